"""New outputs of a beam-search call are tensors of their own: one can be kept, saved or grown without the others."""
import io

import pytest
import torch

from tests.test_gpu_beam_fast_path import Calls, fast, took  # noqa: F401  (fast: a fixture)

pytestmark = pytest.mark.gpu


def made(calls):
    beam = calls.beam(out_scores=None, parents=None, tokens=None, live_out=None)
    fork = calls.fork(seq_lens_out=None, copies=None, shared_pages=None, free_count_out=None)
    return beam, fork[2:]


def test_each_has_memory_of_its_own(cuda_lib, fast):
    both = made(Calls(cuda_lib))
    torch.cuda.synchronize()
    assert took(fast) == [("beam", True), ("fork", True)]
    for outputs in both:
        spans = []
        for t in outputs:
            store = t.untyped_storage()
            assert t.storage_offset() == 0 and t.is_contiguous() and store.resizable()
            assert store.nbytes() == t.numel() * t.element_size()
            spans.append((store.data_ptr(), store.data_ptr() + store.nbytes()))
        spans.sort()
        assert all(a[1] <= b[0] for a, b in zip(spans, spans[1:]))


def test_one_can_grow_and_be_saved_alone(cuda_lib, fast):
    for outputs in made(Calls(cuda_lib)):
        torch.cuda.synchronize()
        for i, t in enumerate(outputs):
            others = [o.clone() for j, o in enumerate(outputs) if j != i]
            one = t.clone()
            file = io.BytesIO()
            torch.save(t, file)
            assert file.tell() < 4096 + t.numel() * t.element_size()
            t.resize_(4096).fill_(77)
            assert all(torch.equal(a, b) for a, b in zip(others, [o for j, o in enumerate(outputs) if j != i]))
            t.resize_(one.shape).copy_(one)


def test_without_a_request(cuda_lib):
    """Outputs without elements."""
    pa = cuda_lib
    got = pa.beam_select(torch.empty(0, 3, 50, device="cuda"), torch.empty(0, 3, device="cuda"), 4)
    assert [tuple(t.shape) for t in got] == [(0, 4)] * 4
    e = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    fork = pa.paged_fork(e(0, 4), e(0), e(0, 5), e(9), e(1) + 3, 40)
    torch.cuda.synchronize()
    assert fork.free_count.item() == 3 and tuple(fork.copies.shape) == (0, 3)


def test_memory_in_use_on_another_stream_is_not_handed_out(cuda_lib):
    """record_stream holds an output's memory until that stream's work is done."""
    calls = Calls(cuda_lib)
    side = torch.cuda.Stream()
    got = calls.beam(out_scores=None, parents=None, tokens=None, live_out=None)
    want = [t.clone() for t in got]
    torch.cuda.synchronize()
    at = {t.data_ptr() for t in got}
    with torch.cuda.stream(side):
        torch.cuda._sleep(2_000_000)
        kept = [t.clone() for t in got]
        for t in got:
            t.record_stream(side)
    del got, t
    again = [torch.full((2, 4), -5, dtype=torch.int32, device="cuda") for _ in range(8)]
    assert not at & {t.data_ptr() for t in again}
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(kept, want))
