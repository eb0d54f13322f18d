"""The beam-search calls through the binding's two paths: the compiled one gives the same bits as the Python
one, on another stream and captured too, and leaves what is not plainly right to the Python checks."""
import pytest
import torch

from tests.test_gpu_fast_path import Counting, same, slow

pytestmark = pytest.mark.gpu
DIMS = (4, 2, 128, 16)


class Calls:
    """The four calls over small inputs, each returning the tensors that it wrote."""

    def __init__(self, pa):
        g = torch.Generator().manual_seed(3)
        bf = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
        self.pa = pa
        self.k, self.v, self.q = bf(40, 16, 2, 128), bf(40, 16, 2, 128), bf(5, 4, 128)
        self.table = i32([[0, 1, 2, 3], [0, 1, 4, 5], [0, 1, 6, 0], [7, 8, 9, 10], [11, 0, 0, 0]])
        self.lens, self.cu, self.shared = i32([60, 64, 33, 50, 3]), i32([0, 3]), i32([2])
        self.logits, self.scores = bf(2, 3, 500), torch.rand(2, 3, generator=g).cuda()
        self.live = i32([[1, 1, 0], [1, 1, 1]])
        self.parents, self.fork_lens = i32([[1, 1, 0], [2, -1, 2]]), i32([40, 20, 5, 16, 0, 33])
        self.fork_table = i32([[0, 1, 2, -1], [0, 3, -1, -1], [4, -1, -1, -1], [5, -1, -1, -1], [-1] * 4, [6, 7, 8, -1]])
        self.free, self.count = i32(list(range(20, 32))), i32([9])
        self.copies = i32([[1, 30, 5], [-1, -1, 0], [2, 31, 15]])

    def decode_shared(self, **kw):
        a = dict(out=torch.zeros_like(self.q), lse=torch.zeros(5, 4, device="cuda"), dims=DIMS)
        a.update(kw)
        return self.pa.attn_decode_paged_shared(self.q, self.k, self.v, self.table, self.lens, self.cu, self.shared, 64,
                                                0.09, **a)

    def beam(self, **kw):
        e = lambda t: torch.zeros(2, 4, dtype=t, device="cuda")
        a = dict(live=self.live, eos_token=7, out_scores=e(torch.float32), parents=e(torch.int32),
                 tokens=e(torch.int32), live_out=e(torch.int32))
        a.update(kw)
        return tuple(self.pa.beam_select(self.logits, self.scores, 4, **a))

    def fork(self, **kw):
        table, free = self.fork_table.clone(), self.free.clone()
        e = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
        a = dict(seq_lens_out=e(6), copies=e(6, 3), shared_pages=e(2), free_count_out=e(1))
        a.update(kw)
        return table, free, *self.pa.paged_fork(self.parents, self.fork_lens, table, free, self.count, 40, **a)

    def copy_pages(self, **kw):
        pools = kw.pop("pools", None) or [self.k.clone(), self.v.clone(), self.k.clone()]
        self.pa.paged_copy_pages(self.copies, pools, **{"dims": DIMS, **kw})
        return tuple(pools)


CALLS = ["decode_shared", "beam", "fork", "copy_pages"]


@pytest.fixture()
def fast(cuda_lib, monkeypatch):
    assert cuda_lib._FAST is not None, "the fast path was not built"
    f = Counting(cuda_lib._FAST)
    monkeypatch.setattr(cuda_lib, "_FAST", f)
    return f


def took(fast):
    return [(n, bool(r)) for n, r in fast.seen]


@pytest.mark.parametrize("name", CALLS)
def test_same_results_on_any_stream_and_captured(cuda_lib, fast, monkeypatch, name):
    fn = getattr(Calls(cuda_lib), name)
    got = fn()
    assert took(fast) == [(name, True)]
    want = slow(cuda_lib, monkeypatch, fn)
    same(got, want)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        got = fn(stream=st)
    same(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = fn()
    for _ in range(2):
        g.replay()
    same(got, want)
    assert took(fast) == [(name, True)] * 3


@pytest.mark.parametrize("name", ["decode_shared", "beam", "fork"])
def test_new_outputs_and_workspaces(cuda_lib, fast, monkeypatch, name):
    c = Calls(cuda_lib)
    fn = getattr(c, name)
    want = slow(cuda_lib, monkeypatch, fn)
    none = {"decode_shared": ["out", "lse"], "beam": ["out_scores", "parents", "tokens", "live_out"],
            "fork": ["seq_lens_out", "copies", "shared_pages", "free_count_out"]}[name]
    same(fn(**{k: None for k in none}), want)
    size = {"decode_shared": lambda: cuda_lib.decode_shared_workspace_size(5, 1, 5, DIMS),
            "beam": lambda: cuda_lib.beam_workspace_size(2, 3, 500, 4),
            "fork": lambda: cuda_lib.fork_workspace_size(2, 3, 4)}[name]()
    ws = torch.full((max(size, 256),), 255, dtype=torch.uint8, device="cuda")
    same(fn(workspace=ws), want)
    assert took(fast) == [(name, True)] * 2
    with pytest.raises(cuda_lib.PagedAttnError):
        fn(workspace=ws[:0])
    # new outputs on a given stream come from the wrapper
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = fn(**{k: None for k in none}, stream=st)
    st.synchronize()
    same(got, want)


@pytest.mark.parametrize("name", CALLS)
def test_anything_else_is_left_to_the_checks(cuda_lib, fast, name):
    c = Calls(cuda_lib)
    fn = getattr(c, name)
    if name == "copy_pages":
        for bad, error in (([c.k.cpu()], ValueError), ([c.k.float()], TypeError), ([c.k, c.v[:-1]], ValueError),
                           ([c.k[:, :8]], ValueError), (["x"], (TypeError, AttributeError))):
            with pytest.raises(error):
                fn(pools=bad)
            assert took(fast)[-1] == (name, False)
        return
    out, like = {"decode_shared": ("out", c.q), "beam": ("parents", torch.zeros(2, 4, dtype=torch.int32, device="cuda")),
                 "fork": ("seq_lens_out", c.fork_lens)}[name]
    for bad, error in ((like.cpu(), ValueError), (like.double(), TypeError), (like[:-1], ValueError),
                       (like.unsqueeze(0), ValueError), (torch.stack([like, like], -1)[..., 0], ValueError),
                       ("x", TypeError)):
        with pytest.raises(error):
            fn(**{out: bad})
        assert took(fast)[-1] == (name, False)


def test_wrong_inputs_name_themselves(cuda_lib):
    c, pa = Calls(cuda_lib), cuda_lib
    with pytest.raises(TypeError, match="logits"):
        pa.beam_select(c.logits.half(), c.scores, 4)
    with pytest.raises(ValueError, match="scores"):
        pa.beam_select(c.logits, c.scores[:1], 4)
    with pytest.raises(pa.PagedAttnError, match="beam_select"):
        pa.beam_select(c.logits, c.scores, 65)
    with pytest.raises(pa.PagedAttnError):
        pa.beam_select(c.logits, c.scores, 4, out_scores=torch.zeros(2, 4, device="cuda"), eos_token=500)
    with pytest.raises(ValueError, match="seq_lens"):
        pa.paged_fork(c.parents, c.lens, c.fork_table, c.free, c.count, 40)
    with pytest.raises(ValueError, match="block_table"):
        pa.paged_fork(c.parents, c.fork_lens, c.fork_table[:5], c.free, c.count, 40)
    with pytest.raises(pa.PagedAttnError):
        pa.paged_fork(torch.zeros(1, 65, dtype=torch.int32, device="cuda"), torch.zeros(65, dtype=torch.int32, device="cuda"),
                      torch.zeros(65, 4, dtype=torch.int32, device="cuda"), c.free, c.count, 40)
    with pytest.raises(ValueError, match="copies"):
        pa.paged_copy_pages(c.copies[:, :2].contiguous(), [c.k], dims=DIMS)
    with pytest.raises(ValueError, match="cu_group_rows"):
        pa.attn_decode_paged_shared(c.q, c.k, c.v, c.table, c.lens, c.cu[:1], c.shared, 64, 0.1, dims=DIMS)
    for bad in (0.0, -1.0, float("nan")):
        with pytest.raises(pa.PagedAttnError):
            pa.attn_decode_paged_shared(c.q, c.k, c.v, c.table, c.lens, c.cu, c.shared, 64, bad, dims=DIMS)
    with pytest.raises(ValueError, match="v_pool"):
        pa.attn_decode_paged_shared(c.q, c.k, c.v[:-1], c.table, c.lens, c.cu, c.shared, 64, 0.1, dims=DIMS)
