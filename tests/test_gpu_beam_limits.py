"""The largest calls that the beam-search operators take: rows, groups, beams, keys, vocabularies, far pages."""
import math

import numpy as np
import pytest
import torch

from oracle import beam as O
from tests.test_gpu_fork import check as check_fork
from tests.test_gpu_fork import grown
from tests.test_gpu_shared_decode import Inputs

pytestmark = pytest.mark.gpu
INF = float("inf")


def room(gib):
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"needs {gib} GB")


@pytest.mark.parametrize("groups,rows", [(4096, 1), (64, 64), (1, 4096), (455, 9), (0, 0)])
def test_shared_decode_of_4096_rows(cuda_lib, groups, rows):
    alone = 4096 - groups * rows
    x = Inputs([(1, [16 + (g + 3 * i) % 9 for i in range(rows)]) for g in range(groups)], [i % 7 for i in range(alone)],
               hkv=1, seed=groups)
    assert len(x.lens) == 4096
    out, lse = x.check(cuda_lib)
    again = x.call(cuda_lib, max_group_rows=None)
    assert x.flags == 0 and torch.equal(out, again[0]) and torch.equal(lse, again[1])


def test_shared_decode_of_131072_keys(cuda_lib):
    """The longest sequence, with all of it shared, with most of it, and with none."""
    x = Inputs([(8192, [131072, 131072]), (8000, [128500])], [131071], hkv=1, seed=1, extra=0)
    x.check(cuda_lib)


def test_fork_of_4096_rows(cuda_lib):
    check_fork(cuda_lib, *grown(64, 64, 12, 5))
    check_fork(cuda_lib, *grown(4096, 1, 7, 6), inplace=True)


def test_copies_of_pages_past_4_gib(cuda_lib):
    room(20)
    n = 140_000
    pools = [torch.zeros(n, 16, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    g = torch.Generator(device="cuda").manual_seed(1)
    for p in pools:
        p[n - 8:] = torch.randn(8, 16, 8, 128, generator=g, device="cuda").to(torch.bfloat16)
    copies = [(n - 8, n - 1, 5), (-1, -1, 0), (n - 7, 0, 16), (3, n - 2, 1)]
    tail = [p[n - 8:].clone() for p in pools]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cuda_lib.paged_copy_pages(torch.tensor(copies, dtype=torch.int32, device="cuda"), pools, status=status)
    torch.cuda.synchronize()
    assert cuda_lib.read_device_status(status) == 0
    for p, t in zip(pools, tail):
        want = t.clone()
        want[7, :5] = t[0, :5]
        want[6, :1] = 0
        assert torch.equal(p[n - 8:], want) and torch.equal(p[0], t[1]) and not p[1:n - 8].any()


@pytest.mark.parametrize("N,W,V,k", [(65535, 1, 7, 1), (1023, 64, 33, 64), (16383, 4, 300, 4)])
def test_selection_of_65535_rows(cuda_lib, N, W, V, k):
    g = torch.Generator(device="cuda").manual_seed(N)
    x = torch.randn(N, W, V, generator=g, device="cuda") * 3
    s = -6 * torch.rand(N, W, generator=g, device="cuda")
    got = cuda_lib.beam_select(x, s, k)
    torch.cuda.synchronize()
    exact = (s.double().unsqueeze(2) + torch.log_softmax(x.double(), 2)).view(N, -1)
    want, place = exact.sort(dim=1, descending=True, stable=True)
    want, place = want[:, :k], place[:, :k]
    mine = got.parents.long() * V + got.tokens.long()
    at = exact.gather(1, mine)
    assert ((at - want).abs()[mine != place] <= 2.0 ** -17).all()
    assert ((got.scores.double() - at).abs() <= 2.0 ** -18 + 2.0 ** -24 * at.abs()).all()
    ordered = mine.sort(dim=1).values
    assert k == 1 or (ordered[:, 1:] != ordered[:, :-1]).all()


@pytest.mark.parametrize("W,V", [(1, 2 ** 31 - 1), (2, 2 ** 30 - 1), (63, 34_087_041)])
def test_selection_over_2_31_candidates(cuda_lib, W, V):
    """Tokens at both ends and in the middle of the largest vocabularies."""
    assert 0 < 2 ** 31 - W * V < 128
    room(16)
    x = torch.full((1, W, V), -9.0, dtype=torch.bfloat16, device="cuda")
    best = [(W - 1, V - 1, 20.0), (0, 0, 19.0), (W // 2, V // 2, 18.5), (W - 1, 1, 18.0), (0, V - 2, 17.5)]
    for b, v, value in best:
        x[0, b, v] = value
    s = torch.zeros(1, W, device="cuda")
    got = cuda_lib.beam_select(x, s, 5)
    torch.cuda.synchronize()
    norm = {}
    for b in range(W):
        values = [val for c, _, val in best if c == b]
        norm[b] = math.log(sum(math.exp(v) for v in values) + (V - len(values)) * math.exp(-9.0))
    want = sorted(((val - norm[b], b, v) for b, v, val in best), reverse=True)
    assert [(p, t) for p, t in zip(got.parents[0].tolist(), got.tokens[0].tolist())] == [(b, v) for _, b, v in want]
    assert all(abs(a - w) <= 2.0 ** -17 + 2.0 ** -24 * abs(w) for a, (w, _, _) in zip(got.scores[0].tolist(), want))


def test_selection_of_rows_past_2_31_elements_apart(cuda_lib):
    room(16)
    apart, V = 1_600_000_001, 5000
    store = torch.empty(3 * apart, dtype=torch.bfloat16, device="cuda")
    x = store.as_strided((3, 1, V), (apart, apart, 1))
    rows = torch.randn(3, 1, V, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    x.copy_(rows)
    s = torch.tensor([[0.0], [-1.0], [-INF]])
    got = cuda_lib.beam_select(x, s.cuda(), 7)
    want = cuda_lib.beam_select(rows.cuda(), s.cuda(), 7)
    torch.cuda.synchronize()
    (ws, wp, wt, _), _ = O.select(rows.float().numpy(), s.numpy(), 7)
    assert np.array_equal(got.tokens.cpu().numpy(), wt) and np.array_equal(got.parents.cpu().numpy(), wp)
    assert torch.equal(got.tokens, want.tokens) and torch.equal(got.parents, want.parents)
    gs = got.scores.cpu().numpy()
    assert np.array_equal(np.isneginf(gs), np.isneginf(ws))
    live = np.isfinite(ws)
    assert (np.abs(gs[live] - ws[live]) <= 2.0 ** -18 + 2.0 ** -24 * np.abs(ws[live])).all()
