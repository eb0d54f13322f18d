"""beam_select against the fp64 definition.

Places are compared exactly, except where two candidates' 64-bit scores lie within the kernel's error
of each other: its normaliser is an fp32 sum of exponentials (each off by 2^-22 of itself for the
exponential and, at most 100 below the maximum here, 2^-24 * 1.45 * 40 for its argument, 2^-18 in
all terms that matter at once would be the worst; the logits here put it below 2^-19). So a place may
hold another candidate only if that one's score is within 2^-18 of the place's; scores then differ by
that and the rounding to fp32, 2^-24 of the score.
"""
import numpy as np
import pytest
import torch

from oracle import beam as O

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def logits_of(N, W, V, dtype, seed, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(N, W, V, generator=g) * spread
    x.view(-1)[torch.randint(0, N * W * V, (max(1, N * W * 3),), generator=g)] += 9.0
    return x.to(dtype).cuda()


def scores_of(N, W, seed):
    g = torch.Generator().manual_seed(seed + 1)
    return (-torch.rand(N, W, generator=g) * 6).cuda()


def check(pa, logits, scores, k, live=None, eos=-1, **kw):
    got = pa.beam_select(logits, scores, k, live=live, eos_token=eos, **kw)
    torch.cuda.synchronize()
    host = logits.float().cpu().numpy()
    lv = None if live is None else live.cpu().numpy()
    (s, p, t, a), every = O.select(host, scores.cpu().numpy(), k, lv, eos)
    gs, gp, gt, ga = (x.cpu().numpy() for x in got)
    tol = 2.0 ** -18
    for n in range(len(gs)):
        known = {(b, v): x for x, b, v in every[n]}
        seen = set()
        for i in range(k):
            if np.isneginf(s[n, i]):
                assert (gs[n, i], gp[n, i], gt[n, i], ga[n, i]) == (-INF, -1, -1, 0), (n, i)
                continue
            place = (int(gp[n, i]), int(gt[n, i]))
            assert place in known and place not in seen, (n, i, place)
            seen.add(place)
            if place != (p[n, i], t[n, i]):
                assert abs(known[place] - s[n, i]) <= tol, (n, i, place, known[place], s[n, i])
                assert place[0] != p[n, i], "the order within a beam is exact"
            assert abs(gs[n, i] - s[n, i]) <= tol + 2.0 ** -24 * abs(s[n, i]), (n, i, gs[n, i], s[n, i])
            ended = lv is not None and lv[n, place[0]] == 0
            assert ga[n, i] == (0 if ended or place[1] == eos else 1)
    return got


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,W,V,k", [(1, 1, 1, 1), (1, 1, 7, 7), (2, 3, 5, 15), (1, 4, 33, 64), (3, 2, 1000, 8),
                                     (2, 5, 4099, 10), (1, 4, 51865, 4), (5, 1, 9001, 3), (1, 64, 77, 64)])
def test_matches_the_definition(cuda_lib, dtype, N, W, V, k):
    check(cuda_lib, logits_of(N, W, V, dtype, N + V), scores_of(N, W, V), k)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_beams_that_ended_or_are_not_in_use(cuda_lib, dtype):
    x, s = logits_of(4, 4, 300, dtype, 3), scores_of(4, 4, 3)
    live = torch.tensor([[1, 1, 1, 1], [0, 1, 0, 1], [0, 0, 0, 0], [1, 0, 1, 1]], dtype=torch.int32).cuda()
    s[0, 1:] = -INF            # the first step
    s[3, 1] = -INF             # ended and not in use: no candidate
    s[3, 2], s[3, 3] = NAN, INF
    x[3, 2:] = NAN             # (nor read)
    x[1, 0] = NAN              # an ended beam's logits are not read
    got = check(cuda_lib, x, s, 6, live, eos=11)
    assert (got.parents[0] == 0).all() and got.parents[2].tolist()[4:] == [-1, -1]
    assert (got.live[2] == 0).all()
    check(cuda_lib, x, s, 6, live, eos=-1)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_without_a_distribution(cuda_lib, dtype):
    x, s = logits_of(3, 3, 700, dtype, 5), scores_of(3, 3, 5)
    x[0, 0] = -INF             # nothing allowed
    x[0, 1, 44] = NAN
    x[0, 2, 699] = INF
    x[1, 1] = -INF
    x[1, 1, 613] = 2.0         # one token allowed
    x[2, :, 5:] = torch.finfo(dtype).min
    got = check(cuda_lib, x, s, 9)
    assert (got.parents[0] == -1).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [50, 6000])
def test_equal_scores_in_the_order_of_beam_and_token(cuda_lib, dtype, V):
    x = torch.zeros(2, 3, V, dtype=dtype, device="cuda")
    x[1, :, ::7] = -0.0
    s = torch.full((2, 3), -2.0, device="cuda")
    got = cuda_lib.beam_select(x, s, 40)
    assert (got.parents == 0).all() and got.tokens.tolist() == [list(range(40))] * 2
    x[:, :, V - 1] = 1.0       # the same best token in three beams alike
    got = cuda_lib.beam_select(x, s, 4)
    assert got.parents.tolist() == [[0, 1, 2, 0]] * 2 and got.tokens.tolist() == [[V - 1] * 3 + [0]] * 2


@pytest.mark.parametrize("V", [2000, 70000])
def test_the_best_in_one_place(cuda_lib, V):
    """All of a beam's best side by side, at the start, the end, or a stride apart."""
    base = torch.linspace(-1, 0, V).expand(1, 4, V).clone()
    base[0, 1, :100] += 5
    base[0, 2, -100:] += 5
    base[0, 3, 64::2048 if V > 2048 * 8 else 8][:60] += 7
    for dtype in (torch.float32, torch.bfloat16):
        check(cuda_lib, base.to(dtype).cuda(), torch.zeros(1, 4, device="cuda"), 64)


def test_strides_offsets_and_large_values(cuda_lib):
    wide = logits_of(2, 3, 1234, torch.bfloat16, 9)
    for cut in (slice(0, 1001), slice(1, 1001), slice(3, 700), slice(8, 1233)):
        check(cuda_lib, wide[..., cut], scores_of(2, 3, 1), 5)
    f = logits_of(1, 2, 4001, torch.float32, 9) * 20
    check(cuda_lib, f[:, :, 1:], scores_of(1, 2, 1) - 300, 5)
    first = wide[:, 0]
    check(cuda_lib, first.unsqueeze(1), scores_of(2, 1, 1), 5)   # rows three apart
    with pytest.raises(ValueError):
        cuda_lib.beam_select(wide[..., ::2], scores_of(2, 3, 1), 5)
    with pytest.raises(ValueError):
        cuda_lib.beam_select(wide[:, :2], scores_of(2, 2, 1), 5)  # not equally far apart


def test_in_place_on_a_stream_in_a_graph_and_with_a_workspace(cuda_lib):
    pa = cuda_lib
    x, s = logits_of(3, 4, 5000, torch.bfloat16, 21), scores_of(3, 4, 21)
    live = torch.ones(3, 4, dtype=torch.int32, device="cuda")
    want = pa.beam_select(x, s, 4, live=live, eos_token=9)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = pa.beam_select(x, s, 4, live=live, eos_token=9, stream=st)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    ws = torch.empty(pa.beam_workspace_size(3, 4, 5000, 4), dtype=torch.uint8, device="cuda")
    s0, l0 = s.clone(), live.clone()
    p, t = torch.zeros(3, 4, dtype=torch.int32, device="cuda"), torch.zeros(3, 4, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.beam_select(x, s, 4, live=live, eos_token=9, out_scores=s, live_out=live, parents=p, tokens=t, workspace=ws)
    for _ in range(3):
        s.copy_(s0)
        live.copy_(l0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(s, want.scores) and torch.equal(live, want.live)
        assert torch.equal(p, want.parents) and torch.equal(t, want.tokens)


def test_no_requests(cuda_lib):
    got = cuda_lib.beam_select(torch.empty(0, 4, 100, device="cuda"), torch.empty(0, 4, device="cuda"), 4)
    assert got.scores.shape == (0, 4)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [511, 512, 513, 1023, 1024, 1025, 1032, 2049])
def test_lengths_about_whole_units_at_every_offset(cuda_lib, dtype, V):
    """Units of 512 or 1,024 logits, rows that start anywhere in 16 bytes, the best at both ends."""
    wide = logits_of(1, 2, V + 8, dtype, V)
    for cut in range(8):
        x = wide[:, :, cut:cut + V].clone() if cut == 0 else wide[:, :, cut:cut + V]
        x[0, 0, 0], x[0, 0, V - 1], x[0, 1, V // 2] = 14.0, 15.0, 14.5
        check(cuda_lib, x, scores_of(1, 2, cut), 12)


def test_more_units_alike_than_are_ranked_at_once(cuda_lib):
    """The first step of a constrained search: three tokens allowed, the others at the type's lowest value."""
    x = torch.full((1, 4, 300001), torch.finfo(torch.float32).min, device="cuda")
    x[0, 0, [5, 170000, 300000]] = torch.tensor([1.0, 2.0, 3.0], device="cuda")
    s = torch.tensor([[0.0, -INF, -INF, -INF]], device="cuda")
    got = check(cuda_lib, x, s, 20)
    assert got.tokens[0].tolist() == [300000, 170000, 5] + [i for i in range(18) if i != 5]


def test_a_few_units_with_all_of_the_best(cuda_lib):
    """More candidates than are ranked at once reach the worst of the k best units' largest."""
    x = torch.full((2, 2, 40000), -4.0)
    for u in range(8):
        x[0, 0, 1024 * u: 1024 * u + 500] = torch.arange(500) / 500.0 + u % 3
    x[1] = torch.randn(2, 40000, generator=torch.Generator().manual_seed(1))
    check(cuda_lib, x.cuda(), torch.zeros(2, 2, device="cuda"), 8)
    check(cuda_lib, x.to(torch.bfloat16).cuda(), torch.zeros(2, 2, device="cuda"), 64)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_one_beam_far_ahead_with_few_units(cuda_lib, dtype):
    x, s = logits_of(3, 8, 9000, dtype, 31), scores_of(3, 8, 31)
    s[:, 3] += 40
    check(cuda_lib, x, s, 32)
    live = torch.ones(3, 8, dtype=torch.int32, device="cuda")
    live[1, 3] = live[2, 0] = 0
    check(cuda_lib, x, s, 32, live, eos=3)


@pytest.mark.parametrize("W,V", [(16, 2080), (3, 9000), (5, 1030), (2, 66)])
def test_last_units_of_a_few_logits(cuda_lib, W, V):
    for dtype in (torch.bfloat16, torch.float32):
        check(cuda_lib, logits_of(2, W, V, dtype, V), scores_of(2, W, V), 31)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_nan_before_anything_else_that_a_thread_reads(cuda_lib, dtype):
    wide = logits_of(2, 2, 9000, dtype, 8)
    for cut, V, where in [(3, 28, 0), (1, 7, 6), (0, 4, 3), (0, 8000, slice(0, 8)), (5, 8000, slice(3, 40)), (6, 30, 29)]:
        x = wide.clone()[:, :, cut:cut + V]
        x[0, 1, where] = NAN
        got = check(cuda_lib, x, scores_of(2, 2, 8), 4)
        assert (got.parents[0] <= 0).all()
