"""attn_prefill_chunk with score options against the fp64 definition.

Tolerance: an output is a mean of |v| < 6 under weights that are rounded to bf16 for the second product
(half a step: 2^-9 .. 2^-8 of each weight, so at most 2^-8 * 6 of the mean, and far less where signs
vary; the normaliser sums the unrounded weights), then rounded to bf16 (2^-8 of the value); the
scores' fp32 error moves weights by 2^-13. So 2^-8 |o| + 2^-8 max|v seen| + 6 * 2^-13; max|v| is
taken as 6. The log-sum-exp: 2^-13 + 2^-23 |lse|, as in the decode.
"""
import numpy as np
import pytest
import torch

import workloads as W
from oracle import as_f64
from oracle import serving as S
from tests.helpers import bits

pytestmark = pytest.mark.gpu

SLOPES = 2.0 ** (-0.5 * np.arange(1, 17))


def dev(a, dtype=torch.int32):
    return torch.tensor(np.asarray(a), dtype=dtype, device="cuda")


def close(out, lse, ref_o, ref_l, rows=None, what=""):
    o, l = as_f64(bits(out)), lse.cpu().numpy().astype(np.float64)
    if rows is not None:
        rows = sorted(rows)
        o, l, ref_o, ref_l = o[rows], l[rows], ref_o[rows], ref_l[rows]
    ok = np.abs(o - ref_o) <= 2.0 ** -8 * np.abs(ref_o) + 6 * (2.0 ** -8 + 2.0 ** -13)
    assert ok.all(), (what, int((~ok).sum()), np.argwhere(~ok)[:4], o[~ok][:4], ref_o[~ok][:4])
    # and in the norm, where the weights' roundings average: each side of a row is off by rounding
    # errors that are independent of one another, uniform within half a step
    n = np.linalg.norm(o - ref_o) / max(np.linalg.norm(ref_o), 1e-30)
    assert n <= 2.0 ** -8, (what, n)
    inf = np.isneginf(ref_l)
    assert np.array_equal(np.isneginf(l), inf), what
    assert not o[inf].any(), what
    d = np.abs(l[~inf] - ref_l[~inf]) - 2.0 ** -23 * np.abs(ref_l[~inf])
    assert d.size == 0 or d.max() <= 2.0 ** -13, (what, d.max())


def unseen(inp, o):
    """NaN into every slot that no row of the call sees."""
    cu = np.concatenate([[0], np.cumsum(inp.host_q_lens)])
    seen = np.zeros((inp.num_pages, 16), bool)
    for b, L in enumerate(inp.host_seq_lens):
        n = int(inp.host_q_lens[b])
        any_row = np.zeros(int(L), bool)
        for r in range(n):
            any_row |= S.visible(int(L) - n + r, int(L), **S._opts(o, b, int(cu[b]) + r))
        for lp in range(-(-int(L) // 16)):
            v = any_row[lp * 16:(lp + 1) * 16]
            seen[inp.host_block_table[b, lp], :len(v)] |= v
    mask = torch.tensor(~seen, device="cuda")
    for p in (inp.k_pools[0], inp.v_pools[0]):
        p[mask] = float("nan")


def call(pa, inp, o, *, status=None, max_ctas=None, q=None, table=None, **kw):
    k = dict(softcap=o.get("softcap", 0.0), window=o.get("window", 0))
    if o.get("slopes") is not None:
        k["alibi_slopes"] = dev(o["slopes"], torch.float32)
    if o.get("prefix") is not None:
        k["prefix_lens"] = dev(o["prefix"])
    if o.get("row_start") is not None:
        k["row_start"] = dev(o["row_start"])
    return pa.attn_prefill_chunk(
        inp.q[0] if q is None else q, inp.cu_q_lens, inp.k_pools[0], inp.v_pools[0],
        inp.block_table if table is None else table, inp.seq_lens, int(inp.host_q_lens.max()),
        int(inp.host_seq_lens.max()), inp.scale, status=status, max_ctas=max_ctas, **k, **kw)


def reference(inp, o, rows=None):
    cu = np.concatenate([[0], np.cumsum(inp.host_q_lens)])
    return S.prefill_scored(bits(inp.q[0]), cu, bits(inp.k_pools[0]), bits(inp.v_pools[0]),
                            inp.host_block_table, inp.host_seq_lens, inp.scale, rows=rows, **o)


def check(pa, inp, o, *, rows=None, poison=True, max_ctas=None, what=""):
    if poison:
        unseen(inp, o)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = call(pa, inp, o, status=status, max_ctas=max_ctas)
    torch.cuda.synchronize()
    assert pa.read_device_status(status) == 0
    close(out, lse, *reference(inp, o, rows), rows=rows, what=what or str(o)[:80])
    return out, lse


OPTIONS = [
    dict(window=1), dict(window=16), dict(window=100), dict(softcap=30.0), dict(softcap=0.5),
    dict(slopes=SLOPES), dict(prefix="p"), dict(window=50, prefix="p"), dict(row_start="r"),
    dict(row_start="r", prefix="p", slopes=SLOPES),
    dict(softcap=20.0, slopes=SLOPES, window=200, prefix="p", row_start="r"),
]


def options(o, q_lens, lens, rng):
    o = dict(o)
    if o.get("prefix") == "p":
        o["prefix"] = np.array([rng.integers(0, l + 1) for l in lens])
        o["prefix"][1::3] = 0
    if o.get("row_start") == "r":
        starts = []
        for n, l in zip(q_lens, lens):
            cuts = np.sort(np.concatenate([[0], rng.integers(0, l, 4)]))
            pos = np.arange(l - n, l)
            s = cuts[np.searchsorted(cuts, pos, side="right") - 1]
            s = np.where(rng.random(n) < 0.1, pos + 1, s)        # rows with no key of their own
            starts.append(np.where(rng.random(n) < 0.1, rng.integers(-5, l + 5, n), s))
        o["row_start"] = np.concatenate(starts)
    return o


SHAPES = [([1], [0]), ([17], [100]), ([129], [0]), ([7, 128, 1, 70], [0, 333, 600, 16]),
          ([300], [37])]


@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("k", range(len(OPTIONS)))
def test_options(cuda_lib, k, shape):
    q_lens, offs = (np.array(a) for a in SHAPES[shape])
    rng = np.random.default_rng(10 * k + shape)
    o = options(OPTIONS[k], q_lens, offs + q_lens, rng)
    inp = W.make_paged(300 + shape, offs + q_lens, q_lens, device="cuda", q_scale=3.0)
    check(cuda_lib, inp, o)


@pytest.mark.parametrize("k", [0, 2, 5, 7, 10])
@pytest.mark.parametrize("max_ctas", [1, 3, 40])
def test_jobs_cut_between_ctas(cuda_lib, k, max_ctas):
    """Few CTAs run many pieces each; an odd number of CTAs cuts jobs into partial results."""
    q_lens, offs = np.array([260, 40]), np.array([1500, 0])
    rng = np.random.default_rng(k)
    o = options(OPTIONS[k], q_lens, offs + q_lens, rng)
    inp = W.make_paged(40, offs + q_lens, q_lens, device="cuda", q_scale=2.0)
    check(cuda_lib, inp, o, max_ctas=max_ctas)


def sample(rng, n, count):
    return set(int(x) for x in rng.integers(0, n, count)) | {0, n - 1}


@pytest.mark.parametrize("n,off,o", [
    (2048, 20_000, dict(window=4096, prefix=[375])),
    (1500, 30_001, dict(softcap=30.0)),
    (1100, 9000, dict(slopes=SLOPES)),
    (2000, 7000, dict(row_start="far", prefix=[50], slopes=SLOPES)),
    (4096, 4000, dict(window=128)),
])
def test_long_chunks_sampled(cuda_lib, n, off, o):
    rng = np.random.default_rng(n)
    o = dict(o)
    if o.get("row_start") == "far":   # every other row sees the far prefix alone
        pos = np.arange(off, off + n)
        o["row_start"] = np.where(pos % 2, pos + 1, pos - pos % 500)
    inp = W.make_paged(50, [off + n], [n], device="cuda", q_scale=4.0)
    check(cuda_lib, inp, o, rows=sample(rng, n, 40), poison=False)


def test_head_partition(cuda_lib):
    inp = W.make_paged(3, [700, 333], [150, 30], device="cuda", q_scale=2.0)
    for hkv in (1, 2, 4):
        q = inp.q[0][:, :2 * hkv].contiguous()
        kp, vp = (p[:, :, :hkv].contiguous() for p in (inp.k_pools[0], inp.v_pools[0]))
        o = dict(softcap=15.0, slopes=SLOPES[:2 * hkv], window=200, prefix=[60, 0])
        out, lse = cuda_lib.attn_prefill_chunk(
            q, inp.cu_q_lens, kp, vp, inp.block_table, inp.seq_lens, 150, 700, inp.scale,
            dims=(2 * hkv, hkv, 128, 16), softcap=15.0, window=200,
            alibi_slopes=dev(o["slopes"], torch.float32), prefix_lens=dev(o["prefix"]))
        ref = S.prefill_scored(bits(q), [0, 150, 180], bits(kp), bits(vp), inp.host_block_table,
                               inp.host_seq_lens, inp.scale, **o)
        close(out, lse, *ref, what=f"{hkv} KV heads")


def test_no_option_that_excludes_a_key_equals_the_plain_call(cuda_lib):
    inp = W.make_paged(61, [3000, 500], [700, 40], device="cuda")
    a, la = cuda_lib.attn_prefill_chunk(inp.q[0], inp.cu_q_lens, inp.k_pools[0], inp.v_pools[0],
                                        inp.block_table, inp.seq_lens, 700, 3000, inp.scale)
    b, lb = call(cuda_lib, inp, dict(window=3000))
    torch.cuda.synchronize()
    assert (a.float() - b.float()).norm() <= 2.0 ** -8 * a.float().norm()
    assert torch.allclose(la, lb, atol=2.0 ** -13)


def test_a_non_finite_value_reaches_only_the_rows_that_see_it(cuda_lib):
    """V rows of NaN / inf inside the chunk: rows before them, and rows of other documents in the same
    tile, keep their values (recomputed with unrounded weights, so within the tolerance above of the
    definition on their visible keys, not bit for bit)."""
    n, off = 200, 130
    pos = np.arange(off, off + n)
    start = np.where(pos < off + 100, 0, off + 100)               # two documents
    inp = W.make_paged(62, [off + n], [n], device="cuda", q_scale=2.0)
    bt = inp.host_block_table
    at = lambda p: (int(bt[0, p // 16]), p % 16)
    inp.v_pools[0][at(off + 60)] = float("nan")                   # seen by rows 60 .. 99
    inp.v_pools[0][at(off + 150)][3] = float("inf")               # head 3: rows 150 .. 199
    inp.k_pools[0][at(off + 170)] = float("nan")                  # rows 170 .. 199
    same = list(range(60)) + list(range(100, 150))
    ref_o, ref_l = reference(inp, dict(row_start=start), rows=set(same) | set(range(150, 170)))
    heads = [h for h in range(16) if h // 2 != 3]
    for cap in (None, 1, 3):
        out, lse = call(cuda_lib, inp, dict(row_start=start), max_ctas=cap)
        torch.cuda.synchronize()
        close(out, lse, ref_o, ref_l, rows=same, what=str(cap))
        assert bool(out[60:100].isnan().all())
        close(out[:, heads].contiguous(), lse[:, heads], ref_o[:, heads], ref_l[:, heads],
              rows=range(150, 170), what=str(cap))
        assert not bool(out[150:170, 6:8].isfinite().any())
        assert bool(out[170:].isnan().all()) and bool(lse[170:].isnan().all())
        assert bool(lse[:170].isfinite().all())


def test_pages_left_behind_by_the_window_may_be_gone(cuda_lib):
    n, off = 40, 700
    inp = W.make_paged(63, [off + n], [n], device="cuda")
    o = dict(window=64, prefix=[20])
    want = call(cuda_lib, inp, o)
    t = inp.block_table.clone()
    first = (off - 63) // 16
    t[0, 2:first] = -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = call(cuda_lib, inp, o, table=t, status=status)
    assert cuda_lib.read_device_status(status) == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    t[0, first] = -1                                              # one that is seen
    call(cuda_lib, inp, o, table=t, status=status)
    assert cuda_lib.read_device_status(status) == cuda_lib.DEV_ERR_PAGE_OOB


def test_chunks_that_do_not_fit_are_flagged_and_left_alone(cuda_lib):
    inp = W.make_paged(64, [50, 60, 70], [20, 30, 10], device="cuda")
    out = torch.full((60, 16, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((60, 16), 9.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    inp.seq_lens[1] = 29                                          # fewer keys than the chunk
    call(cuda_lib, inp, dict(window=8), status=status, out=out, lse=lse)
    assert cuda_lib.read_device_status(status) == cuda_lib.DEV_ERR_LENGTH
    assert bool((out[20:50] == 9.0).all()) and bool((lse[20:50] == 9.0).all())
    inp.seq_lens[1] = 60
    want = call(cuda_lib, inp, dict(window=8))
    assert torch.equal(out[:20], want[0][:20]) and torch.equal(out[50:], want[0][50:])
    out.fill_(9.0)
    inp.cu_q_lens[3] = 75                                         # past the packed rows
    call(cuda_lib, inp, dict(window=8), status=status, out=out)
    assert cuda_lib.read_device_status(status) == cuda_lib.DEV_ERR_LENGTH
    assert torch.equal(out[:50], want[0][:50]) and bool((out[50:] == 9.0).all())


def test_a_prefix_longer_than_what_is_cached_is_seen_as_far_as_it_goes(cuda_lib):
    """A prompt of 300 tokens in chunks of 128: every chunk sees what has been appended."""
    inp = W.make_paged(65, [128], [128], device="cuda", q_scale=2.0)
    out, lse = call(cuda_lib, inp, dict(prefix=[300]), max_prefix_len=300)
    ref = reference(inp, dict(prefix=[128]))
    close(out, lse, *ref)


def test_replayed_from_a_graph_with_new_masks(cuda_lib):
    q_lens, lens = np.array([100, 60]), np.array([900, 60])
    inp = W.make_paged(66, lens, q_lens, device="cuda", q_scale=2.0)
    prefix, start = dev([0, 0]), dev(np.zeros(160))
    slopes = dev(SLOPES, torch.float32)
    out, lse = torch.empty_like(inp.q[0]), torch.empty(160, 16, device="cuda")
    ws = torch.empty(cuda_lib.prefill_score_workspace_size(2, 160), dtype=torch.uint8, device="cuda")

    def go():
        cuda_lib.attn_prefill_chunk(inp.q[0], inp.cu_q_lens, inp.k_pools[0], inp.v_pools[0],
                                    inp.block_table, inp.seq_lens, 100, 900, inp.scale, out=out,
                                    lse=lse, workspace=ws, softcap=25.0, alibi_slopes=slopes,
                                    prefix_lens=prefix, row_start=start)
    go()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go()
    rng = np.random.default_rng(1)
    for _ in range(3):
        o = options(OPTIONS[10], q_lens, lens, rng)
        o.update(softcap=25.0, window=0)
        prefix.copy_(dev(o["prefix"]))
        start.copy_(dev(o["row_start"]))
        g.replay()
        torch.cuda.synchronize()
        close(out, lse, *reference(inp, o))


@pytest.mark.parametrize("cap", [8.0, 50.0, 300.0])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_large_capped_scores_of_one_sign(cuda_lib, cap, sign):
    """Scores near +-60 (all of one sign): the exponents' reference is the largest magnitude's score
    while that stays near the max, else the max itself."""
    n, off = 70, 180
    inp = W.make_paged(67, [off + n], [n], device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    u = torch.randn(16, 128, generator=g, device="cuda")
    k = u[::2] + 0.2 * torch.randn(inp.num_pages, 16, 8, 128, generator=g, device="cuda")
    inp.k_pools[0] = k.to(torch.bfloat16)
    q = sign * 5.0 * u[::2].repeat_interleave(2, 0) * (0.5 + torch.rand(n, 16, 1, generator=g, device="cuda"))
    inp.q[0] = q.to(torch.bfloat16)
    check(cuda_lib, inp, dict(softcap=cap))
    check(cuda_lib, inp, dict(softcap=cap, slopes=SLOPES, window=150), poison=False)


@pytest.mark.parametrize("o", [dict(), dict(softcap=12.0), dict(slopes=SLOPES)])
def test_rows_that_see_no_key_of_a_tile(cuda_lib, o):
    """Rows that see nothing, or only tiles before or after the one at hand, beside rows that see it:
    also where the keys they do not see are NaN (their own document's are not)."""
    n, off = 256, 384
    pos = np.arange(off, off + n)
    start = np.where(pos % 7 == 3, pos + 1, np.where(pos % 2, off + 128 * ((pos - off) // 128), 0))
    o = dict(o, row_start=start)
    inp = W.make_paged(68, [off + n], [n], device="cuda", q_scale=2.0)
    check(cuda_lib, inp, o, poison=False)
    # NaN keys and values at positions 100 .. 105: rows of the documents that start later are unmoved
    bt = inp.host_block_table
    clean = call(cuda_lib, inp, o)
    for p in range(100, 106):
        inp.k_pools[0][int(bt[0, p // 16]), p % 16] = float("nan")
        inp.v_pools[0][int(bt[0, p // 16]), p % 16] = float("nan")
    later = [r for r in range(n) if start[r] > 105]
    ref_o, ref_l = reference(inp, o, rows=set(later))
    for cap in (None, 1, 5):
        out, lse = call(cuda_lib, inp, o, max_ctas=cap)
        torch.cuda.synchronize()
        close(out, lse, ref_o, ref_l, rows=later, what=str(cap))
        assert torch.equal(lse[later], clean[1][later]) or cap is not None
        first = [r for r in range(n) if start[r] == 0]
        assert bool(out[first].isnan().all())


@pytest.mark.parametrize("o,scale", [
    (dict(softcap=1e4), None), (dict(softcap=1e20), None), (dict(softcap=1e-4), None),
    (dict(softcap=200.0, slopes=SLOPES), None), (dict(softcap=30.0), 1e-4), (dict(softcap=30.0), 3.0),
    (dict(slopes=-0.1 * SLOPES, window=100), None), (dict(slopes=-0.3 * SLOPES, softcap=20.0), None),
    (dict(slopes=np.where(np.arange(16) % 2, 9.0, 0.0)), None),
])
def test_caps_scales_and_slopes_far_from_the_usual(cuda_lib, o, scale):
    """A cap far above the scores is no cap (not a loss of their low bits), one far below makes all
    weights equal; scores of every size, slopes of either sign and steep ones."""
    q_lens, offs = np.array([140, 33]), np.array([200, 0])
    inp = W.make_paged(69, offs + q_lens, q_lens, device="cuda", q_scale=2.0)
    if scale is not None:
        inp.scale = scale
    check(cuda_lib, inp, o)
    d = W.make_paged(70, [400, 33], [1, 1], device="cuda", q_scale=2.0)
    if scale is not None:
        d.scale = scale
    for split in (0, 32):
        out, lse = cuda_lib.attn_decode_paged(
            d.q[0], d.k_pools[0], d.v_pools[0], d.block_table, d.seq_lens, 400, d.scale,
            split_tokens=split, softcap=o.get("softcap", 0.0), window=o.get("window", 0),
            alibi_slopes=None if o.get("slopes") is None else dev(o["slopes"], torch.float32))
        close(out, lse, *S.decode_scored(bits(d.q[0]), bits(d.k_pools[0]), bits(d.v_pools[0]),
                                         d.host_block_table, d.host_seq_lens, d.scale, **o))


@pytest.mark.parametrize("off", [0, 3000])
def test_chunks_longer_than_the_bound_are_flagged_and_left_alone(cuda_lib, off):
    q_lens, lens = np.array([40, 300, 20]), np.array([40, 300, 20]) + off
    inp = W.make_paged(69, lens, q_lens, device="cuda")
    want = call(cuda_lib, inp, dict(window=500))
    out = torch.full((360, 16, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cuda_lib.attn_prefill_chunk(inp.q[0], inp.cu_q_lens, inp.k_pools[0], inp.v_pools[0], inp.block_table,
                                inp.seq_lens, 299, int(lens.max()), inp.scale, out=out, status=status,
                                window=500)
    assert cuda_lib.read_device_status(status) == cuda_lib.DEV_ERR_LENGTH
    assert bool((out[40:340] == 9.0).all())
    # (the split of the work differs, and with it the order of a row's sums: 2^-8 of a value in bf16,
    # and the weights' roundings, as above)
    for r in (slice(0, 40), slice(340, 360)):
        a, b = out[r].double(), want[0][r].double()
        assert bool(((a - b).abs() <= 2.0 ** -7 * b.abs() + 6 * (2.0 ** -7 + 2.0 ** -12)).all())


@pytest.mark.parametrize("off", [0, 3000])
@pytest.mark.parametrize("slope", [float("inf"), float("-inf"), float("nan")])
def test_rows_without_keys_under_any_slope(cuda_lib, off, slope):
    n = 150
    inp = W.make_paged(70, [off + n], [n], device="cuda")
    start = np.zeros(n, int)
    start[::3] = off + n                                          # rows that see nothing
    slopes = SLOPES.copy()
    slopes[5] = slope
    for cap in (0.0, 20.0):
        out, lse = call(cuda_lib, inp, dict(slopes=slopes, row_start=start, softcap=cap), max_ctas=7)
        assert bool((lse[::3] == float("-inf")).all()) and not bool(out[::3].any())
        keep = [h for h in range(16) if h != 5]
        assert bool(lse[1::3][:, keep].isfinite().all()) and bool(out[1::3][:, keep].isfinite().all())


@pytest.mark.parametrize("cap", [1e-4, 30.0, 200.0, 1e5])
@pytest.mark.parametrize("bias", [False, True])
def test_products_that_are_all_zero(cuda_lib, cap, bias):
    """Zero q rows and zeroed keys, a warp's worth and a tile's and more of each: every score of such a
    row is 0 before the bias, also under caps that the folded polynomial does not serve."""
    o = dict(softcap=cap, **(dict(slopes=SLOPES) if bias else {}))
    for seed in range(3):
        inp = W.make_paged(520 + seed, [530], [260], device="cuda", q_scale=3.0)
        inp.q[0][32:96] = 0
        inp.q[0][200:260, 5:] = 0
        for p in range(0, 272):
            inp.k_pools[0][int(inp.host_block_table[0, p // 16]), p % 16] = 0
        check(cuda_lib, inp, o)
