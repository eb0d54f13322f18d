"""attn_prefill_chunk with score options on K and V that hold NaN and infinities: who sees such a value
gets it, who does not is unmoved, over caches of every length and at a bounded cost.

Tolerance of the finite values: that of test_gpu_score_prefill.close (2^-8 |o| + 6 (2^-8 + 2^-13), and
2^-13 + 2^-23 |lse|). Rows that are computed again do not round their weights, which only takes an error
away. Scores are small here (q_scale 1, a bias of at most 2^-8 a key over at most 2,000 keys), so that no
weight of a key that holds an infinity underflows in fp32, but where a test says so.
"""
import numpy as np
import pytest
import torch

import workloads as W
from oracle import as_f64
from tests.helpers import bits
from tests.test_gpu_score_prefill import call, reference

pytestmark = pytest.mark.gpu

FLAT = 2.0 ** (-8 - 0.25 * np.arange(16))


def same(out, lse, ref_o, ref_l, rows):
    o, l = as_f64(bits(out))[rows], lse.cpu().numpy().astype(np.float64)[rows]
    ref_o, ref_l = ref_o[rows], ref_l[rows]
    assert np.array_equal(np.isnan(o), np.isnan(ref_o)), np.argwhere(np.isnan(o) != np.isnan(ref_o))[:5]
    inf = np.isinf(ref_o)
    assert np.array_equal(np.isinf(o), inf) and np.array_equal(o[inf], ref_o[inf])
    fin = np.isfinite(ref_o)
    d = np.abs(o[fin] - ref_o[fin]) - 2.0 ** -8 * np.abs(ref_o[fin])
    assert d.size == 0 or d.max() <= 6 * (2.0 ** -8 + 2.0 ** -13), d.max()
    assert np.array_equal(np.isnan(l), np.isnan(ref_l))
    inf = np.isinf(ref_l)
    assert np.array_equal(l[inf], ref_l[inf])
    fin = np.isfinite(ref_l)
    d = np.abs(l[fin] - ref_l[fin]) - 2.0 ** -23 * np.abs(ref_l[fin])
    assert d.size == 0 or d.max() <= 2.0 ** -13, d.max()


def run(pa, inp, o, rows=None, **kw):
    status = torch.full((1,), 0, dtype=torch.int32, device="cuda")
    out = torch.full_like(inp.q[0], 9.0)          # what is not written, shows
    lse = torch.full(inp.q[0].shape[:2], 9.0, device="cuda")
    call(pa, inp, o, status=status, out=out, lse=lse, **kw)
    torch.cuda.synchronize()
    assert pa.read_device_status(status) == 0
    with np.errstate(invalid="ignore", over="ignore"):
        ref = reference(inp, o, None if rows is None else set(rows))
    same(out, lse, *ref, sorted(rows) if rows is not None else slice(None))


def put(pool, inp, b, key, value, heads=slice(None), dims=slice(None)):
    pool[int(inp.host_block_table[b, key // 16]), key % 16, heads, dims] = value


INSTANCES = [dict(), dict(softcap=8.0), dict(slopes=FLAT), dict(softcap=8.0, slopes=FLAT)]


@pytest.mark.parametrize("max_ctas", [None, 40, 7])
@pytest.mark.parametrize("k", range(4))
def test_values_and_rows_of_every_kind(cuda_lib, k, max_ctas):
    """NaN, +inf and -inf in single heads and dims, some in one dim together, seen by all rows, by the
    rows from some position on, by one document, by a window, by none; a NaN key; whole jobs and jobs
    cut between CTAs."""
    nan, inf = float("nan"), float("inf")
    rng = np.random.default_rng(k)
    for seed, q_lens, offs in ((0, [260, 40], [500, 90]), (1, [130, 1, 300], [1700, 40, 0])):
        q_lens, offs = np.array(q_lens), np.array(offs)
        lens = q_lens + offs
        inp = W.make_paged(600 + seed, lens, q_lens, device="cuda")
        K, V = inp.k_pools[0], inp.v_pools[0]
        for b, (n, off) in enumerate(zip(q_lens, offs)):
            put(V, inp, b, 3, nan, 1, 7)                              # early
            put(V, inp, b, 4, inf, 1, slice(7, 10))
            put(V, inp, b, 5, -inf, 1, slice(9, 12))
            if n > 1:
                put(V, inp, b, off + n // 3, nan, 2, slice(0, 64))    # inside the chunk
                put(V, inp, b, off + n // 2, -inf, 2, slice(60, 100))
                put(V, inp, b, off + n // 2 + 1, inf, slice(2, 4), slice(90, 128))
                put(K, inp, b, off + n - n // 8, nan, 5)              # rows from here on: NaN in head 5
                put(K, inp, b, off + n - n // 9, inf, 6)
        T = int(q_lens.sum())
        pos = np.concatenate([np.arange(l - n, l) for l, n in zip(lens, q_lens)])
        start = np.where(rng.random(T) < 0.5, 8, np.maximum(pos - rng.integers(0, 200, T), 0))
        start = np.where(rng.random(T) < 0.1, pos + 1, start)         # no key of their own
        for masks in (dict(), dict(window=150), dict(row_start=start, prefix=np.minimum(lens, 4)),
                      dict(row_start=start)):
            o = dict(INSTANCES[k], **masks)
            if not o:
                o = dict(window=10_000)
            run(cuda_lib, inp, o, max_ctas=max_ctas)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("k", range(4))
def test_pool_slots_behind_the_sequence(cuda_lib, k, value):
    """K and V behind the last key, as an unwritten pool may hold them; the last key tile is one that
    most rows of its query tile see nothing of."""
    for n, off in ((300, 87), (90, 40), (128, 1 + 128 * 9), (17, 512)):
        inp = W.make_paged(640, [off + n], [n], device="cuda")
        for key in range(off + n, -(-(off + n) // 16) * 16):
            put(inp.k_pools[0], inp, 0, key, value)
            put(inp.v_pools[0], inp, 0, key, value)
        run(cuda_lib, inp, dict(INSTANCES[k], window=10_000))


def long_call(o, n=256, L=131_072):
    inp = W.make_paged(650, [L], [n], device="cuda")
    return inp, dict(o, softcap=8.0)


ROWS = [0, 1, 31, 32, 127, 128, 200, 255]


@pytest.mark.parametrize("max_ctas", [8, None])
def test_one_early_value_in_a_long_cache(cuda_lib, max_ctas):
    """A NaN and an infinity that every row of the call sees: every warp meets them in every row, over
    131,072 keys in one piece (8 CTAs), within the waits of the other warps."""
    inp, o = long_call({})
    put(inp.v_pools[0], inp, 0, 3, float("nan"), slice(0, 8, 2), 7)
    put(inp.v_pools[0], inp, 0, 70_000, float("inf"), slice(None), slice(20, 22))
    run(cuda_lib, inp, o, ROWS, max_ctas=max_ctas)


def test_values_that_no_row_sees_in_a_long_cache(cuda_lib):
    """Keys behind a prompt that every row is kept from, in the prompt's page: every row of the call
    would meet them, and every row is computed from its own keys, 131,072 of them in one piece."""
    inp, o = long_call(dict(prefix=[5], row_start=np.full(256, 8)))
    for key in (5, 6, 7):
        put(inp.v_pools[0], inp, 0, key, float("nan"))
    run(cuda_lib, inp, o, ROWS, max_ctas=8)


def test_what_non_finite_values_cost(cuda_lib):
    """Against the same call on finite inputs (38 us): a value that all rows see costs one walk over V
    (115 us), one that a row or none sees the rows' own attention (1.7 ms; 11.3 ms a row at a time), and
    what an unwritten pool holds behind the sequence costs nothing. The limits leave a factor of two and
    more to each."""
    def us(change, o):
        inp = W.make_paged(660, [1021], [128], device="cuda")
        change(inp)
        best = float("inf")
        for _ in range(5):
            t = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
            t[0].record()
            for _ in range(4):
                call(cuda_lib, inp, o)
            t[1].record()
            torch.cuda.synchronize()
            best = min(best, t[0].elapsed_time(t[1]) * 250)
        return best

    def behind(inp):
        for k in (1021, 1022, 1023):
            put(inp.k_pools[0], inp, 0, k, nan)
            put(inp.v_pools[0], inp, 0, k, nan)

    nan, wide = float("nan"), dict(window=5000)
    hide = dict(prefix=[5], row_start=np.full(128, 8))
    clean = us(lambda inp: None, wide)
    assert us(lambda inp: put(inp.v_pools[0], inp, 0, 3, nan), wide) < 10 * clean
    assert us(lambda inp: put(inp.v_pools[0], inp, 0, 1020, nan), wide) < 120 * clean
    assert us(lambda inp: [put(inp.v_pools[0], inp, 0, k, nan) for k in (5, 6, 7)], hide) < 120 * clean
    assert us(behind, wide) < 3 * clean


@pytest.mark.parametrize("max_ctas", [None, 5])
def test_infinities_under_weights_of_zero_and_far_below_one(cuda_lib, max_ctas):
    """A key whose score is -inf has a weight of exactly 0: an infinity of its V makes the row NaN, as the
    formula's 0 times infinity does, beside rows that do not see it; a weight of e^-100 is none that fp32
    holds, and its infinity stays one; rows whose scores are all -inf are 0 whatever their V holds."""
    n, off = 150, 90
    for seed in range(4):
        inp = W.make_paged(680 + seed, [off + n], [n], device="cuda")
        K, V, inf = inp.k_pools[0], inp.v_pools[0], float("inf")
        inp.q[0][:, :, 0] = inp.q[0][:, :, 0].abs() + 0.5      # the sign of dim 0 is known
        put(K, inp, 0, 20, -inf, slice(0, 4), 0)               # score -inf in heads 0 .. 7
        put(V, inp, 0, 20, inf, slice(0, 4), slice(0, 20))
        put(V, inp, 0, 21, -inf, slice(0, 8), slice(10, 30))   # an ordinary weight
        put(V, inp, 0, off + 70, inf, slice(0, 8), slice(25, 40))   # not seen by the rows before it
        put(K, inp, 0, off + 40, -inf, slice(0, 2), 0)         # later rows: -inf again, finite V
        for o in (dict(window=1000), dict(softcap=8.0, window=70), dict(window=60, slopes=FLAT),
                  dict(row_start=np.full(n, 20), window=50), dict(row_start=np.maximum(off + np.arange(n) - 3, 0))):
            run(cuda_lib, inp, o, max_ctas=max_ctas)
        # one key far above the others: weights of e^-100 and less
        put(K, inp, 0, 5, 0.0, slice(4, 8))
        K[int(inp.host_block_table[0, 0]), 5, 4:8, 0] = 1280.0
        put(V, inp, 0, 8, inf, slice(4, 8), slice(60, 70))
        inp.q[0][:, :, 0] = 1.0
        run(cuda_lib, inp, dict(window=1000), max_ctas=max_ctas)


def test_rows_whose_scores_are_all_minus_infinity_are_zero(cuda_lib):
    n, off = 40, 100
    inp = W.make_paged(690, [off + n], [n], device="cuda")
    inp.q[0][:, :, 0] = 1.0
    for key in range(off + 10, off + 14):
        put(inp.k_pools[0], inp, 0, key, float("-inf"), slice(None), 0)
        put(inp.v_pools[0], inp, 0, key, float("nan"), slice(None), slice(0, 64))
        put(inp.v_pools[0], inp, 0, key, float("inf"), slice(None), slice(64, 100))
    for o in (dict(window=1), dict(window=3), dict(window=1, slopes=FLAT)):
        for max_ctas in (None, 3):
            run(cuda_lib, inp, o, max_ctas=max_ctas)


@pytest.mark.parametrize("split_tokens", [0, 16, 64])
@pytest.mark.parametrize("hkv", [8, 2])
def test_decode_rows_whose_scores_are_all_minus_infinity_are_zero(cuda_lib, hkv, split_tokens):
    """One launch, and split with its merges: the keys seen have scores of -inf, their V holds NaN and
    infinities; a row that also sees an ordinary key is NaN there, as the formula's 0 times infinity is."""
    hq, dims = 2 * hkv, (2 * hkv, hkv, 128, 16)
    lens = [3, 40, 700, 5000, 90, 1]
    seen = [3, 40, 33, 300, 7, 1]                       # keys of the window
    B = len(lens)
    pages = [-(-n // 16) for n in lens]
    g = torch.Generator(device="cuda").manual_seed(5)
    kp, vp = (torch.randn(sum(pages), 16, hkv, 128, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn(B, hq, 128, generator=g, device="cuda").to(torch.bfloat16)
    q[:, :, 0] = 1.0
    table = torch.zeros(B, max(pages), dtype=torch.int32, device="cuda")
    at = np.concatenate([[0], np.cumsum(pages)])
    for b in range(B):
        table[b, :pages[b]] = torch.arange(at[b], at[b + 1], device="cuda")
    for b, n in enumerate(lens):
        for key in range(n - seen[b], n):
            kp[int(at[b]) + key // 16, key % 16, :, 0] = float("-inf")
            vp[int(at[b]) + key // 16, key % 16, :, 5:60] = float("inf") if key % 2 else float("nan")
    start = torch.tensor([n - s for n, s in zip(lens, seen)], dtype=torch.int32, device="cuda")
    call = lambda start: cuda_lib.attn_decode_paged(
        q, kp, vp, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), max(lens), 0.09,
        split_tokens=split_tokens, row_start=start, dims=dims)
    out, lse = call(start)
    assert bool((out == 0).all()) and bool((lse == float("-inf")).all())
    more = torch.clamp(start - 1, min=0)
    out, lse = call(more)
    for b in range(B):
        if int(more[b]) < int(start[b]):               # the ordinary key carries the row
            assert bool(out[b, :, 5:60].isnan().all()) and bool(out[b, :, 60:].isfinite().all())
            assert bool(lse[b].isfinite().all())
        else:
            assert bool((out[b] == 0).all())
