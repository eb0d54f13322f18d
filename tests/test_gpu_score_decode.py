"""attn_decode_paged with score options against the fp64 definition.

Tolerance: fp32 throughout and one rounding to bf16, so an output may be off by half a bf16 step
(2^-8 of the value) plus the weights' error, below 2^-16 of the largest value entering the mean: a
score in log2 units errs by the product's 128 terms (2^-24 * 128^0.5 of |q||k|, under 2^-15 for the
scores here, |s| < 60), the cap (2^-22 of it) and the exponential. |v| < 6 here: 6 * 2^-13 covers
weights off by 2^-13 in both numerator and denominator. The log-sum-exp moves by the scores' error
and its own rounding: 2^-13 + 2^-23 |lse|.
"""
import numpy as np
import pytest
import torch

import workloads as W
from oracle import as_f64
from oracle import serving as S
from tests.helpers import bits

pytestmark = pytest.mark.gpu


def close(out, lse, ref_o, ref_l, what=""):
    o, l = as_f64(bits(out)), lse.cpu().numpy().astype(np.float64)
    ok = np.abs(o - ref_o) <= 2.0 ** -8 * np.abs(ref_o) + 6 * 2.0 ** -13
    assert ok.all(), (what, int((~ok).sum()), np.argwhere(~ok)[:4], o[~ok][:4], ref_o[~ok][:4])
    inf = np.isneginf(ref_l)
    assert np.array_equal(np.isneginf(l), inf), what
    assert not o[inf].any(), what
    d = np.abs(l[~inf] - ref_l[~inf]) - 2.0 ** -23 * np.abs(ref_l[~inf])
    assert d.size == 0 or d.max() <= 2.0 ** -13, (what, d.max())


def dev(a, dtype=torch.int32):
    return torch.tensor(np.asarray(a), dtype=dtype, device="cuda")


def poison_unseen(inp, o, Hkv=8):
    """NaN into every slot that the definition says no row sees; -1 into unseen pages' entries."""
    bt = inp.host_block_table.copy()
    seen = np.zeros((inp.num_pages, 16), bool)
    for b, L in enumerate(inp.host_seq_lens):
        vis = S.visible(L - 1, int(L), **S._opts(o, b, b))
        for lp in range(-(-int(L) // 16)):
            v = vis[lp * 16:(lp + 1) * 16]
            if v.any():
                seen[bt[b, lp], :len(v)] |= v
            else:
                bt[b, lp] = -1
    mask = torch.tensor(~seen, device="cuda")
    for p in (inp.k_pools[0], inp.v_pools[0]):
        p[mask] = float("nan")
    inp.host_block_table = bt
    inp.block_table = dev(bt)


def run(pa, inp, o, *, split=0, max_ctas=None, bound=None, poison=True, scale=None, status=None,
        check=True, what=""):
    if poison:
        poison_unseen(inp, o)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(softcap=o.get("softcap", 0.0), window=o.get("window", 0))
    if o.get("slopes") is not None:
        kw["alibi_slopes"] = dev(o["slopes"], torch.float32)
    if o.get("prefix") is not None:
        kw["prefix_lens"] = dev(o["prefix"])
        kw["max_prefix_len"] = o.get("max_prefix")
    if o.get("row_start") is not None:
        kw["row_start"] = dev(o["row_start"])
    scale = inp.scale if scale is None else scale
    out, lse = pa.attn_decode_paged(inp.q[0], inp.k_pools[0], inp.v_pools[0], inp.block_table,
                                    inp.seq_lens, bound or max(1, int(inp.host_seq_lens.max())),
                                    scale, split_tokens=split, max_ctas=max_ctas, status=status, **kw)
    torch.cuda.synchronize()
    assert pa.read_device_status(status) == 0
    if check:
        ref = S.decode_scored(bits(inp.q[0]), bits(inp.k_pools[0]), bits(inp.v_pools[0]),
                              np.maximum(inp.host_block_table, 0), inp.host_seq_lens, scale, **o)
        close(out, lse, *ref, what=what or str(o))
    return out, lse


SLOPES = 2.0 ** (-0.5 * np.arange(1, 17))
OPTIONS = [
    dict(softcap=30.0), dict(softcap=0.5), dict(slopes=SLOPES), dict(window=1), dict(window=16),
    dict(window=100), dict(window=17, prefix="p"), dict(prefix="p"), dict(row_start="r"),
    dict(row_start="r", prefix="p", slopes=SLOPES),
    dict(softcap=20.0, slopes=SLOPES, window=300, prefix="p", row_start="r"),
]


def options(o, lens, rng):
    o = dict(o)
    if o.get("prefix") == "p":
        o["prefix"] = rng.integers(0, np.maximum(lens, 1) + 40)
        o["prefix"][::3] = 0
    if o.get("row_start") == "r":
        o["row_start"] = rng.integers(-3, lens + 2)
        o["row_start"][::4] = lens[::4]     # nothing of its own
    return o


@pytest.mark.parametrize("k", range(len(OPTIONS)))
@pytest.mark.parametrize("path", ["one launch", "split", "split 32"])
def test_options(cuda_lib, k, path):
    rng = np.random.default_rng(100 + k)
    lens = np.array([1, 0, 15, 16, 17, 500, 33, 1000]) if path != "split" else np.concatenate(
        [rng.integers(1, 3000, 20), [1, 16, 4097]])
    o = options(OPTIONS[k], lens, rng)
    inp = W.make_paged(200 + k, lens, np.ones(len(lens), np.int64), device="cuda", q_scale=3.0)
    run(cuda_lib, inp, o, split={"one launch": 0, "split": 0, "split 32": 32}[path],
        max_ctas=3 if path == "split" else None)


@pytest.mark.parametrize("lens,o", [
    ([40_000], dict(window=4096, prefix=[1000])),
    ([40_000], dict(slopes=SLOPES * 8)),
    ([30_000, 5], dict(row_start=[30_000, 0], prefix=[77, 0], slopes=SLOPES)),  # far prefix alone
    ([20_001, 20_002, 19_999], dict(softcap=50.0, slopes=SLOPES, window=8192)),
])
def test_long_sequences(cuda_lib, lens, o):
    inp = W.make_paged(7, lens, [1] * len(lens), device="cuda", q_scale=4.0)
    run(cuda_lib, inp, o)
    run(cuda_lib, inp, o, split=512, poison=False)


@pytest.mark.parametrize("hkv", [1, 2, 4])
def test_head_partitions(cuda_lib, hkv):
    rng = np.random.default_rng(hkv)
    lens = np.array([700, 33, 2100, 1, 16, 999])
    inp = W.make_paged(3, lens, np.ones(6, np.int64), device="cuda", q_scale=2.0)
    q = inp.q[0][:, :2 * hkv].contiguous()
    kp, vp = (p[:, :, :hkv].contiguous() for p in (inp.k_pools[0], inp.v_pools[0]))
    o = dict(softcap=15.0, slopes=SLOPES[:2 * hkv], window=333, prefix=rng.integers(0, 200, 6),
             row_start=rng.integers(0, lens))
    for split in (0, 48):
        for cap in (None, 2):
            out, lse = cuda_lib.attn_decode_paged(
                q, kp, vp, inp.block_table, inp.seq_lens, 2100, inp.scale, split_tokens=split,
                max_ctas=cap, dims=(2 * hkv, hkv, 128, 16), softcap=15.0, window=333,
                alibi_slopes=dev(o["slopes"], torch.float32), prefix_lens=dev(o["prefix"]),
                row_start=dev(o["row_start"]))
            ref = S.decode_scored(bits(q), bits(kp), bits(vp), inp.host_block_table,
                                  inp.host_seq_lens, inp.scale, **o)
            close(out, lse, *ref, what=f"{hkv} heads, split {split}, cap {cap}")


def test_no_option_set_equals_the_plain_call(cuda_lib):
    """A window and a prefix that exclude nothing: the plain call's values up to rounding."""
    inp = W.make_paged(11, [3000, 17, 900], [1, 1, 1], device="cuda")
    plain = cuda_lib.attn_decode_paged(inp.q[0], inp.k_pools[0], inp.v_pools[0], inp.block_table,
                                       inp.seq_lens, 3000, inp.scale)
    out, lse = run(cuda_lib, inp, dict(window=3000), poison=False)
    assert torch.equal(out, plain[0]) and torch.allclose(lse, plain[1], atol=1e-6)


def test_visible_scores_of_minus_infinity(cuda_lib):
    """A bias that drives every visible score to -inf leaves o = 0, lse = -inf; an infinite or NaN
    key among the visible ones reaches its row alone."""
    inp = W.make_paged(12, [50, 60, 70], [1, 1, 1], device="cuda")
    bt = inp.host_block_table
    inp.k_pools[0][int(bt[1, 0]), 3, 2] = float("nan")
    o, l = cuda_lib.attn_decode_paged(
        inp.q[0], inp.k_pools[0], inp.v_pools[0], inp.block_table, inp.seq_lens, 70, inp.scale,
        alibi_slopes=dev(np.full(16, 3e38), torch.float32), prefix_lens=dev([0, 60, 3]),
        row_start=dev([0, 0, 70]))
    torch.cuda.synchronize()
    # own key at distance 0 carries all the weight
    v = inp.v_pools[0][int(bt[0, 3]), 1].repeat_interleave(2, 0)
    assert torch.equal(o[0], v)
    assert bool(o[1, 4:6].isnan().all()) and bool(o[1, :4].isfinite().all())
    # nearest key of the prefix carries all of row 2's weight; its lse is out of fp32's range
    v = inp.v_pools[0][int(bt[2, 0]), 2].repeat_interleave(2, 0)
    assert torch.equal(o[2], v) and bool(torch.isneginf(l[2]).all())
    inp.k_pools[0][int(bt[2, 0]), :3] = float("inf")
    q = -inp.q[0].abs()
    o, l = cuda_lib.attn_decode_paged(q, inp.k_pools[0], inp.v_pools[0], inp.block_table,
                                      inp.seq_lens, 70, inp.scale, prefix_lens=dev([0, 0, 3]),
                                      row_start=dev([0, 0, 70]))
    assert not bool(o[2].any()) and bool(torch.isneginf(l[2]).all())


def test_prefix_lengths_outside_the_bound_are_cut_and_flagged(cuda_lib):
    inp = W.make_paged(13, [400, 400], [1, 1], device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = cuda_lib.attn_decode_paged(inp.q[0], inp.k_pools[0], inp.v_pools[0], inp.block_table,
                                          inp.seq_lens, 400, inp.scale, window=20, status=status,
                                          prefix_lens=dev([-5, 300]), max_prefix_len=32)
    assert cuda_lib.read_device_status(status) == cuda_lib.DEV_ERR_LENGTH
    ref = S.decode_scored(bits(inp.q[0]), bits(inp.k_pools[0]), bits(inp.v_pools[0]),
                          inp.host_block_table, inp.host_seq_lens, inp.scale, window=20,
                          prefix=[0, 32])
    close(out, lse, *ref)


def test_bad_pages_that_are_seen_are_flagged(cuda_lib):
    inp = W.make_paged(14, [100], [1], device="cuda")
    bt = inp.block_table.clone()
    bt[0, :5] = -1                       # window 20 of 100 keys: pages 5 and 6
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for split in (0, 16):
        cuda_lib.attn_decode_paged(inp.q[0], inp.k_pools[0], inp.v_pools[0], bt, inp.seq_lens, 100,
                                   inp.scale, window=20, status=status, split_tokens=split)
        assert cuda_lib.read_device_status(status) == 0
        cuda_lib.attn_decode_paged(inp.q[0], inp.k_pools[0], inp.v_pools[0], bt, inp.seq_lens, 100,
                                   inp.scale, window=21, status=status, split_tokens=split)
        assert cuda_lib.read_device_status(status) == cuda_lib.DEV_ERR_PAGE_OOB


def test_replayed_from_a_graph_with_new_lengths(cuda_lib):
    inp = W.make_paged(15, [900, 2000], [1, 1], device="cuda", q_scale=2.0)
    kw = dict(softcap=10.0, window=512, prefix_lens=dev([40, 0]), max_prefix_len=100)
    out, lse = torch.empty_like(inp.q[0]), torch.empty(2, 16, device="cuda")
    ws = torch.empty(cuda_lib.decode_workspace_size(2, 2000), dtype=torch.uint8, device="cuda")

    def call():
        cuda_lib.attn_decode_paged(inp.q[0], inp.k_pools[0], inp.v_pools[0], inp.block_table,
                                   inp.seq_lens, 2000, inp.scale, out=out, lse=lse, workspace=ws, **kw)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for lens in ([900, 2000], [1, 1999], [700, 0]):
        inp.seq_lens.copy_(dev(lens))
        g.replay()
        torch.cuda.synchronize()
        ref = S.decode_scored(bits(inp.q[0]), bits(inp.k_pools[0]), bits(inp.v_pools[0]),
                              inp.host_block_table, lens, inp.scale, softcap=10.0, window=512,
                              prefix=[40, 0])
        close(out, lse, *ref, what=str(lens))


@pytest.mark.parametrize("lens", [[40, 900], [40, 50000]])
@pytest.mark.parametrize("slope", [float("inf"), float("-inf"), float("nan")])
def test_rows_without_keys_under_any_slope(cuda_lib, lens, slope):
    inp = W.make_paged(71, lens, [1, 1], device="cuda")
    slopes = torch.full((16,), 0.25, device="cuda")
    slopes[5] = slope
    out, lse = cuda_lib.attn_decode_paged(inp.q[0], inp.k_pools[0], inp.v_pools[0], inp.block_table,
                                          inp.seq_lens, max(lens), inp.scale, alibi_slopes=slopes,
                                          row_start=dev([0, lens[1]]))
    assert bool((lse[1] == float("-inf")).all()) and not bool(out[1].any())
    keep = [h for h in range(16) if h != 5]
    assert bool(lse[0, keep].isfinite().all()) and bool(out[0, keep].isfinite().all())
