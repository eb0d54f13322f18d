"""rope_append_paged against the fp64 definition.

Tolerance: one rounding to bf16 (half a step, 2^-8 of the value, at most) of a value computed in fp32
from x1 cos - x2 sin. The fp32 side errs by at most (|x1| + |x2|) * 2^-20 * attn_factor: the angle's
fp32 fraction of a turn (2^-25 turns, 2^-22.3 rad), sincospif (2 ulp, 2^-22), the norm's factor
(sum of 128 squares, sqrt, divide, two products: 8 roundings, 2^-21) and three more roundings.
"""
import numpy as np
import pytest
import torch

from oracle import as_f64
from oracle import serving as S
from tests.helpers import bits

pytestmark = pytest.mark.gpu


def bf(*shape, seed=0, scale=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def assert_rounded(got, want, mag):
    """got bf16 tensor, want fp64, mag: |x1| + |x2| bound of each value's terms."""
    g = as_f64(bits(got))
    bound = 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * mag + 2.0 ** -133
    bad = ~(np.abs(g - want) <= bound)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3], g[bad][:3], want[bad][:3])


def run_case(pa, T, hkv, rot, interleaved, norm, pos, seed=0, pad=0, fused=True, factor=1.0,
             scaling="none"):
    hq = 2 * hkv
    rng = np.random.default_rng(seed)
    if fused:
        qkv = bf(T + pad, hq + 2 * hkv, 128, seed=seed)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    else:
        q, k, v = bf(T + pad, hq, 128, seed=seed), bf(T + pad, hkv, 128, seed=seed + 1), bf(
            T + pad, hkv, 128, seed=seed + 2)
    pages = -(-T // 16) + 3
    slots = np.concatenate([rng.permutation(pages * 16)[:T], -np.ones(pad, np.int64)])
    kp, vp = bf(pages, 16, hkv, 128, seed=seed + 3), bf(pages, 16, hkv, 128, seed=seed + 4)
    kp0, vp0 = bits(kp).copy(), bits(vp).copy()
    freq, fac = pa.rope_inv_freq(rot, 1e6, scaling=scaling, factor=4.0)
    fac *= factor
    gq = 1 + 0.2 * torch.randn(128, device="cuda") if norm else None
    gk = 1 + 0.2 * torch.randn(128, device="cuda") if norm else None
    out = torch.full((T + pad, hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pos = np.concatenate([pos, np.zeros(pad, np.int64)])
    pa.rope_append_paged(q, k, v, torch.tensor(pos, dtype=torch.int32, device="cuda"),
                         torch.tensor(slots, device="cuda"), kp, vp, freq, interleaved=interleaved,
                         attn_factor=fac, q_gamma=gq, k_gamma=gk, eps=1e-6, q_out=out, status=status,
                         dims=(hq, hkv, 128, 16))
    torch.cuda.synchronize()
    assert pa.read_device_status(status) == 0
    f = freq.cpu().numpy()
    for x, gamma, got in ((q, gq, out[:T]), (k, gk, None)):
        x = as_f64(bits(x[:T].contiguous()))
        gm = None if gamma is None else gamma.cpu().numpy()
        want = S.rope_rows(x, pos[:T], f, interleaved, fac, gm)
        # the terms' magnitudes: a row's largest normalised value bounds both
        y = x if gm is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6) * gm
        mag = 2 * np.abs(y).max(-1, keepdims=True) * max(1.0, abs(fac))
        if got is None:
            flat = kp.view(-1, hkv, 128)[torch.tensor(slots[:T], device="cuda")]
            assert_rounded(flat, want, mag)
        else:
            assert_rounded(got, want, mag)
    # v bit for bit, untouched slots and padding rows bit for bit
    s = slots[:T]
    assert np.array_equal(bits(vp).reshape(-1, hkv, 128)[s], bits(v[:T].contiguous()))
    rest = np.setdiff1d(np.arange(pages * 16), s)
    assert np.array_equal(bits(kp).reshape(-1, hkv, 128)[rest], kp0.reshape(-1, hkv, 128)[rest])
    assert np.array_equal(bits(vp).reshape(-1, hkv, 128)[rest], vp0.reshape(-1, hkv, 128)[rest])
    assert bool((out[T:] == 7.0).all())


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("T,hkv,rot", [(1, 8, 128), (3, 4, 96), (17, 2, 64), (33, 1, 32), (5, 8, 16),
                                       (250, 8, 112), (31, 8, 128)])
def test_rows_match_the_definition(cuda_lib, T, hkv, rot, norm, interleaved):
    pos = np.random.default_rng(T).integers(0, 131072, T)
    run_case(cuda_lib, T, hkv, rot, interleaved, norm, pos, seed=T, pad=T % 4)


@pytest.mark.parametrize("interleaved", [False, True])
def test_positions_at_the_ends_of_int32(cuda_lib, interleaved):
    pos = np.array([0, 1, -1, 131071, 2**24 + 1, 2**31 - 1, -2**31, 99_999_999])
    run_case(cuda_lib, len(pos), 8, 128, interleaved, False, pos, seed=5, fused=False)


@pytest.mark.parametrize("scaling", ["linear", "ntk", "llama3", "yarn"])
def test_long_context_scalings(cuda_lib, scaling):
    pos = np.random.default_rng(2).integers(0, 131072, 40)
    run_case(cuda_lib, 40, 8, 128, False, True, pos, seed=8, scaling=scaling, factor=0.75)


def test_many_rows_over_several_passes(cuda_lib):
    """More passes than CTAs hold at once: the table buffers of a CTA are reused."""
    T = 152 * 8 * 2 * 2 + 77
    hq, hkv = 16, 8
    q, k, v = bf(T, hq, 128, seed=1), bf(T, hkv, 128, seed=2), bf(T, hkv, 128, seed=3)
    pages = -(-T // 16)
    kp, vp = bf(pages, 16, hkv, 128, seed=4), bf(pages, 16, hkv, 128, seed=5)
    freq, fac = cuda_lib.rope_inv_freq()
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 31
    out = cuda_lib.rope_append_paged(q, k, v, pos, torch.arange(T, device="cuda"), kp, vp, freq)
    torch.cuda.synchronize()
    rows = np.unique(np.concatenate([np.random.default_rng(0).integers(0, T, 300), [0, T - 1]]))
    for x, got in ((q, out), (k, kp.view(-1, hkv, 128))):
        y = as_f64(bits(x[rows].contiguous()))
        want = S.rope_rows(y, pos.cpu().numpy()[rows], freq.cpu().numpy(), False)
        assert_rounded(got[rows].contiguous(), want, 2 * np.abs(y).max(-1, keepdims=True))
    assert torch.equal(vp.view(-1, hkv, 128)[:T], v)


def test_in_place_q_and_replay(cuda_lib):
    """q_out = q, captured in a graph and replayed: each replay rotates by one more position."""
    q = bf(9, 16, 128, seed=1)
    k, v = bf(9, 8, 128, seed=2), bf(9, 8, 128, seed=3)
    kp, vp = bf(2, 16, 8, 128, seed=4), bf(2, 16, 8, 128, seed=5)
    freq, _ = cuda_lib.rope_inv_freq(64)
    pos = torch.full((9,), 3, dtype=torch.int32, device="cuda")
    slots = torch.arange(9, device="cuda")
    first = q.clone()
    want1 = cuda_lib.rope_append_paged(first, k, v, pos, slots, kp, vp, freq)
    want2 = cuda_lib.rope_append_paged(want1, k, v, pos, slots, kp, vp, freq)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cuda_lib.rope_append_paged(q, k, v, pos, slots, kp, vp, freq, q_out=q)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(q, want1)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(q, want2)


def test_slots_past_the_pool_are_flagged_and_left_alone(cuda_lib):
    q, k, v = bf(4, 16, 128), bf(4, 8, 128), bf(4, 8, 128)
    kp, vp = bf(2, 16, 8, 128, seed=4), bf(2, 16, 8, 128, seed=5)
    k0, v0 = kp.clone(), vp.clone()
    out = torch.full((4, 16, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    freq, _ = cuda_lib.rope_inv_freq()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    slots = torch.tensor([32, -1, 2**40, -2**62], device="cuda")
    cuda_lib.rope_append_paged(q, k, v, pos, slots, kp, vp, freq, q_out=out, status=status)
    torch.cuda.synchronize()
    assert cuda_lib.read_device_status(status) == 1
    assert torch.equal(kp, k0) and torch.equal(vp, v0) and bool((out == 3.0).all())


def test_non_finite_rows_stay_in_their_row(cuda_lib):
    q, k, v = bf(3, 16, 128), bf(3, 8, 128), bf(3, 8, 128)
    q[1, 4, 9] = float("nan")
    k[1, 2, 100] = float("inf")
    v[1, 0, 0] = float("nan")
    kp, vp = bf(1, 16, 8, 128, seed=4), bf(1, 16, 8, 128, seed=5)
    freq, _ = cuda_lib.rope_inv_freq()
    pos = torch.full((3,), 5, dtype=torch.int32, device="cuda")
    gamma = torch.ones(128, device="cuda")
    out = cuda_lib.rope_append_paged(q, k, v, pos, torch.arange(3, device="cuda"), kp, vp, freq,
                                     q_gamma=gamma, k_gamma=gamma)
    assert not bool(out[1, 4].isfinite().any())
    mask = torch.ones(3, 16, dtype=torch.bool, device="cuda")
    mask[1, 4] = False
    assert bool(out[mask].isfinite().all())
    kk = kp.view(-1, 8, 128)[:3]
    assert bool(kk[0].isfinite().all()) and bool(kk[2].isfinite().all())
    assert torch.equal(vp.view(-1, 8, 128)[:3].view(torch.int16), v.view(torch.int16))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("hkv", [1, 2, 8])
def test_rows_past_a_cta_s_first_table(cuda_lib, hkv, interleaved):
    """21,001 rows: every CTA fills its table of angles at least three times on any GPU of up to 152 SMs
    (two CTAs an SM, 32 tokens a table: 9,728 tokens are held at once)."""
    T, hq = 21_001, 2 * hkv
    qkv = bf(T, hq + 2 * hkv, 128, seed=1)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    pages = -(-T // 16)
    kp = torch.zeros(pages, 16, hkv, 128, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    freq, fac = cuda_lib.rope_inv_freq(scaling="yarn", factor=4.0)
    rng = np.random.default_rng(hkv)
    pos = rng.integers(0, 131072, T)
    slots = torch.tensor(rng.permutation(pages * 16)[:T], device="cuda")
    gamma = 1 + 0.2 * torch.randn(128, device="cuda")
    out = cuda_lib.rope_append_paged(q, k, v, torch.tensor(pos, dtype=torch.int32, device="cuda"), slots, kp, vp,
                                     freq, interleaved=interleaved, attn_factor=fac, q_gamma=gamma, k_gamma=gamma,
                                     dims=(hq, hkv, 128, 16))
    torch.cuda.synchronize()
    # rows of every table of a CTA, its first and last tokens among them
    rows = np.unique(np.concatenate([rng.integers(0, T, 500), np.arange(9700, 9760), [0, 31, 32, T - 1]]))
    gm = gamma.cpu().numpy()
    at = torch.tensor(rows, device="cuda")
    for x, got in ((q, out[at]), (k, kp.view(-1, hkv, 128)[slots[at]])):
        y = as_f64(bits(x[at].contiguous()))
        want = S.rope_rows(y, pos[rows], freq.cpu().numpy(), interleaved, fac, gm)
        n = y / np.sqrt((y * y).mean(-1, keepdims=True) + 1e-6) * gm
        assert_rounded(got.contiguous(), want, 2 * np.abs(n).max(-1, keepdims=True) * fac)
    assert torch.equal(vp.view(-1, hkv, 128)[slots], v)
