"""attn_decode_paged_shared keeps the softmax weights of beams and single rows to 2^-15, as two bf16s; those of pages
that more than 8 rows share are one bf16.

Tolerance: with q at 0.05 of the usual size the sums |q_i k_i| of a score stay below 2 in log2 units, so an fp32 sum of
128 products moves a weight by 2^-17 at most and the exponential by 2^-22; the weights' own rounding is 2^-15 and 2^-20.
Together below 2^-14 of the mean of |v| under the weights, and 2^-8 of the output for its rounding. (One bf16 for a
weight is off by up to 2^-8 of it.)"""
import numpy as np
import pytest
import torch

from oracle import as_f64
from tests.helpers import bits
from tests.test_gpu_shared_decode import SCALE, Inputs, dev

pytestmark = pytest.mark.gpu

FEW = [
    ([(0, [2, 3, 16, 40])], []),                      # rows alone
    ([(1, [17, 18])], [7]),                           # a small group
    ([(2, [33 + i % 20 for i in range(8)])], []),
]
MANY = [
    ([(1, [17 + i % 3 for i in range(9)])], []),      # a row more than the form for small groups takes
    ([(2, [32] * 64)], [2]),
    ([(9, [145 + i % 40 for i in range(131)])], []),
]


def alternating(groups, alone, seed, hkv=2):
    """V of 4 and -4 in turn: what is left of a row's sum is the difference of its weights."""
    x = Inputs(groups, alone, hkv=hkv, seed=seed, qscale=0.05)
    sign = 4.0 * (1 - 2 * (torch.arange(16, device="cuda") % 2)).view(1, 16, 1, 1)
    x.v = torch.where(torch.isnan(x.v), x.v, sign.expand_as(x.v).to(torch.bfloat16)).contiguous()
    return x


@pytest.mark.parametrize("groups,alone,step", [(*g, 2.0 ** -14) for g in FEW] + [(*g, 2.0 ** -8 + 2.0 ** -14) for g in MANY])
def test_weights(cuda_lib, groups, alone, step):
    x = alternating(groups, alone, len(groups[0][1]))
    out, lse = x.call(cuda_lib)
    assert x.flags == 0
    ref, ref_l, mag = x.reference()
    off = np.abs(as_f64(bits(out)) - ref)
    assert (off <= 2.0 ** -8 * np.abs(ref) + step * mag).all(), float((off - 2.0 ** -8 * np.abs(ref)).max())
    assert np.abs(lse.cpu().numpy() - ref_l).max() <= 2.0 ** -13


def test_the_last_few_rows_of_a_large_group(cuda_lib):
    """67 rows: 64 in one piece, three in another, whose weights are kept."""
    x = alternating([(3, [48] * 67)], [], 3)
    out, _ = x.call(cuda_lib)
    ref, _, mag = x.reference()
    off = np.abs(as_f64(bits(out)) - ref)[64:]
    assert (off <= 2.0 ** -8 * np.abs(ref[64:]) + 2.0 ** -14 * mag[64:]).all()


@pytest.mark.parametrize("groups,alone", FEW)
def test_as_the_plain_decode(cuda_lib, groups, alone):
    """Both keep the weights, so they differ where a rounding of the output falls the other way, and not by more."""
    x = alternating(groups, alone, 7, hkv=8)
    out, _ = x.call(cuda_lib)
    plain, _ = cuda_lib.attn_decode_paged(x.q, x.k, x.v, dev(np.maximum(x.table, 0)), dev(x.lens), max(x.lens), SCALE)
    torch.cuda.synchronize()
    a, b = out.double(), plain.double()
    # (a step of bf16 is 2^-7 of a value at most; below that, the weights' own 2^-14 of 4)
    assert ((a - b).abs() <= 2.0 ** -7 * torch.maximum(a.abs(), b.abs()) + 2.0 ** -13 * 4).all()


@pytest.mark.parametrize("groups,alone", FEW[1:] + MANY)
def test_an_infinity_of_v_counts_as_one(cuda_lib, groups, alone):
    """A key with any weight whose V is infinite makes its rows' outputs infinite, of its sign, and not NaN."""
    x = Inputs(groups, alone, hkv=2, seed=5)
    clean, _ = x.call(cuda_lib)
    page = int(x.table[0, 0])                          # shared by the first group's rows
    for token in range(16):                            # (weights of every kind, exact in 8 bits and not)
        x.v[page, token, 1, token] = float("inf")
        x.v[page, token, 1, 64 + token] = float("-inf")
    out, _ = x.call(cuda_lib)
    n = len(groups[0][1])
    for row in range(len(x.lens)):
        got = out[row, 2:4]
        if row >= n:
            assert torch.equal(out[row], clean[row])
            continue
        assert (got[:, :16] == float("inf")).all() and (got[:, 64:80] == float("-inf")).all()
        got[:, :16], got[:, 64:80] = clean[row, 2:4, :16], clean[row, 2:4, 64:80]
        assert torch.equal(out[row], clean[row])
