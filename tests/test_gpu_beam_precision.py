"""What beam_select's scores are worth: the normaliser's error at logits made to bring it out, and grids that are cut
by the number of rows.

Bounds. A term of the sum is 2^((x - ref) log2 e) against a reference ref of its thread, which the thread's
largest logit is at most 4.5 above: with y = |x - ref|, the difference and the product round by y 2^-24 each
(relative to the term), the constant's own error is 1.4e-8 y, the exponential's 2^-22: 1.4e-7 y + 2.4e-7. Terms
take at most 6 roundings of 2^-24 to enter their thread's sum, a pair of floats; lanes, warps and pieces 12 more
and three factors of 2^-23: 24 * 2^-24 = 1.43e-6. The terms that matter lie up to the logarithm of their number
below their thread's reference, for fewer than 2^25 logits 10 on the average: 3.1e-6, and a sum that is rescaled as
its reference moves gets 2^-22 more where it still matters: 2^-18 in all cases. In a row of one warp whose terms
all lie within 4.5 of the reference: 1.4e-7 * 4.5 + 2.4e-7 + (6 + 1 + 5) * 2^-24 = 1.59e-6, under 28 * 2^-24.
Scores are rounded to fp32 at the end: 2^-24 of them."""
import pytest
import torch

pytestmark = pytest.mark.gpu
INF = float("inf")


def normaliser_error(pa, x):
    """One beam with score 0: what its best score says of ln sum exp, less the 64-bit one."""
    got = pa.beam_select(x.view(1, 1, -1).cuda(), torch.zeros(1, 1, device="cuda"), 1)
    torch.cuda.synchronize()
    d = x.double()
    want = float(d.max() - torch.logsumexp(d, 0))
    return abs(float(got.scores[0, 0]) - want) - 2.0 ** -24 * abs(want)


# (top, how far the logits that each thread reads first lie below it, how far the others do)
FP32 = [(15.9, 36.1, 0.5122034), (15.9, 36.1, 0.5271186), (20.3, 39.9, 0.5271186), (15.9, 39.9, 0.51220338),
        (3.1, 39.3, 0.37), (7.7, 38.7, 0.81), (1.3, 20.2, 0.44), (11.2, 12.7, 0.23), (11.2, 8.9, 0.61), (2.7, 4.4, 0.3),
        (2.7, 4.1, 0.3), (2.7, 3.9, 0.3)]
BF16 = [(3.0, 37.0, 0.375), (7.75, 37.0, 0.375), (1.25, 37.0, 0.375), (11.25, 20.0, 0.625), (11.25, 5.0, 0.875)]


@pytest.mark.parametrize("dtype,case", [(torch.float32, c) for c in FP32] + [(torch.bfloat16, c) for c in BF16])
def test_logits_that_start_far_below_the_best(cuda_lib, dtype, case):
    """A short row is read by one warp, four vectors a thread: the first 32 vectors are the first that each reads."""
    top, low, near = case
    vec = 16 // dtype.itemsize
    x = torch.full((127 * vec,), top - near, dtype=torch.float32)
    x[:32 * vec] = top - low
    x[-1] = top
    assert normaliser_error(cuda_lib, x.to(dtype)) <= 28 * 2.0 ** -24


@pytest.mark.parametrize("rows,V", [(1, 150_000), (900, 40_000), (3000, 9_000)])
def test_normalisers_of_rows_made_of_two_values(cuda_lib, rows, V):
    """Sums of equal terms, whose roundings all go the same way, at every distance that matters."""
    g = torch.Generator().manual_seed(V)
    near = torch.rand(rows, generator=g) * 12
    x = (20 * torch.rand(rows, generator=g) - near).unsqueeze(1).repeat(1, V)
    best = torch.randint(0, V, (rows,), generator=g)
    x[torch.arange(rows), best] += near
    x[::3, :V // 3] -= 25                                     # (a third starts low)
    x = x.cuda()
    got = cuda_lib.beam_select(x.unsqueeze(1), torch.zeros(rows, 1, device="cuda"), 1)
    torch.cuda.synchronize()
    assert torch.equal(got.tokens[:, 0].cpu().long(), x.argmax(1).cpu())
    d = x.double()
    want = d.amax(1) - torch.logsumexp(d, 1)
    off = (got.scores[:, 0].double() - want).abs() - 2.0 ** -24 * want.abs()
    assert float(off.max()) <= 2.0 ** -18


@pytest.mark.parametrize("N,W,V,dtype", [(100, 8, 30_000, torch.bfloat16), (40, 8, 30_001, torch.float32),
                                         (400, 8, 9_000, torch.bfloat16), (1000, 4, 2_500, torch.float32)])
def test_more_rows_than_pieces(cuda_lib, N, W, V, dtype):
    """So many rows that a piece of one is several units a warp, down to a row a piece."""
    g = torch.Generator(device="cuda").manual_seed(V)
    x = (torch.randn(N, W, V, generator=g, device="cuda") * 3).to(dtype)
    s = -6 * torch.rand(N, W, generator=g, device="cuda")
    k = 12
    got = cuda_lib.beam_select(x, s, k)
    torch.cuda.synchronize()
    exact = (s.double().unsqueeze(2) + torch.log_softmax(x.double(), 2)).view(N, -1)
    want, place = exact.sort(dim=1, descending=True, stable=True)
    want, place = want[:, :k], place[:, :k]
    mine = got.parents.long() * V + got.tokens.long()
    assert (mine >= 0).all() and all(len(set(r)) == k for r in mine.tolist())
    # another candidate only where its score is within two normalisers' error of the place's
    at = exact.gather(1, mine)
    assert ((at - want).abs()[mine != place] <= 2.0 ** -17).all()
    assert ((got.scores.double() - at).abs() <= 2.0 ** -18 + 2.0 ** -24 * at.abs()).all()
    # within a beam the order is that of the logits
    logit = x.view(N, -1).gather(1, mine).double()
    for b in range(W):
        one = torch.where(got.parents == b, logit, torch.full_like(logit, -INF))
        runs = [[v for v in r if v > -INF] for r in one.tolist()]
        assert all(r == sorted(r, reverse=True) for r in runs)
