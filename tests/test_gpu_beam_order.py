"""beam_select's order within a beam: that of its logits, down to 2^-45 of the score that they are added to; and the
last beams and tokens of what a request can have.

Scores are pairs of floats. The sum of a beam's shift (score less normaliser), a pair, with a logit is rounded once,
where the low parts are added: by 2^-24 of them, which are 2^-24 of the shift and of the score at most. Two logits
tie or change places only if they lie closer together than two such roundings, 2^-47 (|shift| + |score|), which is
2^-45 of the larger of a beam's score and its normaliser at most."""
import pytest
import torch

from tests.test_gpu_beam import check

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.mark.parametrize("V", [100, 20_000])
@pytest.mark.parametrize("score", [-300.0, -3.0e6, 40.0, -0.25])
@pytest.mark.parametrize("near", [0.0, 1.0e-6, 1.52587890625e-5, -3.0517578125e-5, 0.125])
def test_the_order_within_a_beam_is_that_of_its_logits(cuda_lib, V, score, near):
    """Logits 2^-45 of the score apart or, where that is more, steps of their own type; about halves of a step of the
    score too."""
    x = torch.full((2, 3, V), -25.0)
    apart = max(abs(score), 2.0) * 2.0 ** -45               # (six logits near 0: the normaliser is below 2)
    steps = []
    at32 = torch.tensor(near, dtype=torch.float32)
    for _ in range(6):
        steps.append(float(at32))
        least = torch.tensor(steps[-1] + apart, dtype=torch.float32)
        if float(least) - steps[-1] < apart:
            least = torch.nextafter(least, torch.tensor(INF))
        at32 = least
    at = [3, 7, V // 2, V // 2 + 1, V - 2, V - 1]
    for order in ([0, 1, 2, 3, 4, 5], [5, 4, 3, 2, 1, 0], [2, 0, 5, 1, 4, 3]):
        for b in range(3):
            for i, o in enumerate(order):
                x[:, b, at[i]] = steps[o]
        s = torch.full((2, 3), score)
        s[1, 1] = -INF
        want = [at[order.index(o)] for o in (5, 4, 3, 2, 1, 0)]
        for k in (1, 4, 6, 18):
            got = cuda_lib.beam_select(x.cuda(), s.cuda(), k)
            torch.cuda.synchronize()
            for n in range(2):
                parents, tokens = got.parents[n].tolist(), got.tokens[n].tolist()
                for b in range(3):
                    mine = [t for p, t in zip(parents, tokens) if p == b]
                    assert mine[:6] == want[:len(mine)], (n, b, k, mine)


@pytest.mark.parametrize("W,V", [(64, 4097), (33, 70_001), (1, 1), (2, 2), (64, 1), (7, 1024), (3, 1025)])
def test_places_of_the_last_beam_and_token(cuda_lib, W, V):
    """Beams and tokens at the ends of what their bits hold."""
    x = torch.full((1, W, V), -3.0)
    x[0, W - 1, V - 1] = 9.0
    x[0, 0, V - 1] = 8.0
    s = torch.zeros(1, W)
    live = torch.ones(1, W, dtype=torch.int32)
    got = check(cuda_lib, x.cuda(), s.cuda(), 5)
    if V > 1:
        assert (got.parents[0, 0].item(), got.tokens[0, 0].item()) == (W - 1, V - 1)
    live[0, W - 1] = 0
    s[0, W - 1] = 2.0
    got = check(cuda_lib, x.cuda(), s.cuda(), 5, live.cuda(), eos=V - 1)
    assert (got.parents[0, 0].item(), got.tokens[0, 0].item(), got.live[0, 0].item()) == (W - 1, V - 1, 0)
