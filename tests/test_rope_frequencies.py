"""rope_inv_freq against the definitions at every pair. Both sides are 64-bit: a power of theta and at
most six roundings apart, so 2^-48 of the value; the factor of cos and sin is rounded to fp32 once."""
import numpy as np
import pytest

from oracle import serving as S


@pytest.fixture(scope="module")
def pa():
    from long_context_paged_gb300 import build as b
    b.build()
    import long_context_paged_gb300 as pa
    return pa


CASES = [dict(kind="none"), dict(kind="linear", factor=8.0), dict(kind="ntk", factor=3.0),
         dict(kind="llama3", factor=8.0, original=8192), dict(kind="llama3", factor=32.0, original=8192),
         dict(kind="llama3", factor=4.0, original=2048, low_freq_factor=2.0, high_freq_factor=40.0),
         dict(kind="yarn", factor=4.0, original=32768), dict(kind="yarn", factor=40.0, original=4096),
         dict(kind="yarn", factor=2.5, original=1000, beta_fast=8.0, beta_slow=2.0, attn_factor=1.25),
         dict(kind="yarn", factor=0.5, original=32768)]


@pytest.mark.parametrize("rot,theta", [(128, 1e6), (64, 1e4), (96, 5e5), (16, 1e6), (4, 1e4)])
@pytest.mark.parametrize("k", range(len(CASES)))
def test_every_pair(pa, k, rot, theta):
    c = dict(CASES[k])
    want, scale = S.rope_frequencies(rot, theta, **c)
    kind, original = c.pop("kind"), c.pop("original", 32768)
    got, factor = pa.rope_inv_freq(rot, theta, scaling=kind, original_max_position=original, device="cpu", **c)
    got = got.numpy()
    assert got.shape == want.shape
    assert (np.abs(got - want) <= 2.0 ** -48 * want).all(), np.argmax(np.abs(got / want - 1))
    assert abs(factor - scale) <= 2.0 ** -24 * scale
    if kind in ("llama3", "yarn") and rot >= 64 and c["factor"] > 1:  # (a blend to check is there)
        plain, _ = S.rope_frequencies(rot, theta)
        ratio = want / plain
        assert ((ratio < 1 - 1e-6) & (ratio > 1 / c["factor"] + 1e-6)).any()
