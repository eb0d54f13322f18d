"""Host-side refusals of the page-table and rotary calls (no GPU: each is returned before any
CUDA call; the pointers are fake, aligned addresses and never read)."""
import ctypes

import pytest

INVALID, UNSUPPORTED, OK = 1, 2, 0
A = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 4)


@pytest.fixture(scope="module")
def lib():
    from long_context_paged_gb300 import build as b
    b.build()
    import long_context_paged_gb300 as pa
    return pa.load()


def test_step_plan(lib):
    def call(cached=A, new=A, batch=2, bt=A, stride=4, free=A, cap=8, count=A, pages=64, rows=3,
             count_out=A, cu=A, seq=A, pos=A, slots=A):
        return lib.paged_step_plan(cached, new, batch, bt, stride, free, cap, count, pages, rows,
                                   count_out, cu, seq, pos, slots, None, None)
    for bad in (dict(batch=-1), dict(stride=0), dict(stride=1 << 28), dict(cap=-1), dict(pages=0),
                dict(rows=-1), dict(slots=ODD)):
        assert call(**bad) == INVALID, bad
    for name in ("cached", "new", "bt", "free", "count", "count_out", "cu", "seq", "pos", "slots"):
        assert call(**{name: None}) == INVALID, name
    assert call(batch=4097) == UNSUPPORTED


def test_release(lib):
    def call(begin=A, end=A, batch=2, bt=A, stride=4, free=A, cap=8, count=A, pages=64, out=A):
        return lib.paged_release(begin, end, batch, bt, stride, free, cap, count, pages, out, None, None)
    for bad in (dict(batch=-1), dict(stride=0), dict(cap=-1), dict(pages=0)):
        assert call(**bad) == INVALID, bad
    for name in ("begin", "end", "bt", "free", "count", "out"):
        assert call(**{name: None}) == INVALID, name
    assert call(batch=4097) == UNSUPPORTED


def test_rope_append(lib):
    import long_context_paged_gb300 as pa

    def call(dims=(16, 8, 128, 16), rot=128, freq=A, factor=1.0, q=A, qs=2048, k=A, ks=1024, v=A,
             vs=1024, rows=2, pos=A, slots=A, qg=None, kg=None, eps=1e-6, out=ctypes.c_void_p(1 << 22),
             kp=A, vp=A, pages=8):
        return lib.rope_append_paged(pa.Dims(*dims), rot, 0, freq, factor, q, qs, k, ks, v, vs, rows,
                                     pos, slots, qg, kg, eps, out, kp, vp, pages, None, None)
    assert call(dims=(16, 4, 128, 16)) == UNSUPPORTED
    for rot in (0, 8, 24, 136, 144, -16):
        assert call(rot=rot) == UNSUPPORTED, rot
    nan = float("nan")
    for bad in (dict(rows=-1), dict(pages=0), dict(eps=-1.0), dict(eps=nan), dict(factor=nan),
                dict(qs=2040), dict(ks=1023), dict(vs=512), dict(qs=2052), dict(ks=1028),
                dict(out=A, qs=4096)):  # in place over strided rows
        assert call(**bad) == INVALID, bad
    for name in ("freq", "q", "k", "v", "pos", "slots", "out", "kp", "vp"):
        assert call(**{name: None}) == INVALID, name
    for name in ("freq", "q", "k", "v", "slots", "qg", "kg", "out", "kp", "vp"):
        assert call(**{name: ODD}) == INVALID, name
    assert call(rows=0, q=None) == OK


def test_rope_inv_freq(lib):
    import math

    import long_context_paged_gb300 as pa
    f, a = pa.rope_inv_freq(64, 1e4, device="cpu")
    assert a == 1.0 and f.shape == (32,) and f[0] == 1.0
    assert math.isclose(f[31].item(), 1e4 ** (-62 / 64), rel_tol=1e-15)
    assert pa.rope_inv_freq(64, 1e4, scaling="linear", factor=8, device="cpu")[0][0] == 0.125
    # ntk: the fastest pair is kept, the slowest one stretched by the factor
    n = pa.rope_inv_freq(64, 1e4, scaling="ntk", factor=8, device="cpu")[0]
    assert n[0] == 1.0 and math.isclose(n[31].item(), f[31].item() / 8, rel_tol=1e-12)
    for kind in ("llama3", "yarn"):  # fast pairs kept, slow pairs divided
        s, b = pa.rope_inv_freq(64, 1e6, scaling=kind, factor=8, original_max_position=8192, device="cpu")
        base = pa.rope_inv_freq(64, 1e6, device="cpu")[0]
        assert s[0] == base[0] and math.isclose(s[31].item(), base[31].item() / 8, rel_tol=1e-12)
        assert ((s <= base * (1 + 1e-15)) & (s >= base / 8 * (1 - 1e-15))).all()
        assert math.isclose(b, 0.1 * math.log(8) + 1 if kind == "yarn" else 1.0, rel_tol=1e-6)
    assert pa.rope_inv_freq(64, scaling="yarn", factor=4, attn_factor=1.5, device="cpu")[1] == 1.5
    with pytest.raises(ValueError):
        pa.rope_inv_freq(64, scaling="other")
    with pytest.raises(ValueError):
        pa.rope_inv_freq(63)
    for bad in (dict(theta=0.0), dict(theta=float("inf")), dict(scaling="linear", factor=0.0),
                dict(scaling="llama3", low_freq_factor=4.0), dict(scaling="yarn", beta_slow=40.0)):
        with pytest.raises(pa.PagedAttnError):
            pa.rope_inv_freq(64, device="cpu", **bad)


def test_python_argument_checks(lib):
    torch = pytest.importorskip("torch")
    import long_context_paged_gb300 as pa
    x = torch.zeros(2, 16, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):  # not on a CUDA device
        pa.rope_append_paged(x, x, x, x, x, x, x, x)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        pa.paged_step_plan(i, i, i, i, i, 4, total_rows=2)
    with pytest.raises(TypeError):
        pa.paged_release(i.float(), i, i, i, i, 4)


def test_score_options(lib):
    """Options are checked before any CUDA call, for both attention calls; NULL options and an empty
    batch pass."""
    import long_context_paged_gb300 as pa
    good = pa.Dims(*pa.DEFAULT_DIMS)
    nan = float("nan")

    def both(softcap=0.0, window=0, max_prefix=0, prefix=0, batch=1):
        o = ctypes.byref(pa.ScoreOpts(softcap, 0, window, prefix, max_prefix, 0))
        # null q: refused too, so only an option error can be told apart by the empty batch's OK
        d = lib.attn_decode_paged_score(good, None, None, None, 1, None, 1, None, batch, 16, 1.0, 0, None,
                                        None, None, 0, None, None, None, o)
        p = lib.attn_prefill_chunk_score(good, None, None, 1, None, None, 1, None, 1, None, batch, 1, 16,
                                         1.0, None, None, None, 0, None, None, None, o)
        assert d == p
        return d

    assert both(batch=0) == OK and both() == INVALID     # null pointers
    assert both(softcap=30.0, window=5, max_prefix=131072, batch=0) == OK
    for bad in (dict(softcap=-1.0), dict(softcap=nan), dict(softcap=float("inf")), dict(softcap=1e-9),
                dict(window=-1), dict(max_prefix=-1), dict(max_prefix=131073)):
        assert both(batch=0, **bad) == INVALID, bad
    bad_cap = pa.LaunchOpts(-1)
    assert lib.attn_decode_paged_score(good, None, None, None, 1, None, 1, None, 0, 16, 1.0, 0, None, None,
                                       None, 0, None, None, ctypes.byref(bad_cap), None) == INVALID
    assert lib.attn_prefill_chunk_score(pa.Dims(16, 4, 128, 16), None, None, 1, None, None, 1, None, 1, None,
                                        1, 1, 16, 1.0, None, None, None, 0, None, None, None, None) == UNSUPPORTED


def test_fast_path_takes_nothing_without_a_gpu(lib):
    """Whatever it is given, the compiled path answers False, never an exception: the binding's own
    checks name the error."""
    import torch

    import long_context_paged_gb300 as pa
    fast = pa._FAST
    assert fast is not None, "the fast path was not built"
    t = torch.zeros(4, dtype=torch.int32)
    for f in (fast.decode, fast.prefill, fast.rope, fast.step_plan, fast.release):
        for n in range(24):
            for x in (None, t, 1, -1, 1 << 70, 0.5, "x", (16, 8, 128, 16)):
                assert f(*[x] * n) is False


def test_release_of_a_table_past_32_bit_counts(lib):
    for batch, stride, want in ((64, 1 << 25, UNSUPPORTED), (4096, 1 << 19, UNSUPPORTED)):
        assert lib.paged_release(A, A, batch, A, stride, A, 8, A, 64, A, None, None) == want
