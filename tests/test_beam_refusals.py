"""Host-side refusals of the beam-search calls (no GPU: each is returned before any CUDA call; the
pointers are fake, aligned addresses and never read), and the oracle of the fork and the selection on
small cases worked by hand."""
import ctypes

import numpy as np
import pytest

INVALID, UNSUPPORTED, SMALL, OK = 1, 2, 3, 0
A = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 2)
NAN = float("nan")


@pytest.fixture(scope="module")
def lib():
    from long_context_paged_gb300 import build as b
    b.build()
    import long_context_paged_gb300 as pa
    return pa.load()


def test_beam_select(lib):
    def call(x=A, kind=0, stride=100, n=2, w=4, v=100, s=A, live=None, k=4, eos=-1, o=A, p=A, t=A, l=A, ws=A,
             size=1 << 30):
        return lib.beam_select(x, kind, stride, n, w, v, s, live, k, eos, o, p, t, l, ws, size, None)
    for bad in (dict(n=-1), dict(w=0), dict(v=0), dict(k=0), dict(k=-1), dict(stride=99), dict(eos=-2),
                dict(eos=100), dict(kind=2), dict(kind=-1), dict(x=ODD, kind=1), dict(ws=ODD),
                dict(x=ctypes.c_void_p((1 << 20) + 1)), dict(k=3, o=A, s=A), dict(k=5, live=A, l=A, o=None)):
        assert call(**bad) == INVALID, bad
    for name in ("x", "s", "o", "p", "t", "l"):
        assert call(**{name: None}) == INVALID, name
    for bad in (dict(w=65), dict(k=65), dict(w=64, v=1 << 26, stride=1 << 26), dict(n=1 << 20, w=2)):
        assert call(**bad) == UNSUPPORTED, bad
    other = ctypes.c_void_p(1 << 21)
    assert call(ws=None, o=other) == SMALL and call(size=0, o=other) == SMALL
    assert call(size=lib.pa_beam_workspace_size(2, 4, 100, 4) - 1, o=other) == SMALL
    assert call(n=0, x=None) == OK
    assert lib.pa_beam_workspace_size(2, 65, 100, 4) == 0 and lib.pa_beam_workspace_size(2, 4, 100, 0) == 0


def test_fork(lib):
    def call(pa=A, sl=A, g=2, w=4, bt=A, stride=8, free=A, cap=8, cnt=A, pages=64, co=A, so=A, c=A, sh=A, ws=A,
             size=1 << 20):
        return lib.paged_fork(pa, sl, g, w, bt, stride, free, cap, cnt, pages, co, so, c, sh, ws, size, None, None)
    for bad in (dict(g=-1), dict(w=0), dict(stride=0), dict(stride=1 << 28), dict(cap=-1), dict(pages=0),
                dict(ws=ODD)):
        assert call(**bad) == INVALID, bad
    for name in ("pa", "sl", "bt", "free", "cnt", "co", "so", "c", "sh"):
        assert call(**{name: None}) == INVALID, name
    assert call(w=65) == UNSUPPORTED and call(g=1025) == UNSUPPORTED
    assert call(ws=None) == SMALL and call(size=64) == SMALL
    assert call(g=0, pa=None, bt=None) == OK
    assert lib.pa_fork_workspace_size(2, 65, 8) == 0


def test_copy_pages(lib):
    import long_context_paged_gb300 as pa
    good = pa.Dims(*pa.DEFAULT_DIMS)

    def call(dims=good, c=A, rows=2, pools=(1 << 20, 1 << 21), n=None, pages=4):
        p = (ctypes.c_void_p * max(1, len(pools)))(*pools)
        return lib.paged_copy_pages(dims, c, rows, p, len(pools) if n is None else n, pages, None, None)
    assert call(dims=pa.Dims(16, 8, 64, 16)) == UNSUPPORTED
    for bad in (dict(rows=-1), dict(n=-1), dict(pages=0), dict(c=None), dict(pools=(1 << 20, None)),
                dict(pools=((1 << 20) + 8,))):
        assert call(**bad) == INVALID, bad
    assert call(rows=0, c=None) == OK and call(pools=()) == OK


def test_decode_shared(lib):
    import long_context_paged_gb300 as pa

    def call(dims=(16, 8, 128, 16), q=A, k=A, v=A, pages=64, bt=A, stride=8, sl=A, b=4, cu=A, sh=A, g=1, most=4,
             bound=128, scale=0.1, out=A, ws=None, size=0):
        return lib.attn_decode_paged_shared(pa.Dims(*dims), q, k, v, pages, bt, stride, sl, b, cu, sh, g, most, bound,
                                            scale, out, None, ws, size, None, None)
    assert call(dims=(16, 4, 128, 16)) == UNSUPPORTED
    for bad in (dict(b=-1), dict(g=-1), dict(most=-1), dict(pages=0), dict(stride=0), dict(stride=1 << 28),
                dict(bound=-1), dict(bound=131073), dict(scale=0.0), dict(scale=-1.0), dict(scale=NAN),
                dict(scale=float("inf"))):
        assert call(**bad) == INVALID, bad
    for name in ("q", "k", "v", "bt", "sl", "cu", "sh", "out"):
        assert call(**{name: None}) == INVALID, name
    for name in ("q", "k", "v", "out"):
        assert call(**{name: ctypes.c_void_p((1 << 20) + 8)}) == INVALID, name
    for bad in (dict(b=4097), dict(g=4097), dict(pages=1 << 27)):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(b=0, q=None) == OK


def test_oracle_fork_by_hand():
    from oracle import beam as O
    # two beams of 20 and 18 tokens share page 3; beam 1 has the only children
    f = O.fork([[1, 1]], [20, 18], [[3, 4, -1], [3, 5, -1]], [8, 9, 0, 0], 2, 10)
    assert f["lens"] == [18, 18] and f["table"].tolist() == [[3, 5, -1], [3, 9, -1]]
    assert f["copies"] == [(-1, -1, 0), (5, 9, 2)] and f["shared"] == [1]
    assert f["count"] == 2 and f["free"].tolist() == [8, 4, 0, 0] and not f["flags"]
    # filled pages are shared without a copy
    f = O.fork([[0, 0, -1]], [32, 0, 5], [[1, 2], [-1, -1], [7, -1]], [0, 0, 0], 0, 10)
    assert f["table"].tolist() == [[1, 2], [1, 2], [-1, -1]] and f["shared"] == [2]
    assert f["free"][:f["count"]].tolist() == [7]
    # no page for the copy: nothing changes
    f = O.fork([[0, 0]], [5, 0], [[1], [-1]], [0], 0, 10)
    assert f["flags"] == {"no_pages"} and f["table"].tolist() == [[1], [-1]] and f["lens"] == [5, 0]


def test_oracle_select_by_hand():
    from oracle import beam as O
    x = np.log(np.array([[[0.5, 0.25, 0.25], [0.1, 0.1, 0.8]]]))
    (s, p, t, live), _ = O.select(x, np.log(np.array([[0.5, 0.5]])), 4, np.array([[1, 1]]), eos=2)
    assert np.allclose(np.exp(s), [[0.4, 0.25, 0.125, 0.125]])
    assert p.tolist() == [[1, 0, 0, 0]] and t.tolist() == [[2, 0, 1, 2]] and live.tolist() == [[0, 1, 1, 0]]
    (s, p, t, live), _ = O.select(x, np.log(np.array([[0.5, 0.5]])), 3, np.array([[0, 0]]), eos=2)
    assert p.tolist() == [[0, 1, -1]] and t.tolist() == [[2, 2, -1]] and live.tolist() == [[0, 0, 0]]
