"""The binding's two paths: the compiled one makes the same launches as the Python one (results bit
for bit the same, on another stream and captured too), takes only what is plainly right, and leaves
every other call to the Python checks."""
import pytest
import torch

pytestmark = pytest.mark.gpu

HQ, HKV, D = 4, 2, 128
DIMS = (HQ, HKV, D, 16)
LENS = [1, 16, 37, 300, 2100]
NEW = [1, 16, 5, 44, 100]
PAGES = 200


class Calls:
    """The five calls over one small batch, each returning the tensors that it wrote."""

    def __init__(self, pa):
        g = torch.Generator().manual_seed(29)
        bf = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
        self.pa = pa
        self.k, self.v = bf(PAGES, 16, HKV, D), bf(PAGES, 16, HKV, D)
        width = (max(LENS) + 15) // 16
        perm = torch.randperm(PAGES, generator=g)
        table, at = torch.zeros(len(LENS), width, dtype=torch.int32), 0
        for b, n in enumerate(LENS):
            used = (n + 15) // 16
            table[b, :used] = perm[at:at + used].int()
            at += used
        self.table, self.lens = table.cuda(), i32(LENS)
        self.qd, self.T = bf(len(LENS), HQ, D), sum(NEW)
        self.qp = bf(self.T, HQ, D)
        self.kn, self.vn = bf(self.T, HKV, D), bf(self.T, HKV, D)
        self.cu = i32([0] + [sum(NEW[:b + 1]) for b in range(len(NEW))])
        self.pos = i32([n - m + j for n, m in zip(LENS, NEW) for j in range(m)])
        self.slots = torch.randperm(PAGES * 16, generator=g)[:self.T].cuda()
        self.slopes = torch.rand(HQ, generator=g).cuda()
        self.prefix, self.start = i32([0, 3, 20, 40, 64]), i32([0, 2, 30, 0, 2000])
        self.freq = pa.rope_inv_freq(D)[0]
        self.gamma = torch.rand(D, generator=g).cuda()
        self.cached, self.new = i32([0, 15, 16, 40, 0]), i32([1, 2, 0, 30, 5])
        self.free, self.count = torch.randperm(PAGES, generator=g).int().cuda(), i32([PAGES])
        self.begin, self.end = i32([0, 0, 1, 2, 0]), i32([1, 1, 1, 9, 40])

    def decode(self, **kw):
        a = dict(out=torch.zeros_like(self.qd), lse=torch.zeros(len(LENS), HQ, device="cuda"), dims=DIMS)
        a.update(kw)
        return self.pa.attn_decode_paged(self.qd, self.k, self.v, self.table, self.lens, max(LENS),
                                         D ** -0.5, **a)

    def decode_score(self, **kw):
        return self.decode(softcap=20.0, alibi_slopes=self.slopes, window=50, prefix_lens=self.prefix,
                           max_prefix_len=64, row_start=self.start, **kw)

    def prefill(self, **kw):
        a = dict(out=torch.zeros_like(self.qp), lse=torch.zeros(self.T, HQ, device="cuda"), dims=DIMS)
        a.update(kw)
        return self.pa.attn_prefill_chunk(self.qp, self.cu, self.k, self.v, self.table, self.lens,
                                          max(NEW), max(LENS), D ** -0.5, **a)

    def prefill_score(self, **kw):
        return self.prefill(softcap=20.0, alibi_slopes=self.slopes, window=50, prefix_lens=self.prefix, **kw)

    def rope(self, **kw):
        k, v = self.k.clone(), self.v.clone()
        a = dict(interleaved=True, q_gamma=self.gamma, k_gamma=self.gamma, q_out=torch.zeros_like(self.qp),
                 dims=DIMS)
        a.update(kw)
        q = self.pa.rope_append_paged(self.qp, self.kn, self.vn, self.pos, self.slots, k, v, self.freq, **a)
        return q, k, v

    def plan(self, **kw):
        table, rows = torch.arange(40, dtype=torch.int32, device="cuda").view(5, 8).clone(), 40
        e = lambda n, t=torch.int32: torch.zeros(n, dtype=t, device="cuda")
        a = dict(total_rows=rows, free_count_out=e(1), cu_new_lens=e(6), seq_lens=e(5), positions=e(rows),
                 slot_map=e(rows, torch.int64))
        a.update(kw)
        return (table, *self.pa.paged_step_plan(self.cached, self.new, table, self.free, self.count,
                                                PAGES, **a))

    def release(self, **kw):
        table, free = self.table.clone(), torch.full((PAGES,), -1, dtype=torch.int32, device="cuda")
        a = dict(free_count_out=torch.zeros(1, dtype=torch.int32, device="cuda"))
        a.update(kw)
        n = self.pa.paged_release(self.begin, self.end, table, free, torch.zeros_like(self.count), PAGES, **a)
        return table, free, n


CALLS = {"decode": "decode", "decode_score": "decode", "prefill": "prefill", "prefill_score": "prefill",
         "rope": "rope", "plan": "step_plan", "release": "release"}


class Counting:
    """The fast path's module, with what each call returned."""

    def __init__(self, mod):
        self.mod, self.seen = mod, []

    def __getattr__(self, name):
        f = getattr(self.mod, name)

        def call(*args):
            self.seen.append((name, f(*args)))
            return self.seen[-1][1]
        return call


@pytest.fixture()
def fast(cuda_lib, monkeypatch):
    assert cuda_lib._FAST is not None, "the fast path was not built"
    f = Counting(cuda_lib._FAST)
    monkeypatch.setattr(cuda_lib, "_FAST", f)
    return f


def slow(pa, monkeypatch, fn, **kw):
    with monkeypatch.context() as m:
        m.setattr(pa, "_FAST", None)
        return fn(**kw)


def same(a, b):
    torch.cuda.synchronize()
    for x, y in zip(a, b, strict=True):
        assert x.dtype == y.dtype and x.shape == y.shape
        raw = {2: torch.int16, 4: torch.int32, 8: torch.int64}[x.element_size()]
        assert torch.equal(x.view(raw), y.view(raw))


@pytest.mark.parametrize("name", CALLS)
def test_same_results(cuda_lib, fast, monkeypatch, name):
    fn = getattr(Calls(cuda_lib), name)
    got = fn()
    assert fast.seen == [(CALLS[name], True)]
    same(got, slow(cuda_lib, monkeypatch, fn))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    more = dict(status=status, **({"max_ctas": 40} if "de" in name or "pre" in name else {}))
    same(fn(**more), slow(cuda_lib, monkeypatch, fn, **more))
    assert fast.seen[1:] == [(CALLS[name], True)] and int(status) == 0


@pytest.mark.parametrize("name", CALLS)
def test_other_stream_and_captured(cuda_lib, fast, monkeypatch, name):
    fn = getattr(Calls(cuda_lib), name)
    want = slow(cuda_lib, monkeypatch, fn)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):  # (the outputs' zeros are on this stream)
        got = fn(stream=st)
    same(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = fn()
    for _ in range(2):
        g.replay()
    same(got, want)
    assert fast.seen == [(CALLS[name], True)] * 2


@pytest.mark.parametrize("name", CALLS)
def test_anything_else_is_left_to_the_checks(cuda_lib, fast, name):
    c = Calls(cuda_lib)
    fn = getattr(c, name)
    out = {"decode": "out", "prefill": "out", "rope": "q_out", "step_plan": "seq_lens",
           "release": "free_count_out"}[CALLS[name]]
    like = {"decode": c.qd, "prefill": c.qp, "rope": c.qp, "step_plan": c.lens, "release": c.count}[CALLS[name]]
    for bad, error in ((like.cpu(), ValueError), (like.double(), TypeError), (like[:-1], ValueError),
                       (like.unsqueeze(0), ValueError),
                       (torch.stack([like, like], -1)[..., 0], None if like.numel() == 1 else ValueError),
                       ("x", TypeError)):
        if error is not None:
            with pytest.raises(error):
                fn(**{out: bad})
            assert fast.seen[-1] == (CALLS[name], False)
    if "dims" in fn.__code__.co_varnames or CALLS[name] in ("decode", "prefill", "rope"):
        for dims in ((4, 4, 128, 16), [4, 2, 128, 16], (4, 2, 64, 16)):
            if isinstance(dims, list):
                fn(dims=dims)  # (a list is served, by the slower path)
            else:
                with pytest.raises((cuda_lib.PagedAttnError, ValueError)):
                    fn(dims=dims)
            assert fast.seen[-1] == (CALLS[name], False)
    if CALLS[name] in ("decode", "prefill"):
        with pytest.raises(ValueError):
            fn(max_ctas=-1)
        assert fast.seen[-1] == (CALLS[name], False)


def test_a_code_of_the_library_is_raised_by_its_name(cuda_lib, fast):
    c = Calls(cuda_lib)
    for fn, call in ((c.decode, "attn_decode_paged_score"), (c.prefill, "attn_prefill_chunk_score")):
        with pytest.raises(cuda_lib.PagedAttnError, match=call):
            fn(window=-1)
    with pytest.raises(cuda_lib.PagedAttnError, match="rope_append_paged"):
        c.rope(eps=-1.0)
    assert [ok for _, ok in fast.seen] == [False] * 3


@pytest.mark.parametrize("name", ["decode", "decode_score", "prefill", "prefill_score", "rope"])
def test_outputs_and_workspaces_of_the_caller_or_not(cuda_lib, fast, monkeypatch, name):
    c = Calls(cuda_lib)
    fn, out = getattr(c, name), "q_out" if name == "rope" else "out"
    want = slow(cuda_lib, monkeypatch, fn)
    same(fn(**{out: None}), want)
    if name != "rope":
        same(fn(out=None, lse=None), want)
        assert fn(lse=None, want_lse=False)[1] is None
        size = {"decode": lambda: cuda_lib.decode_workspace_size(len(LENS), max(LENS), 0, DIMS),
                "prefill": lambda: cuda_lib.prefill_workspace_size(len(LENS), max(NEW), max(LENS), DIMS),
                "prefill_score": lambda: cuda_lib.prefill_score_workspace_size(len(LENS), c.T, DIMS)}
        n = size[CALLS[name] if name != "prefill_score" else name]()
        ws = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
        same(fn(workspace=ws), want)
        assert [ok for _, ok in fast.seen] == [True] * 4
        with pytest.raises(cuda_lib.PagedAttnError):
            fn(workspace=ws[:0])
        same(fn(workspace=torch.empty(n // 4 + 64, dtype=torch.int32, device="cuda")), want)
        assert [ok for _, ok in fast.seen[4:]] == [False] * 2  # (any tensor will do, by the slower path)
    else:
        assert [ok for _, ok in fast.seen] == [True]
