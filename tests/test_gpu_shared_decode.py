"""attn_decode_paged_shared against the fp64 definition of the plain decode.

Tolerance: the weights are rounded to bf16 before they meet V (2^-8 of each at most, so 2^-8 of the
mean of |v| under the weights, which the oracle gives on |V|), fp32 sums and scores (6 * 2^-13, as for
the decode with options: |v| < 6), and one rounding of the output, 2^-8 of it. The log-sum-exp is of
unrounded weights: 2^-13 + 2^-23 |lse|.
"""
import numpy as np
import pytest
import torch

import oracle
from oracle import as_f64
from tests.helpers import bits

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5


def dev(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


class Inputs:
    """groups: list of (shared pages, [keys of each row]); rows in no group behind them. Slots that no
    row holds are NaN, entries past a row's pages -1."""

    def __init__(self, groups, alone=(), hkv=8, seed=0, qscale=1.0, extra=3):
        g = torch.Generator().manual_seed(seed)
        self.hkv, self.dims = hkv, (2 * hkv, hkv, 128, 16)
        self.lens = [n for _, rows in groups for n in rows] + list(alone)
        self.cu = np.cumsum([0] + [len(rows) for _, rows in groups])
        self.shared = [s for s, _ in groups]
        need = [s for s, _ in groups] + [max(-(-n // 16) - s, 0) if n >= 16 * s else -(-n // 16)
                                         for s, rows in groups for n in rows] + [-(-n // 16) for n in alone]
        self.pages = sum(need) + 2
        perm, at = torch.randperm(self.pages, generator=g).tolist(), 0
        stride = max([1] + [-(-n // 16) for n in self.lens]) + extra
        self.table = np.full((len(self.lens), stride), -1)
        self.k = torch.full((self.pages, 16, hkv, 128), float("nan"))
        self.v = self.k.clone()
        r = 0

        def fill(page, n):
            self.k[page, :n] = torch.randn(n, hkv, 128, generator=g)
            self.v[page, :n] = torch.randn(n, hkv, 128, generator=g).clamp(-5.9, 5.9)

        for s, rows in list(groups) + [(0, [n]) for n in alone]:
            common = perm[at:at + s]
            at += s
            for p in common:
                fill(p, 16)
            for n in rows:
                j = 0
                if n >= 16 * s:
                    self.table[r, :s] = common
                    j = s
                for j in range(j, -(-n // 16)):
                    self.table[r, j] = perm[at]
                    fill(perm[at], min(16, n - 16 * j))
                    at += 1
                r += 1
        self.k, self.v = self.k.to(torch.bfloat16).cuda(), self.v.to(torch.bfloat16).cuda()
        self.q = (torch.randn(len(self.lens), 2 * hkv, 128, generator=g) * qscale).to(torch.bfloat16).cuda()
        self.most = max([len(rows) for _, rows in groups] + [0])

    def call(self, pa, **kw):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        kw.setdefault("max_group_rows", self.most)
        kw.setdefault("status", status)
        out = pa.attn_decode_paged_shared(self.q, self.k, self.v, dev(self.table), dev(self.lens), dev(self.cu),
                                          dev(self.shared), max(self.lens), SCALE, dims=self.dims, **kw)
        torch.cuda.synchronize()
        self.flags = pa.read_device_status(kw["status"])
        return out

    def reference(self):
        args = bits(self.q), bits(self.k), bits(self.v), self.table, np.array(self.lens), SCALE
        o, l = oracle.decode(*args)
        mag, _ = oracle.decode(args[0], args[1], bits(self.v.abs()), *args[3:])
        return np.asarray(o), np.asarray(l), np.asarray(mag)

    def check(self, pa, flags=0, **kw):
        out, lse = self.call(pa, **kw)
        assert self.flags == flags
        self.close(out, lse)
        return out, lse

    def close(self, out, lse):
        ref, ref_l, mag = self.reference()
        o, l = as_f64(bits(out)), lse.cpu().numpy().astype(np.float64)
        bad = ~(np.abs(o - ref) <= 2.0 ** -8 * (np.abs(ref) + mag) + 6 * 2.0 ** -13)
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4], o[bad][:4], ref[bad][:4])
        inf = np.isneginf(ref_l)
        assert np.array_equal(np.isneginf(l), inf) and not o[inf].any()
        d = np.abs(l[~inf] - ref_l[~inf]) - 2.0 ** -23 * np.abs(ref_l[~inf])
        assert d.size == 0 or d.max() <= 2.0 ** -13, d.max()


@pytest.mark.parametrize("hkv", [8, 4, 2, 1])
def test_one_group(cuda_lib, hkv):
    Inputs([(3, [49, 60, 48, 64, 65])], hkv=hkv).check(cuda_lib)


@pytest.mark.parametrize("groups,alone", [
    ([], [1]), ([], [0]), ([], [1, 16, 17, 128, 129, 400]),
    ([(0, [5, 20])], []),                                   # nothing shared
    ([(1, [16])], []), ([(1, [17, 16, 16])], []),           # the shared page alone
    ([(8, [128, 129, 257, 300])], []), ([(9, [145, 144])], [3]),
    ([(20, [321, 0, 400, 0])], []),                         # beams not in use
    ([(20, [0, 0])], [7]),                                  # none in use
    ([(20, [100, 333, 319, 320])], []),                     # rows shorter than the shared pages
    ([(4, [64 + i for i in range(1, 9)]), (0, []), (2, [40] * 3), (30, [481, 500])], [0, 77]),
    ([(5, [81 + (i * 7) % 50 for i in range(64)])], []),
    ([(5, [81 + (i * 7) % 50 for i in range(65)])], []),
    ([(17, [300 - (i % 3) for i in range(131)])], [9]),
    ([(3, [50])] * 40, []),
])
def test_groups(cuda_lib, groups, alone):
    x = Inputs(groups, alone, seed=len(groups) + len(alone))
    # (more shared pages than the table has: flagged, and nothing is shared)
    x.check(cuda_lib, flags=2 if max(x.shared, default=0) > x.table.shape[1] else 0)


def test_long_prefixes_and_peaked_scores(cuda_lib):
    Inputs([(300, [4801, 4900, 4816, 5003]), (70, [1121, 1200])], [2500], seed=4, qscale=6.0).check(cuda_lib)
    Inputs([(1100, [17601, 17700])], hkv=1, seed=5, qscale=3.0).check(cuda_lib)


def test_matches_the_plain_decode_on_random_batches(cuda_lib):
    rng = np.random.default_rng(3)
    for seed in range(6):
        groups = []
        for _ in range(rng.integers(1, 9)):
            s = int(rng.integers(0, 40))
            groups.append((s, [int(16 * s + rng.integers(0, 200)) if rng.random() < 0.9 else 0
                               for _ in range(rng.integers(1, 20))]))
        Inputs(groups, [int(n) for n in rng.integers(0, 700, 3)], hkv=int(rng.choice([8, 4, 2, 1])), seed=seed).check(cuda_lib)


def test_non_finite_keys_and_values(cuda_lib):
    """A NaN in a row's own page moves that row alone; one in a shared page all rows that see it; an
    infinite score of one sign takes all the weight or none."""
    inp = Inputs([(4, [70, 90, 100])], [40], seed=8)
    clean, _ = inp.call(cuda_lib)
    page = int(inp.table[1, 5])
    inp.v[page, 3, 2, 7] = float("nan")
    out, _ = inp.call(cuda_lib)
    assert torch.isnan(out[1, 4:6, 7]).all()
    out[1, 4:6, 7] = clean[1, 4:6, 7]
    assert torch.equal(out, clean)
    inp.v[page, 3, 2, 7] = 0.0
    clean, clean_l = inp.call(cuda_lib)
    inp.k[int(inp.table[0, 1]), 9, 1] = float("nan")
    out, lse = inp.call(cuda_lib)
    assert torch.isnan(out[:3, 2:4]).all() and torch.isnan(lse[:3, 2:4]).all()
    out[:3, 2:4] = clean[:3, 2:4]
    assert torch.equal(out, clean)
    # every score of one row is -inf: nothing is left
    inp = Inputs([(2, [33, 40])], seed=9)
    inp.k[:] = float("inf")
    inp.q[0] = -inp.q[0].abs().clamp(min=0.01)
    inp.q[1] = 0.01
    out, lse = inp.call(cuda_lib)
    assert not out[0].any() and torch.isneginf(lse[0]).all() and torch.isnan(out[1]).all()


def test_pages_and_lengths_that_do_not_fit(cuda_lib):
    inp = Inputs([(4, [70, 90])], [40], seed=2)
    good = inp.table.copy()
    for r, j in ((0, 2), (1, 5), (2, 0)):
        inp.table = good.copy()
        inp.table[r, j] = inp.pages
        inp.k.nan_to_num_(0.0)
        inp.v.nan_to_num_(0.0)
        inp.call(cuda_lib)
        assert inp.flags == 1, (r, j)
    inp.table = good
    lens = inp.lens
    for bad in ([70, -3, 40], [70, 90, 16 * good.shape[1] + 1]):
        inp.lens = bad
        inp.table = np.maximum(good, 0)
        inp.call(cuda_lib)
        assert inp.flags == 2
    inp.table, inp.lens = good, lens
    for cu, shared, most in (([0, 3], [4], 2), ([-1, 2], [4], 3), ([2, 0], [4], 3), ([0, 4], [4], 4),
                             ([0, 2], [-1], 2), ([0, 2], [good.shape[1] + 1], 2)):
        inp.cu, inp.shared = cu, shared
        inp.check(cuda_lib, flags=2, max_group_rows=most)


def test_streams_graphs_and_workspaces(cuda_lib):
    pa = cuda_lib
    a = Inputs([(6, [100, 111, 97]), (2, [33, 60])], [12], seed=1)
    b = Inputs([(30, [500, 490])], [3], seed=2)
    want = [x.check(pa) for x in (a, b)]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for x, w in zip((a, b), want):
        got = x.call(pa, stream=st)
        assert torch.equal(got[0], w[0]) and torch.equal(got[1], w[1])
    # two captured calls that share a workspace, replayed in turn
    n = max(pa.decode_shared_workspace_size(len(x.lens), len(x.shared), x.most) for x in (a, b))
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    graphs = []
    for x in (a, b):
        args = (x.q, x.k, x.v, dev(x.table), dev(x.lens), dev(x.cu), dev(x.shared), max(x.lens), SCALE)
        out, lse = torch.zeros_like(x.q), torch.zeros(x.q.shape[:2], device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pa.attn_decode_paged_shared(*args, max_group_rows=x.most, out=out, lse=lse, workspace=ws)
        graphs.append((g, out, lse, args))
    for i in (0, 1, 1, 0, 1):
        g, out, lse, _ = graphs[i]
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])


def test_rows_before_the_first_group_and_between(cuda_lib):
    x = Inputs([(3, [50, 60, 48]), (12, [200] * 20)], [33, 150], seed=11)
    x.table, x.lens = np.roll(x.table, 2, 0), x.lens[-2:] + x.lens[:-2]
    x.q = x.q.roll(2, 0).contiguous()
    x.cu = x.cu + 2
    x.check(cuda_lib)
    # a group that vouches for nothing, between two that do
    y = Inputs([(3, [50, 60, 48]), (0, [20, 100]), (4, [64, 77])], seed=12)
    y.check(cuda_lib)
    y.cu, y.shared = [0, 3, 3, 5, 5, 7], [3, 2, 0, 9, 4]   # empty groups among them
    y.check(cuda_lib)


def test_calls_side_by_side(cuda_lib):
    """Two streams at once, each call with scratch of its own."""
    xs = [Inputs([(40, [700, 650, 777])], [100], seed=s) for s in (1, 2)]
    want = [x.check(cuda_lib) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    args = [(x.q, x.k, x.v, dev(x.table), dev(x.lens), dev(x.cu), dev(x.shared), max(x.lens), SCALE) for x in xs]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for st, a in zip(streams, args):
            got.append(cuda_lib.attn_decode_paged_shared(*a, max_group_rows=3, stream=st))
    torch.cuda.synchronize()
    for i, (o, l) in enumerate(got):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(l, want[i % 2][1])


def test_a_table_past_2_gib_of_entries_and_far_pages(cuda_lib):
    """A row's entries and a page's keys at offsets past 32 bits."""
    x = Inputs([(2, [40, 50])], [20], hkv=8, seed=13)
    stride = 1 << 27
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    table = torch.zeros(3, stride, dtype=torch.int32, device="cuda")      # row 2 starts at 2^30 bytes
    table[:, :x.table.shape[1]] = dev(x.table)
    far = 70_000                                                          # 2.3 GB into the pool
    k = torch.zeros(far + x.pages, 16, 8, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    k[far:], v[far:] = x.k, x.v
    table[table > 0] += far
    zero = [(r, j) for r in range(3) for j in range(x.table.shape[1]) if x.table[r, j] == 0]
    for r, j in zero:
        table[r, j] = far
    table[table < 0] = -1
    with pytest.raises(cuda_lib.PagedAttnError):                          # (a stride the lengths' type does not hold)
        cuda_lib.attn_decode_paged_shared(x.q, k, v, table, dev(x.lens), dev(x.cu), dev(x.shared), 64, SCALE)
    table = table[:, :stride - 64].contiguous()
    out, lse = cuda_lib.attn_decode_paged_shared(x.q, k, v, table, dev(x.lens), dev(x.cu), dev(x.shared), 64, SCALE)
    torch.cuda.synchronize()
    x.close(out, lse)


def test_a_larger_bound_gives_the_same_bits(cuda_lib):
    """The bound sizes the workspace; up to 512 segments are planned by every CTA, more in a launch of their own."""
    for x in (Inputs([(6, [100, 111, 97] * 30), (2, [33, 60]), (17, [300] * 70)], [12, 0, 700] * 40, seed=23),
              Inputs([(2, [40, 33])] * 150 + [(9, [150] * 66)], [30] * 60, hkv=2, seed=24),
              Inputs([(6, [100, 111, 97]), (2, [33, 60]), (0, []), (9, [150] * 8)], [12, 0, 700], seed=21),
              Inputs([(3, [50, 60])] * 90 + [(200, [3300, 3210])], [5] * 3, hkv=1, seed=22)):
        few = x.check(cuda_lib)
        many = x.call(cuda_lib, max_group_rows=128)
        assert x.flags == 0
        assert torch.equal(few[0], many[0]) and torch.equal(few[1], many[1])


def test_the_same_bits_every_time(cuda_lib):
    x = Inputs([(40, [700 + 5 * i for i in range(9)]), (3, [60] * 4)], [300], seed=6)
    first = x.call(cuda_lib)
    for _ in range(5):
        again = x.call(cuda_lib)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_no_lse_empty_batch_and_given_outputs(cuda_lib):
    x = Inputs([(2, [33, 40])], seed=3)
    want, _ = x.check(cuda_lib)
    out = torch.zeros_like(x.q)
    got, lse = x.call(cuda_lib, out=out, want_lse=False)
    assert got is out and lse is None and torch.equal(out, want)
    got, lse = cuda_lib.attn_decode_paged_shared(x.q[:0], x.k, x.v, dev(x.table), dev([]), dev([0]), dev([]), 1, SCALE)
    assert got.shape[0] == 0


@pytest.mark.parametrize("rows", [19, 20, 76, 77])
def test_rows_on_either_side_of_the_merge_s_widths(cuda_lib, rows):
    """8 KV heads make 19 slices of a GB300: up to 19 rows, up to 76 and more are merged by CTAs of three sizes."""
    one = rows // 2
    Inputs([(40, [640 + (i * 37) % 400 for i in range(one)]), (3, [48 + (i * 53) % 300 for i in range(one)])],
           [200] * (rows - 2 * one), seed=rows).check(cuda_lib)


def test_many_results_of_many_rows(cuda_lib):
    """One KV head: 152 slices, so 620 rows are merged by the smallest CTAs, 100 of them from dozens of results."""
    Inputs([(1250, [20000 + 3 * i for i in range(100)])], [i % 40 for i in range(520)], hkv=1, seed=5).check(cuda_lib)
