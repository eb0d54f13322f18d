"""paged_step_plan and paged_release against the sequential definition, value for value."""
import numpy as np
import pytest
import torch

from oracle import serving as S

pytestmark = pytest.mark.gpu


def dev(a, dtype=torch.int32):
    return torch.tensor(np.asarray(a), dtype=dtype, device="cuda")


def make(seed, B, lmax, new_max, free_share=1.0, pad=0, chunk_share=0.1):
    rng = np.random.default_rng(seed)
    cached = rng.integers(0, lmax, B)
    new = np.where(rng.random(B) < chunk_share, rng.integers(0, new_max + 1, B),
                   rng.integers(0, 2, B))
    held = -(-cached // 16)
    need = -(-(cached + new) // 16) - held
    stride = max(1, int((held + need).max())) if B else 1
    num_pages = int(held.sum() + need.sum()) + 7
    perm = rng.permutation(num_pages)
    table = np.full((B, stride), -1)
    at = 0
    for b in range(B):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
    free = perm[at:]
    count = int(min(len(free), round(free_share * need.sum())))
    return cached, new, table, free, count, num_pages, int(new.sum()) + pad


def run_plan(pa, cached, new, table, free, count, num_pages, rows, **kw):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    t = dev(table)
    got = pa.paged_step_plan(dev(cached), dev(new), t, dev(free), dev([count]), num_pages,
                             total_rows=rows, status=status, **kw)
    return got, t, pa.read_device_status(status)


BITS = {"page": 1, "length": 2, "no_pages": 16}


def check_plan(got, table, flags, want):
    assert np.array_equal(got.cu_new_lens.cpu().numpy(), want["cu"])
    assert np.array_equal(got.seq_lens.cpu().numpy(), want["seq_lens"])
    assert np.array_equal(got.positions.cpu().numpy(), want["positions"])
    assert np.array_equal(got.slot_map.cpu().numpy(), want["slots"])
    assert np.array_equal(table.cpu().numpy(), want["table"])
    assert got.free_count.item() == want["count"]
    assert flags == sum(BITS[f] for f in want["flags"])


@pytest.mark.parametrize("B,lmax,new_max,free_share,pad", [
    (1, 1, 1, 1.0, 0), (1, 40, 0, 1.0, 3), (1, 17, 4096, 1.0, 0), (3, 16, 33, 1.0, 1),
    (31, 5000, 4096, 1.0, 0), (32, 100, 100, 0.5, 9), (33, 33, 33, 0.0, 0),
    (1023, 300, 50, 1.0, 5), (1025, 300, 50, 0.7, 0), (4096, 200, 60, 1.0, 13),
    (4096, 100, 20, 0.31, 0), (4095, 17, 17, 0.9, 1),
])
def test_step_plan_matches_the_definition(cuda_lib, B, lmax, new_max, free_share, pad):
    a = make(B * 7 + lmax, B, lmax, new_max, free_share, pad)
    want = S.step_plan(*a)
    check_plan(*run_plan(cuda_lib, *a), want)


def test_step_plan_lengths_that_do_not_fit(cuda_lib):
    cached, new = [3, -1, 5, 60, 64, 0, 2**31 - 1, 7], [2, 4, -3, 5, 0, 64, 2, 2]
    table = np.arange(8 * 4).reshape(8, 4)
    free = np.arange(40, 60)
    a = (cached, new, table, free, 20, 64, 90)
    want = S.step_plan(*a)
    assert want["flags"] == {"length"}
    check_plan(*run_plan(cuda_lib, *a), want)


def test_step_plan_bad_pages_and_counts(cuda_lib):
    # a held page and a free page outside the pool; a free count past the list; too few rows
    table = np.array([[70, 0], [1, 0]])
    a = ([5, 16], [3, 20], table, np.array([2, 99, -4]), 7, 64, 20)
    want = S.step_plan(*a)
    assert want["flags"] == {"page", "length"}
    check_plan(*run_plan(cuda_lib, *a), want)
    a = ([5], [3], np.array([[2, 0]]), np.array([1]), -2, 64, 3)
    want = S.step_plan(*a)
    check_plan(*run_plan(cuda_lib, *a), want)


def test_step_plan_empty_batch_and_no_rows(cuda_lib):
    z = torch.zeros(0, dtype=torch.int32, device="cuda")
    p = cuda_lib.paged_step_plan(z, z, torch.zeros(0, 3, dtype=torch.int32, device="cuda"),
                                 dev([4, 5]), dev([2]), 9, total_rows=3)
    assert p.cu_new_lens.tolist() == [0] and p.free_count.tolist() == [2]
    assert p.positions.tolist() == [0, 0, 0] and p.slot_map.tolist() == [-1, -1, -1]
    p = cuda_lib.paged_step_plan(dev([16]), dev([0]), dev([[3]]), dev([4]), dev([1]), 9, total_rows=0)
    assert p.seq_lens.tolist() == [16] and p.free_count.tolist() == [1]


@pytest.mark.parametrize("B", [5, 4000])
def test_step_plan_in_place_and_replayed_from_a_graph(cuda_lib, B):
    """seq_lens in cached_lens' own buffer and the free count in place: a captured step replays as a
    decode loop that allocates a page whenever a request crosses a page boundary."""
    rng = np.random.default_rng(B)
    cached = rng.integers(0, 40, B)
    steps = 20
    held = -(-cached // 16)
    stride, num_pages = 4, int(held.sum()) + 2 * B + 3
    perm = rng.permutation(num_pages)
    table = np.full((B, stride), -1)
    at = 0
    for b in range(B):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
    free = perm[at:]
    lens, new, t, f, n = dev(cached), dev(np.ones(B)), dev(table), dev(free), dev([len(free)])
    pos = torch.empty(B, dtype=torch.int32, device="cuda")
    slots = torch.empty(B, dtype=torch.int64, device="cuda")
    cu = torch.empty(B + 1, dtype=torch.int32, device="cuda")

    def step():
        cuda_lib.paged_step_plan(lens, new, t, f, n, num_pages, total_rows=B, free_count_out=n,
                                 seq_lens=lens, positions=pos, slot_map=slots, cu_new_lens=cu)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    want = dict(seq_lens=cached, table=table, count=len(free))
    for _ in range(steps):
        want = S.step_plan(want["seq_lens"], np.ones(B, int), want["table"], free, want["count"],
                           num_pages, B)
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(slots.cpu().numpy(), want["slots"])
        assert np.array_equal(lens.cpu().numpy(), want["seq_lens"])
    assert np.array_equal(t.cpu().numpy(), want["table"]) and n.item() == want["count"]
    assert len(set(slots.tolist())) == B


@pytest.mark.parametrize("B,stride,seed", [(1, 1, 0), (1, 700, 1), (7, 130, 2), (32, 33, 3),
                                           (33, 129, 4), (511, 64, 5), (4096, 20, 6)])
def test_release_matches_the_definition(cuda_lib, B, stride, seed):
    rng = np.random.default_rng(seed)
    num_pages = B * stride + 9
    table = rng.permutation(num_pages)[:B * stride].reshape(B, stride)
    table = np.where(rng.random((B, stride)) < 0.1, -1, table)
    begin = rng.integers(0, stride + 1, B) * rng.integers(0, 2, B)
    end = np.where(rng.random(B) < 0.3, 0, rng.integers(0, stride + 1, B))  # some ranges are empty
    free = np.full(num_pages + 3, 77)
    want_t, want_f, want_n, flags = S.release(begin, end, table, free, 3, num_pages)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    t, f = dev(table), dev(free)
    n = cuda_lib.paged_release(dev(begin), dev(end), t, f, dev([3]), num_pages, status=status)
    assert np.array_equal(t.cpu().numpy(), want_t) and np.array_equal(f.cpu().numpy(), want_f)
    assert n.item() == want_n and cuda_lib.read_device_status(status) == 0


def test_release_flags(cuda_lib):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    # a range past its row, a page outside the pool (dropped from the table, not pushed)
    t, f = dev([[1, 99, 2], [3, 4, 5]]), dev(np.zeros(8))
    n = cuda_lib.paged_release(dev([-2, 1]), dev([3, 9]), t, f, dev([0]), 50, status=status)
    assert t.tolist() == [[-1, -1, -1], [3, -1, -1]] and n.item() == 4
    assert f[:4].tolist() == [1, 2, 4, 5] and cuda_lib.read_device_status(status) == 1 + 2
    # no room: nothing is released
    t, f = dev([[1, 2, 3]]), dev([7, 0])
    n = cuda_lib.paged_release(dev([0]), dev([3]), t, f, dev([1]), 50, status=status)
    assert t.tolist() == [[1, 2, 3]] and f.tolist() == [7, 0] and n.item() == 1
    assert cuda_lib.read_device_status(status) == 2


def test_plan_and_release_on_another_stream(cuda_lib):
    a = make(9, 600, 500, 60)
    want = S.step_plan(*a)
    st = torch.cuda.Stream()
    args = dev(a[0]), dev(a[1]), dev(a[2]), dev(a[3]), dev([a[4]])
    st.wait_stream(torch.cuda.current_stream())
    p = cuda_lib.paged_step_plan(*args, a[5], total_rows=a[6], stream=st)
    st.synchronize()
    assert np.array_equal(p.slot_map.cpu().numpy(), want["slots"])
    zero = dev(np.zeros(600))
    full = dev(-(-want["seq_lens"] // 16))
    room = torch.cat([args[3], dev(np.zeros(a[5]))])
    torch.cuda.synchronize()
    n = cuda_lib.paged_release(zero, full, args[2], room, p.free_count, a[5], stream=st)
    st.synchronize()
    # every page is free again, once
    assert n.item() == a[4] + int((-(-a[0] // 16)).sum())
    assert len(set(room[:n.item()].tolist())) == n.item()


@pytest.mark.parametrize("B", [33, 129, 257, 4096])
def test_release_with_ctas_that_have_nothing_to_count(cuda_lib, B):
    """Only the last request gives pages back: the other CTAs of the cluster are at the exchange of
    their counts at once. Calls in a row, each launched during the tail of the one before."""
    table = np.full((B, 40), -1)
    table[-1] = np.arange(40)
    begin, end = np.zeros(B), np.zeros(B)
    end[-1] = 40
    b, e, t = dev(begin), dev(end), dev(table)
    runs = [(t.clone(), dev(np.full(50, 7)), dev([3])) for _ in range(50)]
    torch.cuda.synchronize()
    for ti, f, n in runs:
        cuda_lib.paged_release(b, e, ti, f, n, 64, free_count_out=n)
    want_t, want_f, want_n, _ = S.release(begin, end, table, np.full(50, 7), 3, 64)
    for ti, f, n in runs:
        assert n.item() == want_n and np.array_equal(f.cpu().numpy(), want_f)
        assert np.array_equal(ti.cpu().numpy(), want_t)


@pytest.mark.parametrize("B", [1, 8, 200])
def test_release_of_ranges_that_begin_past_their_row(cuda_lib, B):
    """A begin past the row, up to the largest int32, is an empty range, whatever its end."""
    top = 2**31 - 1
    begin = np.resize([top, top - 30, top - 31, top - 127, 40, 41, 0, top], B)
    end = np.resize([0, top, 40, -5, 40, 40, 40, -2**31], B)
    table = np.arange(B * 40).reshape(B, 40)
    free = np.full(B * 40 + 5, 77)
    want_t, want_f, want_n, flags = S.release(begin, end, table, free, 2, B * 40)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    t, f = dev(table), dev(free)
    n = cuda_lib.paged_release(dev(begin), dev(end), t, f, dev([2]), B * 40, status=status)
    assert n.item() == want_n and np.array_equal(f.cpu().numpy(), want_f)
    assert np.array_equal(t.cpu().numpy(), want_t)
    assert cuda_lib.read_device_status(status) == sum(BITS[x] for x in flags)


@pytest.mark.parametrize("rows", [0, 1, 20, 300])
@pytest.mark.parametrize("page", [99, 64, -4])
def test_step_plan_flags_a_bad_page_that_no_row_reaches(cuda_lib, rows, page):
    """A page of the free list outside the pool is flagged where it goes into a table, not only where a
    row of the call lands on it; the entry and the lengths are as the definition says."""
    a = ([5, 16, 0], [3, 250, 40], np.full((3, 20), 7), np.array(list(range(20, 30)) + [page] + list(range(30, 46))), 27, 64, rows)
    want = S.step_plan(*a)
    assert "page" in want["flags"]
    check_plan(*run_plan(cuda_lib, *a), want)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("new", [[2**31 - 1, 3, 40, 0, 1], [5, 2**31 - 1, 2**31 - 1, 3, 40],
                                 [2**30, 2**30, 1, 2**30, 17]])
def test_step_plan_lengths_that_sum_past_32_bits(cuda_lib, new, in_place):
    """Requests that do not fit keep their rows in the packing, whose offsets end at 2^31 - 1; the ones
    that fit get their pages and lengths all the same."""
    cached = [0, 5, 16, 7, 30]
    table, free = np.arange(5 * 20).reshape(5, 20), np.arange(200, 260)
    a = (cached, new, table, free, 60, 300, 64)
    # (the sequential definition walks every row, so it is given the rows that do not fit as few)
    few = [n if n < 1000 else 400 for n in new]
    want = S.step_plan(cached, few, table, free, 60, 300, 64)
    lens = dev(cached)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    t, count = dev(table), dev([60])
    got = cuda_lib.paged_step_plan(lens, dev(new), t, dev(free), count, 300, total_rows=64, status=status,
                                   **(dict(seq_lens=lens, free_count_out=count) if in_place else {}))
    assert got.cu_new_lens.tolist() == [min(2**31 - 1, int(x)) for x in np.cumsum([0] + new)]
    assert got.seq_lens.tolist() == want["seq_lens"].tolist()
    assert got.free_count.item() == want["count"] and np.array_equal(t.cpu().numpy(), want["table"])
    first = next(i for i, n in enumerate(new) if n >= 1000)
    rows = min(64, sum(new[:first]))
    assert np.array_equal(got.slot_map.cpu().numpy()[:rows], want["slots"][:rows])
    assert (got.slot_map[rows:] == -1).all() and (got.positions[rows:] == 0).all()
    assert cuda_lib.read_device_status(status) == BITS["length"] and want["flags"] == {"length"}


@pytest.mark.parametrize("at", [(0, 1), (1, 0), (2, 0), (3, 3)])
@pytest.mark.parametrize("B", [1, 37, 4000])
def test_step_plan_into_part_of_a_larger_buffer(cuda_lib, B, at):
    """positions and slot_map at offsets that 16-byte stores cannot take; what lies around them stays."""
    a = make(B + 5, B, 60, 50, 1.0, 3)
    want = S.step_plan(*a)
    rows = a[6]
    pos = torch.full((rows + 8,), 77, dtype=torch.int32, device="cuda")
    slots = torch.full((rows + 8,), 77, dtype=torch.int64, device="cuda")
    p, m = pos[at[0]:at[0] + rows], slots[at[1]:at[1] + rows]
    check_plan(*run_plan(cuda_lib, *a, positions=p, slot_map=m), want)
    assert bool((pos[:at[0]] == 77).all()) and bool((pos[at[0] + rows:] == 77).all())
    assert bool((slots[:at[1]] == 77).all()) and bool((slots[at[1] + rows:] == 77).all())


@pytest.mark.parametrize("rows", [1, 2, 3, 5, 6, 7])
def test_step_plan_looks_at_no_page_of_rows_that_it_does_not_write(cuda_lib, rows):
    """Rows past total_rows are not written, and the pages that they would land on are not flagged."""
    table = np.array([[3, -1], [99, -1]])
    a = ([0, 5], [rows, 2], table, np.array([7, 8]), 2, 64, rows)
    want = S.step_plan(*a)
    assert want["flags"] == {"length"}
    check_plan(*run_plan(cuda_lib, *a), want)
