"""paged_fork and paged_copy_pages against the sequential definition: whole numbers and copied bits, so
every comparison is exact."""
import numpy as np
import pytest
import torch

from oracle import beam as O

pytestmark = pytest.mark.gpu
BITS = {"length": 2, "no_pages": 16, "page": 1}


def dev(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def grown(G, W, stride, seed, spare=None, most=None):
    """A pool in the middle of a search: tables that earlier forks and appends have shared, lengths, free
    list. Every page is either in some table (at one place) or free."""
    rng = np.random.default_rng(seed)
    most = stride * 16 if most is None else most
    pages = G * W * stride + (G * W if spare is None else spare)
    free, count = rng.permutation(pages).astype(np.int32), pages
    table = np.full((G * W, stride), -1, np.int32)
    lens = np.zeros(G * W, np.int64)
    for g in range(G):
        lens[g * W] = rng.integers(1, most + 1)
        n = -(-lens[g * W] // 16)
        count -= n
        table[g * W, :n] = free[count:count + n][::-1]
    parents = np.zeros((G, W), int)
    for _ in range(4):
        f = O.fork(parents, lens, table, free, count, pages)
        assert not f["flags"]
        lens, table, free, count = np.array(f["lens"]), f["table"], f["free"], f["count"]
        for r in range(G * W):  # a few tokens each
            add = int(rng.integers(0, 20))
            new = int(min(lens[r] + add, most)) if lens[r] else 0
            for j in range(-(-lens[r] // 16), -(-new // 16)):
                count -= 1
                table[r, j] = free[count]
            lens[r] = new
        parents = rng.integers(-1, W, (G, W))
        parents[rng.random(G) < 0.3] = np.arange(W)
    if spare is not None:  # a pool with this many free pages
        free[:spare], count = free[count - spare:count].copy(), min(spare, count)
    return parents, lens, table, free, count, pages


def check(pa, parents, lens, table, free, count, pages, inplace=False, **kw):
    want = O.fork(parents, lens, table, free, count, pages)
    t, f, c, n = dev(table), dev(free), dev([count]), dev(lens)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    if inplace:
        kw.update(seq_lens_out=n, free_count_out=c)
    got = pa.paged_fork(dev(parents), n, t, f, c, pages, status=status, **kw)
    torch.cuda.synchronize()
    assert pa.read_device_status(status) == sum(BITS[x] for x in want["flags"])
    assert got.seq_lens.tolist() == list(want["lens"])
    assert [tuple(x) for x in got.copies.tolist()] == [tuple(int(v) for v in x) for x in want["copies"]]
    assert got.shared_pages.tolist() == want["shared"]
    assert got.free_count.item() == want["count"]
    assert np.array_equal(t.cpu().numpy(), want["table"])
    assert np.array_equal(f.cpu().numpy(), want["free"])
    if not inplace:
        assert c.item() == count and n.tolist() == [int(x) for x in lens]
    return want, got


@pytest.mark.parametrize("G,W,stride", [(1, 1, 1), (1, 4, 3), (3, 4, 20), (2, 5, 300), (7, 8, 33), (1, 64, 40),
                                        (40, 3, 9), (1, 2, 1100), (600, 2, 300)])
@pytest.mark.parametrize("inplace", [False, True])
def test_matches_the_definition(cuda_lib, G, W, stride, inplace):
    for seed in range(3 if G * W * stride < 50000 else 1):
        state = grown(G, W, stride, 10 * seed + inplace)
        want, _ = check(cuda_lib, *state, inplace=inplace)
        parents, lens, table, free, count, pages = state
        held = {int(e) for b, n in enumerate(want["lens"]) for e in want["table"][b, :-(-n // 16)]}
        assert sorted(list(held) + [int(e) for e in want["free"][:want["count"]]]) == list(range(pages))


def test_a_prompt_is_handed_to_all_beams_and_given_back(cuda_lib):
    for n in (1, 15, 16, 17, 100, 112):
        table = np.full((4, 8), -1)
        k = -(-n // 16)
        table[0, :k] = np.arange(k) + 3
        free = np.array([20, 21, 22, 23, 24, 0, 0, 0, 0, 0, 0, 0])
        want, got = check(cuda_lib, [[0, 0, 0, 0]], [n, 0, 0, 0], table, free, 5, 30)
        assert got.shared_pages.item() == n // 16
        check(cuda_lib, [[-1] * 4], want["lens"], want["table"], want["free"], want["count"], 30)


def test_a_filled_holder_keeps_the_page(cuda_lib):
    """The partial holder of a page that another row has filled gets the copy, wherever it stands."""
    table = np.array([[5, -1], [5, 7]])
    check(cuda_lib, [[0, 1]], [9, 20], table, [1, 2, 3], 2, 30)
    check(cuda_lib, [[1, 0]], [9, 20], table, [1, 2, 3], 2, 30)
    check(cuda_lib, [[0, 0]], [9, 20], table, [1, 2, 3], 2, 30)


@pytest.mark.parametrize("case", ["parent_high", "parent_low", "length", "negative", "no_pages", "capacity",
                                  "count_high", "count_low", "bad_entry", "bad_source", "bad_free", "released"])
def test_what_is_refused_changes_nothing_and_bad_pages_go_nowhere(cuda_lib, case):
    parents, lens, table, free, count, pages = grown(3, 4, 6, 77, spare=12)
    parents, lens = parents.copy(), lens.copy()
    if case == "parent_high":
        parents[1, 2] = 4
    elif case == "parent_low":
        parents[2, 3] = -2
    elif case == "length":
        lens[5] = 6 * 16 + 1
    elif case == "negative":
        lens[0] = -1
    elif case == "no_pages":
        lens[:] = np.where(lens > 0, np.minimum(lens | 1, 95), 0)
        parents[:] = np.argmax(lens.reshape(3, 4) > 0, 1)[:, None]
        count = 2
    elif case == "capacity":
        parents[:] = -1
        free = free[:count + 1]
    elif case == "count_high":
        count = len(free) + 3
    elif case == "count_low":
        count = -1
        parents[:] = np.arange(4)
    elif case == "bad_entry":
        parents[:] = -1
        table[table >= 0] = np.where(np.arange((table >= 0).sum()) % 3 == 0, pages + 7, table[table >= 0])
    elif case == "bad_source":
        lens[:] = np.where(lens > 0, np.minimum(lens | 1, 95), 0)
        parents[:] = np.argmax(lens.reshape(3, 4) > 0, 1)[:, None]
        table[:, :] = np.where(table >= 0, -3, table)
    elif case == "bad_free":
        lens[:] = np.where(lens > 0, np.minimum(lens | 1, 95), 0)
        parents[:] = np.argmax(lens.reshape(3, 4) > 0, 1)[:, None]
        free[:] = pages + 1
    elif case == "released":  # leading pages given back by a window
        table[:, :2] = -1
    check(cuda_lib, parents, lens, table, free, count, pages)


def test_streams_graphs_and_entries_past_the_pages(cuda_lib):
    pa = cuda_lib
    parents, lens, table, free, count, pages = grown(5, 4, 30, 8, most=300)
    table[:, 25:] = 12345      # never held, never touched
    check(pa, parents, lens, table, free, count, pages)
    want = O.fork(parents, lens, table, free, count, pages)
    args = [dev(parents), dev(lens), dev(table), dev(free), dev([count])]
    keep = [a.clone() for a in args]
    ws = torch.empty(pa.fork_workspace_size(5, 4, 30), dtype=torch.uint8, device="cuda")
    copies, shared = torch.zeros(20, 3, dtype=torch.int32, device="cuda"), torch.zeros(5, dtype=torch.int32, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            pa.paged_fork(*args, pages, seq_lens_out=args[1], free_count_out=args[4], copies=copies,
                          shared_pages=shared, workspace=ws)
        for _ in range(3):
            for a, b in zip(args, keep):
                a.copy_(b)
            g.replay()
            st.synchronize()
            assert np.array_equal(args[2].cpu().numpy(), want["table"]) and args[4].item() == want["count"]
            assert args[1].tolist() == list(want["lens"]) and shared.tolist() == want["shared"]
            assert np.array_equal(args[3].cpu().numpy(), want["free"])


@pytest.mark.parametrize("hkv", [8, 4, 2, 1])
@pytest.mark.parametrize("pools", [1, 2, 56, 130])
def test_copied_bits(cuda_lib, hkv, pools):
    g = torch.Generator().manual_seed(pools)
    P = 40
    ps = [torch.randint(-2 ** 15, 2 ** 15, (P, 16, hkv, 128), dtype=torch.int16, generator=g).cuda().view(torch.bfloat16)
          for _ in range(pools)]
    perm = torch.randperm(P, generator=g).tolist()
    copies = [(perm[i], perm[i + 18], i) if i else (-1, -1, 0) for i in range(17)]
    want = [O.copy_pages(copies, p.view(torch.int16).cpu().numpy()) for p in ps]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cuda_lib.paged_copy_pages(dev(copies), ps, status=status, dims=(2 * hkv, hkv, 128, 16))
    torch.cuda.synchronize()
    assert cuda_lib.read_device_status(status) == 0
    for p, w in zip(ps, want):
        assert np.array_equal(p.view(torch.int16).cpu().numpy(), w)


def test_copies_that_name_no_page(cuda_lib):
    pool = torch.randn(8, 16, 8, 128).to(torch.bfloat16).cuda()
    before = pool.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for bad, bit in (([8, 1, 4], 1), ([1, 8, 4], 1), ([-1, 2, 4], 1), ([2, -1, 4], 1), ([1, 2, 17], 2), ([1, 2, -1], 2)):
        cuda_lib.paged_copy_pages(dev([[-1, -1, 0], bad]), [pool], status=status)
        assert cuda_lib.read_device_status(status) == bit, bad
        assert torch.equal(pool, before)
    cuda_lib.paged_copy_pages(dev([[3, 3, 5], [4, 5, 0]]), [pool], status=status)
    assert cuda_lib.read_device_status(status) == 0 and torch.equal(pool, before)
    cuda_lib.paged_copy_pages(dev(np.zeros((0, 3))), [pool])
    cuda_lib.paged_copy_pages(dev([[0, 1, 3]]), [])


def test_a_bad_parent_beside_groups_short_of_pages_is_one_error(cuda_lib):
    """Two groups of a prompt handed to three beams need four pages and there is one; a third group's parent is bad."""
    table = np.full((9, 2), -1, np.int32)
    table[[0, 3, 6], 0] = [0, 1, 2]
    lens = np.array([5, 0, 0, 7, 0, 0, 9, 0, 0])
    parents = np.array([[0, 0, 0], [0, 0, 0], [0, 3, 0]])
    want, _ = check(cuda_lib, parents, lens, table, np.array([3], np.int32), 1, 4)
    assert want["flags"] == {"length"}
