"""Tables and pools whose offsets pass 32 bits, and forks whose blocks hold several rounds of pages."""
import numpy as np
import pytest
import torch

from oracle import beam as O
from tests.test_gpu_fork import check, grown
from tests.test_gpu_shared_decode import SCALE, Inputs, dev

pytestmark = pytest.mark.gpu
STRIDE = (1 << 27) - 64


def room(gib):
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"needs {gib} GB")


def test_entries_past_2_31_and_pages_past_4_gib(cuda_lib):
    """Rows 17 to 19 have their entries more than 2^31 places into the table (the last group's shared pages and a row's
    own among them); the pages lie 4.6 GB into the pools."""
    room(60)
    x = Inputs([(1, [17] * 17), (2, [40, 50])], [300], hkv=8, seed=13)
    assert 17 * STRIDE > 1 << 31
    far = 140_000
    assert far * 16 * 8 * 128 * 2 > 1 << 32
    table = torch.zeros(len(x.lens), STRIDE, dtype=torch.int32, device="cuda")
    table[:, :x.table.shape[1]] = dev(np.where(x.table >= 0, x.table + far, -1))
    k = torch.zeros(far + x.pages, 16, 8, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    k[far:], v[far:] = x.k, x.v
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = cuda_lib.attn_decode_paged_shared(x.q, k, v, table, dev(x.lens), dev(x.cu), dev(x.shared), 300, SCALE,
                                                 status=status)
    torch.cuda.synchronize()
    assert cuda_lib.read_device_status(status) == 0
    x.close(out, lse)


def test_a_fork_of_entries_past_2_31(cuda_lib):
    room(30)
    G, W, stride = 5, 4, 12
    parents, lens, small, free, count, pages = grown(G, W, stride, 3)
    want = O.fork(parents, lens, small, free, count, pages)
    assert not want["flags"]
    table = torch.full((G * W, STRIDE), -1, dtype=torch.int32, device="cuda")
    table[:, :stride] = dev(small)
    f, status = dev(free), torch.zeros(1, dtype=torch.int32, device="cuda")
    got = cuda_lib.paged_fork(dev(parents), dev(lens), table, f, dev([count]), pages, status=status)
    torch.cuda.synchronize()
    assert cuda_lib.read_device_status(status) == 0
    assert got.seq_lens.tolist() == list(want["lens"]) and got.shared_pages.tolist() == want["shared"]
    assert [tuple(x) for x in got.copies.tolist()] == [tuple(int(v) for v in x) for x in want["copies"]]
    assert got.free_count.item() == want["count"]
    assert np.array_equal(table[:, :stride].cpu().numpy(), want["table"])
    assert np.array_equal(f.cpu().numpy(), want["free"])
    assert int(table[:, stride:].max()) == -1


def many(G, W, stride, seed):
    """grown() for many groups: four of them over and over, with pages of their own (made quickly)."""
    parents, lens, table, free, count, pages = grown(4, W, stride, seed)
    times = G // 4
    at = np.arange(times)[:, None, None] * pages
    tables = np.where(table[None] >= 0, table[None] + at, -1).reshape(G * W, stride)
    spare = np.concatenate([free[:count] + i * pages for i in range(times)])
    frees = np.concatenate([spare, np.zeros(times * pages - len(spare), np.int64)])
    return np.tile(parents, (times, 1)), np.tile(lens, times), tables, frees, len(spare), times * pages


@pytest.mark.parametrize("G,W,stride,inplace", [(1000, 2, 1100, False), (1400, 2, 1200, True), (372, 11, 2817, False)])
def test_blocks_of_several_rounds_of_pages(cuda_lib, G, W, stride, inplace):
    """4,096 blocks of 256 pages and more: a block then takes them in rounds."""
    assert G * -(-stride // 256) >= 4096
    check(cuda_lib, *many(G, W, stride, G), inplace=inplace)
