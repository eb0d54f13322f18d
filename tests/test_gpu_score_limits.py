"""The calls with options, the rotary append and the step plan at their limits: offsets past 32 bits,
the largest batches, rows behind the last sequence, two calls at once, capped grids."""
import numpy as np
import pytest
import torch

import workloads as W
from oracle import serving as S
from tests.helpers import bits
from tests.test_gpu_score_decode import close as close_decode
from tests.test_gpu_score_prefill import call, close as close_prefill, reference

pytestmark = pytest.mark.gpu

SLOPES = 2.0 ** (-0.5 * np.arange(1, 17))


def dev(a, dtype=torch.int32):
    return torch.tensor(np.asarray(a), dtype=dtype, device="cuda")


def test_pools_past_4_gib(cuda_lib):
    """Pages whose byte offset in a pool is past 2^32 (32 KB each; pages from 131,072 on)."""
    pages, L, n = 140_000, 300, 40
    g = torch.Generator(device="cuda").manual_seed(1)
    kp = torch.zeros(pages, 16, 8, 128, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    used = torch.arange(pages - 19, pages, device="cuda")[torch.randperm(19, generator=g, device="cuda")]
    for p in (kp, vp):
        p[used] = torch.randn(19, 16, 8, 128, generator=g, device="cuda").to(torch.bfloat16)
    table = used.to(torch.int32)[None, :].contiguous()
    qkv = torch.randn(n, 32, 128, generator=g, device="cuda").to(torch.bfloat16)
    pos = torch.arange(L - n, L, dtype=torch.int32, device="cuda")
    slots = table[0, pos.long() // 16].long() * 16 + pos.long() % 16
    freq, f = cuda_lib.rope_inv_freq()
    q = cuda_lib.rope_append_paged(qkv[:, :16], qkv[:, 16:24], qkv[:, 24:], pos, slots, kp, vp, freq)
    torch.cuda.synchronize()
    assert torch.equal(vp.view(-1, 8, 128)[slots], qkv[:, 24:])
    small_k, small_v = kp[table[0].long()], vp[table[0].long()]      # the sequence's pages, in order
    bt = np.arange(19)[None, :]
    lens = dev([L])
    o = dict(softcap=20.0, window=150, prefix=[30], slopes=SLOPES)
    kw = dict(softcap=20.0, window=150, prefix_lens=dev([30]), alibi_slopes=dev(SLOPES, torch.float32))
    out, lse = cuda_lib.attn_prefill_chunk(q, dev([0, n]), kp, vp, table, lens, n, L, 0.09, **kw)
    ref = S.prefill_scored(bits(q), [0, n], bits(small_k), bits(small_v), bt, [L], 0.09, **o)
    close_prefill(out, lse, *ref)
    for split in (0, 64):
        out, lse = cuda_lib.attn_decode_paged(q[-1:], kp, vp, table, lens, L, 0.09, split_tokens=split, **kw)
        close_decode(out, lse, ref[0][-1:], ref[1][-1:])


def test_decode_of_4096_sequences_with_options(cuda_lib):
    rng = np.random.default_rng(2)
    lens = rng.integers(0, 300, 4096)
    inp = W.make_paged(61, lens, np.ones(4096, np.int64), device="cuda", q_scale=2.0)
    o = dict(softcap=30.0, slopes=SLOPES, window=100, prefix=rng.integers(0, 50, 4096),
             row_start=rng.integers(0, np.maximum(lens, 1) + 1))
    out, lse = cuda_lib.attn_decode_paged(
        inp.q[0], inp.k_pools[0], inp.v_pools[0], inp.block_table, inp.seq_lens, 300, inp.scale,
        softcap=30.0, window=100, alibi_slopes=dev(SLOPES, torch.float32), prefix_lens=dev(o["prefix"]),
        max_prefix_len=50, row_start=dev(o["row_start"]))
    rows = sorted(set(rng.integers(0, 4096, 80).tolist()) | {0, 4095} | set(np.flatnonzero(lens == 0)[:2].tolist()))
    ref_o, ref_l = S.decode_scored(bits(inp.q[0]), bits(inp.k_pools[0]), bits(inp.v_pools[0]),
                                   inp.host_block_table, inp.host_seq_lens, inp.scale, rows=set(rows), **o)
    close_decode(out[rows], lse[rows], ref_o[rows], ref_l[rows])


def test_128_chunks_with_options_and_rows_behind_them(cuda_lib):
    rng = np.random.default_rng(3)
    q_lens, offs = rng.integers(1, 40, 128), rng.integers(0, 300, 128)
    inp = W.make_paged(62, offs + q_lens, q_lens, device="cuda", q_scale=2.0)
    T = int(q_lens.sum())
    o = dict(window=90, prefix=rng.integers(0, 60, 128), slopes=SLOPES, softcap=15.0)
    q = torch.cat([inp.q[0], inp.q[0][:9]])                          # 9 rows no sequence owns
    out = torch.full((T + 9, 16, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T + 9, 16), 5.0, device="cuda")
    call(cuda_lib, inp, o, q=q, out=out, lse=lse)
    torch.cuda.synchronize()
    assert bool((out[T:] == 5.0).all()) and bool((lse[T:] == 5.0).all())
    rows = set(rng.integers(0, T, 150).tolist()) | {0, T - 1}
    close_prefill(out[:T], lse[:T], *reference(inp, o, rows), rows=rows)
    with pytest.raises(cuda_lib.PagedAttnError):
        big = W.make_paged(63, [5] * 129, [1] * 129, device="cuda")
        call(cuda_lib, big, dict(window=3))


def test_two_prefills_and_a_decode_at_once(cuda_lib):
    """Three streams on shares of the SMs, each call with its own workspace."""
    a = W.make_paged(70, [900, 400], [200, 100], device="cuda", q_scale=2.0)
    b = W.make_paged(71, [1500], [300], device="cuda", q_scale=2.0)
    c = W.make_paged(72, [3000, 2500, 10], [1, 1, 1], device="cuda", q_scale=2.0)
    oa, ob = dict(window=120, softcap=20.0), dict(slopes=SLOPES, prefix=[64])
    oc = dict(window=700, softcap=9.0)
    alone = [call(cuda_lib, a, oa, max_ctas=40), call(cuda_lib, b, ob, max_ctas=50)]
    dec = lambda **kw: cuda_lib.attn_decode_paged(c.q[0], c.k_pools[0], c.v_pools[0], c.block_table,
                                                  c.seq_lens, 3000, c.scale, max_ctas=60, window=700,
                                                  softcap=9.0, **kw)
    alone.append(dec())
    torch.cuda.synchronize()
    st = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(5):
        got = [call(cuda_lib, a, oa, max_ctas=40, stream=st[0]), call(cuda_lib, b, ob, max_ctas=50, stream=st[1]),
               dec(stream=st[2])]
        torch.cuda.synchronize()
        for (o1, l1), (o2, l2) in zip(alone, got):
            assert torch.equal(o1, o2) and torch.equal(l1, l2)       # the same split: the same bits
    close_prefill(*got[0], *reference(a, oa))
    close_prefill(*got[1], *reference(b, ob))
    ref = S.decode_scored(bits(c.q[0]), bits(c.k_pools[0]), bits(c.v_pools[0]), c.host_block_table,
                          c.host_seq_lens, c.scale, **oc)
    close_decode(*got[2], *ref)


def test_results_repeat_bit_for_bit(cuda_lib):
    inp = W.make_paged(73, [5000, 700], [600, 130], device="cuda", q_scale=3.0)
    rng = np.random.default_rng(4)
    o = dict(softcap=25.0, slopes=SLOPES, window=2000, prefix=[100, 40], row_start=rng.integers(0, 300, 730))
    first = call(cuda_lib, inp, o)
    for _ in range(4):
        again = call(cuda_lib, inp, o)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_workspaces_that_are_too_small_are_refused(cuda_lib):
    inp = W.make_paged(74, [300], [40], device="cuda")
    need = cuda_lib.prefill_score_workspace_size(1, 40)
    ws = torch.empty(need - 256, dtype=torch.uint8, device="cuda")
    with pytest.raises(cuda_lib.PagedAttnError) as e:
        call(cuda_lib, inp, dict(window=8), workspace=ws)
    assert e.value.code == 3
    call(cuda_lib, inp, dict(window=8), workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()


def test_option_tensors_are_checked(cuda_lib):
    inp = W.make_paged(75, [300], [4], device="cuda")
    ok = dev(SLOPES, torch.float32)
    for bad in (dict(alibi_slopes=ok[:8]), dict(prefix_lens=dev(np.zeros(0))), dict(row_start=dev([0] * 3))):
        with pytest.raises(ValueError):
            cuda_lib.attn_prefill_chunk(inp.q[0], inp.cu_q_lens, inp.k_pools[0], inp.v_pools[0],
                                        inp.block_table, inp.seq_lens, 4, 300, inp.scale, **bad)
    for bad in (dict(alibi_slopes=ok.double()), dict(prefix_lens=dev([0]).long()), dict(row_start=[0] * 4)):
        with pytest.raises(TypeError):
            cuda_lib.attn_prefill_chunk(inp.q[0], inp.cu_q_lens, inp.k_pools[0], inp.v_pools[0],
                                        inp.block_table, inp.seq_lens, 4, 300, inp.scale, **bad)
    for bad in (dict(softcap=-1.0), dict(softcap=float("nan")), dict(softcap=1e-9), dict(window=-3),
                dict(prefix_lens=dev([0]), max_prefix_len=131073)):
        with pytest.raises(cuda_lib.PagedAttnError):
            cuda_lib.attn_prefill_chunk(inp.q[0], inp.cu_q_lens, inp.k_pools[0], inp.v_pools[0],
                                        inp.block_table, inp.seq_lens, 4, 300, inp.scale, **bad)
        with pytest.raises(cuda_lib.PagedAttnError):
            cuda_lib.attn_decode_paged(inp.q[0][:1], inp.k_pools[0], inp.v_pools[0], inp.block_table,
                                       inp.seq_lens, 300, inp.scale, **bad)
