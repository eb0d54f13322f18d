"""Cases of the serving operators around the paged KV cache: scored attention (decode and
chunked prefill), rotary positions with the KV append, and page tables built on the GPU.

``run`` computes a case in plain torch operations, or, where ``own`` is set, through the
framework's calls. ``exact`` gives the definition in 64 bits. Lengths, masks and page counts of
a case follow from the case alone; tensor values and page placement follow from the seed.
"""
import math

import numpy as np
import torch

own = False

PAGE = 16
DIM = 128
SCALE = 1.0 / math.sqrt(DIM)
DEV = "cuda"


# ----------------------------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------------------------
def _decode(batch, lmin, lmax, mix, *, hkv=8, softcap=0.0, alibi=False, window=0, prefix=0,
            docs=0, empty=False, qscale=1.0, name=None):
    c = dict(op="decode", batch=batch, lmin=lmin, lmax=lmax, mix=mix, hkv=hkv, softcap=softcap,
             alibi=alibi, window=window, prefix=prefix, docs=docs, empty=empty, qscale=qscale)
    return dict(c, name=name) if name else c


def _prefill(chunks, mix, *, hkv=8, softcap=0.0, alibi=False, window=0, prefix=0, docs=0,
             empty=False, qscale=1.0, name=None):
    c = dict(op="prefill", chunks=chunks, mix=mix, hkv=hkv, softcap=softcap, alibi=alibi,
             window=window, prefix=prefix, docs=docs, empty=empty, qscale=qscale)
    return dict(c, name=name) if name else c


def _rope(rows, pad, mix, *, hkv=8, rot=128, interleaved=False, scaling="none", norm=True,
          maxpos=131072, name=None):
    c = dict(op="rope", rows=rows, pad=pad, mix=mix, hkv=hkv, rot=rot, interleaved=interleaved,
             scaling=scaling, norm=norm, maxpos=maxpos)
    return dict(c, name=name) if name else c


def _plan(batch, chunks, chunk, pad, mix, *, lmax=90_000, short=False, name=None):
    c = dict(op="plan", batch=batch, chunks=chunks, chunk=chunk, pad=pad, mix=mix, lmax=lmax,
             short=short)
    return dict(c, name=name) if name else c


def _release(batch, lmax, mix, *, name=None):
    c = dict(op="release", batch=batch, lmax=lmax, mix=mix)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one request of 80 s of audio, capped scores: a call whose latency is what counts
        _decode(1, 1000, 1000, 1, softcap=30.0, name="decode_cap_b1_l1000"),
        # 16 concurrent 38-minute meetings: the last 4,096 tokens and a prompt of up to 750
        _decode(16, 27_000, 30_000, 2, window=4096, prefix=750, name="decode_window_b16_l27k"),
        # 64 recordings of 30 s to 90 min, capped scores and a distance bias: bound by the cache
        _decode(64, 375, 70_000, 3, softcap=50.0, alibi=True, qscale=4.0, name="decode_cap_bias_b64"),
        # a chunk of a long recording under a sliding window with its prompt kept in view
        _prefill("4096@32768", 4, window=4096, prefix=375, name="prefill_window_4096_at_32768"),
        # the last chunk of a 90-minute recording with capped scores: the most work of all
        _prefill("4096@61440", 5, softcap=30.0, qscale=4.0, name="prefill_cap_4096_at_61440"),
        # several requests in one call, recordings packed behind each other, distance bias
        _prefill("4096@28672,2048@61440,1024@10000,512@0,1@5000,2@20000", 6, alibi=True, docs=9,
                 empty=True, name="prefill_docs_bias_mix"),
        # the first chunk of a request whose prompt is seen in both directions
        _prefill("375@0", 7, prefix=375, name="prefill_prefix_375_at_0"),
        # one decode step of 31 requests, batch padded to 32 rows for a graph
        _rope(31, 1, 8, name="rope_31_rows"),
        # a prompt chunk and 31 decodes in one step, positions stretched for long recordings
        _rope(4096 + 31, 0, 9, scaling="yarn", name="rope_yarn_4127_rows"),
        # the same step's tables: one chunk of 4,096 tokens and 31 decodes
        _plan(32, 1, 4096, 0, 10, name="plan_32_requests"),
        # the largest batch, most of it decoding
        _plan(4096, 12, 4096, 13, 11, lmax=8000, name="plan_4096_requests"),
        # requests that finish or leave a window behind give their pages back
        _release(512, 8000, 12, name="release_512_requests"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    mix = rng.randrange(1 << 30)
    kind = rng.choice(["decode", "decode", "prefill", "prefill", "rope", "plan", "release"])
    hkv = rng.choice([8, 8, 8, 4, 2, 1])
    masks = dict(hkv=hkv, softcap=rng.choice([0.0, 0.0, 20.0, 30.0, 50.0]),
                 alibi=rng.random() < 0.4, window=rng.choice([0, 0, _log_int(rng, 16, 16_384)]),
                 prefix=rng.choice([0, 0, _log_int(rng, 1, 2000)]),
                 docs=rng.choice([0, 0, rng.randint(1, 12)]), empty=rng.random() < 0.3,
                 qscale=rng.choice([1.0, 1.0, 4.0]))
    if kind == "decode":
        batch = _log_int(rng, 1, 256)
        lmax = _log_int(rng, 1, min(70_000, 2_000_000 // batch))
        return _decode(batch, rng.randint(1, lmax), lmax, mix, **masks)
    if kind == "prefill":
        chunks = []
        for _ in range(rng.choice([1, 1, 2, 4, 7])):
            n = _log_int(rng, 1, 4096 if not chunks else 1024)
            chunks.append("%d@%d" % (n, rng.choice([0, _log_int(rng, 1, 40_000)])))
        return _prefill(",".join(chunks), mix, **masks)
    if kind == "rope":
        return _rope(_log_int(rng, 1, 8192), rng.choice([0, rng.randint(0, 40)]), mix, hkv=hkv,
                     rot=rng.choice([128, 128, 96, 64, 32]), interleaved=rng.random() < 0.5,
                     scaling=rng.choice(["none", "linear", "ntk", "llama3", "yarn"]),
                     norm=rng.random() < 0.5, maxpos=_log_int(rng, 1000, 1_000_000))
    if kind == "plan":
        batch = _log_int(rng, 1, 4096)
        return _plan(batch, rng.randint(0, min(batch, 12)), _log_int(rng, 2, 4096),
                     rng.randint(0, 64), mix, lmax=_log_int(rng, 10, 8000),
                     short=rng.random() < 0.3)
    return _release(_log_int(rng, 1, 512), _log_int(rng, 16, 8000), mix)


# ----------------------------------------------------------------------------------------------
# what a case fixes on the host: lengths, masks, page counts
# ----------------------------------------------------------------------------------------------
def _attn_host(case):
    """q_lens, seq_lens, prefix lengths and each row's first own key of an attention case."""
    rng = np.random.Generator(np.random.PCG64(case["mix"]))
    if case["op"] == "decode":
        lens = np.exp(rng.uniform(math.log(case["lmin"]), math.log(case["lmax"]), case["batch"]))
        lens = np.clip(np.round(lens).astype(np.int64), case["lmin"], case["lmax"])
        n = np.ones(len(lens), np.int64)
    else:
        pairs = [c.split("@") for c in case["chunks"].split(",")]
        n = np.array([int(a) for a, _ in pairs], np.int64)
        lens = n + np.array([int(b) for _, b in pairs], np.int64)
    prefix = np.zeros(len(lens), np.int64)
    if case["prefix"]:  # prompts of different lengths, one of them the longest
        prefix = rng.integers(0, case["prefix"], len(lens), endpoint=True)
        prefix[0] = case["prefix"]
    pos = np.concatenate([np.arange(l - k, l) for l, k in zip(lens, n)])
    start = np.zeros(len(pos), np.int64)
    if case["docs"]:  # each sequence packs up to docs + 1 documents
        at = 0
        for l, k in zip(lens, n):
            cuts = np.sort(np.concatenate([[0], rng.integers(0, l, case["docs"])]))
            p = pos[at:at + k]
            start[at:at + k] = cuts[np.searchsorted(cuts, p, side="right") - 1]
            at += k
    if case["empty"]:  # some rows have no key of their own (padding inside a batch)
        start = np.where(rng.random(len(pos)) < 0.03, pos + 1, start)
    lo = np.maximum(start, pos - case["window"] + 1 if case["window"] else 0)
    return dict(n=n, lens=lens, prefix=prefix, pos=pos, start=start, lo=np.minimum(lo, pos + 1),
                seq=np.repeat(np.arange(len(lens)), n))


def _rope_host(case):
    rng = np.random.Generator(np.random.PCG64(case["mix"]))
    rows = case["rows"]
    chunk = rows - rows // 8 if rows > 64 else 0  # a prompt chunk, the rest single tokens
    first = int(rng.integers(0, max(1, case["maxpos"] - chunk)))
    pos = np.concatenate([np.arange(first, first + chunk),
                          rng.integers(0, case["maxpos"], rows - chunk)])
    return pos, -(-rows // PAGE) * 2 + 1


def _plan_host(case):
    rng = np.random.Generator(np.random.PCG64(case["mix"]))
    B = case["batch"]
    new = np.ones(B, np.int64)
    at = rng.permutation(B)[:case["chunks"]]
    new[at] = rng.integers(max(1, case["chunk"] // 2), case["chunk"], len(at), endpoint=True)
    if len(at):
        new[at[0]] = case["chunk"]
    cached = np.round(np.exp(rng.uniform(0, math.log(case["lmax"]), B))).astype(np.int64) - 1
    held = -(-cached // PAGE)
    need = -(-(cached + new) // PAGE) - held
    free = int(need.sum()) + 5
    if case["short"]:  # fewer free pages than the step asks for: the last requests wait
        free = int(need.sum() * 0.7)
    return cached, new, held, need, free


def _release_host(case):
    rng = np.random.Generator(np.random.PCG64(case["mix"]))
    B = case["batch"]
    pages = -(-np.round(np.exp(rng.uniform(0, math.log(case["lmax"]), B))).astype(np.int64) // PAGE)
    kind = rng.integers(0, 3, B)  # 0: still running, 1: finished, 2: a window moved on
    end = np.where(kind == 1, pages, np.where(kind == 2, pages // 2, 0))
    begin = np.where(kind == 2, pages // 8, 0)
    gone = rng.integers(0, np.maximum(1, pages // 3), B)  # entries from begin given back earlier
    return pages, begin, end, np.where(kind > 0, gone, 0)


def _visible_keys(h):
    """Keys that some row of their sequence sees (a lower bound of what has to be read)."""
    total, at = 0, 0
    for l, k, p in zip(h["lens"], h["n"], h["prefix"]):
        lo, pos = h["lo"][at:at + k], h["pos"][at:at + k]
        own_rows = lo <= pos
        mark = np.zeros(int(l) + 1, np.int64)
        np.add.at(mark, lo[own_rows], 1)
        np.add.at(mark, pos[own_rows] + 1, -1)
        seen = np.cumsum(mark)[:l] > 0
        seen[:min(int(p), int(l))] = True
        total += int(seen.sum())
        at += int(k)
    return total


def _pairs(h):
    p = np.minimum(h["prefix"], h["lens"])[h["seq"]]
    last = h["pos"] + 1
    both = np.maximum(0, np.minimum(p, last) - h["lo"])
    return int((p + (last - h["lo"]) - both).sum())


def work(case):
    if case["op"] in ("decode", "prefill"):
        h = _attn_host(case)
        hkv, rows = case["hkv"], len(h["pos"])
        kv = _visible_keys(h) * hkv * DIM * 2 * 2
        io = rows * 2 * hkv * (DIM * 2 * 2 + 4)
        return {"bytes": kv + io + 4 * rows, "flops": 4 * DIM * 2 * hkv * _pairs(h)}
    if case["op"] == "rope":
        hkv = case["hkv"]
        return {"bytes": case["rows"] * (4 * hkv * DIM * 2 * 2 + 12), "flops": 0}
    if case["op"] == "plan":
        cached, new, held, need, free = _plan_host(case)
        rows = int(new.sum()) + case["pad"]
        return {"bytes": 8 * len(new) + 8 * len(new) + 8 * min(free, int(need.sum())) + 12 * rows, "flops": 0}
    pages, begin, end, gone = _release_host(case)
    return {"bytes": 8 * len(pages) + 12 * int((end - begin).sum()), "flops": 0}


# ----------------------------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------------------------
def _randn(shape, g, scale=1.0):
    out = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 27):
        part = flat[i:i + (1 << 27)]
        part.copy_(torch.randn(part.numel(), generator=g, device=DEV).mul_(scale))
    return out


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _table(pages, num_pages, g, stride=None):
    """A block table whose pages are drawn from one permutation of the pool; the rest is page 0.
    Returns it with the pages left over."""
    perm = torch.randperm(num_pages, generator=g, device=DEV).to(torch.int32)
    stride = max(1, int(pages.max())) if stride is None else stride
    n = torch.from_numpy(pages).to(DEV)
    cell = torch.arange(stride, device=DEV)[None, :]
    index = (n.cumsum(0) - n)[:, None] + cell
    table = torch.where(cell < n[:, None], perm[index.clamp(max=num_pages - 1)], 0)
    return table.to(torch.int32).contiguous(), perm[int(pages.sum()):].contiguous()


def _inv_freq(case):
    """Frequencies of the rotated pairs in 64 bits and the factor on cos and sin."""
    rot, theta = case["rot"], 1e6
    i = np.arange(rot // 2, dtype=np.float64)
    f = theta ** (-2.0 * i / rot)
    kind, factor, original = case["scaling"], 4.0, 32768
    if kind == "linear":
        return f / factor, 1.0
    if kind == "ntk":
        return (theta * factor ** (rot / (rot - 2.0))) ** (-2.0 * i / rot), 1.0
    if kind == "llama3":
        low, high = 1.0, 4.0
        turns = original * f / (2 * math.pi)
        mid = np.clip((turns - low) / (high - low), 0.0, 1.0)
        return f / factor * (1 - mid) + f * mid, 1.0
    if kind == "yarn":
        def dim_of(turns):
            return rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(theta))
        low, high = max(math.floor(dim_of(32.0)), 0), min(math.ceil(dim_of(1.0)), rot - 1)
        ramp = np.clip((i - low) / max(high - low, 1e-3), 0.0, 1.0)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    if case["op"] in ("decode", "prefill"):
        h = _attn_host(case)
        hkv, hq, rows = case["hkv"], 2 * case["hkv"], len(h["pos"])
        pages = -(-h["lens"] // PAGE)
        num_pages = int(pages.sum()) + 17
        table, _ = _table(pages, num_pages, g)
        slopes = torch.exp2(-8.0 * torch.arange(1, hq + 1, device=DEV, dtype=torch.float32) / hq)
        slopes = slopes * (0.9 + 0.2 * torch.rand(hq, generator=g, device=DEV))
        return dict(
            case=case, q=_randn((rows, hq, DIM), g, case["qscale"]),
            k_pool=_randn((num_pages, PAGE, hkv, DIM), g),
            v_pool=_randn((num_pages, PAGE, hkv, DIM), g),
            table=table, seq_lens=_i32(h["lens"]), max_len=int(h["lens"].max()),
            max_n=int(h["n"].max()), cu=_i32(np.concatenate([[0], np.cumsum(h["n"])])),
            bounds=[(int(a), int(a + n), int(l)) for a, n, l in
                    zip(np.cumsum(h["n"]) - h["n"], h["n"], h["lens"])],
            slopes=slopes if case["alibi"] else None,
            prefix=_i32(h["prefix"]) if case["prefix"] else None,
            start=_i32(h["start"]) if case["docs"] or case["empty"] else None,
            out=torch.empty(rows, hq, DIM, dtype=torch.bfloat16, device=DEV),
            lse=torch.empty(rows, hq, dtype=torch.float32, device=DEV))
    if case["op"] == "rope":
        pos, num_pages = _rope_host(case)
        hkv, hq, rows, pad = case["hkv"], 2 * case["hkv"], case["rows"], case["pad"]
        qkv = _randn((rows + pad, hq + 2 * hkv, DIM), g, 2.0)  # one projection's output
        slots = torch.randperm(num_pages * PAGE, generator=g, device=DEV)[:rows]
        freq, factor = _inv_freq(case)
        gamma = [1.0 + 0.1 * torch.randn(DIM, generator=g, device=DEV) for _ in range(2)]
        return dict(
            case=case, q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:],
            positions=_i32(np.concatenate([pos, np.zeros(pad)])),
            slots=torch.cat([slots, torch.full((pad,), -1, device=DEV, dtype=torch.int64)]),
            k_pool=_randn((num_pages, PAGE, hkv, DIM), g),
            v_pool=_randn((num_pages, PAGE, hkv, DIM), g),
            inv_freq=torch.from_numpy(freq).to(DEV), factor=factor,
            q_gamma=gamma[0] if case["norm"] else None, k_gamma=gamma[1] if case["norm"] else None,
            q_out=torch.zeros(rows + pad, hq, DIM, dtype=torch.bfloat16, device=DEV))
    if case["op"] == "plan":
        cached, new, held, need, free = _plan_host(case)
        spare = max(free, int(need.sum())) + 3
        num_pages = int(held.sum()) + spare
        stride = int((held + need).max()) + 1
        table, stack = _table(held, num_pages, g, stride)
        rows, B = int(new.sum()) + case["pad"], len(new)
        e = dict(dtype=torch.int32, device=DEV)
        return dict(case=case, cached=_i32(cached), new=_i32(new), table=table, stack=stack,
                    count=torch.full((1,), free, **e), num_pages=num_pages, rows=rows,
                    count_out=torch.empty(1, **e), cu=torch.empty(B + 1, **e),
                    seq_lens=torch.empty(B, **e), positions=torch.empty(rows, **e),
                    slots=torch.empty(rows, dtype=torch.int64, device=DEV))
    pages, begin, end, gone = _release_host(case)
    num_pages = int(pages.sum()) + 64
    table, spare = _table(pages, num_pages, g)
    cell = torch.arange(table.shape[1], device=DEV)[None, :]
    b, n = (torch.from_numpy(x).to(DEV)[:, None] for x in (begin, gone))
    table = torch.where((cell >= b) & (cell < b + n), -1, table).to(torch.int32)
    stack = torch.zeros(num_pages, dtype=torch.int32, device=DEV)
    stack[:len(spare)] = spare
    return dict(case=case, begin=_i32(begin), end=_i32(end), first=table, table=table.clone(),
                stack=stack, count=torch.full((1,), len(spare), dtype=torch.int32, device=DEV),
                count_out=torch.empty(1, dtype=torch.int32, device=DEV), num_pages=num_pages)


# ----------------------------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s, op)
    return {"decode": _plain_decode, "prefill": _plain_prefill, "rope": _plain_rope,
            "plan": _plain_plan, "release": _plain_release}[op](s)


def _own(s, op):
    import long_context_paged_gb300 as pa
    c = s["case"]
    dims = None
    if "hkv" in c and c["hkv"] != 8:
        dims = (2 * c["hkv"], c["hkv"], DIM, PAGE)
    if op == "decode":
        return pa.attn_decode_paged(
            s["q"], s["k_pool"], s["v_pool"], s["table"], s["seq_lens"], s["max_len"], SCALE,
            out=s["out"], lse=s["lse"], dims=dims, softcap=c["softcap"],
            alibi_slopes=s["slopes"], window=c["window"], prefix_lens=s["prefix"],
            max_prefix_len=c["prefix"], row_start=s["start"])
    if op == "prefill":
        return pa.attn_prefill_chunk(
            s["q"], s["cu"], s["k_pool"], s["v_pool"], s["table"], s["seq_lens"], s["max_n"],
            s["max_len"], SCALE, out=s["out"], lse=s["lse"], dims=dims, softcap=c["softcap"],
            alibi_slopes=s["slopes"], window=c["window"], prefix_lens=s["prefix"],
            max_prefix_len=c["prefix"], row_start=s["start"])
    if op == "rope":
        q = pa.rope_append_paged(
            s["q"], s["k"], s["v"], s["positions"], s["slots"], s["k_pool"], s["v_pool"],
            s["inv_freq"], interleaved=c["interleaved"], attn_factor=s["factor"],
            q_gamma=s["q_gamma"], k_gamma=s["k_gamma"], q_out=s["q_out"], dims=dims)
        return q, s["k_pool"], s["v_pool"]
    if op == "plan":
        p = pa.paged_step_plan(
            s["cached"], s["new"], s["table"], s["stack"], s["count"], s["num_pages"],
            total_rows=s["rows"], free_count_out=s["count_out"], cu_new_lens=s["cu"],
            seq_lens=s["seq_lens"], positions=s["positions"], slot_map=s["slots"])
        return p.cu_new_lens, p.seq_lens, p.positions, p.slot_map, p.free_count, s["table"]
    s["table"].copy_(s["first"])
    n = pa.paged_release(s["begin"], s["end"], s["table"], s["stack"], s["count"], s["num_pages"],
                         free_count_out=s["count_out"])
    return s["table"], s["stack"], n


def _softmax_rows(x, v, vis, dist, slopes, cap):
    """x [..., H, R, K] scores, v [..., H, K, D] values, vis and dist [..., R, K] of each row and
    key, slopes [H, R, 1] or None -> (o, lse) in 32 bits. Distances are counted from the nearest
    visible key, so that a large bias common to a row leaves the scores' low bits alone."""
    if cap:
        x = x.div_(cap).tanh_().mul_(cap)
    shift = 0.0
    if slopes is not None:
        near = torch.where(vis, dist, float("inf")).amin(-1, keepdim=True)
        near = torch.where(torch.isinf(near), 0.0, near).unsqueeze(-3)
        x = x.sub_(slopes * (dist.unsqueeze(-3) - near))
        shift = slopes * near
    x = x.masked_fill_(~vis.unsqueeze(-3), float("-inf"))
    m = x.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), 0.0, m)
    x = x.sub_(m).exp_()
    l = x.sum(-1, keepdim=True)
    o = (x @ v) / torch.where(l > 0, l, 1.0)
    return o, (torch.log(l) + m - shift).squeeze(-1)


def _plain_decode(s):
    c = s["case"]
    B, hkv, L = c["batch"], c["hkv"], s["max_len"]
    key = torch.arange(L, device=DEV)
    page, slot = s["table"].long()[:, key // PAGE], key % PAGE  # entries past a sequence: page 0
    k = s["k_pool"][page, slot].float().permute(0, 2, 3, 1)     # [B, Hkv, D, L]
    q = s["q"].float().view(B, hkv, 2, DIM)
    x = (q @ k).mul_(SCALE)  # both query heads of a KV head as rows of one product
    del k
    n = s["seq_lens"].long()[:, None, None]
    start = None if s["start"] is None else s["start"].long()[:, None, None]
    prefix = None if s["prefix"] is None else s["prefix"].long()[:, None, None]
    vis, dist = _mask(c["window"], key, n - 1, n, start, prefix)
    v = s["v_pool"][page, slot].float().permute(0, 2, 1, 3)
    slopes = None if s["slopes"] is None else s["slopes"].view(hkv, 2, 1)
    o, lse = _softmax_rows(x, v, vis, dist, slopes, c["softcap"])
    s["out"].copy_(o.reshape(B, 2 * hkv, DIM))
    s["lse"].copy_(lse.reshape(B, 2 * hkv))
    return s["out"], s["lse"]


def _mask(window, key, pos, n, start, prefix):
    """Visibility and distance of every (row, key) of sequences of n keys: a key of the prefix,
    or one between the row's first own key and its position."""
    vis = key <= pos
    if start is not None:
        vis &= key >= start
    if window:
        vis &= key > pos - window
    if prefix is not None:
        vis |= key < torch.minimum(prefix, n)
    return vis, (pos - key).abs().float()


def _plain_prefill(s):
    c = s["case"]
    hkv = c["hkv"]
    # each chunk has keys of its own; padding them to one length would need 100s of GB
    for b, (r0, r1, L) in enumerate(s["bounds"]):
        R = r1 - r0
        key = torch.arange(L, device=DEV)
        page, slot = s["table"][b].long()[key // PAGE], key % PAGE
        k = s["k_pool"][page, slot].float().permute(1, 2, 0)     # [Hkv, D, L]
        v = s["v_pool"][page, slot].float().permute(1, 0, 2)
        # rows ordered head of the group, then query
        q = s["q"][r0:r1].float().view(R, hkv, 2, DIM).permute(1, 2, 0, 3).reshape(hkv, 2 * R, DIM)
        x = (q @ k).mul_(SCALE)
        pos = torch.arange(L - R, L, device=DEV)[:, None].repeat(2, 1)
        start = None if s["start"] is None else s["start"][r0:r1, None].long().repeat(2, 1)
        prefix = None if s["prefix"] is None else s["prefix"][b].long()
        vis, dist = _mask(c["window"], key, pos, s["seq_lens"][b].long(), start, prefix)
        slopes = None if s["slopes"] is None else s["slopes"].view(hkv, 2, 1).repeat_interleave(R, 1)
        o, lse = _softmax_rows(x, v, vis, dist, slopes, c["softcap"])
        s["out"][r0:r1] = o.view(hkv, 2, R, DIM).permute(2, 0, 1, 3).reshape(R, 2 * hkv, DIM)
        s["lse"][r0:r1] = lse.view(hkv, 2, R).permute(2, 0, 1).reshape(R, 2 * hkv)
    return s["out"], s["lse"]


def _plain_rope(s):
    c = s["case"]
    rows, rot = c["rows"], c["rot"]
    angle = s["positions"][:rows].double()[:, None] * s["inv_freq"]
    cos, sin = (t.mul(s["factor"]).float()[:, None, :] for t in (angle.cos(), angle.sin()))

    def turn(x, gamma):
        x = x[:rows].float()
        if gamma is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * gamma
        if c["interleaved"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([y, x[..., rot:]], -1).to(torch.bfloat16)

    s["q_out"][:rows] = turn(s["q"], s["q_gamma"])
    at = s["slots"][:rows]
    s["k_pool"].view(-1, c["hkv"], DIM)[at] = turn(s["k"], s["k_gamma"])
    s["v_pool"].view(-1, c["hkv"], DIM)[at] = s["v"][:rows]
    return s["q_out"], s["k_pool"], s["v_pool"]


def _plain_plan(s):
    cached, new, table = s["cached"].long(), s["new"].long(), s["table"]
    held = (cached + PAGE - 1) // PAGE
    need = (cached + new + PAGE - 1) // PAGE - held
    cum = need.cumsum(0)
    ok = (need == 0) | (cum <= s["count"])
    first = s["count"].long() - 1 - (cum - need)  # stack index of a request's first new page
    cell = torch.arange(table.shape[1], device=DEV)[None, :]
    k = cell - held[:, None]
    fresh = (k >= 0) & (k < need[:, None]) & ok[:, None]
    table.copy_(torch.where(fresh, s["stack"][(first[:, None] - k).clamp(0, len(s["stack"]) - 1)], table))
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), new.cumsum(0)])
    t = torch.arange(s["rows"], device=DEV)
    b = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=len(new) - 1)
    pos = cached[b] + t - cu[b]
    live = (t < cu[-1]) & ok[b]
    page = table[b, (pos // PAGE).clamp(max=table.shape[1] - 1)].long()
    s["cu"].copy_(cu)
    s["seq_lens"].copy_(torch.where(ok, cached + new, cached))
    s["positions"].copy_(torch.where(live, pos, 0))
    s["slots"].copy_(torch.where(live, page * PAGE + pos % PAGE, -1))
    s["count_out"].copy_(s["count"] - torch.where(ok, need, 0).sum())
    return s["cu"], s["seq_lens"], s["positions"], s["slots"], s["count_out"], table


def _plain_release(s):
    s["table"].copy_(s["first"])
    table, stack = s["table"], s["stack"]
    cell = torch.arange(table.shape[1], device=DEV)[None, :]
    give = (cell >= s["begin"][:, None]) & (cell < s["end"][:, None]) & (table >= 0)
    at = (give.flatten().cumsum(0) - 1 + s["count"]).view_as(give)
    stack.scatter_(0, torch.where(give, at, len(stack) - 1).flatten(),
                   torch.where(give, table, stack[-1]).flatten())
    s["count_out"].copy_(s["count"] + give.sum())
    table.masked_fill_(give, -1)
    return table, stack, s["count_out"]


# ----------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] in ("decode", "prefill"):
        return _exact_attention(case, seed)
    if case["op"] == "rope":
        return _exact_rope(case, seed)
    return None


def _exact_attention(case, seed):
    s, h = prepare(case, seed), _attn_host(case)
    hkv, group = case["hkv"], 2
    out = torch.zeros(len(h["pos"]), hkv * group, DIM, dtype=torch.float64, device=DEV)
    lse = torch.full((len(h["pos"]), hkv * group), -math.inf, dtype=torch.float64, device=DEV)
    at = 0
    for b, (L, n) in enumerate(zip(h["lens"].tolist(), h["n"].tolist())):
        pages = s["table"][b, :-(-L // PAGE)].long()
        j = torch.arange(L, device=DEV, dtype=torch.float64)
        for r0 in range(0, n, 1024):  # row blocks and heads bound the memory
            r = slice(at + r0, at + min(n, r0 + 1024))
            i = torch.from_numpy(h["pos"][r]).to(DEV).double()[:, None]
            lo = torch.from_numpy(h["start"][r]).to(DEV).double()[:, None]
            seen = (j <= i) & (j >= lo)
            if case["window"]:
                seen &= i - j < case["window"]
            seen |= j < float(h["prefix"][b])
            for head in range(hkv * group):
                keys = s["k_pool"][pages, :, head // group].reshape(-1, DIM)[:L].double()
                values = s["v_pool"][pages, :, head // group].reshape(-1, DIM)[:L].double()
                z = SCALE * (s["q"][r, head].double() @ keys.T)
                if case["softcap"]:
                    z = case["softcap"] * torch.tanh(z / case["softcap"])
                if s["slopes"] is not None:
                    z = z - s["slopes"][head].double() * (i - j).abs()
                z = torch.where(seen, z, -math.inf)
                total = torch.logsumexp(z, 1)
                w = torch.exp(z - torch.where(torch.isinf(total), 0.0, total)[:, None])
                out[r, head] = w @ values
                lse[r, head] = total
        at += n
    return out, lse


def _exact_rope(case, seed):
    s = prepare(case, seed)
    rows, half = case["rows"], case["rot"] // 2
    i = torch.arange(half, device=DEV)
    one, two = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
    phase = torch.polar(torch.full((rows, half), s["factor"], dtype=torch.float64, device=DEV),
                        s["positions"][:rows, None].double() * s["inv_freq"][None, :])[:, None]
    results = []
    for x, gamma in ((s["q"], s["q_gamma"]), (s["k"], s["k_gamma"])):
        x = x[:rows].double()
        if gamma is not None:
            x = x / ((x ** 2).sum(-1, keepdim=True) / DIM + 1e-6).sqrt() * gamma.double()
        z = torch.complex(x[..., one], x[..., two]) * phase
        x = x.clone()
        x[..., one], x[..., two] = z.real, z.imag
        results.append(x)
    q_out = torch.zeros(s["q_out"].shape, dtype=torch.float64, device=DEV)
    q_out[:rows] = results[0]
    pools = [s["k_pool"].double(), s["v_pool"].double()]
    for pool, x in zip(pools, (results[1], s["v"][:rows].double())):
        pool.view(-1, case["hkv"], DIM).index_copy_(0, s["slots"][:rows], x)
    return q_out, pools[0], pools[1]
