"""Cases of the operators of a beam-search step over the paged KV cache: decode attention of rows that
share a prefix, the selection over beams and vocabulary, the fork of the beams' page tables, and the
page copies that a fork orders.

``run`` computes a case in plain torch operations, or, where ``own`` is set, through the framework's
calls. ``exact`` gives the definition in 64 bits. Lengths, parents and page counts of a case follow
from the case alone; tensor values and page placement follow from the seed.
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
def _shared(groups, rmin, rmax, lmin, lmax, own_max, mix, *, hkv=8, empty=False, qscale=1.0, name=None):
    c = dict(op="shared", groups=groups, rmin=rmin, rmax=rmax, lmin=lmin, lmax=lmax, own_max=own_max, mix=mix,
             hkv=hkv, empty=empty, qscale=qscale)
    return dict(c, name=name) if name else c


def _beam(requests, beams, vocab, k, mix, *, dtype="bf16", first=False, done=0.0, banned=False, name=None):
    c = dict(op="beam", requests=requests, beams=beams, vocab=vocab, k=k, mix=mix, dtype=dtype, first=first,
             done=done, banned=banned)
    return dict(c, name=name) if name else c


def _fork(groups, beams, lmin, lmax, own_max, mix, *, first=False, ended=False, name=None):
    c = dict(op="fork", groups=groups, beams=beams, lmin=lmin, lmax=lmax, own_max=own_max, mix=mix, first=first,
             ended=ended)
    return dict(c, name=name) if name else c


def _copy(rows, layers, mix, *, hkv=8, share=0.5, name=None):
    c = dict(op="copy", rows=rows, layers=layers, mix=mix, hkv=hkv, share=share)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one request of 80 s of audio decoded with 4 beams: a call whose latency is what counts
        _shared(1, 4, 4, 1000, 1000, 60, 1, name="shared_1x4_l1000"),
        # one 90-minute recording, 8 beams: its audio prompt is read once instead of 8 times
        _shared(1, 8, 8, 67_500, 67_500, 400, 2, name="shared_1x8_l67500"),
        # 16 concurrent meetings of up to 38 minutes, 4 beams each, some beams not in use
        _shared(16, 4, 4, 5_000, 30_000, 500, 3, empty=True, name="shared_16x4_l30k"),
        # 131 requests of different lengths behind one long instruction, and 3 smaller such sets
        _shared(4, 11, 131, 2_000, 8_000, 900, 4, qscale=4.0, name="shared_4x131_l8000"),
        # the first selection of one request: only its first beam counts
        _beam(1, 4, 151_936, 4, 5, first=True, name="beam_first_1x4"),
        # 16 requests with 5 beams, 10 candidates kept, an odd vocabulary, logits in 32 bits
        _beam(16, 5, 51_865, 10, 6, dtype="fp32", done=0.1, name="beam_16x5_fp32"),
        # a full batch: 64 requests with 8 beams, tokens banned in some rows
        _beam(64, 8, 151_936, 8, 7, done=0.05, banned=True, name="beam_64x8"),
        # one request's prompt handed to its 4 beams
        _fork(1, 4, 1000, 1000, 0, 8, first=True, name="fork_first_1x4"),
        # a full batch in the middle of its transcripts, some requests at their end
        _fork(64, 8, 2_000, 67_500, 500, 9, ended=True, name="fork_64x8_l67500"),
        # one request's 3 copied pages in the 28 layers' pools
        _copy(4, 28, 10, share=0.75, name="copy_4_rows"),
        # a full batch's copies: 512 rows, half of them need one
        _copy(512, 28, 11, name="copy_512_rows"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    mix = rng.randrange(1 << 30)
    kind = rng.choice(["shared", "shared", "shared", "beam", "beam", "beam", "fork", "copy"])
    if kind == "shared":
        groups = _log_int(rng, 1, 32)
        rmax = _log_int(rng, 1, min(150, 512 // groups))
        lmax = _log_int(rng, 1, min(67_500, 200_000 // groups, 2_000_000 // (groups * rmax)))
        return _shared(groups, rng.randint(1, rmax), rmax, rng.randint(1, lmax), lmax,
                       _log_int(rng, 1, min(1000, 30_000 // (groups * rmax))), mix, hkv=rng.choice([8, 8, 4, 2, 1]),
                       empty=rng.random() < 0.3, qscale=rng.choice([1.0, 1.0, 4.0]))
    if kind == "beam":
        beams = rng.choice([1, 2, 3, 4, 5, 8, 10, 16])
        vocab = _log_int(rng, 40, 200_000)
        requests = _log_int(rng, 1, max(1, min(256, 35_000_000 // (beams * vocab))))
        k = rng.choice([beams, beams, 2 * beams, rng.randint(1, 32)])
        return _beam(requests, beams, vocab, k, mix, dtype=rng.choice(["bf16", "fp32"]), first=rng.random() < 0.2,
                     done=rng.choice([0.0, 0.2]), banned=rng.random() < 0.3)
    if kind == "fork":
        beams = rng.choice([1, 2, 3, 4, 5, 8, 16])
        groups = _log_int(rng, 1, 512 // beams)
        lmax = _log_int(rng, 1, 60_000)
        return _fork(groups, beams, rng.randint(1, lmax), lmax, _log_int(rng, 1, 500), mix, first=rng.random() < 0.2,
                     ended=rng.random() < 0.3)
    return _copy(_log_int(rng, 1, 400), rng.randint(1, 28), mix, hkv=rng.choice([8, 8, 4, 2, 1]),
                 share=rng.uniform(0.1, 0.6))


# ----------------------------------------------------------------------------------------------
# what a case fixes on the host
# ----------------------------------------------------------------------------------------------
def _spread(rng, lo, hi, n):
    """n lengths between lo and hi, spread over their logarithm, the first one hi."""
    x = np.clip(np.round(np.exp(rng.uniform(math.log(lo), math.log(hi), n))).astype(np.int64), lo, hi)
    x[0] = hi
    return x


def _shared_host(case):
    """Rows of each group, shared pages of each group, and keys of each row."""
    rng = np.random.Generator(np.random.PCG64(case["mix"]))
    G = case["groups"]
    rows = _spread(rng, case["rmin"], case["rmax"], G)
    prompt = _spread(rng, case["lmin"], case["lmax"], G)
    shared = prompt // PAGE
    group = np.repeat(np.arange(G), rows)
    # a row's own keys: what the prompt has in its last page, and the row's own tokens
    lens = prompt[group] + _spread(rng, 1, case["own_max"], len(group))
    if case["empty"]:
        lens = np.where(rng.random(len(group)) < 0.1, 0, lens)
    return rows, shared, group, lens


def _beam_host(case):
    """Scores and live flags of the beams."""
    rng = np.random.Generator(np.random.PCG64(case["mix"]))
    shape = (case["requests"], case["beams"])
    if case["first"]:
        scores = np.full(shape, -np.inf, np.float32)
        scores[:, 0] = 0.0
        return scores, np.ones(shape, np.int32)
    scores = -np.sort(rng.uniform(0.5, 20.0) + rng.exponential(2.0, shape), axis=1).astype(np.float32)
    live = (rng.random(shape) >= case["done"]).astype(np.int32)
    return scores, live


def _fork_host(case):
    """Parents [G, W], lengths [G, W], and for each row the row whose pages it has up to which page."""
    rng = np.random.Generator(np.random.PCG64(case["mix"]))
    G, W = case["groups"], case["beams"]
    prompt = _spread(rng, case["lmin"], case["lmax"], G)
    if case["first"]:
        lens = np.zeros((G, W), np.int64)
        lens[:, 0] = prompt
        parents = np.zeros((G, W), np.int64)
        kin = np.zeros((G, W), np.int64)
        upto = np.zeros((G, W), np.int64)
    else:
        step = rng.integers(1, case["own_max"], G, endpoint=True)
        lens = np.repeat((prompt + step)[:, None], W, 1)
        ended = rng.random((G, W)) < 0.1  # finished transcripts are shorter
        lens = np.where(ended, prompt[:, None] + rng.integers(0, np.repeat(step[:, None], W, 1)), lens)
        # better beams have more children
        parents = np.minimum(rng.geometric(0.5, (G, W)) - 1, W - 1)
        kin = rng.integers(0, np.maximum(1, np.arange(W)), (G, W))
        first = prompt // PAGE
        last = np.minimum(np.take_along_axis(lens, kin, 1), lens) // PAGE  # only whole pages are shared
        upto = rng.integers(np.repeat(first[:, None], W, 1), last, endpoint=True)
    if case["ended"]:
        parents = np.where(rng.random((G, 1)) < 0.15, -1, parents)
    return parents, lens, kin, upto


def _copy_host(case):
    rng = np.random.Generator(np.random.PCG64(case["mix"]))
    n = rng.integers(1, PAGE, case["rows"])
    n = np.where(rng.random(case["rows"]) < case["share"], n, 0)
    n[-1] = PAGE - 1
    return n


def work(case):
    if case["op"] == "shared":
        rows, shared, group, lens = _shared_host(case)
        hkv = case["hkv"]
        used = np.zeros(len(rows), bool)
        used[group[lens > 0]] = True
        keys = int((shared * PAGE)[used].sum()) + int(np.maximum(lens - shared[group] * PAGE, 0).sum())
        return {"bytes": keys * hkv * DIM * 4 + len(lens) * 2 * hkv * (DIM * 4 + 4),
                "flops": 4 * DIM * 2 * hkv * int(lens.sum())}
    if case["op"] == "beam":
        scores, live = _beam_host(case)
        rows = int(((scores > -np.inf) & (live > 0)).sum())
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": rows * case["vocab"] * size + case["requests"] * (case["beams"] * 8 + case["k"] * 16),
                "flops": 0}
    if case["op"] == "fork":
        parents, lens, kin, upto = _fork_host(case)
        pages = -(-lens // PAGE)
        return {"bytes": 4 * int(pages.sum()) + 32 * lens.size, "flops": 0}
    n = int(_copy_host(case).sum())
    return {"bytes": 2 * 2 * case["layers"] * n * case["hkv"] * DIM * 2, "flops": 0}


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


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return {"shared": _prepare_shared, "beam": _prepare_beam, "fork": _prepare_fork,
            "copy": _prepare_copy}[case["op"]](case, g)


def _prepare_shared(case, g):
    rows, shared, group, lens = _shared_host(case)
    hkv, hq, B = case["hkv"], 2 * case["hkv"], len(lens)
    mine = np.maximum(-(-lens // PAGE) - shared[group], 0)  # pages of a row's own
    num_pages = int(shared.sum() + mine.sum()) + 17
    perm = torch.randperm(num_pages, generator=g, device=DEV).to(torch.int32)
    stride = int((-(-lens // PAGE)).max(initial=1)) + 3
    cell = torch.arange(stride, device=DEV)[None, :]
    sh, first = (torch.from_numpy(x[group]).to(DEV)[:, None] for x in (shared, np.cumsum(shared) - shared))
    own_first = torch.from_numpy(shared.sum() + np.cumsum(mine) - mine).to(DEV)[:, None]
    index = torch.where(cell < sh, first + cell, own_first + cell - sh)
    held = cell < torch.from_numpy(-(-lens // PAGE)).to(DEV)[:, None]
    table = torch.where(held, perm[index.clamp(max=num_pages - 1)], 0).to(torch.int32).contiguous()
    at = np.concatenate([[0], np.cumsum(rows)])
    return dict(
        case=case, q=_randn((B, hq, DIM), g, case["qscale"]), k_pool=_randn((num_pages, PAGE, hkv, DIM), g),
        v_pool=_randn((num_pages, PAGE, hkv, DIM), g), table=table, seq_lens=_i32(lens),
        max_len=int(lens.max()), cu=_i32(at), shared=_i32(shared), max_rows=int(rows.max()),
        bounds=[(int(a), int(b), int(n)) for a, b, n in zip(at[:-1], at[1:], shared * PAGE)],
        own_max=int((lens - shared[group] * PAGE).max()),
        out=torch.empty(B, hq, DIM, dtype=torch.bfloat16, device=DEV),
        lse=torch.empty(B, hq, dtype=torch.float32, device=DEV))


def _prepare_beam(case, g):
    N, W, V = case["requests"], case["beams"], case["vocab"]
    scores, live = _beam_host(case)
    logits = torch.randn(N, W, V, generator=g, device=DEV).mul_(2.5)
    # a model's logits: a few tokens far above the rest
    at = torch.randint(0, V, (N, W, 24), generator=g, device=DEV)
    logits.scatter_add_(2, at, 8.0 * torch.rand(N, W, 24, generator=g, device=DEV))
    if case["banned"]:
        ban = torch.randint(0, V, (N, W, max(1, V // 16)), generator=g, device=DEV)
        logits[::2].scatter_(2, ban[::2], float("-inf"))
    return dict(case=case, logits=logits.to(torch.bfloat16) if case["dtype"] == "bf16" else logits,
                scores=torch.from_numpy(scores).to(DEV) + 0.01 * torch.rand(N, W, generator=g, device=DEV),
                live=torch.from_numpy(live).to(DEV), eos=min(V - 1, 7))


def _prepare_fork(case, g):
    parents, lens, kin, upto = _fork_host(case)
    G, W = lens.shape
    pages = -(-lens // PAGE)
    stride = int(pages.max(initial=1)) + 2
    fresh = np.where(np.arange(W)[None, :] > 0, np.maximum(pages - upto, 0), pages)
    spare = G * W + 5
    num_pages = int(fresh.sum()) + spare
    perm = torch.randperm(num_pages, generator=g, device=DEV).to(torch.int32)
    cell = torch.arange(stride, device=DEV)[None, :]
    base = torch.from_numpy((np.cumsum(fresh.ravel()) - fresh.ravel()).reshape(G, W)).to(DEV)
    n, u, from_row = (torch.from_numpy(x).to(DEV) for x in (pages, upto, kin))
    table = torch.full((G, W, stride), -1, dtype=torch.int32, device=DEV)
    every = torch.arange(G, device=DEV)
    for w in range(W):  # a row has its kin's pages up to a page, then its own
        u_w = u[:, w:w + 1] if w else torch.zeros(G, 1, dtype=torch.int64, device=DEV)
        mine = perm[(base[:, w:w + 1] + cell - u_w).clamp(0, num_pages - 1)]
        row = torch.where(cell < u_w, table[every, from_row[:, w]], mine)
        table[:, w] = torch.where(cell < n[:, w:w + 1], row, -1)
    stack = torch.zeros(num_pages, dtype=torch.int32, device=DEV)
    stack[:spare] = perm[num_pages - spare:]
    e = dict(dtype=torch.int32, device=DEV)
    return dict(case=case, parents=_i32(parents), seq_lens=_i32(lens.ravel()), first=table.view(G * W, stride),
                table=table.view(G * W, stride).clone(), first_stack=stack, stack=stack.clone(),
                count=torch.full((1,), spare, **e), num_pages=num_pages, lens_out=torch.empty(G * W, **e),
                copies=torch.empty(G * W, 3, **e), shared=torch.empty(G, **e), count_out=torch.empty(1, **e))


def _prepare_copy(case, g):
    n = _copy_host(case)
    B, hkv = case["rows"], case["hkv"]
    num_pages = 2 * B + 3
    perm = torch.randperm(num_pages, generator=g, device=DEV).to(torch.int32)
    tokens = _i32(n)
    copies = torch.stack([torch.where(tokens > 0, perm[:B], -1), torch.where(tokens > 0, perm[B:2 * B], -1),
                          tokens], 1).contiguous()
    one = _randn((num_pages, PAGE, hkv, DIM), g)
    # (pools of the layers: shifted copies of one, so that inputs are made quickly)
    pools = [one.roll(i, 0) for i in range(2 * case["layers"])]
    return dict(case=case, copies=copies, pools=pools)


# ----------------------------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s, op)
    return {"shared": _plain_shared, "beam": _plain_beam, "fork": _plain_fork, "copy": _plain_copy}[op](s)


def _own(s, op):
    import long_context_paged_gb300 as pa
    c = s["case"]
    dims = None
    if "hkv" in c and c["hkv"] != 8:
        dims = (2 * c["hkv"], c["hkv"], DIM, PAGE)
    if op == "shared":
        return pa.attn_decode_paged_shared(
            s["q"], s["k_pool"], s["v_pool"], s["table"], s["seq_lens"], s["cu"], s["shared"], s["max_len"], SCALE,
            max_group_rows=s["max_rows"], out=s["out"], lse=s["lse"], dims=dims)
    if op == "beam":
        return tuple(pa.beam_select(s["logits"], s["scores"], c["k"], live=s["live"], eos_token=s["eos"]))
    if op == "fork":
        s["table"].copy_(s["first"])
        s["stack"].copy_(s["first_stack"])
        f = pa.paged_fork(s["parents"], s["seq_lens"], s["table"], s["stack"], s["count"], s["num_pages"],
                          seq_lens_out=s["lens_out"], copies=s["copies"], shared_pages=s["shared"],
                          free_count_out=s["count_out"])
        return f.seq_lens, f.copies, f.shared_pages, f.free_count, s["table"], s["stack"]
    pa.paged_copy_pages(s["copies"], s["pools"], dims=dims)
    return s["pools"]


def _plain_shared(s):
    hkv = s["case"]["hkv"]
    for r0, r1, n in s["bounds"]:  # the groups' prefixes have lengths of their own
        R = r1 - r0
        table, lens = s["table"][r0:r1].long(), s["seq_lens"][r0:r1].long()[:, None]
        last = table.shape[1] - 1
        # the group's pages, from a row that is in use; then each row's own keys, padded to one length
        pages = table.gather(0, lens.argmax(0, keepdim=True).expand(1, table.shape[1]))[0, :n // PAGE]
        j = n + torch.arange(s["own_max"], device=DEV)
        page, slot = table[:, (j // PAGE).clamp(max=last)], (j % PAGE).expand(R, -1)
        q = s["q"][r0:r1].float().view(R, hkv, 2, DIM).permute(1, 0, 2, 3)           # [Hkv, R, 2, D]
        k = s["k_pool"][pages].view(n, hkv, DIM).float().permute(1, 2, 0)             # [Hkv, D, n]
        x = (q.reshape(hkv, 2 * R, DIM) @ k).view(hkv, R, 2, n)
        k = s["k_pool"][page, slot].float().permute(2, 0, 3, 1)                       # [Hkv, R, D, own]
        x = torch.cat([x, q @ k], -1).mul_(SCALE)
        seen = torch.cat([(lens > 0).expand(R, n), j < lens], 1)[None, :, None, :]
        x = x.masked_fill_(~seen, float("-inf"))
        m = x.amax(-1, keepdim=True)
        m = torch.where(torch.isinf(m), 0.0, m)
        x = x.sub_(m).exp_()
        l = x.sum(-1, keepdim=True)
        v = s["v_pool"][pages].view(n, hkv, DIM).float().permute(1, 0, 2)
        o = (x[..., :n].reshape(hkv, 2 * R, n) @ v).view(hkv, R, 2, DIM)
        o += x[..., n:] @ s["v_pool"][page, slot].float().permute(2, 0, 1, 3)
        o /= torch.where(l > 0, l, 1.0)
        s["out"][r0:r1] = o.permute(1, 0, 2, 3).reshape(R, 2 * hkv, DIM)
        s["lse"][r0:r1] = (torch.log(l) + m).permute(1, 0, 2, 3).reshape(R, 2 * hkv)
    return s["out"], s["lse"]


def _plain_beam(s):
    # in 64 bits: candidates of different beams lie close to each other
    N, W, V = s["logits"].shape
    x = s["logits"].double()
    m = x.amax(-1, keepdim=True)
    x = s["scores"].double()[..., None] + (x - m - torch.log(torch.exp(x - m).sum(-1, keepdim=True)))
    token = torch.arange(V, device=DEV)
    done = (s["live"] == 0)[..., None]
    # a finished beam has one candidate, itself
    x = torch.where(done, torch.where(token == s["eos"], s["scores"].double()[..., None], -math.inf), x)
    x = torch.where(torch.isnan(x), -math.inf, x).view(N, W * V)
    scores, index = [], []
    for _ in range(s["case"]["k"]):  # the lowest index of the largest
        best = x.argmax(-1, keepdim=True)
        scores.append(x.gather(1, best))
        index.append(best)
        x.scatter_(1, best, -math.inf)
    scores, index = torch.cat(scores, 1), torch.cat(index, 1)
    none = torch.isinf(scores)
    parents = torch.where(none, -1, index // V)
    tokens = torch.where(none, -1, index % V)
    live = s["live"].long().gather(1, parents.clamp(min=0)) * (tokens != s["eos"]) * ~none
    return scores.float(), parents.int(), tokens.int(), live.int()


def _plain_fork(s):
    s["table"].copy_(s["first"])
    s["stack"].copy_(s["first_stack"])
    G, W = s["parents"].shape
    old, lens, parents = s["table"].view(G, W, -1), s["seq_lens"].view(G, W).long(), s["parents"].long()
    stride = old.shape[2]
    cell = torch.arange(stride, device=DEV)
    held = -(-lens // PAGE)
    row = torch.arange(W, device=DEV)
    # pages of the children before any copy
    at = parents.clamp(min=0)
    n = torch.where(parents >= 0, lens.gather(1, at), 0)
    pages = -(-n // PAGE)
    new = old.gather(1, at[..., None].expand(-1, -1, stride))
    new = torch.where(cell < pages[..., None], new, -1)
    # a child that writes into a page that another one holds too gets a copy, but the first of them
    last = (pages - 1).clamp(min=0)
    mine = new.gather(2, last[..., None])                                     # [G, W, 1]
    theirs = new.gather(2, last[:, None, :].expand(-1, W, -1)).transpose(1, 2)  # [G, W, W]: row b's page of row b'
    there = theirs.eq(mine) & (pages[:, None, :] > last[..., None]) & (row[:, None] != row)
    whole = n[:, None, :] >= PAGE * (last[..., None] + 1)
    copy = (n % PAGE > 0) & (there & ((row < row[:, None]) | whole)).any(-1)
    stack, F, C = s["stack"], s["count"].long(), copy.sum()
    i = copy.flatten().cumsum(0) - 1
    fresh = stack[(F - 1 - i).clamp(min=0)].view(G, W)
    s["copies"].copy_(torch.stack([torch.where(copy, mine[..., 0], -1), torch.where(copy, fresh, -1),
                                   torch.where(copy, (n % PAGE).int(), 0)], -1).view(G * W, 3))
    # pages that no child has: of the rows without children, from the first row that holds the page
    used = (parents[:, None, :] == row[:, None]).any(-1)                      # [G, W]
    own_page = cell < held[..., None]
    gone = own_page & ~used[..., None] & (old >= 0)
    for r in range(W):
        same = (old == old[:, r:r + 1]) & own_page[:, r:r + 1] & (used[:, r, None, None] | (row[:, None] > r))
        gone &= ~same
    give = gone.transpose(1, 2).reshape(-1)                                   # by group, page, row
    to = torch.where(give, F - C + give.cumsum(0) - 1, len(stack))
    grown = torch.cat([stack, stack[:1]]).scatter_(0, to, old.transpose(1, 2).reshape(-1))
    stack.copy_(grown[:-1])
    s["count_out"].copy_(F - C + give.sum())
    # whole pages that all rows in use have
    rows = (n > 0)[..., None]
    one = new.masked_fill(~rows, -1).amax(1, keepdim=True)
    common = ((new == one) & (cell < (n // PAGE)[..., None]) | ~rows).all(1) & rows.any(1)
    s["shared"].copy_(common.long().cumprod(1).sum(1))
    new = torch.where(copy[..., None] & (cell == last[..., None]), fresh[..., None], new)
    old.copy_(torch.where(cell < torch.maximum(held, pages)[..., None], new, old))
    s["lens_out"].copy_(n.flatten())
    return s["lens_out"], s["copies"], s["shared"], s["count_out"], s["table"], s["stack"]


def _plain_copy(s):
    src, dst, n = s["copies"].long().unbind(1)
    slot = torch.arange(PAGE, device=DEV)
    take = slot < n[:, None]
    src = (src[:, None] * PAGE + slot)[take]
    dst = (dst[:, None] * PAGE + slot)[take]
    for pool in s["pools"]:
        rows = pool.view(-1, pool.shape[2] * DIM)
        rows[dst] = rows[src]
    return s["pools"]


# ----------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "shared":
        return _exact_shared(case, seed)
    if case["op"] == "beam":
        return _exact_beam(case, seed)
    if case["op"] == "copy":
        return _exact_copy(case, seed)
    return None  # (a fork's outputs are whole numbers)


def _exact_shared(case, seed):
    s = prepare(case, seed)
    hkv, lens = case["hkv"], s["seq_lens"].tolist()
    out = torch.zeros(len(lens), hkv * 2, DIM, dtype=torch.float64, device=DEV)
    lse = torch.full((len(lens), hkv * 2), -math.inf, dtype=torch.float64, device=DEV)
    if sum(lens) * hkv > 64_000_000:  # (about 20 s)
        return None
    for b, L in enumerate(lens):
        if L == 0:
            continue
        pages = s["table"][b, :-(-L // PAGE)].long()
        keys = s["k_pool"][pages].reshape(-1, hkv, DIM)[:L].double()
        values = s["v_pool"][pages].reshape(-1, hkv, DIM)[:L].double()
        z = SCALE * torch.einsum("hgd,lhd->hgl", s["q"][b].double().view(hkv, 2, DIM), keys)
        total = torch.logsumexp(z, -1)
        out[b] = torch.einsum("hgl,lhd->hgd", torch.exp(z - total[..., None]), values).reshape(2 * hkv, DIM)
        lse[b] = total.reshape(-1)
    return out, lse


def _exact_beam(case, seed):
    s = prepare(case, seed)
    N, W, V = s["logits"].shape
    best = torch.full((N, case["k"]), -math.inf, dtype=torch.float64, device=DEV)
    for i in range(N):
        z = torch.log_softmax(s["logits"][i].double(), -1) + s["scores"][i].double()[:, None]
        stays = s["live"][i] == 0
        z[stays] = -math.inf
        z[stays, s["eos"]] = s["scores"][i][stays].double()
        z = torch.nan_to_num(z, nan=-math.inf, posinf=math.inf, neginf=-math.inf)
        top = torch.sort(z.flatten(), descending=True).values[:case["k"]]
        best[i, :len(top)] = top
    return best, None, None, None


def _exact_copy(case, seed):
    s = prepare(case, seed)
    pools = []
    for pool in s["pools"]:
        x = pool.double()
        for n in range(1, PAGE):  # the copies of n tokens
            some = s["copies"][s["copies"][:, 2] == n].long()
            x[some[:, 1], :n] = pool[some[:, 0], :n].double()
        pools.append(x)
    return pools
