"""The serving calls together, as a scheduler uses them: step plan, rotate-and-append through its slot
map, attention with score options through its table, pages left behind by the window released, all
against the fp64 definitions on the history of every request."""
import numpy as np
import pytest
import torch

from oracle import as_f64
from oracle import serving as S
from tests.helpers import bits
from tests.test_gpu_rope import assert_rounded
from tests.test_gpu_score_decode import close as close_decode
from tests.test_gpu_score_prefill import close as close_prefill

pytestmark = pytest.mark.gpu

HQ, HKV, D = 16, 8, 128
SCALE = D ** -0.5


def dev(a, dtype=torch.int32):
    return torch.tensor(np.asarray(a), dtype=dtype, device="cuda")


class Server:
    """Three requests over one pool; the host keeps each request's appended rows."""

    def __init__(self, pa, prefix, window, softcap, slopes, pages=64, stride=24, seed=0):
        self.pa, self.prefix, self.window, self.softcap, self.slopes = pa, prefix, window, softcap, slopes
        self.B = len(prefix)
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.rng = np.random.default_rng(seed)
        self.num_pages = pages
        nan = torch.full((pages, 16, HKV, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.kp, self.vp = nan.clone(), nan.clone()   # unwritten slots are poison
        self.table = dev(np.full((self.B, stride), -1))
        self.free = dev(self.rng.permutation(pages))
        self.count, self.lens = dev([pages]), dev(np.zeros(self.B))
        self.freq, self.factor = pa.rope_inv_freq(96, 1e5, scaling="yarn", factor=4.0,
                                                  original_max_position=256)
        self.gq = 1 + 0.1 * torch.randn(D, generator=self.gen, device="cuda")
        self.gk = 1 + 0.1 * torch.randn(D, generator=self.gen, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.kh = [np.zeros((0, HKV, D), np.int16) for _ in prefix]
        self.vh = [np.zeros((0, HKV, D), np.int16) for _ in prefix]
        self.prefix_d = dev(prefix)
        self.slopes_d = dev(slopes, torch.float32)

    def project(self, rows):
        return torch.randn(rows, HQ + 2 * HKV, D, generator=self.gen, device="cuda").to(torch.bfloat16)

    def options(self):
        return dict(softcap=self.softcap, window=self.window, alibi_slopes=self.slopes_d,
                    prefix_lens=self.prefix_d, max_prefix_len=int(max(self.prefix)))

    def check(self, new, qkv, qr, out, lse, slots, close):
        """Rotated q and k, appended v, and the attention of this step's rows."""
        at, rows_o, rows_l = 0, [], []
        for b, n in enumerate(new):
            past = len(self.kh[b])
            pos = np.arange(past, past + n)
            raw = qkv[at:at + n]
            s = slots[at:at + n]
            k_now, v_now = self.kp.view(-1, HKV, D)[s], self.vp.view(-1, HKV, D)[s]
            f = self.freq.cpu().numpy()
            for x, g, got in ((raw[:, :HQ], self.gq, qr[at:at + n]), (raw[:, HQ:HQ + HKV], self.gk, k_now)):
                x, g = as_f64(bits(x.contiguous())), g.cpu().numpy()
                y = x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6) * g
                mag = 2 * np.abs(y).max(-1, keepdims=True) * max(1.0, self.factor) if n else 1.0
                assert_rounded(got.contiguous(), S.rope_rows(x, pos, f, False, self.factor, g), mag)
            assert torch.equal(v_now, raw[:, HQ + HKV:])
            self.kh[b] = np.concatenate([self.kh[b], bits(k_now.contiguous())])
            self.vh[b] = np.concatenate([self.vh[b], bits(v_now.contiguous())])
            q = bits(qr[at:at + n].contiguous())
            L = past + n
            o, l = np.zeros((n, HQ, D)), np.zeros((n, HQ))
            for r in range(n):
                vis = S.visible(past + r, L, min(self.prefix[b], L), 0, self.window)
                for h in range(HQ):
                    o[r, h], l[r, h] = S.attend_scored(q[r, h], as_f64(self.kh[b][:, h // 2]),
                                                       as_f64(self.vh[b][:, h // 2]), past + r, vis,
                                                       SCALE, self.softcap, self.slopes[h])
            rows_o.append(o)
            rows_l.append(l)
            at += n
        close(out[:at], lse[:at], np.concatenate(rows_o), np.concatenate(rows_l))

    def leave_window_behind(self):
        """Pages that no later row sees go back: after the prefix, before the window of the next row."""
        lens = np.array([len(k) for k in self.kh])
        begin = -(-np.asarray(self.prefix) // 16)
        end = np.maximum(begin, (lens + 1 - self.window) // 16)
        self.pa.paged_release(dev(begin), dev(end), self.table, self.free, self.count, self.num_pages,
                              free_count_out=self.count, status=self.status)

    def finish(self, b):
        """Request b is done: all it still holds goes back."""
        begin, end = np.zeros(self.B), np.zeros(self.B)
        end[b] = -(-len(self.kh[b]) // 16)
        self.pa.paged_release(dev(begin), dev(end), self.table, self.free, self.count, self.num_pages,
                              free_count_out=self.count, status=self.status)


@pytest.mark.parametrize("stream", [False, True])
def test_chunks_then_decodes_over_a_recycled_pool(cuda_lib, stream):
    s = Server(cuda_lib, [20, 0, 33], 40, 25.0, 2.0 ** (-0.5 * np.arange(1, 17)), pages=26, seed=int(stream))
    st = torch.cuda.Stream() if stream else None
    kw = {} if st is None else dict(stream=st)

    def step(new, decode):
        rows = int(sum(new)) + 3                        # three padding rows behind the last request
        qkv = s.project(rows)
        n = dev(new)
        if st is not None:
            st.wait_stream(torch.cuda.current_stream())
        plan = cuda_lib.paged_step_plan(s.lens, n, s.table, s.free, s.count, s.num_pages, total_rows=rows,
                                        free_count_out=s.count, seq_lens=s.lens, status=s.status, **kw)
        qr = cuda_lib.rope_append_paged(qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:], plan.positions,
                                        plan.slot_map, s.kp, s.vp, s.freq, attn_factor=s.factor,
                                        q_gamma=s.gq, k_gamma=s.gk, status=s.status, **kw)
        bound = max(len(k) for k in s.kh) + max(new)
        if decode:
            out, lse = cuda_lib.attn_decode_paged(qr[:s.B].contiguous() if st is None else qr[:s.B], s.kp,
                                                  s.vp, s.table, plan.seq_lens, bound, SCALE,
                                                  status=s.status, **kw, **s.options())
        else:
            out, lse = cuda_lib.attn_prefill_chunk(qr, plan.cu_new_lens, s.kp, s.vp, s.table, plan.seq_lens,
                                                   max(new), bound, SCALE, status=s.status, **kw,
                                                   **s.options())
        torch.cuda.synchronize()
        assert cuda_lib.read_device_status(s.status) == 0
        s.check(new, qkv, qr, out, lse, plan.slot_map, close_decode if decode else close_prefill)
        s.leave_window_behind()

    step([70, 33, 1], False)
    step([50, 1, 64], False)
    for _ in range(18):
        step([1, 1, 1], True)
    s.finish(0)
    held = (s.table >= 0).sum().item()
    assert s.count.item() + held == s.num_pages
    owned = s.free[:s.count.item()].tolist() + s.table[s.table >= 0].tolist()
    assert sorted(owned) == list(range(s.num_pages))    # every page once


def test_a_decode_step_replayed_as_one_graph(cuda_lib):
    """Plan in place, rotate-and-append, attention: one graph; each replay is the next token."""
    s = Server(cuda_lib, [5, 0, 0], 64, 0.0, np.zeros(16), pages=40, seed=9)
    qkv = s.project(4)
    new, pos = dev([1, 1, 1]), dev(np.zeros(4))
    slots, cu = dev(np.zeros(4), torch.int64), dev(np.zeros(4))
    qr = torch.zeros(4, HQ, D, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.empty(3, HQ, D, dtype=torch.bfloat16, device="cuda"), torch.empty(3, HQ, device="cuda")
    ws = torch.empty(cuda_lib.decode_workspace_size(3, 384), dtype=torch.uint8, device="cuda")

    def step():
        p = cuda_lib.paged_step_plan(s.lens, new, s.table, s.free, s.count, s.num_pages, total_rows=4,
                                     free_count_out=s.count, seq_lens=s.lens, positions=pos, slot_map=slots,
                                     cu_new_lens=cu, status=s.status)
        cuda_lib.rope_append_paged(qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:], p.positions,
                                   p.slot_map, s.kp, s.vp, s.freq, attn_factor=s.factor, q_gamma=s.gq,
                                   k_gamma=s.gk, q_out=qr, status=s.status)
        cuda_lib.attn_decode_paged(qr[:3], s.kp, s.vp, s.table, s.lens, 384, SCALE, out=out, lse=lse,
                                   workspace=ws, status=s.status, window=64, prefix_lens=s.prefix_d,
                                   max_prefix_len=5)
    warm = Server(cuda_lib, [5, 0, 0], 64, 0.0, np.zeros(16), pages=40, seed=9)
    real, s = s, warm
    step()                                              # loads every kernel before the capture
    torch.cuda.synchronize()
    s = real
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(70):
        qkv.copy_(s.project(4))
        g.replay()
        torch.cuda.synchronize()
        assert cuda_lib.read_device_status(s.status) == 0
        s.check([1, 1, 1], qkv, qr, out, lse, slots, close_decode)
    assert s.lens.tolist() == [70, 70, 70] and s.count.item() == 40 - 15
