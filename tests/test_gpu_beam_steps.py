"""Beam search over the paged cache as a scheduler runs it: selection, fork of the tables, page copies in all
layers, step plan, append, attention over the shared pages; step by step, and as one captured graph. The
host keeps every beam's own history; selection, tables and attention are held against it."""
import numpy as np
import pytest
import torch

from oracle import as_f64, attend_rows
from oracle import beam as O
from tests.helpers import bits

pytestmark = pytest.mark.gpu
HQ, HKV, D = 16, 8, 128
SCALE = D ** -0.5
V, EOS = 60, 3


def dev(a, dtype=torch.int32):
    return torch.tensor(np.asarray(a), dtype=dtype, device="cuda")


class Search:
    def __init__(self, pa, prompts, beams, pages, stride, layers=2, seed=0):
        self.pa, self.G, self.W, self.pages = pa, len(prompts), beams, pages
        self.B = self.G * beams
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        nan = torch.full((pages, 16, HKV, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.k = [nan.clone() for _ in range(layers)]
        self.v = [nan.clone() for _ in range(layers)]
        self.table = dev(np.full((self.B, stride), -1))
        self.free = dev(np.random.default_rng(seed).permutation(pages))
        self.count, self.lens = dev([pages]), dev(np.zeros(self.B))
        self.scores = dev([[0.0] + [-np.inf] * (beams - 1)] * self.G, torch.float32)
        self.live = dev(np.ones((self.G, beams)))
        self.cu = dev(np.arange(self.G + 1) * beams)
        self.freq = torch.zeros(64, dtype=torch.float64, device="cuda")   # angles of 0: rows as they are
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        # buffers of a step
        self.logits = torch.zeros(self.G, beams, V, device="cuda")
        self.qkv = torch.zeros(layers, self.B, HQ + 2 * HKV, D, dtype=torch.bfloat16, device="cuda")
        self.out = [torch.zeros(self.B, HQ, D, dtype=torch.bfloat16, device="cuda") for _ in range(layers)]
        self.lse = [torch.zeros(self.B, HQ, device="cuda") for _ in range(layers)]
        self.history = [[(np.zeros((0, HKV, D), np.int16),) * 2 for _ in range(self.B)] for _ in range(layers)]
        # prompts: in the first row of each group
        new = np.zeros(self.B, int)
        new[::beams] = prompts
        plan = pa.paged_step_plan(self.lens, dev(new), self.table, self.free, self.count, pages,
                                  total_rows=int(new.sum()), free_count_out=self.count, seq_lens=self.lens,
                                  status=self.status)
        for layer in range(layers):
            rows = self.random(int(new.sum()), 2 * HKV)
            at = 0
            for g, n in enumerate(prompts):
                s = plan.slot_map[at:at + n]
                kk, vv = rows[at:at + n, :HKV].contiguous(), rows[at:at + n, HKV:].contiguous()
                self.k[layer].view(-1, HKV, D)[s], self.v[layer].view(-1, HKV, D)[s] = kk, vv
                self.history[layer][g * beams] = bits(kk), bits(vv)
                at += n

    def random(self, *shape):
        return torch.randn(*shape, D, generator=self.gen, device="cuda").clamp(-5.9, 5.9).to(torch.bfloat16)

    def draw(self):
        self.logits.copy_(2 * torch.randn(self.G, self.W, V, generator=self.gen, device="cuda"))
        self.logits[..., EOS] += 1.0
        self.qkv.copy_(self.random(*self.qkv.shape[:3]))

    def step(self):
        """One step, from the logits and the projections of the new tokens; all buffers in place."""
        pa = self.pa
        self.chosen = pa.beam_select(self.logits, self.scores, self.W, live=self.live, eos_token=EOS,
                                     out_scores=self.scores, live_out=self.live)
        fork = pa.paged_fork(self.chosen.parents, self.lens, self.table, self.free, self.count, self.pages,
                             seq_lens_out=self.lens, free_count_out=self.count, status=self.status)
        pa.paged_copy_pages(fork.copies, self.k + self.v, status=self.status)
        plan = pa.paged_step_plan(self.lens, self.live.view(-1), self.table, self.free, self.count, self.pages,
                                  total_rows=self.B, free_count_out=self.count, seq_lens=self.lens,
                                  status=self.status)
        # packed rows are the live beams'
        t = torch.arange(self.B, device="cuda")
        row = (torch.searchsorted(plan.cu_new_lens, t, right=True) - 1).clamp(max=self.B - 1)
        packed = plan.cu_new_lens[:-1].long().clamp(max=self.B - 1)
        for layer in range(len(self.k)):
            x = self.qkv[layer][row]
            q = pa.rope_append_paged(x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:], plan.positions, plan.slot_map,
                                     self.k[layer], self.v[layer], self.freq, status=self.status)
            q = torch.where(self.live.view(-1, 1, 1) > 0, q[packed], self.qkv[layer][:, :HQ])
            pa.attn_decode_paged_shared(q.contiguous(), self.k[layer], self.v[layer], self.table, self.lens, self.cu,
                                        fork.shared_pages, 16 * self.table.shape[1], SCALE, max_group_rows=self.W,
                                        out=self.out[layer], lse=self.lse[layer], status=self.status)
        self.fork = fork

    def check(self, before):
        """What the step came to, against the host's account of it."""
        scores, live, lens = before
        (s, p, t, a), _ = O.select(self.logits.cpu().numpy(), scores, self.W, live, EOS)
        assert np.array_equal(self.chosen.parents.cpu().numpy(), p) and np.array_equal(self.chosen.tokens.cpu().numpy(), t)
        assert np.array_equal(self.live.cpu().numpy(), a)
        assert np.allclose(self.scores.cpu().numpy(), s, rtol=2.0 ** -24, atol=2.0 ** -18)
        assert self.pa.read_device_status(self.status) == 0
        want = [0 if p[b // self.W, b % self.W] < 0 else lens[b // self.W * self.W + p[b // self.W, b % self.W]]
                + a[b // self.W, b % self.W] for b in range(self.B)]
        assert self.lens.tolist() == want
        for layer in range(len(self.k)):
            old, x = self.history[layer], self.qkv[layer]
            self.history[layer] = []
            for b in range(self.B):
                g, parent = b // self.W * self.W, int(p[b // self.W, b % self.W])
                kh, vh = old[g + parent] if parent >= 0 else (np.zeros((0, HKV, D), np.int16),) * 2
                if a[b // self.W, b % self.W]:
                    kh = np.concatenate([kh, bits(x[b:b + 1, HQ:HQ + HKV].contiguous())])
                    vh = np.concatenate([vh, bits(x[b:b + 1, HQ + HKV:].contiguous())])
                self.history[layer].append((kh, vh))
                n = len(kh)
                assert n == want[b]
                pages = self.table[b, :-(-n // 16)].long()
                assert np.array_equal(bits(self.k[layer][pages].reshape(-1, HKV, D)[:n].contiguous()), kh)
                assert np.array_equal(bits(self.v[layer][pages].reshape(-1, HKV, D)[:n].contiguous()), vh)
                q, o = as_f64(bits(x[b, :HQ].contiguous())), as_f64(bits(self.out[layer][b]))
                for h in range(HQ):
                    if n == 0:
                        assert not o[h].any()
                        continue
                    K, Vv = as_f64(kh[:, h // 2]), as_f64(vh[:, h // 2])
                    ref, lse = attend_rows(q[h][None], K, Vv, [n], SCALE)
                    mag, _ = attend_rows(q[h][None], K, np.abs(Vv), [n], SCALE)
                    assert (np.abs(o[h] - ref[0]) <= 2.0 ** -8 * (np.abs(ref[0]) + mag[0]) + 6 * 2.0 ** -13).all()
                    assert abs(self.lse[layer][b, h].item() - lse[0]) <= 2.0 ** -13 + 2.0 ** -23 * abs(lse[0])
        # every page is free or held, and only rows of one group hold it, at one place
        count = self.count.item()
        held = {}
        for b, n in enumerate(want):
            for j, e in enumerate(self.table[b, :-(-n // 16)].tolist()):
                assert held.setdefault(e, (b // self.W, j)) == (b // self.W, j)
        assert sorted(self.free[:count].tolist() + list(held)) == list(range(self.pages))

    def before(self):
        return self.scores.cpu().numpy().copy(), self.live.cpu().numpy().copy(), self.lens.cpu().numpy().copy()

    def end(self):
        """The transcripts are done: all pages go back."""
        self.pa.paged_fork(torch.full((self.G, self.W), -1, dtype=torch.int32, device="cuda"), self.lens, self.table,
                           self.free, self.count, self.pages, seq_lens_out=self.lens, free_count_out=self.count,
                           status=self.status)
        assert self.pa.read_device_status(self.status) == 0
        assert sorted(self.free[:self.count.item()].tolist()) == list(range(self.pages))


@pytest.mark.parametrize("prompts,beams,steps", [((37, 70), 3, 22), ((16,), 5, 18), ((130, 1, 48), 2, 10)])
def test_step_by_step(cuda_lib, prompts, beams, steps):
    s = Search(cuda_lib, prompts, beams, pages=90, stride=14, seed=beams)
    for _ in range(steps):
        s.draw()
        before = s.before()
        s.step()
        torch.cuda.synchronize()
        s.check(before)
    s.end()


def test_one_graph_replayed(cuda_lib):
    warm = Search(cuda_lib, (40, 70), 4, pages=90, stride=14, seed=9)
    warm.draw()
    warm.step()                     # loads every kernel before the capture
    s = Search(cuda_lib, (40, 70), 4, pages=90, stride=14, seed=10)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.step()
    for _ in range(20):
        s.draw()
        before = s.before()
        g.replay()
        torch.cuda.synchronize()
        s.check(before)
    s.end()
