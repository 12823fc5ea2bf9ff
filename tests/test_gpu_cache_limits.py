"""The paged cache at its stated limits, and its calls captured, replayed and side by side."""
import numpy as np
import pytest
import torch

import step_flow_map_b200 as fmb
from oracle import cache as oc
from test_gpu_cache import DT, World, check_attention, cu_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,dh", [("bf16", 64), ("bf16", 128), ("f32", 64)])
@pytest.mark.parametrize("G", [33, 100, 128])
@pytest.mark.parametrize("rows", [1, 3])
@pytest.mark.parametrize("window,sinks", [(0, 0), (130, 5)])
def test_many_query_heads_per_head(dtype, dh, G, rows, window, sinks):
    w = World([700, 3, 260], 1, dh, 32, dtype, seed=G + rows, weight=True)
    check_attention(w, [rows] * 3, G, window, sinks, accumulate=True, sharp=2.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 5])
def test_as_many_sequences_as_a_call_may_have(dtype, rows):
    rng = np.random.default_rng(rows)
    lens = rng.integers(rows, 90, fmb.FM_MAX_CALL_SEQS).tolist()
    lens[7] = lens[100] = 0
    n = [min(rows, L) for L in lens]
    w = World(lens, 1, 64, 16, dtype, seed=rows, weight=True)
    check_attention(w, n, 8, accumulate=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,G", [(1, 1), (20, 1)])
def test_as_many_heads_as_a_cache_may_have(dtype, rows, G):
    w = World([40, 25], 1024, 64, 16, dtype, seed=rows, weight=True)
    check_attention(w, [rows, rows], G, accumulate=True)


def test_evict_as_many_rows_as_a_call_may_have():
    L = fmb.FM_MAX_EVICT_ROWS
    w = World([L, 100], 1, 64, 128, "bf16", pos=True, weight=True)
    for budget, sinks, recent in ((L - 1, 0, 0), (L // 2, 4, 1000), (3, 1, 1)):
        wt = np.round(np.exp(w.rng.normal(size=(L, 1)) * 2), 1)
        w.put(w.weight, 0, torch.tensor(wt))
        w.put(w.pos, 0, torch.tensor(w.rng.permutation(L)[:, None]))
        old = {n: getattr(w, n).clone() for n in ("k", "v", "pos", "weight")}
        kv = torch.tensor([L, 100], dtype=torch.int32).cuda()
        left = w.cache.evict(kv, kv, budget, max_kv=L, sinks=sinks, recent=recent)
        assert left.cpu().tolist() == [min(x, budget) for x in (L, 100)]
        for b, n in enumerate((L, 100)):
            pos, weight = w.get(old["pos"], b)[:, 0], w.get(old["weight"], b)[:, 0]
            moves = oc.evict(weight, pos, n, budget, sinks, recent)
            if moves:
                P, O = (t.cuda() for t in w.where(b, n))
                to, come = (torch.tensor(m).cuda() for m in zip(*moves))
                for t in old:
                    old[t][P[to], 0, O[to]] = old[t][P[come], 0, O[come]]
        for t in old:
            assert torch.equal(torch.nan_to_num(getattr(w, t), 123.0), torch.nan_to_num(old[t], 123.0)), t
            getattr(w, t).copy_(old[t])


# ------------------------------------------------------------------ a round of all three, captured
class Round:
    """One round of a budgeted cache on buffers that stay: append, attend with weights, cut."""

    def __init__(self, dtype, rows, seed):
        self.B, self.rows, self.budget, hq, hkv, dh = 3, rows, 96, 8, 2, 64
        self.w = w = World([96, 50, 96], hkv, dh, 16, dtype, seed=seed, pos=True, weight=True, extra=rows + 46)
        T = self.B * rows
        self.qkv = torch.zeros(T, hq + 2 * hkv, dh, dtype=DT[dtype]).cuda()
        self.q, self.k, self.v = self.qkv[:, :hq], self.qkv[:, hq:hq + hkv], self.qkv[:, hq + hkv:]
        self.cu, self.kv = cu_of([rows] * self.B), w.kv.clone()
        self.q_pos = torch.zeros(T, dtype=torch.int32).cuda()
        self.next_pos = torch.tensor([400, 50, 97], dtype=torch.int32).cuda()
        self.freq = torch.tensor([0.8 ** i for i in range(16)], dtype=torch.float64).cuda()
        self.gain = torch.ones(dh, dtype=DT[dtype]).cuda()
        self.qr = torch.zeros(T, hq, dh, dtype=DT[dtype]).cuda()
        self.out, self.left = torch.zeros_like(self.qr), torch.zeros_like(self.kv)

    def feed(self, i):
        g = torch.Generator(device="cuda").manual_seed(i)
        self.qkv.copy_(torch.randn(self.qkv.shape, generator=g, device="cuda"))
        self.q_pos.copy_((self.next_pos[:, None] + torch.arange(self.rows, device="cuda")).flatten())
        self.next_pos += self.rows
        self.kv += self.rows

    def run(self, **on):
        c = self.w.cache
        c.append(self.q, self.k, self.v, self.cu, self.kv, q_pos=self.q_pos, q_gain=self.gain, k_gain=self.gain,
                 inv_freq=self.freq, out=self.qr, **on)
        c.attend(self.qr, self.cu, self.kv, max_rows=self.rows, max_kv=self.budget + self.rows, q_pos=self.q_pos, window=200,
                 sinks=4, accumulate=True, out=self.out, **on)
        c.evict(self.kv, self.next_pos, self.budget, max_kv=self.budget + self.rows, sinks=4, recent=8, new_len=self.left, **on)

    def close(self):
        self.kv.copy_(self.left)

    def state(self):
        return [torch.nan_to_num(t.float(), 9.0).clone() for t in
                (self.out, self.qr, self.left, self.w.k, self.w.v, self.w.pos, self.w.weight)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 17, 40])
def test_a_captured_round_follows_its_inputs(dtype, rows):
    eager, played = Round(dtype, rows, 3), Round(dtype, rows, 3)
    first = played.state()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        played.run()
    assert all(torch.equal(a, b) for a, b in zip(played.state(), first)), "the capture ran something"
    for i in range(6):
        for r in (eager, played):
            r.feed(i)
        eager.run()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager.state(), played.state()):
            assert torch.equal(a, b), i
        for r in (eager, played):
            r.close()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rounds_on_two_streams_and_in_two_graphs_at_once(dtype):
    alone, at_once, graphs = ([Round(dtype, 17, s) for s in (1, 2)] for _ in range(3))
    streams = [torch.cuda.Stream() for _ in range(2)]
    played = []
    torch.cuda.synchronize()
    for r, st in zip(graphs, streams):
        played.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(played[-1], stream=st):
            r.run()
    for i in range(5):
        for group in (alone, at_once, graphs):
            for j, r in enumerate(group):
                r.feed(10 * i + j)
        torch.cuda.synchronize()
        for r in alone:
            r.run()
            torch.cuda.synchronize()
        for r, st in zip(at_once, streams):
            r.run(stream=st)
        torch.cuda.synchronize()
        for g, st in zip(played, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for j in range(2):
            for a, b, c in zip(*(group[j].state() for group in (alone, at_once, graphs))):
                assert torch.equal(a, b) and torch.equal(a, c), (i, j)
        for group in (alone, at_once, graphs):
            for r in group:
                r.close()
