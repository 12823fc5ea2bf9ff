"""Forms of the paged cache's calls that combine what other tests take one by one."""
import numpy as np
import pytest
import torch

import step_flow_map_b200 as fmb
from oracle import cache as oc
from test_gpu_cache import World, check_attention, cu_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 4, 17, 150])
@pytest.mark.parametrize("window,sinks", [(0, 0), (60, 3), (200, 40)])
def test_weights_under_a_window_of_stored_positions(dtype, rows, window, sinks):
    """Width 128, positions in any order and of each head its own."""
    lens = [500, 155, 160]
    w = World(lens, 2, 128, 32, dtype, seed=rows + window, pos=True, weight=True)
    for b, L in enumerate(lens):
        w.put(w.pos, b, torch.tensor(np.stack([w.rng.permutation(L) * (b + 1) for _ in range(2)], 1)))
    q_pos = np.concatenate([np.sort(w.rng.integers(0, L * (b + 1), rows)) for b, L in enumerate(lens)])
    check_attention(w, [rows] * 3, 4, window, sinks, q_pos=q_pos, accumulate=True)


@pytest.mark.parametrize("max_kv,budget", [(500, 64), (500, 499), (400, 600), (64, 64)])
def test_evict_cuts_a_sequence_longer_than_max_kv(max_kv, budget):
    """Its rows from max_kv on are dropped, whatever their weight; the others go by the rule."""
    lens = [700, 30, 500]
    w = World(lens, 2, 64, 16, "bf16", seed=budget, pos=True, weight=True)
    old = {n: getattr(w, n).clone() for n in ("k", "v", "pos", "weight")}
    left = w.cache.evict(w.kv, w.kv, budget, max_kv=max_kv, sinks=4, recent=8)
    assert left.cpu().tolist() == [min(L, max_kv, budget) for L in lens]
    for b, L in enumerate(lens):
        cut = min(L, max_kv)
        pos, wt = w.get(old["pos"], b, cut), w.get(old["weight"], b, cut)
        P, O = (t.cuda() for t in w.where(b, L))
        for h in range(2):
            for to, come in oc.evict(wt[:, h], pos[:, h], L, budget, 4, 8):
                for n in old:
                    old[n][P[to], h, O[to]] = old[n][P[come], h, O[come]]
    for n in old:
        assert torch.equal(torch.nan_to_num(getattr(w, n), 123.0), torch.nan_to_num(old[n], 123.0)), n


def test_evict_takes_lengths_side_by_side():
    """Old and new lengths and the positions as parts of one tensor."""
    lens = [100, 30, 75, 64]
    w = World(lens, 2, 64, 16, "bf16", pos=True, weight=True)
    for order in ((0, 1, 2), (2, 0, 1), (1, 2, 0)):
        box = torch.zeros(3, 4, dtype=torch.int32).cuda()
        box[order[0]], box[order[1]] = w.kv, w.kv
        left = w.cache.evict(box[order[0]], box[order[1]], 64, max_kv=100, sinks=4, recent=8, new_len=box[order[2]])
        assert left.cpu().tolist() == [64, 30, 64, 64]


FEW = [(1, 4), (2, 8), (3, 5)]   # new rows, query heads per key/value head: at most 16 packed rows


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,G", FEW)
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 3)])
@pytest.mark.parametrize("pos", [False, True])
def test_kept_scores_take_what_the_cache_holds_whatever_max_kv_says(dtype, rows, G, window, sinks, pos):
    B, most = 9, 2 ** 24
    w = World([130, 0, 600, 141, 7, 16, 17, 64, 65], 2, 64, 16, dtype, seed=rows, pos=pos, weight=True)
    n = [min(rows, L) for L in w.lens]
    a = fmb.fm_attention_args(T=sum(n), B=B, n_heads=2 * G, max_rows=rows, max_kv=most, accumulate=0)
    plain = fmb.fm_cache_attention_workspace(w.cache._c, a)
    a.accumulate = 1
    extra = fmb.fm_cache_attention_workspace(w.cache._c, a) - plain
    assert 0 < extra <= 2 * (w.k.shape[0] * 16 + B * 64) * rows * G * 4 + sum(n) * 2 * G * 4 + 512
    q_pos = np.concatenate([np.arange(L - m, L) for L, m in zip(w.lens, n)]) if pos else None
    check_attention(w, n, G, window, sinks, q_pos=q_pos, accumulate=True, max_kv=most)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,G", FEW)
@pytest.mark.parametrize("window,sinks", [(0, 0), (2500, 40)])
def test_weights_of_lengths_past_the_rows_that_the_cache_has(dtype, rows, G, window, sinks):
    """Most pages of the tables do not exist; there is no room for the scores of the last units."""
    lens = [3000, 2900]
    w = World(lens, 2, 64, 16, dtype, seed=rows, weight=True)
    m, (cache_k, cache_v, cache_w) = 30, (w.k, w.v, w.weight)
    keep = w.rng.permutation(sum(w.pages))[:m].tolist()          # pages that go on to exist, numbered anew
    owned = [int(p) for row, c in zip(w.table, w.pages) for p in row[:c]]
    new = {owned[i]: j for j, i in enumerate(keep)}
    idx = torch.tensor([p for p, _ in sorted(new.items(), key=lambda x: x[1])]).cuda()
    w.k, w.v, w.weight = (t[idx].contiguous() for t in (cache_k, cache_v, cache_w))
    full = w.table.copy()
    w.table = np.array([[new.get(int(p), -1) for p in row] for row in full], np.int32)
    there = [(w.table[b, np.arange(L) // 16] >= 0) for b, L in enumerate(lens)]
    assert all(t.any() and not t.all() for t in there)
    w.t = torch.tensor(w.table).cuda()
    w.cache = type(w.cache)(w.k, w.v, w.t, weight=w.weight)
    a = fmb.fm_attention_args(T=2 * rows, B=2, n_heads=2 * G, max_rows=rows, max_kv=3000, accumulate=1)
    assert fmb.fm_cache_attention_workspace(w.cache._c, a) < 2 ** 23
    # (World reads rows of pages that do not exist as those of the last page; the oracle masks them)
    check_attention(w, [rows] * 2, G, window, sinks, accumulate=False, there=there)
    had = w.weight.clone()
    q = torch.tensor(w.rng.normal(size=(2 * rows, 2 * G, 64))).to(w.k.dtype).cuda()
    cu = torch.tensor([0, rows, 2 * rows], dtype=torch.int32).cuda()
    w.cache.attend(q, cu, w.kv, max_rows=rows, max_kv=3000, window=window, sinks=sinks, accumulate=True)
    got = (w.weight - had).double().cpu().numpy()
    want = np.zeros_like(got)
    for b, L in enumerate(lens):
        k, v = np.nan_to_num(w.get(w.k, b)), np.nan_to_num(w.get(w.v, b))
        _, _, wt, _, _ = oc.attention(q[b * rows:(b + 1) * rows].double().cpu().numpy(), k, v, np.arange(L - rows, L),
                                      np.arange(L)[:, None].repeat(2, 1), 64 ** -0.5, window, sinks, there[b])
        for r in np.flatnonzero(there[b]):
            want[w.table[b, r // 16], :, r % 16] += wt[r]
    # p off by 4 d = 2^-21 (dh + 8) big + 2^-18 relatively, with sum |q k| scale below 32: 2^-9.8; the weight is rounded once
    assert (np.abs(got - want) <= 2.0 ** -9.8 * (want + 1e-7) + 2.0 ** -22).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G", [2, 8])
def test_weights_of_accepted_rows_alone(dtype, G):
    """A scored block whose drafts are accepted in part: attended without weights, and the rows that
    stay once more with them.  The rejected rows leave no weight behind, and the next block takes
    their places."""
    rows, lens, accepted = 17, [150, 90, 133], [5, 17, 1]
    w = World(lens, 2, 64, 16, dtype, seed=G, weight=True)
    q = torch.tensor(w.rng.normal(size=(3 * rows, 2 * G, 64))).to(w.k.dtype).cuda()
    cu = cu_of([rows] * 3)
    before = [w.get(w.weight, b) for b in range(3)]
    full = w.cache.attend(q, cu, w.kv, max_rows=rows, max_kv=150)
    for b in range(3):
        assert np.array_equal(w.get(w.weight, b), before[b])
    kept = torch.cat([q[b * rows:b * rows + n] for b, n in enumerate(accepted)])
    short = [L - rows + n for L, n in zip(lens, accepted)]
    again = w.cache.attend(kept, cu_of(accepted), torch.tensor(short, dtype=torch.int32).cuda(), max_rows=rows, max_kv=150,
                           accumulate=True)
    at = 0
    for b, (L, n) in enumerate(zip(short, accepted)):
        k, v = (w.get(t, b, L) for t in (w.k, w.v))
        o, _, wt, mag, _ = oc.attention(q[b * rows:b * rows + n].double().cpu().numpy(), k, v, np.arange(L - n, L),
                                        np.arange(L)[:, None].repeat(2, 1), 64 ** -0.5)
        # scores off by d = 2^-23 (dh + 8) 32 + 2^-20 < 2^-11.8 (sum |q k| scale below 32), p by 4 d; outputs as in
        # the attention tests: 2 u and 4 d of sum p |v|, one rounding
        u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
        for got in (full[b * rows:b * rows + n], again[at:at + n]):
            assert (np.abs(got.double().cpu().numpy() - o) <= u * np.abs(o) + (2 * u + 2.0 ** -9.8) * mag).all()
        gain = w.get(w.weight, b) - before[b]
        assert (np.abs(gain[:L] - wt) <= 2.0 ** -9.8 * (wt + 1e-7) + 2.0 ** -22 * (1 + wt)).all() and (gain[L:] == 0).all()
        at += n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 3, 12, 60])
def test_a_query_whose_scores_are_all_minus_infinity(dtype, rows):
    """It gets zeros and gives no weight, as one that sees nothing; the others go on without it."""
    w = World([200, 90], 2, 64, 16, dtype, seed=rows, weight=True)
    for b, L in enumerate(w.lens):
        k = torch.tensor(w.get(w.k, b))
        k[..., 0] = k[..., 0].abs() + 0.1
        w.put(w.k, b, k)
    q = torch.tensor(w.rng.normal(size=(2 * rows, 8, 64))).to(w.k.dtype).cuda()
    cu, args = cu_of([rows] * 2), dict(max_rows=rows, max_kv=200, lse=True)
    had = w.weight.clone()
    want, wl = w.cache.attend(q, cu, w.kv, accumulate=True, **args)
    all_heads = torch.nan_to_num(w.weight - had)
    bad = q.clone()
    bad[rows - 1, 5, 0] = -float("inf")
    w.weight.copy_(had)
    got, gl = w.cache.attend(bad, cu, w.kv, accumulate=True, **args)
    assert (got[rows - 1, 5] == 0).all() and gl[rows - 1, 5] == -float("inf")
    got[rows - 1, 5], gl[rows - 1, 5] = want[rows - 1, 5], wl[rows - 1, 5]
    assert torch.equal(got, want) and torch.equal(gl, wl)
    gain = torch.nan_to_num(w.weight - had, nan=-9.0)
    # its head's rows lose its one unit of weight, no other row changes (fp32 sums of 200 terms below 61)
    assert (gain >= 0).all() and (gain <= all_heads + 1e-4).all()
    lost = (all_heads - gain).sum((0, 2)).cpu()
    assert abs(lost[1] - 1) < 1e-2 and lost[0].abs() < 1e-4
