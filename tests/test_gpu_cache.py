"""The paged-cache operators on the GPU against their fp64 oracle.

Tolerances count roundings (u = eps / 2 of the type: bf16 2^-8, fp32 2^-24):

* attention: the output is rounded once (u |o|); with A = sum p |v|, bf16
  probabilities enter the products rounded (u A) and, as the sum that divides
  may be taken over the unrounded ones, shift the quotient by up to u A more;
  a score is a dh-term fp32 sum and its exponential, off by at most
  d = 2^-23 (dh + 8) max sum |q k| scale + 2^-20 absolutely, so p by about d
  relatively, numerator and denominator both (2 d A, taken as 4 d A); the
  row's sums are fp32 over L terms in runs (2^-24 (64 + L / 8) A).
* lse: d plus the sum's error, relative to 1, plus u_32 |lse| for its rounding.
* weights: p's error times the weight, plus fp32 sums over the new rows.
* append: the norm and the turned pair are fp32 (8 roundings and an angle good
  to 2^-22), the result is rounded once.
* evict: exact.
"""
import math

import numpy as np
import pytest
import torch

from oracle import cache as oc

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def host():
    from step_flow_map_b200 import host as h
    return h


class World:
    """Sequences in a paged cache with shuffled pages; everything no sequence owns is NaN."""

    def __init__(self, lens, hkv, dh, page, dtype, seed=0, pos=False, weight=False, spare=2, extra=0):
        self.rng = np.random.default_rng(seed)
        self.lens, self.hkv, self.dh, self.page, self.dtype = list(lens), hkv, dh, page, dtype
        self.pages = [-(-(L + extra) // page) for L in lens]
        n = sum(self.pages) + spare
        order = self.rng.permutation(n)
        self.table = np.full((len(lens), max(1, max(self.pages)) + 1), -1, np.int32)
        at = 0
        for b, c in enumerate(self.pages):
            self.table[b, :c] = order[at:at + c]
            at += c
        nan = torch.full((n, hkv, page, dh), float("nan"))
        self.k, self.v = nan.clone().to(DT[dtype]).cuda(), nan.clone().to(DT[dtype]).cuda()
        self.pos = torch.full((n, hkv, page), -7, dtype=torch.int32).cuda() if pos else None
        self.weight = torch.zeros(n, hkv, page).cuda() if weight else None
        for b, L in enumerate(lens):
            self.put(self.k, b, torch.tensor(self.rng.normal(size=(L, hkv, dh))))
            self.put(self.v, b, torch.tensor(self.rng.normal(size=(L, hkv, dh)) + 0.3))
            if pos:
                self.put(self.pos, b, torch.arange(L)[:, None].expand(L, hkv))
            if weight:
                self.put(self.weight, b, torch.tensor(self.rng.random((L, hkv))))
        self.t = torch.tensor(self.table).cuda()
        self.cache = host().PagedCache(self.k, self.v, self.t, pos=self.pos, weight=self.weight)
        self.kv = torch.tensor(self.lens, dtype=torch.int32).cuda()

    def where(self, b, L):
        r = torch.arange(L)
        return torch.tensor(self.table[b].astype(np.int64))[r // self.page], r % self.page

    def put(self, buf, b, rows):
        p, o = self.where(b, rows.shape[0])
        buf[p.cuda(), :, o.cuda()] = rows.to(buf.dtype).cuda()

    def get(self, buf, b, L=None):
        p, o = self.where(b, self.lens[b] if L is None else L)
        return buf[p.cuda(), :, o.cuda()].double().cpu().numpy()


def cu_of(rows):
    return torch.tensor(np.concatenate([[0], np.cumsum(rows)]), dtype=torch.int32).cuda()


def check_attention(w, rows, G, window=0, sinks=0, q_pos=None, accumulate=False, tail=2, max_rows=None,
                    there=None, sharp=1.0, strided=False, run=None, max_kv=None):
    hq, dh, T = w.hkv * G, w.dh, sum(rows)
    q = torch.tensor(w.rng.normal(size=(T + tail, hq, dh)) * sharp).to(DT[w.dtype]).cuda()
    out = torch.full((T + tail, hq, dh), 77.0, dtype=DT[w.dtype]).cuda()
    if strided:   # rows inside a wider buffer
        wide = torch.full((T + tail, hq + 3, dh), 55.0, dtype=DT[w.dtype]).cuda()
        wide[:, :hq] = q
        q = wide[:, :hq]
        out = torch.full((T + tail, hq + 1, dh), 77.0, dtype=DT[w.dtype]).cuda()[:, :hq]
    pq = None
    if q_pos is not None:
        pq = torch.tensor(np.concatenate([q_pos, np.zeros(tail)]), dtype=torch.int32).cuda()
    before = w.weight.clone() if w.weight is not None else None
    args = dict(max_rows=max_rows or max(1, max(rows)), max_kv=max_kv or max(1, max(w.lens)), q_pos=pq, window=window,
                sinks=sinks, accumulate=accumulate, lse=True, out=out)
    got, lse = (run or (lambda: w.cache.attend(q, cu_of(rows), w.kv, **args)))()
    again, lse2 = w.cache.attend(q, cu_of(rows), w.kv, **{**args, "accumulate": False, "out": torch.empty_like(out)})
    assert torch.equal(got[:T], again[:T]) and torch.equal(lse[:T], lse2[:T]), "two runs differ"
    assert (got[T:] == 77.0).all(), "rows behind the last sequence were written"
    scale, u, at = dh ** -0.5, U[w.dtype], 0
    g64, l64, q64 = got.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().cpu().numpy()
    for b, n in enumerate(rows):
        L = w.lens[b]
        k, v = np.nan_to_num(w.get(w.k, b)), np.nan_to_num(w.get(w.v, b))
        pk = w.get(w.pos, b) if w.pos is not None else np.arange(L)[:, None].repeat(w.hkv, 1)
        mine = q_pos[at:at + n] if q_pos is not None else np.arange(L - n, L)
        o, ls, wt, mag, big = oc.attention(q64[at:at + n], k, v, mine, pk, scale, window, sinks,
                                           there[b] if there is not None else None)
        d = 2.0 ** -23 * (dh + 8) * big + 2.0 ** -20
        sums = 2.0 ** -24 * (64 + L / 8)
        tol = u * np.abs(o) + ((2 * u if w.dtype == "bf16" else 0) + 4 * d + sums) * mag + 1e-30
        err = np.abs(g64[at:at + n] - o)
        assert (err <= tol).all(), f"seq {b}: out off by {(err / tol).max():.3g} of the bound"
        seen = np.isfinite(ls)
        assert (np.isfinite(l64[at:at + n]) == seen).all() and (l64[at:at + n][~seen] == -np.inf).all()
        le = np.abs(l64[at:at + n][seen] - ls[seen])
        assert (le <= 2 * d + sums + 2.0 ** -23 * np.abs(ls[seen])).all(), f"seq {b}: lse off by {le.max():.3g}"
        if accumulate:
            had, has = (np.where(np.isnan(x), 0, x) for x in (w.get(before, b), w.get(w.weight, b)))
            we = np.abs(has - had - wt)
            assert (we <= (4 * d + sums + 2.0 ** -24 * (n * G + 8)) * (wt + 1e-7) + 2.0 ** -23 * (had + wt)).all(), \
                f"seq {b}: weight off by {we.max():.3g}"
        at += n
    if accumulate:   # rows of no sequence keep their bits
        owned = torch.zeros(w.weight.shape, dtype=torch.bool)
        for b, L in enumerate(w.lens):
            p, o = w.where(b, L)
            owned[p, :, o] = True
        assert torch.equal(w.weight.cpu()[~owned], before.cpu()[~owned])
    return got, lse


TYPES = [("bf16", 64), ("bf16", 128), ("f32", 32), ("f32", 64), ("f32", 128)]


@pytest.mark.parametrize("dtype,dh", TYPES)
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("G", [1, 4, 5, 16])
def test_one_token_over_ragged_lengths(dtype, dh, page, G):
    w = World([1, 0, 15, 16, 17, 63, 64, 65, 300], 2, dh, page, dtype, seed=page + G)
    check_attention(w, [1, 0, 1, 1, 1, 1, 1, 1, 1], G)


@pytest.mark.parametrize("dtype,dh", TYPES)
@pytest.mark.parametrize("rows,lens", [([17, 3, 0, 17], [17, 40, 9, 200]), ([33, 1, 2], [33, 129, 258]),
                                       ([130], [130]), ([70, 201], [333, 201])])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (7, 3), (64, 20), (1000, 4)])
def test_blocks_and_prompts(dtype, dh, rows, lens, window, sinks):
    w = World(lens, 2, dh, 32, dtype, seed=window + len(rows))
    check_attention(w, rows, 3, window, sinks)


@pytest.mark.parametrize("dtype,dh", [("bf16", 128), ("f32", 64)])
@pytest.mark.parametrize("rows", [1, 17, 257])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 5), (513, 130)])
def test_long_caches_are_split_and_joined(dtype, dh, rows, window, sinks):
    w = World([5000, 1700], 2, dh, 64, dtype, seed=rows)
    check_attention(w, [rows, rows], 4, window, sinks, sharp=3.0, strided=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 17, 150])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3)])
def test_stored_positions_decide(dtype, rows, window, sinks):
    """Rows in any order; each head its own; some queries see nothing."""
    lens = [200, 155, 160]
    w = World(lens, 3, 64, 16, dtype, seed=rows, pos=True, weight=True)
    for b, L in enumerate(lens):
        p = np.stack([w.rng.permutation(L) for _ in range(3)], 1) + (1000 if b == 1 else 0)
        w.put(w.pos, b, torch.tensor(p))
    q_pos = np.concatenate([np.arange(L - rows, L) for L in lens])   # sequence 1's rows all lie in the future
    q_pos[-1] = 2 ** 31 - 1
    _, lse = check_attention(w, [rows] * 3, 2, window, sinks, q_pos=q_pos, accumulate=True)
    assert (lse[rows:2 * rows] == -math.inf).all()


@pytest.mark.parametrize("dtype,dh", [("bf16", 64), ("bf16", 128), ("f32", 128)])
@pytest.mark.parametrize("rows,G", [(1, 4), (1, 1), (3, 5), (17, 4), (140, 2)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 6)])
def test_weights_add_up(dtype, dh, rows, G, window, sinks):
    w = World([140, 600, 141, 0], 2, dh, 32, dtype, seed=rows, weight=True)
    check_attention(w, [rows, rows, rows, 0], G, window, sinks, accumulate=True, sharp=2.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 40])
def test_more_rows_than_the_cache_holds_see_nothing_before_it(dtype, rows):
    """A sequence shorter than its new rows: the first of them lie before row 0."""
    w = World([7, 0, 64], 1, 64, 16, dtype)
    _, lse = check_attention(w, [rows + 7, rows, 64], 8)
    assert (lse[:rows] == -math.inf).all() and (lse[rows + 7:2 * rows + 7] == -math.inf).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 30])
def test_pages_that_do_not_exist_hold_no_rows(dtype, rows):
    w = World([150, 100, 90], 2, 64, 16, dtype, weight=True)
    bad = {0: [0, 3], 1: [6], 2: list(range(6))}
    there = [np.ones(L, bool) for L in w.lens]
    t = w.t.clone()
    for b, ps in bad.items():
        for i, p in enumerate(ps):
            t[b, p] = [-1, w.k.shape[0], 2 ** 31 - 1][i % 3]
            there[b][p * 16:(p + 1) * 16] = False
    w.cache.page_table = t
    _, lse = check_attention(w, [rows] * 3, 4, there=there, accumulate=True)
    assert (lse[2 * rows:3 * rows] == -math.inf).all()


def test_rows_past_max_rows_are_not_computed():
    w = World([90, 90], 2, 128, 16, "bf16")
    q = torch.randn(12, 8, 128, device="cuda").bfloat16()
    out = torch.full_like(q, 77.0)
    w.cache.attend(q, cu_of([6, 6]), w.kv, max_rows=4, max_kv=90, out=out)
    full = w.cache.attend(q, cu_of([6, 6]), w.kv, max_rows=6, max_kv=90)
    for at in (0, 6):
        assert (out[at + 4:at + 6] == 77.0).all()
        torch.testing.assert_close(out[at:at + 4].float(), full[at:at + 4].float(), rtol=2.0 ** -6, atol=2.0 ** -6)


@pytest.mark.parametrize("rows", [1, 17, 100])
def test_captured_call_follows_lengths_and_tables(rows):
    """One captured graph serves lengths, tables and queries that change between replays."""
    w = World([400, 300], 2, 128, 32, "bf16")
    cu = cu_of([rows, rows])
    q = torch.randn(2 * rows, 8, 128, device="cuda").bfloat16()
    kv, out = w.kv.clone(), torch.empty_like(q)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        w.cache.attend(q, cu, kv, max_rows=rows, max_kv=400, out=out)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        w.cache.attend(q, cu, kv, max_rows=rows, max_kv=400, out=out)
    for lens in ([400, 300], [101, 299], [rows, 400 - 100]):
        kv.copy_(torch.tensor(lens, dtype=torch.int32))
        q.normal_()
        graph.replay()
        torch.cuda.synchronize()
        want = w.cache.attend(q, cu, kv, max_rows=rows, max_kv=400)
        torch.cuda.synchronize()
        assert torch.equal(out, want), lens


def test_two_streams_at_once():
    ws = [World([2000, 900], 2, 128, 16, "bf16", seed=i) for i in range(2)]
    qs = [torch.randn(2, 8, 128, device="cuda").bfloat16() for _ in ws]
    want = [w.cache.attend(q, cu_of([1, 1]), w.kv, max_rows=1, max_kv=2000) for w, q in zip(ws, qs)]
    cu = cu_of([1, 1])
    torch.cuda.synchronize()
    st = [torch.cuda.Stream() for _ in ws]
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            got[i].append(ws[i].cache.attend(qs[i], cu, ws[i].kv, max_rows=1, max_kv=2000, stream=st[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g, want[i]) for g in got[i])


def test_offsets_past_31_bits():
    """A cache whose element offsets need more than 32 bits: its last pages."""
    n_pages, hkv, page, dh = 4700, 8, 128, 128   # 6.2e8 elements ... times 8 heads' pages: 4.9 GB each
    n_pages *= 4
    k = torch.zeros(n_pages, hkv, page, dh, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    assert k.numel() > 2 ** 31
    table = torch.tensor([[n_pages - 1, 0, n_pages - 2]], dtype=torch.int32, device="cuda")
    for i, p in enumerate(table[0].tolist()):
        k[p].normal_()
        v[p] = float(i + 1)
    c = host().PagedCache(k, v, table)
    L = 300
    kv = torch.tensor([L], dtype=torch.int32, device="cuda")
    for rows in (1, 20):
        q = torch.randn(rows, 8, dh, device="cuda").bfloat16()
        out = c.attend(q, cu_of([rows]), kv, max_rows=rows, max_kv=L)
        kk = torch.cat([k[p] for p in table[0].tolist()], 1)[:, :L].double().cpu().numpy().transpose(1, 0, 2)
        vv = torch.cat([v[p] for p in table[0].tolist()], 1)[:, :L].double().cpu().numpy().transpose(1, 0, 2)
        o, _, _, mag, _ = oc.attention(q.double().cpu().numpy(), kk, vv, np.arange(L - rows, L),
                                       np.arange(L)[:, None].repeat(8, 1), dh ** -0.5)
        assert (np.abs(out.double().cpu().numpy() - o) <= 2.0 ** -6 * mag).all()
    new = torch.randn(1, 8 * 3, dh, device="cuda").bfloat16()
    c.append(new[:, :8], new[:, 8:16], new[:, 16:], cu_of([1]), kv)
    assert torch.equal(k[n_pages - 2, :, (L - 1) % page], new[0, 8:16])
    assert torch.equal(v[n_pages - 2, :, (L - 1) % page], new[0, 16:])


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("dtype,dh", TYPES)
@pytest.mark.parametrize("heads", [(1, 1), (8, 2), (40, 8)])
@pytest.mark.parametrize("rot,inter", [(0, False), (16, False), (16, True), ("half", False), ("all", False), ("all", True)])
@pytest.mark.parametrize("norm", [False, True])
def test_append(dtype, dh, heads, rot, inter, norm):
    hq, hkv = heads
    rot = {"half": dh // 2, "all": dh}.get(rot, rot)
    rows, lens = [1, 0, 33, 5], [70, 3, 33, 18]
    w = World(lens, hkv, dh, 16, dtype, seed=hq + dh, pos=True, weight=True)
    T, u = sum(rows), U[dtype]
    qkv = torch.tensor(w.rng.normal(size=(T + 2, hq + 2 * hkv, dh)) * 3).to(DT[dtype]).cuda()
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    pos = w.rng.integers(0, 2 ** 20, T + 2)
    pos[:2] = [0, 2 ** 31 - 1]
    f = 10000.0 ** (-np.arange(rot // 2) / max(1, rot // 2))
    gq, gk = ((torch.tensor(w.rng.normal(size=dh)).to(DT[dtype]).cuda() for _ in range(2)) if norm else (None, None))
    old = {n: getattr(w, n).clone() for n in ("k", "v", "pos", "weight")}
    out = torch.full((T + 2, hq, dh), 77.0, dtype=DT[dtype]).cuda()
    w.cache.append(q, k, v, cu_of(rows), w.kv, q_pos=torch.tensor(pos, dtype=torch.int32).cuda(), q_gain=gq, k_gain=gk,
                   eps=1e-5, inv_freq=torch.tensor(f, dtype=torch.float64).cuda() if rot else None, interleaved=inter,
                   out=out)
    assert (out[T:] == 77.0).all()
    x = qkv.double().cpu().numpy()

    def close(got, want, size):
        # pair and norm in fp32: 8 roundings and an angle good to 2^-22 of the pair's size; one rounding of the result
        tol = u * np.abs(want) + 2.0 ** -20 * size + 1e-30
        err = np.abs(got.double().cpu().numpy() - want)
        assert (err <= tol).all(), (err / tol).max()

    def want(x, gain):
        g = gain.double().cpu().numpy() if gain is not None else None
        y = oc.norm_rotate(x, g, 1e-5, pos[:T], f, inter)
        z = oc.norm_rotate(x, g, 1e-5, np.zeros(T), [], inter)
        return y, np.abs(z).max(-1, keepdims=True) * np.ones_like(y)

    close(out[:T], *want(x[:T, :hq], gq))
    kw, ks = want(x[:T, hq:hq + hkv], gk)
    at = 0
    for b, n in enumerate(rows):
        p, o = (t.cuda() for t in w.where(b, lens[b]))
        p, o = p[lens[b] - n:], o[lens[b] - n:]
        close(w.k[p, :, o], kw[at:at + n], ks[at:at + n])
        assert torch.equal(w.v[p, :, o], v[at:at + n])
        assert (w.pos[p, :, o].cpu() == torch.tensor(pos[at:at + n, None], dtype=torch.int32)).all()
        assert (w.weight[p, :, o] == 0).all()
        for name in old:   # nothing else changes
            old[name][p, :, o] = getattr(w, name)[p, :, o]
        at += n
    for name in old:
        a, b = getattr(w, name), old[name]
        assert torch.equal(torch.nan_to_num(a, 123.0), torch.nan_to_num(b, 123.0)), name


def test_append_default_positions_in_place_and_missing_pages():
    w = World([20, 40], 2, 64, 16, "f32")
    t = w.t.clone()
    t[1, 2] = -1   # rows 32.. of sequence 1 do not exist
    w.cache.page_table = t
    q = torch.randn(25, 4, 64, device="cuda")
    k, v = torch.randn(25, 2, 64, device="cuda"), torch.randn(25, 2, 64, device="cuda")
    f = torch.tensor([0.5 ** i for i in range(32)], dtype=torch.float64).cuda()
    old = w.k.clone()
    q0 = q.double().cpu().numpy()
    got = w.cache.append(q, k, v, cu_of([5, 20]), w.kv, inv_freq=f, out=q)
    assert got.data_ptr() == q.data_ptr()
    pos = np.concatenate([np.arange(15, 20), np.arange(20, 40)])
    np.testing.assert_allclose(q.cpu().numpy(), oc.norm_rotate(q0, None, 0, pos, f.cpu().numpy(), False), atol=2e-6, rtol=0)
    gone = int(w.table[1, 2])
    assert torch.equal(torch.nan_to_num(w.k[gone], 1.0), torch.nan_to_num(old[gone], 1.0))
    p, o = w.where(1, 32)
    assert torch.equal(w.v[p[20:].cuda(), :, o[20:].cuda()], v[5:17])


# ------------------------------------------------------------------ evict
@pytest.mark.parametrize("dtype,dh,page", [("bf16", 128, 16), ("bf16", 64, 128), ("f32", 32, 32), ("f32", 128, 64)])
@pytest.mark.parametrize("lens,budget,sinks,recent", [
    ([40, 0, 33, 32, 1], 32, 4, 8), ([500, 300, 700], 1, 0, 0), ([1000, 513], 512, 0, 0),
    ([1000, 999, 17], 64, 30, 34), ([9000, 20, 4500], 4096, 4, 100), ([20000], 19990, 4, 100)])
def test_evict(dtype, dh, page, lens, budget, sinks, recent):
    w = World(lens, 2, dh, page, dtype, seed=budget, pos=True, weight=True)
    nxt = []
    for b, L in enumerate(lens):
        p = np.stack([w.rng.permutation(L + 50)[:L] for _ in range(2)], 1) if L else np.zeros((0, 2))
        w.put(w.pos, b, torch.tensor(p))
        x = np.round(np.exp(w.rng.normal(size=(L, 2)) * 2), 1)   # many ties
        x[w.rng.random((L, 2)) < 0.2] = 0.0
        if L > 30:
            x[5], x[6], x[7], x[8] = np.inf, np.nan, -3.0, 1e-42
        w.put(w.weight, b, torch.tensor(x))
        nxt.append(L + 50)
    old = {n: getattr(w, n).clone() for n in ("k", "v", "pos", "weight")}
    left = w.cache.evict(w.kv, torch.tensor(nxt, dtype=torch.int32).cuda(), budget, max_kv=max(lens), sinks=sinks, recent=recent)
    assert left.cpu().tolist() == [min(L, budget) for L in lens]
    for b, L in enumerate(lens):
        if L <= budget:
            continue
        pos, wt = w.get(old["pos"], b), w.get(old["weight"], b)
        P, O = (t.cuda() for t in w.where(b, L))
        for h in range(2):
            for n in old:
                moves = oc.evict(wt[:, h], pos[:, h], nxt[b], budget, sinks, recent)
                if moves:
                    to, come = (torch.tensor(m).cuda() for m in zip(*moves))
                    old[n][P[to], h, O[to]] = old[n][P[come], h, O[come]]
    for n in old:
        assert torch.equal(torch.nan_to_num(getattr(w, n), 123.0), torch.nan_to_num(old[n], 123.0)), n


def test_evict_skips_rows_that_do_not_exist():
    w = World([80], 1, 64, 16, "bf16", pos=True, weight=True)
    t = w.t.clone()
    t[0, 1] = -1      # rows 16..31 are gone: they rank below every other row
    w.cache.page_table = t
    wt, pos = w.get(w.weight, 0)[:, 0], np.arange(80)
    k = w.get(w.k, 0)
    w.cache.evict(w.kv, w.kv, 40, max_kv=80, sinks=2, recent=5)
    wt[16:32], pos[16:32] = -1, 40   # neither safe nor weighted: sorted last of all
    order = [r for r in range(80) if not 16 <= r < 32]
    safe = [r for r in order if r < 2 or r >= 75]
    kept = (safe + sorted((r for r in order if r not in safe), key=lambda r: (-wt[r], r)))[:40]
    holes, movers = [r for r in range(40) if r not in kept], sorted(r for r in kept if r >= 40)
    for to, come in zip(holes, movers):
        if not 16 <= to < 32:
            k[to] = k[come]
    got = w.get(w.k, 0)
    assert np.array_equal(got, k)


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rounds_of_append_attend_evict(dtype):
    """A budgeted cache over several rounds: each appends a block, attends with
    weights, and is cut back; the oracle follows with the same rows."""
    B, hq, hkv, dh, budget, rows = 3, 8, 2, 64, 48, 17
    w = World([budget, 30, 40], hkv, dh, 16, dtype, seed=5, pos=True, weight=True, extra=3 * rows)
    lens, nxt = list(w.lens), np.array([400, 30, 41])
    f = torch.tensor([100.0 ** (-i / 32) for i in range(32)], dtype=torch.float64).cuda()
    gain = torch.ones(dh, dtype=DT[dtype]).cuda()
    kv = w.kv
    for _ in range(5):
        T = B * rows
        qkv = torch.tensor(w.rng.normal(size=(T, hq + 2 * hkv, dh))).to(DT[dtype]).cuda()
        pos = np.concatenate([np.arange(n, n + rows) for n in nxt])
        q_pos, cu = torch.tensor(pos, dtype=torch.int32).cuda(), cu_of([rows] * B)
        kv = kv + rows
        lens = [n + rows for n in lens]
        nxt = nxt + rows
        q = w.cache.append(qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], cu, kv, q_pos=q_pos, q_gain=gain,
                           k_gain=gain, inv_freq=f)
        before = [w.get(w.weight, b, lens[b]) for b in range(B)]
        out = w.cache.attend(q, cu, kv, max_rows=rows, max_kv=budget + rows, q_pos=q_pos, window=200, sinks=4, accumulate=True)
        o64, q64 = out.double().cpu().numpy(), q.double().cpu().numpy()
        for b in range(B):
            k, v, pk = (w.get(t, b, lens[b]) for t in (w.k, w.v, w.pos))
            o, _, wt, mag, _ = oc.attention(q64[b * rows:(b + 1) * rows], k, v, pos[b * rows:(b + 1) * rows], pk, dh ** -0.5, 200, 4)
            u = U[dtype]
            assert (np.abs(o64[b * rows:(b + 1) * rows] - o) <= u * np.abs(o) + (2 * u + 1e-4) * mag).all()
            np.testing.assert_allclose(w.get(w.weight, b, lens[b]) - before[b], wt, rtol=1e-4, atol=1e-5)
        state = [[w.get(t, b, lens[b]) for t in (w.k, w.v, w.pos, w.weight)] for b in range(B)]
        kv = w.cache.evict(kv, torch.tensor(nxt, dtype=torch.int32).cuda(), budget, max_kv=budget + rows, sinks=4, recent=rows)
        for b in range(B):
            for h in range(hkv):
                for to, come in oc.evict(state[b][3][:, h], state[b][2][:, h], nxt[b], budget, 4, rows):
                    for t in state[b]:
                        t[to, h] = t[come, h]
        lens = [min(n, budget) for n in lens]
        assert kv.cpu().tolist() == lens
        for b in range(B):
            for t, buf in zip(state[b], (w.k, w.v, w.pos, w.weight)):
                assert np.array_equal(w.get(buf, b, lens[b]), t[:lens[b]])


# ------------------------------------------------------------------ calls that nothing above makes
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 17, 150])
def test_a_nan_query_spoils_its_own_row_alone(dtype, rows):
    """Its output and its lse are NaN, as the formula's; every other row is as without it."""
    w = World([700, 260], 2, 64, 16, dtype, seed=rows)
    q = torch.tensor(w.rng.normal(size=(2 * rows, 8, 64))).to(DT[dtype]).cuda()
    args = dict(max_rows=rows, max_kv=700, lse=True)
    want, wl = w.cache.attend(q, cu_of([rows, rows]), w.kv, **args)
    bad = q.clone()
    bad[rows - 1, 3, 5] = float("nan")
    got, gl = w.cache.attend(bad, cu_of([rows, rows]), w.kv, **args)
    assert got[rows - 1, 3].isnan().all() and gl[rows - 1, 3].isnan()
    got[rows - 1, 3], gl[rows - 1, 3] = want[rows - 1, 3], wl[rows - 1, 3]
    assert torch.equal(got, want) and torch.equal(gl, wl)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_more_tiles_than_a_call_can_have_are_cut_off(dtype):
    """cu_rows that goes back, so that every sequence claims all rows: no error to return (it
    lies on the device), but nothing out of range is touched and the next call is right."""
    B, rows = 40, 300
    w = World([rows] * B, 1, 64, 16, dtype, seed=3)
    q = torch.tensor(w.rng.normal(size=(rows, 8, 64))).to(DT[dtype]).cuda()
    cu = torch.tensor([0, rows] * (B // 2) + [0], dtype=torch.int32).cuda()
    w.cache.attend(q, cu, w.kv, max_rows=rows, max_kv=rows)
    torch.cuda.synchronize()
    w = World([rows], 1, 64, 16, dtype, seed=4)
    check_attention(w, [rows], 8)


def test_a_stream_of_another_kind_of_handle():
    """A raw stream number serves as a stream object does."""
    w = World([90], 2, 64, 16, "bf16")
    q = torch.randn(3, 4, 64, device="cuda").bfloat16()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    a = w.cache.attend(q, cu_of([3]), w.kv, max_rows=3, max_kv=90)
    torch.cuda.synchronize()
    b = w.cache.attend(q, cu_of([3]), w.kv, max_rows=3, max_kv=90, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 17, 150])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3)])
def test_stored_positions_decide_at_width_128(dtype, rows, window, sinks):
    """Positions far apart, in any order, over caches of several blocks."""
    lens = [500, 155, 160]
    w = World(lens, 2, 128, 32, dtype, seed=rows, pos=True)
    for b, L in enumerate(lens):
        w.put(w.pos, b, torch.tensor(np.stack([w.rng.permutation(L) * (b + 1) for _ in range(2)], 1)))
    q_pos = np.concatenate([np.sort(w.rng.integers(0, L * (b + 1), rows)) for b, L in enumerate(lens)])
    check_attention(w, [rows] * 3, 4, window, sinks, q_pos=q_pos)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 17, 140])
@pytest.mark.parametrize("max_kv", [1, 100, 129])
def test_a_sequence_longer_than_max_kv_is_cut(dtype, rows, max_kv):
    """Its rows keep their positions; the cached rows from max_kv on are not read."""
    w = World([300, 60, 128], 2, 64, 16, dtype, seed=max_kv, weight=True)
    n = [rows, min(rows, 60), min(rows, 128)]
    there = [np.arange(L) < max_kv for L in w.lens]
    check_attention(w, n, 4, 0, 0, there=there, max_kv=max_kv, accumulate=True)
    check_attention(w, n, 4, 250, 2, there=there, max_kv=max_kv)


@pytest.mark.parametrize("dtype,dh", [("bf16", 64), ("bf16", 128), ("f32", 64)])
@pytest.mark.parametrize("rows", [1, 40, 200])
def test_largest_window_and_sinks(dtype, dh, rows):
    """The largest numbers mean no window at all, also before row 0."""
    w = World([7, 0, 64, 300], 1, dh, 16, dtype)
    for window, sinks in ((2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1), (5, 2 ** 31 - 1)):
        check_attention(w, [rows + 7, rows, 64, rows], 8, window, sinks)
