"""What the paged cache's append passes on as it is, and which pages it may share.

Columns past rot_dim are not turned, and without a gain heads are not scaled: such
values are copies, infinities and -0 among them, and are compared bit for bit (a
NaN stays one).  With a gain and a finite row they are x r g, two products after the norm:
8 fp32 roundings (2^-21 relative) and one of the result (2^-8 for bf16, 2^-24).
"""
import math

import numpy as np
import pytest
import torch

from oracle import cache as oc
from test_gpu_cache import DT, TYPES, U, World, cu_of

pytestmark = pytest.mark.gpu


def bits(t):
    return torch.where(t.isnan(), math.nan, t).view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


def odd_values(x, cols):
    """Infinities, NaN, zeros of both signs and the largest and smallest numbers in some columns."""
    fi = torch.finfo(x.dtype)
    for i, v in enumerate([math.inf, -math.inf, math.nan, -0.0, 0.0, fi.max, -fi.max, fi.smallest_normal]):
        x[i % x.shape[0], :, cols[(3 * i + 1) % len(cols)]] = v
    return x


@pytest.mark.parametrize("dtype,dh", TYPES)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rot", [0, 16, "half", "all but 16"])
def test_values_past_the_rotation_are_copies(dtype, dh, inter, rot):
    rot = {"half": dh // 2, "all but 16": dh - 16}.get(rot, rot)
    if rot % 16:
        rot -= rot % 16
    hq, hkv, rows, lens = 6, 2, [4, 7], [9, 40]
    w = World(lens, hkv, dh, 16, dtype, seed=rot)
    T = sum(rows)
    qkv = odd_values(torch.tensor(w.rng.normal(size=(T, hq + 2 * hkv, dh))).to(DT[dtype]).cuda(), range(rot, dh))
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    f = torch.tensor([0.7 ** i for i in range(rot // 2)], dtype=torch.float64).cuda() if rot else None
    got = w.cache.append(q, k, v, cu_of(rows), w.kv, inv_freq=f, interleaved=inter)
    assert torch.equal(bits(got[..., rot:]), bits(q[..., rot:]))
    at = 0
    for b, n in enumerate(rows):
        p, o = (t.cuda()[lens[b] - n:] for t in w.where(b, lens[b]))
        assert torch.equal(bits(w.k[p, :, o][..., rot:]), bits(k[at:at + n][..., rot:]))
        assert torch.equal(bits(w.v[p, :, o]), bits(v[at:at + n]))
        if rot:   # and the turned ones are finite, as their pairs are
            assert got[at:at + n, :, :rot].isfinite().all() and w.k[p, :, o][..., :rot].isfinite().all()
        at += n


@pytest.mark.parametrize("dtype,dh", TYPES)
@pytest.mark.parametrize("inter", [False, True])
def test_a_gain_scales_values_past_the_rotation_by_themselves(dtype, dh, inter):
    """An infinite gain reaches its own column alone."""
    hq, hkv, rot = 6, 2, 16
    w = World([30], hkv, dh, 16, dtype, seed=3)
    x = torch.tensor(w.rng.normal(size=(5, hq + 2 * hkv, dh))).to(DT[dtype]).cuda()
    gain = torch.tensor(w.rng.normal(size=dh)).to(DT[dtype]).cuda()
    want = oc.norm_rotate(x[:, :hq].double().cpu().numpy(), gain.double().cpu().numpy(), 1e-6, np.arange(25, 30),
                          [1.0 / (i + 1) for i in range(rot // 2)], inter)
    f = torch.tensor([1.0 / (i + 1) for i in range(rot // 2)], dtype=torch.float64).cuda()
    gain[rot + 3] = math.inf
    got = w.cache.append(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], cu_of([5]), w.kv, q_gain=gain, k_gain=gain,
                         inv_freq=f, interleaved=inter).double().cpu().numpy()
    assert (np.abs(got[..., rot + 3]) == np.inf).all()
    got[..., rot + 3] = want[..., rot + 3]
    tol = (U[dtype] + 2.0 ** -21) * np.abs(want) + 2.0 ** -20 * np.abs(want).max(-1, keepdims=True) * (np.arange(dh) < rot)
    assert (np.abs(got - want) <= tol).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 40, 3000])
@pytest.mark.parametrize("where", ["in place", "beside"])
def test_queries_go_to_a_slice_of_the_same_buffer(dtype, T, where):
    """The projection's own query slice, or another slice of the same rows."""
    hq, hkv, dh = 8, 2, 64
    w = World([T + 5], hkv, dh, 16, dtype, seed=T)
    wide = torch.tensor(w.rng.normal(size=(T, 2 * hq + 2 * hkv, dh))).to(DT[dtype]).cuda()
    q, k, v, spare = wide.split([hq, hkv, hkv, hq], 1)
    f = torch.tensor([0.5 ** i for i in range(16)], dtype=torch.float64).cuda()
    gain = torch.tensor(w.rng.normal(size=dh)).to(DT[dtype]).cuda()
    args = dict(cu_rows=cu_of([T]), kv_len=w.kv, q_gain=gain, k_gain=gain, inv_freq=f)
    want = w.cache.append(q, k, v, **args)
    cached = w.k.clone(), w.v.clone()
    out = q if where == "in place" else spare
    got = w.cache.append(q, k, v, **args, out=out)
    assert got.data_ptr() == out.data_ptr() and torch.equal(got, want)
    for now, old in zip((w.k, w.v), cached):
        assert torch.equal(torch.nan_to_num(now, 9.0), torch.nan_to_num(old, 9.0))


def test_sequences_may_share_the_pages_before_their_new_rows():
    """Drafts of one prefix: each has its own last page, the pages before it are the same."""
    w = World([64], 2, 64, 16, "bf16", extra=16, spare=6)
    B, rows = 3, 5
    own = [i for i in range(w.k.shape[0]) if i not in w.table[0, :4].tolist()][:B]
    t = torch.tensor([w.table[0, :4].tolist() + [p] for p in own], dtype=torch.int32).cuda()
    c = w.cache
    c.page_table = t
    old = w.k.clone(), w.v.clone()
    kv = torch.full((B,), 64 + rows, dtype=torch.int32).cuda()
    qkv = torch.tensor(w.rng.normal(size=(B * rows, 8, 64))).to(torch.bfloat16).cuda()
    q = c.append(qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], cu_of([rows] * B), kv)
    for i, (now, x) in enumerate(((w.k, qkv[:, 4:6]), (w.v, qkv[:, 6:]))):
        want = old[i].clone()
        for b, p in enumerate(own):
            want[p, :, :rows] = x[b * rows:(b + 1) * rows].transpose(0, 1)
        assert torch.equal(torch.nan_to_num(now, 9.0), torch.nan_to_num(want, 9.0))
    out = c.attend(q, cu_of([rows] * B), kv, max_rows=rows, max_kv=64 + rows)
    for b in range(B):
        k, v = (torch.cat([x[p] for p in t[b].tolist()], 1)[:, :64 + rows].transpose(0, 1).double().cpu().numpy() for x in (w.k, w.v))
        o, _, _, mag, _ = oc.attention(q[b * rows:(b + 1) * rows].double().cpu().numpy(), k, v, np.arange(64, 64 + rows),
                                       np.arange(64 + rows)[:, None].repeat(2, 1), 64 ** -0.5)
        # the bound of the attention tests with every score error below 2^-10
        assert (np.abs(out[b * rows:(b + 1) * rows].double().cpu().numpy() - o) <= 2.0 ** -8 * np.abs(o) + 2.0 ** -6 * mag).all()
