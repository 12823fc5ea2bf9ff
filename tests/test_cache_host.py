"""The paged-cache operators on the host: what they refuse, and their oracle's pins (no GPU needed)."""
import numpy as np
import pytest
import torch

import step_flow_map_b200 as fmb
from oracle import cache as oc
from step_flow_map_b200 import build
from step_flow_map_b200.host import PagedCache

P = 1 << 20   # a non-null, aligned address that no refused call reads


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()


def cache(**kw):
    d = dict(dtype=fmb.FM_BF16, n_pages=8, page_size=16, n_kv_heads=2, head_dim=64, table_stride=4,
             k=P, v=P, pos=P, weight=P, page_table=P)
    return fmb.fm_paged_cache(**{**d, **kw})


def append_args(**kw):
    d = dict(T=3, B=2, n_heads=4, q=P, k=P, v=P, q_stride=256, k_stride=128, v_stride=128, eps=1e-6,
             inv_freq=P, rot_dim=64, cu_rows=P, kv_len=P, q_pos=P, q_out=P, q_out_stride=256)
    return fmb.fm_append_args(**{**d, **kw})


def attn_args(**kw):
    d = dict(T=3, B=2, n_heads=4, max_rows=2, max_kv=64, q=P, q_stride=256, cu_rows=P, kv_len=P,
             q_pos=P, scale=0.125, out=P + 4096, out_stride=256)
    return fmb.fm_attention_args(**{**d, **kw})


def refused(status, fn, *a):
    with pytest.raises(fmb.FlashmapError) as e:
        fn(*a)
    assert e.value.status == status, str(e.value)


BAD_CACHE = [
    (dict(k=None), fmb.FM_ERR_ARG), (dict(v=None), fmb.FM_ERR_ARG), (dict(page_table=None), fmb.FM_ERR_ARG),
    (dict(dtype=2), fmb.FM_ERR_ARG), (dict(n_pages=0), fmb.FM_ERR_ARG), (dict(n_kv_heads=0), fmb.FM_ERR_ARG),
    (dict(table_stride=0), fmb.FM_ERR_ARG), (dict(page_size=24), fmb.FM_ERR_UNSUPPORTED),
    (dict(page_size=8), fmb.FM_ERR_UNSUPPORTED), (dict(page_size=256), fmb.FM_ERR_UNSUPPORTED),
    (dict(head_dim=32), fmb.FM_ERR_UNSUPPORTED), (dict(head_dim=96), fmb.FM_ERR_UNSUPPORTED),
    (dict(n_pages=1 << 30), fmb.FM_ERR_UNSUPPORTED), (dict(table_stride=1 << 24), fmb.FM_ERR_UNSUPPORTED),
    (dict(k=P + 8), fmb.FM_ERR_ARG), (dict(pos=P + 2), fmb.FM_ERR_ARG),
]


@pytest.mark.parametrize("kw,status", BAD_CACHE)
def test_bad_cache_is_refused(kw, status):
    refused(status, fmb.fm_cache_append, cache(**kw), append_args())
    refused(status, fmb.fm_cache_attention, cache(**kw), attn_args(), P, 1 << 40)
    refused(status, fmb.fm_cache_evict, cache(**kw), P, P, 2, 64, 32, 4, 8, P + 64)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), fmb.FM_ERR_ARG), (dict(B=0), fmb.FM_ERR_ARG), (dict(B=257), fmb.FM_ERR_UNSUPPORTED),
    (dict(n_heads=3), fmb.FM_ERR_ARG), (dict(n_heads=0), fmb.FM_ERR_ARG), (dict(q=None), fmb.FM_ERR_ARG),
    (dict(k=None), fmb.FM_ERR_ARG), (dict(v=None), fmb.FM_ERR_ARG), (dict(q_out=None), fmb.FM_ERR_ARG),
    (dict(cu_rows=None), fmb.FM_ERR_ARG), (dict(kv_len=None), fmb.FM_ERR_ARG), (dict(q_pos=None), fmb.FM_ERR_ARG),
    (dict(q_stride=255), fmb.FM_ERR_ARG), (dict(q_stride=128), fmb.FM_ERR_ARG), (dict(k_stride=64), fmb.FM_ERR_ARG),
    (dict(q=P + 8), fmb.FM_ERR_ARG), (dict(rot_dim=24), fmb.FM_ERR_ARG), (dict(rot_dim=80), fmb.FM_ERR_ARG),
    (dict(inv_freq=None), fmb.FM_ERR_ARG), (dict(eps=-1.0), fmb.FM_ERR_ARG), (dict(eps=float("nan")), fmb.FM_ERR_ARG),
    (dict(q_gain=P + 4), fmb.FM_ERR_ARG), (dict(T=1 << 25), fmb.FM_ERR_UNSUPPORTED),
])
def test_bad_append_is_refused(kw, status):
    refused(status, fmb.fm_cache_append, cache(), append_args(**kw))


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), fmb.FM_ERR_ARG), (dict(B=0), fmb.FM_ERR_ARG), (dict(n_heads=5), fmb.FM_ERR_ARG),
    (dict(max_rows=0), fmb.FM_ERR_ARG), (dict(max_kv=0), fmb.FM_ERR_ARG), (dict(max_kv=1 << 25), fmb.FM_ERR_UNSUPPORTED),
    (dict(window=-1), fmb.FM_ERR_ARG), (dict(sinks=-1), fmb.FM_ERR_ARG), (dict(scale=0.0), fmb.FM_ERR_ARG),
    (dict(scale=float("nan")), fmb.FM_ERR_ARG), (dict(scale=float("inf")), fmb.FM_ERR_ARG), (dict(q=None), fmb.FM_ERR_ARG),
    (dict(out=None), fmb.FM_ERR_ARG), (dict(q_pos=None), fmb.FM_ERR_ARG), (dict(out_stride=100), fmb.FM_ERR_ARG),
    (dict(cu_rows=None), fmb.FM_ERR_ARG),
])
def test_bad_attention_is_refused(kw, status):
    refused(status, fmb.fm_cache_attention, cache(), attn_args(**kw), P, 1 << 40)


def test_accumulate_without_weights_and_bad_workspace_are_refused():
    refused(fmb.FM_ERR_ARG, fmb.fm_cache_attention, cache(weight=None), attn_args(accumulate=1), P, 1 << 40)
    refused(fmb.FM_ERR_ARG, fmb.fm_cache_attention, cache(), attn_args(), None, 1 << 40)
    refused(fmb.FM_ERR_ARG, fmb.fm_cache_attention, cache(), attn_args(), P + 16, 1 << 40)


def test_attention_in_place_is_refused():
    refused(fmb.FM_ERR_ARG, fmb.fm_cache_attention, cache(), attn_args(out=P, q=P), P, 1 << 40)


def test_a_cache_off_the_gpu_is_refused_before_any_launch():
    k = torch.zeros(6, 2, 16, 64, dtype=torch.bfloat16)
    pos, weight = torch.zeros(6, 2, 16, dtype=torch.int32), torch.zeros(6, 2, 16)
    c = PagedCache(k, k.clone(), torch.zeros(2, 3, dtype=torch.int32), pos, weight)
    cu, kv = torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    q, kr = torch.zeros(4, 4, 64, dtype=torch.bfloat16), torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    qp = torch.zeros(4, dtype=torch.int32)
    for stream in (None, 0):
        with pytest.raises(ValueError, match="GPU"):
            c.append(q, kr, kr, cu, kv, q_pos=qp, stream=stream)
        with pytest.raises(ValueError, match="GPU"):
            c.attend(q, cu, kv, max_rows=4, max_kv=16, q_pos=qp, stream=stream)
        with pytest.raises(ValueError, match="GPU"):
            c.evict(kv, kv, 8, max_kv=16, stream=stream)


@pytest.mark.parametrize("a,status", [
    ((None, P, 2, 64, 32, 4, 8, P + 64), fmb.FM_ERR_ARG), ((P, None, 2, 64, 32, 4, 8, P + 64), fmb.FM_ERR_ARG),
    ((P, P, 2, 64, 32, 4, 8, None), fmb.FM_ERR_ARG), ((P, P, 2, 64, 32, 4, 8, P), fmb.FM_ERR_ARG),
    ((P, P, 0, 64, 32, 4, 8, P + 64), fmb.FM_ERR_ARG), ((P, P, 2, 64, 0, 0, 0, P + 64), fmb.FM_ERR_ARG),
    ((P, P, 2, 64, 32, 25, 8, P + 64), fmb.FM_ERR_ARG), ((P, P, 2, 64, 32, -1, 8, P + 64), fmb.FM_ERR_ARG),
    ((P, P, 2, 64, 32, 4, -8, P + 64), fmb.FM_ERR_ARG), ((P, P, 257, 64, 32, 4, 8, P + 64), fmb.FM_ERR_UNSUPPORTED),
    ((P, P, 2, fmb.FM_MAX_EVICT_ROWS + 1, 32, 4, 8, P + 64), fmb.FM_ERR_UNSUPPORTED),
    ((P, P, 2, 64, 1 << 30, 1 << 30, 1 << 30, P + 64), fmb.FM_ERR_ARG),
])
def test_bad_evict_is_refused(a, status):
    refused(status, fmb.fm_cache_evict, cache(), *a)


def test_evict_without_positions_or_weights_is_refused():
    a = (P, P, 2, 64, 32, 4, 8, P + 64)
    refused(fmb.FM_ERR_ARG, fmb.fm_cache_evict, cache(pos=None), *a)
    refused(fmb.FM_ERR_ARG, fmb.fm_cache_evict, cache(weight=None), *a)


def test_a_call_without_rows_does_nothing():
    fmb.fm_cache_append(cache(), append_args(T=0, q=None, k=None, v=None, q_out=None))
    fmb.fm_cache_attention(cache(), attn_args(T=0, q=None, out=None), None, 0)


def test_paged_cache_checks_its_tensors():
    k = torch.zeros(6, 2, 16, 64, dtype=torch.bfloat16)
    table = torch.zeros(2, 3, dtype=torch.int32)
    pos, weight = torch.zeros(6, 2, 16, dtype=torch.int32), torch.zeros(6, 2, 16)
    PagedCache(k, k.clone(), table, pos, weight)
    for bad in (dict(v=k.float()), dict(v=k[:5]), dict(page_table=table.long()), dict(page_table=table[0]),
                dict(pos=pos.long()), dict(weight=weight[:, :, :8]), dict(k=k.half()),
                dict(v=k.transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises(ValueError):
            PagedCache(**{**dict(k=k, v=k.clone(), page_table=table, pos=pos, weight=weight), **bad})
    c = PagedCache(k, k.clone(), table, pos, weight)
    cu, kv = torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    q = torch.zeros(4, 4, 64, dtype=torch.bfloat16)
    kr = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    qp = torch.zeros(4, dtype=torch.int32)
    for bad in (dict(q=q.float()), dict(q=q[0]), dict(q=q.transpose(0, 1)), dict(q=q[..., :32]),
                dict(cu_rows=cu[:2]), dict(kv_len=kv.long()), dict(q_pos=qp[:3])):
        with pytest.raises(ValueError):
            c.attend(**{**dict(q=q, cu_rows=cu, kv_len=kv, q_pos=qp, max_rows=2, max_kv=16), **bad})
    for bad in (dict(k=kr[:3]), dict(k=kr[:, :1]), dict(v=kr.float()), dict(q_gain=torch.ones(64)),
                dict(inv_freq=torch.ones(32))):
        with pytest.raises(ValueError):
            c.append(**{**dict(q=q, k=kr, v=kr, cu_rows=cu, kv_len=kv, q_pos=qp), **bad})
    with pytest.raises(ValueError):   # more sequences than the table has rows
        c.evict(torch.zeros(3, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), 8, max_kv=16)


# ------------------------------------------------------------------ the oracle's own pins
def test_oracle_rotation_is_a_rotation():
    rng = np.random.default_rng(1)
    x, f = rng.normal(size=(2, 3, 32)), np.array([1.0, 0.1, 0.01, 0.001])
    for inter in (False, True):
        y = oc.norm_rotate(x, None, 0.0, [7, 11], f, inter)
        np.testing.assert_allclose((y * y).sum(-1), (x * x).sum(-1), rtol=1e-13)
        assert (y[..., 8:] == x[..., 8:]).all()
        # scores depend on the difference of positions only
        z = oc.norm_rotate(x, None, 0.0, [107, 111], f, inter)
        np.testing.assert_allclose((y[0] * y[1]).sum(), (z[0] * z[1]).sum(), rtol=1e-11)
    # a quarter turn of pair 0 takes (a, b) to (-b, a)
    y = oc.norm_rotate(x, None, 0.0, [1, 1], [np.pi / 2], True)
    np.testing.assert_allclose(y[..., 0], -x[..., 1], atol=1e-15)
    np.testing.assert_allclose(y[..., 1], x[..., 0], atol=1e-15)
    y = oc.norm_rotate(x, np.full(32, 2.0), 0.0, [0, 0], [], False)
    np.testing.assert_allclose((y * y).mean(-1), 4.0)


def test_oracle_mask():
    see = oc.visible([5], [0, 1, 2, 3, 4, 5, 6], 3, 1)[0]
    assert see.tolist() == [True, False, False, True, True, True, False]
    assert oc.visible([5], [0, 5, 6], 0, 0)[0].tolist() == [True, True, False]


def test_oracle_attention_closed_forms():
    v = np.arange(6.0).reshape(3, 1, 2)
    q, k = np.zeros((1, 2, 2)), np.zeros((3, 1, 2))
    o, lse, w, _, _ = oc.attention(q, k, v, [2], np.arange(3)[:, None], 1.0)
    np.testing.assert_allclose(o[0, 0], [2, 3])
    np.testing.assert_allclose(lse, np.log(3))
    np.testing.assert_allclose(w[:, 0], 2 / 3)
    o, lse, w, _, _ = oc.attention(q, k, v, [-1], np.arange(3)[:, None], 1.0)
    assert (o == 0).all() and (lse == -np.inf).all() and (w == 0).all()
    q[0, 1, 0] = np.log(4)   # head 1 weighs row 1 four times
    k[1, 0, 0] = 1.0
    o, _, w, _, _ = oc.attention(q, k, v, [2], np.arange(3)[:, None], 1.0)
    np.testing.assert_allclose(o[0, 1], [(0 + 4 * 2 + 4) / 6, (1 + 4 * 3 + 5) / 6])
    np.testing.assert_allclose(w[:, 0], [1 / 3 + 1 / 6, 1 / 3 + 4 / 6, 1 / 3 + 1 / 6])


def test_oracle_evict_by_hand():
    #        row   0    1    2    3    4    5
    w = [0.1, 0.9, 0.0, 0.5, 0.9, 0.0]
    pos = [0, 1, 2, 3, 4, 5]
    # row 5 is recent, row 0 a sink, then rows 1 and 4 by weight: 2 <- 4, 3 <- 5
    assert oc.evict(w, pos, 6, 4, 1, 1) == [(2, 4), (3, 5)]
    # ties: rows 2 and 5 both 0, the lower stays
    assert oc.evict(w, pos, 6, 5, 0, 0) == []
    assert oc.evict([0, np.nan, -1.0, 2.0], [9, 8, 7, 6], 10, 2, 0, 0) == [(1, 3)]
    assert oc.evict(w, pos, 6, 6, 1, 1) == []
