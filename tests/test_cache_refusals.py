"""Calls of the paged cache that would fault, race or mean something else on the GPU are
refused on the host (no GPU needed)."""
import pytest
import torch

import step_flow_map_b200 as fmb
from step_flow_map_b200.host import PagedCache
from test_cache_host import P, _lib, append_args, attn_args, cache, refused  # noqa: F401


@pytest.mark.parametrize("name", ["cu_rows", "kv_len", "q_pos"])
@pytest.mark.parametrize("off", [1, 2])
def test_misaligned_numbers_are_refused(name, off):
    refused(fmb.FM_ERR_ARG, fmb.fm_cache_append, cache(), append_args(**{name: P + off}))
    refused(fmb.FM_ERR_ARG, fmb.fm_cache_attention, cache(), attn_args(**{name: P + off}), P, 1 << 40)


@pytest.mark.parametrize("off", [1, 2])
def test_misaligned_outputs_and_lengths_are_refused(off):
    refused(fmb.FM_ERR_ARG, fmb.fm_cache_attention, cache(), attn_args(lse=P + off), P, 1 << 40)
    at = [P, P + 4096, P + 8192]
    for i in range(3):
        kv, nxt, new = (p + off * (i == j) for j, p in enumerate(at))
        refused(fmb.FM_ERR_ARG, fmb.fm_cache_evict, cache(), kv, nxt, 2, 64, 32, 4, 8, new)


@pytest.mark.parametrize("d", [0, 4, 28, -4, -28])
def test_eviction_refuses_lengths_that_overlap_its_inputs(d):
    """Eight sequences: the new lengths lie d bytes from the old ones, or from the positions."""
    kv, nxt = P, P + 4096
    refused(fmb.FM_ERR_ARG, fmb.fm_cache_evict, cache(), kv, nxt, 8, 64, 32, 4, 8, kv + d)
    refused(fmb.FM_ERR_ARG, fmb.fm_cache_evict, cache(), kv, nxt, 8, 64, 32, 4, 8, nxt + d)


# ------------------------------------------------------------------ outputs that overlap inputs
ROW = 256 * 2   # bytes of a row of 4 heads of width 64 in bf16
AT = dict(q=P, k=P + (1 << 16), v=P + (2 << 16), q_out=P + (3 << 16))


def message(fn, *a):
    with pytest.raises(fmb.FlashmapError) as e:
        fn(*a)
    assert e.value.status == fmb.FM_ERR_ARG, str(e.value)
    return str(e.value)


@pytest.mark.parametrize("kw", [
    dict(q_out=P + 16), dict(q_out=P + 2 * ROW), dict(q_out=P - 2 * ROW), dict(q_out=P + ROW - 16),   # q, shifted
    dict(q_out=P, q_out_stride=264), dict(q_out=P, q_stride=512),                                     # q, another stride
    dict(q_out=AT["k"]), dict(q_out=AT["k"] - 3 * ROW + 16), dict(q_out=AT["v"] + 2 * 256 + 240),
    # slices of one buffer (768 values a row) that reach into one another
    dict(q_stride=768, k_stride=768, v_stride=768, q_out_stride=768, k=P + ROW, v=P + ROW + 256, q_out=P + ROW + 496),
    dict(q_stride=768, k_stride=768, v_stride=768, q_out_stride=768, k=P + ROW, v=P + ROW + 256, q_out=P + 768 * 2 - 16),
])
def test_append_refuses_queries_that_overlap_what_it_reads(kw):
    assert "overlap" in message(fmb.fm_cache_append, cache(), append_args(**{**AT, **kw}))


@pytest.mark.parametrize("kw", [
    dict(out=P), dict(out=P + 16), dict(out=P + 3 * ROW - 16), dict(out=P - 2 * ROW - 16), dict(out=P + 16, out_stride=264),
    dict(q_stride=512, out_stride=512, out=P + ROW - 16), dict(q_stride=512, out_stride=512, out=P - 512 * 2 + ROW + 16),
    dict(lse=P + 4), dict(lse=P + 3 * ROW - 4), dict(lse=P + 4096 + ROW), dict(lse=P + 4096 - 44),
    dict(T=1, out=P + ROW - 16, out_stride=8), dict(T=1, out=P, q_stride=1024),
])
def test_attention_refuses_outputs_that_overlap(kw):
    assert "overlap" in message(fmb.fm_cache_attention, cache(), attn_args(**kw), P, 1 << 40)


@pytest.mark.parametrize("kw", [
    dict(), dict(out=P + 3 * ROW), dict(out=P - 3 * ROW), dict(lse=P + 3 * ROW), dict(lse=P - 48), dict(lse=P + 4096 - 48),
    # slices of one buffer
    dict(q_stride=512, out_stride=512, out=P + ROW), dict(q_stride=512, out_stride=512, out=P - ROW),
    dict(q_stride=1024, out_stride=1024, out=P + ROW + 16), dict(q_stride=1024, out_stride=1024, out=P - 2048 * 2 + ROW),
    dict(q_stride=512, out_stride=2048, out=P + ROW), dict(T=1, out=P + ROW, out_stride=8),
])
def test_attention_takes_outputs_beside_its_queries(kw):
    """The only complaint is the one that comes next: no workspace."""
    assert "workspace" in message(fmb.fm_cache_attention, cache(), attn_args(**kw), None, 0)


def test_overlap_of_rows_is_found_byte_by_byte():
    """Against the sets of bytes, for strides and distances around every border."""
    def touched(at, stride, width, n):
        return {at + i * stride + x for i in range(n) for x in range(0, width, 16)}
    n, width = 3, 2 * 64 * 2
    base = P + (1 << 14)
    for qs in (256, 272, 512, 784):
        for os in (256, 272, 512, 784):
            mine = touched(0, qs, width, n)
            for d in range(-1600, 1601, 16):
                a = attn_args(n_heads=2, T=n, q=base, q_stride=qs // 2, out=base + d, out_stride=os // 2)
                got = "overlap" in message(fmb.fm_cache_attention, cache(), a, None, 0)
                assert got == bool(mine & touched(d, os, width, n)), (qs, os, d)


# the refusals of an append once more where nothing overlaps
@pytest.mark.parametrize("kw,status", [
    (dict(q=None), fmb.FM_ERR_ARG), (dict(k=None), fmb.FM_ERR_ARG), (dict(v=None), fmb.FM_ERR_ARG),
    (dict(q_out=None), fmb.FM_ERR_ARG), (dict(cu_rows=None), fmb.FM_ERR_ARG), (dict(kv_len=None), fmb.FM_ERR_ARG),
    (dict(q_pos=None), fmb.FM_ERR_ARG), (dict(q_stride=255), fmb.FM_ERR_ARG), (dict(q_stride=128), fmb.FM_ERR_ARG),
    (dict(k_stride=64), fmb.FM_ERR_ARG), (dict(q=P + 8), fmb.FM_ERR_ARG), (dict(rot_dim=24), fmb.FM_ERR_ARG),
    (dict(rot_dim=80), fmb.FM_ERR_ARG), (dict(inv_freq=None), fmb.FM_ERR_ARG), (dict(eps=-1.0), fmb.FM_ERR_ARG),
    (dict(eps=float("nan")), fmb.FM_ERR_ARG), (dict(q_gain=P + 4), fmb.FM_ERR_ARG), (dict(n_heads=3), fmb.FM_ERR_ARG),
    (dict(inv_freq=P + 4), fmb.FM_ERR_ARG), (dict(T=1 << 25), fmb.FM_ERR_UNSUPPORTED), (dict(B=257), fmb.FM_ERR_UNSUPPORTED),
])
def test_bad_append_is_refused_for_its_own_reason(kw, status):
    with pytest.raises(fmb.FlashmapError) as e:
        fmb.fm_cache_append(cache(), append_args(**{**AT, **kw}))
    assert e.value.status == status and "overlap" not in str(e.value)


# ------------------------------------------------------------------ numbers that C would wrap
@pytest.mark.parametrize("name", ["max_rows", "max_kv", "window", "sinks"])
@pytest.mark.parametrize("x", [2 ** 31, 2 ** 32, 2 ** 32 + 7, 2 ** 64 + 5, -2 ** 31 - 1])
def test_attend_refuses_numbers_past_32_bits(name, x):
    c, q, cu, kv, _ = a_cache_off_the_gpu()
    with pytest.raises(ValueError, match=name):
        c.attend(q, cu, kv, **{**dict(max_rows=4, max_kv=16, window=3, sinks=1), name: x})


@pytest.mark.parametrize("name", ["max_kv", "budget", "sinks", "recent"])
@pytest.mark.parametrize("x", [2 ** 31, 2 ** 32, 2 ** 32 + 7, 2 ** 64 + 5, -2 ** 31 - 1])
def test_evict_refuses_numbers_past_32_bits(name, x):
    c, _, _, kv, _ = a_cache_off_the_gpu()
    with pytest.raises(ValueError, match=name):
        c.evict(kv, kv, **{**dict(budget=8, max_kv=16, sinks=1, recent=2), name: x})


def a_cache_off_the_gpu():
    """Calls with it end in ValueError at the latest when they ask for its GPU."""
    k = torch.zeros(6, 2, 16, 64, dtype=torch.bfloat16)
    c = PagedCache(k, k.clone(), torch.zeros(2, 3, dtype=torch.int32), None, torch.zeros(6, 2, 16))
    return (c, torch.zeros(4, 4, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32),
            torch.zeros(2, dtype=torch.int32), torch.zeros(4, 2, 64, dtype=torch.bfloat16))


def test_outputs_are_looked_at_before_a_stream_is():
    """What is wrong with an output is said as for any other tensor, whatever stream is given."""
    c, q, cu, kv, kr = a_cache_off_the_gpu()
    for stream in (None, 0):
        with pytest.raises(ValueError, match="out must"):
            c.append(q, kr, kr, cu, kv, out=q.float(), stream=stream)
        with pytest.raises(ValueError, match="out must"):
            c.attend(q, cu, kv, max_rows=4, max_kv=16, out=q[:3], stream=stream)
        with pytest.raises(ValueError, match="new_len must"):
            c.evict(kv, kv, 8, max_kv=16, new_len=kv[:1], stream=stream)
