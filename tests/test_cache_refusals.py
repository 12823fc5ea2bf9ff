"""Calls of the paged cache that would fault, race or mean something else on the GPU are
refused on the host (no GPU needed)."""
import pytest

import step_flow_map_b200 as fmb
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
