"""What must not move a bit of the paged cache's attention: packed rows that are
none of the result's.

bf16 tiles of 128 packed rows hold whole queries, so for G = 3 or 5 query heads per
key/value head the last rows of a tile belong to no query, and past a
sequence's end they belong to its neighbour.
"""
import numpy as np
import pytest
import torch

from test_gpu_cache import DT, World, cu_of

pytestmark = pytest.mark.gpu


def attend(w, q, rows, window=0):
    out, lse = w.cache.attend(q, cu_of(rows), w.kv, max_rows=max(rows), max_kv=max(w.lens), window=window, lse=True)
    return out.clone(), lse.clone()


def queries(w, T, heads, sharp=1.0):
    return torch.tensor(w.rng.normal(size=(T, heads, w.dh)) * sharp).to(DT[w.dtype]).cuda()


# (rows, G, key/value heads): one query tile and two of them, with enough heads that a
# CTA takes many blocks of a tile
MANY = [(5, 5, 24), (20, 3, 24), (26, 5, 2), (60, 3, 2)]


@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("rows,G,hkv", MANY)
def test_a_neighbours_queries_leave_a_sequences_bits_alone(dh, rows, G, hkv):
    w = World([5000, 4000], hkv, dh, 32, "bf16", seed=rows)
    q = queries(w, 2 * rows, hkv * G, 3.0)
    want, wl = attend(w, q, [rows, rows])
    for size in (0.0, 40.0, 1000.0):
        other = q.clone()
        other[rows:] *= size
        got, gl = attend(w, other, [rows, rows])
        assert torch.equal(got[:rows], want[:rows]) and torch.equal(gl[:rows], wl[:rows]), size


@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("rows,G,hkv", MANY)
def test_what_ran_before_leaves_the_bits_alone(dh, rows, G, hkv):
    """Between two equal calls another one leaves large values wherever it kept its queries."""
    w = World([5000, 4000], hkv, dh, 32, "bf16", seed=rows)
    q = queries(w, 2 * rows, hkv * G, 3.0)
    filler = World([6000] * 8, 2, dh, 32, "bf16", seed=1)
    huge = queries(filler, 8 * 64, 2 * 4, 1000.0)
    want, wl = attend(w, q, [rows, rows])
    for scale in (1.0, 0.0):
        attend(filler, huge * scale, [64] * 8)
        got, gl = attend(w, q, [rows, rows])
        assert torch.equal(got, want) and torch.equal(gl, wl)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,G,hkv", MANY + [(1, 5, 2), (3, 5, 2)])
def test_rows_behind_the_last_sequence_leave_the_bits_alone(dtype, rows, G, hkv):
    w = World([1500, 1300], hkv, 64, 16, dtype, seed=rows)
    q = queries(w, 2 * rows + 9, hkv * G, 3.0)
    want, wl = attend(w, q, [rows, rows])
    for fill in (0.0, 500.0, float("inf"), float("nan")):
        q[2 * rows:] = fill
        got, gl = attend(w, q, [rows, rows])
        assert torch.equal(got[:2 * rows], want[:2 * rows]) and torch.equal(gl[:2 * rows], wl[:2 * rows]), fill
