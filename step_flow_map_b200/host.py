"""Host-side marshalling helpers built on torch device memory.

Uploads host arrays into device tensors of the library's storage type and
wraps the C context in a small object.  No step of the draft or verify
runs here.
"""
from __future__ import annotations

import contextlib

import numpy as np
import torch

from . import (FM_BF16, FM_F32, fm_append_args, fm_attention_args, fm_cache_append,
               fm_cache_attention, fm_cache_attention_workspace, fm_cache_evict, fm_draft,
               fm_draft_factorised, fm_free, fm_load_weights, fm_paged_cache, fm_project_context,
               fm_verify_greedy, fm_verify_sample)

TORCH_DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}
FM_DTYPE = {"f32": FM_F32, "bf16": FM_BF16}


def to_device(a, dtype: str = "f32", device="cuda") -> torch.Tensor:
    """Host array -> contiguous device tensor of storage type ``dtype``.

    fp64 arrays (uniforms) stay fp64; integer arrays keep their type; other
    floating arrays become ``dtype``.  For bf16 the values must already be
    bf16-representable; the cast is then exact.
    """
    t = torch.from_numpy(np.ascontiguousarray(a))
    if t.dtype == torch.float64:   # uniforms cross the ABI as fp64
        return t.to(device=device).contiguous()
    t = t.to(device=device, dtype=TORCH_DTYPE[dtype] if t.is_floating_point() else t.dtype)
    return t.contiguous()


class Context:
    """A loaded drafter: device weights plus the C context that borrows them."""

    def __init__(self, shape, dtype: str, weights: dict, max_ctx: int, max_seqs: int,
                 max_noise: int, max_new: int, device="cuda", stream=None):
        self.shape, self.dtype = shape, dtype
        self.weights = {k: to_device(v, dtype, device) for k, v in weights.items()}
        cfg = dict(V=shape.V, d=shape.d, n_blocks=shape.n_blocks, n_heads=shape.n_heads,
                   mlp=shape.mlp, K=shape.K, target_hidden=shape.hidden, n_taps=shape.n_taps,
                   dtype=FM_DTYPE[dtype], max_ctx=max_ctx, max_seqs=max_seqs,
                   max_noise=max_noise, max_new=max_new)
        self.cfg = cfg
        self.ctx = fm_load_weights(cfg, self.weights, stream)

    def close(self):
        if self.ctx:
            fm_free(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def project(self, seq_ids, hidden: torch.Tensor, pos0, stream=None):
        n_new = hidden.shape[1]
        fm_project_context(self.ctx, seq_ids, hidden, n_new, pos0, stream)

    def draft(self, seq_ids, noise: torch.Tensor, t_grid, temps, u_draft=None, logits=True,
              stream=None):
        n_seqs, n_noise, K, V = noise.shape
        tokens = torch.empty((n_seqs, n_noise, K), dtype=torch.int32, device=noise.device)
        out_logits = (torch.empty((n_seqs, n_noise, K, V), dtype=torch.float32, device=noise.device)
                      if logits else None)
        fm_draft(self.ctx, seq_ids, noise, n_noise, t_grid, temps, u_draft, tokens, out_logits,
                 stream)
        return tokens, out_logits

    def draft_factorised(self, seq_ids, noise: torch.Tensor, t_grid, temps, u_draft=None,
                         logits=True, stream=None):
        """noise [n_seqs, K, K, V]: position i of each block from noise block i."""
        n_seqs, K, _, V = noise.shape
        tokens = torch.empty((n_seqs, K), dtype=torch.int32, device=noise.device)
        out_logits = (torch.empty((n_seqs, K, V), dtype=torch.float32, device=noise.device)
                      if logits else None)
        fm_draft_factorised(self.ctx, seq_ids, noise, t_grid, temps, u_draft, tokens, out_logits,
                            stream)
        return tokens, out_logits

    def verify_greedy(self, target: torch.Tensor, draft: torch.Tensor, stream=None):
        B, N, K1, V = target.shape
        dev = target.device
        n = torch.empty(B, dtype=torch.int32, device=dev)
        br = torch.empty(B, dtype=torch.int32, device=dev)
        out = torch.empty((B, K1), dtype=torch.int32, device=dev)
        fm_verify_greedy(self.ctx, target, draft, B, N, K1 - 1, V, n, br, out, stream)
        return n, br, out

    def verify_sample(self, target, draft_logits, draft, T, u_accept, u_res, stream=None):
        B, N, K1, V = target.shape
        dev = target.device
        n = torch.empty(B, dtype=torch.int32, device=dev)
        br = torch.empty(B, dtype=torch.int32, device=dev)
        out = torch.empty((B, K1), dtype=torch.int32, device=dev)
        fm_verify_sample(self.ctx, target, draft_logits, draft, B, N, K1 - 1, V, T, u_accept,
                         u_res, n, br, out, stream)
        return n, br, out


_HERE = contextlib.nullcontext()   # the current device and stream serve as they are


class PagedCache:
    """One layer of the target's paged key/value cache: torch tensors in the
    library's layout, and the operators that work on them (argument checks and
    marshalling only; see the C header for every argument's meaning).

    k, v [n_pages, n_kv_heads, page_size, head_dim] (bf16 or fp32), page_table
    [n_seqs, table_stride] int32, pos [n_pages, n_kv_heads, page_size] int32 or
    None, weight (same shape) fp32 or None; all contiguous, on one GPU.  The
    tensors may be changed in place between calls; `page_table` may be
    replaced.

    Calls run on `stream`, or on the current stream of the cache's device;
    outputs and workspaces are allocated on that stream, one workspace per
    call, so calls on different streams (or captured in different graphs)
    share nothing but what they are given.  Given `stream`, a call keeps the
    allocator from handing out the memory of its tensors again, the cache's
    included, before that stream is done with them, so that they may be
    dropped at once; that they are written before it begins is up to the caller.
    """

    def __init__(self, k, v, page_table, pos=None, weight=None):
        if k.dtype not in (torch.bfloat16, torch.float32) or k.dim() != 4:
            raise ValueError("k must be [n_pages, n_kv_heads, page_size, head_dim], bf16 or fp32")
        self.k, self.v, self.pos, self.weight = k, v, pos, weight
        self.device = k.device
        self._ws_bytes = {}
        n_pages, n_kv, ps, dh = k.shape
        if k.is_cuda and k.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self._check("v", v, k.dtype, k.shape)
        for name, t, dt in (("pos", pos, torch.int32), ("weight", weight, torch.float32)):
            if t is not None:
                self._check(name, t, dt, k.shape[:3])
        if not k.is_contiguous():
            raise ValueError("k must be contiguous")
        self._c = fm_paged_cache(
            dtype=FM_BF16 if k.dtype == torch.bfloat16 else FM_F32, n_pages=n_pages, page_size=ps,
            n_kv_heads=n_kv, head_dim=dh, k=k.data_ptr(), v=v.data_ptr(),
            pos=pos.data_ptr() if pos is not None else None,
            weight=weight.data_ptr() if weight is not None else None)
        self.page_table = page_table

    @property
    def page_table(self):
        return self._table

    @page_table.setter
    def page_table(self, t):
        if t.dim() != 2:
            raise ValueError("page_table must be [n_seqs, table_stride]")
        self._check("page_table", t, torch.int32, t.shape)
        self._table = t
        self._lent = set()         # streams that the cache's tensors are lent to
        self._c.page_table, self._c.table_stride = t.data_ptr(), t.shape[1]

    def _check(self, name, t, dtype, shape):
        if t.shape != shape or t.dtype != dtype or t.device != self.device or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} "
                             f"on {self.device}")

    def _rows(self, name, t, T, heads):
        """Row stride of a [T, heads, head_dim] tensor whose heads are contiguous."""
        dh = self._c.head_dim
        if t.shape != (T, heads, dh) or t.dtype != self.k.dtype or t.device != self.device:
            raise ValueError(f"{name} must be [{T}, {heads}, {dh}] {self.k.dtype} on {self.device}")
        st = t.stride()
        if st[2] != 1 or (heads > 1 and st[1] != dh):
            if t.numel():
                raise ValueError(f"{name} must have contiguous heads")
        # one row's stride says nothing; any aligned one will do
        return st[0] if T > 1 else heads * dh

    def _seqs(self, T, cu_rows, kv_len, q_pos):
        B = kv_len.shape[0]
        self._check("kv_len", kv_len, torch.int32, (B,))
        self._check("cu_rows", cu_rows, torch.int32, (B + 1,))
        if B > self._table.shape[0]:
            raise ValueError(f"{B} sequences, {self._table.shape[0]} rows of page_table")
        if q_pos is not None:
            self._check("q_pos", q_pos, torch.int32, (T,))
        return B

    @staticmethod
    def _sizes(**given):
        """Whole numbers that the C structures hold in 32 bits (ctypes would wrap larger ones)."""
        for name, x in given.items():
            if not -2**31 <= x < 2**31:
                raise ValueError(f"{name} = {x} does not fit 32 bits")

    def _on(self, stream, *lent):
        """A context under which tensors are allocated on the cache's device and on
        `stream` (None: the device's current stream), and that stream, to which the
        tensors `lent` (None among them) and the cache's are lent."""
        if self.device.type != "cuda":
            raise ValueError(f"the cache is on {self.device}; its operators run on a GPU")
        if stream is None:   # (the public accessors cost 5 us, as much as a small call's kernels)
            dev = self.device.index
            st = torch._C._cuda_getCurrentRawStream(dev)
            return (_HERE if torch._C._cuda_getDevice() == dev else torch.cuda.device(dev)), st
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=self.device)
        elif stream.device != self.device:
            raise ValueError(f"stream of {stream.device}, cache on {self.device}")
        if stream.cuda_stream not in self._lent:   # (held until they are freed: once per stream is enough)
            self._lent.add(stream.cuda_stream)
            lent += (self.k, self.v, self.pos, self.weight, self._table)
        for t in lent:
            if t is not None:
                t.record_stream(stream)
        return torch.cuda.stream(stream), stream.cuda_stream

    def append(self, q, k, v, cu_rows, kv_len, q_pos=None, *, q_gain=None, k_gain=None, eps=1e-6,
               inv_freq=None, interleaved=False, out=None, stream=None):
        """Norms, rotates and appends the new rows; returns the queries [T, n_heads, head_dim]."""
        n_kv, dh = self._c.n_kv_heads, self._c.head_dim
        if q.dim() != 3:
            raise ValueError("q must be [T, n_heads, head_dim]")
        T, n_heads = q.shape[0], q.shape[1]
        qs = self._rows("q", q, T, n_heads)
        ks, vs = self._rows("k", k, T, n_kv), self._rows("v", v, T, n_kv)
        B = self._seqs(T, cu_rows, kv_len, q_pos)
        for name, g in (("q_gain", q_gain), ("k_gain", k_gain)):
            if g is not None:
                self._check(name, g, self.k.dtype, (dh,))
        rot = 0
        if inv_freq is not None:
            rot = 2 * inv_freq.shape[0]
            self._check("inv_freq", inv_freq, torch.float64, (rot // 2,))
        os = n_heads * dh if out is None else self._rows("out", out, T, n_heads)
        ctx, st = self._on(stream, q, k, v, cu_rows, kv_len, q_pos, q_gain, k_gain, inv_freq, out)
        with ctx:
            if out is None:
                out = q.new_empty(T, n_heads, dh)
            # positional, in the structure's order
            fm_cache_append(self._c, fm_append_args(
                T, B, n_heads, q.data_ptr(), k.data_ptr(), v.data_ptr(), qs, ks, vs,
                None if q_gain is None else q_gain.data_ptr(),
                None if k_gain is None else k_gain.data_ptr(), eps,
                inv_freq.data_ptr() if rot else None, rot, int(bool(interleaved)),
                cu_rows.data_ptr(), kv_len.data_ptr(),
                None if q_pos is None else q_pos.data_ptr(), out.data_ptr(), os), st)
        return out

    def attend(self, q, cu_rows, kv_len, *, max_rows, max_kv, q_pos=None, scale=None, window=0,
               sinks=0, accumulate=False, lse=False, out=None, stream=None):
        """Attention of the new rows; returns out, or (out, lse) with ``lse=True``."""
        if q.dim() != 3:
            raise ValueError("q must be [T, n_heads, head_dim]")
        T, n_heads, dh = q.shape
        qs = self._rows("q", q, T, n_heads)
        B = self._seqs(T, cu_rows, kv_len, q_pos)
        self._sizes(max_rows=max_rows, max_kv=max_kv, window=window, sinks=sinks)
        os = n_heads * dh if out is None else self._rows("out", out, T, n_heads)
        ctx, st = self._on(stream, q, cu_rows, kv_len, q_pos, out)
        with ctx:
            if out is None:
                out = q.new_empty(T, n_heads, dh)
            got = q.new_empty((T, n_heads), dtype=torch.float32) if lse else None
            a = fm_attention_args(
                T, B, n_heads, max_rows, max_kv, q.data_ptr(), qs, cu_rows.data_ptr(),
                kv_len.data_ptr(), None if q_pos is None else q_pos.data_ptr(),
                dh ** -0.5 if scale is None else scale, window, sinks, int(bool(accumulate)),
                out.data_ptr(), os, got.data_ptr() if lse else None)
            # a function of the sizes alone
            key = (T, B, n_heads, max_rows, max_kv, a.accumulate)
            ws_bytes = self._ws_bytes.get(key)
            if ws_bytes is None:
                if len(self._ws_bytes) > 256:
                    self._ws_bytes.clear()
                ws_bytes = self._ws_bytes[key] = fm_cache_attention_workspace(self._c, a)
            ws = self._table.new_empty(ws_bytes // 4)   # int32; (new_empty parses its arguments fastest)
            fm_cache_attention(self._c, a, ws, ws_bytes, st)
        return (out, got) if lse else out

    def evict(self, kv_len, next_pos, budget, *, max_kv, sinks=0, recent=0, new_len=None,
              stream=None):
        """Cuts every (sequence, head) to `budget` rows in place; returns the new lengths [B]."""
        B = kv_len.shape[0]
        self._check("kv_len", kv_len, torch.int32, (B,))
        self._check("next_pos", next_pos, torch.int32, (B,))
        if B > self._table.shape[0]:
            raise ValueError(f"{B} sequences, {self._table.shape[0]} rows of page_table")
        self._sizes(max_kv=max_kv, budget=budget, sinks=sinks, recent=recent)
        if new_len is not None:
            self._check("new_len", new_len, torch.int32, (B,))
        ctx, st = self._on(stream, kv_len, next_pos, new_len)
        with ctx:
            if new_len is None:
                new_len = kv_len.new_empty(B)
            fm_cache_evict(self._c, kv_len.data_ptr(), next_pos.data_ptr(), B, max_kv, budget, sinks,
                           recent, new_len.data_ptr(), st)
        return new_len
