"""What calls with sequences that overlap, and workspaces of the least size, leave alone:
the memory around outputs and workspaces, the cache and its tables."""
import pytest
import torch

import step_flow_map_b200 as fmb
from test_gpu_cache import DT, World, cu_of

pytestmark = pytest.mark.gpu

PAT = 0x5A


class Guarded:
    """A buffer with a patterned margin on either side."""

    def __init__(self, nbytes, margin=4096):
        self.n, self.margin = nbytes, margin
        self.buf = torch.full((nbytes + 2 * margin + 256,), PAT, dtype=torch.uint8, device="cuda")
        self.off = margin + (-(self.buf.data_ptr() + margin)) % 256
        self.ptr = self.buf.data_ptr() + self.off

    def intact(self):
        return bool((self.buf[:self.off] == PAT).all()) and bool((self.buf[self.off + self.n:] == PAT).all())


# decode, one query tile, pairs of them (bf16) / prompt tiles (fp32)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("max_rows", [2, 12, 300])
@pytest.mark.parametrize("accumulate", [0, 1])
def test_sequences_that_overlap_touch_nothing_else(dtype, max_rows, accumulate):
    """cu_rows that goes back and forth, against the rules, with a workspace of the least size:
    the margins around workspace, output and lse, the cache and the tables keep their bits."""
    B, T, G, L = 40, 300, 8, 300
    w = World([L] * B, 1, 64, 16, dtype, seed=3, weight=True)
    es = 2 if dtype == "bf16" else 4
    q = torch.tensor(w.rng.normal(size=(T, G, 64))).to(DT[dtype]).cuda()
    out, lse = Guarded(T * G * 64 * es), Guarded(T * G * 4)
    view = w.cache._c
    for cu in ([0, T] * (B // 2) + [0], [0] + [T] * B, [0] + [2 ** 31 - 1] * B, [-5, T] * (B // 2) + [7], list(range(0, 8 * B + 1, 8))):
        cu = torch.tensor(cu, dtype=torch.int32).cuda()
        a = fmb.fm_attention_args(T=T, B=B, n_heads=G, max_rows=max_rows, max_kv=L, q=q.data_ptr(), q_stride=G * 64,
                                  cu_rows=cu.data_ptr(), kv_len=w.kv.data_ptr(), scale=0.125, accumulate=accumulate,
                                  out=out.ptr, out_stride=G * 64, lse=lse.ptr)
        need = fmb.fm_cache_attention_workspace(view, a)
        ws = Guarded(need)
        same = {n: getattr(w, n).clone() for n in ("k", "v", "kv", "t")}
        fmb.fm_cache_attention(view, a, ws.ptr, need, torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert ws.intact() and out.intact() and lse.intact(), cu.tolist()[:4]
        for n, x in same.items():
            assert torch.equal(torch.nan_to_num(getattr(w, n).float()), torch.nan_to_num(x.float())), n
        with pytest.raises(fmb.FlashmapError):
            fmb.fm_cache_attention(view, a, ws.ptr, need - 1, None)


def test_a_workspace_of_the_least_size_serves():
    for dtype in ("bf16", "f32"):
        for rows, acc in ((1, 1), (2, 0), (12, 1), (40, 0), (40, 1)):
            w = World([500, 0, 777], 2, 64, 16, dtype, seed=rows, weight=True)
            n = [rows, 0, rows]
            q = torch.tensor(w.rng.normal(size=(2 * rows, 8, 64))).to(DT[dtype]).cuda()
            had = w.weight.clone()
            want = w.cache.attend(q, cu_of(n), w.kv, max_rows=rows, max_kv=777, accumulate=bool(acc))
            got_w = w.weight.clone()
            w.weight.copy_(had)
            out, cu = Guarded(want.numel() * want.element_size()), cu_of(n)
            a = fmb.fm_attention_args(T=2 * rows, B=3, n_heads=8, max_rows=rows, max_kv=777, q=q.data_ptr(), q_stride=8 * 64,
                                      cu_rows=cu.data_ptr(), kv_len=w.kv.data_ptr(), scale=64 ** -0.5, accumulate=acc,
                                      out=out.ptr, out_stride=8 * 64)
            need = fmb.fm_cache_attention_workspace(w.cache._c, a)
            ws = Guarded(need)
            fmb.fm_cache_attention(w.cache._c, a, ws.ptr, need, torch.cuda.current_stream().cuda_stream)
            torch.cuda.synchronize()
            assert ws.intact() and out.intact()
            got = out.buf[out.off:out.off + out.n].view(want.dtype).view(want.shape)
            assert torch.equal(got, want) and torch.equal(w.weight, got_w)
