// Accumulated attention weight of many new rows (bf16): weight_r += sum over
// the packed rows of e^(s - lse), see fm_cache_attn.cuh.
//
// D = K Q^T with the keys on the MMA's M side (mma.sync m16n8k16): a warp holds
// 16 keys as A fragments for the whole call, walks over the queries in chunks
// of 64 that its CTA stages in shared memory, and adds the probabilities of its
// rows up in registers -- a column sum of the attention matrix without a
// transpose or an atomic.  Bound: HBM (the keys once, 256 bytes a row of width
// 128) for drafted blocks, the exponentials for prompts.
#pragma once
#include "fm_cache_attn.cuh"
#include "fm_ptx.cuh"

namespace fm {

constexpr int WM_THREADS = 256;    // 8 warps of 16 keys
constexpr int WM_KEYS = 128;
constexpr int WM_CHUNK = 64;       // packed rows staged at a time

template <int DH>
struct WmCfg {
  static constexpr int SMEM = (WM_KEYS + WM_CHUNK) * DH * 2;
};

template <int DH>
__global__ void __launch_bounds__(WM_THREADS) k_cache_weights_mma(const CacheAttnArgs a) {
  constexpr int CH = DH / 8;       // 16-byte pieces of a row
  extern __shared__ __align__(16) uint8_t smb[];
  __shared__ float s_lse[WM_CHUNK];
  __shared__ int s_pq[WM_CHUNK];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = blockIdx.y, b = blockIdx.z;
  const int gr = lane >> 2, t4 = lane & 3;
  pdl_wait();
  pdl_trigger();
  const NewRows s = new_rows(a.cu, a.kv_len, b, a.T);
  const int n = min(s.n, a.max_rows), rows = n * a.G;
  if (n == 0) return;
  const SeenRows seen = seen_rows(a, s, 0, n - 1);
  const uint32_t sk = (uint32_t)__cvta_generic_to_shared(smb), sq = sk + WM_KEYS * DH * 2;
  for (int r0 = blockIdx.x * WM_KEYS; r0 < seen.hi; r0 += gridDim.x * WM_KEYS) {
    // blocks that nobody sees (the same decision in every thread)
    if (!(r0 < seen.s_end || r0 + WM_KEYS > seen.lo)) continue;
    __syncthreads();
    for (int i = tid; i < WM_KEYS * CH; i += WM_THREADS) {
      const int y = i / CH, c = i % CH, r = r0 + y;
      const int page = row_seen(seen, r) ? cache_page(a.c, b, r) : -1;
      const bf16* src = (const bf16*)a.c.k + cache_row(a.c, max(page, 0), g, r) * DH;
      cp_async16_if(sk + y * (DH * 2) + ((c ^ (y & 7)) << 4), src + c * 8, page >= 0);
    }
    cp_commit();
    int pk[2];
    size_t at[2];
    bool ok[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = r0 + warp * 16 + gr + 8 * h;
      const int page = row_seen(seen, r) ? cache_page(a.c, b, r) : -1;
      ok[h] = page >= 0;
      at[h] = cache_row(a.c, max(page, 0), g, r);
      pk[h] = ok[h] && a.c.pos ? a.c.pos[at[h]] : r;
    }
    cp_wait<0>();
    __syncthreads();
    uint32_t ka[DH / 16][4];
#pragma unroll
    for (int k = 0; k < DH / 16; ++k) {
      const int y = warp * 16 + (lane & 15), c = 2 * k + (lane >> 4);
      ldsm_x4(sk + y * (DH * 2) + ((c ^ (y & 7)) << 4), ka[k][0], ka[k][1], ka[k][2], ka[k][3]);
    }
    float sum[2] = {0.f, 0.f};
    for (int x0 = 0; x0 < rows; x0 += WM_CHUNK) {
      // chunks whose queries all come before these keys see none of them
      if (!a.c.pos && s.L - s.n + min(x0 + WM_CHUNK - 1, rows - 1) / a.G < r0) continue;
      __syncthreads();
      for (int i = tid; i < WM_CHUNK * CH; i += WM_THREADS) {
        const int y = i / CH, c = i % CH, x = x0 + y;
        const bool live = x < rows;
        const int qi = live ? x / a.G : 0;
        const bf16* src = (const bf16*)a.q + (s.first + qi) * a.qs + (g * a.G + (live ? x % a.G : 0)) * DH;
        cp_async16_if(sq + y * (DH * 2) + ((c ^ (y & 7)) << 4), src + c * 8, live);
      }
      cp_commit();
      if (tid < WM_CHUNK) {
        const int x = x0 + tid;
        float l = INFINITY;        // 2^(s - inf) = 0: rows past the end, rows that see nothing
        int pq = 0;
        if (x < rows) {
          const int t = s.first + x / a.G;
          const float v = a.lse[(size_t)t * a.n_heads + g * a.G + x % a.G];
          if (v != -INFINITY) l = v * 1.4426950408889634f;
          pq = a.q_pos ? __ldg(a.q_pos + t) : s.L - s.n + x / a.G;
        }
        s_lse[tid] = l;
        s_pq[tid] = pq;
      }
      cp_wait<0>();
      __syncthreads();
#pragma unroll 2
      for (int q0 = 0; q0 < WM_CHUNK; q0 += 16) {
        float d[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) d[i][0] = d[i][1] = d[i][2] = d[i][3] = 0.f;
#pragma unroll
        for (int k = 0; k < DH / 16; ++k) {
          const int y = q0 + (lane & 7) + ((lane >> 4) << 3), c = 2 * k + ((lane >> 3) & 1);
          uint32_t b0, b1, b2, b3;
          ldsm_x4(sq + y * (DH * 2) + ((c ^ (y & 7)) << 4), b0, b1, b2, b3);
          mma_bf16(d[0], ka[k], b0, b1);
          mma_bf16(d[1], ka[k], b2, b3);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int y = q0 + i * 8 + 2 * t4 + (e & 1), h = e >> 1;
            const float p = ex2(fmaf(d[i][e], a.scale_log2, -s_lse[y]));
            if (sees(s_pq[y], pk[h], a.window, a.sinks)) sum[h] += p;
          }
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 1);
      sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 2);
      if (t4 == 0 && ok[h]) a.c.weight[at[h]] += sum[h];
    }
  }
}

}  // namespace fm
