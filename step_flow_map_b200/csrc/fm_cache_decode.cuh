// Attention of few new rows over the paged cache (bf16, at most 16 packed
// rows per key/value head: one token, or a short block).
//
// Bound: HBM -- every visible key and value is read once and used by at most
// 16 rows, 16 FLOP per byte and below, so the kernel is a stream with an
// online softmax (mma.sync m16n8k16, whose M is the 16 packed rows; at this
// ratio the legacy tensor path is far from its limit and needs no TMEM round
// trip per 16 keys).  A unit is 64 cache rows of one (sequence, head); each of
// the four warps owns 16 of them and its own three-stage cp.async ring (16
// rows of a head are one contiguous block of a page), so the loop has no CTA
// barrier, and the ring runs on across tiles of different sequences.  The
// lengths' prefix sum (at most 256 sequences) is taken by every CTA itself,
// which is cheaper than a launch.
#pragma once
#include "fm_cache_attn.cuh"
#include "fm_ptx.cuh"

namespace fm {

constexpr int CD_THREADS = 128;
constexpr int CD_KB = 64;          // cache rows per unit
constexpr int CD_STAGES = 3;
constexpr int CD_QT = 16;

// Where every sequence's units begin, and what it sees.
struct DecodeSeqs {
  int first[257];                  // prefix sums of blocks (heads apart)
  int s_end[256], lo[256], hi[256];
  int row0[256], n[256], len[256];
};
template <int KB>
__device__ __forceinline__ void decode_scan(const CacheAttnArgs& a, DecodeSeqs& s, int* sh) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int nb[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int b = tid * 2 + k;
    nb[k] = 0;
    if (b < a.B) {
      const NewRows r = new_rows(a.cu, a.kv_len, b, a.T);
      const int n = min(r.n, a.max_rows);
      const SeenRows v = seen_rows(a, r, 0, max(0, n - 1));
      if (n > 0) nb[k] = SeenBlocks<KB>(v).nb;
      s.s_end[b] = v.s_end;
      s.lo[b] = v.lo;
      s.hi[b] = v.hi;
      s.row0[b] = r.first;
      s.n[b] = n;
      s.len[b] = r.L - r.n;        // position of its first new row
    }
  }
  int x = nb[0] + nb[1];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sh[warp] = x;
  __syncthreads();
  int add = 0;
#pragma unroll
  for (int i = 0; i < CD_THREADS / 32; ++i)
    if (i < warp) add += sh[i];
  s.first[tid * 2 + 1] = add + x - nb[1];
  s.first[tid * 2 + 2] = add + x;
  if (tid == 0) s.first[0] = 0;
  __syncthreads();
}
__device__ __forceinline__ int decode_find(const CacheAttnArgs& a, const DecodeSeqs& s, int u) {
  int b = 0;
#pragma unroll
  for (int step = 128; step > 0; step >>= 1)
    if (s.first[b + step] * a.c.n_kv <= u) b += step;
  return b;
}

// A unit of the CTA's run: block j of head g of sequence b.
struct DecodeCursor {
  int b, g, j, nb;
  __device__ __forceinline__ void seek(const CacheAttnArgs& a, const DecodeSeqs& s, int u) {
    b = decode_find(a, s, u);
    nb = s.first[b + 1] - s.first[b];
    const int at = u - s.first[b] * a.c.n_kv;
    g = at / nb;
    j = at - g * nb;
  }
  __device__ __forceinline__ void next(const CacheAttnArgs& a, const DecodeSeqs& s) {
    if (++j < nb) return;
    j = 0;
    if (++g < a.c.n_kv) return;
    g = 0;
    do {
      ++b;
      nb = b < 256 ? s.first[b + 1] - s.first[b] : 1;
    } while (nb == 0);
  }
};

template <int DH>
struct CdCfg {
  static constexpr int TILE = 16 * DH * 2;             // bytes of a warp's 16 keys (or values)
  static constexpr int STAGE = 2 * TILE + 64;          // keys, values, positions
  static constexpr int RING = CD_STAGES * STAGE;
  static constexpr int MLD = DH + 4;                   // merge buffer row
  static constexpr int SMEM = 4 * RING + 4 * 4 * MLD * 4;
};

template <int DH>
__global__ void __launch_bounds__(CD_THREADS, 2) k_cache_decode(const CacheAttnArgs a) {
  using C = CdCfg<DH>;
  constexpr int CH = DH / 8;       // 16-byte pieces of a row
  extern __shared__ __align__(16) uint8_t smb[];
  __shared__ DecodeSeqs s;
  __shared__ int s_scan[4];
  __shared__ float2 s_ml[4][CD_QT];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_trigger();
  decode_scan<CD_KB>(a, s, s_scan);
  const WorkRun w(s.first[256] * a.c.n_kv, gridDim.x);
  if ((int)blockIdx.x >= w.g || w.N == 0) {
    if (tid == 0) a.plan_join[2 * blockIdx.x] = make_int4(-1, 0, 0, 0);
    return;
  }
  const int u0 = w.start(blockIdx.x), count = w.start(blockIdx.x + 1) - u0;
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smb) + warp * C::RING;
  float* merge = (float*)(smb + 4 * C::RING);

  DecodeCursor ld, cu;
  ld.seek(a, s, u0);
  cu = ld;
  if (tid == 0)
    put_join(a, w, blockIdx.x, u0 - ld.j, ld.nb, s.row0[ld.b], ld.g, 0, s.n[ld.b] * a.G);
  auto tile_row = [&](const DecodeCursor& c) {
    const SeenRows v = {s.s_end[c.b], s.lo[c.b], s.hi[c.b]};
    return SeenBlocks<CD_KB>(v).row(c.j) + 16 * warp;
  };
  int ld_row = tile_row(ld), ld_page = cache_page(a.c, ld.b, ld_row);
  // stage `st` <- the load cursor's unit; then the cursor moves on and its
  // page number starts loading
  auto load = [&](int st, bool more) {
    const SeenRows v = {s.s_end[ld.b], s.lo[ld.b], s.hi[ld.b]};
    const uint32_t dst = ring + st * C::STAGE;
    const size_t at = cache_row(a.c, max(ld_page, 0), ld.g, ld_row);
    const char* gk = (const char*)a.c.k + at * (DH * 2);
    const char* gv = (const char*)a.c.v + at * (DH * 2);
#pragma unroll
    for (int i = 0; i < CH / 2; ++i) {
      const int x = lane + 32 * i, r = x / CH, c = x % CH;
      const bool live = ld_page >= 0 && row_seen(v, ld_row + r);
      const uint32_t o = r * (DH * 2) + ((c ^ (r & 7)) << 4);
      cp_async16_if(dst + o, gk + x * 16, live);
      cp_async16_if(dst + C::TILE + o, gv + x * 16, live);
    }
    if (a.c.pos && lane < 4)
      cp_async16_if(dst + 2 * C::TILE + lane * 16, a.c.pos + at + lane * 4, ld_page >= 0);
    if (more) {
      ld.next(a, s);
      ld_row = tile_row(ld);
      ld_page = cache_page(a.c, ld.b, ld_row);
    }
  };
  int issued = 0;
#pragma unroll
  for (int i = 0; i < CD_STAGES - 1; ++i) {
    if (issued < count) {
      ++issued;
      load(i, issued < count);
    }
    cp_commit();
  }
  int cu_page = cache_page(a.c, cu.b, tile_row(cu));

  const int gr = lane >> 2, t4 = lane & 3;
  int done = 0, stage = 0;
  while (done < count) {
    // ---- one tile: the units of (cu.b, cu.g) in this run
    const int b = cu.b, g = cu.g, j0 = cu.j, nb = cu.nb;
    const int todo = min(nb - j0, count - done);
    const int rows = s.n[b] * a.G, row0 = s.row0[b], p0 = s.len[b];
    const SeenRows seen = {s.s_end[b], s.lo[b], s.hi[b]};
    uint32_t qa[DH / 16][4];
    int pq[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int x = gr + 8 * h;
      const bool live = x < rows;
      const int qi = live ? x / a.G : 0;
      const bf16* qr = (const bf16*)a.q + (row0 + qi) * a.qs + (g * a.G + (live ? x % a.G : 0)) * DH;
      pq[h] = a.q_pos ? __ldg(a.q_pos + row0 + qi) : p0 + qi;
#pragma unroll
      for (int k = 0; k < DH / 16; ++k) {
        qa[k][h] = live ? *(const uint32_t*)(qr + k * 16 + 2 * t4) : 0u;
        qa[k][2 + h] = live ? *(const uint32_t*)(qr + k * 16 + 8 + 2 * t4) : 0u;
      }
    }
    const int p_last = p0 + s.n[b] - 1;
    float o[DH / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int n = 0; n < DH / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;

    for (int it = 0; it < todo; ++it) {
      cp_wait<CD_STAGES - 2>();
      __syncwarp();
      {
        // refill the stage freed by the previous unit
        const int st = stage == 0 ? CD_STAGES - 1 : stage - 1;
        if (issued < count) {
          ++issued;
          load(st, issued < count);
        }
        cp_commit();
      }
      const int r0 = tile_row(cu);
      const bool there = cu_page >= 0;
      if (it + 1 < todo) {
        cu.next(a, s);
        cu_page = cache_page(a.c, cu.b, tile_row(cu));
      }
      const uint32_t kt = ring + stage * C::STAGE, vt = kt + C::TILE;
      const int* kp = (const int*)(smb + warp * C::RING + stage * C::STAGE + 2 * C::TILE);
      // nothing of the tile is visible: skip it
      if (there && (r0 < seen.s_end || (r0 + 16 > seen.lo && r0 < seen.hi))) {
        float sc[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.f;
#pragma unroll
        for (int k = 0; k < DH / 16; ++k) {
          const int r = (lane & 7) + ((lane >> 4) << 3), c = 2 * k + ((lane >> 3) & 1);
          uint32_t b0, b1, b2, b3;
          ldsm_x4(kt + r * (DH * 2) + ((c ^ (r & 7)) << 4), b0, b1, b2, b3);
          mma_bf16(sc[0], qa[k], b0, b1);
          mma_bf16(sc[1], qa[k], b2, b3);
        }
        // every row visible to every query?
        const bool open = !a.c.pos && r0 >= seen.lo && r0 + 15 <= p0 && r0 + 16 <= seen.hi &&
                          (a.window == 0 || p_last - r0 < a.window);
        float mx[2] = {m[0], m[1]};
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float v = sc[n][e] * a.scale_log2;
            if (!open) {
              const int kr = n * 8 + 2 * t4 + (e & 1), r = r0 + kr;
              const int pk = a.c.pos ? kp[kr] : r;
              if (!(row_seen(seen, r) && sees(pq[e >> 1], pk, a.window, a.sinks))) v = -INFINITY;
            }
            sc[n][e] = v;
            mx[e >> 1] = fmaxf(mx[e >> 1], v);
          }
        if (a.scores) {            // kept for the weights: 2 keys, 8 bytes, a thread and row
          float* dst = a.scores + score_at(a, b, g, r0, 0) + 2 * t4;
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (gr + 8 * h < rows)
#pragma unroll
              for (int n = 0; n < 2; ++n)
                *(float2*)(dst + (gr + 8 * h) * 16 + n * 8) = make_float2(sc[n][2 * h], sc[n][2 * h + 1]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
          mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
        }
        if (__any_sync(0xffffffffu, mx[0] > m[0] || mx[1] > m[1])) {
          float cr[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            cr[h] = mx[h] == -INFINITY ? 1.f : ex2(m[h] - mx[h]);
            m[h] = mx[h];
            l[h] *= cr[h];
          }
#pragma unroll
          for (int n = 0; n < DH / 8; ++n) {
            o[n][0] *= cr[0]; o[n][1] *= cr[0];
            o[n][2] *= cr[1]; o[n][3] *= cr[1];
          }
        }
        const float ref0 = m[0] == -INFINITY ? 0.f : m[0], ref1 = m[1] == -INFINITY ? 0.f : m[1];
        // probabilities enter the product rounded to bf16 (the tensor path's
        // type); the sum, and so lse, takes them as they are
        uint32_t pa[4];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[n][e] = ex2(sc[n][e] - (e < 2 ? ref0 : ref1));
          l[0] += sc[n][0] + sc[n][1];
          l[1] += sc[n][2] + sc[n][3];
          pa[2 * n] = pack_bf16x2(sc[n][0], sc[n][1]);
          pa[2 * n + 1] = pack_bf16x2(sc[n][2], sc[n][3]);
        }
#pragma unroll
        for (int n = 0; n < DH / 16; ++n) {
          const int r = lane & 15, c = 2 * n + (lane >> 4);
          uint32_t b0, b1, b2, b3;
          ldsm_x4_t(vt + r * (DH * 2) + ((c ^ (r & 7)) << 4), b0, b1, b2, b3);
          mma_bf16(o[2 * n], pa, b0, b1);
          mma_bf16(o[2 * n + 1], pa, b2, b3);
        }
      }
      stage = stage + 1 == CD_STAGES ? 0 : stage + 1;
    }
    // ---- the four warps' states into one
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      if (t4 == 0) s_ml[warp][gr + 8 * h] = make_float2(m[h], l[h]);
    }
    const bool whole = j0 == 0 && todo == nb;
    const int slot = done == 0 ? 0 : 1;
    // four rows at a time through the merge buffer
    for (int x0 = 0; x0 < rows; x0 += 4) {
      __syncthreads();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int x = gr + 8 * h - x0;
        if (x >= 0 && x < 4) {
          float* dst = merge + (warp * 4 + x) * C::MLD + 2 * t4;
#pragma unroll
          for (int n = 0; n < DH / 8; ++n) *(float2*)(dst + n * 8) = make_float2(o[n][2 * h], o[n][2 * h + 1]);
        }
      }
      __syncthreads();
      const int x = x0 + warp;     // a warp finishes a row, DH / 32 columns a lane
      if (x < rows) {
        float mm = -INFINITY, ll = 0.f, f[4], acc[DH / 32];
#pragma unroll
        for (int i = 0; i < 4; ++i) mm = fmaxf(mm, s_ml[i][x].x);
        const float ref = mm == -INFINITY ? 0.f : mm;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f[i] = ex2(s_ml[i][x].x - ref);
          ll = fmaf(s_ml[i][x].y, f[i], ll);
        }
#pragma unroll
        for (int k = 0; k < DH / 32; ++k) acc[k] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int k = 0; k < DH / 32; ++k)
            acc[k] = fmaf(merge[(i * 4 + warp) * C::MLD + lane * (DH / 32) + k], f[i], acc[k]);
        if (whole) {
          const int t = row0 + x / a.G, h = g * a.G + x % a.G;
          const float inv = ll != 0.f ? 1.f / ll : 0.f;
          uint32_t* dst = (uint32_t*)((bf16*)a.out + t * a.os + h * DH) + lane * (DH / 64);
#pragma unroll
          for (int k = 0; k < DH / 64; ++k) dst[k] = pack_bf16x2(acc[2 * k] * inv, acc[2 * k + 1] * inv);
          if (a.lse && lane == 0)
            a.lse[(size_t)t * a.n_heads + h] =
                ll != 0.f ? (mm + log2f(ll)) * 0.69314718055994531f : -INFINITY;
        } else {
          const size_t p = ((size_t)blockIdx.x * 2 + slot) * CD_QT + x;
#pragma unroll
          for (int k = 0; k < DH / 32; ++k) a.part[p * DH + lane * (DH / 32) + k] = acc[k];
          if (lane == 0) a.part_ml[p] = make_float2(mm, ll);
        }
      }
    }
    __syncthreads();               // s_ml and the buffer are free again
    done += todo;
    if (done < count) {
      cu.next(a, s);
      cu_page = cache_page(a.c, cu.b, tile_row(cu));
    }
  }
  cp_wait<0>();
}

}  // namespace fm
