// The target's paged key/value cache: norms, rotation and append of new rows,
// and eviction by accumulated attention weight.  (The attention over the
// pages is in fm_cache_attn.cuh.)
//
// Layout of one layer: k, v [n_pages][n_kv_heads][page_size][head_dim], so a
// head's rows of a page are one contiguous block, which a tensor map or a
// warp of 16-byte loads reads without a gap; pos and weight
// [n_pages][n_kv_heads][page_size].
#pragma once
#include "fm_common.cuh"

namespace fm {

struct CacheView {
  int n_pages, ps_log2, n_kv, table_stride;
  void *k, *v;
  int* pos;
  float* weight;
  const int* table;
};

// Page of row r of sequence b, -1 when the row does not exist.
__device__ __forceinline__ int cache_page(const CacheView& c, int b, int r) {
  const int i = r >> c.ps_log2;
  if (r < 0 || i >= c.table_stride) return -1;
  const int pg = __ldg(c.table + (size_t)b * c.table_stride + i);
  return (unsigned)pg < (unsigned)c.n_pages ? pg : -1;
}
// Index of (page, head, row in page) in units of rows.
__device__ __forceinline__ size_t cache_row(const CacheView& c, int page, int g, int r) {
  return (((size_t)page * c.n_kv + g) << c.ps_log2) + (r & ((1 << c.ps_log2) - 1));
}

// New rows of sequence b: [first, first + n) of the T given ones; L: its
// length with them.
struct NewRows {
  int first, n, L;
};
__device__ __forceinline__ NewRows new_rows(const int* cu, const int* kv_len, int b, int T) {
  NewRows s;
  const int a = min(max(__ldg(cu + b), 0), T), e = min(max(__ldg(cu + b + 1), a), T);
  s.first = a;
  s.n = e - a;
  s.L = max(__ldg(kv_len + b), 0);
  return s;
}

// ------------------------------------------------------------------ append
// y = x / sqrt(mean(x^2) + eps) * gain per head, then pair i of the first
// rot_dim values turns by position * inv_freq[i]: (a, b) -> (a cos - b sin,
// b cos + a sin).
//
// Bound: for many rows the instructions per 16 bytes (12,709 rows, ncu: 0.71
// issued a cycle and scheduler, DRAM at 55 % of the copy rate; stalls are fixed
// latencies and the norm's shuffles), then HBM (every value read once and
// written once); launch and one chain of dependent loads for few.  A thread holds 16 bytes of one
// head, head_dim * size / 16 neighbouring lanes hold the head, so the norm is
// a few shuffles and a half-split pair one shuffle.  A CTA takes `tok` rows:
// its warps find the rows' sequences, pages and angles side by side (one fp64
// product and reduction per pair) while the first row's values are already
// loading, and leave for every value of a head the cosine and the signed sine
// of its term, in the order the threads read them; a row's angles then sit in
// registers for all its heads.  Each row is loaded while the row before it is
// worked on.  (Angles looked up by pair at each use
// took 108 us for 12,709 rows of 48 heads of width 128 in bf16; this takes 72,
// 4.3 TB/s.  At 80 registers three CTAs fit an SM; four at 64 took 80 us, two
// at 96 85.)  tok, the rows over four per SM, is 1 while rows are fewer than eight
// per SM and grows to 8, so that the chain at a CTA's start is paid once per 8
// rows.
constexpr int CA_THREADS = 256;
constexpr int CA_MAX_TOK = 8;     // rows of one CTA
constexpr int CA_UNROLL = 3;      // 16-byte loads in flight per thread

struct AppendArgs {
  CacheView c;
  int T, B, n_heads, tok;         // tok: rows per CTA
  const void *q, *k, *v;
  int64_t qs, ks, vs, os;         // row strides (elements)
  const void *qg, *kg;
  float eps;
  const double* inv_freq;
  int rot, interleaved;
  const int *cu, *kv_len, *q_pos;
  void* q_out;
};

template <typename T> struct Vec16;
template <> struct Vec16<bf16> {
  static constexpr int N = 8;
  __device__ static void unpack(const uint4& u, float* f) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ static uint4 pack(const float* f) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
  }
};
template <> struct Vec16<float> {
  static constexpr int N = 4;
  __device__ static void unpack(const uint4& u, float* f) {
    f[0] = __uint_as_float(u.x); f[1] = __uint_as_float(u.y);
    f[2] = __uint_as_float(u.z); f[3] = __uint_as_float(u.w);
  }
  __device__ static uint4 pack(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
};

template <typename T, int DH, bool INTER>
__global__ void __launch_bounds__(CA_THREADS, 3) k_cache_append(const AppendArgs a) {
  constexpr int VE = Vec16<T>::N, LPH = DH / VE;   // values per thread, lanes per head
  constexpr int STEP = CA_THREADS / LPH;           // heads the CTA covers at once
  constexpr int PAIRS = (DH / 2 + 31) / 32;
  // (cosine, signed sine) of value c of a head at [c % VE][c / VE]
  __shared__ float2 s_cs[CA_MAX_TOK][VE][LPH];
  __shared__ int s_page[CA_MAX_TOK], s_row[CA_MAX_TOK], s_pos[CA_MAX_TOK];
  const int t0 = blockIdx.x * a.tok, nt = min(a.tok, a.T - t0);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int heads = a.n_heads + 2 * a.c.n_kv;
  const int sub = tid & (LPH - 1);
  pdl_wait();
  pdl_trigger();

  // rows side by side when their heads are fewer than STEP; this thread's
  // first row and head
  const int side = max(1, STEP / heads), slot = tid / LPH;
  const int j0 = side == 1 ? 0 : slot / heads, h0 = side == 1 ? slot : slot - j0 * heads;
  const int j_end = j0 < side ? nt : 0;
  // heads are numbered q, k, v; the k and v row pointers stand so far back
  // that head h of any kind lies h DH values on
  const int k_at = a.n_heads, v_at = a.n_heads + a.c.n_kv;
  const T *pq = (const T*)a.q + (t0 + j0) * a.qs + sub * VE,
          *pk = (const T*)a.k + (t0 + j0) * a.ks + sub * VE - k_at * DH,
          *pv = (const T*)a.v + (t0 + j0) * a.vs + sub * VE - v_at * DH;
  auto load = [&](int h) -> uint4 {
    return *(const uint4*)((h < k_at ? pq : h < v_at ? pk : pv) + h * DH);
  };
  uint4 x[CA_UNROLL];
#pragma unroll
  for (int u = 0; u < CA_UNROLL; ++u)
    if (j0 < j_end && h0 + u * STEP < heads) x[u] = load(h0 + u * STEP);
  uint4 gq = make_uint4(0, 0, 0, 0), gk = gq;
  if (a.qg) gq = __ldg((const uint4*)a.qg + sub);
  if (a.kg) gk = __ldg((const uint4*)a.kg + sub);

  // a warp per row: its sequence (all of cu_rows and kv_len in one round of
  // loads), page and angles
  for (int j = warp; j < nt; j += CA_THREADS / 32) {
    const int t = t0 + j;
    const int given = a.q_pos ? __ldg(a.q_pos + t) : 0;
    double f[PAIRS];
#pragma unroll
    for (int k = 0; k < PAIRS; ++k) {
      const int i = lane + 32 * k;
      f[k] = i < a.rot / 2 ? a.inv_freq[i] : 0.0;
    }
    int row = -1, seq = -1;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      const int b = b0 + lane;
      if (b < a.B) {
        const NewRows s = new_rows(a.cu, a.kv_len, b, a.T);
        if (t >= s.first && t < s.first + s.n) {
          row = s.L - s.n + (t - s.first);
          seq = b;
        }
      }
    }
    const unsigned hit = __ballot_sync(0xffffffffu, seq >= 0);
    if (hit) {
      row = __shfl_sync(0xffffffffu, row, __ffs((int)hit) - 1);
      seq = __shfl_sync(0xffffffffu, seq, __ffs((int)hit) - 1);
    }
    const int p = a.q_pos ? given : row;
    if (lane == 0) {
      s_pos[j] = p;
      s_row[j] = row;
      s_page[j] = hit ? cache_page(a.c, seq, row) : -2;   // -2: a row of no sequence
    }
    // turns = position * f / (2 pi), whose whole part drops out: two products and
    // a constant rounded to fp64, so off by at most 3 2^-53 of the turns, 1e-10 of
    // a turn up to 300,000 turns and 1.2e-7 at the last 32-bit position (f = 1)
#pragma unroll
    for (int k = 0; k < PAIRS; ++k) {
      const int i = lane + 32 * k;
      if (i < a.rot / 2) {
        const double turns = (double)p * f[k] * 0.15915494309189533577;
        float c, s;
        sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
        const int lo = INTER ? 2 * i : i, hi = INTER ? 2 * i + 1 : i + a.rot / 2;
        s_cs[j][lo % VE][lo / VE] = make_float2(c, -s);
        s_cs[j][hi % VE][hi / VE] = make_float2(c, s);
      }
    }
  }
  __syncthreads();

  if (a.c.pos || a.c.weight)
    for (int i = tid; i < nt * a.c.n_kv; i += CA_THREADS) {
      const int j = i / a.c.n_kv, g = i - j * a.c.n_kv;
      if (s_page[j] < 0) continue;
      const size_t at = cache_row(a.c, s_page[j], g, s_row[j]);
      if (a.c.pos) a.c.pos[at] = s_pos[j];
      if (a.c.weight) a.c.weight[at] = 0.f;
    }

  // shuffles stay among a head's lanes, which always branch together
  const unsigned m = LPH == 32 ? 0xffffffffu : ((1u << (LPH & 31)) - 1u) << (lane & ~(LPH - 1));
  // half-split pairs: a thread's values pair with those rot/2 on (or back), a
  // whole number of lanes away (rot is a multiple of 16)
  const int c0 = sub * VE, far = (a.rot >> 1) / VE;
  // values past rot stay as they are: an angle of zero would not do, as 0 x inf
  // is no 0 (rot is a multiple of 16, so this holds for all of a thread's values
  // or none; 12,709 rows 72 us against 70 without the choice, 78 when such a
  // thread keeps the 16 bytes it loaded)
  const bool turned = c0 < a.rot;
  const int peer = (lane & ~(LPH - 1)) +
                   (c0 >= a.rot ? sub : c0 < (a.rot >> 1) ? sub + far : sub - far);
  for (int j = j0; j < j_end; j += side) {
    float cs[VE], sn[VE];
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      const float2 v = s_cs[j][e][sub];
      cs[e] = v.x;
      sn[e] = v.y;
    }
    // where head h's result goes: + h DH (queries), + h page rows (keys, values)
    const int page = s_page[j];
    const size_t at0 = cache_row(a.c, max(page, 0), 0, s_row[j]);
    T* const dq = (T*)a.q_out + (t0 + j) * a.os + sub * VE;
    T* const dk = (T*)a.c.k + (at0 - ((size_t)k_at << a.c.ps_log2)) * DH + sub * VE;
    T* const dv = (T*)a.c.v + (at0 - ((size_t)v_at << a.c.ps_log2)) * DH + sub * VE;
    for (int hb = h0; hb < heads; hb += STEP * CA_UNROLL) {
      // the next group: further heads of this row, or the next row
      uint4 y[CA_UNROLL];
      int nh = hb + STEP * CA_UNROLL;
      if (nh >= heads) {
        nh = j + side < j_end ? h0 : heads;
        pq += side * a.qs;
        pk += side * a.ks;
        pv += side * a.vs;
      }
#pragma unroll
      for (int u = 0; u < CA_UNROLL; ++u)
        if (nh + u * STEP < heads) y[u] = load(nh + u * STEP);
#pragma unroll
      for (int u = 0; u < CA_UNROLL; ++u) {
        const int h = hb + u * STEP;
        if (h >= heads) break;
        const bool is_q = h < k_at;
        uint4 out = x[u];
        if (h < v_at) {
          float f[VE], r = 1.f;
          Vec16<T>::unpack(x[u], f);
          if (is_q ? a.qg != nullptr : a.kg != nullptr) {
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < VE; ++e) ss = fmaf(f[e], f[e], ss);
#pragma unroll
            for (int z = LPH / 2; z > 0; z >>= 1) ss += __shfl_xor_sync(m, ss, z);
            r = rsqrtf(ss * (1.f / DH) + a.eps);
            float g[VE];
            Vec16<T>::unpack(is_q ? gq : gk, g);
#pragma unroll
            for (int e = 0; e < VE; ++e) f[e] *= g[e];
          }
          float o[VE];
#pragma unroll
          for (int e = 0; e < VE; ++e) o[e] = INTER ? f[e ^ 1] : __shfl_sync(m, f[e], peer);
#pragma unroll
          for (int e = 0; e < VE; ++e) {
            const float y = fmaf(o[e], sn[e], f[e] * cs[e]);
            f[e] = r * (turned ? y : f[e]);
          }
          out = Vec16<T>::pack(f);
        }
        if (is_q) {
          if (page != -2) *(uint4*)(dq + h * DH) = out;
        } else if (page >= 0) {
          *(uint4*)((h < v_at ? dk : dv) + ((size_t)h << a.c.ps_log2) * DH) = out;
        }
      }
#pragma unroll
      for (int u = 0; u < CA_UNROLL; ++u) x[u] = y[u];
    }
  }
}

// ------------------------------------------------------------------ evict
// One cluster of C CTAs per (sequence, head); CTA z owns the contiguous slice
// [z S, (z + 1) S) of the L rows and keeps its rows' 32-bit sort keys in
// shared memory, so positions and weights are read once.  Selection: three
// radix passes (11, 11, 10 bits) of cluster-wide histograms give the budget-th
// largest key and how many of its ties stay; ballots and prefix sums give every
// hole and every mover its rank; entry i of both lists lives in
// CTA i mod C's shared memory.  Movers come from rows >= budget, holes are
// rows < budget, so no move can overwrite another's source and they all run
// at once.
//
// Bound: the latency of the passes for few rows (each a few shared-memory
// round trips and a barrier: 256 pairs of 1,041 rows 15 us); 8 bytes per row
// plus the moved rows beyond that (64 pairs of up to 16,384 rows cut to 2,048:
// 47 us, of which 22 move the rows at 4.7 TB/s).
constexpr int EV_THREADS = 512;
constexpr int EV_SLICE = 32768;    // most rows of one CTA (64 steps of a warp: one flag word)
constexpr int EV_MAX_CLUSTER = 8;
constexpr int EV_BINS = 2048;

struct EvictArgs {
  CacheView c;
  const int *kv_len, *next_pos;
  int* new_len;
  int max_kv, budget, sinks, recent, row_bytes;
  int slice_cap;                   // rows the shared-memory key array holds
};

__host__ __device__ constexpr int evict_smem(int slice_cap) {
  return slice_cap * 4 + 2 * EV_BINS * 4 + 64 * 4 + 64 * 4;
}

// 32-bit key, larger = kept first.  A non-negative float's bits order as its
// value; 0 is left for rows that do not exist.
__device__ __forceinline__ uint32_t evict_key(float w) {
  return w > 0.f ? __float_as_uint(w) + 1u : 1u;
}

// Exclusive prefix of v over the EV_THREADS threads, and the block's total.
__device__ __forceinline__ unsigned block_prefix(unsigned v, unsigned* sh, unsigned& total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  unsigned x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) sh[w] = x;
  __syncthreads();
  unsigned base = 0, sum = 0;
#pragma unroll
  for (int i = 0; i < EV_THREADS / 32; ++i) {
    const unsigned y = sh[i];
    if (i < w) base += y;
    sum += y;
  }
  total = sum;
  return base + x - v;
}
// The same over the warps, for a value that is the same in all lanes.
__device__ __forceinline__ unsigned warp_prefix(unsigned v, unsigned* sh, unsigned& total) {
  const int w = threadIdx.x >> 5;
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[w] = v;
  __syncthreads();
  unsigned base = 0, sum = 0;
#pragma unroll
  for (int i = 0; i < EV_THREADS / 32; ++i) {
    const unsigned y = sh[i];
    if (i < w) base += y;
    sum += y;
  }
  total = sum;
  return base;
}
__device__ __forceinline__ unsigned dsmem_ldu(uint32_t addr) {
  unsigned v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint4 dsmem_ld4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void dsmem_stu(uint32_t addr, unsigned v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__global__ void __launch_bounds__(EV_THREADS) k_cache_evict(const EvictArgs a) {
  extern __shared__ __align__(16) uint32_t sm[];
  uint32_t* key = sm;                               // [slice_cap]; later the two lists
  uint32_t* hist = sm + a.slice_cap;                // two buffers of EV_BINS
  uint32_t* scan = hist + 2 * EV_BINS;              // [64] block scans
  uint32_t* xch = scan + 64;                        // [64] values other CTAs read
  pdl_wait();
  pdl_trigger();
  const int C = (int)cluster_size(), z = (int)cluster_rank();
  const int pair = blockIdx.x / C, b = pair / a.c.n_kv, g = pair % a.c.n_kv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto sync_cluster = [&]() {
    if (C > 1) cluster_sync_all();
    else __syncthreads();
  };
  const int cap = min(a.max_kv, a.c.table_stride << a.c.ps_log2);
  const int L = min(max(__ldg(a.kv_len + b), 0), cap);
  if (g == 0 && z == 0 && tid == 0) a.new_len[b] = min(L, a.budget);
  if (L <= a.budget) return;                        // the whole cluster leaves
  const int S = (L + C - 1) / C, r0 = z * S, n = max(0, min(S, L - r0));
  // rows at or past this position are protected (64 bits: no overflow)
  const long long fresh = (long long)__ldg(a.next_pos + b) - a.recent;
  for (int i = tid; i < 2 * EV_BINS; i += EV_THREADS) hist[i] = 0u;
  __syncthreads();
  // four rows a thread at a time: their pages, then their positions and weights
  constexpr int LD = 4;
  for (int i0 = tid; i0 < n; i0 += EV_THREADS * LD) {
    int page[LD], pos[LD];
    float w[LD];
#pragma unroll
    for (int k = 0; k < LD; ++k) {
      const int i = i0 + k * EV_THREADS;
      page[k] = i < n ? cache_page(a.c, b, r0 + i) : -1;
    }
#pragma unroll
    for (int k = 0; k < LD; ++k) {
      pos[k] = 0;
      w[k] = 0.f;
      if (page[k] >= 0) {
        const size_t at = cache_row(a.c, page[k], g, r0 + i0 + k * EV_THREADS);
        pos[k] = a.c.pos[at];
        w[k] = a.c.weight[at];
      }
    }
#pragma unroll
    for (int k = 0; k < LD; ++k) {
      const int i = i0 + k * EV_THREADS;
      if (i >= n) continue;
      uint32_t kk = 0u;
      if (page[k] >= 0) kk = (pos[k] < a.sinks || pos[k] >= fresh) ? 0xffffffffu : evict_key(w[k]);
      key[i] = kk;
      atomicAdd(hist + (kk >> 21), 1u);
    }
  }
  // the budget-th largest key: bits 31..21, 20..10, 9..0
  uint32_t prefix = 0u, want = (uint32_t)a.budget;  // want: keys still to take below `prefix`'s range
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    uint32_t* h = hist + (pass & 1) * EV_BINS;
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const int bins = pass == 2 ? 1024 : EV_BINS;
    if (pass > 0) {
      const int up = pass == 1 ? 21 : 10;
      for (int i = tid; i < n; i += EV_THREADS)
        if ((key[i] >> up) == (prefix >> up)) atomicAdd(h + ((key[i] >> shift) & (bins - 1)), 1u);
    }
    sync_cluster();
    // thread t holds bins 4t..4t+3 counted from the top, one 16-byte load from
    // every CTA's histogram, all in flight at once
    unsigned cnt[4] = {0, 0, 0, 0}, sum = 0;
    if (tid * 4 < bins) {
      const uint32_t at = (uint32_t)__cvta_generic_to_shared(h + bins - 4 - tid * 4);
      uint4 v[EV_MAX_CLUSTER];
#pragma unroll
      for (int p = 0; p < EV_MAX_CLUSTER; ++p)
        if (p < C) v[p] = dsmem_ld4(dsmem_addr(at, p));
#pragma unroll
      for (int p = 0; p < EV_MAX_CLUSTER; ++p)
        if (p < C) {
          cnt[0] += v[p].w;
          cnt[1] += v[p].z;
          cnt[2] += v[p].y;
          cnt[3] += v[p].x;
        }
      sum = (cnt[0] + cnt[1]) + (cnt[2] + cnt[3]);
    }
    unsigned total;
    unsigned above = block_prefix(sum, scan, total);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (above < want && want <= above + cnt[e]) {
        scan[32] = (uint32_t)(bins - 1 - (tid * 4 + e));
        scan[33] = want - above;
      }
      above += cnt[e];
    }
    __syncthreads();
    prefix |= scan[32] << shift;
    want = scan[33];
    // the other buffer is empty for the next pass; this one is cleared for the
    // pass after it once every CTA has read it
    if (pass == 0) {
      sync_cluster();
      for (int i = tid; i < EV_BINS; i += EV_THREADS) h[i] = 0u;
    }
  }
  // `want` rows whose key is the threshold itself stay, lowest rows first.
  // Warp w owns the run [w q 32, (w + 1) q 32) of the slice (q <= 64), 32 rows a
  // step: ballots rank the rows within a step, a running count over the steps,
  // block prefixes over the warps and the cluster.
  const int q = (n + EV_THREADS - 1) / EV_THREADS, i0 = warp * q * 32;
  const unsigned lt = (1u << lane) - 1u;
  unsigned ties = 0;
  for (int k = 0; k < q; ++k) {
    const int i = i0 + k * 32 + lane;
    ties += __popc(__ballot_sync(0xffffffffu, i < n && key[i] == prefix));
  }
  unsigned cta_ties;
  unsigned tie = warp_prefix(ties, scan, cta_ties);
  if (tid == 0) xch[0] = cta_ties;
  sync_cluster();
  for (int p = 0; p < z; ++p) tie += dsmem_ldu(dsmem_addr((uint32_t)__cvta_generic_to_shared(xch), p));
  unsigned long long keep = 0ull;   // bit k: the row of step k stays
  unsigned holes = 0, movers = 0;
  for (int k = 0; k < q; ++k) {
    const int i = i0 + k * 32 + lane;
    const uint32_t kk = i < n ? key[i] : 0u;
    const unsigned at = __ballot_sync(0xffffffffu, i < n && kk == prefix);
    const bool in = i < n && (kk > prefix || (kk == prefix && tie + __popc(at & lt) < want));
    tie += __popc(at);
    if (in) keep |= 1ull << k;
    const bool low = r0 + i < a.budget;
    holes += __popc(__ballot_sync(0xffffffffu, i < n && low && !in));
    movers += __popc(__ballot_sync(0xffffffffu, i < n && !low && in));
  }
  unsigned cta_holes, cta_movers;
  unsigned hole = warp_prefix(holes, scan, cta_holes);
  unsigned mover = warp_prefix(movers, scan + EV_THREADS / 32, cta_movers);
  if (tid == 0) {
    xch[1] = cta_holes;
    xch[2] = cta_movers;
  }
  sync_cluster();   // also: no CTA reads its keys after this point
  unsigned moves = 0;
  for (int p = 0; p < C; ++p) {
    const uint32_t at = dsmem_addr((uint32_t)__cvta_generic_to_shared(xch + 1), p);
    const unsigned ph = dsmem_ldu(at), pm = dsmem_ldu(at + 4);
    if (p < z) {
      hole += ph;
      mover += pm;
    }
    moves += pm;
  }
  // entry e of the lists: CTA e mod C, slot e / C.  At most min(budget,
  // L - budget) <= L / 2 entries, so two lists fit the key array.  The entries
  // are row indices of the whole cache (31 bits; all ones: the row does not
  // exist), looked up here, where every thread has its own.
  const uint32_t lists = (uint32_t)__cvta_generic_to_shared(key);
  const uint32_t half = (uint32_t)(a.slice_cap / 2) * 4u;
  for (int k = 0; k < q; ++k) {
    const int i = i0 + k * 32 + lane;
    const bool in = (keep >> k) & 1ull, low = r0 + i < a.budget;
    const bool is_hole = i < n && low && !in, is_mover = i < n && !low && in;
    const unsigned hm = __ballot_sync(0xffffffffu, is_hole), mm = __ballot_sync(0xffffffffu, is_mover);
    if (is_hole || is_mover) {
      const int page = cache_page(a.c, b, r0 + i);
      const unsigned at = page < 0 ? 0xffffffffu : (unsigned)cache_row(a.c, page, g, r0 + i);
      const unsigned e = is_hole ? hole + __popc(hm & lt) : mover + __popc(mm & lt);
      dsmem_stu(dsmem_addr(is_hole ? lists : lists + half, e % C) + (e / C) * 4u, at);
    }
    hole += __popc(hm);
    mover += __popc(mm);
  }
  sync_cluster();
  const int mine = ((int)moves - z + C - 1) / C;
  const uint32_t* to_row = key;
  const uint32_t* from_row = key + a.slice_cap / 2;
  const int per = a.row_bytes >> 4;                 // 16-byte pieces of a row: 4 .. 32
  // a row's keys and values are 2 per pieces of 16 bytes; a warp moves UN rows
  // at a time, all loads before the first store
  constexpr int W = EV_THREADS / 32, UN = 4;
  for (int e0 = warp; e0 < mine; e0 += W * UN) {
    size_t d[UN], s[UN];
    bool ok[UN];
#pragma unroll
    for (int k = 0; k < UN; ++k) {
      const int e = e0 + k * W;
      const unsigned dr = e < mine ? to_row[e] : ~0u, sr = e < mine ? from_row[e] : ~0u;
      ok[k] = dr != ~0u && sr != ~0u;
      d[k] = dr;
      s[k] = sr;
    }
    for (int i = lane; i < 2 * per; i += 32) {
      const int o = i >= per ? i - per : i;
      char* base = (char*)(i >= per ? a.c.v : a.c.k);
      uint4 v[UN];
#pragma unroll
      for (int k = 0; k < UN; ++k)
        if (ok[k]) v[k] = *((const uint4*)(base + s[k] * a.row_bytes) + o);
#pragma unroll
      for (int k = 0; k < UN; ++k)
        if (ok[k]) *((uint4*)(base + d[k] * a.row_bytes) + o) = v[k];
    }
#pragma unroll
    for (int k = 0; k < UN; ++k) {
      if (ok[k] && lane == 2 * k) a.c.pos[d[k]] = a.c.pos[s[k]];
      if (ok[k] && lane == 2 * k + 1) a.c.weight[d[k]] = a.c.weight[s[k]];
    }
  }
}

}  // namespace fm
