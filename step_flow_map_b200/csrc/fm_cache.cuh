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
// Bound: HBM (every value read once and written once) for many rows, launch
// and one chain of dependent loads for few.  A thread holds 16 bytes of one
// head, head_dim * size / 16 neighbouring lanes hold the head, so the norm is
// a few shuffles and a half-split pair one shuffle; a CTA takes whole rows,
// whose angles (one fp64 product and reduction per pair, shared by all heads)
// wait in shared memory while the heads' loads are in flight.
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

template <typename T, int DH>
__global__ void __launch_bounds__(CA_THREADS) k_cache_append(const AppendArgs a) {
  constexpr int VE = Vec16<T>::N, LPH = DH / VE;   // values per thread, lanes per head
  __shared__ float2 s_cs[CA_MAX_TOK][DH / 2];      // (cos, sin) per row and pair
  __shared__ int s_page[CA_MAX_TOK], s_row[CA_MAX_TOK], s_pos[CA_MAX_TOK];
  const int t0 = blockIdx.x * a.tok, nt = min(a.tok, a.T - t0);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int heads = a.n_heads + 2 * a.c.n_kv;
  const int sub = tid & (LPH - 1), tasks = nt * heads;
  constexpr int STEP = CA_THREADS / LPH;
  pdl_wait();
  pdl_trigger();

  auto src = [&](int task) -> const T* {
    const int t = t0 + task / heads;
    int h = task % heads;
    if (h < a.n_heads) return (const T*)a.q + t * a.qs + h * DH;
    h -= a.n_heads;
    if (h < a.c.n_kv) return (const T*)a.k + t * a.ks + h * DH;
    return (const T*)a.v + t * a.vs + (h - a.c.n_kv) * DH;
  };
  // the first heads' loads go out before anything else
  uint4 x[CA_UNROLL];
#pragma unroll
  for (int u = 0; u < CA_UNROLL; ++u) {
    const int task = tid / LPH + u * STEP;
    if (task < tasks) x[u] = *((const uint4*)src(task) + sub);
  }
  // a warp per row: its sequence (all of cu_rows and kv_len in one round of
  // loads), page and position
  for (int j = warp; j < nt; j += CA_THREADS / 32) {
    const int t = t0 + j;
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
    if (lane == 0) {
      const int p = a.q_pos ? __ldg(a.q_pos + t) : row;
      s_pos[j] = p;
      s_row[j] = row;
      s_page[j] = hit ? cache_page(a.c, seq, row) : -2;   // -2: a row of no sequence
    }
    const int p = __shfl_sync(0xffffffffu, lane == 0 ? s_pos[j] : 0, 0);
    // turns = position * f / (2 pi): its whole part drops out in fp64, so the
    // fraction is good to 1e-10 of a turn at any 32-bit position
    for (int i = lane; i < a.rot / 2; i += 32) {
      const double turns = (double)p * a.inv_freq[i] * 0.15915494309189533577;
      float c, s;
      sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
      s_cs[j][i] = make_float2(c, s);
    }
  }
  __syncthreads();

  // shuffles stay among a head's lanes, which always branch together
  const unsigned m = LPH == 32 ? 0xffffffffu : ((1u << (LPH & 31)) - 1u) << (lane & ~(LPH - 1));
  for (int task0 = 0; task0 < tasks; task0 += STEP * CA_UNROLL) {
    if (task0 > 0) {
#pragma unroll
      for (int u = 0; u < CA_UNROLL; ++u) {
        const int task = task0 + tid / LPH + u * STEP;
        if (task < tasks) x[u] = *((const uint4*)src(task) + sub);
      }
    }
#pragma unroll
    for (int u = 0; u < CA_UNROLL; ++u) {
      const int task = task0 + tid / LPH + u * STEP;
      if (task >= tasks) continue;
      const int j = task / heads, t = t0 + j;
      int h = task % heads;
      const int page = s_page[j];
      if (h >= a.n_heads + a.c.n_kv) {
        h -= a.n_heads + a.c.n_kv;
        if (page >= 0)
          *((uint4*)((T*)a.c.v + cache_row(a.c, page, h, s_row[j]) * DH) + sub) = x[u];
        continue;
      }
      const bool is_q = h < a.n_heads;
      if (!is_q) h -= a.n_heads;
      float f[VE];
      Vec16<T>::unpack(x[u], f);
      const T* gain = (const T*)(is_q ? a.qg : a.kg);
      if (gain) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < VE; ++e) ss = fmaf(f[e], f[e], ss);
#pragma unroll
        for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(m, ss, o);
        const float r = rsqrtf(ss * (1.f / DH) + a.eps);
        float gv[VE];
        Vec16<T>::unpack(__ldg((const uint4*)gain + sub), gv);
#pragma unroll
        for (int e = 0; e < VE; ++e) f[e] *= r * gv[e];
      }
      const int c0 = sub * VE;   // this thread's first value of the head
      if (a.interleaved) {
        if (c0 < a.rot) {
#pragma unroll
          for (int e = 0; e < VE; e += 2) {
            const float2 cs = s_cs[j][(c0 + e) >> 1];
            const float lo = f[e], hi = f[e + 1];
            f[e] = lo * cs.x - hi * cs.y;
            f[e + 1] = hi * cs.x + lo * cs.y;
          }
        }
      } else if (a.rot > 0) {
        // the partner of values c0.. lies rot/2 values on (or back), a whole
        // number of lanes away (rot is a multiple of 16)
        const int half = a.rot >> 1, d = half / VE;
        const bool low = c0 < half, in = c0 < a.rot;
        const int peer = (lane & ~(LPH - 1)) + (!in ? sub : low ? sub + d : sub - d);
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          const float o = __shfl_sync(m, f[e], peer);
          if (in) {
            const float2 cs = s_cs[j][(low ? c0 : c0 - half) + e];
            f[e] = low ? f[e] * cs.x - o * cs.y : f[e] * cs.x + o * cs.y;
          }
        }
      }
      if (is_q) {
        if (page != -2) *((uint4*)((T*)a.q_out + t * a.os + h * DH) + sub) = Vec16<T>::pack(f);
      } else if (page >= 0) {
        const size_t at = cache_row(a.c, page, h, s_row[j]);
        *((uint4*)((T*)a.c.k + at * DH) + sub) = Vec16<T>::pack(f);
        if (sub == 0) {
          if (a.c.pos) a.c.pos[at] = s_pos[j];
          if (a.c.weight) a.c.weight[at] = 0.f;
        }
      }
    }
  }
}

// ------------------------------------------------------------------ evict
// One cluster of C CTAs per (sequence, head); CTA z owns the contiguous slice
// [z S, (z + 1) S) of the L rows and keeps its rows' 32-bit sort keys in
// shared memory, so positions and weights are read once.  Selection: three
// radix passes (11, 11, 10 bits) of cluster-wide histograms give the budget-th
// largest key and how many of its ties stay; one ordered scan per thread run
// gives every hole and every mover its rank; entry i of both lists lives in
// CTA i mod C's shared memory.  Movers come from rows >= budget, holes are
// rows < budget, so no move can overwrite another's source and they all run
// at once.
//
// Bound: the latency of the passes for few rows (each a few shared-memory
// round trips and a cluster barrier); 8 bytes per row plus the moved rows
// beyond that.
constexpr int EV_THREADS = 512;
constexpr int EV_SLICE = 32768;    // most rows of one CTA (64 per thread: one flag word)
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
__device__ __forceinline__ unsigned dsmem_ldu(uint32_t addr) {
  unsigned v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void dsmem_stu(uint32_t addr, unsigned v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__global__ void __launch_bounds__(EV_THREADS) k_cache_evict(const EvictArgs a) {
  extern __shared__ uint32_t sm[];
  uint32_t* key = sm;                               // [slice_cap]; later the two lists
  uint32_t* hist = sm + a.slice_cap;                // two buffers of EV_BINS
  uint32_t* scan = hist + 2 * EV_BINS;              // [64] block scans
  uint32_t* xch = scan + 64;                        // [64] values other CTAs read
  pdl_wait();
  pdl_trigger();
  const int C = (int)cluster_size(), z = (int)cluster_rank();
  const int pair = blockIdx.x / C, b = pair / a.c.n_kv, g = pair % a.c.n_kv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cap = min(a.max_kv, a.c.table_stride << a.c.ps_log2);
  const int L = min(max(__ldg(a.kv_len + b), 0), cap);
  if (g == 0 && z == 0 && tid == 0) a.new_len[b] = min(L, a.budget);
  if (L <= a.budget) return;                        // the whole cluster leaves
  const int S = (L + C - 1) / C, r0 = z * S, n = max(0, min(S, L - r0));
  // rows at or past this position are protected (64 bits: no overflow)
  const long long fresh = (long long)__ldg(a.next_pos + b) - a.recent;
  for (int i = tid; i < 2 * EV_BINS; i += EV_THREADS) hist[i] = 0u;
  __syncthreads();
  for (int i = tid; i < n; i += EV_THREADS) {
    const int r = r0 + i, page = cache_page(a.c, b, r);
    uint32_t k = 0u;
    if (page >= 0) {
      const size_t at = cache_row(a.c, page, g, r);
      const int p = a.c.pos[at];
      k = (p < a.sinks || p >= fresh) ? 0xffffffffu : evict_key(a.c.weight[at]);
    }
    key[i] = k;
    atomicAdd(hist + (k >> 21), 1u);
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
    cluster_sync_all();
    // thread t holds bins 4t..4t+3 counted from the top
    unsigned cnt[4], sum = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int bin = bins - 1 - (tid * 4 + e);
      cnt[e] = 0;
      if (bin >= 0)
        for (int q = 0; q < C; ++q)
          cnt[e] += dsmem_ldu(dsmem_addr((uint32_t)__cvta_generic_to_shared(h + bin), q));
      sum += cnt[e];
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
      cluster_sync_all();
      for (int i = tid; i < EV_BINS; i += EV_THREADS) h[i] = 0u;
    }
  }
  // `want` rows whose key is the threshold itself stay, lowest rows first.
  // Thread t owns the run [t q, (t + 1) q) of the slice (q <= 64).
  const int q = (n + EV_THREADS - 1) / EV_THREADS;
  const int i0 = min(tid * q, n), i1 = min(i0 + q, n);
  unsigned ties = 0;
  for (int i = i0; i < i1; ++i) ties += key[i] == prefix;
  unsigned cta_ties;
  unsigned tie = block_prefix(ties, scan, cta_ties);
  if (tid == 0) xch[0] = cta_ties;
  cluster_sync_all();
  for (int p = 0; p < z; ++p) tie += dsmem_ldu(dsmem_addr((uint32_t)__cvta_generic_to_shared(xch), p));
  unsigned long long keep = 0ull;
  unsigned holes = 0, movers = 0;
  for (int i = i0; i < i1; ++i) {
    const uint32_t k = key[i];
    bool in = k > prefix;
    if (k == prefix) in = tie++ < want;
    if (in) keep |= 1ull << (i - i0);
    if (r0 + i < a.budget) holes += !in;
    else movers += in;
  }
  unsigned cta_holes, cta_movers;
  unsigned hole = block_prefix(holes, scan, cta_holes);
  unsigned mover = block_prefix(movers, scan, cta_movers);
  if (tid == 0) {
    xch[1] = cta_holes;
    xch[2] = cta_movers;
  }
  cluster_sync_all();   // also: no CTA reads its keys after this point
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
  // L - budget) <= L / 2 entries, so two lists fit the key array.
  const uint32_t lists = (uint32_t)__cvta_generic_to_shared(key);
  const uint32_t half = (uint32_t)(a.slice_cap / 2) * 4u;
  for (int i = i0; i < i1; ++i) {
    const bool in = (keep >> (i - i0)) & 1ull;
    if (r0 + i < a.budget) {
      if (!in) {
        dsmem_stu(dsmem_addr(lists, hole % C) + (hole / C) * 4u, (unsigned)(r0 + i));
        ++hole;
      }
    } else if (in) {
      dsmem_stu(dsmem_addr(lists + half, mover % C) + (mover / C) * 4u, (unsigned)(r0 + i));
      ++mover;
    }
  }
  cluster_sync_all();
  const int mine = ((int)moves - z + C - 1) / C;
  const uint32_t* to_row = key;
  const uint32_t* from_row = key + a.slice_cap / 2;
  const int per = a.row_bytes >> 4;                 // 16-byte pieces of a row: 4 .. 32
  for (int e = warp; e < mine; e += EV_THREADS / 32) {
    const int dr = (int)to_row[e], sr = (int)from_row[e];
    const int dp = cache_page(a.c, b, dr), sp = cache_page(a.c, b, sr);
    if (dp < 0 || sp < 0) continue;
    const size_t d = cache_row(a.c, dp, g, dr), s = cache_row(a.c, sp, g, sr);
    for (int i = lane; i < 2 * per; i += 32) {
      const bool val = i >= per;
      const int o = val ? i - per : i;
      const char* base = (const char*)(val ? a.c.v : a.c.k);
      *((uint4*)(base + d * a.row_bytes) + o) = *((const uint4*)(base + s * a.row_bytes) + o);
    }
    if (lane == 0) a.c.pos[d] = a.c.pos[s];
    if (lane == 1) a.c.weight[d] = a.c.weight[s];
  }
}

}  // namespace fm
