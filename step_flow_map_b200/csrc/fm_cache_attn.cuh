// Attention of new rows over the target's paged key/value cache.
//
//   s = scale q.k,  p = softmax of s over the rows a query sees,  o = sum p v,
//   lse = log sum e^s,  weight_r += sum of p over queries and query heads
//
// The query heads of one key/value head share its rows, so they are packed:
// packed row x = i G + j is query i, head g G + j (G query heads per
// key/value head).  A tile is QT packed rows of one (sequence, key/value
// head); its unit of work is one block of KB cache rows.  Lengths live on the
// device (a captured launch serves them as they change), so the split is
// decided there: all units of all tiles, in order, are dealt to the CTAs in
// equal runs, whatever the lengths.  A CTA keeps (max, sum, O) over the
// blocks of a tile that fall in its run and writes the result when it had all
// of them, else a partial; at most two partials per CTA (its first and its
// last tile), so their number does not grow with the lengths.  A second
// kernel joins the partials of split tiles in CTA order.
#pragma once
#include "fm_cache.cuh"
#include "fm_ptx.cuh"

namespace fm {

struct CacheAttnArgs {
  CacheView c;
  int T, B, n_heads, G, max_rows, max_kv;
  int rt, tile_rows;               // packed rows of a (half) tile that are used; of a tile
  int ov;                          // units a tile's start and end cost beyond its blocks
  int max_tiles;                   // entries of the plan
  const void* q;
  int64_t qs, os;
  const int *cu, *kv_len, *q_pos;
  float scale_log2;                // scale * log2(e)
  int window, sinks;
  void* out;
  float* lse;                      // or null
  // workspace
  int* plan_n;                     // number of tiles
  int* plan_first;                 // [tiles + 1]: first unit of each tile, heads apart; few packed
                                   //   rows: [B + 1], of each sequence
  int4* plan_tile;                 // [tiles][2]: (b, first packed row, first new row, packed rows
                                   //   of the sequence), (s_end, lo, hi, position of new row 0)
  int4* plan_join;                 // [grid][2], see JoinItem
  float* part;                     // [grid][2][QT][DH]
  float2* part_ml;                 // [grid][2][QT]: (max, sum), log2 units
  float* scores;                   // see score_at
  int score_units;                 // units it has room for
};

// Rows a tile can see: [0, s_end) and [lo, hi), s_end <= lo.
struct SeenRows {
  int s_end, lo, hi;
};
__device__ __forceinline__ SeenRows seen_rows(const CacheAttnArgs& a, const NewRows& s, int i0,
                                              int i1) {
  SeenRows r;
  const int len = min(s.L, min(a.max_kv, a.c.table_stride << a.c.ps_log2));
  r.s_end = 0;
  r.lo = 0;
  r.hi = len;
  if (a.c.pos) return r;           // any row may hold any position
  const long long p0 = (long long)s.L - s.n + i0, p1 = (long long)s.L - s.n + i1;
  r.hi = (int)max(0ll, min((long long)len, p1 + 1));
  if (a.window > 0) {
    r.lo = (int)min((long long)r.hi, max(0ll, p0 - a.window + 1));
    r.s_end = min(a.sinks, r.lo);
  }
  return r;
}
// Its blocks of KB rows: nb in all, the j-th at row block_row(j).
template <int KB>
struct SeenBlocks {
  int ns, b0, nb;                  // blocks of [0, s_end), first block of [lo, hi), all
  __device__ __forceinline__ explicit SeenBlocks(const SeenRows& r) {
    b0 = r.lo / KB;
    ns = min((r.s_end + KB - 1) / KB, b0);
    // a tile that sees nothing still has one (masked) block, which writes its zeros
    nb = max(1, ns + max(0, (r.hi + KB - 1) / KB - b0));
  }
  __device__ __forceinline__ int row(int j) const { return (j < ns ? j : j - ns + b0) * KB; }
  __device__ __forceinline__ int at(int r) const {   // the block of a row that is seen
    const int j = r / KB;
    return j < ns ? j : j - b0 + ns;
  }
};
__device__ __forceinline__ bool row_seen(const SeenRows& s, int r) {
  return r < s.s_end || (r >= s.lo && r < s.hi);
}
// The mask of one (query position, row position) pair.  The difference is
// taken unsigned once the order is known, so no pair of positions overflows.
__device__ __forceinline__ bool sees(int pq, int pk, int window, int sinks) {
  return pk <= pq && (window == 0 || (unsigned)pq - (unsigned)pk < (unsigned)window || pk < sinks);
}

constexpr int CD_KB = 64;          // cache rows of a unit of few packed rows
// Masked scores (log2 units) of the 16 cache rows `sub` of unit u (CD_KB rows of a
// sequence and head, numbered over the call) against packed row x of at most
// a.max_rows G <= 16, the 16 rows' side by side.
__device__ __forceinline__ size_t score_at(const CacheAttnArgs& a, int u, int sub, int x) {
  return (((size_t)u * 4 + sub) * (a.max_rows * a.G) + x) * 16;
}

// ------------------------------------------------------------------ plan
// One CTA lists the tiles of every sequence and prefix-sums their blocks.
// Sequences that overlap, against the rules, can ask for more tiles than the
// plan holds: the sums stop there.
constexpr int CP_THREADS = 1024;
template <int KB>
__global__ void __launch_bounds__(CP_THREADS) k_cache_plan(const CacheAttnArgs a) {
  __shared__ int s_tiles[257];
  __shared__ int s_warp[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int QT = a.tile_rows;
  pdl_wait();
  pdl_trigger();
  if (tid < 256) {
    int n = 0;
    if (tid < a.B) n = min(new_rows(a.cu, a.kv_len, tid, a.T).n, a.max_rows);
    s_tiles[tid + 1] = min((n * a.G + QT - 1) / QT, a.max_tiles);
  }
  if (tid == 0) s_tiles[0] = 0;
  __syncthreads();
  if (warp == 0) {                 // prefix sum, eight sequences a lane
    int v[8], sum = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) sum = min(sum + (v[k] = s_tiles[lane * 8 + k + 1]), a.max_tiles);
    int at = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, at, o);
      if (lane >= o) at = min(at + y, a.max_tiles);
    }
    at = __shfl_up_sync(0xffffffffu, at, 1);
    if (lane == 0) at = 0;
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 8; ++k) s_tiles[lane * 8 + k + 1] = at = min(at + v[k], a.max_tiles);
  }
  __syncthreads();
  const int E = s_tiles[256];
  int base = 0;
  for (int e0 = 0; e0 < E; e0 += CP_THREADS) {
    const int e = e0 + tid;
    int nb = 0;                      // units: the blocks, and the tile's overhead
    if (e < E) {
      int b = 0;                   // largest b with s_tiles[b] <= e
      for (int step = 128; step > 0; step >>= 1)
        if (s_tiles[b + step] <= e) b += step;
      const int tile = e - s_tiles[b];
      const NewRows s = new_rows(a.cu, a.kv_len, b, a.T);
      const int rows = min(s.n, a.max_rows) * a.G;
      const SeenRows r = seen_rows(a, s, tile * QT / a.G, (min(rows, (tile + 1) * QT) - 1) / a.G);
      nb = SeenBlocks<KB>(r).nb + a.ov;
      a.plan_tile[2 * e] = make_int4(b, tile * QT, s.first, rows);
      a.plan_tile[2 * e + 1] = make_int4(r.s_end, r.lo, r.hi, s.L - s.n);
    }
    int x = nb;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    int add = base, sum = 0;
    for (int i = 0; i < 32; ++i) {
      if (i < warp) add += s_warp[i];
      sum += s_warp[i];
    }
    if (e < E) a.plan_first[e] = add + x - nb;
    base += sum;
  }
  if (tid == 0) {
    a.plan_first[E] = base;
    a.plan_n[0] = E;
  }
}

// The run of units of CTA c of `grid`, and the tile a unit falls in.  Units of
// a tile: for head 0 `ov` units that stand for its start and end and then its
// blocks, then the same for head 1, and so on.
// There are fewer than 2^31 units (checked by the host from the bounds it was
// given).
struct WorkRun {
  int N, g, q, rem;                // units; CTAs that have work; N = g q + rem
  __device__ __forceinline__ WorkRun(int N_, int grid) : N(N_), g(max(1, min(grid, N_))) {
    q = N / g;
    rem = N - q * g;
  }
  __device__ __forceinline__ int start(int c) const { return q * c + min(c, rem); }
  __device__ __forceinline__ int cta_of(int u) const {
    const int t = rem * (q + 1);
    return u < t ? u / (q + 1) : rem + (u - t) / q;
  }
};
// Largest e with plan_first[e] n_kv <= u; every lane of the warp takes part,
// 32 probes a round.
__device__ __forceinline__ int find_tile(const CacheAttnArgs& a, int E, int u) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = E;               // the answer lies in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int at = lo + lane * step;
    const bool ok = lane * step < n && a.plan_first[at] * a.c.n_kv <= u;
    const int k = 31 - __clz((int)__ballot_sync(0xffffffffu, ok));   // lane 0 always holds
    n = min(step, n - k * step);
    lo += k * step;
  }
  return lo;
}
// What the second kernel joins at the start of run c: the tile that run c0 =
// c - 1 began (its partial in slot slot0) and runs .. last continue, when run
// c's start is the first to fall among its blocks; else c0 = -1.  Every CTA
// writes its own entry: {c0, last, slot0, packed rows of the sequence}, {first
// new row, head, first packed row, -}.
__device__ __forceinline__ void put_join(const CacheAttnArgs& a, const WorkRun& w, int c, int first,
                                         int units, int row0, int g, int x0, int all) {
  const int u = w.start(c), real = first + a.ov;
  int c0 = -1;
  if (c > 0 && c < w.g && u > real && w.start(c - 1) <= real) c0 = c - 1;
  a.plan_join[2 * c] = make_int4(c0, c0 < 0 ? 0 : w.cta_of(first + units - 1),
                                 c0 < 0 || w.start(c0) >= first ? 0 : 1, all);
  a.plan_join[2 * c + 1] = make_int4(row0, g, x0, 0);
}

// ------------------------------------------------------------------ CUDA-core kernel (fp32)
// More than 16 packed rows in fp32: tiles of 64 packed rows against blocks of
// 64 cache rows, 16 x 16 threads with 4 x 4 scores and 4 x DH / 16 outputs
// each; scores, probabilities and O stay fp32.  The next block's keys and
// values come by cp.async while this one is worked on, one CTA barrier a block.
// Bound: shared memory beside the FMAs (12 wavefronts per 64 FMA instructions of
// a warp; ncu: its data path 68-73 % busy, the FMA pipe 48 %, 0.65 instructions a
// cycle and scheduler).  513 rows over 1,500, 2 x 12 heads of width 64: 163 us with
// plan and join, 24 TFLOP/s, a third of the FMA rate (128 threads and loads between
// the barriers were 1.7 times slower).
constexpr int CS_THREADS = 256;
constexpr int CS_KB = 64;
constexpr int CS_QT = 64;

template <int DH>
struct CsCfg {
  static constexpr int TC = 16, TR = CS_THREADS / TC;
  static constexpr int RPT = CS_QT / TR, KPT = CS_KB / TC, CPT = DH / TC;
  static constexpr int LD = DH + 4, PLD = CS_KB + 4;
  static constexpr int STAGE = CS_KB * (LD + DH + 2);  // keys, values, positions, "exists"
  static constexpr int SMEM = (CS_QT * LD + 2 * STAGE + CS_QT * PLD) * 4;
};

template <int DH>
__global__ void __launch_bounds__(CS_THREADS, DH == 128 ? 1 : 2) k_cache_attn_simt(const CacheAttnArgs a) {
  using C = CsCfg<DH>;
  constexpr int VW = C::CPT < 4 ? C::CPT : 4;      // neighbouring O columns of a thread
  constexpr int CH = DH / 4;                       // 16-byte pieces of a row
  extern __shared__ __align__(16) float smf[];
  float* sq = smf;                                 // [QT][LD]
  float* ring = sq + CS_QT * C::LD;                // two stages: keys [KB][LD], values [KB][DH],
                                                   //   positions [KB], 1 where the row exists [KB]
  float* sp = ring + 2 * C::STAGE;                 // [QT][PLD]
  const int tid = threadIdx.x, tr = tid / C::TC, tc = tid % C::TC;
  pdl_wait();
  pdl_trigger();
  const int E = a.plan_n[0];
  const WorkRun w(a.plan_first[E] * a.c.n_kv, gridDim.x);
  if ((int)blockIdx.x >= w.g || w.N == 0) {
    if (tid == 0) a.plan_join[2 * blockIdx.x] = make_int4(-1, 0, 0, 0);
    return;
  }
  int u = w.start(blockIdx.x);
  const int u1 = w.start(blockIdx.x + 1), u0 = u;
  int e = find_tile(a, E, u);
  while (u < u1) {
    const int t0 = a.plan_first[e], nb = a.plan_first[e + 1] - t0;
    const int g = (u - t0 * a.c.n_kv) / nb, j0 = u - t0 * a.c.n_kv - g * nb;
    const int j1 = min(nb, j0 + (u1 - u));
    const int4 pt = a.plan_tile[2 * e], ps = a.plan_tile[2 * e + 1];
    const int b = pt.x;
    const SeenRows seen = {ps.x, ps.y, ps.z};
    const SeenBlocks<CS_KB> blocks(seen);
    const int x0 = pt.y, row0 = pt.z, rows = min(CS_QT, pt.w - x0);
    if (u == u0 && tid == 0) put_join(a, w, blockIdx.x, u - j0, nb, row0, g, x0, pt.w);
    auto load = [&](int j) {
      const int r0 = blocks.row(j);
      float* st = ring + (j & 1) * C::STAGE;
      int* info = (int*)(st + CS_KB * (C::LD + DH));
      const uint32_t k32 = (uint32_t)__cvta_generic_to_shared(st), v32 = k32 + CS_KB * C::LD * 4;
#pragma unroll
      for (int i = tid; i < CS_KB * CH; i += CS_THREADS) {
        const int r = i / CH, c = i % CH, cr = r0 + r;
        const int page = row_seen(seen, cr) ? cache_page(a.c, b, cr) : -1;
        const size_t at = cache_row(a.c, max(page, 0), g, cr);
        cp_async16_if(k32 + (r * C::LD + c * 4) * 4, (const float*)a.c.k + at * DH + c * 4, page >= 0);
        cp_async16_if(v32 + (r * DH + c * 4) * 4, (const float*)a.c.v + at * DH + c * 4, page >= 0);
        if (c == 0) {
          info[r] = a.c.pos && page >= 0 ? a.c.pos[at] : cr;
          info[CS_KB + r] = page >= 0;
        }
      }
      cp_commit();
    };
    __syncthreads();                               // the tile before is done with the buffers
    load(j0);
    for (int i = tid; i < CS_QT * CH; i += CS_THREADS) {
      const int r = i / CH, c = (i % CH) * 4;
      float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rows) {
        const int x = x0 + r;
        f = *(const float4*)((const float*)a.q + (row0 + x / a.G) * a.qs + (g * a.G + x % a.G) * DH + c);
        f.x *= a.scale_log2; f.y *= a.scale_log2; f.z *= a.scale_log2; f.w *= a.scale_log2;
      }
      *(float4*)(sq + r * C::LD + c) = f;
    }
    int pq[C::RPT];
    float m[C::RPT], l[C::RPT], o[C::RPT][C::CPT];
#pragma unroll
    for (int i = 0; i < C::RPT; ++i) {
      const int r = tr + C::TR * i;
      const int qi = (x0 + (r < rows ? r : 0)) / a.G;
      pq[i] = a.q_pos ? __ldg(a.q_pos + row0 + qi) : ps.w + qi;
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int c = 0; c < C::CPT; ++c) o[i][c] = 0.f;
    }
    // positions of the tile's first and last query
    const int pmin = ps.w + x0 / a.G, pmax = ps.w + (x0 + rows - 1) / a.G;
    for (int j = j0; j < j1; ++j) {
      const int r0 = blocks.row(j);
      cp_wait<0>();
      __syncthreads();
      if (j + 1 < j1) load(j + 1);
      const float* sk = ring + (j & 1) * C::STAGE;
      const float* sv = sk + CS_KB * C::LD;
      const int* s_pos = (const int*)(sv + CS_KB * DH);
      const int* s_ok = s_pos + CS_KB;
      // every row that exists is seen by every query
      const bool open = !a.c.pos && r0 >= seen.lo && r0 + CS_KB <= seen.hi && r0 + CS_KB - 1 <= pmin &&
                        (a.window == 0 || pmax - r0 < a.window);
      float sc[C::RPT][C::KPT];
#pragma unroll
      for (int i = 0; i < C::RPT; ++i)
#pragma unroll
        for (int k = 0; k < C::KPT; ++k) sc[i][k] = 0.f;
#pragma unroll 4
      for (int d = 0; d < DH; d += 4) {
        float4 qv[C::RPT];
#pragma unroll
        for (int i = 0; i < C::RPT; ++i) qv[i] = *(const float4*)(sq + (tr + C::TR * i) * C::LD + d);
#pragma unroll
        for (int k = 0; k < C::KPT; ++k) {
          const float4 kv = *(const float4*)(sk + (tc + C::TC * k) * C::LD + d);
#pragma unroll
          for (int i = 0; i < C::RPT; ++i) {
            sc[i][k] = fmaf(qv[i].x, kv.x, sc[i][k]);
            sc[i][k] = fmaf(qv[i].y, kv.y, sc[i][k]);
            sc[i][k] = fmaf(qv[i].z, kv.z, sc[i][k]);
            sc[i][k] = fmaf(qv[i].w, kv.w, sc[i][k]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < C::RPT; ++i) {
        float mx = m[i];
#pragma unroll
        for (int k = 0; k < C::KPT; ++k) {
          const int kr = tc + C::TC * k;
          if (!s_ok[kr] || !(open || sees(pq[i], s_pos[kr], a.window, a.sinks))) sc[i][k] = -INFINITY;
          mx = fmaxf(mx, sc[i][k]);
        }
#pragma unroll
        for (int d = 1; d < C::TC; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
        const float ref = mx == -INFINITY ? 0.f : mx;
        const float corr = exp2f(m[i] - ref);      // 0 while nothing was seen
        m[i] = mx;
        l[i] *= corr;
#pragma unroll
        for (int c = 0; c < C::CPT; ++c) o[i][c] *= corr;
#pragma unroll
        for (int k = 0; k < C::KPT; ++k) {
          const float p = exp2f(sc[i][k] - ref);
          l[i] += p;
          sp[(tr + C::TR * i) * C::PLD + tc + C::TC * k] = p;
        }
      }
      __syncwarp();                                // a row's probabilities come from its own warp
#pragma unroll 2
      for (int k = 0; k < CS_KB; k += 4) {
        float4 pv[C::RPT];
#pragma unroll
        for (int i = 0; i < C::RPT; ++i) pv[i] = *(const float4*)(sp + (tr + C::TR * i) * C::PLD + k);
#pragma unroll
        for (int y = 0; y < 4; ++y)
#pragma unroll
          for (int c = 0; c < C::CPT; c += VW) {
            float vv[VW];
            const float* src = sv + (k + y) * DH + c * C::TC + tc * VW;
            if constexpr (VW == 4) *(float4*)vv = *(const float4*)src;
            else *(float2*)vv = *(const float2*)src;
#pragma unroll
            for (int i = 0; i < C::RPT; ++i) {
              const float p = y == 0 ? pv[i].x : y == 1 ? pv[i].y : y == 2 ? pv[i].z : pv[i].w;
#pragma unroll
              for (int z = 0; z < VW; ++z) o[i][c + z] = fmaf(p, vv[z], o[i][c + z]);
            }
          }
      }
      __syncwarp();
    }
    const bool whole = j0 == 0 && j1 == nb;
    const int slot = u == u0 ? 0 : 1;
#pragma unroll
    for (int i = 0; i < C::RPT; ++i) {
#pragma unroll
      for (int d = 1; d < C::TC; d <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);
      const int r = tr + C::TR * i;
      if (r >= rows) continue;
      if (whole) {
        const int x = x0 + r, t = row0 + x / a.G, h = g * a.G + x % a.G;
        const float inv = l[i] != 0.f ? 1.f / l[i] : 0.f;
        float* dst = (float*)a.out + t * a.os + h * DH;
#pragma unroll
        for (int c = 0; c < C::CPT; ++c) dst[(c / VW) * VW * C::TC + tc * VW + c % VW] = o[i][c] * inv;
        if (a.lse && tc == 0)
          a.lse[(size_t)t * a.n_heads + h] =
              l[i] != 0.f ? (m[i] + log2f(l[i])) * 0.69314718055994531f : -INFINITY;
      } else {
        const size_t p = ((size_t)blockIdx.x * 2 + slot) * CS_QT + r;
#pragma unroll
        for (int c = 0; c < C::CPT; ++c)
          a.part[p * DH + (c / VW) * VW * C::TC + tc * VW + c % VW] = o[i][c];
        if (tc == 0) a.part_ml[p] = make_float2(m[i], l[i]);
      }
    }
    u += j1 - j0;
    if (u - t0 * a.c.n_kv >= nb * a.c.n_kv) ++e;
  }
}

// ------------------------------------------------------------------ join
// The partials of split tiles, in run order.  blockIdx.x is the entry of
// plan_join (1 .. grid - 1).  Bound: latency, one round of loads for the
// entry, one for the sums, one for the partials.
constexpr int CJ_THREADS = 128;

__device__ __forceinline__ void join_store_lse(const CacheAttnArgs& a, int t, int h, float m, float l) {
  if (a.lse)
    a.lse[(size_t)t * a.n_heads + h] = l != 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

// Partials [row][column] (tiles of at most 64 rows).  Few packed rows: a CTA per
// row, its warps take every fourth run, so that a long cache's many runs are
// read at once.  64-row tiles: a warp per row (a CTA per row took 18 us for 28
// tiles of 51 rows, most of it CTAs that come and go).
template <typename T, int DH, int QT>
__global__ void __launch_bounds__(CJ_THREADS) k_cache_join_rows(const CacheAttnArgs a) {
  constexpr int W = QT == 64 ? 1 : CJ_THREADS / 32;  // warps of a row
  __shared__ float s_l[W], s_o[W][DH];
  const int lane = threadIdx.x & 31, warp = W == 1 ? 0 : threadIdx.x >> 5;
  pdl_wait();
  pdl_trigger();
  const int4 ja = a.plan_join[2 * blockIdx.x + 2], jb = a.plan_join[2 * blockIdx.x + 3];
  const int r = W == 1 ? blockIdx.y * (CJ_THREADS / 32) + (threadIdx.x >> 5) : blockIdx.y;
  const int c0 = ja.x, last = ja.y, x = jb.z + r;
  if (c0 < 0 || r >= QT || x >= ja.w) return;
  auto at = [&](int i) { return ((size_t)i * 2 + (i == c0 ? ja.z : 0)) * QT + r; };
  float m = -INFINITY;
  for (int i = c0 + lane; i <= last; i += 32) m = fmaxf(m, a.part_ml[at(i)].x);
  m = warp_max(m);
  const float ref = m == -INFINITY ? 0.f : m;
  float l = 0.f, o[DH / 32];
#pragma unroll
  for (int k = 0; k < DH / 32; ++k) o[k] = 0.f;
#pragma unroll 8
  for (int i = c0 + warp; i <= last; i += W) {
    const size_t p = at(i);
    const float2 ml = a.part_ml[p];
    const float f = exp2f(ml.x - ref);
    l = fmaf(ml.y, f, l);
#pragma unroll
    for (int k = 0; k < DH / 32; ++k) o[k] = fmaf(a.part[p * DH + lane + 32 * k], f, o[k]);
  }
  const int t = jb.x + x / a.G, h = jb.y * a.G + x % a.G;
  T* const dst = (T*)a.out + t * a.os + h * DH;
  if constexpr (W == 1) {
    const float inv = l != 0.f ? 1.f / l : 0.f;
#pragma unroll
    for (int k = 0; k < DH / 32; ++k) dst[lane + 32 * k] = from_f<T>(o[k] * inv);
    if (lane == 0) join_store_lse(a, t, h, m, l);
  } else {
    if (lane == 0) s_l[warp] = l;
#pragma unroll
    for (int k = 0; k < DH / 32; ++k) s_o[warp][lane + 32 * k] = o[k];
    __syncthreads();
    const int col = threadIdx.x;
    l = (s_l[0] + s_l[1]) + (s_l[2] + s_l[3]);
    const float inv = l != 0.f ? 1.f / l : 0.f;
    if (col < DH) dst[col] = from_f<T>(((s_o[0][col] + s_o[1][col]) + (s_o[2][col] + s_o[3][col])) * inv);
    if (threadIdx.x == 0) join_store_lse(a, t, h, m, l);
  }
}

// Partials [column][row] (the 128-row tiles): a lane per row, a warp per
// DH / 4 columns.  Partial row r is row r % 128 of half tile r / 128.
template <int DH, int QT>
__global__ void __launch_bounds__(CJ_THREADS) k_cache_join_cols(const CacheAttnArgs a) {
  constexpr int COLS = DH / (CJ_THREADS / 32);
  pdl_wait();
  pdl_trigger();
  const int4 ja = a.plan_join[2 * blockIdx.x + 2], jb = a.plan_join[2 * blockIdx.x + 3];
  const int first = ja.x, last = ja.y;
  const int r = blockIdx.y * 32 + (threadIdx.x & 31), c0 = (threadIdx.x >> 5) * COLS;
  const int x = jb.z + (r >> 7) * a.rt + (r & 127);
  if (first < 0 || (r & 127) >= a.rt || x >= ja.w) return;
  float m = -INFINITY, l = 0.f, o[COLS];
  auto slot = [&](int i) { return (size_t)i * 2 + (i == first ? ja.z : 0); };
#pragma unroll 4
  for (int i = first; i <= last; ++i) m = fmaxf(m, a.part_ml[slot(i) * QT + r].x);
  const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
  for (int k = 0; k < COLS; ++k) o[k] = 0.f;
#pragma unroll 2
  for (int i = first; i <= last; ++i) {
    const float2 ml = a.part_ml[slot(i) * QT + r];
    const float f = exp2f(ml.x - ref);
    l = fmaf(ml.y, f, l);
    const float* p = a.part + (slot(i) * DH + c0) * QT + r;
#pragma unroll
    for (int k = 0; k < COLS; ++k) o[k] = fmaf(p[(size_t)k * QT], f, o[k]);
  }
  const float inv = l != 0.f ? 1.f / l : 0.f;
  const int t = jb.x + x / a.G, h = jb.y * a.G + x % a.G;
  bf16* dst = (bf16*)a.out + t * a.os + h * DH + c0;
#pragma unroll
  for (int k = 0; k < COLS; k += 8) {
    float v[8];
#pragma unroll
    for (int z = 0; z < 8; ++z) v[z] = o[k + z] * inv;
    *(uint4*)(dst + k) = Vec16<bf16>::pack(v);
  }
  if (c0 == 0) join_store_lse(a, t, h, m, l);
}

// ------------------------------------------------------------------ weights
// weight_r += sum over queries and heads of e^(s - lse), added up in the order
// of the packed rows (no atomics, so the sum does not depend on scheduling).

constexpr int CW_THREADS = 256;

// One cached row by the whole warp, the key in registers, the scores once more.
template <typename T, int DH>
__device__ __forceinline__ void weigh_row(const CacheAttnArgs& a, const NewRows& s, int n, int g, int r,
                                          size_t at) {
  const int lane = threadIdx.x & 31;
  const int pk = a.c.pos ? a.c.pos[at] : r;
  float kv[DH / 32];
#pragma unroll
  for (int k = 0; k < DH / 32; ++k) kv[k] = to_f(((const T*)a.c.k)[at * DH + lane + 32 * k]);
  float sum = 0.f;
  for (int x = 0; x < n * a.G; ++x) {
    const int t = s.first + x / a.G, h = g * a.G + x % a.G;
    const int pq = a.q_pos ? __ldg(a.q_pos + t) : s.L - s.n + x / a.G;
    const float lse = a.lse[(size_t)t * a.n_heads + h];
    // (lse is -inf where all scores are: such a query gives no weight, as its output is 0)
    if (lse == -INFINITY || !sees(pq, pk, a.window, a.sinks)) continue;
    float d = 0.f;
#pragma unroll
    for (int k = 0; k < DH / 32; ++k)
      d = fmaf(to_f(((const T*)a.q)[t * a.qs + h * DH + lane + 32 * k]), kv[k], d);
    d = warp_sum(d);
    sum += exp2f(d * a.scale_log2 - lse * 1.4426950408889634f);
  }
  if (lane == 0) a.c.weight[at] += sum;
}

// Few packed rows: from the scores the attention kernel left, a thread per
// cache row.  Bound: HBM, 4 bytes per score and 8 per weight -- for four query
// heads per key/value head 24 bytes a row against the 256 that reading the
// keys again would take.  Units that the scores have no room for (lengths past
// the rows that the cache has: pages that do not exist) go row by row; to do
// so for all rows would take 1,195 us where the scores take 216 (64 sequences of
// 4,096 rows, 8 heads, with the attention's 189).
template <typename T, int DH>
__global__ void __launch_bounds__(CW_THREADS) k_cache_weights_scores(const CacheAttnArgs a) {
  __shared__ float s_lse[16];
  const int g = blockIdx.y, b = blockIdx.z, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  const NewRows s = new_rows(a.cu, a.kv_len, b, a.T);
  const int n = min(s.n, a.max_rows), rows = n * a.G;
  if (n == 0) return;
  if (threadIdx.x < rows) {
    const int x = threadIdx.x;
    const float v = a.lse[(size_t)(s.first + x / a.G) * a.n_heads + g * a.G + x % a.G];
    s_lse[x] = v == -INFINITY ? INFINITY : v * 1.4426950408889634f;   // 2^(s - inf) = 0
  }
  __syncthreads();
  const SeenRows seen = seen_rows(a, s, 0, n - 1);
  const SeenBlocks<CD_KB> blocks(seen);
  const int first = a.plan_first[b];
  const int u0 = first * a.c.n_kv + g * (a.plan_first[b + 1] - first);   // this head's first unit
  for (int r0 = blockIdx.x * CW_THREADS + threadIdx.x - lane; r0 < seen.hi; r0 += gridDim.x * CW_THREADS) {
    const int r = r0 + lane, u = u0 + blocks.at(r);
    const int page = r < seen.hi && row_seen(seen, r) ? cache_page(a.c, b, r) : -1;
    const size_t at = cache_row(a.c, max(page, 0), g, r);
    if (page >= 0 && u < a.score_units) {
      float* w = a.c.weight + at;
      const float had = *w;
      const float* p = a.scores + score_at(a, u, (r >> 4) & 3, 0) + (r & 15);
      float sum = 0.f;
#pragma unroll 4
      for (int x = 0; x < rows; ++x) sum += exp2f(p[x * 16] - s_lse[x]);
      *w = had + sum;
    }
    for (unsigned rest = __ballot_sync(0xffffffffu, page >= 0 && u >= a.score_units); rest; rest &= rest - 1) {
      const int i = __ffs((int)rest) - 1;
      weigh_row<T, DH>(a, s, n, g, r0 + i, __shfl_sync(0xffffffffu, at, i));
    }
  }
}

// Many packed rows, fp32: one warp per cache row.
template <typename T, int DH>
__global__ void __launch_bounds__(CW_THREADS) k_cache_weights(const CacheAttnArgs a) {
  const int g = blockIdx.y, b = blockIdx.z;
  pdl_wait();
  pdl_trigger();
  const NewRows s = new_rows(a.cu, a.kv_len, b, a.T);
  const int n = min(s.n, a.max_rows);
  if (n == 0) return;
  const SeenRows seen = seen_rows(a, s, 0, n - 1);
  for (int r = blockIdx.x * (CW_THREADS / 32) + (threadIdx.x >> 5); r < seen.hi;
       r += gridDim.x * (CW_THREADS / 32)) {
    const int page = row_seen(seen, r) ? cache_page(a.c, b, r) : -1;
    if (page >= 0) weigh_row<T, DH>(a, s, n, g, r, cache_row(a.c, page, g, r));
  }
}

}  // namespace fm
