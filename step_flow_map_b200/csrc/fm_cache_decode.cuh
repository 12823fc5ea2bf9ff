// Attention of few new rows over the paged cache (at most 16 packed rows per
// key/value head: one token, or a short block).
//
// Bound: HBM -- every visible key and value is read once and used by at most
// 16 rows, 16 FLOP per byte and below, so the kernel is a stream with an
// online softmax.  bf16: mma.sync m16n8k16, whose M is the 16 packed rows (at
// this ratio the legacy tensor path is far from its limit and needs no TMEM
// round trip per 16 keys).  fp32: FMAs, two lanes per key for the scores and
// DH / 32 columns a lane for the output, four rows at a time, so that few rows
// cost few instructions.  Measured: one token over 131,071 rows of 8 heads of
// width 128 in bf16 98 us with the join (107 when both cursors worked out their
// rows anew for every unit), 64 tokens with weights 171 us (186); 8 tokens over
// 3,000 rows of 4 heads of width 64 in fp32 25 us with the join (108 in tiles of
// the prompt kernel).  A unit is 64 cache rows of one (sequence, head); each of
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
constexpr int CD_STAGES = 3;
constexpr int CD_QT = 16;

// Where every sequence's units begin, and what it sees.
struct DecodeSeqs {
  int first[257];                  // prefix sums of blocks (heads apart)
  int lo[256], hi[256];
  int row0[256], n[256], len[256];
  __device__ __forceinline__ SeenRows seen(const CacheAttnArgs& a, int b) const {
    return {a.window > 0 && !a.c.pos ? min(a.sinks, lo[b]) : 0, lo[b], hi[b]};   // as seen_rows
  }
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

// A unit of the CTA's run, block j of head g of sequence b, and the first of
// this warp's 16 rows in it; stepping on is an addition but where the sequence
// changes.
struct DecodeCursor {
  int b, g, j, nb, row;
  int ns, main;                    // blocks of [0, s_end); this warp's row of the first one past them
  SeenRows v;
  __device__ __forceinline__ void open(const CacheAttnArgs& a, const DecodeSeqs& s) {
    v = s.seen(a, b);
    const SeenBlocks<CD_KB> k(v);
    ns = k.ns;
    main = k.b0 * CD_KB + 16 * (threadIdx.x >> 5);
  }
  __device__ __forceinline__ void seek(const CacheAttnArgs& a, const DecodeSeqs& s, int u) {
    b = decode_find(a, s, u);
    nb = s.first[b + 1] - s.first[b];
    open(a, s);
    const int at = u - s.first[b] * a.c.n_kv;
    g = at / nb;
    j = at - g * nb;
    row = j < ns ? j * CD_KB + 16 * (threadIdx.x >> 5) : (j - ns) * CD_KB + main;
  }
  __device__ __forceinline__ void next(const CacheAttnArgs& a, const DecodeSeqs& s) {
    row += CD_KB;
    if (++j == ns) row = main;
    if (j < nb) return;
    j = 0;
    if (++g == a.c.n_kv) {
      g = 0;
      do {
        ++b;                       // (there is a next unit, so there is a next sequence)
        nb = s.first[b + 1] - s.first[b];
      } while (nb == 0);
      open(a, s);
    }
    row = ns > 0 ? 16 * (threadIdx.x >> 5) : main;
  }
};

template <typename T, int DH>
struct CdCfg {
  static constexpr int ROW = DH * (int)sizeof(T);      // bytes of a cache row
  static constexpr int TILE = 16 * ROW;                // a warp's 16 keys (or values)
  static constexpr int STAGE = 2 * TILE + 64;          // keys, values, positions
  static constexpr int RING = CD_STAGES * STAGE;
  static constexpr int MLD = DH + 4;                   // merge buffer row
  // a warp's merge rows (4), which also hold its 16 x 16 probabilities (fp32)
  static constexpr int SLOT = 4 * MLD > 256 ? 4 * MLD : 256;
  static constexpr int QLD = DH + 4;                   // fp32 query row, its second half 4 on
  static constexpr int SMEM = 4 * RING + 4 * SLOT * 4 + (sizeof(T) == 4 ? 16 * (QLD + 1) * 4 : 0);
  static constexpr int CTAS = SMEM > 110 * 1024 ? 1 : 2;   // per SM
};

// The tile in hand, and what a warp needs of it.
struct DecodeTile {
  int rows, row0, p0, p_last, g;   // packed rows; first new row; positions of the first and last one
  SeenRows seen;
};
// Sixteen cached rows in shared memory: 16-byte piece c of row r at c ^ (r % 8).
struct DecodeKeys {
  uint32_t k, v;
  const int* pos;
  int r0;
  float* scores;                   // of row r0 and packed row 0, or null
  bool open;                       // seen by every query
};

// A warp's running state over its keys.
template <typename T, int DH> struct DecodeState;

template <int DH> struct DecodeState<bf16, DH> {
  uint32_t qa[DH / 16][4];
  int pq[2];
  float o[DH / 8][4], m[2], l[2];
  int gr, t4;

  __device__ __forceinline__ void begin(const CacheAttnArgs& a, const DecodeTile& t, float*) {
    const int lane = threadIdx.x & 31;
    gr = lane >> 2;
    t4 = lane & 3;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int x = gr + 8 * h;
      const bool live = x < t.rows;
      const int qi = live ? x / a.G : 0;
      const bf16* qr = (const bf16*)a.q + (t.row0 + qi) * a.qs + (t.g * a.G + (live ? x % a.G : 0)) * DH;
      pq[h] = a.q_pos ? __ldg(a.q_pos + t.row0 + qi) : t.p0 + qi;
#pragma unroll
      for (int k = 0; k < DH / 16; ++k) {
        qa[k][h] = live ? *(const uint32_t*)(qr + k * 16 + 2 * t4) : 0u;
        qa[k][2 + h] = live ? *(const uint32_t*)(qr + k * 16 + 8 + 2 * t4) : 0u;
      }
      m[h] = -INFINITY;
      l[h] = 0.f;
    }
#pragma unroll
    for (int n = 0; n < DH / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
  }

  __device__ __forceinline__ void tile(const CacheAttnArgs& a, const DecodeTile& t, const DecodeKeys& y,
                                       const float*, float*) {
    const int lane = threadIdx.x & 31;
    float sc[2][4];
#pragma unroll
    for (int n = 0; n < 2; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.f;
#pragma unroll
    for (int k = 0; k < DH / 16; ++k) {
      const int r = (lane & 7) + ((lane >> 4) << 3), c = 2 * k + ((lane >> 3) & 1);
      uint32_t b0, b1, b2, b3;
      ldsm_x4(y.k + r * (DH * 2) + ((c ^ (r & 7)) << 4), b0, b1, b2, b3);
      mma_bf16(sc[0], qa[k], b0, b1);
      mma_bf16(sc[1], qa[k], b2, b3);
    }
    float mx[2] = {m[0], m[1]};
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float v = sc[n][e] * a.scale_log2;
        if (!y.open) {
          const int kr = n * 8 + 2 * t4 + (e & 1), r = y.r0 + kr;
          const int pk = a.c.pos ? y.pos[kr] : r;
          if (!(row_seen(t.seen, r) && sees(pq[e >> 1], pk, a.window, a.sinks))) v = -INFINITY;
        }
        sc[n][e] = v;
        mx[e >> 1] = fmaxf(mx[e >> 1], v);
      }
    if (y.scores) {                // kept for the weights: 2 keys, 8 bytes, a thread and row
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (gr + 8 * h < t.rows)
#pragma unroll
          for (int n = 0; n < 2; ++n)
            *(float2*)(y.scores + 2 * t4 + (gr + 8 * h) * 16 + n * 8) =
                make_float2(sc[n][2 * h], sc[n][2 * h + 1]);
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
      ldsm_x4_t(y.v + r * (DH * 2) + ((c ^ (r & 7)) << 4), b0, b1, b2, b3);
      mma_bf16(o[2 * n], pa, b0, b1);
      mma_bf16(o[2 * n + 1], pa, b2, b3);
    }
  }

  // (max, sum) of its 16 rows
  __device__ __forceinline__ void stats(float2* ml) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      if (t4 == 0) ml[gr + 8 * h] = make_float2(m[h], l[h]);
    }
  }
  // rows x0 .. x0 + 3 of O
  __device__ __forceinline__ void put(float* dst, int ld, int x0) const {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int x = gr + 8 * h - x0;
      if (x >= 0 && x < 4)
#pragma unroll
        for (int n = 0; n < DH / 8; ++n)
          *(float2*)(dst + x * ld + 2 * t4 + n * 8) = make_float2(o[n][2 * h], o[n][2 * h + 1]);
    }
  }
};

template <int DH> struct DecodeState<float, DH> {
  static constexpr int CPL = DH / 32, CH = DH / 4, QLD = CdCfg<float, DH>::QLD;
  float o[16][CPL], m[16], l[16];  // m the same in all lanes, l a lane's own keys

  // the tile's queries, scaled, and their positions, for all warps
  __device__ __forceinline__ void begin(const CacheAttnArgs& a, const DecodeTile& t, float* sq) {
    for (int i = threadIdx.x; i < 16 * CH; i += CD_THREADS) {
      const int x = i / CH, c = (i % CH) * 4;
      float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
      if (x < t.rows) {
        f = *(const float4*)((const float*)a.q + (t.row0 + x / a.G) * a.qs + (t.g * a.G + x % a.G) * DH + c);
        f.x *= a.scale_log2; f.y *= a.scale_log2; f.z *= a.scale_log2; f.w *= a.scale_log2;
      }
      *(float4*)(sq + x * QLD + c + (c >= DH / 2 ? 4 : 0)) = f;
    }
    if (threadIdx.x < 16) {
      const int qi = (int)threadIdx.x < t.rows ? threadIdx.x / a.G : 0;
      ((int*)(sq + 16 * QLD))[threadIdx.x] = a.q_pos ? __ldg(a.q_pos + t.row0 + qi) : t.p0 + qi;
    }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < 16; ++x) {
      m[x] = -INFINITY;
      l[x] = 0.f;
#pragma unroll
      for (int c = 0; c < CPL; ++c) o[x][c] = 0.f;
    }
  }

  __device__ __forceinline__ void tile(const CacheAttnArgs& a, const DecodeTile& t, const DecodeKeys& y,
                                       const float* sq, float* sp) {
    const int lane = threadIdx.x & 31, key = lane & 15, half = lane >> 4;
    const int r = y.r0 + key, pk = a.c.pos ? y.pos[key] : r;
    const bool there = row_seen(t.seen, r);
    const int* pq = (const int*)(sq + 16 * QLD);
#pragma unroll
    for (int x0 = 0; x0 < 16; x0 += 4) {
      if (x0 >= t.rows) break;
      float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
      for (int c = 0; c < CH / 2; ++c) {
        const float4 k = lds128(y.k + key * (DH * 4) + (((half * (CH / 2) + c) ^ (key & 7)) << 4));
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          const float4 q = *(const float4*)(sq + (x0 + z) * QLD + half * (DH / 2 + 4) + 4 * c);
          s[z] = fmaf(q.x, k.x, s[z]);
          s[z] = fmaf(q.y, k.y, s[z]);
          s[z] = fmaf(q.z, k.z, s[z]);
          s[z] = fmaf(q.w, k.w, s[z]);
        }
      }
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        const int x = x0 + z;
        s[z] += __shfl_xor_sync(0xffffffffu, s[z], 16);
        if (!y.open && !(there && sees(pq[x], pk, a.window, a.sinks))) s[z] = -INFINITY;
        if (y.scores && half == 0 && x < t.rows) y.scores[x * 16 + key] = s[z];
        float mx = s[z];
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
        if (mx > m[x]) {           // the same in all lanes
          const float f = exp2f(m[x] - mx);
          m[x] = mx;
          l[x] *= f;
#pragma unroll
          for (int c = 0; c < CPL; ++c) o[x][c] *= f;
        }
        const float p = exp2f(s[z] - (m[x] == -INFINITY ? 0.f : m[x]));
        l[x] += p;
        if (half == 0) sp[x * 16 + key] = p;
      }
    }
    __syncwarp();
#pragma unroll
    for (int k0 = 0; k0 < 16; k0 += 4) {
      float v[4][CPL];
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        const int c = lane * CPL / 4;
        const uint32_t at = y.v + (k0 + z) * (DH * 4) + ((c ^ ((k0 + z) & 7)) << 4) + (lane * CPL % 4) * 4;
        if constexpr (CPL == 4) *(float4*)v[z] = lds128(at);
        else if constexpr (CPL == 2) *(float2*)v[z] = lds64(at);
        else v[z][0] = lds32(at);
      }
#pragma unroll
      for (int x0 = 0; x0 < 16; x0 += 4) {
        if (x0 >= t.rows) break;
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          const float4 p = *(const float4*)(sp + (x0 + z) * 16 + k0);
#pragma unroll
          for (int c = 0; c < CPL; ++c) {
            float& d = o[x0 + z][c];
            d = fmaf(p.x, v[0][c], d);
            d = fmaf(p.y, v[1][c], d);
            d = fmaf(p.z, v[2][c], d);
            d = fmaf(p.w, v[3][c], d);
          }
        }
      }
    }
    __syncwarp();
  }

  __device__ __forceinline__ void stats(float2* ml) {
#pragma unroll
    for (int x = 0; x < 16; ++x) {
#pragma unroll
      for (int d = 8; d > 0; d >>= 1) l[x] += __shfl_xor_sync(0xffffffffu, l[x], d);
      if ((threadIdx.x & 31) == 0) ml[x] = make_float2(m[x], l[x]);
    }
  }
  __device__ __forceinline__ void put(float* dst, int ld, int x0) const {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int x = 0; x < 16; ++x)
      if (x >= x0 && x < x0 + 4)
#pragma unroll
        for (int c = 0; c < CPL; ++c) dst[(x - x0) * ld + lane * CPL + c] = o[x][c];
  }
};

template <typename T, int DH>
__global__ void __launch_bounds__(CD_THREADS, (CdCfg<T, DH>::CTAS)) k_cache_decode(const CacheAttnArgs a) {
  using C = CdCfg<T, DH>;
  constexpr int CH = C::ROW / 16;  // 16-byte pieces of a row
  extern __shared__ __align__(16) uint8_t smb[];
  __shared__ DecodeSeqs s;
  __shared__ int s_scan[4];
  __shared__ float2 s_ml[4][CD_QT];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_trigger();
  decode_scan<CD_KB>(a, s, s_scan);
  if (blockIdx.x == 0 && a.score_units > 0)            // for the weights
    for (int b = tid; b <= a.B; b += CD_THREADS) a.plan_first[b] = s.first[b];
  const WorkRun w(s.first[256] * a.c.n_kv, gridDim.x);
  if ((int)blockIdx.x >= w.g || w.N == 0) {
    if (tid == 0) a.plan_join[2 * blockIdx.x] = make_int4(-1, 0, 0, 0);
    return;
  }
  const int u0 = w.start(blockIdx.x), count = w.start(blockIdx.x + 1) - u0;
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smb) + warp * C::RING;
  float* merge = (float*)(smb + 4 * C::RING);
  float* sq = merge + 4 * C::SLOT;                     // fp32: queries and positions

  DecodeCursor ld, cu;
  ld.seek(a, s, u0);
  cu = ld;
  if (tid == 0)
    put_join(a, w, blockIdx.x, u0 - ld.j, ld.nb, s.row0[ld.b], ld.g, 0, s.n[ld.b] * a.G);
  int ld_page = cache_page(a.c, ld.b, ld.row);
  uint32_t there = 0;              // bit k % 32: the page of the run's unit k exists
  // stage `st` <- the load cursor's unit, the run's unit k; then the cursor moves
  // on and its page number starts loading
  auto load = [&](int st, int k, bool more) {
    const uint32_t dst = ring + st * C::STAGE;
    const size_t at = cache_row(a.c, max(ld_page, 0), ld.g, ld.row);
    const char* gk = (const char*)a.c.k + at * C::ROW + lane * 16;
    const char* gv = (const char*)a.c.v + at * C::ROW + lane * 16;
    there = (there & ~(1u << (k & 31))) | (uint32_t)(ld_page >= 0) << (k & 31);
    const bool all = ld_page >= 0 && ld.row >= ld.v.lo && ld.row + 16 <= ld.v.hi;
#pragma unroll
    for (int i = 0; i < CH / 2; ++i) {
      const int x = lane + 32 * i, r = x / CH, c = x % CH;
      const bool live = all || (ld_page >= 0 && row_seen(ld.v, ld.row + r));
      const uint32_t o = r * C::ROW + ((c ^ (r & 7)) << 4);
      cp_async16_if(dst + o, gk + i * 512, live);
      cp_async16_if(dst + C::TILE + o, gv + i * 512, live);
    }
    if (a.c.pos && lane < 4)
      cp_async16_if(dst + 2 * C::TILE + lane * 16, a.c.pos + at + lane * 4, ld_page >= 0);
    if (more) {
      ld.next(a, s);
      ld_page = cache_page(a.c, ld.b, ld.row);
    }
  };
  int issued = 0;
#pragma unroll
  for (int i = 0; i < CD_STAGES - 1; ++i) {
    if (issued < count) {
      ++issued;
      load(i, i, issued < count);
    }
    cp_commit();
  }

  int done = 0, stage = 0;
  while (done < count) {
    // ---- one tile: the units of (cu.b, cu.g) in this run
    const int b = cu.b, g = cu.g, j0 = cu.j, nb = cu.nb;
    const int todo = min(nb - j0, count - done);
    const int rows = s.n[b] * a.G, row0 = s.row0[b], p0 = s.len[b];
    const SeenRows seen = cu.v;
    const DecodeTile tile = {rows, row0, p0, p0 + s.n[b] - 1, g, seen};
    DecodeState<T, DH> state;
    state.begin(a, tile, sq);

    for (int it = 0; it < todo; ++it) {
      cp_wait<CD_STAGES - 2>();
      __syncwarp();
      {
        // refill the stage freed by the previous unit
        const int st = stage == 0 ? CD_STAGES - 1 : stage - 1;
        if (issued < count) {
          ++issued;
          load(st, issued - 1, issued < count);
        }
        cp_commit();
      }
      const int r0 = cu.row;
      const bool here = there >> ((done + it) & 31) & 1u;
      if (it + 1 < todo) cu.next(a, s);
      const uint32_t kt = ring + stage * C::STAGE;
      // nothing of the tile is visible: skip it
      if (here && (r0 < seen.s_end || (r0 + 16 > seen.lo && r0 < seen.hi))) {
        const DecodeKeys keys = {
            kt, kt + C::TILE, (const int*)(smb + warp * C::RING + stage * C::STAGE + 2 * C::TILE), r0,
            u0 + done + it < a.score_units ? a.scores + score_at(a, u0 + done + it, warp, 0) : nullptr,
            !a.c.pos && r0 >= seen.lo && r0 + 15 <= p0 && r0 + 16 <= seen.hi &&
                (a.window == 0 || tile.p_last - r0 < a.window)};
        state.tile(a, tile, keys, sq, merge + warp * C::SLOT);
      }
      stage = stage + 1 == CD_STAGES ? 0 : stage + 1;
    }
    // ---- the four warps' states into one
    state.stats(s_ml[warp]);
    const bool whole = j0 == 0 && todo == nb;
    const int slot = done == 0 ? 0 : 1;
    // four rows at a time through the merge buffer
    for (int x0 = 0; x0 < rows; x0 += 4) {
      __syncthreads();
      state.put(merge + warp * C::SLOT, C::MLD, x0);
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
            acc[k] = fmaf(merge[i * C::SLOT + warp * C::MLD + lane * (DH / 32) + k], f[i], acc[k]);
        if (whole) {
          const int t = row0 + x / a.G, h = g * a.G + x % a.G;
          const float inv = ll != 0.f ? 1.f / ll : 0.f;
          T* const dst = (T*)a.out + t * a.os + h * DH + lane * (DH / 32);
          if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int k = 0; k < DH / 32; k += 2)
              *(uint32_t*)(dst + k) = pack_bf16x2(acc[k] * inv, acc[k + 1] * inv);
          } else {
#pragma unroll
            for (int k = 0; k < DH / 32; ++k) dst[k] = acc[k] * inv;
          }
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
    if (done < count) cu.next(a, s);
  }
  cp_wait<0>();
}

}  // namespace fm
