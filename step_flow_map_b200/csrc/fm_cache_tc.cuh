// Attention of many new rows over the paged cache (bf16, more than 16 packed
// rows per key/value head: drafted blocks, prompts) on tcgen05.
//
// Per block of 128 cache rows: S = Q K^T (128 packed rows x 128 keys, fp32 in
// TMEM), P = 2^(S - m) rounded to bf16 (the tensor path's type; the sums take p
// as it is), O += P V with P read from TMEM.  Keys and values come page by page through TMA into a ring
// of 128-row tiles (128-byte swizzle): K as the K-major operand, V as it lies,
// MN-major.  Two S/O pairs fill TMEM (2 x (128 + DH) columns), so one's
// exponentials run under the other's products; two softmax warpgroups work on
// each, a thread on 64 keys of one packed row (one warpgroup per pair, a thread
// on all 128 keys: 75 us for 2,777 rows over 4,001, 16 heads of width 64,
// against 68 when it was tried):
//   PAIR  (more than 128 packed rows) the pairs are two tiles of 128 rows that
//         share every K/V tile;
//   else  one tile of 128 rows: even blocks go to pair 0, odd ones to pair 1,
//         merged at the end of the tile.
// Bound: for prompts the exponentials (16 a clock and SM) and the products, each
// 43-44 % busy at width 128, where a pair's next S waits for the PV that reads
// its P; for drafted blocks HBM.  Whole calls, plan and join with them, their
// inputs not in L2 (the card's power decides the clock, and with it some 3 % of
// the first three): 8,192 rows, 32 heads of width 128, causal 565 us (0.97
// PFLOP/s), under a 2,048 window 322 (0.75); 8,192 causal rows of width 64 382
// (0.72); 2,777 rows over 4,001, 16 heads of width 64, 61 (0.48); 48 blocks of 17
// rows over 2,048..4,096 136, 5.6 TB/s inside the kernel.  Times beside the
// choices below compare two builds on one input that stays in L2, called over and
// over, and are lower.
//
// Roles (640 threads): warp 0 TMA, warp 1 MMA, warps 4-19 softmax.
// O is rescaled by the softmax threads, and only when a row maximum has grown
// by more than 2^8 since the reference in use: p stays below 2^8, which costs
// no precision in bf16 or fp32.  Every wait is bounded; a thread whose wait
// gave up goes on through the same barriers (later waits end at once) and the
// outputs that it may have spoilt are NaN.
#pragma once
#include "fm_cache_attn.cuh"
#include "fm_ptx.cuh"

namespace fm {

constexpr int CT_THREADS = 640;
constexpr int CT_KB = 128;

template <int DH>
struct CtCfg {
  static constexpr int TILE = 128 * DH * 2;            // 128 rows of Q, K or V
  static constexpr int BOX = 128 * 128;                // its 64-column half
  static constexpr int STAGES = DH == 128 ? 5 : 8;
  static constexpr int O_COL = 256;                    // TMEM: S0, S1 (128 each), O0, O1
  // Width 64 leaves TMEM columns for P of its own (after O), so a pair's next S
  // is made while its exponentials run; at 128 P lies over the second half of S,
  // and the next S follows the PV that reads it.  (At 128, S in two halves of 64
  // keys, the first made early, was slower: 8,192 rows under a 2,048 window 286
  // -> 307 us, as the queries are read from shared memory twice.)
  static constexpr bool AHEAD = DH == 64;
  static constexpr int P_COL = AHEAD ? O_COL + 64 : 64;   // of pair 0; pair 1: 128 on
  static constexpr int BARS = 2 * STAGES + 12;         // full, empty; per pair s_full, s_read,
                                                       //   p_full, o_full, q_full, q_empty
  static constexpr int SMEM = 2 * TILE + STAGES * TILE + 4 * 128 * 4 + BARS * 8 + 16 * 4 + 16;
};

// A stretch of one tile's units inside a CTA's run: nv of them, of which the
// last n are blocks, from block j0 on (see WorkRun; n may be 0).
struct TileSeg {
  int e, g, nv, j0, n, nb, b, x0, row0, all, p0;   // row0: first new row; all: its packed rows;
  SeenRows seen;                                   //   p0: position of its first new row
  __device__ __forceinline__ void at(const CacheAttnArgs& a, int u, int u1) {
    const int t0 = a.plan_first[e], units = a.plan_first[e + 1] - t0;
    const int4 t = a.plan_tile[2 * e], s = a.plan_tile[2 * e + 1];
    const int d = u - t0 * a.c.n_kv;
    g = d / units;
    const int v0 = d - g * units;
    nv = min(units - v0, u1 - u);
    nb = units - a.ov;
    j0 = max(0, v0 - a.ov);
    n = max(0, v0 + nv - a.ov) - j0;
    b = t.x;
    x0 = t.y;
    row0 = t.z;
    all = t.w;
    p0 = s.w;
    seen.s_end = s.x;
    seen.lo = s.y;
    seen.hi = s.z;
  }
  __device__ __forceinline__ void done(const CacheAttnArgs& a) {
    if (j0 + n == nb && g + 1 == a.c.n_kv) ++e;
  }
};

// Bits 0 .. n - 1 of a word, for any n.
__device__ __forceinline__ unsigned long long below(int n) {
  return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1ull;
}

template <int DH, bool PAIR>
__global__ void __launch_bounds__(CT_THREADS, 1)
k_cache_attn_tc(const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV,
                const __grid_constant__ CUtensorMap mapQ, const CacheAttnArgs a) {
  using C = CtCfg<DH>;
  constexpr int QT = PAIR ? 256 : 128;                 // partial rows of a tile
  extern __shared__ __align__(1024) uint8_t smem_tc[];
  uint8_t* sQ = smem_tc;                               // two tiles; the second is the merge
  uint8_t* sKV = sQ + 2 * C::TILE;                     //   buffer when there is one Q tile
  // [pair][half][row]: row maxima and sums that the halves exchange; stored key
  // positions of a pair's block lie over its first half's
  float* s_mx = (float*)(sKV + C::STAGES * C::TILE);
  uint64_t* bars = (uint64_t*)(s_mx + 512);
  uint64_t *full = bars, *empty = bars + C::STAGES, *s_full = empty + C::STAGES, *s_read = s_full + 2,
           *p_full = s_read + 2,           *o_full = p_full + 2, *q_full = o_full + 2, *q_empty = q_full + 2;
  // pages of a block that exist, by block of the CTA: written before its keys
  // are asked for, and at most STAGES / 2 + 1 blocks before its values are used
  uint32_t* s_pages = (uint32_t*)(bars + C::BARS);     // [16]
  uint32_t* tmem_slot = s_pages + 16;
  volatile int* abort = (volatile int*)(tmem_slot + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_trigger();
  if (tid == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(smem_u32(&full[i]), 1);
      mbar_init(smem_u32(&empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s_full[i]), 1);
      mbar_init(smem_u32(&p_full[i]), 256);
      mbar_init(smem_u32(&s_read[i]), 256);
      mbar_init(smem_u32(&o_full[i]), 1);
      mbar_init(smem_u32(&q_full[i]), 1);
      mbar_init(smem_u32(&q_empty[i]), PAIR ? 256 : 512);
    }
    *abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  const int E = a.plan_n[0];
  const WorkRun w(a.plan_first[E] * a.c.n_kv, gridDim.x);
  const bool active = (int)blockIdx.x < w.g && w.N > 0;
  const int u0 = active ? w.start(blockIdx.x) : 0, u1 = active ? w.start(blockIdx.x + 1) : 0;
  TileSeg seg;
  seg.e = active && warp != 3 ? find_tile(a, E, u0) : 0;
  if (warp == 0) {
    // ---------------- TMA producer: lane i takes the block's i-th page
    const int np = CT_KB >> a.c.ps_log2, ps = 1 << a.c.ps_log2;
    const int gone = a.c.n_pages * a.c.n_kv * ps;      // past the last row: reads zeros
    int cnt = 0, nseg = 0;
    bool go = true;                                    // the same in every lane
    for (int u = u0; u < u1 && go; u += seg.nv) {
      seg.at(a, u, u1);
      if (seg.n == 0) break;                            // the run ends in a tile's overhead
      // the tile's queries: G heads of a.rt / G rows, in packed order
      if (lane == 0) {
#pragma unroll
        for (int p = 0; p < (PAIR ? 2 : 1) && go; ++p) {
          go = mbar_wait(smem_u32(&q_empty[p]), (nseg & 1) ^ 1, abort);
          if (!go) break;
          mbar_expect_tx(smem_u32(&q_full[p]), a.rt * DH * 2);
#pragma unroll
          for (int h = 0; h < DH / 64; ++h)
            tma_load_4d(smem_u32(sQ + p * C::TILE + h * C::BOX), &mapQ, h * 64, 0, seg.g,
                        seg.row0 + (seg.x0 + p * a.rt) / a.G, smem_u32(&q_full[p]));
        }
      }
      go = __shfl_sync(0xffffffffu, go, 0);
      ++nseg;
      const SeenBlocks<CT_KB> blocks(seg.seen);
      for (int j = 0; j < seg.n && go; ++j) {
        const int r = blocks.row(seg.j0 + j) + lane * ps;
        int row = gone;
        if (lane < np && (r < seg.seen.s_end || (r + ps > seg.seen.lo && r < seg.seen.hi))) {
          const int page = cache_page(a.c, seg.b, r);
          if (page >= 0) row = (page * a.c.n_kv + seg.g) << a.c.ps_log2;
        }
        const uint32_t pages = __ballot_sync(0xffffffffu, row != gone);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv, ++cnt) {
          const int st = cnt % C::STAGES;
          const bool ok = go && mbar_wait(smem_u32(&empty[st]), ((cnt / C::STAGES) & 1) ^ 1, abort);
          go = __all_sync(0xffffffffu, ok);
          if (!go) continue;
          const uint32_t fb = smem_u32(&full[st]);
          if (lane == 0) {
            if (kv == 0) s_pages[(cnt >> 1) & 15] = pages;
            mbar_expect_tx(fb, C::TILE);
          }
          __syncwarp();
          if (lane < np)
#pragma unroll
            for (int h = 0; h < DH / 64; ++h)
              tma_load_2d(smem_u32(sKV + st * C::TILE + h * C::BOX + lane * ps * 128),
                          kv ? &mapV : &mapK, h * 64, row, fb);
        }
        __syncwarp();
      }
      seg.done(a);
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer.  Step s of a segment: PAIR: block s/2 for
    // pair s%2; else block s for pair s%2.  S runs two steps ahead of PV: a
    // pair's next S is issued once its scores have been read (AHEAD), else
    // after the PV that reads the P it overwrites.
    constexpr uint32_t idS = idesc_bf16<128>();
    constexpr uint32_t idO = idesc_bf16<DH>() | (1u << 16);   // V: MN-major
    // a wait that gave up is not acted on here: the remaining products run on
    // whatever is there, every later wait ends at once
    const uint64_t dk = desc_sw128(smem_u32(sKV)), dq = desc_sw128(smem_u32(sQ)),
                   dv = desc_sw128_mn(smem_u32(sKV), C::BOX);
    int cnt = 0, nseg = 0;                              // ring entries of earlier segments
    uint32_t pc0 = 0, pc1 = 0;                          // PV steps of each pair so far
    for (int u = u0; u < u1; u += seg.nv, ++nseg) {
      seg.at(a, u, u1);
      if (seg.n == 0) break;
      const int n = __shfl_sync(0xffffffffu, seg.n, 0);
      const int steps = PAIR ? 2 * n : n;
      auto issue_s = [&](int s) {
        const int j = PAIR ? s >> 1 : s, p = s & 1;
        const int c = cnt + 2 * j, st = c % C::STAGES;
        if (s < (PAIR ? 2 : 1)) (void)mbar_wait(smem_u32(&q_full[p]), nseg & 1, abort);
        if (!PAIR || p == 0) (void)mbar_wait(smem_u32(&full[st]), (c / C::STAGES) & 1, abort);
        tc_fence_after();
#pragma unroll
        for (int h = 0; h < DH / 64; ++h)
          tc_mma4(tmem + p * 128, (uint32_t)dq + (((PAIR ? p * C::TILE : 0) + h * C::BOX) >> 4),
                  (uint32_t)dk + ((st * C::TILE + h * C::BOX) >> 4), (uint32_t)(dk >> 32), idS, h > 0);
        if (!PAIR || p == 1) tc_commit_elect(smem_u32(&empty[st]));
        tc_commit_elect(smem_u32(&s_full[p]));
      };
      auto issue_pv = [&](int s) {
        const int j = PAIR ? s >> 1 : s, p = s & 1;
        const int c = cnt + 2 * j + 1, st = c % C::STAGES;
        (void)mbar_wait(smem_u32(&full[st]), (c / C::STAGES) & 1, abort);
        (void)mbar_wait(smem_u32(&p_full[p]), (p ? pc1 : pc0) & 1, abort);
        tc_fence_after();
#pragma unroll
        for (int h = 0; h < 2; ++h)
          tc_mma4_ts(tmem + C::O_COL + p * 128, tmem + C::P_COL + p * 128 + h * 32,
                     (uint32_t)dv + ((st * C::TILE + h * 64 * 128) >> 4), (uint32_t)(dv >> 32), idO,
                     s >= 2 || h > 0);
        if (!PAIR || p == 1) tc_commit_elect(smem_u32(&empty[st]));
        if (C::AHEAD || s + 2 >= steps) tc_commit_elect(smem_u32(&o_full[p]));
      };
      issue_s(0);
      if (steps > 1) issue_s(1);
      for (int s = 0; s < steps; ++s) {
        const int p = s & 1;
        const bool more = s + 2 < steps;
        if (C::AHEAD && more) {
          // (a pair's s_read and p_full complete once a step, so they share the count)
          (void)mbar_wait(smem_u32(&s_read[p]), (p ? pc1 : pc0) & 1, abort);
          issue_s(s + 2);
        }
        issue_pv(s);
        if (!C::AHEAD && more) issue_s(s + 2);
        p ? ++pc1 : ++pc0;
      }
      cnt += 2 * n;
      seg.done(a);
    }
  } else if (warp == 2) {
    // ---------------- what the join kernel finds at this run's start
    if (lane == 0 && !active) a.plan_join[2 * blockIdx.x] = make_int4(-1, 0, 0, 0);
    if (lane == 0 && active) {
      seg.at(a, u0, u1);
      const int t0 = a.plan_first[seg.e] * a.c.n_kv;
      put_join(a, w, blockIdx.x, t0 + seg.g * (seg.nb + a.ov), seg.nb + a.ov, seg.row0, seg.g, seg.x0,
               seg.all);
    }
  } else if (warp >= 4) {
    // ---------------- softmax: thread = 64 keys (`half`) of packed row `r` of pair `p`
    const int p = (warp - 4) >> 3, half = ((warp - 4) >> 2) & 1, r = tid & 127;
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t tS = tl + p * 128, tO = tl + C::O_COL + p * 128 + half * (DH / 2),
                   tP = tl + C::P_COL + p * 128 + half * 32;
    const int rows_bar = 1 + p * 4 + (warp & 3), pair_bar = 9 + p;   // two warps, eight warps
    float* const mine = s_mx + (p * 2 + half) * 128 + r;
    const float* const others = s_mx + (p * 2 + (half ^ 1)) * 128 + r;
    int* const s_kpos = (int*)(s_mx + p * 256);
    uint32_t sc = 0, oc = 0;                            // phases of s_full and o_full seen
    int cnt = 0;                                        // ring entries of earlier segments
    const int np = CT_KB >> a.c.ps_log2;
    const uint32_t all_pages = (1u << np) - 1u;
    for (int u = u0; u < u1; u += seg.nv) {
      seg.at(a, u, u1);
      if (seg.n == 0) break;
      const SeenBlocks<CT_KB> blocks(seg.seen);
      const int all = seg.all;
      const int xw = seg.x0 + (PAIR ? p * a.rt : 0);    // this pair's first packed row
      const int x = xw + r;
      const bool live = r < a.rt && x < all;
      const int qi = live ? x / a.G : 0, hq = seg.g * a.G + (live ? x - qi * a.G : 0);
      const int pq = a.q_pos ? __ldg(a.q_pos + seg.row0 + qi) : seg.p0 + qi;
      // blocks that every row of this pair sees whole: those from row `open_lo` to
      // row `open_hi` on (p_first, p_last: the pair's first and last position)
      const int p_first = seg.p0 + min(xw, all - 1) / a.G;
      const int p_last = seg.p0 + (min(xw + a.rt, all) - 1) / a.G;
      const int open_lo = max(seg.seen.lo, a.window > 0 && p_last >= a.window ? p_last - a.window + 1 : 0);
      const int open_hi = a.c.pos ? -1 : min(seg.seen.hi - CT_KB, p_first - (CT_KB - 1));
      float m = -INFINITY, l = 0.f;                     // l: this thread's keys
      bool first = true;
      for (int j = PAIR ? 0 : p; j < seg.n; j += PAIR ? 1 : 2) {
        const int r0 = blocks.row(seg.j0 + j);
        // The scores or the V tile say that the block's pages are noted down.  The
        // V tile where it is there already as a rule and this thread, waiting for
        // the scores, can decide about masks meanwhile (8,192 rows under a 2,048
        // window, width 128: 283 us against 292).  The scores where the loop is
        // bound by this thread's instructions (width 64, 8,192 causal rows: 376 us
        // against 396) or by the tiles' arrival (one Q tile).
        const int ring = cnt + 2 * j + 1;               // the block's V tile
        auto wait_v = [&]() {
          (void)mbar_wait(smem_u32(&full[ring % C::STAGES]), (ring / C::STAGES) & 1, abort);
        };
        auto wait_s = [&]() { (void)mbar_wait(smem_u32(&s_full[p]), sc++ & 1, abort); };
        constexpr bool BY_V = PAIR && !C::AHEAD;
        if constexpr (BY_V) wait_v();
        else wait_s();
        const uint32_t pages = s_pages[(ring >> 1) & 15];
        const bool open = r0 >= open_lo && r0 <= open_hi && pages == all_pages;
        uint32_t see0 = ~0u, see1 = ~0u;                // this thread's mask of its 64 keys
        if (!open) {
          const int kr = r0 + r;
          const bool inside = r0 >= seg.seen.lo && r0 + CT_KB <= seg.seen.hi;
          if (!inside || a.c.pos) {
            named_sync(pair_bar, 256);                  // the last block's readers are done
            if (a.c.pos && half == 0) {
              int kp = 0;
              if (row_seen(seg.seen, kr) && ((pages >> (r >> a.c.ps_log2)) & 1u))
                kp = a.c.pos[cache_row(a.c, cache_page(a.c, seg.b, kr), seg.g, kr)];
              s_kpos[r] = kp;
            }
            // value rows in pages that exist but that nobody sees may hold
            // anything: zero them, as 0 x NaN would not be 0
            if (!inside) {
              if constexpr (!BY_V) wait_v();
              if (!row_seen(seg.seen, kr)) {
                uint8_t* v = sKV + (ring % C::STAGES) * C::TILE + r * 128;
#pragma unroll
                for (int z = 0; z < DH / 16; ++z) {     // neighbouring rows on different banks
                  const int c = half * (DH / 16) + z;
                  *(uint4*)(v + (c >> 3) * C::BOX + (((c + r) & 7) << 4)) = make_uint4(0, 0, 0, 0);
                }
              }
              asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            }
            named_sync(pair_bar, 256);
          }
          // without stored positions a row sees keys [0, c_sink) and [c_lo, c_hi)
          // of the block (counted from r0; r0 and the ends are cache rows, and
          // pq + 1 only matters up to hi)
          const int c_hi = min(seg.seen.hi, min(pq, seg.seen.hi) + 1) - r0;
          const int c_lo = a.window > 0 && pq >= a.window ? pq - a.window + 1 - r0 : 0;
          const int c_sink = a.window > 0 ? min(a.sinks - r0, c_hi) : 0;
          const int c0 = half * 64, c = c0 + lane;
          const uint32_t k0 = __ballot_sync(
              0xffffffffu, row_seen(seg.seen, r0 + c) && ((pages >> (c >> a.c.ps_log2)) & 1u));
          const uint32_t k1 = __ballot_sync(
              0xffffffffu,
              row_seen(seg.seen, r0 + c + 32) && ((pages >> ((c + 32) >> a.c.ps_log2)) & 1u));
          unsigned long long see = 0ull;
          if (a.c.pos) {
#pragma unroll 4
            for (int i = 0; i < 64; ++i)
              see |= (unsigned long long)sees(pq, s_kpos[c0 + i], a.window, a.sinks) << i;
            named_sync(pair_bar, 256);                  // the maxima go where the positions are
          } else {
            see = (below(c_hi - c0) & ~below(c_lo - c0)) | below(c_sink - c0);
          }
          see0 = (uint32_t)see & k0;
          see1 = (uint32_t)(see >> 32) & k1;
        }
        if constexpr (BY_V) wait_s();
        // the tile's last scores are there: its queries may be replaced
        if (j + (PAIR ? 1 : 2) >= seg.n) mbar_arrive(smem_u32(&q_empty[PAIR ? p : 0]));
        tc_fence_after();
        uint32_t s[64];
        tmem_ld64(tS + half * 64, s);
        if (!open) {
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (!(((c < 32 ? see0 : see1) >> (c & 31)) & 1u)) s[c] = 0xff800000u;   // -inf
        }
        float mx[2] = {__uint_as_float(s[0]), __uint_as_float(s[1])};
#pragma unroll
        for (int c = 2; c < 62; c += 4)
#pragma unroll
          for (int z = 0; z < 2; ++z)
            mx[z] = max3(mx[z], __uint_as_float(s[c + 2 * z]), __uint_as_float(s[c + 2 * z + 1]));
        const float my_top = max3(fmaxf(mx[0], mx[1]), __uint_as_float(s[62]), __uint_as_float(s[63]));
        *mine = my_top;
        // also: both halves of the scores are in registers, P may overwrite them
        tc_fence_before();
        named_sync(rows_bar, 64);
        tc_fence_after();
        const float top = fmaxf(my_top, *others) * a.scale_log2;
        if (C::AHEAD) mbar_arrive(smem_u32(&s_read[p]));
        // (both halves of a row come to the same m and f; rows of no query, whose
        // scores are of whatever the tile held or of the next sequence's queries,
        // have no vote, so they cannot change how the others are rounded)
        const bool grow = !first && __any_sync(0xffffffffu, live && top > m + 8.f);
        float f = 1.f;
        if (first) {
          m = top;
        } else if (grow) {
          const float mn = fmaxf(m, top);
          if (mn != -INFINITY) f = ex2(m - mn);
          m = mn;
          l *= f;
        }
        const float ref = m == -INFINITY ? 0.f : m;
        const uint64_t scale2 = pack2(a.scale_log2, a.scale_log2), ref2 = pack2(-ref, -ref);
        uint64_t ls[2] = {0ull, 0ull};
#pragma unroll
        for (int c = 0; c < 64; c += 2) {
          const uint64_t t =
              fma2(pack2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), scale2, ref2);
          float p0, p1;
          unpack2(t, p0, p1);
          p0 = ex2(p0);
          p1 = ex2(p1);
          ls[(c >> 1) & 1] = add2(ls[(c >> 1) & 1], pack2(p0, p1));
          s[c >> 1] = pack_bf16x2(p0, p1);
        }
        if (C::AHEAD && !first) {                        // the PV before has read P and left O alone
          (void)mbar_wait(smem_u32(&o_full[p]), oc++ & 1, abort);
          tc_fence_after();
        }
        first = false;
        tmem_st32(tP, s);
        float l0, l1;
        unpack2(add2(ls[0], ls[1]), l0, l1);
        l += l0 + l1;
        if (grow) {
#pragma unroll 1
          for (int c = 0; c < DH / 2; c += 32) {
            uint32_t o[32];
            tmem_ld32(tO + c, o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            tmem_st32(tO + c, o);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(smem_u32(&p_full[p]));
      }
      if (!PAIR && p >= seg.n) mbar_arrive(smem_u32(&q_empty[0]));   // it had no block
      // ---- the segment's result: half of a row's columns a thread
      const bool whole = seg.j0 == 0 && seg.n == seg.nb;
      const size_t prt = (size_t)blockIdx.x * 2 + (u == u0 ? 0 : 1);   // its slot
      const int pr = (PAIR ? p * 128 : 0) + r;
      const int t = seg.row0 + qi;
      auto put = [&](int c0, const uint32_t* o, float f) {   // 32 columns, from c0 of this half on
        if (!live) return;
        c0 += half * (DH / 2);
        if (whole) {
          bf16* const dst = (bf16*)a.out + t * a.os + hq * DH + c0;
#pragma unroll
          for (int i = 0; i < 32; i += 8) {
            uint32_t v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              v[k] = pack_bf16x2(__uint_as_float(o[i + 2 * k]) * f, __uint_as_float(o[i + 2 * k + 1]) * f);
            *(uint4*)(dst + i) = make_uint4(v[0], v[1], v[2], v[3]);
          }
        } else {
          // [column][row], so that a warp's store is one line
          float* const dst = a.part + (prt * DH + c0) * QT + pr;
#pragma unroll
          for (int i = 0; i < 32; ++i) dst[(size_t)i * QT] = __uint_as_float(o[i]);
        }
      };
      auto stats = [&](float mm, float ll) {
        if (!live || half) return;
        if (!whole) a.part_ml[prt * QT + pr] = make_float2(mm, ll);
        else if (a.lse)
          a.lse[(size_t)t * a.n_heads + hq] =
              ll != 0.f ? (mm + log2f(ll)) * 0.69314718055994531f : -INFINITY;
      };
      if (PAIR || p == 0 || seg.n > 1) (void)mbar_wait(smem_u32(&o_full[p]), oc++ & 1, abort);
      tc_fence_after();
      if (*abort) l = NAN;                              // a wait gave up: no result, and none to trust
      *mine = l;
      named_sync(rows_bar, 64);
      l += *others;
      named_sync(rows_bar, 64);                         // before the next maximum replaces it
      if constexpr (PAIR) {
        const float f = l != 0.f ? 1.f / l : 0.f;
#pragma unroll 1
        for (int c = 0; c < DH / 2; c += 32) {
          uint32_t o[32];
          tmem_ld32(tO + c, o);
          put(c, o, f);
        }
        stats(m, l);
      } else {
        // pair 1's state goes to pair 0: (max, sum) in its two slots of s_mx, O
        // through the second Q tile (64 columns at width 128, 32 at 64) in two
        // rounds; the four warps of a row meet
        const int merge_bar = 11 + (warp & 3);
        if (p == 1) *mine = half ? l : m;
#pragma unroll 1
        for (int k = 0; k < 2; ++k) {
          const bool on = DH == 128 || half == k;
          const int c = DH == 128 ? 32 * k : 0;
          float* const buf = (float*)(sQ + C::TILE) + (DH == 128 ? half * 32 * 128 : 0) + r;
          if (p == 1 && on && seg.n > 1) {
            uint32_t o[32];
            tmem_ld32(tO + c, o);
#pragma unroll
            for (int i = 0; i < 32; ++i) buf[i * 128] = __uint_as_float(o[i]);
          }
          named_sync(merge_bar, 128);
          if (p == 0 && on) {
            const float m1 = s_mx[256 + r], l1 = s_mx[384 + r];
            const float mm = fmaxf(m, m1), rf = mm == -INFINITY ? 0.f : mm;
            const float f0 = ex2(m - rf), f1 = seg.n > 1 ? ex2(m1 - rf) : 0.f;
            const float ll = l * f0 + (seg.n > 1 ? l1 * f1 : 0.f);
            const float f = ll != 0.f ? 1.f / ll : 0.f;
            uint32_t o[32];
            tmem_ld32(tO + c, o);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              float v = __uint_as_float(o[i]) * f0;
              if (seg.n > 1) v = fmaf(buf[i * 128], f1, v);
              o[i] = __float_as_uint(v);
            }
            put(c, o, f);
            if (k == 0) stats(mm, ll);
          }
          named_sync(merge_bar, 128);
        }
      }
      tc_fence_before();
      cnt += 2 * seg.n;
      seg.done(a);
    }
  }

  // ---------------- teardown
  tc_fence_before();
  __syncthreads();
  if (*abort) {
    // let copies and MMAs already issued land before the memory goes away
    const unsigned long long t0 = gtimer();
    while (gtimer() - t0 < 50000ull) {
    }
    __syncthreads();
  }
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace fm
