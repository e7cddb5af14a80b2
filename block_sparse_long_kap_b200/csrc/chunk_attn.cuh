// Attention of a ragged batch of new tokens over the paged cache (cosa_chunk_attention),
// from one token a sequence to whole prompts, on the sm_100a tensor cores.
//
// A tile is 128 rows of (token, query head of the KV head's group): G heads share every
// K / V block whatever the number of tokens.  Sequences with more than 128 rows take tiles in
// pairs (NT = 2), which halves the K / V traffic from L2; up to 128 rows a sequence run one
// tile (NT = 1).  (Up to 16 rows at D = 128: chunk_decode.cuh.)
//
// The work is cut by blocks of 128 keys, not by tiles: chunk_plan_kernel lists every
// tile's block range [jb, jb + nb) (window, documents and prefix shrink it) and the running
// sum of nb and a tile's setup; the 148 CTAs of chunk_attn_kernel (one per SM, each resident for the whole
// launch) take equal shares of that sum, a share running over the end of one tile into the
// next.  A tile cut between CTAs leaves unnormalised fp32 partial rows (at most two a CTA),
// which chunk_combine_kernel joins; so one long sequence, a ragged batch and a prompt
// whose tile count does not divide by 148 all end together.
//
// A block is worked off in halves of 64 keys, with two S buffers a tile: the scores of a half
// come in while the softmax is on the one before, so neither waits for the other (whole
// blocks with one buffer: 4.6 k cycles for 128 keys of a pair of tiles; halves with one warp
// issuing for both tiles: 6.7 k; halves with a warp a tile: 3.8 k, the products alone 2.6 k).
//
// Roles of the 4 + 4 NT warps:
//   warp 0     Q and K loads (TMA through the page table, lane t takes page t)
//   warp 1     MMA issue of tile 0, and
//   warp 3     of tile 1; warp 3 also owns the TMEM allocation
//   warp 2     V loads; values behind the sequence's end are zeroed (they may hold NaN,
//              and a zero weight times NaN is NaN); the join list
//   warps 4..  softmax of tile 0 / 1, one row per thread (its TMEM lane)
// S, P (bf16, over S) and O live in TMEM; the exponent base m_ref moves only when the row
// max passes it by 2^8.  Row max, sums and O are fp32; P is rounded to bf16 for the second
// product (relative error 2^-8 a weight at most, averaged over the keys), its sum is not: the output is off
// by 2.0e-3 to 2.3e-3 of its norm, of which its own rounding makes 1.6e-3.  P as a high and a low bf16
// half (chunk_decode.cuh) leaves 1.6e-3, for half as much again in products: 2,048 tokens on 32K
// keys 1,515 against 1,170 us, packed documents 244 against 212, prefix with bias (D = 64) 87 against
// 84.
// Every wait is bounded, as in the dense kernel.
//
// Measured: 1,010-1,090 TFLOP/s on a 16K prompt (32 / 8 heads, D = 128; the dense kernel beside it
// 930-960), and 1.20 ms for 2,048 tokens on 32K keys in a long run, 0.58 of the burst rate: the
// power cap holds the clock at 1.65 GHz there.  Moving a quarter of the exponentials to the FMA
// pipe shortens the softmax and lengthens the run (1.30 -> 1.33 ms): what costs then is energy.
#pragma once

#include <type_traits>

#include "chunk_common.cuh"
#include "chunk_list.h"

namespace cosa {

struct ChunkAttnParams {
  ChunkSeqs seqs;
  ChunkMask mask;
  const int32_t* page_table;
  const float* slopes;  // [H_q] or null
  __nv_bfloat16* out;   // [total_q][H_q][D]
  float* lse;           // [total_q][H_q] or null
  ChunkTile* tiles;     // workspace [max tiles]
  long long* cum;       // workspace [max tiles + 1]
  int* n_tiles;         // workspace
  ChunkJoin* joins;     // workspace [NUM_SMS]
  float* part_o;        // workspace [2 NUM_SMS][part_rows][D]
  float2* part_ml;      // workspace [2 NUM_SMS][part_rows]: exponent base, sum
  int num_q_heads, num_kv_heads, group, page_size, pages_per_seq, num_phys_pages;
  int tile_tokens;  // 128 / G
  int nt;           // tiles a CTA works on at once
  int part_rows;
  int max_tiles;    // room in the workspace
  ScoreShape score;
  unsigned long long timeout_ns;
};

__device__ __forceinline__ ChunkBounds chunk_bounds(const ChunkAttnParams& p) {
  return ChunkBounds{p.seqs.batch, p.seqs.total_q, p.seqs.max_kv, p.num_kv_heads,
                     p.tile_tokens * p.nt, p.max_tiles, NUM_SMS};
}

// Half blocks of 64 keys that nb blocks from one with `keys` keys left on hold.
__device__ __forceinline__ int half_blocks(int nb, int keys) {
  return min(2 * nb, max((keys + 63) >> 6, 1));
}

// A CTA's walk over its share [w, w_end) of the plan; every role walks by itself.
struct ChunkWalk {
  long long w, w_end, per_head;
  int hk, t, n_tiles;
  // the segment
  ChunkTile tile;
  int jb, nb;       // its blocks
  int part;         // -1: the whole tile; else partial slot 0 (starts inside) / 1
  int lead;         // units of the tile's setup that fall into the share
  // (an entry that does not fit the call is reported, and ends the walk)
  __device__ __forceinline__ bool next(const ChunkAttnParams& p) {
    if (w >= w_end) return false;
    const int4 x = __ldcg(reinterpret_cast<const int4*>(p.tiles + t));
    const int4 y = __ldcg(reinterpret_cast<const int4*>(p.tiles + t) + 1);
    const long long behind = w - hk * per_head - __ldcg(p.cum + t);
    tile.tok0 = x.x; tile.ntok = x.y; tile.pos0 = x.z; tile.b = x.w;
    tile.jb = y.x; tile.nb = y.y; tile.kv = y.z; tile.prefix = y.w;
    if (!tile_fits(chunk_bounds(p), tile, behind, hk)) {
      set_status(COSA_ERR_WORKSPACE);
      w = w_end;
      return false;
    }
    const int at = (int)behind - CHUNK_SETUP;  // negative: in front of the tile's blocks
    const int off = max(at, 0);
    lead = max(-at, 0);
    const long long left = w_end - w - lead;
    if (left <= 0) return false;
    jb = tile.jb + off;
    nb = left < tile.nb - off ? (int)left : tile.nb - off;
    part = off > 0 ? 0 : (nb < tile.nb ? 1 : -1);
    return true;
  }
  __device__ __forceinline__ void advance() {
    w += lead + nb;
    if (jb + nb == tile.jb + tile.nb && ++t == n_tiles) {
      t = 0;
      ++hk;
    }
  }
};

// What a row's sum l makes of its O, and its lse.  l = 0: it sees no key.  A NaN among the scores
// that it sees makes l NaN, and the row with it.
__device__ __forceinline__ float row_scale(float l) { return l != 0.f ? 1.f / l : 0.f; }
__device__ __forceinline__ float row_lse(float m, float l) {
  return l != 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

// ---- plan -----------------------------------------------------------------------------
constexpr int PLAN_THREADS = 1024;

__device__ __forceinline__ long long plan_scan(long long v, long long* red, long long& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  long long inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) red[warp] = inc;
  __syncthreads();
  long long w = lane < PLAN_THREADS / 32 ? red[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const long long before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
  __syncthreads();
  return (warp ? before : 0) + inc - v;
}

// One CTA.  Dynamic shared memory: first tile of each sequence, [batch + 1] int.
__global__ void __launch_bounds__(PLAN_THREADS) chunk_plan_kernel(const ChunkAttnParams p) {
  extern __shared__ int first_tile[];
  __shared__ long long red[32];
  pdl_launch();
  const int tid = threadIdx.x, B = p.seqs.batch;
  const int span = p.tile_tokens * p.nt;  // tokens a tile (pair)
  long long base = 0, total;
  for (int b0 = 0; b0 < B; b0 += PLAN_THREADS) {
    const int b = b0 + tid;
    long long n = 0;
    if (b < B) n = (chunk_seq(p.seqs, b).q_len + span - 1) / span;
    const long long before = plan_scan(n, red, total);
    if (b < B) first_tile[b] = (int)(base + before);
    base += total;
  }
  // overlapping sequences (cu_q going back and forth) can add up to more tiles than
  // total_q tokens give: nothing is run then
  if (base > p.max_tiles && tid == 0) set_status(COSA_ERR_INVALID_ARG);
  const int T = base > p.max_tiles ? 0 : (int)base;
  if (tid == 0) {
    first_tile[B] = T;
    *p.n_tiles = T;
  }
  __syncthreads();
  base = 0;
  for (int t0 = 0; t0 < T; t0 += PLAN_THREADS) {
    const int t = t0 + tid;
    ChunkTile d;
    d.nb = 0;
    if (t < T) {
      int lo = 0, hi = B - 1;  // the last sequence whose first tile is at or before t
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first_tile[mid] <= t) lo = mid;
        else hi = mid - 1;
      }
      const ChunkSeq s = chunk_seq(p.seqs, lo);
      const int i0 = (t - first_tile[lo]) * span;
      d.b = lo;
      d.tok0 = s.q0 + i0;
      d.ntok = min(span, s.q_len - i0);
      d.pos0 = s.kv - s.q_len + i0;
      d.kv = s.kv;
      d.prefix = p.mask.prefix_len ? __ldg(p.mask.prefix_len + lo) : 0;
      int kmin = INT_MAX, kmax = -1;
      if (p.mask.first_key) {
        for (int i = 0; i < d.ntok; ++i) {
          int a, z;
          token_range(p.mask, d.tok0 + i, d.pos0 + i, d.kv, d.prefix, a, z);
          if (a <= z) {
            kmin = min(kmin, a);
            kmax = max(kmax, z);
          }
        }
      } else {  // both ends grow with the position
        int z;
        token_range(p.mask, d.tok0, d.pos0, d.kv, d.prefix, kmin, z);
        int a;
        token_range(p.mask, d.tok0 + d.ntok - 1, d.pos0 + d.ntok - 1, d.kv, d.prefix, a, kmax);
      }
      // a tile without any visible key works through one masked block: zeros and -inf
      d.jb = kmax >= 0 ? kmin >> 7 : 0;
      d.nb = kmax >= 0 ? (kmax >> 7) + 1 - d.jb : 1;
    }
    const long long before = plan_scan(t < T ? d.nb + CHUNK_SETUP : 0, red, total);
    if (t < T) {
      p.tiles[t] = d;
      p.cum[t] = base + before;
    }
    base += total;
  }
  if (tid == 0) p.cum[T] = base;
}

// ---- attention ------------------------------------------------------------------------
template <int D, int NT>
struct ChunkCfg {
  static constexpr int KB = 128;                    // keys a block
  static constexpr int THREADS = 128 + 128 * NT;
  static constexpr uint32_t Q_BYTES = 128 * D * 2;  // one tile
  static constexpr uint32_t BLK_BYTES = KB * D * 2;
  static constexpr int KS = D == 128 ? 3 : 5;       // K ring slots
  static constexpr int VS = D == 128 ? (NT == 1 ? 3 : 2) : 5;
  static constexpr uint32_t OFF_Q = 0;
  static constexpr uint32_t OFF_K = OFF_Q + NT * Q_BYTES;
  static constexpr uint32_t OFF_V = OFF_K + KS * BLK_BYTES;
  static constexpr uint32_t OFF_BAR = OFF_V + VS * BLK_BYTES;
  // q full / empty, k full / empty, v full / empty, v tail, s full[2][2], p full[2][2],
  // o full[2], pv done[2], done[2]
  static constexpr int NBAR = 2 + 2 * KS + 2 * VS + 1 + 8 + 4 + 2;
  static constexpr uint32_t OFF_MISC = (OFF_BAR + NBAR * 8 + 15) & ~15u;
  static constexpr uint32_t SMEM = OFF_MISC + 32;   // TMEM address, abort, start tile
  static constexpr uint32_t SMEM_ALLOC = SMEM + 1024;  // 1024-byte alignment slack
  static constexpr int COL_O = 256;                 // S buffers: tile i at 128 i, 64 columns each
  static constexpr float kRescale = 8.0f;
  static_assert(SMEM_ALLOC <= 227 * 1024, "shared memory budget");
};

template <int D, int NT, CapForm CAP, bool BIAS>  // CAP: none, or the form beyond y = 0.625
__global__ void __launch_bounds__(128 + 128 * NT, 1)
    chunk_attn_kernel(const __grid_constant__ CUtensorMap tm_q,
                      const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const ChunkAttnParams prm) {
  using C = ChunkCfg<D, NT>;
  using namespace tc;
  // A bias makes the near keys' scores the largest: a segment's half blocks go from the last to the
  // first then, and the exponent base seldom moves (1,510 tokens on 7,339 keys, 16 heads with
  // slopes 2^-0.5 to 2^-8, D = 64: 92 us from the first to the last, 82 this way)
  constexpr bool REV = BIAS;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t sraw = static_cast<uint32_t>(__cvta_generic_to_shared(smem_raw));
  const uint32_t sb0 = (sraw + 1023u) & ~1023u;
  uint8_t* sg = smem_raw + (sb0 - sraw);
  const uint32_t sQ = sb0 + C::OFF_Q, sK = sb0 + C::OFF_K, sV = sb0 + C::OFF_V;
  const uint32_t bar = sb0 + C::OFF_BAR;
  const uint32_t b_qfull = bar, b_qempty = bar + 8;
  auto b_kfull = [&](int s) { return bar + 8u * (2 + s); };
  auto b_kempty = [&](int s) { return bar + 8u * (2 + C::KS + s); };
  auto b_vfull = [&](int s) { return bar + 8u * (2 + 2 * C::KS + s); };
  auto b_vempty = [&](int s) { return bar + 8u * (2 + 2 * C::KS + C::VS + s); };
  constexpr int B0 = 2 + 2 * C::KS + 2 * C::VS;
  const uint32_t b_vtail = bar + 8u * B0;
  auto b_sfull = [&](int i, int buf) { return bar + 8u * (B0 + 1 + 2 * i + buf); };
  auto b_pfull = [&](int i, int buf) { return bar + 8u * (B0 + 5 + 2 * i + buf); };
  auto b_ofull = [&](int i) { return bar + 8u * (B0 + 9 + i); };
  auto b_pv = [&](int i) { return bar + 8u * (B0 + 11 + i); };
  auto b_done = [&](int i) { return bar + 8u * (B0 + 13 + i); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sg + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sg + C::OFF_MISC + 4);
  volatile int* start_tile = reinterpret_cast<volatile int*>(sg + C::OFF_MISC + 8);

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform for the compiler too
  if (__syncthreads_or(*(volatile int*)&g_status == COSA_ERR_TIMEOUT)) {
    // an earlier launch timed out: nothing is run, and the join (which comes all the same) must
    // not take what the workspace holds for a list
    // (the plan writes to the workspace: this grid, and the join behind it, end after it)
    pdl_wait();
    if (tid == 0) prm.joins[blockIdx.x].ntok = 0;
    return;
  }
  const int G = prm.group, TOK = prm.tile_tokens, P = prm.page_size;

  if (tid == 0) {
    mbar_init(b_qfull, 1);
    // a slot is free when the issuers of both tiles have let it go
    mbar_init(b_qempty, NT);
    for (int s = 0; s < C::KS; ++s) { mbar_init(b_kfull(s), 1); mbar_init(b_kempty(s), NT); }
    for (int s = 0; s < C::VS; ++s) { mbar_init(b_vfull(s), 1); mbar_init(b_vempty(s), NT); }
    mbar_init(b_vtail, 1);
    for (int i = 0; i < 2; ++i) {
      for (int buf = 0; buf < 2; ++buf) {
        mbar_init(b_sfull(i, buf), 1);
        mbar_init(b_pfull(i, buf), 4);
      }
      mbar_init(b_ofull(i), 1);
      mbar_init(b_pv(i), 1);
    }
    mbar_init(b_done(0), 1);
    mbar_init(b_done(1), 1);
    *abort_flag = 0;
    *start_tile = 0;
    fence_barrier_init();
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  if (warp == 3) {
    tmem_alloc(sb0 + C::OFF_MISC, 512);
    tmem_relinquish();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);

  // ---- this CTA's share of the plan
  pdl_wait();
  ChunkWalk walk;
  walk.n_tiles = __ldcg(prm.n_tiles);
  walk.per_head = 0;
  if (walk.n_tiles >= 0 && walk.n_tiles <= prm.max_tiles) walk.per_head = __ldcg(prm.cum + walk.n_tiles);
  if (!plan_fits(chunk_bounds(prm), walk.n_tiles, walk.per_head)) {
    set_status(COSA_ERR_WORKSPACE);
    walk.n_tiles = 0;
    walk.per_head = 0;
  }
  const long long total = walk.per_head * prm.num_kv_heads;
  const long long quota = (total + gridDim.x - 1) / gridDim.x;
  walk.w = min((long long)blockIdx.x * quota, total);
  walk.w_end = min(walk.w + quota, total);
  walk.hk = 0;
  walk.t = 0;
  if (walk.w < walk.w_end) {
    walk.hk = (int)(walk.w / walk.per_head);
    const long long rem = walk.w - walk.hk * walk.per_head;
    for (int t = tid; t < walk.n_tiles; t += C::THREADS)
      if (__ldcg(prm.cum + t) <= rem && rem < __ldcg(prm.cum + t + 1)) *start_tile = t;
  }
  __syncthreads();
  walk.t = *start_tile;

  const unsigned long long tmo = prm.timeout_ns;
  // bounded waits on an mbarrier phase; false on timeout or abort
  const uint32_t abort_at = sb0 + C::OFF_MISC + 4;
  auto wait = [&](uint32_t bar_addr, uint32_t parity) -> bool {
    return mbar_try_wait(bar_addr, parity) || wait_on(bar_addr, parity, abort_at, tmo);
  };
  auto wait_warp = [&](uint32_t bar_addr, uint32_t parity) -> bool {
    int okl = 1;
    if (lane == 0) okl = wait(bar_addr, parity) ? 1 : 0;
    return __shfl_sync(0xffffffffu, okl, 0) != 0;
  };
  // the same without suspending: for the softmax's wait, which starts its cycle (the MMA warps
  // suspend: their polling took issue slots and, under the power cap, clock)
  auto wait_warp_hot = [&](uint32_t bar_addr, uint32_t parity) -> bool {
    int okl = 1;
    if (lane == 0)
      okl = mbar_test_wait(bar_addr, parity) || wait_on_hot(bar_addr, parity, abort_at, tmo) ? 1 : 0;
    return __shfl_sync(0xffffffffu, okl, 0) != 0;
  };
  const int pshift = 31 - __clz(P);        // P is a power of two
  const int ppb = C::KB >> pshift;         // pages a block, at most 8: one a lane
  // coordinate of page `lane` of block j (-1: outside the pool or given up, read as zeros)
  auto page_coord = [&](const ChunkTile& tile, int hk, int j, int np) -> int {
    if (lane >= np) return 0;
    if ((j * ppb + lane + 1) << pshift <= window_start(prm.mask, tile.pos0)) return -1;
    const int ph = __ldg(prm.page_table + (long long)tile.b * prm.pages_per_seq + j * ppb + lane);
    if (ph < 0 || ph >= prm.num_phys_pages) {
      set_status(COSA_ERR_INVALID_ARG);
      return -1;
    }
    return ph * prm.num_kv_heads + hk;
  };
  auto blk_pages = [&](int kv, int j) {
    return min(ppb, (kv - j * C::KB + P - 1) >> pshift);
  };

  if (warp < 4) {
  if (warp == 0) {
    // ================= Q and K ========================================================
    int it = 0, seg = 0;
    bool ok = true;
    const int qtok_bytes = G * TOK * 128 * (D / 64);
    for (; ok && walk.next(prm); walk.advance(), ++seg) {
      const int nt = (NT == 2 && walk.tile.ntok > TOK) ? 2 : 1;
      if (seg > 0 && !wait_warp(b_qempty, (seg - 1) & 1)) { ok = false; break; }
      if (lane == 0) {
        mbar_arrive_expect_tx(b_qfull, (uint32_t)(nt * qtok_bytes));
        for (int i = 0; i < nt; ++i)
#pragma unroll
          for (int kb = 0; kb < D / 64; ++kb)
            tma_load_3d(sQ + i * C::Q_BYTES + kb * (128 * 128), &tm_q, b_qfull, kb * 64,
                        walk.hk * G, walk.tile.tok0 + i * TOK);
      }
      constexpr int DIR = REV ? -1 : 1;
      int jx = walk.jb + (REV ? walk.nb - 1 : 0);
      int cz = page_coord(walk.tile, walk.hk, jx, blk_pages(walk.tile.kv, jx));
      for (int j = 0; j < walk.nb; ++j, ++it, jx += DIR) {
        const int s = it % C::KS, np = blk_pages(walk.tile.kv, jx);
        int cz_next = 0;
        if (j + 1 < walk.nb)
          cz_next = page_coord(walk.tile, walk.hk, jx + DIR, blk_pages(walk.tile.kv, jx + DIR));
        if (it >= C::KS && !wait_warp(b_kempty(s), ((it / C::KS) - 1) & 1)) { ok = false; break; }
        if (lane == 0) mbar_arrive_expect_tx(b_kfull(s), (uint32_t)(np * P * D * 2));
        __syncwarp();
        if (lane < np)
#pragma unroll
          for (int kb = 0; kb < D / 64; ++kb)
            tma_load_3d(sK + s * C::BLK_BYTES + kb * (C::KB * 128) + lane * (P * 128), &tm_k,
                        b_kfull(s), kb * 64, 0, cz);
        cz = cz_next;
      }
      if (!ok) { ++seg; break; }
    }
    // loads never consumed (abort only) land before the CTA leaves
    if (lane == 0) {
      const uint64_t t0 = globaltimer_ns();
      if (seg > 0) drain_wait(b_qfull, (seg - 1) & 1, t0, tmo);
      for (int x = max(0, it - C::KS); x < it; ++x)
        drain_wait(b_kfull(x % C::KS), (x / C::KS) & 1, t0, tmo);
    }
  } else if (warp == 2) {
    // ================= V ==============================================================
    int it = 0, tails = 0;
    bool ok = true;
    ChunkJoin jn;  // the tile that this share starts and does not finish
    jn.ntok = jn.tok0 = jn.hk = jn.last = 0;
    for (; ok && walk.next(prm); walk.advance()) {
      if (walk.part == 1) {
        jn.tok0 = walk.tile.tok0;
        jn.ntok = walk.tile.ntok;
        jn.hk = walk.hk;
        jn.last = (int)((walk.w + walk.lead + walk.tile.nb - 1) / quota);
      }
      constexpr int DIR = REV ? -1 : 1;
      int jx = walk.jb + (REV ? walk.nb - 1 : 0);
      int cz = page_coord(walk.tile, walk.hk, jx, blk_pages(walk.tile.kv, jx));
      for (int j = 0; j < walk.nb; ++j, ++it, jx += DIR) {
        const int s = it % C::VS, np = blk_pages(walk.tile.kv, jx);
        const int keys = walk.tile.kv - jx * C::KB;
        int cz_next = 0;
        if (j + 1 < walk.nb)
          cz_next = page_coord(walk.tile, walk.hk, jx + DIR, blk_pages(walk.tile.kv, jx + DIR));
        if (it >= C::VS && !wait_warp(b_vempty(s), ((it / C::VS) - 1) & 1)) { ok = false; break; }
        // the MMA reads the keys of whole 16-key steps: those behind the end are zeroed
        const bool tail = keys < C::KB && (keys & 15) != 0;
        const uint32_t full = tail ? b_vtail : b_vfull(s);
        const uint32_t dst = sV + s * C::BLK_BYTES;
        if (lane == 0) mbar_arrive_expect_tx(full, (uint32_t)(np * P * D * 2));
        __syncwarp();
        if (lane < np)
#pragma unroll
          for (int kb = 0; kb < D / 64; ++kb)
            tma_load_3d(dst + kb * (C::KB * 128) + lane * (P * 128), &tm_v, full, kb * 64, 0, cz);
        cz = cz_next;
        if (tail) {
          // (on a timeout here the slot is reported full all the same: the MMA thread leaves
          // through the abort flag)
          const bool have = wait_warp(b_vtail, tails & 1);
          ++tails;
          const int nz = 16 - (keys & 15);
          for (int x = lane; have && x < nz * 8 * (D / 64); x += 32) {
            const int c = x & 7, r = keys + (x >> 3) % nz, kb = (x >> 3) / nz;
            st_shared_v4(dst + kb * (C::KB * 128) + r * 128 + c * 16, 0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(b_vfull(s));
          if (!have) { ++it; ok = false; break; }
        }
      }
      if (!ok) break;
    }
    if (lane == 0) {
      ChunkJoin* o = prm.joins + blockIdx.x;
      o->ntok = jn.ntok;
      o->tok0 = jn.tok0;
      o->hk = jn.hk;
      o->last = jn.last;
      const uint64_t t0 = globaltimer_ns();
      for (int x = max(0, it - C::VS); x < it; ++x)
        drain_wait(b_vfull(x % C::VS), (x / C::VS) & 1, t0, tmo);
      if (tails > 0) drain_wait(b_vtail, (tails - 1) & 1, t0, tmo);
    }
  } else if (warp == 1 || (NT == 2 && warp == 3)) {
    // ================= MMA issue of tile i ============================================
    // The whole warp walks, one elected lane issues: with warp-uniform control flow the
    // operands stay in uniform registers.  Issued from a branch that one lane takes, every
    // MMA first moved its five operands there, and cost 85-140 cycles instead of 64.  A warp a
    // tile: the barriers and commits of one cost as much as its products take (1.4 k of 3.4 k
    // cycles a half block of two tiles when one warp did both).
    const int i = warp >> 1;
    const uint32_t lead = elect_one();
    constexpr uint32_t ID_QK = idesc_bf16_f32(128, 64, 0);
    constexpr uint32_t ID_PV = idesc_bf16_f32(128, D, 1);
    const uint64_t dq = smem_desc_sw128(sQ + i * C::Q_BYTES, 16, 1024);
    const uint64_t dk = smem_desc_sw128(sK, 16, 1024);
    const uint64_t dv = smem_desc_sw128(sV, C::KB * 128, 1024);
    const uint32_t t_s = tmem + i * 128, t_o = tmem + C::COL_O + i * D;
    int it = 0, seg = 0, cnt = 0;  // blocks of the CTA, segments, half blocks of the tile
    bool ok = true;
    auto all = [&](bool v) { return __all_sync(0xffffffffu, v) != 0; };
    for (; ok; ++seg) {
      if (!all(walk.next(prm))) break;
      const int nb = __shfl_sync(0xffffffffu, walk.nb, 0);
      const int keys0 = __shfl_sync(0xffffffffu, walk.tile.kv - walk.jb * C::KB, 0);
      if (!all(wait(b_qfull, seg & 1))) { ok = false; break; }
      if (i == 1 && all(walk.tile.ntok <= TOK)) {
        // no second tile here: hand every slot on once it has been filled (not before: an
        // arrival ahead of the slot's phase would count for an earlier one)
        if (lane == 0) mbar_arrive(b_qempty);
        for (int x = it; ok && x < it + nb; ++x) {
          ok = all(wait(b_kfull(x % C::KS), (x / C::KS) & 1));
          if (ok && lane == 0) mbar_arrive(b_kempty(x % C::KS));
          ok = ok && all(wait(b_vfull(x % C::VS), (x / C::VS) & 1));
          if (ok && lane == 0) mbar_arrive(b_vempty(x % C::VS));
        }
      } else {
        const int ns = half_blocks(nb, keys0);  // 2 nb, or one less
        // half block of step n, its block's place in the ring, whether the step is the first or the
        // last on that block
        auto half = [&](int n) { return REV ? ns - 1 - n : n; };
        auto block = [&](int n) { return it + (REV ? nb - 1 - (half(n) >> 1) : n >> 1); };
        auto opens = [&](int n) { return REV ? n == 0 || (half(n) & 1) : !(n & 1); };
        auto closes = [&](int n) { return REV ? !(half(n) & 1) : (n & 1) || n + 1 == ns; };
        // Step n: S(n) = Q K(n)^T, then O += P(n - 1) V(n - 1): the scores of a half block come in
        // under the softmax of the one before
        for (int n = 0; n <= ns; ++n) {
          if (n < ns) {
            const int x = block(n), s = x % C::KS, buf = (cnt + n) & 1;
            if (opens(n)) {
              if (!all(wait(b_kfull(s), (x / C::KS) & 1))) { ok = false; break; }
              tc_fence_after();
            }
            const uint64_t dks = dk + (((uint32_t)s * C::BLK_BYTES + (half(n) & 1) * (64 * 128)) >> 4);
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              mma_bf16_ss_if(lead, t_s + buf * 64, dq + (((k >> 2) * (128 * 128) + (k & 3) * 32) >> 4),
                             dks + (((k >> 2) * (C::KB * 128) + (k & 3) * 32) >> 4), ID_QK,
                             k > 0 ? 1u : 0u);
            mma_commit_if(lead, b_sfull(i, buf));
            if (closes(n)) mma_commit_if(lead, b_kempty(s));
            if (n + 1 == ns) mma_commit_if(lead, b_qempty);
          }
          if (n > 0) {
            const int m = n - 1, x = block(m), s = x % C::VS, c = cnt + m, buf = c & 1;
            if (opens(m) && !all(wait(b_vfull(s), (x / C::VS) & 1))) { ok = false; break; }
            if (!all(wait(b_pfull(i, buf), (c >> 1) & 1))) { ok = false; break; }
            tc_fence_after();
            const int keys = keys0 - half(m) * 64;
            const uint64_t dvs = dv + (((uint32_t)s * C::BLK_BYTES + (half(m) & 1) * (64 * 128)) >> 4);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_bf16_ts_if(k * 16 < keys ? lead : 0u, t_o, t_s + buf * 64 + k * 8,
                             dvs + ((k * 16 * 128) >> 4), ID_PV, (m > 0 || k > 0) ? 1u : 0u);
            mma_commit_if(lead, b_pv(i));
            if (n == ns) mma_commit_if(lead, b_ofull(i));
            if (closes(m)) mma_commit_if(lead, b_vempty(s));
          }
        }
        cnt += ns;
      }
      if (!ok) break;
      it += nb;
      walk.advance();
    }
    // every issued MMA completes before teardown frees TMEM
    mma_commit_if(lead, b_done(i));
    const uint64_t t0 = globaltimer_ns();
    if (lane == 0) drain_wait(b_done(i), 0, t0, tmo);
  }
  } else {
    // ================= softmax of tile i, one row per thread ==========================
    const int i = (warp - 4) >> 2, q4 = warp & 3, row = q4 * 32 + lane;
    const uint32_t t_row = tmem + ((uint32_t)(q4 * 32) << 16);
    const uint32_t t_o = t_row + C::COL_O + i * D;
    const int row_tok = row / G, row_g = row - row_tok * G;
    int cnt = 0, nseg = 0;  // half blocks and segments of this tile
    bool ok = true;
    for (; ok && walk.next(prm); walk.advance()) {
      const int ntok = walk.tile.ntok - i * TOK;
      if (ntok <= 0) continue;  // a lone tile: the second group of warps has no rows
      const int token = walk.tile.tok0 + i * TOK + row_tok;
      const int pos = walk.tile.pos0 + i * TOK + row_tok;
      const bool row_valid = row_tok < min(TOK, ntok);
      const int head = walk.hk * G + row_g;
      int lo = 0, hi = INT_MAX;  // rows without a token need no mask: their result goes nowhere
      float slope = 0.f;
      if (row_valid) {
        token_range(prm.mask, token, pos, walk.tile.kv, walk.tile.prefix, lo, hi);
        if (BIAS) slope = __ldg(prm.slopes + head) * 1.4426950408889634f;
      }
      const bool warp_works = __any_sync(0xffffffffu, row_valid);
      // the keys that every row of the warp sees: [alo, ahi]
      const int alo = __reduce_max_sync(0xffffffffu, lo), ahi = __reduce_min_sync(0xffffffffu, hi);
      float m_ref = -INFINITY, l = 0.f;
      const int ns = half_blocks(walk.nb, walk.tile.kv - walk.jb * C::KB);
      for (int n = 0; n < ns; ++n, ++cnt) {
        const int buf = cnt & 1;
        const uint32_t t_s = t_row + i * 128 + buf * 64;
        if (!wait_warp_hot(b_sfull(i, buf), (cnt >> 1) & 1)) { ok = false; break; }
        tc_fence_after();
        const int key0 = walk.jb * C::KB + (REV ? ns - 1 - n : n) * 64;
        if (warp_works) {
          uint32_t sc[64];
          tmem_ld64(t_s, sc);
          const bool plain = alo <= key0 && ahi >= key0 + 63;
          // ---- scores in log2 units where they are shaped (otherwise the scale goes into the
          // exponent below), the unseen ones -inf
          if (CAP) {
            float far = 0.f;
#pragma unroll
            for (int e = 0; e < 64; e += 2)
              far = fmax3f(far, fabsf(__uint_as_float(sc[e])), fabsf(__uint_as_float(sc[e + 1])));
            auto shape = [&](auto form_tag) {
#pragma unroll
              for (int e = 0; e < 64; e += 2) {
                float x0, x1;
                unpack2(score2_log2<decltype(form_tag)::value>(
                            prm.score, pack2(__uint_as_float(sc[e]), __uint_as_float(sc[e + 1])),
                            both(0.f)),
                        x0, x1);
                sc[e] = __float_as_uint(x0);
                sc[e + 1] = __float_as_uint(x1);
              }
            };
            if (__all_sync(0xffffffffu, !row_valid || far <= prm.score.lim))
              shape(std::integral_constant<CapForm, CAP_NEAR>{});
            else
              shape(std::integral_constant<CapForm, CAP>{});
          }
          if (BIAS) {
            const f32x2 d0 = both((float)(key0 - pos)), mul = both(CAP ? 1.f : prm.score.a);
#pragma unroll
            for (int e = 0; e < 64; e += 2) {
              float a0, a1;
              unpack2(add2(d0, pack2((float)e, (float)(e + 1))), a0, a1);
              const f32x2 x = mul2(pack2(__uint_as_float(sc[e]), __uint_as_float(sc[e + 1])), mul);
              unpack2(fma2(both(-slope), pack2(fabsf(a0), fabsf(a1)), x), a0, a1);
              sc[e] = __float_as_uint(a0);
              sc[e + 1] = __float_as_uint(a1);
            }
          }
          if (!plain) {
            const int r0 = max(lo - key0, 0), r1 = min(hi - key0, 63);  // one bit a column: seen
            const uint64_t bits = r0 > r1 ? 0ull : (~0ull << r0) & (~0ull >> (63 - r1));
            const uint32_t b0 = (uint32_t)bits, b1 = (uint32_t)(bits >> 32);
#pragma unroll
            for (int e = 0; e < 64; ++e)
              if (!(((e < 32 ? b0 : b1) >> (e & 31)) & 1u)) sc[e] = 0xff800000u;  // -inf
          }
          // ---- row max
          float a[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) a[e] = fmaxf(__uint_as_float(sc[e]), __uint_as_float(sc[e + 4]));
#pragma unroll
          for (int e = 8; e < 64; e += 8)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              a[x] = fmax3f(a[x], __uint_as_float(sc[e + 2 * x]), __uint_as_float(sc[e + 2 * x + 1]));
          const float m_loc = fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3])) * (CAP || BIAS ? 1.f : prm.score.a);
          const bool resc = m_loc > m_ref + C::kRescale;
          if (__any_sync(0xffffffffu, resc)) {
            // a bias still rises on the way from a prefix's later keys down to the row's own
            // position: the base takes that rise in advance (up to 2^60, which P, l and O have
            // room for)
            const float m_new =
                BIAS ? m_loc + fminf(fmaxf(slope * (float)(key0 - pos), 0.f), 60.f) : m_loc;
            if (n > 0) {  // O is at rest once the previous half block's product is done
              if (!wait_warp(b_pv(i), (cnt - 1) & 1)) { ok = false; break; }
              tc_fence_after();
              const float alpha = resc ? ex2_approx(m_ref - m_new) : 1.f;
#pragma unroll 1
              for (int k = 0; k < D / 32; ++k) {
                uint32_t r[32];
                tmem_ld32(t_o + k * 32, r);
#pragma unroll
                for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * alpha);
                tmem_st32(t_o + k * 32, r);
              }
              l *= alpha;
            }
            if (resc) m_ref = m_new;
          }
          // ---- P = 2^(score - m_ref) as bf16 pairs over the first half of the S columns
          const float nb = m_ref == -INFINITY ? 0.f : -m_ref;
          const f32x2 nb2 = both(nb), mul = both(prm.score.a);
          f32x2 sum[2] = {both(0.f), both(0.f)};
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              f32x2 x = pack2(__uint_as_float(sc[32 * c + 2 * e]), __uint_as_float(sc[32 * c + 2 * e + 1]));
              x = (CAP || BIAS) ? add2(x, nb2) : fma2(x, mul, nb2);
              float x0, x1;
              unpack2(x, x0, x1);
              const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
              sum[e & 1] = add2(sum[e & 1], pack2(p0, p1));
              __nv_bfloat162 v2 = __floats2bfloat162_rn(p0, p1);
              w[e] = *reinterpret_cast<uint32_t*>(&v2);
            }
            tmem_st16(t_s + c * 16, w);
          }
          float t0, t1;
          unpack2(add2(sum[0], sum[1]), t0, t1);
          l += t0 + t1;
          tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        // one barrier a buffer: a warp without rows may be a half block ahead of the others, and
        // its arrival must not count for theirs
        if (lane == 0) mbar_arrive(b_pfull(i, buf));
      }
      // ---- epilogue: O / l, or the partial rows of a tile cut between CTAs
      const bool have = ok && wait_warp(b_ofull(i), nseg & 1);
      ++nseg;
      if (!have) ok = false;
      if (!have || !warp_works) continue;
      tc_fence_after();
      const bool whole = walk.part < 0;
      const float inv = row_scale(l);
      const long long r_out = (long long)token * prm.num_q_heads + head;
      const long long r_part =
          (long long)(2 * blockIdx.x + (walk.part > 0 ? 1 : 0)) * prm.part_rows + i * 128 + row;
#pragma unroll 1
      for (int k = 0; k < D / 32; ++k) {
        uint32_t r[32];
        tmem_ld32(t_o + k * 32, r);
        if (!row_valid) continue;
        if (whole) {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            __nv_bfloat162 v2 = __floats2bfloat162_rn(__uint_as_float(r[2 * e]) * inv,
                                                      __uint_as_float(r[2 * e + 1]) * inv);
            w[e] = *reinterpret_cast<uint32_t*>(&v2);
          }
          uint4* dst = reinterpret_cast<uint4*>(prm.out + r_out * D + k * 32);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            dst[e] = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
        } else {
          uint4* dst = reinterpret_cast<uint4*>(prm.part_o + r_part * D + k * 32);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            dst[e] = make_uint4(r[4 * e], r[4 * e + 1], r[4 * e + 2], r[4 * e + 3]);
        }
      }
      if (row_valid) {
        if (whole) {
          if (prm.lse)
            prm.lse[r_out] = row_lse(m_ref, l);
        } else {
          prm.part_ml[r_part] = make_float2(m_ref, l);
        }
      }
      tc_fence_before();
    }
  }

  // ---- teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 3) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---- join of the tiles that were cut ----------------------------------------------------
constexpr int JOIN_WARPS = 8;
constexpr int JOIN_ROWS = 4;  // rows of a warp, JOIN_WARPS apart

// grid (NUM_SMS, groups of JOIN_WARPS * JOIN_ROWS rows).  All latency: the loads of all a warp's
// rows (a prompt's tile: two or three parts each) or of 16 parts of one row (a decode step's)
// are in flight together.
template <int D>
__global__ void __launch_bounds__(32 * JOIN_WARPS) chunk_combine_kernel(const ChunkAttnParams p) {
  constexpr int EPL = D / 32;  // floats a lane
  pdl_wait();
  const int4 jn = __ldcg(reinterpret_cast<const int4*>(p.joins + blockIdx.x));
  if (!jn.x) return;  // ntok = 0: this CTA cut no tile
  const int last = __ldcg(&p.joins[blockIdx.x].last);
  if (!join_fits(chunk_bounds(p), jn.x, jn.y, jn.z, blockIdx.x, last)) {
    set_status(COSA_ERR_WORKSPACE);
    return;
  }
  const int lane = threadIdx.x & 31, G = p.group;
  const int c0 = blockIdx.x, n = last - c0 + 1;
  const int row0 = blockIdx.y * (JOIN_WARPS * JOIN_ROWS) + (threadIdx.x >> 5);
  auto tok_of = [&](int row) { return (row >> 7) * p.tile_tokens + (row & 127) / G; };
  auto real = [&](int row) {
    return row < p.part_rows && (row & 127) < p.tile_tokens * G && tok_of(row) < jn.x;
  };
  auto slot = [&](int s, int row) {
    return (long long)(s == 0 ? 2 * c0 + 1 : 2 * (c0 + s)) * p.part_rows + row;
  };
  auto load = [&](long long at, float* v) {
    const float* src = p.part_o + at * D + lane * EPL;
    if (EPL == 4) {
      const float4 t = __ldcg(reinterpret_cast<const float4*>(src));
      v[0] = t.x, v[1] = t.y, v[EPL - 2] = t.z, v[EPL - 1] = t.w;
    } else {
      const float2 t = __ldcg(reinterpret_cast<const float2*>(src));
      v[0] = t.x, v[1] = t.y;
    }
  };
  auto finish = [&](int row, float m, float l, const float* o) {
    const float inv = row_scale(l);
    const long long out =
        (long long)(jn.y + tok_of(row)) * p.num_q_heads + jn.z * G + (row & 127) % G;
#pragma unroll
    for (int e = 0; e < EPL; e += 2)
      *reinterpret_cast<__nv_bfloat162*>(p.out + out * D + lane * EPL + e) =
          __floats2bfloat162_rn(o[e] * inv, o[e + 1] * inv);
    if (p.lse && lane == 0)
      p.lse[out] = row_lse(m, l);
  };
  if (n <= 3) {
    float2 ml[JOIN_ROWS][3];
    float v[JOIN_ROWS][3][EPL];
#pragma unroll
    for (int k = 0; k < JOIN_ROWS; ++k)
#pragma unroll
      for (int s = 0; s < 3; ++s) {
        ml[k][s] = make_float2(-INFINITY, 0.f);
        if (s < n && real(row0 + k * JOIN_WARPS)) {
          const long long at = slot(s, row0 + k * JOIN_WARPS);
          ml[k][s] = __ldcg(p.part_ml + at);
          load(at, v[k][s]);
        }
      }
#pragma unroll
    for (int k = 0; k < JOIN_ROWS; ++k) {
      if (!real(row0 + k * JOIN_WARPS)) continue;
      const float m = fmaxf(fmaxf(ml[k][0].x, ml[k][1].x), ml[k][2].x);
      float l = 0.f, o[EPL];
#pragma unroll
      for (int e = 0; e < EPL; ++e) o[e] = 0.f;
#pragma unroll
      for (int s = 0; s < 3; ++s)
        if (ml[k][s].y != 0.f) {  // (a part without keys has no weight, whatever its O holds)
          const float w = tc::ex2_approx(ml[k][s].x - m);
          l = fmaf(w, ml[k][s].y, l);
#pragma unroll
          for (int e = 0; e < EPL; ++e) o[e] = fmaf(w, v[k][s][e], o[e]);
        }
      finish(row0 + k * JOIN_WARPS, m, l, o);
    }
    return;
  }
#pragma unroll 1
  for (int k = 0; k < JOIN_ROWS; ++k) {
    const int row = row0 + k * JOIN_WARPS;
    if (!real(row)) continue;
    float l = 0.f, m = -INFINITY, o[EPL];
#pragma unroll
    for (int e = 0; e < EPL; ++e) o[e] = 0.f;
    // 32 parts at a time: a lane holds one part's base and sum
    for (int s0 = 0; s0 < n; s0 += 32) {
      const int cnt = min(32, n - s0);
      const float2 ml =
          lane < cnt ? __ldcg(p.part_ml + slot(s0 + lane, row)) : make_float2(-INFINITY, 0.f);
      if (!__any_sync(0xffffffffu, ml.y != 0.f)) continue;
      const float mx = fmaxf(m, warp_max(ml.x));
      const float back = tc::ex2_approx(m - mx);  // (from -inf: 0)
      const float w = ml.y != 0.f ? tc::ex2_approx(ml.x - mx) : 0.f;
      float part = w * ml.y;
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) part += __shfl_xor_sync(0xffffffffu, part, x);
      l = fmaf(l, back, part);
      m = mx;
#pragma unroll
      for (int e = 0; e < EPL; ++e) o[e] *= back;
      for (int s = 0; s < cnt; s += 16) {
        float v[16][EPL];
#pragma unroll
        for (int x = 0; x < 16; ++x) load(slot(s0 + min(s + x, cnt - 1), row), v[x]);
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          const float ws = __shfl_sync(0xffffffffu, w, min(s + x, 31));
          if (s + x < cnt && ws != 0.f)
#pragma unroll
            for (int e = 0; e < EPL; ++e) o[e] = fmaf(ws, v[x][e], o[e]);
        }
      }
    }
    finish(row, m, l, o);
  }
}

}  // namespace cosa
