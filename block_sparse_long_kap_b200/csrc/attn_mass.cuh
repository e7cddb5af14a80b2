// Accumulated attention mass of the cached keys (cosa_attention_mass):
//   mass[k] = (k is older than the chunk ? decay * mass[k] : 0)
//             + sum over rows (token, head of the group) of e^(s - lse_row).
// The softmax normaliser is known (the lse that the attention left), so no running maximum
// is needed and the sum over rows is a plain column sum of the weights.  The product is
// taken transposed, S^T = K Q^T: a thread owns one key (its TMEM lane) and adds the weights
// of all rows in registers, in a fixed order, without atomics or shuffles.
//
// 148 CTAs, one per SM, share the pairs of 128-key blocks of all (KV head, sequence)s.  With at
// most two tiles of 128 rows a chunk (HELD: decode steps, the last tokens of a prompt) a CTA
// takes a contiguous run of pairs, and the tiles' Q and row constants stay in shared memory
// while the sequence and head do; else every 148th pair (under a causal mask the late pairs
// of a long chunk see fewer tiles; striping evens that out), past which the tiles stream, each
// serving both blocks.
//   warp 0  K loads      warp 2  Q loads
//   warp 1  MMA issue    warp 3  TMEM allocation
//   warps 4-7 / 8-11     weights and sums of the first / second block of a pair; two S
//                        buffers each, so the next tile's product runs under this one's
//                        exponentials.
// Bound by the K bytes for a few rows: a decode step of eight sequences of up to 16K keys (218 MB)
// takes 43 us, 0.78 of a copy's rate, the rest is the start of the stream and the last pair's
// way through.  For many rows by the exponentials (16 a cycle and SM): the last 64 tokens of 32
// heads on 64K keys are 134 M of them, 30 us, and take 62 us (special-function unit 50 % busy,
// tensor core 25 %); a quarter of them as a polynomial on the FMA pipe gave nothing.  All 2,048 tokens of a
// chunk on 8K keys (470 M of them, 103 us at the unit's rate) take 257 us, the unit 56 % busy.
// A softmax warp whose wait ran out keeps meeting the others at their named barrier, so that
// none waits there for good.
#pragma once

#include <type_traits>

#include "chunk_common.cuh"

namespace cosa {

struct MassParams {
  ChunkSeqs seqs;
  ChunkMask mask;
  const int32_t* page_table;
  const float* slopes;
  const float* lse;  // [total_q][H_q]
  float* mass;       // [B][H_kv][mass_stride]
  long long mass_stride;
  int num_q_heads, num_kv_heads, group, page_size, pages_per_seq, num_phys_pages;
  int tile_tokens;   // 128 / G
  int box_tokens;    // tokens a Q load brings (fewer where no chunk has as many)
  int last_q;        // 0: all
  int cols;          // columns of the product: rows of a tile rounded up to 16
  int held;          // no chunk has more than two tiles
  float decay;
  ScoreShape score;
  unsigned long long timeout_ns;
};

// A tile's rows as the softmax reads them: constants in arrays of 128.
struct MassRows {
  float c[128];    // -lse in log2 units
  int lo[128], hi[128];
  float slope[128], tok[128];  // tok: counted from the first row's, as the keys are
                               // (a float does not hold every position past 2^24)
};

template <int D>
struct MassCfg {
  static constexpr int KB = 128;
  static constexpr int THREADS = 384;
  static constexpr uint32_t BLK_BYTES = KB * D * 2;
  static constexpr int KS = 4;  // K slots
  static constexpr int QS = 2;  // Q slots
  static constexpr uint32_t OFF_K = 0;
  static constexpr uint32_t OFF_Q = OFF_K + KS * BLK_BYTES;
  static constexpr uint32_t OFF_ROW = OFF_Q + QS * BLK_BYTES;  // [2 groups][2 buffers]
  static constexpr uint32_t OFF_BAR = OFF_ROW + 4 * sizeof(MassRows);
  static constexpr int NBAR = 2 * KS + 2 * QS + 8 + 1;  // k, q full / empty; s full / free [4]; done
  static constexpr uint32_t OFF_MISC = (OFF_BAR + NBAR * 8 + 15) & ~15u;
  static constexpr uint32_t OFF_CUM = OFF_MISC + 32;  // pairs before each sequence [B + 1]
  static constexpr uint32_t smem(int batch) { return OFF_CUM + (batch + 1) * 4 + 1024; }
  static_assert(OFF_CUM + (CHUNK_MAX_BATCH + 1) * 4 + 1024 <= 227 * 1024, "shared memory budget");
};

template <int D, CapForm CAP, bool BIAS>  // CAP: none, or each where not all are near
__global__ void __launch_bounds__(384, 1)
    attn_mass_kernel(const __grid_constant__ CUtensorMap tm_q,
                     const __grid_constant__ CUtensorMap tm_k, const MassParams prm) {
  using C = MassCfg<D>;
  using namespace tc;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int G = prm.group, TOK = prm.tile_tokens, P = prm.page_size, B = prm.seqs.batch;
  if (__syncthreads_or(*(volatile int*)&g_status == COSA_ERR_TIMEOUT)) return;

  extern __shared__ uint8_t smem_raw[];
  const uint32_t sraw = static_cast<uint32_t>(__cvta_generic_to_shared(smem_raw));
  const uint32_t sb0 = (sraw + 1023u) & ~1023u;
  uint8_t* sg = smem_raw + (sb0 - sraw);
  const uint32_t sK = sb0 + C::OFF_K, sQ = sb0 + C::OFF_Q, bar = sb0 + C::OFF_BAR;
  auto b_kfull = [&](int s) { return bar + 8u * s; };
  auto b_kempty = [&](int s) { return bar + 8u * (C::KS + s); };
  auto b_qfull = [&](int s) { return bar + 8u * (2 * C::KS + s); };
  auto b_qempty = [&](int s) { return bar + 8u * (2 * C::KS + C::QS + s); };
  auto b_sfull = [&](int s) { return bar + 8u * (2 * C::KS + 2 * C::QS + s); };
  auto b_sfree = [&](int s) { return bar + 8u * (2 * C::KS + 2 * C::QS + 4 + s); };
  const uint32_t b_done = bar + 8u * (C::NBAR - 1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sg + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sg + C::OFF_MISC + 4);
  int* scan_s = reinterpret_cast<int*>(sg + C::OFF_ROW);  // (before the rows are needed)
  int* cum = reinterpret_cast<int*>(sg + C::OFF_CUM);

  if (tid == 0) {
    for (int s = 0; s < C::KS; ++s) { mbar_init(b_kfull(s), 1); mbar_init(b_kempty(s), 1); }
    for (int s = 0; s < C::QS; ++s) { mbar_init(b_qfull(s), 1); mbar_init(b_qempty(s), 1); }
    for (int s = 0; s < 4; ++s) { mbar_init(b_sfull(s), 1); mbar_init(b_sfree(s), 4); }
    mbar_init(b_done, 1);
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
  }
  if (warp == 3) {
    tmem_alloc(sb0 + C::OFF_MISC, 512);
    tmem_relinquish();
  }
  // rows of a Q slot that no load writes (128 is not a multiple of G) are zero: their product
  // has to be finite to vanish under a weight of zero
  const int r0 = G * prm.box_tokens, nr = prm.cols - r0;
  for (int x = tid; x < C::QS * (D / 64) * nr * 8; x += C::THREADS) {
    const int piece = x & 7, r = r0 + (x >> 3) % nr, h = (x >> 3) / nr;  // h: slot and half
    st_shared_v4(sQ + h * (128 * 128) + r * 128 + piece * 16, 0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
  // pairs of key blocks before each sequence
  int base = 0;
  for (int b0 = 0; b0 < B; b0 += C::THREADS) {
    const int b = b0 + tid;
    int n = 0;
    if (b < B) {
      const ChunkSeq s = chunk_seq(prm.seqs, b);
      if (s.ok) n = (s.kv + 2 * C::KB - 1) / (2 * C::KB);
    }
    int inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) scan_s[warp] = inc;
    __syncthreads();
    int before = 0, total = 0;
    for (int w = 0; w < C::THREADS / 32; ++w) {
      const int v = scan_s[w];
      if (w < warp) before += v;
      total += v;
    }
    if (b < B) cum[b] = base + before + inc - n;
    base += total;
    __syncthreads();
  }
  if (tid == 0) cum[B] = base;
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  const long long npairs = (long long)base * prm.num_kv_heads;

  // ---- this CTA's pairs; every role walks by itself
  const long long share = (npairs + gridDim.x - 1) / gridDim.x;
  const long long first = prm.held ? blockIdx.x * share : blockIdx.x;
  const int step = prm.held ? 1 : gridDim.x;
  const long long last = prm.held ? min(first + share, npairs) : npairs;
  struct Walk {
    long long p;
    int w, hk, b;                  // pair within the head, head, sequence
    int from, to;                  // the sequence's pairs
    bool fresh;                    // another head or sequence than the pair before
    ChunkSeq seq;
    int tok0, ntok, pos0, prefix, ntile;  // rows: the last tokens of the chunk
    int kb, nw;                    // first block, blocks (1 or 2)
    int t0, t1;                    // tiles that may see a key of the pair
  };
  auto find = [&](Walk& r) {
    r.fresh = false;
    if (r.w < r.from || r.w >= r.to) {
      r.fresh = true;
      while (r.w >= base) {
        r.w -= base;
        ++r.hk;
      }
      int lo = 0, hi = B - 1;  // the last sequence whose first pair is at or before w
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cum[mid] <= r.w) lo = mid;
        else hi = mid - 1;
      }
      r.b = lo;
      r.from = cum[lo];
      r.to = cum[lo + 1];
      r.seq = chunk_seq(prm.seqs, lo);
      const int skip = (prm.last_q > 0 && prm.last_q < r.seq.q_len) ? r.seq.q_len - prm.last_q : 0;
      r.tok0 = r.seq.q0 + skip;
      r.ntok = r.seq.q_len - skip;
      r.pos0 = r.seq.kv - r.ntok;
      r.prefix = prm.mask.prefix_len ? __ldg(prm.mask.prefix_len + lo) : 0;
      r.ntile = (r.ntok + TOK - 1) / TOK;
    }
    r.kb = 2 * (r.w - r.from);
    r.nw = min(2, (r.seq.kv + C::KB - 1) / C::KB - r.kb);
    r.t0 = 0;
    r.t1 = r.ntile;
    const int key0 = r.kb * C::KB, key1 = key0 + r.nw * C::KB - 1;
    if (r.prefix <= key0 && key0 > r.pos0) r.t0 = min((key0 - r.pos0) / TOK, r.ntile);
    if (prm.mask.window > 0) {  // tiles from the first token on that no longer sees key1
      const long long i = (long long)key1 + prm.mask.window - r.pos0;
      r.t1 = i <= 0 ? 0 : (int)min((i + TOK - 1) / TOK, (long long)r.ntile);
    }
    if (r.t1 < r.t0) r.t1 = r.t0;
  };
  Walk r;
  r.p = first;
  r.hk = 0;
  r.w = r.from = r.to = 0;
  if (first < last) {
    r.hk = (int)(first / base);
    r.w = (int)(first - (long long)r.hk * base);
    find(r);
  }
  auto next = [&]() {
    r.p += step;
    r.w += step;
    if (r.p < last) find(r);
  };

  const unsigned long long tmo = prm.timeout_ns;
  const uint32_t abort_at = sb0 + C::OFF_MISC + 4;
  auto wait = [&](uint32_t bar_addr, uint32_t parity) -> bool {
    return mbar_try_wait(bar_addr, parity) || wait_on(bar_addr, parity, abort_at, tmo);
  };
  auto wait_warp = [&](uint32_t bar_addr, uint32_t parity) -> bool {
    int okl = 1;
    if (lane == 0) okl = wait(bar_addr, parity) ? 1 : 0;
    return __shfl_sync(0xffffffffu, okl, 0) != 0;
  };
  // A loader that is ahead waits for whole pairs: a K slot comes free once all the chunk's tiles have
  // passed it (a tile takes a pair one to two microseconds; half a million of them were past the
  // limit), held tiles once the CTA's pairs of their sequence are through.  Its limit grows with that.
  auto wait_long = [&](uint32_t bar_addr, uint32_t parity, long long steps) -> bool {
    return mbar_try_wait(bar_addr, parity) || wait_on(bar_addr, parity, abort_at, tmo + 20000ull * steps);
  };
  auto all = [&](bool v) { return __all_sync(0xffffffffu, v) != 0; };

  if (warp == 0) {
    // ================= K ==============================================================
    const int pshift = 31 - __clz(P), ppb = C::KB >> pshift;
    const int most_tiles = (prm.seqs.max_q + TOK - 1) / TOK;
    int x = 0;  // blocks loaded
    bool ok = true;
    for (; ok && r.p < last; next()) {
      if (r.t0 == r.t1) continue;  // nobody sees the pair
      for (int w = 0; w < r.nw; ++w) {
        const int kb = r.kb + w;
        const int s = x % C::KS, np = min(ppb, (r.seq.kv - kb * C::KB + P - 1) >> pshift);
        int cz = 0;
        if (lane < np) {
          cz = -1;
          if ((kb * ppb + lane + 1) << pshift > window_start(prm.mask, r.pos0)) {
            const int ph = __ldg(prm.page_table + (long long)r.b * prm.pages_per_seq + kb * ppb + lane);
            if (ph >= 0 && ph < prm.num_phys_pages) cz = ph * prm.num_kv_heads + r.hk;
            else set_status(COSA_ERR_INVALID_ARG);
          }
        }
        if (x >= C::KS) {
          int free = 1;
          if (lane == 0) free = wait_long(b_kempty(s), ((x / C::KS) - 1) & 1, prm.held ? 0 : most_tiles) ? 1 : 0;
          if (!__shfl_sync(0xffffffffu, free, 0)) { ok = false; break; }
        }
        if (lane == 0) mbar_arrive_expect_tx(b_kfull(s), (uint32_t)(np * P * D * 2));
        __syncwarp();
        if (lane < np)
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
            tma_load_3d(sK + s * C::BLK_BYTES + h * (C::KB * 128) + lane * (P * 128), &tm_k,
                        b_kfull(s), h * 64, 0, cz);
        ++x;
      }
    }
    if (lane == 0) {
      const uint64_t t0 = globaltimer_ns();
      for (int y = max(0, x - C::KS); y < x; ++y)
        drain_wait(b_kfull(y % C::KS), (y / C::KS) & 1, t0, tmo);
    }
  } else if (warp == 2) {
    if (lane == 0) {
      // ================= Q ============================================================
      int x = 0;
      bool ok = true;
      const uint32_t bytes = (uint32_t)(G * prm.box_tokens * 128 * (D / 64));
      for (; ok && r.p < last; next()) {
        // held: both slots at once (the second tile may be empty: loaded all the same)
        if (prm.held && !r.fresh) continue;
        const int ta = prm.held ? 0 : r.t0, tb = prm.held ? C::QS : r.t1;
        for (int t = ta; t < tb; ++t) {
          const int s = x % C::QS;
          if (x >= C::QS && !wait_long(b_qempty(s), ((x / C::QS) - 1) & 1, prm.held ? share : 0)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(b_qfull(s), bytes);
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
            tma_load_3d(sQ + s * C::BLK_BYTES + h * (128 * 128), &tm_q, b_qfull(s), h * 64,
                        r.hk * G, r.tok0 + t * TOK);
          ++x;
        }
      }
      const uint64_t t0 = globaltimer_ns();
      for (int y = max(0, x - C::QS); y < x; ++y)
        drain_wait(b_qfull(y % C::QS), (y / C::QS) & 1, t0, tmo);
    }
  } else if (warp == 1) {
    // ================= MMA issue: S^T = K Q^T (the whole warp walks, one lane issues) ====
    const uint32_t lead = elect_one();
    const uint32_t id = idesc_bf16_f32(128, prm.cols, 0);
    const uint64_t dq = smem_desc_sw128(sQ, 16, 1024);
    const uint64_t dk = smem_desc_sw128(sK, 16, 1024);
    int xk = 0, xq = 0, n0 = 0, n1 = 0;  // blocks and tiles taken, products of each group
    bool ok = true;
    for (; ok && r.p < last; next()) {
      const int t0 = __shfl_sync(0xffffffffu, r.t0, 0), t1 = __shfl_sync(0xffffffffu, r.t1, 0);
      const int nw = __shfl_sync(0xffffffffu, r.nw, 0);
      if (prm.held && all(r.fresh)) {
        if (xq > 0)
          for (int s = 0; s < C::QS; ++s) mma_commit_if(lead, b_qempty(s));
        for (int s = 0; ok && s < C::QS; ++s) ok = all(wait(b_qfull(s), (xq / C::QS) & 1));
        xq += C::QS;
      }
      if (t0 == t1) continue;
      for (int t = t0; ok && t < t1; ++t) {
        const int qs = prm.held ? t : xq % C::QS;
        if (!prm.held) {
          ok = all(wait(b_qfull(qs), (xq / C::QS) & 1));
          ++xq;
        }
#pragma unroll 1
        for (int w = 0; ok && w < nw; ++w) {
          const int ks = (xk + w) % C::KS, n = w ? n1 : n0, sbuf = 2 * w + (n & 1);
          if (t == t0 && !all(wait(b_kfull(ks), ((xk + w) / C::KS) & 1))) { ok = false; break; }
          if (n >= 2 && !all(wait(b_sfree(sbuf), ((n >> 1) - 1) & 1))) { ok = false; break; }
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = ((k >> 2) * (128 * 128) + (k & 3) * 32) >> 4;
            mma_bf16_ss_if(lead, tmem + sbuf * 128, dk + ((uint32_t)ks * C::BLK_BYTES >> 4) + off,
                           dq + ((uint32_t)qs * C::BLK_BYTES >> 4) + off, id, k > 0 ? 1u : 0u);
          }
          mma_commit_if(lead, b_sfull(sbuf));
          if (w) ++n1;
          else ++n0;
          if (t + 1 == t1) mma_commit_if(lead, b_kempty(ks));
        }
        if (!prm.held) mma_commit_if(lead, b_qempty(qs));
      }
      xk += nw;
    }
    mma_commit_if(lead, b_done);
    const uint64_t t0 = globaltimer_ns();
    if (lane == 0) drain_wait(b_done, 0, t0, tmo);
  } else if (warp >= 4) {
    // ================= weights and sums, one key per thread ===========================
    const int w = (warp - 4) >> 2, q4 = warp & 3, row = q4 * 32 + lane;
    const uint32_t t_row = tmem + ((uint32_t)(q4 * 32) << 16);
    const int row_tok = row / G, row_g = row - row_tok * G;
    MassRows* rows_s = reinterpret_cast<MassRows*>(sg + C::OFF_ROW) + 2 * w;
    int n = 0, nrow = 0;
    bool ok = true;
    // one row's constants from global memory
    struct Row {
      float c, slope, tok;
      int lo, hi;
    };
    auto load_row = [&](int t) {
      Row v;
      const int i = t * TOK + row_tok;
      const bool valid = row_tok < TOK && i < r.ntok;
      v.lo = INT_MAX;
      v.hi = -1;
      v.c = -INFINITY;
      v.slope = 0.f;
      v.tok = (float)i;
      if (valid) {
        v.c = __ldg(prm.lse + (long long)(r.tok0 + i) * prm.num_q_heads + r.hk * G + row_g);
        token_range(prm.mask, r.tok0 + i, r.pos0 + i, r.seq.kv, r.prefix, v.lo, v.hi);
        if (BIAS) v.slope = __ldg(prm.slopes + r.hk * G + row_g);
      } else if (row >= G * prm.box_tokens) {
        v.lo = INT_MIN;  // zero in shared memory: needs no mask
        v.hi = INT_MAX;
      }
      return v;
    };
    auto put_row = [&](MassRows* m, const Row& v) {
      m->c[row] = v.c == -INFINITY ? v.c : -1.4426950408889634f * v.c;
      m->lo[row] = v.lo;
      m->hi[row] = v.hi;
      if (BIAS) {
        m->slope[row] = 1.4426950408889634f * v.slope;
        m->tok[row] = v.tok;
      }
    };
    // the keys that every row of a tile sees: [lo, hi]
    int all_lo[2], all_hi[2];
    auto reach = [&](const MassRows* m, int& lo, int& hi) {
      int a = INT_MIN, z = INT_MAX;
      for (int e = lane; e < prm.cols; e += 32) {
        a = max(a, m->lo[e]);
        z = min(z, m->hi[e]);
      }
      lo = __reduce_max_sync(0xffffffffu, a);
      hi = __reduce_min_sync(0xffffffffu, z);
    };
    for (; r.p < last; next()) {
      if (prm.held && r.fresh) {
        const Row v0 = load_row(0), v1 = load_row(1);
        named_bar_sync(1 + w, 128);  // the rows before these are read
        put_row(rows_s, v0);
        put_row(rows_s + 1, v1);
        named_bar_sync(1 + w, 128);
        reach(rows_s, all_lo[0], all_hi[0]);
        reach(rows_s + 1, all_lo[1], all_hi[1]);
      }
      if (w >= r.nw) continue;
      const int key0 = (r.kb + w) * C::KB, key = key0 + row;
      f32x2 sum[2] = {both(0.f), both(0.f)};
      Row v;
      if (!prm.held && r.t0 < r.t1) v = load_row(r.t0);
      float* mass = prm.mass + ((long long)r.b * prm.num_kv_heads + r.hk) * prm.mass_stride + key;
      float old = 0.f;  // fetched now, needed after the sums
      if (key < r.seq.kv - r.seq.q_len && prm.decay != 0.f) old = *mass;
      for (int t = r.t0; t < r.t1; ++t, ++n) {
        const int sbuf = 2 * w + (n & 1);
        const MassRows* m = rows_s + t;
        int mlo = all_lo[t & 1], mhi = all_hi[t & 1];
        if (!prm.held) {
          // this buffer was last read two fills ago: the meeting between orders it
          MassRows* fill = rows_s + (++nrow & 1);
          put_row(fill, v);
          named_bar_sync(1 + w, 128);
          if (t + 1 < r.t1) v = load_row(t + 1);
          reach(fill, mlo, mhi);
          m = fill;
        }
        const bool plain = mlo <= key0 && mhi >= key0 + C::KB - 1;
        if (ok && !wait_warp(b_sfull(sbuf), (n >> 1) & 1)) ok = false;
        if (!ok) continue;
        tc_fence_after();
        const float fkey = (float)(key - r.pos0);
        auto add_as = [&](auto mask_tag, auto form_tag, const uint32_t* v, int c0) {  // 16 rows
          constexpr bool MASK = decltype(mask_tag)::value;
          constexpr CapForm FORM = decltype(form_tag)::value;
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            const float4 c4 = *reinterpret_cast<const float4*>(m->c + c0 + e);
            f32x2 x0 = score2_log2<FORM>(
                prm.score, pack2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])),
                pack2(c4.x, c4.y));
            f32x2 x1 = score2_log2<FORM>(
                prm.score, pack2(__uint_as_float(v[e + 2]), __uint_as_float(v[e + 3])),
                pack2(c4.z, c4.w));
            if (BIAS) {
              const float4 s4 = *reinterpret_cast<const float4*>(m->slope + c0 + e);
              const float4 p4 = *reinterpret_cast<const float4*>(m->tok + c0 + e);
              x0 = fma2(pack2(-s4.x, -s4.y), pack2(fabsf(fkey - p4.x), fabsf(fkey - p4.y)), x0);
              x1 = fma2(pack2(-s4.z, -s4.w), pack2(fabsf(fkey - p4.z), fabsf(fkey - p4.w)), x1);
            }
            float y[4];
            unpack2(x0, y[0], y[1]);
            unpack2(x1, y[2], y[3]);
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k] = ex2_approx(y[k]);
            if (MASK) {
              const int4 l4 = *reinterpret_cast<const int4*>(m->lo + c0 + e);
              const int4 h4 = *reinterpret_cast<const int4*>(m->hi + c0 + e);
              y[0] = (key >= l4.x && key <= h4.x) ? y[0] : 0.f;
              y[1] = (key >= l4.y && key <= h4.y) ? y[1] : 0.f;
              y[2] = (key >= l4.z && key <= h4.z) ? y[2] : 0.f;
              y[3] = (key >= l4.w && key <= h4.w) ? y[3] : 0.f;
            }
            sum[0] = add2(sum[0], pack2(y[0], y[1]));
            sum[1] = add2(sum[1], pack2(y[2], y[3]));
          }
        };
        auto add = [&](auto mask_tag, const uint32_t* v, int c0) {
          if (CAP) {
            float far = 0.f;
#pragma unroll
            for (int e = 0; e < 16; e += 2)
              far = fmax3f(far, fabsf(__uint_as_float(v[e])), fabsf(__uint_as_float(v[e + 1])));
            if (__all_sync(0xffffffffu, far <= prm.score.lim)) {
              add_as(mask_tag, std::integral_constant<CapForm, CAP_NEAR>{}, v, c0);
              return;
            }
          }
          add_as(mask_tag, std::integral_constant<CapForm, CAP>{}, v, c0);
        };
        auto sweep = [&](auto mask_tag) {
          const uint32_t t_s = t_row + sbuf * 128;
          int c0 = 0;
          if (prm.cols >= 64) {
            uint32_t va[32], vb[32];
            tmem_ld32_async(t_s, va);
#pragma unroll 1
            for (; c0 + 64 <= prm.cols; c0 += 64) {
              tmem_ld_wait32(va);
              tmem_ld32_async(t_s + c0 + 32, vb);
              add(mask_tag, va, c0);
              add(mask_tag, va + 16, c0 + 16);
              tmem_ld_wait32(vb);
              if (c0 + 128 <= prm.cols) tmem_ld32_async(t_s + c0 + 64, va);
              add(mask_tag, vb, c0 + 32);
              add(mask_tag, vb + 16, c0 + 48);
            }
          }
#pragma unroll 1
          for (; c0 < prm.cols; c0 += 16) {
            uint32_t v[16];
            tmem_ld16(t_s + c0, v);
            add(mask_tag, v, c0);
          }
        };
        if (plain) sweep(std::false_type{});
        else sweep(std::true_type{});
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_sfree(sbuf));
      }
      if (ok && key < r.seq.kv) {
        float s0, s1;
        unpack2(add2(sum[0], sum[1]), s0, s1);
        *mass = fmaf(prm.decay, old, s0 + s1);
      }
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

}  // namespace cosa
