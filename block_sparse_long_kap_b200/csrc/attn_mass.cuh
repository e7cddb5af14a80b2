// Accumulated attention mass of the cached keys (cosa_attention_mass):
//   mass[k] = (k is older than the chunk ? decay * mass[k] : 0)
//             + sum over rows (token, head of the group) of e^(s - lse_row).
// The softmax normaliser is known (the lse that the attention left), so no running maximum
// is needed and the sum over rows is a plain column sum of the weights.  The product is
// taken transposed, S^T = K Q^T: a thread owns one key (its TMEM lane) and adds the weights
// of all rows in a register, in a fixed order, without atomics or shuffles.
//
// A CTA takes a run of key blocks of one (sequence, KV head), two at a time (one for each
// group of four softmax warps), and streams the tiles of 128 rows past them; a Q tile is
// loaded once for both blocks, and once in all when the chunk has a single tile.
//   warp 0  K loads      warp 2  Q loads
//   warp 1  MMA issue    warp 3  TMEM allocation
//   warps 4-7 / 8-11     weights and sums of the first / second block of a pair; two S
//                        buffers each, so the next tile's product runs under this one's
//                        exponentials.
// Bound by the K bytes for a few rows, by the exponentials for many.
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
  int last_q;        // 0: all
  int cols;          // columns of the product: rows of a tile rounded up to 16
  float decay;
  ScoreShape score;
  unsigned long long timeout_ns;
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
  static constexpr uint32_t OFF_ROW = OFF_Q + QS * BLK_BYTES;  // per group: rows' constants
  // [2 groups][2 buffers][128] of float4: -lse (log2), first and last key, slope; positions
  static constexpr uint32_t ROW_BYTES = 128 * 20;
  static constexpr uint32_t OFF_BAR = OFF_ROW + 4 * ROW_BYTES;
  static constexpr int NBAR = 2 * KS + 2 * QS + 8 + 1;  // k, q full / empty; s full / free [4]; done
  static constexpr uint32_t OFF_MISC = (OFF_BAR + NBAR * 8 + 15) & ~15u;
  static constexpr uint32_t SMEM = OFF_MISC + 16;
  static constexpr uint32_t SMEM_ALLOC = SMEM + 1024;
  static_assert(SMEM_ALLOC <= 227 * 1024, "shared memory budget");
};

// grid (parts, H_kv, B)
template <int D, bool CAP, bool BIAS>
__global__ void __launch_bounds__(384, 1)
    attn_mass_kernel(const __grid_constant__ CUtensorMap tm_q,
                     const __grid_constant__ CUtensorMap tm_k, const MassParams prm) {
  using C = MassCfg<D>;
  using namespace tc;
  const int hk = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = prm.group, TOK = prm.tile_tokens, P = prm.page_size;
  const ChunkSeq seq = chunk_seq(prm.seqs, b);
  if (!seq.ok) return;
  // this CTA's key blocks
  const int nblk = (seq.kv + C::KB - 1) / C::KB;
  const int per = (nblk + gridDim.x - 1) / gridDim.x;
  const int kb0 = blockIdx.x * per, kb1 = min(kb0 + per, nblk);
  if (kb0 >= kb1) return;
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

  // rows: the last tokens of the chunk
  const int skip = (prm.last_q > 0 && prm.last_q < seq.q_len) ? seq.q_len - prm.last_q : 0;
  const int tok0 = seq.q0 + skip, ntok = seq.q_len - skip;
  const int pos0 = seq.kv - ntok;
  const int prefix = prm.mask.prefix_len ? __ldg(prm.mask.prefix_len + b) : 0;
  const int ntile = (ntok + TOK - 1) / TOK;
  // tiles that may see a key of the pair of blocks starting at kb (documents only narrow it)
  auto tile_range = [&](int kb, int& t0, int& t1) {
    const int key0 = kb * C::KB, key1 = min(kb + 2, kb1) * C::KB - 1;
    t0 = 0;
    t1 = ntile;
    if (prefix <= key0) t0 = min(max(key0 - pos0, 0) / TOK, ntile);
    if (prm.mask.window > 0) {  // the first token that no longer sees key1
      const long long i = (long long)key1 + prm.mask.window - pos0;
      t1 = i <= 0 ? 0 : (int)min((i + TOK - 1) / TOK, (long long)ntile);
    }
    if (t1 < t0) t1 = t0;
  };
  const bool one_tile = ntile == 1;

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
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const unsigned long long tmo = prm.timeout_ns;
  auto wait = [&](uint32_t bar_addr, uint32_t parity) -> bool {
    if (mbar_try_wait(bar_addr, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar_addr, parity)) {
      if (*abort_flag) return false;
      if (*(volatile int*)&g_status == COSA_ERR_TIMEOUT || globaltimer_ns() - t0 > tmo) {
        *abort_flag = 1;
        set_status(COSA_ERR_TIMEOUT);
        return false;
      }
    }
    return true;
  };
  auto wait_warp = [&](uint32_t bar_addr, uint32_t parity) -> bool {
    int okl = 1;
    if (lane == 0) okl = wait(bar_addr, parity) ? 1 : 0;
    return __shfl_sync(0xffffffffu, okl, 0) != 0;
  };

  if (warp == 0) {
    // ================= K ==============================================================
    const int ppb = C::KB / P;
    int x = 0;  // blocks loaded
    for (int kb = kb0; kb < kb1; ++kb) {
      int t0, t1;
      tile_range(kb0 + ((kb - kb0) & ~1), t0, t1);
      if (t0 == t1) continue;  // nobody sees the pair
      const int s = x % C::KS, np = min(ppb, (seq.kv - kb * C::KB + P - 1) / P);
      int cz = 0;
      if (lane < np) {
        const int ph = __ldg(prm.page_table + (long long)b * prm.pages_per_seq + kb * ppb + lane);
        cz = (ph < 0 || ph >= prm.num_phys_pages) ? -1 : ph * prm.num_kv_heads + hk;
        if (cz < 0) set_status(COSA_ERR_INVALID_ARG);
      }
      if (x >= C::KS && !wait_warp(b_kempty(s), ((x / C::KS) - 1) & 1)) break;
      if (lane == 0) mbar_arrive_expect_tx(b_kfull(s), (uint32_t)(np * P * D * 2));
      __syncwarp();
      if (lane < np)
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
          tma_load_3d(sK + s * C::BLK_BYTES + h * (C::KB * 128) + lane * (P * 128), &tm_k,
                      b_kfull(s), h * 64, 0, cz);
      ++x;
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
      const uint32_t bytes = (uint32_t)(G * TOK * 128 * (D / 64));
      for (int kb = kb0; ok && kb < kb1; kb += 2) {
        int t0, t1;
        tile_range(kb, t0, t1);
        for (int t = t0; t < t1; ++t) {
          if (one_tile && x > 0) break;  // stays in its slot
          const int s = x % C::QS;
          if (x >= C::QS && !wait(b_qempty(s), ((x / C::QS) - 1) & 1)) { ok = false; break; }
          mbar_arrive_expect_tx(b_qfull(s), bytes);
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
            tma_load_3d(sQ + s * C::BLK_BYTES + h * (128 * 128), &tm_q, b_qfull(s), h * 64, hk * G,
                        tok0 + t * TOK);
          ++x;
        }
      }
      const uint64_t t0 = globaltimer_ns();
      for (int y = max(0, x - C::QS); y < x; ++y)
        drain_wait(b_qfull(y % C::QS), (y / C::QS) & 1, t0, tmo);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ================= MMA issue: S^T = K Q^T =========================================
      const uint32_t id = idesc_bf16_f32(128, prm.cols, 0);
      const uint64_t dq = smem_desc_sw128(sQ, 16, 1024);
      const uint64_t dk = smem_desc_sw128(sK, 16, 1024);
      int xk = 0, xq = 0, n[2] = {0, 0};  // blocks and tiles taken, products of each group
      bool ok = true;
      for (int kb = kb0; ok && kb < kb1; kb += 2) {
        int t0, t1;
        tile_range(kb, t0, t1);
        if (t0 == t1) continue;
        const int nw = min(2, kb1 - kb);
        for (int t = t0; ok && t < t1; ++t) {
          const int qs = one_tile ? 0 : xq % C::QS;
          if (!one_tile || xq == 0)
            ok = wait(b_qfull(qs), (xq / C::QS) & 1);
          for (int w = 0; ok && w < nw; ++w) {
            const int ks = (xk + w) % C::KS, sbuf = 2 * w + (n[w] & 1);
            if (t == t0 && !wait(b_kfull(ks), ((xk + w) / C::KS) & 1)) { ok = false; break; }
            if (n[w] >= 2 && !wait(b_sfree(sbuf), ((n[w] >> 1) - 1) & 1)) { ok = false; break; }
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint32_t off = ((k >> 2) * (128 * 128) + (k & 3) * 32) >> 4;
              mma_bf16_ss(tmem + sbuf * 128, dk + ((uint32_t)ks * C::BLK_BYTES >> 4) + off,
                          dq + ((uint32_t)qs * C::BLK_BYTES >> 4) + off, id, k > 0 ? 1u : 0u);
            }
            mma_commit(b_sfull(sbuf));
            ++n[w];
            if (t + 1 == t1) mma_commit(b_kempty(ks));
          }
          if (!ok) break;
          if (!one_tile) mma_commit(b_qempty(qs));
          ++xq;
        }
        xk += nw;
      }
      mma_commit(b_done);
      const uint64_t t0 = globaltimer_ns();
      drain_wait(b_done, 0, t0, tmo);
    }
  } else if (warp >= 4) {
    // ================= weights and sums, one key per thread ===========================
    const int w = (warp - 4) >> 2, q4 = warp & 3, row = q4 * 32 + lane;
    const uint32_t t_row = tmem + ((uint32_t)(q4 * 32) << 16);
    const int row_tok = row / G, row_g = row - row_tok * G;
    int n = 0, loaded = 0;
    bool ok = true, plain = false;  // plain: every row of the tile sees every key of the block
    // rows' constants: -lse in log2 units, first and last key, slope, position
    auto row_f = [&](int buf) {
      return reinterpret_cast<float*>(sg + C::OFF_ROW + (w * 2 + buf) * C::ROW_BYTES);
    };
    for (int kb = kb0; ok && kb < kb1; kb += 2) {
      int t0, t1;
      tile_range(kb, t0, t1);
      const int mine = kb + w;
      if (mine >= kb1) break;
      const int key0 = mine * C::KB, key = key0 + row;
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
      for (int t = t0; t < t1; ++t, ++n) {
        const int sbuf = 2 * w + (n & 1);
        float* rc = row_f(one_tile ? 0 : n & 1);
        int* rl = reinterpret_cast<int*>(rc + 128);
        int* rh = rl + 128;
        float* rs = rc + 384;
        float* rp = rc + 512;
        if (!one_tile || loaded == 0) {
          // the buffer was last read two tiles ago: the barrier of the tile between orders it
          const int i = t * TOK + row_tok;
          const bool valid = row_tok < TOK && i < ntok;
          int lo = INT_MAX, hi = -1;
          float c = 0.f;
          if (valid) {
            token_range(prm.mask, tok0 + i, pos0 + i, seq.kv, prefix, lo, hi);
            c = -1.4426950408889634f *
                __ldg(prm.lse + (long long)(tok0 + i) * prm.num_q_heads + hk * G + row_g);
          }
          rc[row] = c;
          rl[row] = lo;
          rh[row] = hi;
          if (BIAS) {
            rs[row] = valid ? 1.4426950408889634f * __ldg(prm.slopes + hk * G + row_g) : 0.f;
            rp[row] = (float)(pos0 + i);
          }
          loaded = 1;
          named_bar_sync(1 + w, 128);
        }
        // does every row of the tile see the whole block?
        {
          bool in = true;
          for (int r = lane; r < prm.cols; r += 32) in = in && rl[r] <= key0 && rh[r] >= key0 + C::KB - 1;
          plain = __all_sync(0xffffffffu, in);
        }
        if (!wait_warp(b_sfull(sbuf), (n >> 1) & 1)) { ok = false; break; }
        tc_fence_after();
        auto add = [&](auto mask_tag) {
          constexpr bool MASK = decltype(mask_tag)::value;
          const float fkey = (float)key;
#pragma unroll 1
          for (int c0 = 0; c0 < prm.cols; c0 += 16) {
            uint32_t v[16];
            tmem_ld16(t_row + sbuf * 128 + c0, v);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int r = c0 + e;
              float x;
              if (!CAP) x = fmaf(__uint_as_float(v[e]), prm.score.a, rc[r]);
              else x = score_log2<true>(prm.score, __uint_as_float(v[e])) + rc[r];
              if (BIAS) x = fmaf(-rs[r], fabsf(fkey - rp[r]), x);
              float pr = ex2_approx(x);
              if (MASK) pr = (key >= rl[r] && key <= rh[r]) ? pr : 0.f;
              sum[e & 3] += pr;
            }
          }
        };
        if (plain) add(std::false_type{});
        else add(std::true_type{});
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_sfree(sbuf));
      }
      if (ok && key < seq.kv) {
        float* m = prm.mass + ((long long)b * prm.num_kv_heads + hk) * prm.mass_stride + key;
        float old = 0.f;
        if (key < seq.kv - seq.q_len && prm.decay != 0.f) old = prm.decay * *m;
        *m = old + ((sum[0] + sum[1]) + (sum[2] + sum[3]));
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
