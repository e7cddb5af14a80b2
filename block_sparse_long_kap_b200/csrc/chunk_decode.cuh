// Attention of a few new tokens a sequence over the paged cache: the decode form of
// cosa_chunk_attention, for at most 16 rows (token, query head) of a sequence and KV head and
// D = 128.
//
// Both products are taken transposed, so that the 128-row side of the tensor core holds keys
// and head dims instead of rows that do not exist:
//   S^T = K Q^T      128 keys x 16 rows
//   O^T = V^T P^T    128 dims x 2 x 16 rows,   V^T read from V as it lies (MN-major A)
// The tiled form spends eight times the multiplications on this (and, under the power cap that
// a stream of the whole cache alone comes near, clock with them), and leaves the softmax of a
// block to the one warp whose rows exist; here a thread owns a key, 128 threads share the
// block, and P goes to the second product through shared memory, as two bf16 halves: rows 0-15
// bf16(p), rows 16-31 bf16(p - high), together within 2^-16 of p.  The products have time for both in one
// instruction of 32 columns (201.5 against 201.3 us for the 32 sequences below, 12.2 against 12.0 for the
// one; as two instructions of 16 each 12.5), O^T comes in two halves that the epilogue adds, and the
// output's error is that of its own rounding: 1.64e-3 of its norm, where one half left 2.1e-3 to 2.3e-3.
//
// The running maximum of a row spans threads: a warp reduces its keys' maxima (one redux a
// row), the four warps vote whether any row passed its exponent base by 2^8, and only then
// exchange the maxima and rescale O; the base is the same in all threads.  Sums stay in the
// threads until the segment ends.
//
// Work split, partial rows and join as in the tiled form, but planned by every CTA for itself
// (a tile is a sequence): equal shares of all (KV head, sequence, block)s, no plan launch.
//   warp 0  Q and K loads     warp 2  V loads, zeroing of the values behind the end, join list
//   warp 1  MMA issue         warp 3  TMEM allocation
//   warps 4-7  softmax, one key per thread
// Bound by the K and V bytes over many blocks: 32 ragged sequences of up to 32K keys (7 rows,
// 1.29 GB) take 198-205 us, 0.96-0.99 of a copy's rate; the tiled form 202 us in short runs and
// 231 us in long ones, where the clock gives way.  One sequence of 2,049 keys (32 / 8 heads) is
// latency: 7 us to the partial rows and 12 us joined, of which the first K tile's way through
// the cold cache and the instructions' own fetch are most (code of rows that do not exist is
// left by one jump: jumping from row to row cost 2 us).  Every wait is bounded; a softmax warp
// whose wait ran out keeps meeting the others at the named barrier.
#pragma once

#include "chunk_attn.cuh"

namespace cosa {

struct DecCfg {
  static constexpr int N = 16;  // rows
  static constexpr int D = 128, KB = 128, THREADS = 256;
  static constexpr uint32_t BLK_BYTES = KB * D * 2;
  static constexpr uint32_t Q_BYTES = N * D * 2;   // two halves of N x 64
  static constexpr int NP = 2 * N;  // rows of P: the high halves of the weights, then the low
  static constexpr uint32_t P_BYTES = NP * KB * 2;
  static constexpr int KS = 3, VS = 3;
  static constexpr uint32_t OFF_K = 0;
  static constexpr uint32_t OFF_V = OFF_K + KS * BLK_BYTES;
  static constexpr uint32_t OFF_Q = OFF_V + VS * BLK_BYTES;  // two segments
  static constexpr uint32_t OFF_P = OFF_Q + 2 * Q_BYTES;     // two blocks
  static constexpr uint32_t OFF_BAR = OFF_P + 2 * P_BYTES;
  // q full / empty [2], k, v full / empty, v tail, s full[2], p full[2], o full, pv done, done
  static constexpr int NBAR = 4 + 2 * KS + 2 * VS + 1 + 4 + 3;
  static constexpr uint32_t OFF_MISC = (OFF_BAR + NBAR * 8 + 15) & ~15u;
  static constexpr uint32_t OFF_ROWS = OFF_MISC + 64;        // lo, hi, slope, pos [2][N]
  static constexpr uint32_t OFF_EXCH = OFF_ROWS + 2 * 4 * N * 4;  // [N][4]
  static constexpr uint32_t SMEM = OFF_EXCH + N * 16 + 1024;  // 1024-byte alignment slack
  static constexpr int TMEM_COLS = 64;  // S at 0 and 16, O at 32 (high) and 48 (low)
  static constexpr float kRescale = 8.0f;
  static_assert(SMEM <= 227 * 1024, "shared memory budget");
};

__device__ __forceinline__ float redux_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
// named barrier of n threads that also ORs a predicate over them
__device__ __forceinline__ bool named_bar_or(int id, int n, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %3, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(n), "r"((uint32_t)v)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void st_shared_b16(uint32_t addr, __nv_bfloat16 v) {
  asm volatile("st.shared.b16 [%0], %1;" ::"r"(addr), "h"(*reinterpret_cast<uint16_t*>(&v))
               : "memory");
}

// Block range of sequence b's tokens (nb = 0: none).
__device__ __forceinline__ ChunkTile decode_tile(const ChunkAttnParams& p, int b) {
  ChunkTile d;
  const ChunkSeq s = chunk_seq(p.seqs, b);
  d.b = b;
  d.tok0 = s.q0;
  d.ntok = s.q_len;
  d.pos0 = s.kv - s.q_len;
  d.kv = s.kv;
  d.prefix = p.mask.prefix_len ? __ldg(p.mask.prefix_len + b) : 0;
  d.jb = d.nb = 0;
  if (!s.ok) return d;
  int kmin = INT_MAX, kmax = -1;
  for (int i = 0; i < s.q_len; ++i) {
    int a, z;
    token_range(p.mask, d.tok0 + i, d.pos0 + i, d.kv, d.prefix, a, z);
    if (a <= z) {
      kmin = min(kmin, a);
      kmax = max(kmax, z);
    }
  }
  d.jb = kmax >= 0 ? kmin >> 7 : 0;  // no visible key: one masked block
  d.nb = kmax >= 0 ? (kmax >> 7) + 1 - d.jb : 1;
  return d;
}

template <bool CAP, bool BIAS>
__global__ void __launch_bounds__(256, 1)
    chunk_decode_kernel(const __grid_constant__ CUtensorMap tm_q,
                        const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const ChunkAttnParams prm) {
  using C = DecCfg;
  using namespace tc;
  constexpr int D = C::D, N = C::N;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t sraw = static_cast<uint32_t>(__cvta_generic_to_shared(smem_raw));
  const uint32_t sb0 = (sraw + 1023u) & ~1023u;
  uint8_t* sg = smem_raw + (sb0 - sraw);
  const uint32_t sK = sb0 + C::OFF_K, sV = sb0 + C::OFF_V, sQ = sb0 + C::OFF_Q, sP = sb0 + C::OFF_P;
  const uint32_t bar = sb0 + C::OFF_BAR;
  auto b_qfull = [&](int i) { return bar + 8u * i; };
  auto b_qempty = [&](int i) { return bar + 8u * (2 + i); };
  auto b_kfull = [&](int s) { return bar + 8u * (4 + s); };
  auto b_kempty = [&](int s) { return bar + 8u * (4 + C::KS + s); };
  auto b_vfull = [&](int s) { return bar + 8u * (4 + 2 * C::KS + s); };
  auto b_vempty = [&](int s) { return bar + 8u * (4 + 2 * C::KS + C::VS + s); };
  constexpr int B0 = 4 + 2 * C::KS + 2 * C::VS;
  const uint32_t b_vtail = bar + 8u * B0;
  auto b_sfull = [&](int i) { return bar + 8u * (B0 + 1 + i); };
  auto b_pfull = [&](int i) { return bar + 8u * (B0 + 3 + i); };
  const uint32_t b_ofull = bar + 8u * (B0 + 5), b_pv = bar + 8u * (B0 + 6), b_done = bar + 8u * (B0 + 7);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sg + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sg + C::OFF_MISC + 4);
  int* start_off = reinterpret_cast<int*>(sg + C::OFF_MISC + 8);
  ChunkTile* start_s = reinterpret_cast<ChunkTile*>(sg + C::OFF_MISC + 16);
  long long* scan_s = reinterpret_cast<long long*>(sg + C::OFF_ROWS);  // (before the rows)

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int G = prm.group, P = prm.page_size, B = prm.seqs.batch;
  // (an earlier launch that timed out: looked at with the plan's loads under way)
  const bool stop = *(volatile int*)&g_status == COSA_ERR_TIMEOUT;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) { mbar_init(b_qfull(i), 1); mbar_init(b_qempty(i), 1); }
    for (int s = 0; s < C::KS; ++s) { mbar_init(b_kfull(s), 1); mbar_init(b_kempty(s), 1); }
    for (int s = 0; s < C::VS; ++s) { mbar_init(b_vfull(s), 1); mbar_init(b_vempty(s), 1); }
    mbar_init(b_vtail, 1);
    for (int i = 0; i < 2; ++i) { mbar_init(b_sfull(i), 1); mbar_init(b_pfull(i), 4); }
    mbar_init(b_ofull, 1);
    mbar_init(b_pv, 1);
    mbar_init(b_done, 1);
    *abort_flag = 0;
    start_s->nb = *start_off = 0;  // (found below, unless the lengths change meanwhile)
    fence_barrier_init();
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  if (warp == 3) {
    tmem_alloc(sb0 + C::OFF_MISC, C::TMEM_COLS);
    tmem_relinquish();
  }
  // ---- plan: blocks of all sequences, a contiguous group of them per thread
  const int per = (B + C::THREADS - 1) / C::THREADS;
  const int bs0 = min(tid * per, B), bs1 = min(bs0 + per, B);
  ChunkTile first;  // the group's first sequence, kept (the only one for up to 256)
  first.nb = 0;
  long long mine = 0;
  for (int b = bs0; b < bs1; ++b) {
    const ChunkTile d = decode_tile(prm, b);
    if (b == bs0) first = d;
    mine += d.nb;
  }
  long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) scan_s[warp] = inc;
  const bool stopped = __syncthreads_or(stop);
  long long before = inc - mine, per_head = 0;
#pragma unroll
  for (int w = 0; w < C::THREADS / 32; ++w) {
    const long long v = scan_s[w];
    if (w < warp) before += v;
    per_head += v;
  }
  // (32-bit divisions where they do: a 64-bit one takes a tenth of a microsecond)
  auto divide = [](long long a, long long d) -> long long {
    return a <= 0xffffffffll && d <= 0xffffffffll ? (long long)((uint32_t)a / (uint32_t)d) : a / d;
  };
  const long long total = stopped ? 0 : per_head * prm.num_kv_heads;
  const long long quota = divide(total + gridDim.x - 1, gridDim.x);
  const long long w0 = min((long long)blockIdx.x * quota, total), w1 = min(w0 + quota, total);
  const int hk0 = w0 < w1 ? (int)divide(w0, per_head) : 0;
  if (w0 < w1) {
    long long rem = w0 - hk0 * per_head - before;
    if (rem >= 0 && rem < mine)
      for (int b = bs0; b < bs1; ++b) {
        const ChunkTile d = b == bs0 ? first : decode_tile(prm, b);
        if (rem < d.nb) {
          *start_s = d;
          *start_off = (int)rem;
          break;
        }
        rem -= d.nb;
      }
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);

  // ---- this CTA's segments; every role walks by itself
  DecodeWalk wk;
  wk.left = w1 - w0;
  wk.hk = hk0;
  wk.b = wk.off = 0;
  wk.lost = false;
  wk.have = wk.left > 0;
  if (wk.have) {
    wk.tile = *start_s;
    wk.b = wk.tile.b;
    wk.off = *start_off;
  }
  auto next = [&]() { return wk.next(B, prm.num_kv_heads, [&](int b) { return decode_tile(prm, b); }); };
  auto advance = [&]() { wk.advance(B); };

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
  auto all = [&](bool v) { return __all_sync(0xffffffffu, v) != 0; };
  const int pshift = 31 - __clz(P), ppb = C::KB >> pshift;
  auto blk_pages = [&](int kv, int j) { return min(ppb, (kv - j * C::KB + P - 1) >> pshift); };
  auto page_coord = [&](int j, int np) -> int {
    if (lane >= np) return 0;
    if ((j * ppb + lane + 1) << pshift <= window_start(prm.mask, wk.tile.pos0)) return -1;
    const int ph = __ldg(prm.page_table + (long long)wk.b * prm.pages_per_seq + j * ppb + lane);
    if (ph < 0 || ph >= prm.num_phys_pages) {
      set_status(COSA_ERR_INVALID_ARG);
      return -1;
    }
    return ph * prm.num_kv_heads + wk.hk;
  };

  if (warp == 0) {
    // ================= Q and K ========================================================
    int it = 0, seg = 0;
    bool ok = true;
    const uint32_t qbytes = (uint32_t)(G * prm.seqs.max_q * 128 * 2);
    for (; ok && next(); advance()) {
      const int qs = seg & 1;
      if (seg >= 2 && !wait_warp(b_qempty(qs), ((seg >> 1) - 1) & 1)) { ok = false; break; }
      if (lane == 0) {
        mbar_arrive_expect_tx(b_qfull(qs), qbytes);
#pragma unroll
        for (int h = 0; h < 2; ++h)
          tma_load_3d(sQ + qs * C::Q_BYTES + h * (N * 128), &tm_q, b_qfull(qs), h * 64, wk.hk * G,
                      wk.tile.tok0);
      }
      ++seg;
      int cz = page_coord(wk.jb, blk_pages(wk.tile.kv, wk.jb));
      for (int j = 0; j < wk.nb; ++j, ++it) {
        const int s = it % C::KS, np = blk_pages(wk.tile.kv, wk.jb + j);
        int cz_next = 0;
        if (j + 1 < wk.nb) cz_next = page_coord(wk.jb + j + 1, blk_pages(wk.tile.kv, wk.jb + j + 1));
        if (it >= C::KS && !wait_warp(b_kempty(s), ((it / C::KS) - 1) & 1)) { ok = false; break; }
        if (lane == 0) mbar_arrive_expect_tx(b_kfull(s), (uint32_t)(np * P * D * 2));
        __syncwarp();
        if (lane < np)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            tma_load_3d(sK + s * C::BLK_BYTES + h * (C::KB * 128) + lane * (P * 128), &tm_k,
                        b_kfull(s), h * 64, 0, cz);
        cz = cz_next;
      }
    }
    // loads never consumed (abort only) land before the CTA leaves
    if (lane == 0) {
      const uint64_t t0 = globaltimer_ns();
      for (int x = max(0, seg - 2); x < seg; ++x) drain_wait(b_qfull(x & 1), (x >> 1) & 1, t0, tmo);
      for (int x = max(0, it - C::KS); x < it; ++x)
        drain_wait(b_kfull(x % C::KS), (x / C::KS) & 1, t0, tmo);
    }
  } else if (warp == 2) {
    // ================= V ==============================================================
    int it = 0, tails = 0;
    bool ok = true;
    ChunkJoin jn;  // the sequence that this share starts and does not finish
    jn.ntok = jn.tok0 = jn.hk = jn.last = 0;
    for (; ok && next(); advance()) {
      if (wk.part == 1) {
        jn.tok0 = wk.tile.tok0;
        jn.ntok = wk.tile.ntok;
        jn.hk = wk.hk;
        jn.last = (int)((w1 - wk.left + wk.tile.nb - 1) / quota);
      }
      int cz = page_coord(wk.jb, blk_pages(wk.tile.kv, wk.jb));
      for (int j = 0; j < wk.nb; ++j, ++it) {
        const int s = it % C::VS, np = blk_pages(wk.tile.kv, wk.jb + j);
        const int keys = wk.tile.kv - (wk.jb + j) * C::KB;
        int cz_next = 0;
        if (j + 1 < wk.nb) cz_next = page_coord(wk.jb + j + 1, blk_pages(wk.tile.kv, wk.jb + j + 1));
        if (it >= C::VS && !wait_warp(b_vempty(s), ((it / C::VS) - 1) & 1)) { ok = false; break; }
        // the MMA reads the keys of whole 16-key steps: those behind the end are zeroed
        const bool tail = keys < C::KB && (keys & 15) != 0;
        const uint32_t full = tail ? b_vtail : b_vfull(s);
        const uint32_t dst = sV + s * C::BLK_BYTES;
        if (lane == 0) mbar_arrive_expect_tx(full, (uint32_t)(np * P * D * 2));
        __syncwarp();
        if (lane < np)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            tma_load_3d(dst + h * (C::KB * 128) + lane * (P * 128), &tm_v, full, h * 64, 0, cz);
        cz = cz_next;
        if (tail) {
          const bool have = wait_warp(b_vtail, tails & 1);
          ++tails;
          const int nz = 16 - (keys & 15);
          for (int x = lane; have && x < nz * 16; x += 32) {
            const int c = x & 7, r = keys + (x >> 3) % nz, h = (x >> 3) / nz;
            st_shared_v4(dst + h * (C::KB * 128) + r * 128 + c * 16, 0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(b_vfull(s));
          if (!have) { ++it; ok = false; break; }
        }
      }
    }
    if (lane == 0) {
      if (wk.lost) set_status(COSA_ERR_INVALID_ARG);
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
  } else if (warp == 1) {
    // ================= MMA issue (the whole warp walks, one lane issues) ==================
    const uint32_t lead = elect_one();
    constexpr uint32_t ID_QK = idesc_bf16_f32(128, N, 0);
    constexpr uint32_t ID_PV = idesc_bf16_f32(128, C::NP, 0) | (1u << 15);  // A = V^T, MN-major
    const uint64_t dq = smem_desc_sw128(sQ, 16, 1024), dk = smem_desc_sw128(sK, 16, 1024);
    const uint64_t dv = smem_desc_sw128(sV, C::KB * 128, 1024), dp = smem_desc_sw128(sP, 16, 1024);
    int it = 0, seg = 0;
    bool ok = true;
    while (ok && all(next())) {
      const int nb = __shfl_sync(0xffffffffu, wk.nb, 0);
      const int keys0 = __shfl_sync(0xffffffffu, wk.tile.kv - wk.jb * C::KB, 0);
      const uint64_t dqs = dq + ((uint32_t)(seg & 1) * C::Q_BYTES >> 4);
      if (!all(wait(b_qfull(seg & 1), (seg >> 1) & 1))) { ok = false; break; }
      // step j: S^T of block j, then O^T += V^T P^T of block j - 1, under the softmax of j
      for (int j = 0; j <= nb; ++j) {
        if (j < nb) {
          const int x = it + j, s = x % C::KS;
          if (!all(wait(b_kfull(s), (x / C::KS) & 1))) { ok = false; break; }
          tc_fence_after();
          const uint64_t dks = dk + ((uint32_t)s * C::BLK_BYTES >> 4);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mma_bf16_ss_if(lead, tmem + (x & 1) * 16, dks + (((k >> 2) * (C::KB * 128) + (k & 3) * 32) >> 4),
                           dqs + (((k >> 2) * (N * 128) + (k & 3) * 32) >> 4), ID_QK, k > 0 ? 1u : 0u);
          mma_commit_if(lead, b_sfull(x & 1));
          mma_commit_if(lead, b_kempty(s));
          if (j + 1 == nb) mma_commit_if(lead, b_qempty(seg & 1));
        }
        if (j > 0) {
          const int x = it + j - 1, s = x % C::VS, keys = keys0 - (j - 1) * C::KB;
          if (!all(wait(b_vfull(s), (x / C::VS) & 1)) || !all(wait(b_pfull(x & 1), (x >> 1) & 1))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t dvs = dv + ((uint32_t)s * C::BLK_BYTES >> 4);
          const uint64_t dps = dp + ((uint32_t)(x & 1) * C::P_BYTES >> 4);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mma_bf16_ss_if(k * 16 < keys ? lead : 0u, tmem + 32, dvs + ((k * 16 * 128) >> 4),
                           dps + (((k >> 2) * (C::NP * 128) + (k & 3) * 32) >> 4), ID_PV,
                           (j > 1 || k > 0) ? 1u : 0u);
          mma_commit_if(lead, b_pv);
          mma_commit_if(lead, b_vempty(s));
          if (j == nb) mma_commit_if(lead, b_ofull);
        }
      }
      if (!ok) break;
      it += nb;
      ++seg;
      advance();
    }
    // every issued MMA completes before teardown frees TMEM
    mma_commit_if(lead, b_done);
    const uint64_t t0 = globaltimer_ns();
    if (lane == 0) drain_wait(b_done, 0, t0, tmo);
  } else if (warp >= 4) {
    // ================= softmax: key `row` of the block, then dim `row` of O ==============
    const int q4 = warp & 3, row = q4 * 32 + lane;
    const uint32_t t_row = tmem + ((uint32_t)(q4 * 32) << 16);
    float* exch = reinterpret_cast<float*>(sg + C::OFF_EXCH);  // [N][4]
    // where this key's weights go in P: row r at + r * 128, its 16-byte piece swizzled by r
    const uint32_t p_col = sP + (row >> 6) * (C::NP * 128) + (row & 7) * 2, p_piece = (row & 63) >> 3;
    int cnt = 0, nseg = 0;
    bool ok = true;
    for (; next(); advance()) {
      const int nrow = wk.tile.ntok * G;
      int* rlo = reinterpret_cast<int*>(sg + C::OFF_ROWS) + (nseg & 1) * 4 * N;
      int* rhi = rlo + N;
      float* rsl = reinterpret_cast<float*>(rhi + N);
      float* rpos = rsl + N;
      if (row < N) {
        int lo = INT_MIN, hi = INT_MAX;  // rows that do not exist see everything
        float slope = 0.f;
        const int tok = row / G;
        if (row < nrow) {
          token_range(prm.mask, wk.tile.tok0 + tok, wk.tile.pos0 + tok, wk.tile.kv, wk.tile.prefix,
                      lo, hi);
          if (BIAS)
            slope = 1.4426950408889634f * __ldg(prm.slopes + wk.hk * G + row - tok * G);
        }
        rlo[row] = lo;
        rhi[row] = hi;
        rsl[row] = slope;
        rpos[row] = (float)tok;  // (a float does not hold every position past 2^24)
      }
      named_bar_sync(1, 128);
      // the keys that every row sees: [alo, ahi]
      const int e_row = lane < N ? lane : 0;
      const int alo = __reduce_max_sync(0xffffffffu, rlo[e_row]);
      const int ahi = __reduce_min_sync(0xffffffffu, rhi[e_row]);
      float m_ref[N], l[N];
#pragma unroll
      for (int r = 0; r < N; ++r) {
        m_ref[r] = -INFINITY;
        l[r] = 0.f;
      }
      for (int j = 0; j < wk.nb; ++j, ++cnt) {
        const int buf = cnt & 1, key0 = (wk.jb + j) * C::KB, key = key0 + row;
        const float ahead = (float)(key - wk.tile.pos0);  // of the first new token
        if (ok && !wait_warp(b_sfull(buf), (cnt >> 1) & 1)) ok = false;
        float x[N], wmax[N];
        bool grow = false;
        if (ok) {
          tc_fence_after();
          uint32_t sc[N];
          tmem_ld16(t_row + buf * 16, sc);
          const bool plain = alo <= key0 && ahi >= key0 + C::KB - 1;
#pragma unroll
          for (int r0 = 0; r0 < N; r0 += 4) {
            if (r0 >= nrow) break;  // one jump past all the code of rows that do not exist
#pragma unroll
            for (int r = r0; r < r0 + 4; r += 2)
              unpack2(score2_log2<CAP ? CAP_EACH : CAP_NONE>(
                          prm.score, pack2(__uint_as_float(sc[r]), __uint_as_float(sc[r + 1])),
                          both(0.f)),
                      x[r], x[r + 1]);
#pragma unroll
            for (int r = r0; r < r0 + 4; ++r) {
              if (BIAS) x[r] = fmaf(-rsl[r], fabsf(ahead - rpos[r]), x[r]);
              if (!plain && (key < rlo[r] || key > rhi[r])) x[r] = -INFINITY;
              wmax[r] = redux_max(x[r]);
              grow = grow || (r < nrow && wmax[r] > m_ref[r] + C::kRescale);
            }
          }
        }
        if (named_bar_or(1, 128, ok && grow)) {
          if (ok) {
            float v = 0.f;
#pragma unroll
            for (int r0 = 0; r0 < N; r0 += 4) {
              if (r0 >= nrow) break;
#pragma unroll
              for (int r = r0; r < r0 + 4; ++r)
                if (lane == r) v = wmax[r];
            }
            if (lane < nrow) exch[lane * 4 + q4] = v;
          }
          named_bar_sync(1, 128);
          if (ok) {
            float alpha[N];
#pragma unroll
            for (int r = 0; r < N; ++r) alpha[r] = 1.f;
#pragma unroll
            for (int r0 = 0; r0 < N; r0 += 4) {
              if (r0 >= nrow) break;
#pragma unroll
              for (int r = r0; r < r0 + 4; ++r) {
                const float4 e4 = *reinterpret_cast<const float4*>(exch + r * 4);
                const float m = fmaxf(fmaxf(e4.x, e4.y), fmaxf(e4.z, e4.w));
                if (r < nrow && m > m_ref[r] + C::kRescale) {
                  alpha[r] = ex2_approx(m_ref[r] - m);
                  m_ref[r] = m;
                  l[r] *= alpha[r];
                }
              }
            }
            if (j > 0) {  // O is at rest once the previous block's product is done
              if (wait_warp(b_pv, (cnt - 1) & 1)) {
                tc_fence_after();
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                  uint32_t o[N];
                  tmem_ld16(t_row + 32 + h * N, o);
#pragma unroll
                  for (int r = 0; r < N; ++r) o[r] = __float_as_uint(__uint_as_float(o[r]) * alpha[r]);
                  tmem_st16(t_row + 32 + h * N, o);
                }
                tmem_st_wait();
              } else {
                ok = false;
              }
            }
          }
        }
        if (ok) {
#pragma unroll
          for (int r0 = 0; r0 < N; r0 += 4) {
            if (r0 >= nrow) break;
#pragma unroll
            for (int r = r0; r < r0 + 4; ++r) {
              const float p = ex2_approx(x[r] - (m_ref[r] == -INFINITY ? 0.f : m_ref[r]));
              l[r] += p;
              const __nv_bfloat16 hi = __float2bfloat16_rn(p);
              const uint32_t at = p_col + buf * C::P_BYTES + r * 128 + ((p_piece ^ (r & 7)) << 4);
              st_shared_b16(at, hi);
              st_shared_b16(at + N * 128, __float2bfloat16_rn(p - __bfloat162float(hi)));
            }
          }
          fence_proxy_async_smem();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(b_pfull(buf));
        }
      }
      // ---- epilogue: the rows' sums over all keys, then dim `row` of every row
      if (ok && !wait_warp(b_ofull, nseg & 1)) ok = false;
      ++nseg;
#pragma unroll
      for (int r0 = 0; r0 < N; r0 += 4) {
        if (r0 >= nrow) break;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
          for (int r = r0; r < r0 + 4; ++r) l[r] += __shfl_xor_sync(0xffffffffu, l[r], o);
        if (lane < 4)
          exch[(r0 + lane) * 4 + q4] = lane < 2 ? (lane ? l[r0 + 1] : l[r0])
                                                : (lane == 2 ? l[r0 + 2] : l[r0 + 3]);
      }
      named_bar_sync(1, 128);
      if (ok) {
        tc_fence_after();
        uint32_t o[N], low[N];
        tmem_ld16(t_row + 32, o);
        tmem_ld16(t_row + 32 + N, low);
#pragma unroll
        for (int r = 0; r < N; ++r) o[r] = __float_as_uint(__uint_as_float(o[r]) + __uint_as_float(low[r]));
        const long long slot = (2 * blockIdx.x + (wk.part > 0 ? 1 : 0)) * (long long)prm.part_rows;
        long long at = (long long)wk.tile.tok0 * prm.num_q_heads + wk.hk * G;  // row 0's
        int g = 0;
#pragma unroll
        for (int r = 0; r < N; ++r) {
          if (r >= nrow) break;
          const float4 e4 = *reinterpret_cast<const float4*>(exch + r * 4);
          const float sum = (e4.x + e4.y) + (e4.z + e4.w);
          if (wk.part < 0) {
            const float inv = row_scale(sum);
            prm.out[at * D + row] = __float2bfloat16_rn(__uint_as_float(o[r]) * inv);
            if (prm.lse && row == r) prm.lse[at] = row_lse(m_ref[r], sum);
          } else {
            prm.part_o[(slot + r) * D + row] = __uint_as_float(o[r]);
            if (row == r) prm.part_ml[slot + r] = make_float2(m_ref[r], sum);
          }
          ++at;  // the next head of the group, or the next token's first
          if (++g == G) {
            g = 0;
            at += prm.num_q_heads - G;
          }
        }
        tc_fence_before();
      }
      named_bar_sync(1, 128);  // the sums are read
    }
  }

  // ---- teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 3) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

}  // namespace cosa
