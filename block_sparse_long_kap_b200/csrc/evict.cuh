// Eviction by accumulated attention mass: per (sequence, KV head) the sink and recent keys
// and the heaviest others up to a budget, then a gather of their K, V and mass into new
// pages.
//
// evict_select_kernel: one cluster of 8 CTAs per (b, h_kv); each CTA owns a contiguous
// eighth of the candidates and holds their keys in shared memory.  The K-th largest mass is
// found by a radix select over the order-preserving 32-bit form of the float (digits of 11,
// 11 and 10 bits); the CTAs add their histograms' non-empty bins into one that is spread
// over the cluster's shared memories, one cluster barrier a digit (reading all eight
// histograms instead cost 5,000 cycles a digit: distributed shared memory moves some 13
// bytes a cycle).  Equal masses at the border go to the lowest positions: the CTAs' counts
// of larger and of equal keys give each one its place, so the kept list comes out ascending
// and is the same on every run.
// Measured, both kernels replayed back to back: 32K keys of 8 heads cut to 4K 20.4 us, six ragged
// sequences of up to 16K keys 25.7 us; the bytes are 5 and 8 us of it.  (Apart and from cold caches the select
// takes 16 us in both, the gather 12 and 16.)  The rest is latency in a chain: three digits of
// counting, cluster barrier and scan, the placing, the gather's two dependent
// loads.
// evict_gather_kernel: a copy, 16 bytes a lane, source pages never written.
#pragma once

#include "chunk_common.cuh"

namespace cosa {

struct EvictParams {
  const float* mass;  // [B][H_kv][mass_stride]
  const int32_t* kv_len;
  const int32_t* page_table;
  const int32_t* dst_table;  // [B][dst_pages]
  __nv_bfloat16 *k_pool, *v_pool;
  int32_t* kept;     // [B][H_kv][budget]
  int32_t* new_len;  // [B]
  float* mass_out;   // [B][H_kv][dst_pages * P] or null
  long long mass_stride;
  int num_kv_heads, page_size, pages_per_seq, num_phys_pages, max_kv, dst_pages;
  int budget, sink, recent;
};

constexpr int EVICT_CL = 8;
constexpr int EVICT_THREADS = 512;
constexpr int EVICT_BINS = 2048;
constexpr int EVICT_SLICE = EVICT_BINS / EVICT_CL;  // bins that a CTA sums
constexpr int EVICT_SEG_MAX = 40960;  // keys of a segment in shared memory (160 KB)

// Larger float, larger key; -0 is +0; a NaN is below everything.
__device__ __forceinline__ uint32_t mass_key(float v) {
  if (v != v) return 0u;
  const uint32_t u = __float_as_uint(v + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
// its two halves: leaving the first means having come, the second waits for all
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}
// words of another CTA of the cluster at the same shared-memory offset
__device__ __forceinline__ uint4 ld_cluster4(const void* p, int rank) {
  const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p));
  uint32_t r;
  uint4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(r)
               : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_cluster(const void* p, int rank) {
  const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p));
  uint32_t r, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(r) : "memory");
  return v;
}

__device__ __forceinline__ void add_cluster(const void* p, int rank, uint32_t v) {
  const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p));
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(r), "r"(v) : "memory");
}

// Exclusive prefix sum over the block; total gets the sum.  red: 32 words.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* red, uint32_t& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) red[warp] = inc;
  __syncthreads();
  uint32_t w = lane < (int)(blockDim.x >> 5) ? red[lane] : 0u;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const uint32_t before = warp ? __shfl_sync(0xffffffffu, w, warp - 1) : 0u;
  __syncthreads();
  return before + inc - v;
}

// HELD: the segment's keys are kept in dynamic shared memory; else they are read again from
// the masses in every pass (caches past 8 * 40960 keys).
template <bool HELD>
__global__ void __cluster_dims__(EVICT_CL, 1, 1) __launch_bounds__(EVICT_THREADS)
    evict_select_kernel(const EvictParams p) {
  extern __shared__ uint32_t keys_s[];
  __shared__ __align__(16) uint32_t hist[3][EVICT_BINS];  // this CTA's counts of each digit
  // the cluster's counts: this CTA's slice of the bins
  __shared__ __align__(16) uint32_t sums[3][EVICT_SLICE];
  __shared__ uint32_t red[32];
  __shared__ uint32_t found[2];  // digit, keys above it
  __shared__ uint32_t cnt_s[2];  // this CTA's keys above / at the border
  __shared__ uint32_t warp_s[2][EVICT_THREADS / 32];
  const int tid = threadIdx.x, rank = blockIdx.x, warp = tid >> 5, lane = tid & 31;
  const int hk = blockIdx.y, b = blockIdx.z;
  pdl_launch();
  const int kv = __ldg(p.kv_len + b);
  if (kv < 0 || kv > p.max_kv) {
    if (tid == 0) set_status(COSA_ERR_INVALID_ARG);
    return;  // the whole cluster
  }
  const long long bh = (long long)b * p.num_kv_heads + hk;
  int32_t* kept = p.kept + bh * p.budget;
  const int gtid = rank * EVICT_THREADS + tid, gstep = EVICT_CL * EVICT_THREADS;
  if (kv <= p.budget) {
    for (int j = gtid; j < p.budget; j += gstep) kept[j] = j < kv ? j : -1;
    return;
  }
  for (int j = gtid; j < p.sink; j += gstep) kept[j] = j;
  for (int j = gtid; j < p.recent; j += gstep) kept[p.budget - p.recent + j] = kv - p.recent + j;
  uint32_t want = p.budget - p.sink - p.recent;  // of the candidates
  if (want == 0) return;
  const int m = kv - p.sink - p.recent;  // > want
  const int seg = (m + EVICT_CL - 1) / EVICT_CL;
  const int s0 = min(rank * seg, m), n = min(s0 + seg, m) - s0;
  const float* mass = p.mass + bh * p.mass_stride + p.sink + s0;
  auto key = [&](int i) { return HELD ? keys_s[i] : mass_key(__ldg(mass + i)); };
  for (int i = tid; i < 3 * EVICT_BINS / 4; i += EVICT_THREADS)
    reinterpret_cast<uint4*>(hist)[i] = make_uint4(0u, 0u, 0u, 0u);
  for (int i = tid; i < 3 * EVICT_SLICE; i += EVICT_THREADS) sums[0][i] = 0u;
  if (HELD) {
    int i = tid;
    for (; i + 7 * EVICT_THREADS < n; i += 8 * EVICT_THREADS) {
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = __ldg(mass + i + e * EVICT_THREADS);
#pragma unroll
      for (int e = 0; e < 8; ++e) keys_s[i + e * EVICT_THREADS] = mass_key(v[e]);
    }
    for (; i < n; i += EVICT_THREADS) keys_s[i] = mass_key(__ldg(mass + i));
  }
  cluster_sync();  // every CTA's sums are zero before any is added to
  uint32_t prefix = 0;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
    const int bits = pass == 2 ? 10 : 11;
    const int top = shift + bits;
    uint32_t* h = hist[pass];
    const uint32_t mask = (1u << bits) - 1u;
    if (pass == 0 || prefix == 0x80000000u >> top) {
      // masses of exactly zero (keys that no token has seen) come in numbers: a warp counts its
      // own with one addition
      for (int i0 = 0; i0 < n; i0 += EVICT_THREADS) {
        const int i = i0 + tid;
        const uint32_t k = i < n ? key(i) : 0u;
        const bool in = i < n && (pass == 0 || (k >> top) == prefix);
        const uint32_t zero = __ballot_sync(0xffffffffu, in && k == 0x80000000u);
        if (in && k != 0x80000000u) atomicAdd(h + ((k >> shift) & mask), 1u);
        if (zero && lane == 0) atomicAdd(h + ((0x80000000u >> shift) & mask), (uint32_t)__popc(zero));
      }
    } else {
#pragma unroll 4
      for (int i = tid; i < n; i += EVICT_THREADS) {
        const uint32_t k = key(i);
        if ((k >> top) == prefix) atomicAdd(h + ((k >> shift) & mask), 1u);
      }
    }
    __syncthreads();
    // a thread's four bins into the slices that their owners hold; few are not empty
    const int bin0 = EVICT_BINS - 4 - 4 * tid;
    const uint4 own = *reinterpret_cast<const uint4*>(&hist[pass][bin0]);
    uint32_t* at = &sums[pass][bin0 % EVICT_SLICE];
    const int owner = bin0 / EVICT_SLICE;
    if (own.x) add_cluster(at, owner, own.x);
    if (own.y) add_cluster(at + 1, owner, own.y);
    if (own.z) add_cluster(at + 2, owner, own.z);
    if (own.w) add_cluster(at + 3, owner, own.w);
    cluster_sync();
    // from the largest digit down: the digit at which `want` keys are reached
    const uint4 t4 = ld_cluster4(at, owner);
    const uint32_t c[4] = {t4.w, t4.z, t4.y, t4.x};
    const uint32_t sum = c[0] + c[1] + c[2] + c[3];
    uint32_t total;
    uint32_t above = block_scan(sum, red, total);
    if (above < want && above + sum >= want) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (above < want && above + c[e] >= want) {
          found[0] = bin0 + 3 - e;
          found[1] = above;
        }
        above += c[e];
      }
    }
    __syncthreads();
    prefix = (prefix << bits) | found[0];
    want -= found[1];
    __syncthreads();
  }
  // keys above the border value are kept, of the equal ones the first `want`.  A warp owns a
  // contiguous run of the segment: its counts, then its place in the list.
  const int run = ((n + EVICT_THREADS - 1) / EVICT_THREADS) * 32;
  const int r0 = min(warp * run, n), r1 = min(r0 + run, n);
  uint32_t gt = 0, eq = 0;
  for (int i0 = r0; i0 < r1; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t k = i < r1 ? key(i) : 0u;
    gt += __popc(__ballot_sync(0xffffffffu, i < r1 && k > prefix));
    eq += __popc(__ballot_sync(0xffffffffu, i < r1 && k == prefix));
  }
  if (lane == 0) {
    warp_s[0][warp] = gt;
    warp_s[1][warp] = eq;
  }
  __syncthreads();
  uint32_t g0 = 0, e0 = 0;  // keys above / equal before this warp's run
  {
    const uint32_t g = lane < EVICT_THREADS / 32 ? warp_s[0][lane] : 0u;
    const uint32_t q = lane < EVICT_THREADS / 32 ? warp_s[1][lane] : 0u;
    if (warp == 0) {
      const int tg = warp_sum_int((int)g), tq = warp_sum_int((int)q);
      if (lane == 0) {
        cnt_s[0] = tg;
        cnt_s[1] = tq;
      }
    }
    g0 = warp_sum_int(lane < warp ? (int)g : 0);
    e0 = warp_sum_int(lane < warp ? (int)q : 0);
  }
  cluster_sync();
  {  // and in the segments before this one
    const bool other = lane < rank;
    g0 += warp_sum_int(other ? (int)ld_cluster(&cnt_s[0], other ? lane : 0) : 0);
    e0 += warp_sum_int(other ? (int)ld_cluster(&cnt_s[1], other ? lane : 0) : 0);
  }
  cluster_arrive();  // the others' counts are read; they may leave once all have come this far
  const uint32_t below = (1u << lane) - 1u;
  for (int i0 = r0; i0 < r1; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t k = i < r1 ? key(i) : 0u;
    const bool above = i < r1 && k > prefix, equal = i < r1 && k == prefix;
    const uint32_t bg = __ballot_sync(0xffffffffu, above), be = __ballot_sync(0xffffffffu, equal);
    const uint32_t eb = e0 + __popc(be & below);
    if (above || (equal && eb < want))
      kept[p.sink + g0 + __popc(bg & below) + min(eb, want)] = p.sink + s0 + i;
    g0 += __popc(bg);
    e0 += __popc(be);
  }
  cluster_wait();
}

constexpr int GATHER_THREADS = 256;
constexpr int GATHER_UNROLL = 4;

// grid (blocks of kept rows, H_kv, B)
template <int D>
__global__ void __launch_bounds__(GATHER_THREADS) evict_gather_kernel(const EvictParams p) {
  constexpr int LPR = D / 8;                     // lanes a row, 16 bytes each
  constexpr int RPB = GATHER_THREADS / LPR;      // rows a pass
  const int hk = blockIdx.y, b = blockIdx.z;
  pdl_wait();
  const int kv = __ldcg(p.kv_len + b);  // new_len may be written over it: the same minimum
  if (kv < 0 || kv > p.max_kv) return;
  const int n = min(kv, p.budget);
  if (blockIdx.x == 0 && hk == 0 && threadIdx.x == 0) p.new_len[b] = n;
  const long long bh = (long long)b * p.num_kv_heads + hk;
  const int32_t* kept = p.kept + bh * p.budget;
  const int r0 = blockIdx.x * RPB * GATHER_UNROLL + threadIdx.x / LPR, l = threadIdx.x % LPR;
  long long from[GATHER_UNROLL], to[GATHER_UNROLL];
  int src[GATHER_UNROLL];
#pragma unroll
  for (int e = 0; e < GATHER_UNROLL; ++e) {
    const int j = r0 + e * RPB;
    src[e] = j < n ? __ldcg(kept + j) : -1;
  }
#pragma unroll
  for (int e = 0; e < GATHER_UNROLL; ++e) {
    const int j = r0 + e * RPB;
    from[e] = to[e] = -1;
    if (src[e] < 0 || src[e] >= p.max_kv) continue;
    const int ps = __ldg(p.page_table + (long long)b * p.pages_per_seq + src[e] / p.page_size);
    const int pd = __ldg(p.dst_table + (long long)b * p.dst_pages + j / p.page_size);
    const bool from_ok = ps >= 0 && ps < p.num_phys_pages, to_ok = pd >= 0 && pd < p.num_phys_pages;
    if (!(from_ok && to_ok) && l == 0) set_status(COSA_ERR_INVALID_ARG);
    if (!to_ok) continue;
    to[e] = (((long long)pd * p.num_kv_heads + hk) * p.page_size + j % p.page_size) * LPR + l;
    if (from_ok)
      from[e] = (((long long)ps * p.num_kv_heads + hk) * p.page_size + src[e] % p.page_size) * LPR + l;
  }
  // a key of a page outside the pool reads as zeros, here as in the attention: its slot must not
  // keep what the new page held
  uint4 k[GATHER_UNROLL], v[GATHER_UNROLL];
#pragma unroll
  for (int e = 0; e < GATHER_UNROLL; ++e) {
    k[e] = v[e] = make_uint4(0u, 0u, 0u, 0u);
    if (from[e] >= 0) {
      k[e] = reinterpret_cast<const uint4*>(p.k_pool)[from[e]];
      v[e] = reinterpret_cast<const uint4*>(p.v_pool)[from[e]];
    }
  }
#pragma unroll
  for (int e = 0; e < GATHER_UNROLL; ++e)
    if (to[e] >= 0) {
      reinterpret_cast<uint4*>(p.k_pool)[to[e]] = k[e];
      reinterpret_cast<uint4*>(p.v_pool)[to[e]] = v[e];
    }
  if (p.mass_out && l == 0) {
    float* mo = p.mass_out + bh * ((long long)p.dst_pages * p.page_size);
#pragma unroll
    for (int e = 0; e < GATHER_UNROLL; ++e) {
      const int j = r0 + e * RPB;
      if (j < n && src[e] >= 0 && src[e] < p.max_kv)
        mo[j] = __ldg(p.mass + bh * p.mass_stride + src[e]);
    }
  }
}

}  // namespace cosa
