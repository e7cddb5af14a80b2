// Eviction by accumulated attention mass: per (sequence, KV head) the sink and recent keys
// and the heaviest others up to a budget, then a gather of their K, V and mass into new
// pages.
//
// evict_select_kernel: one cluster of 8 CTAs per (b, h_kv); each CTA owns a contiguous
// eighth of the candidates.  The K-th largest mass is found by a radix select over the
// order-preserving 32-bit form of the float (digits of 11, 11 and 10 bits: three passes
// over the masses, which stay in L2), the eight histograms summed through distributed
// shared memory.  Equal masses at the border go to the lowest positions: the CTAs' counts
// of larger and of equal keys give each one its place, so the kept list comes out ascending
// and is the same on every run.
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

// Larger float, larger key; -0 is +0; a NaN is below everything.
__device__ __forceinline__ uint32_t mass_key(float v) {
  if (v != v) return 0u;
  const uint32_t u = __float_as_uint(v + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
// word of another CTA of the cluster at the same shared-memory offset
__device__ __forceinline__ uint32_t ld_cluster(const void* p, int rank) {
  const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p));
  uint32_t r, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(r) : "memory");
  return v;
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

__global__ void __cluster_dims__(EVICT_CL, 1, 1) __launch_bounds__(EVICT_THREADS)
    evict_select_kernel(const EvictParams p) {
  __shared__ uint32_t hist[EVICT_BINS];
  __shared__ uint32_t slice[EVICT_BINS / EVICT_CL];
  __shared__ uint32_t red[32];
  __shared__ uint32_t found[2];  // digit, keys above it
  __shared__ uint32_t cnt_s[2];  // this CTA's keys above / at the border
  const int tid = threadIdx.x, rank = blockIdx.x;
  const int hk = blockIdx.y, b = blockIdx.z;
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
  const int s0 = min(rank * seg, m), s1 = min(s0 + seg, m);
  const float* mass = p.mass + bh * p.mass_stride + p.sink;
  uint32_t prefix = 0;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
    const int bits = pass == 2 ? 10 : 11;
    for (int i = tid; i < EVICT_BINS; i += EVICT_THREADS) hist[i] = 0;
    __syncthreads();
    for (int i = s0 + tid; i < s1; i += EVICT_THREADS) {
      const uint32_t k = mass_key(__ldg(mass + i));
      if (pass == 0 || (k >> (shift + bits)) == prefix)
        atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1u)], 1u);
    }
    cluster_sync();
    // this CTA sums its eighth of the bins over the cluster
    if (tid < EVICT_BINS / EVICT_CL) {
      uint32_t t = 0;
#pragma unroll
      for (int r = 0; r < EVICT_CL; ++r) t += ld_cluster(&hist[rank * (EVICT_BINS / EVICT_CL) + tid], r);
      slice[tid] = t;
    }
    cluster_sync();
    // from the largest digit down: the digit at which `want` keys are reached
    uint32_t c[4], sum = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int bin = EVICT_BINS - 1 - (4 * tid + e);
      c[e] = ld_cluster(&slice[bin % (EVICT_BINS / EVICT_CL)], bin / (EVICT_BINS / EVICT_CL));
      sum += c[e];
    }
    uint32_t total;
    uint32_t above = block_scan(sum, red, total);
    if (above < want && above + sum >= want) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (above < want && above + c[e] >= want) {
          found[0] = EVICT_BINS - 1 - (4 * tid + e);
          found[1] = above;
        }
        above += c[e];
      }
    }
    __syncthreads();
    prefix = (prefix << bits) | found[0];
    want -= found[1];
  }
  // keys above the border value are kept, of the equal ones the first `want`
  uint32_t gt = 0, eq = 0;
  for (int i = s0 + tid; i < s1; i += EVICT_THREADS) {
    const uint32_t k = mass_key(__ldg(mass + i));
    gt += k > prefix;
    eq += k == prefix;
  }
  uint32_t tg, te;
  block_scan(gt, red, tg);
  block_scan(eq, red, te);
  if (tid == 0) {
    cnt_s[0] = tg;
    cnt_s[1] = te;
  }
  cluster_sync();
  uint32_t g0 = 0, e0 = 0;  // keys above / equal in the segments before this one
  for (int r = 0; r < rank; ++r) {
    g0 += ld_cluster(&cnt_s[0], r);
    e0 += ld_cluster(&cnt_s[1], r);
  }
  for (int base = s0; base < s1; base += 4 * EVICT_THREADS) {
    uint32_t k[4], mine = 0;  // keys above in the upper half, equal in the lower
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = base + 4 * tid + e;
      k[e] = i < s1 ? mass_key(__ldg(mass + i)) : 0u;
      if (i < s1) mine += (k[e] > prefix ? 0x10000u : 0u) + (k[e] == prefix ? 1u : 0u);
    }
    uint32_t total;
    const uint32_t before = block_scan(mine, red, total);
    uint32_t gb = g0 + (before >> 16), eb = e0 + (before & 0xffffu);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = base + 4 * tid + e;
      if (i < s1) {
        const bool above = k[e] > prefix, equal = k[e] == prefix;
        if (above || (equal && eb < want)) kept[p.sink + gb + min(eb, want)] = p.sink + i;
        gb += above;
        eb += equal;
      }
    }
    g0 += total >> 16;
    e0 += total & 0xffffu;
  }
  cluster_sync();  // the counts above are read by the others
}

constexpr int GATHER_THREADS = 256;
constexpr int GATHER_UNROLL = 4;

// grid (blocks of kept rows, H_kv, B)
template <int D>
__global__ void __launch_bounds__(GATHER_THREADS) evict_gather_kernel(const EvictParams p) {
  constexpr int LPR = D / 8;                     // lanes a row, 16 bytes each
  constexpr int RPB = GATHER_THREADS / LPR;      // rows a pass
  const int hk = blockIdx.y, b = blockIdx.z;
  const int kv = __ldg(p.kv_len + b);  // new_len may be written over it: the same minimum
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
    src[e] = j < n ? __ldg(kept + j) : -1;
  }
#pragma unroll
  for (int e = 0; e < GATHER_UNROLL; ++e) {
    const int j = r0 + e * RPB;
    from[e] = -1;
    if (src[e] < 0 || src[e] >= p.max_kv) continue;
    const int ps = __ldg(p.page_table + (long long)b * p.pages_per_seq + src[e] / p.page_size);
    const int pd = __ldg(p.dst_table + (long long)b * p.dst_pages + j / p.page_size);
    if (ps < 0 || ps >= p.num_phys_pages || pd < 0 || pd >= p.num_phys_pages) {
      if (l == 0) set_status(COSA_ERR_INVALID_ARG);
      continue;
    }
    from[e] = (((long long)ps * p.num_kv_heads + hk) * p.page_size + src[e] % p.page_size) * LPR + l;
    to[e] = (((long long)pd * p.num_kv_heads + hk) * p.page_size + j % p.page_size) * LPR + l;
  }
  uint4 k[GATHER_UNROLL], v[GATHER_UNROLL];
#pragma unroll
  for (int e = 0; e < GATHER_UNROLL; ++e)
    if (from[e] >= 0) {
      k[e] = reinterpret_cast<const uint4*>(p.k_pool)[from[e]];
      v[e] = reinterpret_cast<const uint4*>(p.v_pool)[from[e]];
    }
#pragma unroll
  for (int e = 0; e < GATHER_UNROLL; ++e)
    if (from[e] >= 0) {
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
