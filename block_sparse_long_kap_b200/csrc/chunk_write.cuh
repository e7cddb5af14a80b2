// Rotary positions with several axes, fused with the write of a chunk's Q, K, V: token-major
// inputs (possibly views of a fused projection) to token-major Q and the paged cache.
//
// Pair (x, y) of a head turns by w = positions[axis][token] * inv_freq[pair]:
//   x' = x cos w - y sin w,  y' = y cos w + x sin w.
// w / 2 pi is taken in fp64 and reduced to [-1/2, 1/2] turns before the fp32 sine and
// cosine: at position 10^6 an fp32 angle is off by 0.06 rad.  One (cos, sin) per token and
// pair serves all heads, so the table of a CTA's tokens is made once in shared memory.
// The work is the copy: every element is read and written once, 16 bytes a lane.
//
// Measured: 32K tokens of 80 heads (1.33 GB) 224 us, 0.91 of a copy's rate; 8,191 tokens of 36
// heads (151 MB) 33 us called, 30.5 replayed, 23 of them its bytes': each CTA's first loads come behind its page
// lookup, its table and a barrier, and the issue slots are 56 % busy, a division a unit among what
// fills them; a decode step of 64 sequences 3.3 us, its table and one trip to memory.  Deeper unrolling (2 to 4 units a thread
// in flight) took 249 to 364 us for the first.
#pragma once

#include "chunk_common.cuh"

namespace cosa {

struct ChunkWriteParams {
  ChunkSeqs seqs;
  const __nv_bfloat16 *q_tok, *k_tok, *v_tok;
  __nv_bfloat16 *q, *k_pool, *v_pool;
  long long q_tok_stride, k_tok_stride, v_tok_stride, q_stride;
  const int32_t* positions;  // [axes][total_q]
  const float* inv_freq;     // [half]
  const int32_t* page_table;
  int num_q_heads, num_kv_heads, page_size, pages_per_seq, num_phys_pages;
  int half;         // rotated pairs (a multiple of 8)
  int axes, interleaved, adjacent;
  int sections[COSA_MAX_ROPE_AXES];
  int tokens_per_cta, units_per_part;  // a unit: 32 bytes of a head, one thread
};

constexpr int CHUNK_WRITE_THREADS = 256;

__device__ __forceinline__ int rope_axis(const ChunkWriteParams& p, int j) {
  if (p.interleaved) {
    const int a = j % p.axes;
    int s = p.sections[0];
#pragma unroll
    for (int k = 1; k < COSA_MAX_ROPE_AXES; ++k)
      if (a == k) s = p.sections[k];
    return (a > 0 && j < p.axes * s) ? a : 0;
  }
  int a = 0, end = p.sections[0];
#pragma unroll
  for (int k = 1; k < COSA_MAX_ROPE_AXES; ++k) {
    if (k < p.axes && j >= end) a = k;
    end += p.sections[k];
  }
  return a;
}

__device__ __forceinline__ void unpack8(const uint4& v, float* f) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = __bfloat1622float2(h[i]);
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}
__device__ __forceinline__ uint4 pack8(const float* f) {
  uint4 v;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
  return v;
}

// What the kernel below does not find where cu_q goes back: there its count of ends is no guide to a
// token's sequence, and a token may have several.  A CTA of its own looks every sequence's lengths
// over, and in that case writes the rows of a token's other sequences, or of all of them where the
// counted one is not its own.  (Such a cu_q is an error and recorded as one; the sequences that are
// sound have to come out whole, not fast.)  q is written with a token's first sequence only: in
// place, a second turn would count.
__device__ __forceinline__ void chunk_write_look_over(const ChunkWriteParams& p, int D) {
  const int tid = threadIdx.x, hq = p.num_q_heads, hk = p.num_kv_heads;
  bool back = false;
  for (int b = tid; b < p.seqs.batch; b += CHUNK_WRITE_THREADS) {
    chunk_seq(p.seqs, b);
    back |= __ldg(p.seqs.cu_q + b + 1) < __ldg(p.seqs.cu_q + b);
  }
  if (!__syncthreads_or(back)) return;
  // a warp a token
  const int lane = tid & 31;
  for (int t = tid >> 5; t < p.seqs.total_q; t += CHUNK_WRITE_THREADS / 32) {
    int counted = 0;
    for (int b = lane; b < p.seqs.batch; b += 32) counted += __ldg(p.seqs.cu_q + b + 1) <= t;
    counted = warp_sum_int(counted);
    auto owns = [&](int b) {
      const ChunkSeq s = chunk_seq(p.seqs, b);
      return s.ok && t >= s.q0 && t < s.q0 + s.q_len;
    };
    bool with_q = counted >= p.seqs.batch || !owns(counted);
    for (int b0 = 0; b0 < p.seqs.batch; b0 += 32) {
      const int mine = b0 + lane;
      uint32_t owners = __ballot_sync(0xffffffffu, mine < p.seqs.batch && mine != counted && owns(mine));
      for (; owners; owners &= owners - 1) {
        const int b = b0 + __ffs(owners) - 1;
        const ChunkSeq s = chunk_seq(p.seqs, b);
        const int pos = s.kv - s.q_len + (t - s.q0);
        const int phys = __ldg(p.page_table + (long long)b * p.pages_per_seq + pos / p.page_size);
        const bool page = phys >= 0 && phys < p.num_phys_pages;
        if (!page) set_status(COSA_ERR_INVALID_ARG);
        const long long row = (long long)phys * hk * p.page_size + pos % p.page_size;
        // a lane's item: two elements of a head, a pair that turns together or two that stay
        for (int x = lane; x < (hq + 2 * hk) * (D / 2); x += 32) {
          const int h = x / (D / 2), j = x % (D / 2), g = h < hq ? h : (h - hq) % hk;
          const bool is_v = h >= hq + hk;
          if (h < hq ? !with_q : !page) continue;
          const __nv_bfloat16* src = h < hq ? p.q_tok + t * p.q_tok_stride
                                            : (is_v ? p.v_tok + t * p.v_tok_stride : p.k_tok + t * p.k_tok_stride);
          __nv_bfloat16* dst = h < hq ? p.q + t * p.q_stride + g * D
                                      : (is_v ? p.v_pool : p.k_pool) + (row + (long long)g * p.page_size) * D;
          src += g * D;
          const bool halves = j < p.half && !p.adjacent;
          const int e0 = halves ? j : 2 * j, e1 = halves ? j + p.half : 2 * j + 1;
          const __nv_bfloat16 x0 = src[e0], x1 = src[e1];
          if (is_v || j >= p.half) {
            dst[e0] = x0;
            dst[e1] = x1;
            continue;
          }
          // (not shared with the kernel below: in a common function it cost that a spilled register,
          // and 1 % of the time of 32K tokens)
          const int at = __ldg(p.positions + (long long)rope_axis(p, j) * p.seqs.total_q + t);
          const double w = (double)at * (double)__ldg(p.inv_freq + j) * 0.15915494309189533577;
          float sn, co;
          sincospif(2.f * (float)(w - rint(w)), &sn, &co);
          const float a = __bfloat162float(x0), c = __bfloat162float(x1);
          dst[e0] = __float2bfloat16_rn(a * co - c * sn);
          dst[e1] = __float2bfloat16_rn(c * co + a * sn);
        }
        with_q = false;
      }
    }
  }
}

// Six CTAs an SM (42 registers): 223 us for 32K tokens of 80 heads; with the compiler's 48 and five
// CTAs 232, with seven or eight 235.
// grid (token blocks and one CTA more, parts of a token's units); dynamic shared memory: (cos, sin) of
// tokens_per_cta * half pairs
template <int D>
__global__ void __launch_bounds__(CHUNK_WRITE_THREADS, 6)
    chunk_write_kernel(const ChunkWriteParams p) {
  constexpr int UPH = D / 16;  // units per head
  constexpr int MAX_TOK = 16;
  extern __shared__ float4 cs[];           // [token][4][half / 8]: pairs 8c + 2q, 8c + 2q + 1
  __shared__ long long row_s[MAX_TOK];     // cache row of head 0; -1: no page, -2: no token
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tok0 = blockIdx.x * p.tokens_per_cta;
  const int n = min(p.tokens_per_cta, p.seqs.total_q - tok0);
  const int half = p.half;
  if (n <= 0) {  // the CTA past the last token
    if (blockIdx.y == 0) chunk_write_look_over(p, D);
    return;
  }
  // the sequence of token t: the number of sequences that end at or before it
  for (int i = warp; i < n; i += CHUNK_WRITE_THREADS / 32) {
    const int t = tok0 + i;
    int cnt = 0;
    for (int k = lane; k < p.seqs.batch; k += 32) cnt += __ldg(p.seqs.cu_q + k + 1) <= t;
    const int b = warp_sum_int(cnt);
    if (lane == 0) {
      long long row = -2;
      if (b < p.seqs.batch) {
        const ChunkSeq s = chunk_seq(p.seqs, b);
        if (s.ok && t >= s.q0 && t < s.q0 + s.q_len) {
          const int pos = s.kv - s.q_len + (t - s.q0);
          const int phys = __ldg(p.page_table + (long long)b * p.pages_per_seq + pos / p.page_size);
          row = -1;
          if (phys >= 0 && phys < p.num_phys_pages)
            row = (long long)phys * p.num_kv_heads * p.page_size + pos % p.page_size;
          else
            set_status(COSA_ERR_INVALID_ARG);
        }
      }
      row_s[i] = row;
    }
  }
  for (int x = tid; x < n * half; x += CHUNK_WRITE_THREADS) {
    const int i = x / half, j = x - i * half;
    const int pos = __ldg(p.positions + (long long)rope_axis(p, j) * p.seqs.total_q + tok0 + i);
    const double turns = (double)pos * (double)__ldg(p.inv_freq + j) * 0.15915494309189533577;
    float sn, co;
    sincospif(2.f * (float)(turns - rint(turns)), &sn, &co);
    float2* e = reinterpret_cast<float2*>(cs + (i * 4 + ((j & 7) >> 1)) * (half >> 3) + (j >> 3));
    e[j & 1] = make_float2(co, sn);
  }
  __syncthreads();
  const int units = (p.num_q_heads + 2 * p.num_kv_heads) * UPH;
  const int u0 = blockIdx.y * p.units_per_part;
  const int nu = min(p.units_per_part, units - u0);
  for (int x = tid; x < n * nu; x += CHUNK_WRITE_THREADS) {
    const int i = x / nu, u = u0 + x - i * nu;
    const long long row = row_s[i];
    if (row == -2) continue;
    int h = u / UPH;
    const int c = u % UPH;
    const long long t = tok0 + i;
    const __nv_bfloat16* src;
    __nv_bfloat16* dst;
    bool turn = true;
    if (h < p.num_q_heads) {
      src = p.q_tok + t * p.q_tok_stride + h * D;
      dst = p.q + t * p.q_stride + h * D;
    } else {
      if (row < 0) continue;
      h -= p.num_q_heads;
      const bool is_k = h < p.num_kv_heads;
      if (!is_k) h -= p.num_kv_heads;
      src = (is_k ? p.k_tok + t * p.k_tok_stride : p.v_tok + t * p.v_tok_stride) + h * D;
      dst = (is_k ? p.k_pool : p.v_pool) + (row + (long long)h * p.page_size) * D;
      turn = is_k;
    }
    // the unit's two 16-byte pieces: partners of the same pairs, or neighbours
    turn = turn && 8 * c < half;
    int c0 = 2 * c, c1 = 2 * c + 1;
    if (!p.adjacent) {
      if (8 * c < half) {
        c0 = c;
        c1 = c + (half >> 3);
      }
      // pieces past the rotated dims keep their place: unit c >= half / 8 holds 2c, 2c + 1
    }
    const uint4 r0 = reinterpret_cast<const uint4*>(src)[c0];
    const uint4 r1 = reinterpret_cast<const uint4*>(src)[c1];
    if (!turn) {
      reinterpret_cast<uint4*>(dst)[c0] = r0;
      reinterpret_cast<uint4*>(dst)[c1] = r1;
      continue;
    }
    float a[8], b[8];
    unpack8(r0, a);
    unpack8(r1, b);
    const float4* w = cs + i * 4 * (half >> 3) + c;
    if (p.adjacent) {
      // pairs 8c .. 8c + 3 in the first piece, 8c + 4 .. 8c + 7 in the second
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float4 f = w[q * (half >> 3)];
        float* e = q < 2 ? a + 4 * q : b + 4 * (q - 2);
        const float x0 = e[0], y0 = e[1], x1 = e[2], y1 = e[3];
        e[0] = x0 * f.x - y0 * f.y;
        e[1] = y0 * f.x + x0 * f.y;
        e[2] = x1 * f.z - y1 * f.w;
        e[3] = y1 * f.z + x1 * f.w;
      }
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float4 f = w[q * (half >> 3)];
        const float x0 = a[2 * q], y0 = b[2 * q], x1 = a[2 * q + 1], y1 = b[2 * q + 1];
        a[2 * q] = x0 * f.x - y0 * f.y;
        b[2 * q] = y0 * f.x + x0 * f.y;
        a[2 * q + 1] = x1 * f.z - y1 * f.w;
        b[2 * q + 1] = y1 * f.z + x1 * f.w;
      }
    }
    reinterpret_cast<uint4*>(dst)[c0] = pack8(a);
    reinterpret_cast<uint4*>(dst)[c1] = pack8(b);
  }
}

}  // namespace cosa
