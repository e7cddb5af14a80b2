// Shared pieces of the chunk kernels (cosa_chunk_write, cosa_chunk_attention,
// cosa_attention_mass, cosa_cache_evict): a ragged batch's lengths, the range of keys a
// token sees, and the score's shape.
#pragma once

#include <limits.h>

#include "common.cuh"
#include "tc_ptx.cuh"

namespace cosa {

constexpr int CHUNK_MAX_BATCH = 8192;
constexpr int NUM_SMS = 148;  // B200

struct ChunkSeqs {
  const int32_t* cu_q;    // [B + 1]
  const int32_t* kv_len;  // [B]
  int batch, total_q, max_q, max_kv;
};

struct ChunkSeq {
  int q0, q_len, kv;
  bool ok;  // has new tokens and consistent lengths
};

// Lengths of sequence b; an inconsistent one is reported and counts as having no tokens.
__device__ __forceinline__ ChunkSeq chunk_seq(const ChunkSeqs& s, int b) {
  ChunkSeq r;
  const int q0 = __ldg(s.cu_q + b), q1 = __ldg(s.cu_q + b + 1);
  const int kv = __ldg(s.kv_len + b);
  const bool sane = q0 >= 0 && q1 >= q0 && q1 <= s.total_q && q1 - q0 <= s.max_q &&
                    kv <= s.max_kv && (q1 == q0 || q1 - q0 <= kv);
  if (!sane) set_status(COSA_ERR_INVALID_ARG);
  r.q0 = q0;
  r.q_len = sane ? q1 - q0 : 0;
  r.kv = kv;
  r.ok = r.q_len > 0;
  return r;
}

// Which keys a token sees: an interval [lo, hi] of cache positions (lo > hi: none).
struct ChunkMask {
  const int32_t* first_key;   // [total_q] or null
  const int32_t* prefix_len;  // [B] or null
  int window;
};

__device__ __forceinline__ void token_range(const ChunkMask& m, int token, int pos, int kv,
                                            int prefix, int& lo, int& hi) {
  lo = m.first_key ? max(__ldg(m.first_key + token), 0) : 0;
  if (m.window > 0) lo = max(lo, pos - m.window + 1);
  hi = min(max(pos, prefix - 1), kv - 1);
}

// Score in log2 units from the raw product.  Plain: raw * a.  Capped:
// c tanh(raw * scale / c) = c - 2c / (1 + e^(2 raw scale / c)), with the exponential and
// the reciprocal on the special-function unit: absolute error about c * 2^-23, where the
// hardware tanh (relative error 2^-11) would move a logit near a cap of 50 by 0.02.
struct ScoreShape {
  float a;      // plain: scale * log2 e; capped: 2 * scale / c * log2 e
  float cap2;   // c * log2 e
};

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <bool CAP>
__device__ __forceinline__ float score_log2(const ScoreShape& s, float raw) {
  if (!CAP) return raw * s.a;
  const float r = rcp_approx(1.f + tc::ex2_approx(raw * s.a));
  return fmaf(-2.f * s.cap2, r, s.cap2);
}

// Pairs of floats in one 64-bit register: the FMA pipe takes both in one instruction.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pack2(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(f32x2 v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// 2^x of a pair on the FMA pipe, for x <= 127: x = n + f with n the nearest integer (taken
// from the low mantissa bits of x + 1.5 * 2^23, after Cody and Waite), 2^f on [-1/2, 1/2] by
// a degree-4 polynomial of least relative error (2.6e-6, far below the 2^-9 of the bf16
// weights), n added to the exponent.  x below -126 gives 2^-126.
__device__ __forceinline__ f32x2 exp2_poly2(f32x2 x) {
  float x0, x1;
  unpack2(x, x0, x1);
  x = pack2(fmaxf(x0, -126.f), fmaxf(x1, -126.f));
  const f32x2 magic = pack2(12582912.f, 12582912.f), neg = pack2(-12582912.f, -12582912.f);
  const f32x2 t = add2(x, magic);
  const f32x2 f = fma2(add2(t, neg), pack2(-1.f, -1.f), x);
  f32x2 p = pack2(0.00957010179f, 0.00957010179f);
  p = fma2(p, f, pack2(0.0559178603f, 0.0559178603f));
  p = fma2(p, f, pack2(0.240247448f, 0.240247448f));
  p = fma2(p, f, pack2(0.693121815f, 0.693121815f));
  p = fma2(p, f, pack2(0.999999261f, 0.999999261f));
  float t0, t1, p0, p1;
  unpack2(t, t0, t1);
  unpack2(p, p0, p1);
  return pack2(__int_as_float(__float_as_int(p0) + (__float_as_int(t0) << 23)),
               __int_as_float(__float_as_int(p1) + (__float_as_int(t1) << 23)));
}

// Programmatic dependent launch: wait for the kernels before this one in the stream, and
// let the next one start its prologue.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace cosa
