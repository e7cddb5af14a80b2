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

// Programmatic dependent launch: wait for the kernels before this one in the stream, and
// let the next one start its prologue.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace cosa
