// Shared pieces of the chunk kernels (cosa_chunk_write, cosa_chunk_attention,
// cosa_attention_mass, cosa_cache_evict): a ragged batch's lengths, the range of keys a
// token sees, and the score's shape.
#pragma once

#include <limits.h>

#include "common.cuh"
#include "tc_ptx.cuh"

namespace cosa {

// ---- PTX wrappers that only the chunk kernels use
namespace tc {
// One lane of a converged warp (1 for it, 0 for the others).
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r;
}
// The MMAs and the commit of tc_ptx.cuh, predicated on `on`: a warp in uniform control flow
// issues them from the lane that elect_one chose, without a branch.
__device__ __forceinline__ void mma_bf16_ss_if(uint32_t on, uint32_t d_tmem, uint64_t a_desc,
                                               uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(on)
      : "memory");
}
__device__ __forceinline__ void mma_bf16_ts_if(uint32_t on, uint32_t d_tmem, uint32_t a_tmem,
                                               uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(on)
      : "memory");
}
__device__ __forceinline__ void mma_commit_if(uint32_t on, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(on)
      : "memory");
}
__device__ __forceinline__ uint32_t ld_shared_volatile(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_shared_volatile(uint32_t addr, uint32_t v) {
  asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
}  // namespace tc

constexpr int CHUNK_MAX_BATCH = 4096;
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
  hi = min(max(pos, max(prefix, 0) - 1), kv - 1);
}

// The first key that the window leaves to the token at position pos and to those after it.  Pages
// before it read as zeros whatever the page table says: a server gives them up, and their entries
// may name nothing, or a page that holds something else by now (NaN too, which a weight of zero
// would not keep out of the second product).
__device__ __forceinline__ int window_start(const ChunkMask& m, int pos) {
  return m.window > 0 ? pos - m.window + 1 : 0;
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
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 both(float a) { return pack2(a, a); }

// Scores in log2 units from raw products.  Plain: raw * a.  Capped: with y = raw * scale / c,
// by the size of y:
//   |y| <= 0.625   c (y + y z q(z)), z = y^2: an odd polynomial of degree 9 (least absolute error of
//                  the tanh on that range, 4.3e-8; of the score 2^-22.1), on the FMA pipe
//   beyond         c tanh(y) = c - 2c / (1 + e^2y), the exponential and the reciprocal on the
//                  special-function unit: absolute error about c * 2^-23, a score's own rounding
//                  here, but for a small score under a large cap all of it (9e-3 at a cap of
//                  10^5).  (The hardware tanh, relative error 2^-11, would move a logit near a cap
//                  of 50 by 0.02.)
// The first form leaves the special-function unit two results an element: the tiled attention and the
// mass take it (CAP_NEAR) where all of a warp's scores are in its range, the usual case.  For the
// others:
//   CAP_FAR   the second form for all scores: the tiled attention under caps up to 64, where its error is at
//             most 2^-17, two roundings of a score of 64, and far below that of its weights
//   CAP_EACH  chosen for each score: the tiled attention under larger caps, the mass (a sum of weights
//             as they are), the single-token form for all scores.  (In the tiled attention on packed
//             documents, scores beyond their cap of 2: 276 against 242 us.  In the mass of 64 tokens on
//             64K keys, where CAP_FAR for all takes 121 us whatever the cap: 90 us under a cap of 30,
//             149 under one of 2.  In the single-token form, bound by its bytes, 200 us for 32 ragged
//             sequences either way.)
enum CapForm { CAP_NONE, CAP_NEAR, CAP_FAR, CAP_EACH };
constexpr float kCapFarMax = 64.f;
struct ScoreShape {
  float a;    // scale * log2 e
  float e2;   // capped: 2 * scale / c * log2 e
  float cap;  // capped: c * log2 e
  float y;    // capped: scale / c
  float lim;  // capped: the raw product at y = 0.625
};

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float cap_far(const ScoreShape& s, float raw) {
  return fmaf(-2.f * s.cap, rcp_approx(1.f + tc::ex2_approx(raw * s.e2)), s.cap);
}

// A pair of scores in log2 units plus `add`; CAP_NEAR: both products are within s.lim.
template <CapForm FORM>
__device__ __forceinline__ f32x2 score2_log2(const ScoreShape& s, f32x2 raw, f32x2 add) {
  if (FORM == CAP_NONE) return fma2(raw, both(s.a), add);
  float r0, r1;
  unpack2(raw, r0, r1);
  if (FORM == CAP_FAR) return add2(pack2(cap_far(s, r0), cap_far(s, r1)), add);
  const f32x2 y = mul2(raw, both(s.y)), z = mul2(y, y);
  f32x2 q = fma2(z, both(0.0148892366f), both(-0.0517016767f));
  q = fma2(q, z, both(0.133020084f));
  q = fma2(q, z, both(-0.333318751f));
  const f32x2 x = mul2(raw, both(s.a)), qz = mul2(q, z);
  if (FORM == CAP_NEAR) return fma2(x, qz, fma2(raw, both(s.a), add));
  float x0, x1;
  unpack2(fma2(x, qz, x), x0, x1);
  return add2(pack2(fabsf(r0) <= s.lim ? x0 : cap_far(s, r0), fabsf(r1) <= s.lim ? x1 : cap_far(s, r1)), add);
}

// The waiting itself, kept out of line: two dozen inlined copies of these loops would not
// leave the instruction cache room for the loops that work.
__device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, uint32_t abort_at,
                                     unsigned long long tmo) {
  const uint64_t t0 = tc::globaltimer_ns();
  while (!tc::mbar_try_wait(bar, parity)) {
    if (tc::ld_shared_volatile(abort_at)) return false;
    if (*(volatile int*)&g_status == COSA_ERR_TIMEOUT || tc::globaltimer_ns() - t0 > tmo) {
      tc::st_shared_volatile(abort_at, 1u);
      set_status(COSA_ERR_TIMEOUT);
      return false;
    }
  }
  return true;
}
__device__ __noinline__ bool wait_on_hot(uint32_t bar, uint32_t parity, uint32_t abort_at,
                                         unsigned long long tmo) {
  const uint64_t t0 = tc::globaltimer_ns();
  uint32_t n = 0;
  while (!tc::mbar_test_wait(bar, parity)) {
    if ((++n & 255u) == 0) {
      if (tc::ld_shared_volatile(abort_at)) return false;
      if (*(volatile int*)&g_status == COSA_ERR_TIMEOUT || tc::globaltimer_ns() - t0 > tmo) {
        tc::st_shared_volatile(abort_at, 1u);
        set_status(COSA_ERR_TIMEOUT);
        return false;
      }
    }
  }
  return true;
}

// Programmatic dependent launch: wait for the kernels before this one in the stream, and
// let the next one start its prologue.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace cosa
