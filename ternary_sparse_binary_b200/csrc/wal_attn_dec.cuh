// Shared by the attention kernels of few query rows (wal_attn.cu, wal_attn_ring.cu).
#pragma once

#include "wal_attn.h"

namespace wal {

namespace {

constexpr int kDecWarps = 4;
constexpr int kDecMaxRows = 16;

// Divide, round and store a row held by a warp.  A row that came out as NaN
// beside a non-finite V which it does not see is done again from its own keys.
template <int D, bool GEN>
__device__ __forceinline__ void finish_row(const AttnParams& p, const AttnSeq& s, int b, int head, int tok, const float* acc,
                                           float l) {
  constexpr int VPL = D / 32;
  const int lane = threadIdx.x & 31, lim = attn_limit(s, tok);
  float y[VPL];
  bool nan = false;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    y[i] = lim == 0 ? 0.f : acc[i] / l;
    nan |= y[i] != y[i];
  }
  if (__any_sync(0xffffffffu, nan && l == l)) {
    const int h = head / p.group, row = tok * p.group + head - h * p.group, reach = attn_reach(p, s, row);
    if (lim < reach && attn_last_nonfinite<D>(p, s, b, h, lim, reach) >= 0) {
      attend_row<D, GEN>(p, s, b, head, tok);
      return;
    }
    if (GEN) {
      const int from = attn_from(p, s, row), low = attn_low(p, s, lim);
      if (from < low && attn_last_nonfinite<D>(p, s, b, h, from, low) >= 0) {
        attend_row<D, GEN>(p, s, b, head, tok);
        return;
      }
    }
  }
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.O + (s.q0 + tok) * p.ldo + head * D + lane * VPL);
#pragma unroll
  for (int i = 0; i < VPL / 2; ++i) dst[i] = dev::float2_to_bf16x2(y[2 * i], y[2 * i + 1]);
}

template <bool HALF>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if (HALF)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kDecLazy = 4.f;

}  // namespace
}  // namespace wal
