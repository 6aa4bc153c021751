// Shared by the rotary, cache and attention kernels: argument checks of the
// cache descriptor and conversions of its element types.
#pragma once

#include "wal_internal.h"

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

namespace wal {

constexpr size_t kStatusWs = 512;  // workspace that only holds the 256-byte aligned status word

int check_cache(const wal_kv_cache* c);
inline int32_t* status_word(void* ws) { return !ws ? nullptr : reinterpret_cast<int32_t*>(align_up((uintptr_t)ws, 256)); }
// The status word of a workspace, cleared on `stream`; NULL without one.
int clear_status(void* ws, cudaStream_t stream, int32_t** status);

inline int log2_of(int v) {
  int s = 0;
  while ((1 << s) < v) ++s;
  return s;
}
inline bool misaligned(const void* p, uintptr_t a) { return (uintptr_t)p & (a - 1); }

namespace dev {

__device__ __forceinline__ float2 bf16x2_to_float2(uint32_t v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t float2_to_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t float2_to_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Four 8-bit codes (bytes 0..3 of w) as fp32.
template <int TYPE>
__device__ __forceinline__ void codes4_to_float(uint32_t w, float (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t b = (w >> (8 * i)) & 0xFFu;
    if (TYPE == WAL_KV_INT8)
      v[i] = (float)(int8_t)b;
    else  // s eeee mmm read as an fp32 with exponent field eeee, then times 2^120: exact, subnormals too
      v[i] = __uint_as_float(((b & 0x80u) << 24) | ((b & 0x7Fu) << 20)) * 1.329227995784916e36f;
  }
}

// The same as bf16 pairs: lo = codes 0 and 1, hi = codes 2 and 3.  Both types are
// exact in bf16.
template <int TYPE>
__device__ __forceinline__ void codes4_to_bf16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (TYPE == WAL_KV_INT8) {
    // byte b = 128 s + u stands for u - 128 s.  As the low byte of 0x43xx, u
    // reads 128 + u and the sign bit alone 128 or 256: their difference.
    const uint32_t t0 = __byte_perm(w, 0x43434343u, 0x4140), t1 = __byte_perm(w, 0x43434343u, 0x4342);
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(lo) : "r"(t0 & 0xFF7FFF7Fu), "r"(t0 & 0xFF80FF80u));
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(hi) : "r"(t1 & 0xFF7FFF7Fu), "r"(t1 & 0xFF80FF80u));
  } else {
    // s eeee mmm moved to the sign, the low exponent bits and the high mantissa
    // bits reads 2^-120 times the value, subnormals too
    const uint32_t t0 = __byte_perm(w, 0, 0x1404), t1 = __byte_perm(w, 0, 0x3424);
    const uint32_t e = 0x7B807B80u;  // 2^120 as a bf16 pair
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(lo) : "r"((t0 & 0x80008000u) | ((t0 >> 4) & 0x07F007F0u)), "r"(e));
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(hi) : "r"((t1 & 0x80008000u) | ((t1 >> 4) & 0x07F007F0u)), "r"(e));
  }
}
// And as fp16 pairs, in half the instructions: int8 as the low byte of 0x64xx
// reads 1024 + (code + 128), e4m3 has a conversion of its own.
template <int TYPE>
__device__ __forceinline__ void codes4_to_half(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (TYPE == WAL_KV_INT8) {
    const uint32_t u = w ^ 0x80808080u, off = 0x64806480u;  // 1152
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(__byte_perm(u, 0x64646464u, 0x4140)), "r"(off));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(__byte_perm(u, 0x64646464u, 0x4342)), "r"(off));
  } else {
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  }
}

}  // namespace dev
}  // namespace wal
