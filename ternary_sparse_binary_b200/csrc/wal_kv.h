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
// The status word of a workspace, cleared on `stream`.
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

}  // namespace dev
}  // namespace wal
