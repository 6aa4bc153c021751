// Shared by the kernels that rotate, store and normalise head rows (wal_cache.cu,
// wal_qkv.cu): argument checks, angles, and items of 16 elements of a row.
#pragma once

#include "wal_kv.h"

#include <string>

namespace wal {

namespace {

constexpr int kMaxPairs = 128;

struct Rope {
  const uint64_t* freq;
  int pairs;  // rot_dim / 2; 0: no rotation
  int layout;
  float mscale;
};

int check_rope(const wal_rope_plan* r, int head_dim) {
  if (!r) return fail(WAL_ERR_ARG, "rope plan is NULL");
  if (r->head_dim != head_dim) return fail(WAL_ERR_SHAPE, "the rope plan is for another head_dim");
  if (head_dim <= 0 || r->rot_dim <= 0 || r->rot_dim > head_dim || (r->rot_dim & 1))
    return fail(WAL_ERR_SHAPE, "rot_dim must be even and in [2, head_dim]");
  if (head_dim % 16 || head_dim > 256 || r->rot_dim % 16)
    return fail(WAL_ERR_UNSUPPORTED, "head_dim and rot_dim must be multiples of 16, head_dim at most 256");
  if (r->layout != WAL_ROPE_HALF && r->layout != WAL_ROPE_INTERLEAVED) return fail(WAL_ERR_ARG, "unknown rope layout");
  if (!r->freq || misaligned(r->freq, 8)) return fail(WAL_ERR_ARG, "freq is required, 8-byte aligned");
  return WAL_OK;
}

int check_rows(const void* X, int type, int ld, int64_t width, const char* what) {
  if (type != WAL_F32 && type != WAL_BF16) return fail(WAL_ERR_ARG, "the element type must be WAL_F32 or WAL_BF16");
  if (misaligned(X, 16)) return fail(WAL_ERR_ARG, std::string(what) + " must be 16-byte aligned");
  if (ld < width || ld % (type == WAL_F32 ? 4 : 8))
    return fail(WAL_ERR_ARG, std::string(what) + ": the row stride must cover the heads and be a multiple of 16 bytes");
  return WAL_OK;
}

// Cosine and sine (times mscale) of pair i at position pos.
__device__ __forceinline__ float2 rope_angle(const Rope& r, int pos, int i) {
  const uint64_t turn = (uint64_t)(int64_t)pos * __ldg(r.freq + i);
  const float half_turns = (float)(int32_t)(uint32_t)(turn >> 32) * 4.656612873077393e-10f;  // 2^-31
  float s, c;
  sincospif(half_turns, &s, &c);
  return make_float2(c * r.mscale, s * r.mscale);
}

// The columns of item `it` of a head: two runs of eight, [a, a + 8) and
// [b, b + 8).  Rotated items come first; in the half layout their two runs are
// the two sides of eight pairs, else the runs are adjacent.
struct ItemCols {
  int a, b;
  bool rot;
};
__device__ __forceinline__ ItemCols item_cols(const Rope& r, int it) {
  ItemCols c;
  c.rot = it < (r.pairs >> 3);
  c.a = 16 * it;
  c.b = c.a + 8;
  if (c.rot && r.layout == WAL_ROPE_HALF) {
    c.a = 8 * it;
    c.b = c.a + r.pairs;
  }
  return c;
}

__device__ __forceinline__ uint4 pack8(const float* v) {
  return make_uint4(dev::float2_to_bf16x2(v[0], v[1]), dev::float2_to_bf16x2(v[2], v[3]),
                    dev::float2_to_bf16x2(v[4], v[5]), dev::float2_to_bf16x2(v[6], v[7]));
}

// Turn the 16 elements of item `it` (v[0..7] the first run, v[8..15] the second).
__device__ __forceinline__ void rotate16(float (&v)[16], const Rope& r, int it, const float2* cs) {
  const float2* c = cs + 8 * it;
  if (r.layout == WAL_ROPE_HALF) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = v[i], y = v[8 + i];
      v[i] = x * c[i].x - y * c[i].y;
      v[8 + i] = y * c[i].x + x * c[i].y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = v[2 * i], y = v[2 * i + 1];
      v[2 * i] = x * c[i].x - y * c[i].y;
      v[2 * i + 1] = y * c[i].x + x * c[i].y;
    }
  }
}

template <int XT>
struct Raw16 {  // 16 elements as they lie in memory
  uint4 v[XT == WAL_F32 ? 4 : 2];
};
template <int XT>
__device__ __forceinline__ void load16(const void* row, int a, int b, Raw16<XT>& r) {
  const char* p = static_cast<const char*>(row);
  constexpr int S = XT == WAL_F32 ? 4 : 2, H = S / 2;
#pragma unroll
  for (int i = 0; i < H; ++i) {
    r.v[i] = *reinterpret_cast<const uint4*>(p + (size_t)a * S + 16 * i);
    r.v[H + i] = *reinterpret_cast<const uint4*>(p + (size_t)b * S + 16 * i);
  }
}
template <int XT>
__device__ __forceinline__ void unpack16(const Raw16<XT>& r, float (&v)[16]) {
  if (XT == WAL_F32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 u = r.v[i < (XT == WAL_F32 ? 4 : 2) ? i : 0];
      v[4 * i] = __uint_as_float(u.x); v[4 * i + 1] = __uint_as_float(u.y);
      v[4 * i + 2] = __uint_as_float(u.z); v[4 * i + 3] = __uint_as_float(u.w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t w[4] = {r.v[i].x, r.v[i].y, r.v[i].z, r.v[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = dev::bf16x2_to_float2(w[k]);
        v[8 * i + 2 * k] = f.x;
        v[8 * i + 2 * k + 1] = f.y;
      }
    }
  }
}
// Cosines and sines of tokens t0 .. t0 + n - 1 into cs[token][pair].
__device__ __forceinline__ void angles(const Rope& r, const int32_t* __restrict__ positions, int64_t t0, int n, float2* cs) {
  for (int q = threadIdx.x; q < n * r.pairs; q += blockDim.x) {
    const int t = q / r.pairs, i = q - t * r.pairs;
    cs[t * kMaxPairs + i] = rope_angle(r, __ldg(positions + t0 + t), i);
  }
}

// Codes of a and b as bytes 0 and 1.
template <int TYPE>
__device__ __forceinline__ uint32_t codes2(float a, float b) {
  if (TYPE == WAL_KV_INT8) return ((uint32_t)__float2int_rn(a) & 0xFFu) | (((uint32_t)__float2int_rn(b) & 0xFFu) << 8);
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

int launched(const char* what) {
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(WAL_ERR_CUDA, std::string(what) + " launch: " + cudaGetErrorString(e));
  return WAL_OK;
}

}  // namespace
}  // namespace wal
