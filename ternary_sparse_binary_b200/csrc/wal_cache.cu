// Rotary positions and the paged KV cache: rotate, append, read back.
//
// All three move each byte once and do little arithmetic, so they are bound by
// HBM, or by one launch when there are few rows.  An item is 16 elements of
// one head row, read and written with 16-byte accesses.
//
// Angles.  A pair turns by p * f_i; f_i / 2 pi is a 64-bit fixed-point
// fraction, so the wrapping product p * freq is the turn modulo one exactly,
// however far the position.  Its top 32 bits, as a signed fraction of half a
// turn in [-1, 1), go to fp32 (relative 2^-24, absolute at most 2^-25 of a half
// turn) and sincospif.  Each CTA computes a token's cosines and sines once in
// shared memory and uses them for all heads.
#include "wal_rope.cuh"

#include <cmath>
#include <cstring>

namespace wal {

int check_cache(const wal_kv_cache* c) {
  if (!c) return fail(WAL_ERR_ARG, "cache descriptor is NULL");
  size_t sz[4];
  int st = wal_kv_cache_sizes(c->n_pages, c->page_size, c->n_heads, c->head_dim, c->type, sz);
  if (st) return st;
  if (!c->k || !c->v) return fail(WAL_ERR_ARG, "k and v are required");
  if (c->type != WAL_KV_BF16 && (!c->k_scale || !c->v_scale))
    return fail(WAL_ERR_ARG, "k_scale and v_scale are required for an 8-bit cache");
  if (misaligned(c->k, 16) || misaligned(c->v, 16) || misaligned(c->k_scale, 16) || misaligned(c->v_scale, 16))
    return fail(WAL_ERR_ARG, "cache buffers must be 16-byte aligned");
  return WAL_OK;
}

int clear_status(void* ws, cudaStream_t stream, int32_t** status) {
  *status = status_word(ws);
  if (!ws) return WAL_OK;
  const cudaError_t e = cudaMemsetAsync(*status, 0, 4, stream);
  if (e != cudaSuccess) return fail(WAL_ERR_CUDA, std::string("status clear: ") + cudaGetErrorString(e));
  return WAL_OK;
}

namespace {

constexpr int kThreads = 256;
// ---------------------------------------------------------------------------
// rotate
// ---------------------------------------------------------------------------
// Bound by bytes: 16384 tokens of 40 heads in 54 us, 0.97 of the copy rate; 25 tokens
// take 2.7 us of a graph.  A CTA takes kTokens tokens (one where there are few:
// latency).  A thread has
// the same item of each of them, so that its place is worked out once, and loads
// all of them before the angles are computed.
constexpr int kBatch = 4;

template <int XT, int kTokens>
__global__ void __launch_bounds__(kThreads) rope_kernel(const void* X, uint16_t* Y, const int32_t* __restrict__ positions,
                                                         Rope r, int n_heads, int items, int64_t ldx, int64_t ldy, int T) {
  __shared__ float2 cs[kTokens * kMaxPairs];
  const int64_t t0 = (int64_t)blockIdx.x * kTokens;
  const int n = min(kTokens, (int)(T - t0)), per = n_heads * items;
  bool first = true;
  for (int q = threadIdx.x; first || q - (int)threadIdx.x < per; q += blockDim.x) {
    const int h = q / items, it = q - h * items, col = h * items * 16;
    const ItemCols c = item_cols(r, it);
    Raw16<XT> raw[kTokens];
    if (q < per)
#pragma unroll
      for (int t = 0; t < kTokens; ++t)
        if (t < n) load16<XT>(static_cast<const char*>(X) + (t0 + t) * ldx * (XT == WAL_F32 ? 4 : 2), col + c.a, col + c.b, raw[t]);
    if (first) {
      first = false;
      angles(r, positions, t0, n, cs);
      __syncthreads();
    }
    if (q < per)
#pragma unroll
      for (int t = 0; t < kTokens; ++t)
        if (t < n) {
          float v[16];
          unpack16<XT>(raw[t], v);
          if (c.rot) rotate16(v, r, it, cs + t * kMaxPairs);
          uint16_t* y = Y + (t0 + t) * ldy + col;
          *reinterpret_cast<uint4*>(y + c.a) = pack8(v);
          *reinterpret_cast<uint4*>(y + c.b) = pack8(v + 8);
        }
  }
}

// ---------------------------------------------------------------------------
// append
// ---------------------------------------------------------------------------
struct AppendParams {
  const void* x[2];  // K, V
  int64_t ld[2];
  void* cache[2];
  float* scale[2];
  const int32_t* slots;
  const int32_t* positions;
  Rope rope;
  int n_heads, head_dim, shift, T;
  uint32_t n_slots;
  int32_t* status;  // NULL: nothing is recorded
};

// Whether y = x * (1 / scale) lies so near to a border between two codes that
// x / scale, which decides, may lie on its other side.  y is within 2^-22 of the
// quotient (relative); the margins are several times that.
template <int TYPE>
__device__ __forceinline__ bool near_border(float y) {
  if (TYPE == WAL_KV_INT8) return fabsf(y - rintf(y)) > 0.5f - 0x1p-13f;
  // half way between codes: the fourth mantissa bit and no more; below the
  // smallest normal code the borders lie elsewhere
  return ((__float_as_uint(y) + 8u) & 0xFFFFFu) - 0x80000u < 16u || (fabsf(y) < 0x1p-6f && y != 0.f);
}
// Bound by instructions in the 8-bit types (39 us for 16381 tokens of 8 heads, 0.41 of
// the copy rate, 2.7 of 4 issued a cycle; 25 and 0.82 to a bf16 cache): the reduction, the conversions and the
// border test.  A CTA takes kTokens tokens; a head row (head_dim / 16 items of neighbouring
// threads, 4 or 8) is reduced by shuffles.
template <int XT, int TYPE, int kTokens>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendParams p) {
  __shared__ float2 cs[kTokens * kMaxPairs];
  const int64_t t0 = (int64_t)blockIdx.x * kTokens;
  const int n = min(kTokens, (int)(p.T - t0));
  if (blockIdx.x == 0 && p.status) {  // the first CTA looks at every slot: no CTA has to wait for a cleared word
    bool bad = false;
    for (int t = threadIdx.x; t < p.T; t += blockDim.x) {
      const int s = __ldg(p.slots + t);
      bad |= (uint32_t)s >= p.n_slots && s != -1;
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) *p.status = bad ? (int32_t)WAL_ERR_ARG : 0;
  }
  int slots[kTokens];
#pragma unroll
  for (int t = 0; t < kTokens; ++t) slots[t] = t < n ? __ldg(p.slots + t0 + t) : -1;
  const int items = p.head_dim / 16, shift = items == 8 ? 3 : 2, rows = 2 * p.n_heads, per = rows << shift;
  bool first = true;
  for (int q = threadIdx.x; first || q - (int)threadIdx.x < per; q += blockDim.x) {
    // whole warps go along for the shuffles
    const int row = min(q >> shift, rows - 1), it = q & (items - 1), which = row >= p.n_heads, h = row - (which ? p.n_heads : 0);
    Rope r = p.rope;
    if (which) r.pairs = 0;
    const ItemCols c = item_cols(r, it);
    const char* x = static_cast<const char*>(which ? p.x[1] : p.x[0]);
    const int64_t ld = which ? p.ld[1] : p.ld[0];
    Raw16<XT> raw[kTokens];
#pragma unroll
    for (int t = 0; t < kTokens; ++t)
      load16<XT>(x + (t0 + min(t, n - 1)) * ld * (XT == WAL_F32 ? 4 : 2), h * p.head_dim + c.a, h * p.head_dim + c.b, raw[t]);
    if (first) {
      first = false;
      if (p.rope.pairs) {
        angles(p.rope, p.positions, t0, n, cs);
        __syncthreads();
      }
    }
    char* cache = static_cast<char*>(which ? p.cache[1] : p.cache[0]);
    float* scales = which ? p.scale[1] : p.scale[0];
#pragma unroll
    for (int t = 0; t < kTokens; ++t) {
      const int slot = slots[t];
      const bool live = q < per && (uint32_t)slot < p.n_slots;
      float v[16];
      unpack16<XT>(raw[t], v);
      if (c.rot) rotate16(v, r, it, cs + t * kMaxPairs);
      const int64_t crow = (((int64_t)(slot >> p.shift) * p.n_heads + h) << p.shift) + (slot & ((1 << p.shift) - 1));
      if (TYPE == WAL_KV_BF16) {
        uint16_t* d = reinterpret_cast<uint16_t*>(cache) + crow * p.head_dim;
        if (live) {
          *reinterpret_cast<uint4*>(d + c.a) = pack8(v);
          *reinterpret_cast<uint4*>(d + c.b) = pack8(v + 8);
        }
        continue;
      }
      // the largest magnitude as bits: infinities and NaN come out on top
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
      for (int o = items >> 1; o; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      const bool bad = top >= 0x7F800000u;
      const float scale = fmaxf(__fdiv_rn(__uint_as_float(bad ? 0u : top), TYPE == WAL_KV_INT8 ? 127.f : 448.f), 1.1754943508222875e-38f);
      const float inv = __frcp_rn(scale);
      bool border = false;
      float y[16];
      uint32_t low = ~0u, least = ~0u;  // e4m3: the nearest to half way, and the smallest
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        y[i] = v[i] * inv;
        if (TYPE == WAL_KV_INT8) {
          border |= near_border<TYPE>(y[i]);
        } else {
          low = min(low, (__float_as_uint(y[i]) + 8u - 0x80000u) & 0xFFFFFu);
          least = min(least, __float_as_uint(y[i]) & 0x7FFFFFFFu);
        }
      }
      if (border || low < 16u || least < 0x3C800000u)  // a code is round(x / scale), the quotient being the IEEE one
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (near_border<TYPE>(y[i])) y[i] = __fdiv_rn(v[i], scale);
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = codes2<TYPE>(y[4 * i], y[4 * i + 1]) | (codes2<TYPE>(y[4 * i + 2], y[4 * i + 3]) << 16);
      if (bad) w[0] = w[1] = w[2] = w[3] = 0;
      if (live) {
        uint8_t* d = reinterpret_cast<uint8_t*>(cache) + crow * p.head_dim;
        *reinterpret_cast<uint2*>(d + c.a) = make_uint2(w[0], w[1]);
        *reinterpret_cast<uint2*>(d + c.b) = make_uint2(w[2], w[3]);
        if (it == 0) scales[crow] = bad ? __int_as_float(0x7FC00000) : scale;
      }
    }
  }
}

// Tokens of a CTA: one while the CTAs do not fill the SMs several times, then two.
// One, two, four and eight: 16381 bf16 tokens of 8 heads of 128 to e4m3 43, 38, 53
// and 80 us; rotating half of 16384 tokens of 40 heads 57, 53, 54 and 55; 2000
// tokens, which take two for little (14.4 and 15.9 us with their reading back).
constexpr int kManyTokens = 2, kFewTokens = 148 * 8;

// Threads of a CTA that has `items` of them a token: whole warps, in equal rounds.
int threads_for(int items) {
  const int rounds = (items + kThreads - 1) / kThreads, each = (items + rounds - 1) / rounds;
  return (each + 31) / 32 * 32;
}

template <int XT, int TYPE>
void launch_append(const AppendParams& p, cudaStream_t s) {
  const int threads = threads_for(2 * p.n_heads * (p.head_dim / 16));
  if (p.T <= kFewTokens)
    append_kernel<XT, TYPE, 1><<<p.T, threads, 0, s>>>(p);
  else
    append_kernel<XT, TYPE, kManyTokens><<<(p.T + kManyTokens - 1) / kManyTokens, threads, 0, s>>>(p);
}
template <int XT>
void launch_rope(const void* X, uint16_t* Y, const int32_t* positions, const Rope& r, int n_heads, int items, int ldx, int ldy, int T,
                 cudaStream_t s) {
  const int threads = threads_for(n_heads * items);
  if (T <= kFewTokens)
    rope_kernel<XT, 1><<<T, threads, 0, s>>>(X, Y, positions, r, n_heads, items, ldx, ldy, T);
  else
    rope_kernel<XT, kManyTokens><<<(T + kManyTokens - 1) / kManyTokens, threads, 0, s>>>(X, Y, positions, r, n_heads, items, ldx, ldy, T);
}

// ---------------------------------------------------------------------------
// read back
// ---------------------------------------------------------------------------
struct ReadParams {
  const void* cache[2];
  const float* scale[2];
  void* out[2];
  int64_t ld[2];
  const int32_t* table;
  const int32_t* start;
  int64_t ld_table;
  int n_heads, head_dim, shift, n_pages, max_len, T;
  int halves;  // K and V, or the one that is wanted in the first place
  int32_t* status;
};
constexpr int kReadTokens = 16;  // tokens of one CTA: a divisor of every page size, so one page

// Bound by bytes: 25 sequences of up to 8192 tokens from int8 to bf16 128 us, 0.98
// of the copy rate.  Neighbouring threads take items of a row, then heads of a token (the output's
// rows are contiguous over both), then tokens, then K and V; four items a thread
// at a time, all loaded before the first is stored.
template <int TYPE, int OT>
__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ ReadParams p) {
  const int b = blockIdx.y, j0 = blockIdx.x * kReadTokens;
  const int64_t s0 = p.start[b], s1 = p.start[b + 1];
  if (s0 < 0 || s1 < s0 || s1 > p.T || s1 - s0 > p.max_len) {
    if (j0 == 0 && threadIdx.x == 0 && p.status) atomicExch(p.status, (int32_t)WAL_ERR_ARG);
    return;
  }
  const int n = min((int)(s1 - s0) - j0, kReadTokens);
  if (n <= 0) return;
  const int page = p.table[b * p.ld_table + (j0 >> p.shift)];
  const bool bad = (uint32_t)page >= (uint32_t)p.n_pages;
  if (bad && threadIdx.x == 0 && p.status) atomicExch(p.status, (int32_t)WAL_ERR_ARG);
  const int off = j0 & ((1 << p.shift) - 1);
  const int items = p.head_dim / 16, per = p.n_heads * items, all = p.halves * n * per;
  const int64_t row0 = (((int64_t)(bad ? 0 : page) * p.n_heads) << p.shift) + off;  // head 0, token j0
  struct Place {
    int which, j, h, it;
  };
  auto place = [&](int q) {
    Place x;
    x.which = q >= n * per;
    const int r = q - x.which * n * per;
    x.j = r / per;
    const int e = r - x.j * per;
    x.h = e / items;
    x.it = e - x.h * items;
    return x;
  };
  for (int q0 = threadIdx.x; q0 < all; q0 += kBatch * kThreads) {
    uint4 raw[kBatch][TYPE == WAL_KV_BF16 ? 2 : 1];
    float sc[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const Place x = place(min(q0 + u * kThreads, all - 1));
      const int64_t crow = row0 + ((int64_t)x.h << p.shift) + x.j;
      const char* cache = static_cast<const char*>(x.which ? p.cache[1] : p.cache[0]);
      if (TYPE == WAL_KV_BF16) {
        const uint4* src = reinterpret_cast<const uint4*>(cache + (crow * p.head_dim + 16 * x.it) * 2);
        raw[u][0] = src[0];
        raw[u][TYPE == WAL_KV_BF16 ? 1 : 0] = src[1];
      } else {
        raw[u][0] = *reinterpret_cast<const uint4*>(cache + crow * p.head_dim + 16 * x.it);
        sc[u] = (x.which ? p.scale[1] : p.scale[0])[crow];
      }
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (q0 + u * kThreads >= all) break;
      const Place x = place(q0 + u * kThreads);
      char* out = static_cast<char*>(x.which ? p.out[1] : p.out[0]);
      const int64_t dst = (s0 + j0 + x.j) * (x.which ? p.ld[1] : p.ld[0]) + x.h * p.head_dim + 16 * x.it;
      float v[16];
      if (TYPE == WAL_KV_BF16) {
        Raw16<WAL_BF16> r;
        r.v[0] = raw[u][0];
        r.v[1] = raw[u][TYPE == WAL_KV_BF16 ? 1 : 0];
        unpack16<WAL_BF16>(r, v);
      } else {
        const uint32_t w[4] = {raw[u][0].x, raw[u][0].y, raw[u][0].z, raw[u][0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float f[4];
          dev::codes4_to_float<TYPE>(w[i], f);
#pragma unroll
          for (int k = 0; k < 4; ++k) v[4 * i + k] = f[k] * sc[u];
        }
      }
      if (bad)
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = 0.f;
      if (OT == WAL_BF16) {
        uint4* d = reinterpret_cast<uint4*>(out + dst * 2);
        d[0] = pack8(v);
        d[1] = pack8(v + 8);
      } else {
        float4* d = reinterpret_cast<float4*>(out + dst * 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
      }
    }
  }
}

}  // namespace
}  // namespace wal

using namespace wal;

extern "C" int wal_rope_freqs(int rot_dim, double base, int scaling, double factor, double original_len, double slow,
                              double fast, uint64_t* freq, float* mscale) {
  if (!freq || !mscale) return fail(WAL_ERR_ARG, "freq and mscale are required");
  if (rot_dim < 2 || rot_dim > 2 * kMaxPairs || (rot_dim & 1)) return fail(WAL_ERR_SHAPE, "rot_dim must be even and in [2, 256]");
  if (scaling < WAL_SCALING_NONE || scaling > WAL_SCALING_PARTS) return fail(WAL_ERR_ARG, "unknown scaling");
  if (!(base > 1.0) || !std::isfinite(base)) return fail(WAL_ERR_ARG, "base must be above 1");
  if (scaling != WAL_SCALING_NONE && (!(factor >= 1.0) || !std::isfinite(factor)))
    return fail(WAL_ERR_ARG, "factor must be at least 1");
  if (scaling == WAL_SCALING_PARTS &&
      (!(original_len > 0.0) || !std::isfinite(original_len) || !(slow >= 0.0) || !(fast > slow) || !std::isfinite(fast)))
    return fail(WAL_ERR_ARG, "by-parts scaling needs original_len > 0 and fast > slow >= 0");
  const long double two_pi = 6.283185307179586476925286766559L;
  for (int i = 0; i < rot_dim / 2; ++i) {
    long double f = powl((long double)base, -2.0L * i / rot_dim);
    if (scaling == WAL_SCALING_LINEAR) f /= factor;
    if (scaling == WAL_SCALING_PARTS) {
      const long double t = original_len * f / two_pi;
      long double g = (t - slow) / ((long double)fast - slow);
      g = g < 0 ? 0 : g > 1 ? 1 : g;
      f = (1 - g) * f / factor + g * f;
    }
    // f <= 1, so f / 2 pi < 0.16 of a turn and the product stays below 2^62
    freq[i] = (uint64_t)llroundl(f / two_pi * 18446744073709551616.0L);
  }
  *mscale = scaling == WAL_SCALING_PARTS ? (float)(0.1 * std::log(factor) + 1.0) : 1.f;
  return WAL_OK;
}

extern "C" int wal_rope(const wal_rope_plan* rope, const void* X, int x_type, int T, int n_heads, int ldx,
                        const int32_t* positions, uint16_t* Y, int ldy, wal_stream_t stream) {
  if (!rope) return fail(WAL_ERR_ARG, "rope plan is NULL");
  int st = check_rope(rope, rope->head_dim);
  if (st) return st;
  if (T < 0 || n_heads < 1) return fail(WAL_ERR_SHAPE, "T must be >= 0 and n_heads >= 1");
  const int64_t width = (int64_t)n_heads * rope->head_dim;
  if ((st = check_rows(X, x_type, ldx, width, "X"))) return st;
  if ((st = check_rows(Y, WAL_BF16, ldy, width, "Y"))) return st;
  if (misaligned(positions, 4)) return fail(WAL_ERR_ARG, "positions must be 4-byte aligned");
  if (T == 0) return WAL_OK;
  if (!X || !Y || !positions) return fail(WAL_ERR_ARG, "X, Y and positions are required");
  if ((const void*)Y == X && (x_type != WAL_BF16 || ldx != ldy))
    return fail(WAL_ERR_ARG, "Y may be X only for bf16 rows of the same stride");
  int dev = 0;
  if ((st = current_device(&dev))) return st;
  const Rope r = {rope->freq, rope->rot_dim / 2, rope->layout, rope->mscale};
  const int items = rope->head_dim / 16;
  cudaStream_t s = (cudaStream_t)stream;
  if (x_type == WAL_F32)
    launch_rope<WAL_F32>(X, Y, positions, r, n_heads, items, ldx, ldy, T, s);
  else
    launch_rope<WAL_BF16>(X, Y, positions, r, n_heads, items, ldx, ldy, T, s);
  return launched("rope_kernel");
}

extern "C" int wal_kv_cache_sizes(int n_pages, int page_size, int n_heads, int head_dim, int type, size_t out[4]) {
  if (!out) return fail(WAL_ERR_ARG, "out_bytes is NULL");
  if (n_pages < 1 || n_heads < 1 || page_size < 1 || head_dim < 1)
    return fail(WAL_ERR_SHAPE, "n_pages, page_size, n_heads and head_dim must be positive");
  if (type != WAL_KV_BF16 && type != WAL_KV_INT8 && type != WAL_KV_E4M3) return fail(WAL_ERR_ARG, "unknown cache type");
  if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1)))
    return fail(WAL_ERR_UNSUPPORTED, "page_size must be 16, 32, 64, 128 or 256");
  if (head_dim != 64 && head_dim != 128) return fail(WAL_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
  if (n_heads > 1024) return fail(WAL_ERR_UNSUPPORTED, "at most 1024 K/V heads");
  if ((int64_t)n_pages * page_size > 0x7FFFFFFF) return fail(WAL_ERR_UNSUPPORTED, "n_pages * page_size must be below 2^31");
  const size_t rows = (size_t)n_pages * page_size * n_heads;
  out[0] = out[1] = rows * head_dim * (type == WAL_KV_BF16 ? 2 : 1);
  out[2] = out[3] = type == WAL_KV_BF16 ? 0 : rows * 4;
  return WAL_OK;
}

extern "C" int wal_kv_append(const wal_kv_cache* cache, const void* K, const void* V, int in_type, int T, int ldk,
                             int ldv, const int32_t* slots, const int32_t* positions, const wal_rope_plan* rope,
                             void* ws, size_t ws_bytes, wal_stream_t stream) {
  int st = check_cache(cache);
  if (st) return st;
  if (rope && (st = check_rope(rope, cache->head_dim))) return st;
  if (T < 0) return fail(WAL_ERR_SHAPE, "T must be >= 0");
  const int64_t width = (int64_t)cache->n_heads * cache->head_dim;
  if ((st = check_rows(K, in_type, ldk, width, "K"))) return st;
  if ((st = check_rows(V, in_type, ldv, width, "V"))) return st;
  if (misaligned(slots, 4) || misaligned(positions, 4)) return fail(WAL_ERR_ARG, "slots and positions must be 4-byte aligned");
  if (T > 0 && (!K || !V || !slots)) return fail(WAL_ERR_ARG, "K, V and slots are required");
  if (T > 0 && rope && !positions) return fail(WAL_ERR_ARG, "positions are required with a rope plan");
  if (ws && ws_bytes < kStatusWs) return fail(WAL_ERR_WORKSPACE, "a workspace has at least 512 bytes");
  int dev = 0;
  if ((st = current_device(&dev))) return st;
  AppendParams p = {};
  cudaStream_t s = (cudaStream_t)stream;
  if (T == 0) return clear_status(ws, s, &p.status);
  p.status = status_word(ws);
  p.T = T;
  p.x[0] = K; p.x[1] = V;
  p.ld[0] = ldk; p.ld[1] = ldv;
  p.cache[0] = cache->k; p.cache[1] = cache->v;
  p.scale[0] = cache->k_scale; p.scale[1] = cache->v_scale;
  p.slots = slots;
  p.positions = positions;
  if (rope) p.rope = {rope->freq, rope->rot_dim / 2, rope->layout, rope->mscale};
  p.n_heads = cache->n_heads;
  p.head_dim = cache->head_dim;
  p.shift = log2_of(cache->page_size);
  p.n_slots = (uint32_t)(cache->n_pages * cache->page_size);
  const bool f = in_type == WAL_F32;
  switch (cache->type) {
    case WAL_KV_BF16: f ? launch_append<WAL_F32, WAL_KV_BF16>(p, s) : launch_append<WAL_BF16, WAL_KV_BF16>(p, s); break;
    case WAL_KV_INT8: f ? launch_append<WAL_F32, WAL_KV_INT8>(p, s) : launch_append<WAL_BF16, WAL_KV_INT8>(p, s); break;
    default: f ? launch_append<WAL_F32, WAL_KV_E4M3>(p, s) : launch_append<WAL_BF16, WAL_KV_E4M3>(p, s); break;
  }
  return launched("append_kernel");
}

extern "C" int wal_kv_read(const wal_kv_cache* cache, const int32_t* table, int ld_table, const int32_t* start, int B,
                           int max_len, void* K, void* V, int out_type, int T, int ldk, int ldv, void* ws,
                           size_t ws_bytes, wal_stream_t stream) {
  int st = check_cache(cache);
  if (st) return st;
  if (B < 1 || B > 65535 || max_len < 1 || T < 0) return fail(WAL_ERR_SHAPE, "1 <= B <= 65535, max_len >= 1 and T >= 0");
  const int64_t width = (int64_t)cache->n_heads * cache->head_dim;
  if ((st = check_rows(K, out_type, K ? ldk : (int)align_up((size_t)width, 8), width, "K"))) return st;
  if ((st = check_rows(V, out_type, V ? ldv : (int)align_up((size_t)width, 8), width, "V"))) return st;
  if (!table || !start || misaligned(table, 4) || misaligned(start, 4))
    return fail(WAL_ERR_ARG, "table and start are required, 4-byte aligned");
  if ((int64_t)ld_table * cache->page_size < max_len) return fail(WAL_ERR_ARG, "ld_table pages must cover max_len tokens");
  if (ws && ws_bytes < kStatusWs) return fail(WAL_ERR_WORKSPACE, "a workspace has at least 512 bytes");
  int dev = 0;
  if ((st = current_device(&dev))) return st;
  ReadParams p = {};
  cudaStream_t s = (cudaStream_t)stream;
  if ((st = clear_status(ws, s, &p.status))) return st;
  if (!K && !V) return WAL_OK;
  p.cache[0] = cache->k; p.cache[1] = cache->v;
  p.scale[0] = cache->k_scale; p.scale[1] = cache->v_scale;
  p.out[0] = K; p.out[1] = V;
  p.ld[0] = ldk; p.ld[1] = ldv;
  p.halves = K && V ? 2 : 1;
  if (!K) {
    p.cache[0] = p.cache[1];
    p.scale[0] = p.scale[1];
    p.out[0] = p.out[1];
    p.ld[0] = p.ld[1];
  }
  p.table = table;
  p.start = start;
  p.ld_table = ld_table;
  p.n_heads = cache->n_heads;
  p.head_dim = cache->head_dim;
  p.shift = log2_of(cache->page_size);
  p.n_pages = cache->n_pages;
  p.max_len = max_len;
  p.T = T;
  const dim3 grid((unsigned)((max_len + (int64_t)kReadTokens - 1) / kReadTokens), (unsigned)B);
  const bool f = out_type == WAL_F32;
  switch (cache->type) {
    case WAL_KV_BF16: f ? read_kernel<WAL_KV_BF16, WAL_F32><<<grid, kThreads, 0, s>>>(p) : read_kernel<WAL_KV_BF16, WAL_BF16><<<grid, kThreads, 0, s>>>(p); break;
    case WAL_KV_INT8: f ? read_kernel<WAL_KV_INT8, WAL_F32><<<grid, kThreads, 0, s>>>(p) : read_kernel<WAL_KV_INT8, WAL_BF16><<<grid, kThreads, 0, s>>>(p); break;
    default: f ? read_kernel<WAL_KV_E4M3, WAL_F32><<<grid, kThreads, 0, s>>>(p) : read_kernel<WAL_KV_E4M3, WAL_BF16><<<grid, kThreads, 0, s>>>(p); break;
  }
  return launched("read_kernel");
}
