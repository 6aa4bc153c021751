// What a layer does to the q, k and v of new tokens, in one launch: the norms of
// the q and k heads, the rotation, q to bf16 rows, k and v to the paged cache (or
// k to bf16 rows).
//
//   y = x w / sqrt(mean(x^2) + eps)     over the columns of one head, w of a column
//
// then rotated and rounded once.  Each byte moves once.  An item is 16 elements of a
// head row; the row's items lie in neighbouring lanes, which add their squares (and
// find the largest magnitude, for a code's scale) by shuffles.
#include "wal_ptx.cuh"
#include "wal_rope.cuh"

namespace wal {

namespace {

constexpr int kRows = -1;  // in the place of a cache type: k goes to bf16 rows

struct QkvParams {
  const void* x[3];  // q, k, v
  int64_t ld[3];
  uint16_t* out[2];  // rows of q, and of k without a cache
  int64_t ldo[2];
  void* cache[2];
  float* scale[2];
  const int32_t* slots;
  const int32_t* positions;
  const void* weight[2];  // NULL: no norm
  int weight_type;
  float eps;
  Rope rope;
  int n_heads, n_kv_heads, head_dim;
  int items, lanes_log2;  // of a head row
  int shift, T;
  uint32_t n_slots;
  int32_t* status;  // NULL: nothing is recorded
};

// Reciprocal root of the mean square of a row whose items lie in `lanes` lanes.
// The squares of values beyond 2^64 overflow; such a row is summed again at 2^-80 of
// its size, where eps is nothing beside it.  An infinity stays one: the row's other
// elements become 0 and it becomes NaN, as in the formula.
__device__ __forceinline__ float row_norm(const float (&v)[16], int lanes, float inv_dim, float eps) {
  float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 x = make_float2(v[2 * i], v[2 * i + 1]);
    s2 = ptx::fma2(x, x, s2);
  }
  float s = s2.x + s2.y;
  for (int o = lanes >> 1; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  float r = rsqrtf(s * inv_dim + eps);
  if (__any_sync(0xffffffffu, s == INFINITY)) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float x = v[i] * 0x1p-80f;
      t += x * x;
    }
    for (int o = lanes >> 1; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if (s == INFINITY) r = rsqrtf(t * inv_dim) * 0x1p-80f;
  }
  return r;
}

// Cosines and sines of a token, and the norms' weights, as the items take them: chunk j
// of item `it` at [j][it], so that the lanes of a row read neighbouring chunks.  Angles:
// {cos, cos, sin, sin} of two pairs.
struct Angles {
  float4 v[4][kMaxPairs / 8];
};
struct Weights {
  float4 v[4][kMaxPairs / 8];
};
// rotate16 over them, its products contracted as they are there: the same bits.
__device__ __forceinline__ void turn(float (&v)[16], int layout, const Angles& a, int it) {
  if (layout == WAL_ROPE_HALF) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 t = a.v[j][it];
      const float2 c = make_float2(t.x, t.y), s = make_float2(t.z, t.w), minus = make_float2(-t.z, -t.w);
      const float2 x = make_float2(v[2 * j], v[2 * j + 1]), y = make_float2(v[8 + 2 * j], v[9 + 2 * j]);
      const float2 p = ptx::fma2(x, c, ptx::mul2(y, minus)), q = ptx::fma2(x, s, ptx::mul2(y, c));
      v[2 * j] = p.x;
      v[2 * j + 1] = p.y;
      v[8 + 2 * j] = q.x;
      v[9 + 2 * j] = q.y;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 t = a.v[j][it];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float c = e ? t.y : t.x, s = e ? t.w : t.z, x = v[4 * j + 2 * e], y = v[4 * j + 2 * e + 1];
        v[4 * j + 2 * e] = x * c - y * s;
        v[4 * j + 2 * e + 1] = y * c + x * s;
      }
    }
  }
}

// Bound by bytes.  A CTA takes kTokens tokens (one where there are few: latency), a
// thread the same item of each of them; all of them are loaded before the first
// token's angles are worked out, and a round's loads before the round before is done.
template <int XT, int TYPE, int kTokens>
__global__ void __launch_bounds__(512) qkv_kernel(const __grid_constant__ QkvParams p) {
  constexpr int S = XT == WAL_F32 ? 4 : 2;
  __shared__ Angles angle[kTokens];
  __shared__ Weights weight[2];
  const int64_t t0 = (int64_t)blockIdx.x * kTokens;
  const int n = min(kTokens, (int)(p.T - t0));
  int slots[kTokens];
  if (TYPE != kRows) {
    if (blockIdx.x == 0 && p.status) {  // the first CTA looks at every slot: no CTA has to wait for a cleared word
      bool bad = false;
      for (int t = threadIdx.x; t < p.T; t += blockDim.x) {
        const int s = __ldg(p.slots + t);
        bad |= (uint32_t)s >= p.n_slots && s != -1;
      }
      bad = __syncthreads_or(bad);
      if (threadIdx.x == 0) *p.status = bad ? (int32_t)WAL_ERR_ARG : 0;
    }
#pragma unroll
    for (int t = 0; t < kTokens; ++t) slots[t] = t < n ? __ldg(p.slots + t0 + t) : -1;
  }
  const int lanes = 1 << p.lanes_log2, rows = p.n_heads + p.n_kv_heads * (TYPE == kRows ? 1 : 2), per = rows << p.lanes_log2;
  const float inv_dim = 1.f / (float)p.head_dim;
  const bool norm = p.weight[0] != nullptr;
  // a thread's item is the same in all of its rows
  const int lane = threadIdx.x & (lanes - 1);
  const bool there = lane < p.items;
  const int it = there ? lane : 0;
  Rope rope = p.rope, none = p.rope;
  none.pairs = 0;
  const ItemCols turned = item_cols(rope, it), plain = item_cols(none, it);
  struct Place {
    int which, h;
    ItemCols c;
  };
  auto place = [&](int i) {
    const int row = min(i >> p.lanes_log2, rows - 1);
    Place x;
    x.which = TYPE != kRows && row >= p.n_heads + p.n_kv_heads ? 2 : row >= p.n_heads;
    x.h = row - (x.which == 0 ? 0 : x.which == 1 ? p.n_heads : p.n_heads + p.n_kv_heads);
    x.c = x.which == 2 ? plain : turned;
    return x;
  };
  Raw16<XT> raw[kTokens];
  auto load = [&](const Place& x) {
    const char* from = static_cast<const char*>(x.which == 0 ? p.x[0] : x.which == 1 ? p.x[1] : p.x[2]);
    const int64_t ld = x.which == 0 ? p.ld[0] : x.which == 1 ? p.ld[1] : p.ld[2];
#pragma unroll
    for (int t = 0; t < kTokens; ++t)
      load16<XT>(from + ((t0 + min(t, n - 1)) * ld + x.h * p.head_dim) * S, x.c.a, x.c.b, raw[t]);
  };
  load(place(threadIdx.x));
  if (norm)
    for (int j = threadIdx.x; j < 32 * p.items; j += blockDim.x) {
      const int k = j >= 16 * p.items, e = j - (k ? 16 * p.items : 0), item = e >> 4;
      const ItemCols c = item_cols(rope, item);
      const int col = (e & 8) ? c.b + (e & 7) : c.a + (e & 7);
      const void* w = k ? p.weight[1] : p.weight[0];
      reinterpret_cast<float*>(&weight[k].v[(e & 15) >> 2][item])[e & 3] =
          p.weight_type == WAL_F32 ? __ldg(static_cast<const float*>(w) + col)
                                   : __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t*>(w) + col) << 16);
    }
  for (int q = threadIdx.x; q < n * rope.pairs; q += blockDim.x) {
    const int t = q / rope.pairs, i = q - t * rope.pairs;
    const float2 cs = rope_angle(rope, __ldg(p.positions + t0 + t), i);
    float* f = reinterpret_cast<float*>(&angle[t].v[(i & 7) >> 1][i >> 3]) + (i & 1);
    f[0] = cs.x;
    f[2] = cs.y;
  }
  __syncthreads();
#pragma unroll 1
  for (int i = threadIdx.x; i - (int)threadIdx.x < per; i += blockDim.x) {  // whole warps go along for the shuffles
    const Place x = place(i);
    const bool live = there && i < per;
    float v[kTokens][16];
#pragma unroll
    for (int t = 0; t < kTokens; ++t) unpack16<XT>(raw[t], v[t]);
    if (i - (int)threadIdx.x + (int)blockDim.x < per) load(place(i + blockDim.x));
#pragma unroll
    for (int t = 0; t < kTokens; ++t) {
      if (!there)
#pragma unroll
        for (int e = 0; e < 16; ++e) v[t][e] = 0.f;
      if (norm) {
        const float rn = row_norm(v[t], lanes, inv_dim, p.eps);
        if (x.which < 2) {
          const float2 r2 = make_float2(rn, rn);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float4 w = weight[x.which].v[j][it];
            const float2 y = ptx::mul2(ptx::mul2(make_float2(v[t][4 * j], v[t][4 * j + 1]), r2), make_float2(w.x, w.y));
            const float2 z = ptx::mul2(ptx::mul2(make_float2(v[t][4 * j + 2], v[t][4 * j + 3]), r2), make_float2(w.z, w.w));
            v[t][4 * j] = y.x;
            v[t][4 * j + 1] = y.y;
            v[t][4 * j + 2] = z.x;
            v[t][4 * j + 3] = z.y;
          }
        }
      }
      if (x.c.rot) turn(v[t], rope.layout, angle[t], it);
      if (TYPE == kRows || x.which == 0) {
        if (live && t < n) {
          uint16_t* y = (x.which == 0 ? p.out[0] : p.out[1]) + (t0 + t) * (x.which == 0 ? p.ldo[0] : p.ldo[1]) + x.h * p.head_dim;
          *reinterpret_cast<uint4*>(y + x.c.a) = pack8(v[t]);
          *reinterpret_cast<uint4*>(y + x.c.b) = pack8(v[t] + 8);
        }
      }
      if (TYPE == kRows) continue;
      const int slot = slots[t];
      const bool store = live && x.which > 0 && (uint32_t)slot < p.n_slots;
      char* cache = static_cast<char*>(x.which == 2 ? p.cache[1] : p.cache[0]);
      const int64_t crow = (((int64_t)(slot >> p.shift) * p.n_kv_heads + x.h) << p.shift) + (slot & ((1 << p.shift) - 1));
      if (TYPE == WAL_KV_BF16) {
        if (store) {
          uint16_t* d = reinterpret_cast<uint16_t*>(cache) + crow * p.head_dim;
          *reinterpret_cast<uint4*>(d + x.c.a) = pack8(v[t]);
          *reinterpret_cast<uint4*>(d + x.c.b) = pack8(v[t] + 8);
        }
        continue;
      }
      if (__all_sync(0xffffffffu, x.which == 0)) continue;
      // the largest magnitude as bits: infinities and NaN come out on top
      uint32_t top = 0;
#pragma unroll
      for (int e = 0; e < 16; ++e) top = max(top, __float_as_uint(v[t][e]) & 0x7FFFFFFFu);
      for (int o = lanes >> 1; o; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      const bool bad = top >= 0x7F800000u;
      const float scale = fmaxf(__fdiv_rn(__uint_as_float(bad ? 0u : top), TYPE == WAL_KV_INT8 ? 127.f : 448.f), 1.1754943508222875e-38f);
      // quotients: times the reciprocal, then one step on the exact remainder
      // (Markstein, 1990).  A remainder beside a tiny scale is not exact.
      const float inv = __frcp_rn(scale);
      if (scale < 0x1p-100f) {
#pragma unroll
        for (int e = 0; e < 16; ++e) v[t][e] = __fdiv_rn(v[t][e], scale);
      } else {
        const float2 inv2 = make_float2(inv, inv), minus = make_float2(-scale, -scale);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 u = make_float2(v[t][2 * e], v[t][2 * e + 1]);
          const float2 y = ptx::mul2(u, inv2), z = ptx::fma2(ptx::fma2(y, minus, u), inv2, y);
          v[t][2 * e] = z.x;
          v[t][2 * e + 1] = z.y;
        }
      }
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = codes2<TYPE>(v[t][4 * e], v[t][4 * e + 1]) | (codes2<TYPE>(v[t][4 * e + 2], v[t][4 * e + 3]) << 16);
      if (bad) w[0] = w[1] = w[2] = w[3] = 0;
      if (store) {
        uint8_t* d = reinterpret_cast<uint8_t*>(cache) + crow * p.head_dim;
        *reinterpret_cast<uint2*>(d + x.c.a) = make_uint2(w[0], w[1]);
        *reinterpret_cast<uint2*>(d + x.c.b) = make_uint2(w[2], w[3]);
        if (it == 0) (x.which == 2 ? p.scale[1] : p.scale[0])[crow] = bad ? __int_as_float(0x7FC00000) : scale;
      }
    }
  }
}

// Up to kFewTokens tokens leave SMs idle: one CTA a token, wide, for latency.  More of
// them: CTAs of 128 threads (16381 tokens of 32 + 16 fp32 heads into e4m3: 107 us; 192
// threads 138, 256 the same, 96 108).  Two tokens a CTA halve the weights' loads but
// double the registers: bf16 rows gain (8191 tokens of 80 heads: 57 us, 61 with one), fp32
// rows lose (the former 94 us with one).
constexpr int kFewTokens = 148 * 4;

template <int XT, int TYPE>
void launch_qkv(const QkvParams& p, cudaStream_t s) {
  const int per = (p.n_heads + p.n_kv_heads * (TYPE == kRows ? 1 : 2)) << p.lanes_log2;
  const bool few = p.T <= kFewTokens;
  constexpr int kMany = XT == WAL_F32 ? 1 : 2;
  const int most = few ? 512 : 128, rounds = (per + most - 1) / most;
  const int threads = ((per + rounds - 1) / rounds + 31) / 32 * 32;  // whole warps, in equal rounds
  if (few)
    qkv_kernel<XT, TYPE, 1><<<p.T, threads, 0, s>>>(p);
  else
    qkv_kernel<XT, TYPE, kMany><<<(p.T + kMany - 1) / kMany, threads, 0, s>>>(p);
}

int check_norm(const wal_head_norm* n, int head_dim) {
  if (n->head_dim != head_dim) return fail(WAL_ERR_SHAPE, "the norm is for another head_dim");
  if (n->type != WAL_F32 && n->type != WAL_BF16) return fail(WAL_ERR_ARG, "the weights' type must be WAL_F32 or WAL_BF16");
  if (!n->q_weight || !n->k_weight || misaligned(n->q_weight, 4) || misaligned(n->k_weight, 4))
    return fail(WAL_ERR_ARG, "q_weight and k_weight are required, 4-byte aligned");
  if (!(n->eps > 0.f) || n->eps > 3.4e38f) return fail(WAL_ERR_ARG, "eps must be positive and finite");
  return WAL_OK;
}

// Rows of Y (bf16) may be those of X where X is bf16 of the same stride: a row is read before it is written.
int check_place(const void* X, int x_type, int ldx, const void* Y, int ldy, const char* what) {
  if (X == Y && (x_type != WAL_BF16 || ldx != ldy))
    return fail(WAL_ERR_ARG, std::string(what) + " may be written in place only as bf16 rows of the same stride");
  return WAL_OK;
}

void fill(QkvParams& p, const wal_head_norm* norm, const wal_rope_plan* rope, int head_dim) {
  if (norm) {
    p.weight[0] = norm->q_weight; p.weight[1] = norm->k_weight;
    p.weight_type = norm->type;
    p.eps = norm->eps;
  }
  if (rope) p.rope = {rope->freq, rope->rot_dim / 2, rope->layout, rope->mscale};
  p.head_dim = head_dim;
  p.items = head_dim / 16;
  p.lanes_log2 = log2_of(p.items);
}

}  // namespace
}  // namespace wal

using namespace wal;

extern "C" int wal_qk_norm_rope(const wal_head_norm* norm, const wal_rope_plan* rope, const void* Q, const void* K, int x_type, int T,
                                int n_heads, int n_kv_heads, int ldq, int ldk, const int32_t* positions, uint16_t* Yq, int ldyq,
                                uint16_t* Yk, int ldyk, wal_stream_t stream) {
  if (!rope) return fail(WAL_ERR_ARG, "rope plan is NULL");
  int st = check_rope(rope, rope->head_dim);
  if (st) return st;
  const int D = rope->head_dim;
  if (norm && (st = check_norm(norm, D))) return st;
  if (T < 0 || n_heads < 1 || n_kv_heads < 1) return fail(WAL_ERR_SHAPE, "T must be >= 0, n_heads and n_kv_heads >= 1");
  if (n_heads > 65536 || n_kv_heads > 65536) return fail(WAL_ERR_UNSUPPORTED, "at most 65536 heads");
  const int64_t wq = (int64_t)n_heads * D, wk = (int64_t)n_kv_heads * D;
  if ((st = check_rows(Q, x_type, ldq, wq, "Q")) || (st = check_rows(K, x_type, ldk, wk, "K")) ||
      (st = check_rows(Yq, WAL_BF16, ldyq, wq, "Yq")) || (st = check_rows(Yk, WAL_BF16, ldyk, wk, "Yk")))
    return st;
  if (misaligned(positions, 4)) return fail(WAL_ERR_ARG, "positions must be 4-byte aligned");
  if (T == 0) return WAL_OK;
  if (!Q || !K || !Yq || !Yk || !positions) return fail(WAL_ERR_ARG, "Q, K, Yq, Yk and positions are required");
  if ((st = check_place(Q, x_type, ldq, Yq, ldyq, "Q")) || (st = check_place(K, x_type, ldk, Yk, ldyk, "K"))) return st;
  if ((const void*)Yq == K || (const void*)Yk == Q || Yq == Yk) return fail(WAL_ERR_ARG, "Yq and Yk must not be each other or the other's input");
  int dev = 0;
  if ((st = current_device(&dev))) return st;
  QkvParams p = {};
  fill(p, norm, rope, D);
  p.x[0] = Q; p.x[1] = K;
  p.ld[0] = ldq; p.ld[1] = ldk;
  p.out[0] = Yq; p.out[1] = Yk;
  p.ldo[0] = ldyq; p.ldo[1] = ldyk;
  p.positions = positions;
  p.n_heads = n_heads; p.n_kv_heads = n_kv_heads;
  p.T = T;
  cudaStream_t s = (cudaStream_t)stream;
  if (x_type == WAL_F32)
    launch_qkv<WAL_F32, kRows>(p, s);
  else
    launch_qkv<WAL_BF16, kRows>(p, s);
  return launched("qkv_kernel");
}

extern "C" int wal_qkv_append(const wal_kv_cache* cache, const wal_head_norm* norm, const wal_rope_plan* rope, const void* Q,
                              const void* K, const void* V, int in_type, int T, int n_heads, int ldq, int ldk, int ldv,
                              const int32_t* slots, const int32_t* positions, uint16_t* Yq, int ldy, void* ws, size_t ws_bytes,
                              wal_stream_t stream) {
  int st = check_cache(cache);
  if (st) return st;
  const int D = cache->head_dim;
  if (rope && (st = check_rope(rope, D))) return st;
  if (norm && (st = check_norm(norm, D))) return st;
  if (T < 0 || n_heads < 1) return fail(WAL_ERR_SHAPE, "T must be >= 0 and n_heads >= 1");
  if (n_heads > 65536) return fail(WAL_ERR_UNSUPPORTED, "at most 65536 heads");
  const int64_t wq = (int64_t)n_heads * D, wk = (int64_t)cache->n_heads * D;
  if ((st = check_rows(Q, in_type, ldq, wq, "Q")) || (st = check_rows(K, in_type, ldk, wk, "K")) ||
      (st = check_rows(V, in_type, ldv, wk, "V")) || (st = check_rows(Yq, WAL_BF16, ldy, wq, "Yq")))
    return st;
  if (misaligned(slots, 4) || misaligned(positions, 4)) return fail(WAL_ERR_ARG, "slots and positions must be 4-byte aligned");
  if (T > 0 && (!Q || !K || !V || !Yq || !slots)) return fail(WAL_ERR_ARG, "Q, K, V, Yq and slots are required");
  if (T > 0 && rope && !positions) return fail(WAL_ERR_ARG, "positions are required with a rope plan");
  if (T > 0 && (st = check_place(Q, in_type, ldq, Yq, ldy, "Q"))) return st;
  if (T > 0 && ((const void*)Yq == K || (const void*)Yq == V)) return fail(WAL_ERR_ARG, "Yq must not be K or V");
  if (ws && ws_bytes < kStatusWs) return fail(WAL_ERR_WORKSPACE, "a workspace has at least 512 bytes");
  int dev = 0;
  if ((st = current_device(&dev))) return st;
  QkvParams p = {};
  cudaStream_t s = (cudaStream_t)stream;
  if (T == 0) return clear_status(ws, s, &p.status);
  p.status = status_word(ws);
  fill(p, norm, rope, D);
  p.x[0] = Q; p.x[1] = K; p.x[2] = V;
  p.ld[0] = ldq; p.ld[1] = ldk; p.ld[2] = ldv;
  p.out[0] = Yq;
  p.ldo[0] = ldy;
  p.cache[0] = cache->k; p.cache[1] = cache->v;
  p.scale[0] = cache->k_scale; p.scale[1] = cache->v_scale;
  p.slots = slots;
  p.positions = positions;
  p.n_heads = n_heads; p.n_kv_heads = cache->n_heads;
  p.shift = log2_of(cache->page_size);
  p.T = T;
  p.n_slots = (uint32_t)(cache->n_pages * cache->page_size);
  const bool f = in_type == WAL_F32;
  switch (cache->type) {
    case WAL_KV_BF16: f ? launch_qkv<WAL_F32, WAL_KV_BF16>(p, s) : launch_qkv<WAL_BF16, WAL_KV_BF16>(p, s); break;
    case WAL_KV_INT8: f ? launch_qkv<WAL_F32, WAL_KV_INT8>(p, s) : launch_qkv<WAL_BF16, WAL_KV_INT8>(p, s); break;
    default: f ? launch_qkv<WAL_F32, WAL_KV_E4M3>(p, s) : launch_qkv<WAL_BF16, WAL_KV_E4M3>(p, s); break;
  }
  return launched("qkv_kernel");
}
