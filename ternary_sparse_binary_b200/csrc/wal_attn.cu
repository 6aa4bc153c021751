// Attention entry points and the kernels that run on CUDA cores.
//
//   O[t][h] = sum_j softmax_j(scale * Q[t][h] . K[j]) V[j]
//
// over the keys a token sees: the first len - n_q + i + 1 of its sequence for
// new token i.  One pass over the keys with the running maximum m and sum l:
// when m grows to m', l and the accumulator are multiplied by 2^(m - m').
#include "wal_attn.h"

#include <cmath>

namespace wal {

namespace {

// One row by one warp, in fp32: lane i holds columns [i * VPL, (i + 1) * VPL).
// Only visible keys are touched, and a non-finite one among them acts as in
// the formula: a NaN score, a +inf score, scores that are all -inf, or a
// non-finite value under any weight give NaN.
template <int D>
__device__ void attend_row(const AttnParams& p, const AttnSeq& s, int b, int head, int tok) {
  constexpr int VPL = D / 32;
  const int lane = threadIdx.x & 31, h = head / p.group;
  const int lim = attn_limit(s, tok);
  float q[VPL], acc[VPL];
  const uint16_t* qr = p.Q + (s.q0 + tok) * p.ldq + head * D + lane * VPL;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    q[i] = __uint_as_float((uint32_t)qr[i] << 16);
    acc[i] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < lim; ++j) {
    float k[VPL], v[VPL];
    if (p.table && p.type != WAL_KV_BF16) {
      const int64_t row = attn_page_row(p, b, h, j);
      const uint8_t* kc = static_cast<const uint8_t*>(p.k) + row * D + lane * VPL;
      const uint8_t* vc = static_cast<const uint8_t*>(p.v) + row * D + lane * VPL;
      const float ks = p.ks[row], vs = p.vs[row];
      uint32_t kw = 0, vw = 0;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        kw |= (uint32_t)kc[i] << (8 * i);
        vw |= (uint32_t)vc[i] << (8 * i);
      }
      float kf[4], vf[4];
      if (p.type == WAL_KV_INT8) {
        dev::codes4_to_float<WAL_KV_INT8>(kw, kf);
        dev::codes4_to_float<WAL_KV_INT8>(vw, vf);
      } else {
        dev::codes4_to_float<WAL_KV_E4M3>(kw, kf);
        dev::codes4_to_float<WAL_KV_E4M3>(vw, vf);
      }
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        k[i] = kf[i] * ks;
        v[i] = vf[i] * vs;
      }
    } else {
      const uint16_t *kr, *vr;
      if (p.table) {
        const int64_t row = attn_page_row(p, b, h, j);
        kr = static_cast<const uint16_t*>(p.k) + row * D;
        vr = static_cast<const uint16_t*>(p.v) + row * D;
      } else {
        kr = static_cast<const uint16_t*>(p.k) + (int64_t)(s.q0 + j) * p.ldk + h * D;
        vr = static_cast<const uint16_t*>(p.v) + (int64_t)(s.q0 + j) * p.ldv + h * D;
      }
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        k[i] = __uint_as_float((uint32_t)kr[lane * VPL + i] << 16);
        v[i] = __uint_as_float((uint32_t)vr[lane * VPL + i] << 16);
      }
    }
    float x = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) x += q[i] * k[i];
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    x *= p.scale_log2;
    const float mn = fmaxf(m, x);
    const float c = m == -INFINITY ? 1.f : exp2f(m - mn);  // nothing summed yet, or only weights of zero
    const float w = x == -INFINITY ? 0.f : exp2f(x - mn);
    m = mn;
    l = l * c + w;
#pragma unroll
    for (int i = 0; i < VPL; ++i) acc[i] = acc[i] * c + w * v[i];
  }
  uint16_t* o = p.O + (s.q0 + tok) * p.ldo + head * D + lane * VPL;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const float y = lim == 0 ? 0.f : acc[i] / l;
    o[i] = (uint16_t)(dev::float2_to_bf16x2(y, 0.f) & 0xFFFFu);
  }
}

constexpr int kRowWarps = 4;

template <int D>
__global__ void __launch_bounds__(32 * kRowWarps) attn_rows_kernel(const AttnParams p) {
  const int b = blockIdx.z;
  const AttnSeq s = attn_seq(p, b);
  if (s.bad) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) atomicExch(p.status, (int32_t)WAL_ERR_ARG);
    return;
  }
  const int head = blockIdx.y * kRowWarps + (threadIdx.x >> 5);
  if ((int)blockIdx.x < s.n_q && head < p.n_heads) attend_row<D>(p, s, b, head, blockIdx.x);
}

int check_attn(int n_heads, int n_kv_heads, int head_dim, int T, int B, int max_q, int max_kv, float scale) {
  if (n_heads < 1 || n_kv_heads < 1 || n_heads % n_kv_heads)
    return fail(WAL_ERR_SHAPE, "n_heads must be a positive multiple of the K/V heads");
  if (head_dim != 64 && head_dim != 128) return fail(WAL_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
  if (n_heads / n_kv_heads > 128 || n_kv_heads > 1024) return fail(WAL_ERR_UNSUPPORTED, "at most 128 q heads per K/V head and 1024 K/V heads");
  if (T < 0 || B < 1 || B > 65535 || max_q < 1 || max_kv < 1)
    return fail(WAL_ERR_SHAPE, "T >= 0, 1 <= B <= 65535 and the length bounds >= 1");
  if ((int64_t)max_q * (n_heads / n_kv_heads) > 0x7FFFFF00) return fail(WAL_ERR_UNSUPPORTED, "max_q * group must be below 2^31 - 256");
  if (!std::isfinite(scale)) return fail(WAL_ERR_ARG, "scale must be finite");
  return WAL_OK;
}

int check_bf16_rows(const void* X, int64_t ld, int64_t width, bool needed, const char* what) {
  if (needed && !X) return fail(WAL_ERR_ARG, std::string(what) + " is required");
  if (misaligned(X, 16)) return fail(WAL_ERR_ARG, std::string(what) + " must be 16-byte aligned");
  if (ld < width || ld % 8) return fail(WAL_ERR_ARG, std::string(what) + ": the row stride must cover the heads and be a multiple of 8");
  return WAL_OK;
}

int launch_attn(const AttnParams& p, cudaStream_t stream) {
  const dim3 grid((unsigned)p.max_q, (unsigned)((p.n_heads + kRowWarps - 1) / kRowWarps), (unsigned)p.B);
  if (p.head_dim == 64)
    attn_rows_kernel<64><<<grid, 32 * kRowWarps, 0, stream>>>(p);
  else
    attn_rows_kernel<128><<<grid, 32 * kRowWarps, 0, stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(WAL_ERR_CUDA, std::string("attn_rows_kernel launch: ") + cudaGetErrorString(e));
  return WAL_OK;
}

}  // namespace
}  // namespace wal

using namespace wal;

extern "C" size_t wal_attn_paged_workspace_bytes(const wal_kv_cache* cache, int n_heads, int T, int B, int max_q,
                                                 int max_kv) {
  if (check_cache(cache) != WAL_OK) return 0;
  if (check_attn(n_heads, cache->n_heads, cache->head_dim, T, B, max_q, max_kv, 1.f) != WAL_OK) return 0;
  return kStatusWs;
}

extern "C" int wal_attn_paged(const wal_kv_cache* cache, const uint16_t* Q, int n_heads, int T, int ldq,
                              const int32_t* q_start, const int32_t* kv_len, const int32_t* table, int ld_table,
                              int B, int max_q, int max_kv, float scale, uint16_t* O, int ldo, void* ws,
                              size_t ws_bytes, wal_stream_t stream) {
  int st = check_cache(cache);
  if (st) return st;
  if ((st = check_attn(n_heads, cache->n_heads, cache->head_dim, T, B, max_q, max_kv, scale))) return st;
  const int64_t width = (int64_t)n_heads * cache->head_dim;
  if ((st = check_bf16_rows(Q, ldq, width, T > 0, "Q")) || (st = check_bf16_rows(O, ldo, width, T > 0, "O"))) return st;
  if (!q_start || !kv_len || !table || misaligned(q_start, 4) || misaligned(kv_len, 4) || misaligned(table, 4))
    return fail(WAL_ERR_ARG, "q_start, kv_len and table are required, 4-byte aligned");
  if ((int64_t)ld_table * cache->page_size < max_kv) return fail(WAL_ERR_ARG, "ld_table pages must cover max_kv tokens");
  if (!ws || ws_bytes < wal_attn_paged_workspace_bytes(cache, n_heads, T, B, max_q, max_kv))
    return fail(WAL_ERR_WORKSPACE, "workspace too small");
  int dev = 0;
  if ((st = current_device(&dev))) return st;
  AttnParams p = {};
  cudaStream_t s = (cudaStream_t)stream;
  if ((st = clear_status(ws, s, &p.status))) return st;
  if (T == 0) return WAL_OK;
  p.Q = Q; p.O = O;
  p.k = cache->k; p.v = cache->v;
  p.ks = cache->k_scale; p.vs = cache->v_scale;
  p.q_start = q_start; p.kv_len = kv_len; p.table = table;
  p.ldq = ldq; p.ldo = ldo; p.ld_table = ld_table;
  p.n_heads = n_heads; p.n_kv_heads = cache->n_heads; p.group = n_heads / cache->n_heads;
  p.head_dim = cache->head_dim; p.type = cache->type;
  p.shift = log2_of(cache->page_size); p.n_pages = cache->n_pages;
  p.T = T; p.B = B; p.max_q = max_q < T ? max_q : T; p.max_kv = max_kv;
  p.scale_log2 = scale * 1.4426950408889634f;
  return launch_attn(p, s);
}

extern "C" int wal_attn_prompt(const uint16_t* Q, const uint16_t* K, const uint16_t* V, int n_heads, int n_kv_heads,
                               int head_dim, int T, int ldq, int ldk, int ldv, const int32_t* start, int B,
                               int max_len, float scale, uint16_t* O, int ldo, void* ws, size_t ws_bytes,
                               wal_stream_t stream) {
  int st = check_attn(n_heads, n_kv_heads, head_dim, T, B, max_len, max_len, scale);
  if (st) return st;
  const int64_t width = (int64_t)n_heads * head_dim, kv_width = (int64_t)n_kv_heads * head_dim;
  if ((st = check_bf16_rows(Q, ldq, width, T > 0, "Q")) || (st = check_bf16_rows(K, ldk, kv_width, T > 0, "K")) ||
      (st = check_bf16_rows(V, ldv, kv_width, T > 0, "V")) || (st = check_bf16_rows(O, ldo, width, T > 0, "O")))
    return st;
  if (!start || misaligned(start, 4)) return fail(WAL_ERR_ARG, "start is required, 4-byte aligned");
  if (!ws || ws_bytes < kStatusWs) return fail(WAL_ERR_WORKSPACE, "prompt attention needs a 512-byte workspace");
  int dev = 0;
  if ((st = current_device(&dev))) return st;
  AttnParams p = {};
  cudaStream_t s = (cudaStream_t)stream;
  if ((st = clear_status(ws, s, &p.status))) return st;
  if (T == 0) return WAL_OK;
  p.Q = Q; p.O = O;
  p.k = K; p.v = V;
  p.q_start = start;
  p.ldq = ldq; p.ldo = ldo; p.ldk = ldk; p.ldv = ldv;
  p.n_heads = n_heads; p.n_kv_heads = n_kv_heads; p.group = n_heads / n_kv_heads;
  p.head_dim = head_dim; p.type = WAL_KV_BF16;
  p.T = T; p.B = B; p.max_q = p.max_kv = max_len < T ? max_len : T;
  p.scale_log2 = scale * 1.4426950408889634f;
  return launch_attn(p, s);
}
