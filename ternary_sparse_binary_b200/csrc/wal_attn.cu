// Attention entry points, the single-token kernel and the sum over splits.
//
//   O[t][h] = sum_j softmax_j(scale * Q[t][h] . K[j]) V[j]
//
// over the keys a token sees: the first len - n_q + i + 1 of its sequence for
// new token i.  One pass over the keys with the running maximum m and sum l:
// when m grows to m', l and the accumulator are multiplied by 2^(m - m').
#include "wal_attn.h"

#include <algorithm>
#include <cmath>

namespace wal {

namespace {

constexpr int kRowWarps = 4;

// Divide, round and store a row held by a warp.  A row that does not see every
// key and came out as NaN is done again from its own keys.
template <int D>
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
  if (__any_sync(0xffffffffu, nan) && lim < s.len) {
    attend_row<D>(p, s, b, head, tok);
    return;
  }
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.O + (s.q0 + tok) * p.ldo + head * D + lane * VPL);
#pragma unroll
  for (int i = 0; i < VPL / 2; ++i) dst[i] = dev::float2_to_bf16x2(y[2 * i], y[2 * i + 1]);
}

// ---------------------------------------------------------------------------
// few query rows: keys split over CTAs, mma.sync
// ---------------------------------------------------------------------------
// A CTA takes one (sequence, K/V head, split of the keys) and its 8 * NT query
// rows at most; its four warps take steps of 16 * MT keys in turn.  The keys
// are the M side of both products, so the few query rows waste little:
//   S^T[key][row] = K Q^T,   O^T[d][row] += V^T P^T,   m16n8k16, fp32 sums.
// Both A operands are built from 16-byte global loads without shared memory:
//  - K: the four lanes of a fragment row read neighbouring pieces of a key.  A
//    product over d may take d in any order, so Q is loaded in the same one;
//  - V: a lane reads the same columns of key pairs (2c, 2c + 1) and
//    interleaves them by byte permutes; which d a fragment row stands for is
//    undone when O is written;
//  - P: an 8 x 8 transpose (movmatrix) turns S^T's accumulator layout into the
//    B operand's.
// 8-bit codes are exact in bf16 and go to the tensor cores unscaled: the score
// gets the key's K scale, the weight its V scale, both in fp32.  Weights are
// rounded to bf16 for the second product (the operand type; 2^-8 of a weight,
// averaged over the keys); m, l, scores and O stay fp32.
constexpr int kDecWarps = 4;
constexpr int kDecMaxRows = 16;

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
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

// The loads of one key row by one lane: D / 4 elements of K, the lane's part.
template <int D, int TYPE>
struct RowWords {
  static constexpr int n = TYPE == WAL_KV_BF16 ? D / 8 : D / 16;  // 32-bit words of K (and of V) a lane holds per key
};

template <int D, int TYPE, int NT, int MT>
__global__ void __launch_bounds__(32 * kDecWarps) attn_decode_kernel(const __grid_constant__ AttnParams p) {
  constexpr int KB = TYPE == WAL_KV_BF16 ? 2 : 1;       // bytes of a code
  constexpr int W = RowWords<D, TYPE>::n;               // words of K per lane and key
  constexpr int NW = D * KB / 32;                       // words of V per lane and key (of 8 lanes)
  constexpr int DT = D / 16;                            // fragments along d
  constexpr int STEP = 16 * MT;
  __shared__ float s_o[kDecWarps][8 * NT][D + 4];
  __shared__ float2 s_ml[kDecWarps][8 * NT];
  const int b = blockIdx.z, h = blockIdx.y, split = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const AttnSeq s = attn_seq(p, b);
  if (p.clear) {
    if (split == 0 && h == 0 && b == 0 && threadIdx.x == 0) *p.status = 0;
  } else if (s.bad && h == 0 && threadIdx.x == 0 && p.status) {
    atomicExch(p.status, (int32_t)WAL_ERR_ARG);
  }
  if (s.bad) return;
  const int rows = s.n_q * p.group;
  const int k0 = split * p.split_keys, k1 = min(s.len, k0 + p.split_keys);
  if (rows == 0 || (k0 >= k1 && split > 0)) return;  // split 0 also answers for a sequence without keys

  // Q fragments: row g of tile t, the columns in the order of the K loads
  uint32_t q[NT][DT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int r = 8 * t + g;
    const bool live = r < rows;
    const uint16_t* src = p.Q + (s.q0 + (live ? r / p.group : 0)) * p.ldq + (h * p.group + (live ? r % p.group : 0)) * D;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {  // 16 bytes of Q: two fragments along d
      const int piece = TYPE == WAL_KV_BF16 ? 32 * i + 8 * c : 64 * (i >> 1) + 16 * c + 8 * (i & 1);
      uint4 v = make_uint4(0, 0, 0, 0);
      if (live) v = __ldg(reinterpret_cast<const uint4*>(src + piece));
      q[t][2 * i][0] = v.x;
      q[t][2 * i][1] = v.y;
      q[t][2 * i + 1][0] = v.z;
      q[t][2 * i + 1][1] = v.w;
    }
  }
  // this lane's columns of S^T: rows 8 t + 2 c + {0, 1}
  int lim[NT][2];
  float m[NT][2], l[NT][2];
  int lim_min = s.len;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 8 * t + 2 * c + e;
      lim[t][e] = r < rows ? attn_limit(s, r / p.group) : s.len;
      m[t][e] = -INFINITY;
      l[t][e] = 0.f;
    }
  lim_min = attn_limit(s, 0);
  float o[DT][NT][4];
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[d][t][e] = 0.f;

  const uint8_t* kbase = static_cast<const uint8_t*>(p.k);
  const uint8_t* vbase = static_cast<const uint8_t*>(p.v);
  for (int j0 = k0 + warp * STEP; j0 < k1; j0 += kDecWarps * STEP) {
    // rows of the 16-key tiles: a tile lies in one page
    int64_t row[MT];
#pragma unroll
    for (int u = 0; u < MT; ++u) row[u] = j0 + 16 * u < k1 ? attn_page_row(p, b, h, j0 + 16 * u) : 0;
    uint32_t kw[MT][2][W], vw[MT][4][NW];
    float ks[MT][2], vs[MT][2];
#pragma unroll
    for (int u = 0; u < MT; ++u) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int j = 16 * u + g + 8 * e;
        const bool live = j0 + j < k1;
        const uint8_t* src = kbase + (row[u] + g + 8 * e) * (D * KB) + 16 * c;
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (live) v = __ldg(reinterpret_cast<const uint4*>(src + 64 * i));
          kw[u][e][4 * i] = v.x; kw[u][e][4 * i + 1] = v.y; kw[u][e][4 * i + 2] = v.z; kw[u][e][4 * i + 3] = v.w;
        }
        if (TYPE != WAL_KV_BF16) {
          ks[u][e] = live ? __ldg(p.ks + row[u] + g + 8 * e) : 0.f;
          vs[u][e] = live ? __ldg(p.vs + row[u] + g + 8 * e) : 0.f;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < MT; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int jj = 2 * c + (e & 1) + 8 * (e >> 1);
        const bool live = j0 + 16 * u + jj < k1;
        const uint8_t* src = vbase + (row[u] + jj) * (D * KB);
        if (NW >= 4) {
#pragma unroll
          for (int i = 0; i < NW / 4; ++i) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (live) v = __ldg(reinterpret_cast<const uint4*>(src + 128 * i + 16 * g));
            vw[u][e][4 * i] = v.x; vw[u][e][4 * i + 1] = v.y; vw[u][e][4 * i + 2] = v.z; vw[u][e][4 * i + 3] = v.w;
          }
        } else {  // 8-bit rows of 64: 8 bytes a lane
          uint2 v = make_uint2(0, 0);
          if (live) v = __ldg(reinterpret_cast<const uint2*>(src + 8 * g));
          vw[u][e][0] = v.x; vw[u][e][1] = v.y;
        }
      }

    // S^T = K Q^T
    float sc[MT][NT][4];
#pragma unroll
    for (int u = 0; u < MT; ++u) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[u][t][e] = 0.f;
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        uint32_t a[4];
        if (TYPE == WAL_KV_BF16) {
          a[0] = kw[u][0][2 * d]; a[1] = kw[u][1][2 * d]; a[2] = kw[u][0][2 * d + 1]; a[3] = kw[u][1][2 * d + 1];
        } else {
          dev::codes4_to_bf16<TYPE>(kw[u][0][d], a[0], a[2]);
          dev::codes4_to_bf16<TYPE>(kw[u][1][d], a[1], a[3]);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) mma16816(sc[u][t], a[0], a[1], a[2], a[3], q[t][d][0], q[t][d][1]);
      }
    }
    // scores in log2 units; keys a row does not see get -inf
#pragma unroll
    for (int u = 0; u < MT; ++u)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = sc[u][t][e] * p.scale_log2;
          if (TYPE != WAL_KV_BF16) x *= ks[u][e >> 1];
          sc[u][t][e] = x;
        }
    if (j0 + STEP > lim_min || j0 + STEP > k1) {
#pragma unroll
      for (int u = 0; u < MT; ++u)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = j0 + 16 * u + g + 8 * (e >> 1);
            if (j >= min(k1, lim[t][e & 1])) sc[u][t][e] = -INFINITY;
          }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float corr[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float mx = m[t][e];
#pragma unroll
        for (int u = 0; u < MT; ++u) mx = fmaxf(mx, fmaxf(sc[u][t][e], sc[u][t][e + 2]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
        const float ref = mx == -INFINITY ? 0.f : mx;
        corr[e] = exp2f(m[t][e] - ref);
        m[t][e] = mx;
        l[t][e] *= corr[e];
#pragma unroll
        for (int u = 0; u < MT; ++u)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float w = exp2f(sc[u][t][e + 2 * r] - ref);
            l[t][e] += w;
            sc[u][t][e + 2 * r] = TYPE == WAL_KV_BF16 ? w : w * vs[u][r];
          }
      }
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[d][t][e] *= corr[e & 1];
    }
    // O^T += V^T P^T
#pragma unroll
    for (int u = 0; u < MT; ++u) {
      uint32_t pb[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        pb[t][0] = transpose8x8(dev::float2_to_bf16x2(sc[u][t][0], sc[u][t][1]));
        pb[t][1] = transpose8x8(dev::float2_to_bf16x2(sc[u][t][2], sc[u][t][3]));
      }
      if (TYPE == WAL_KV_BF16) {
#pragma unroll
        for (int d = 0; d < DT; ++d) {  // word d: columns 64 (d / 4) + 8 g + 2 (d % 4) + {0, 1}
          const uint32_t a0 = __byte_perm(vw[u][0][d], vw[u][1][d], 0x5410), a1 = __byte_perm(vw[u][0][d], vw[u][1][d], 0x7632);
          const uint32_t a2 = __byte_perm(vw[u][2][d], vw[u][3][d], 0x5410), a3 = __byte_perm(vw[u][2][d], vw[u][3][d], 0x7632);
#pragma unroll
          for (int t = 0; t < NT; ++t) mma16816(o[d][t], a0, a1, a2, a3, pb[t][0], pb[t][1]);
        }
      } else {
#pragma unroll
        for (int d = 0; d < DT; d += 2) {  // word d / 2: columns (D / 8) g + 2 d + {0 .. 3}
          uint32_t a[2][4];
          const uint32_t w0 = vw[u][0][d / 2], w1 = vw[u][1][d / 2], w2 = vw[u][2][d / 2], w3 = vw[u][3][d / 2];
          dev::codes4_to_bf16<TYPE>(__byte_perm(w0, w1, 0x5140), a[0][0], a[0][1]);
          dev::codes4_to_bf16<TYPE>(__byte_perm(w0, w1, 0x7362), a[1][0], a[1][1]);
          dev::codes4_to_bf16<TYPE>(__byte_perm(w2, w3, 0x5140), a[0][2], a[0][3]);
          dev::codes4_to_bf16<TYPE>(__byte_perm(w2, w3, 0x7362), a[1][2], a[1][3]);
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int t = 0; t < NT; ++t) mma16816(o[d + x][t], a[x][0], a[x][1], a[x][2], a[x][3], pb[t][0], pb[t][1]);
        }
      }
    }
  }

  // join the warps: each leaves its rows, then a warp takes a row
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float x = l[t][e];
      x += __shfl_xor_sync(0xffffffffu, x, 4);
      x += __shfl_xor_sync(0xffffffffu, x, 8);
      x += __shfl_xor_sync(0xffffffffu, x, 16);
      if (g == 0) s_ml[warp][8 * t + 2 * c + e] = make_float2(m[t][e], x);
    }
#pragma unroll
  for (int d = 0; d < DT; ++d) {
    // fragment rows g and g + 8 stand for neighbouring columns
    const int col = TYPE == WAL_KV_BF16 ? 64 * (d >> 2) + 8 * g + 2 * (d & 3) : (D / 8) * g + 2 * d;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) s_o[warp][8 * t + 2 * c + (e & 1)][col + (e >> 1)] = o[d][t][e];
  }
  __syncthreads();
  constexpr int VPL = D / 32;
  for (int r = warp; r < rows; r += kDecWarps) {
    float mm = -INFINITY;
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) mm = fmaxf(mm, s_ml[w][r].x);
    const float ref = mm == -INFINITY ? 0.f : mm;
    float acc[VPL], ll = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) acc[i] = 0.f;
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) {
      const float2 ml = s_ml[w][r];
      const float f = exp2f(ml.x - ref);
      ll += f * ml.y;
#pragma unroll
      for (int i = 0; i < VPL; ++i) acc[i] += f * s_o[w][r][lane * VPL + i];
    }
    const int tok = r / p.group, head = h * p.group + r % p.group;
    if (p.n_split > 1) {
      const int64_t pr = (int64_t)split * p.T * p.n_heads + attn_part_row(p, s, tok, head);
      float* dst = p.part_o + pr * D + lane * VPL;
      if (VPL == 4)
        *reinterpret_cast<float4*>(dst) = make_float4(acc[0], acc[1], acc[VPL - 2], acc[VPL - 1]);
      else
        *reinterpret_cast<float2*>(dst) = make_float2(acc[0], acc[1]);
      if (lane == 0) p.part_ml[pr] = make_float2(mm, ll);
    } else {
      finish_row<D>(p, s, b, head, tok, acc, ll);
    }
  }
}

// Add the splits of a row in order, one warp a row, and report index values out
// of range.
template <int D>
__global__ void __launch_bounds__(32 * kRowWarps) attn_combine_kernel(const __grid_constant__ AttnParams p) {
  constexpr int VPL = D / 32;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int b = blockIdx.z, lane = threadIdx.x & 31;
  const AttnSeq s = attn_seq(p, b);
  if (blockIdx.x == 0) {  // the first kernel cleared the status word; what it skipped is reported here
    bool bad = s.bad;
    const int pages = (s.len + (1 << p.shift) - 1) >> p.shift;
    for (int i = threadIdx.x; i < pages; i += 32 * kRowWarps) bad |= (uint32_t)__ldg(p.table + b * p.ld_table + i) >= (uint32_t)p.n_pages;
    if (bad) atomicExch(p.status, (int32_t)WAL_ERR_ARG);
  }
  const int row = blockIdx.x * kRowWarps + (threadIdx.x >> 5);  // (token, head)
  if (s.bad || row >= s.n_q * p.n_heads) return;
  const int tok = row / p.n_heads, head = row - tok * p.n_heads;
  const int n = max(1, (s.len + p.split_keys - 1) / p.split_keys);
  const int64_t pr = attn_part_row(p, s, tok, head), stride = (int64_t)p.T * p.n_heads;
  float mm = -INFINITY;
  for (int i = lane; i < n; i += 32) mm = fmaxf(mm, p.part_ml[pr + i * stride].x);
#pragma unroll
  for (int o = 16; o; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
  const float ref = mm == -INFINITY ? 0.f : mm;
  float acc[VPL], ll = 0.f;
#pragma unroll
  for (int i = 0; i < VPL; ++i) acc[i] = 0.f;
  for (int i = 0; i < n; ++i) {
    const float2 ml = p.part_ml[pr + i * stride];
    if (ml.x == -INFINITY && ml.y == 0.f) continue;  // a split in which the row sees nothing
    const float f = exp2f(ml.x - ref);
    ll += f * ml.y;
    const float* src = p.part_o + (pr + i * stride) * D + lane * VPL;
#pragma unroll
    for (int k = 0; k < VPL; ++k) acc[k] += f * src[k];
  }
  finish_row<D>(p, s, b, head, tok, acc, ll);
}

int check_attn(int n_heads, int n_kv_heads, int head_dim, int T, int B, int max_q, int max_kv, float scale) {
  if (n_heads < 1 || n_kv_heads < 1 || n_heads % n_kv_heads)
    return fail(WAL_ERR_SHAPE, "n_heads must be a positive multiple of the K/V heads");
  if (head_dim != 64 && head_dim != 128) return fail(WAL_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
  if (n_heads / n_kv_heads > 128 || n_kv_heads > 1024) return fail(WAL_ERR_UNSUPPORTED, "at most 128 q heads per K/V head and 1024 K/V heads");
  if (T < 0 || B < 1 || B > 65535 || max_q < 1 || max_kv < 1)
    return fail(WAL_ERR_SHAPE, "T >= 0, 1 <= B <= 65535 and the length bounds >= 1");
  if ((int64_t)max_q * (n_heads / n_kv_heads) > 0x7FFFFF00) return fail(WAL_ERR_UNSUPPORTED, "max_q * group must be below 2^31 - 256");
  if (((int64_t)T * n_heads / kTcAttnRows + (int64_t)B * n_kv_heads) > 0x7FFFFFFF / 128) return fail(WAL_ERR_UNSUPPORTED, "T * n_heads and B * n_kv_heads must stay below 2^32 and 2^24");
  if (!std::isfinite(scale)) return fail(WAL_ERR_ARG, "scale must be finite");
  return WAL_OK;
}

int check_bf16_rows(const void* X, int64_t ld, int64_t width, bool needed, const char* what) {
  if (needed && !X) return fail(WAL_ERR_ARG, std::string(what) + " is required");
  if (misaligned(X, 16)) return fail(WAL_ERR_ARG, std::string(what) + " must be 16-byte aligned");
  if (ld < width || ld % 8) return fail(WAL_ERR_ARG, std::string(what) + ": the row stride must cover the heads and be a multiple of 8");
  return WAL_OK;
}

size_t attn_ws_bytes(int n_split, int T, int n_heads, int head_dim) {
  if (n_split == 1) return kStatusWs;
  const size_t pr = (size_t)n_split * T * n_heads;
  return kStatusWs + align_up(pr * 8, 256) + pr * head_dim * 4;
}

int launched(cudaError_t e, const char* what) {
  if (e != cudaSuccess) return fail(WAL_ERR_CUDA, std::string(what) + " launch: " + cudaGetErrorString(e));
  return WAL_OK;
}

template <int D, int TYPE>
void launch_decode(const AttnParams& p, const dim3& grid, cudaStream_t s) {
  constexpr int MT2 = TYPE == WAL_KV_BF16 ? 1 : 2;  // sixteen rows: half the keys a step, to stay in registers
  if (p.max_q * p.group <= 8)
    attn_decode_kernel<D, TYPE, 1, 2><<<grid, 32 * kDecWarps, 0, s>>>(p);
  else
    attn_decode_kernel<D, TYPE, 2, MT2><<<grid, 32 * kDecWarps, 0, s>>>(p);
}

int launch_combine(const AttnParams& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(((int64_t)p.max_q * p.n_heads + kRowWarps - 1) / kRowWarps), 1, (unsigned)p.B);
  cfg.blockDim = dim3(32 * kRowWarps);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = p.head_dim == 64 ? cudaLaunchKernelEx(&cfg, attn_combine_kernel<64>, p)
                                         : cudaLaunchKernelEx(&cfg, attn_combine_kernel<128>, p);
  return launched(e, "attn_combine_kernel");
}

constexpr int kPlanSms = 148;  // SMs the splits are planned for: a constant, so that a workspace size holds on any device

// How the keys are split.
// Decode: a CTA holds a quarter to a half of an SM, so two an SM run at once;
// about six times as many pieces even out ragged lengths, and a piece has at
// least 128 keys.
// Tensor-core kernel: the split with the least estimated time, in steps of 128
// keys (about 1.8 us).  A piece costs three steps more than it has; pieces that
// more than fill the SMs leave about 1.2 pieces' time unused at the end, the
// more so as only bounds of the lengths are known here; a split writes and
// reads fp32 partial results at about 5.7 TB/s, and adds a launch.  Measured,
// without and with the split it takes: 2 x 1024 tokens over up to 16384 keys
// 368 and 159 us; 2 x 2048 over 4096 (none) 220, with three 321 us.
void plan_split(int64_t pieces, int64_t part_bytes, int max_kv, bool tc, int* n_split, int* split_keys) {
  const int64_t tiles = ((int64_t)max_kv + 127) / 128;
  int64_t best = 1;
  if (tc) {
    double best_cost = 0;
    for (int64_t s = 1; s <= 128 && s <= (tiles + 1) / 2; ++s) {
      const double r = (double)(pieces * s) / kPlanSms, steps = (double)((tiles + s - 1) / s) + 3;
      double cost = (r <= 1 ? 1 : r + 1.2) * steps;
      if (s > 1) cost += 3 + (double)part_bytes * s * 2 / (5.7e6 * 1.8);
      if (s == 1 || cost < best_cost) {
        best = s;
        best_cost = cost;
      }
    }
  } else {
    const int64_t even = (max_kv * pieces + 12 * kPlanSms - 1) / (12 * kPlanSms);
    best = std::max<int64_t>(1, tiles / std::max<int64_t>(1, (even + 127) / 128));
  }
  const int64_t keys = (tiles + best - 1) / best * 128;
  *split_keys = (int)std::min<int64_t>(keys, 0x7FFFFF80);
  *n_split = (int)((max_kv + keys - 1) / keys);
}

// Pieces of a call whose keys are not split: decode, one a (sequence, K/V head);
// else as many row tiles as T rows of B sequences can have.
int64_t attn_pieces(int B, int n_kv_heads, int group, int T, int max_q) {
  const int64_t rows = (int64_t)max_q * group;
  if (rows <= kDecMaxRows) return (int64_t)B * n_kv_heads;
  const int64_t most = B * ((rows + kTcAttnRows - 1) / kTcAttnRows);
  return n_kv_heads * std::min<int64_t>(most, (int64_t)T * group / kTcAttnRows + B);
}

int launch_attn(const AttnParams& p, cudaStream_t stream) {
  if (!p.table || (int64_t)p.max_q * p.group > kDecMaxRows) {
    const int st = launch_attn_tc(p, stream);
    return st || p.n_split == 1 ? st : launch_combine(p, stream);
  }
  const dim3 grid((unsigned)p.n_split, (unsigned)p.n_kv_heads, (unsigned)p.B);
  const bool wide = p.head_dim == 128;
  switch (p.type) {
    case WAL_KV_BF16: wide ? launch_decode<128, WAL_KV_BF16>(p, grid, stream) : launch_decode<64, WAL_KV_BF16>(p, grid, stream); break;
    case WAL_KV_INT8: wide ? launch_decode<128, WAL_KV_INT8>(p, grid, stream) : launch_decode<64, WAL_KV_INT8>(p, grid, stream); break;
    default: wide ? launch_decode<128, WAL_KV_E4M3>(p, grid, stream) : launch_decode<64, WAL_KV_E4M3>(p, grid, stream); break;
  }
  const int st = launched(cudaGetLastError(), "attn_decode_kernel");
  return st || p.n_split == 1 ? st : launch_combine(p, stream);
}

}  // namespace

}  // namespace wal

using namespace wal;

extern "C" size_t wal_attn_paged_workspace_bytes(const wal_kv_cache* cache, int n_heads, int T, int B, int max_q,
                                                 int max_kv) {
  if (check_cache(cache) != WAL_OK) return 0;
  if (check_attn(n_heads, cache->n_heads, cache->head_dim, T, B, max_q, max_kv, 1.f) != WAL_OK) return 0;
  int n_split, split_keys;
  const int64_t rows = (int64_t)std::max(1, std::min(max_q, T)) * (n_heads / cache->n_heads);
  plan_split(attn_pieces(B, cache->n_heads, n_heads / cache->n_heads, T, std::max(1, std::min(max_q, T))), (int64_t)T * n_heads * cache->head_dim * 4, max_kv, rows > kDecMaxRows, &n_split, &split_keys);
  return attn_ws_bytes(n_split, T, n_heads, cache->head_dim);
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
  int dev = 0;
  AttnParams p = {};
  cudaStream_t s = (cudaStream_t)stream;
  const int64_t rows = (int64_t)std::max(1, std::min(max_q, T)) * (n_heads / cache->n_heads);
  plan_split(attn_pieces(B, cache->n_heads, n_heads / cache->n_heads, T, std::max(1, std::min(max_q, T))), (int64_t)T * n_heads * cache->head_dim * 4, max_kv, rows > kDecMaxRows, &p.n_split, &p.split_keys);
  if ((ws || p.n_split > 1) && (!ws || ws_bytes < attn_ws_bytes(p.n_split, T, n_heads, cache->head_dim)))
    return fail(WAL_ERR_WORKSPACE, "workspace too small");
  if ((st = current_device(&dev))) return st;
  p.clear = T > 0 && p.n_split > 1;
  p.status = status_word(ws);
  if (!p.clear && (st = clear_status(ws, s, &p.status))) return st;
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
  char* part = reinterpret_cast<char*>(p.status) + 256;
  p.part_ml = reinterpret_cast<float2*>(part);
  p.part_o = reinterpret_cast<float*>(part + align_up((size_t)p.n_split * T * n_heads * 8, 256));
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
  if (ws && ws_bytes < kStatusWs) return fail(WAL_ERR_WORKSPACE, "a workspace has at least 512 bytes");
  int dev = 0;
  if ((st = current_device(&dev))) return st;
  AttnParams p = {};
  cudaStream_t s = (cudaStream_t)stream;
  if (T == 0) return clear_status(ws, s, &p.status);
  p.clear = ws != nullptr;
  p.status = status_word(ws);
  p.Q = Q; p.O = O;
  p.k = K; p.v = V;
  p.q_start = start;
  p.ldq = ldq; p.ldo = ldo; p.ldk = ldk; p.ldv = ldv;
  p.n_heads = n_heads; p.n_kv_heads = n_kv_heads; p.group = n_heads / n_kv_heads;
  p.head_dim = head_dim; p.type = WAL_KV_BF16;
  p.T = T; p.B = B; p.max_q = p.max_kv = max_len < T ? max_len : T;
  p.n_split = 1; p.split_keys = p.max_kv;
  p.scale_log2 = scale * 1.4426950408889634f;
  return launch_attn(p, s);
}
