// Attention entry points, the single-token kernel and the sum over splits.
//
//   O[t][h] = sum_j softmax_j(scale * Q[t][h] . K[j]) V[j]
//
// over the keys a token sees: the first len - n_q + i + 1 of its sequence for
// new token i.  One pass over the keys with the running maximum m and sum l:
// when m grows to m', l and the accumulator are multiplied by 2^(m - m').
#include "wal_attn.h"
#include "wal_ptx.cuh"

#include <algorithm>
#include <atomic>
#include <cmath>

namespace wal {

namespace {

constexpr int kRowWarps = 4;

// Divide, round and store a row held by a warp.  A row that came out as NaN
// beside a non-finite V which it does not see is done again from its own keys.
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
  if (__any_sync(0xffffffffu, nan && l == l)) {
    const int h = head / p.group, reach = attn_reach(p, s, tok * p.group + head - h * p.group);
    if (lim < reach && attn_last_nonfinite<D>(p, s, b, h, lim, reach) >= 0) {
      attend_row<D>(p, s, b, head, tok);
      return;
    }
  }
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.O + (s.q0 + tok) * p.ldo + head * D + lane * VPL);
#pragma unroll
  for (int i = 0; i < VPL / 2; ++i) dst[i] = dev::float2_to_bf16x2(y[2 * i], y[2 * i + 1]);
}

// ---------------------------------------------------------------------------
// few query rows: keys split over CTAs, mma.sync
// ---------------------------------------------------------------------------
// Bound by bytes over bf16 (25 sequences of up to 16384 keys, 8 heads of 128: 133 us,
// 0.93 of the copy rate) and by latency over codes (up to 32768 int8 keys: 179 us,
// 0.71; registers allow 8 warps an SM, which use 41 % of the issue slots); one
// sequence of 2048 keys takes 8.9 us of a graph, both kernels.
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
// 8-bit codes go to the tensor cores unscaled, as fp16 (exact, and half the
// instructions of bf16); the score gets the key's K scale in fp32.  Q is then
// fp16 too, each row brought to [1, 2) by a power of two: nothing is lost down to
// 2^-14 of the row's largest, and 2^-25 of it below.  V's scale belongs to the
// weight, and a small one must not cost an fp16 weight its digits: O has a
// reference of its own, m2 = max(score + log2 |V scale|), so that its weights are
// at most about 1 where they count.  bf16 caches stay bf16 (m2 = m).  Weights are
// rounded for the second product (2^-8 or 2^-11 of a weight, averaged over the
// keys); references, l, scores and O are fp32.
// References are lazy: they follow the maximum when it has grown by more than
// 2^4, which a vote finds; most steps have no reduction and leave O alone.
constexpr int kDecWarps = 4;
constexpr int kDecMaxRows = 16;

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

template <int D, int TYPE, int NT, int MT>
__global__ void __launch_bounds__(32 * kDecWarps, TYPE == WAL_KV_BF16 && NT == 1 ? 3 : 2) attn_decode_kernel(const __grid_constant__ AttnParams p) {
  constexpr bool CODES = TYPE != WAL_KV_BF16;
  constexpr int KB = CODES ? 1 : 2;      // bytes of a code
  constexpr int W = D * KB / 16;         // 32-bit words of K per lane and key (of 4 lanes)
  constexpr int NW = D * KB / 32;        // words of V per lane and key (of 8 lanes)
  constexpr int DT = D / 16;             // fragments along d
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
    attn_report(p.status);
  }
  if (s.bad) return;
  const int rows = s.n_q * p.group;
  const int k0 = split * p.split_keys, k1 = min(s.len, k0 + p.split_keys);
  if (rows == 0 || (k0 >= k1 && split > 0)) return;  // split 0 also answers for a sequence without keys

  // K and V of a step, and where they lie: a tile of 16 keys is in one page
  uint32_t kw[MT][2][W], vw[MT][4][NW];
  float ks[MT][2], vs[MT][2];
  int64_t row[MT];
  auto find = [&](int j0) {
#pragma unroll
    for (int u = 0; u < MT; ++u) row[u] = j0 + 16 * u < k1 ? attn_page_row(p, b, h, j0 + 16 * u) : 0;
  };
  auto load_k = [&](int j0) {
    const uint8_t* base = static_cast<const uint8_t*>(p.k);
#pragma unroll
    for (int u = 0; u < MT; ++u)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int j = g + 8 * e;
        const bool live = j0 + 16 * u + j < k1;
        const uint8_t* src = base + (row[u] + j) * (D * KB) + 16 * c;
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (live) v = __ldg(reinterpret_cast<const uint4*>(src + 64 * i));
          kw[u][e][4 * i] = v.x; kw[u][e][4 * i + 1] = v.y; kw[u][e][4 * i + 2] = v.z; kw[u][e][4 * i + 3] = v.w;
        }
        if (CODES) ks[u][e] = live ? __ldg(p.ks + row[u] + j) : 0.f;
      }
  };
  auto load_v = [&](int j0) {
    const uint8_t* base = static_cast<const uint8_t*>(p.v);
#pragma unroll
    for (int u = 0; u < MT; ++u) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = 2 * c + (e & 1) + 8 * (e >> 1);
        const bool live = j0 + 16 * u + j < k1;
        const uint8_t* src = base + (row[u] + j) * (D * KB);
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
      if (CODES)
#pragma unroll
        for (int e = 0; e < 2; ++e) vs[u][e] = j0 + 16 * u + g + 8 * e < k1 ? __ldg(p.vs + row[u] + g + 8 * e) : 0.f;
    }
  };
  int j0 = k0 + warp * STEP;
  find(j0);
  load_k(j0);
  load_v(j0);

  // Q fragments: row g of tile t, the columns in the order of the K loads
  uint32_t q[NT][DT][2];
  float mult[NT][2];  // of the scores of this lane's columns of S^T: rows 8 t + 2 c + {0, 1}
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int r = 8 * t + g;
    const bool live = r < rows;
    const uint16_t* src = p.Q + (s.q0 + (live ? r / p.group : 0)) * p.ldq + (h * p.group + (live ? r % p.group : 0)) * D;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {  // 16 bytes of Q: two fragments along d
      const int piece = CODES ? 64 * (i >> 1) + 16 * c + 8 * (i & 1) : 32 * i + 8 * c;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (live) v = __ldg(reinterpret_cast<const uint4*>(src + piece));
      q[t][2 * i][0] = v.x;
      q[t][2 * i][1] = v.y;
      q[t][2 * i + 1][0] = v.z;
      q[t][2 * i + 1][1] = v.w;
      top = max(max(max(top, v.x & 0x7FFFu), (v.x >> 16) & 0x7FFFu), max(v.y & 0x7FFFu, (v.y >> 16) & 0x7FFFu));
      top = max(max(max(top, v.z & 0x7FFFu), (v.z >> 16) & 0x7FFFu), max(v.w & 0x7FFFu, (v.w >> 16) & 0x7FFFu));
    }
    mult[t][0] = mult[t][1] = p.scale_log2;
    if (CODES) {
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const uint32_t e = min(max(top >> 7, 1u), 253u);  // biased exponent of the row's largest
      const float down = __uint_as_float((254u - e) << 23), up = __uint_as_float(e << 23) * p.scale_log2;
#pragma unroll
      for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float2 f = dev::bf16x2_to_float2(q[t][i][k]);
          q[t][i][k] = dev::float2_to_half2(f.x * down, f.y * down);
        }
      mult[t][0] = __shfl_sync(0xffffffffu, up, 8 * c);
      mult[t][1] = __shfl_sync(0xffffffffu, up, 8 * c + 4);
    }
  }
  int lim[NT][2];
  float m[NT][2], m2[NT][2], l[NT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 8 * t + 2 * c + e;
      lim[t][e] = r < rows ? attn_limit(s, r / p.group) : s.len;
      m[t][e] = m2[t][e] = -INFINITY;
      l[t][e] = 0.f;
    }
  const int lim_min = min(k1, attn_limit(s, 0));
  float o[DT][NT][4];
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[d][t][e] = 0.f;

#pragma unroll 1
  for (; j0 < k1; j0 += kDecWarps * STEP) {
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
        if (CODES) {
          dev::codes4_to_half<TYPE>(kw[u][0][d], a[0], a[2]);
          dev::codes4_to_half<TYPE>(kw[u][1][d], a[1], a[3]);
        } else {
          a[0] = kw[u][0][2 * d]; a[1] = kw[u][1][2 * d]; a[2] = kw[u][0][2 * d + 1]; a[3] = kw[u][1][2 * d + 1];
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) mma16816<CODES>(sc[u][t], a[0], a[1], a[2], a[3], q[t][d][0], q[t][d][1]);
      }
    }
    // scores in log2 units, and (codes) what V's scale adds to them
    float lv[MT][2];
#pragma unroll
    for (int u = 0; u < MT; ++u)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        lv[u][r] = CODES ? lg2(fabsf(vs[u][r])) : 0.f;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float& x = sc[u][t][e + 2 * r];
            x *= mult[t][e];
            if (CODES) x *= ks[u][r];
          }
      }
    if (j0 + STEP > lim_min) {  // keys a row does not see get -inf
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
    // the next step's K, in the registers of this one's
    const int jn = j0 + kDecWarps * STEP;
    find(jn);
    load_k(jn);

    float mx[NT][2], mx2[NT][2];
    bool grow = false;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mx[t][e] = sc[0][t][e];
        mx2[t][e] = sc[0][t][e] + lv[0][0];
#pragma unroll
        for (int u = 0; u < MT; ++u)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            mx[t][e] = fmaxf(mx[t][e], sc[u][t][e + 2 * r]);
            if (CODES) mx2[t][e] = fmaxf(mx2[t][e], sc[u][t][e + 2 * r] + lv[u][r]);
          }
        grow |= mx[t][e] > m[t][e] + kDecLazy || (CODES && mx2[t][e] > m2[t][e] + kDecLazy);
      }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float corr[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          auto join = [&](float x, float old) {
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
            return fmaxf(fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16)), old);
          };
          const float n = join(mx[t][e], m[t][e]);
          const float f = m[t][e] == -INFINITY ? 0.f : ex2(m[t][e] - n);
          m[t][e] = n;
          l[t][e] *= f;
          corr[e] = f;
          if (CODES) {
            const float n2 = join(mx2[t][e], m2[t][e]);
            corr[e] = m2[t][e] == -INFINITY ? 0.f : ex2(m2[t][e] - n2);
            m2[t][e] = n2;
          }
        }
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[d][t][e] *= corr[e & 1];
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float ref = m[t][e] == -INFINITY ? 0.f : m[t][e], ref2 = m2[t][e] == -INFINITY ? 0.f : m2[t][e];
#pragma unroll
        for (int u = 0; u < MT; ++u)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float& x = sc[u][t][e + 2 * r];
            const float w = ex2(x - ref);
            l[t][e] += w;
            x = CODES ? copysignf(ex2(x + lv[u][r] - ref2), vs[u][r]) : w;
          }
      }
    // O^T += V^T P^T
#pragma unroll
    for (int u = 0; u < MT; ++u) {
      uint32_t pb[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        pb[t][0] = transpose8x8(CODES ? dev::float2_to_half2(sc[u][t][0], sc[u][t][1]) : dev::float2_to_bf16x2(sc[u][t][0], sc[u][t][1]));
        pb[t][1] = transpose8x8(CODES ? dev::float2_to_half2(sc[u][t][2], sc[u][t][3]) : dev::float2_to_bf16x2(sc[u][t][2], sc[u][t][3]));
      }
      if (!CODES) {
#pragma unroll
        for (int d = 0; d < DT; ++d) {  // word d: columns 64 (d / 4) + 8 g + 2 (d % 4) + {0, 1}
          const uint32_t a0 = __byte_perm(vw[u][0][d], vw[u][1][d], 0x5410), a1 = __byte_perm(vw[u][0][d], vw[u][1][d], 0x7632);
          const uint32_t a2 = __byte_perm(vw[u][2][d], vw[u][3][d], 0x5410), a3 = __byte_perm(vw[u][2][d], vw[u][3][d], 0x7632);
#pragma unroll
          for (int t = 0; t < NT; ++t) mma16816<CODES>(o[d][t], a0, a1, a2, a3, pb[t][0], pb[t][1]);
        }
      } else {
#pragma unroll
        for (int d = 0; d < DT; d += 2) {  // word d / 2: columns (D / 8) g + 2 d + {0 .. 3}
          uint32_t a[2][4];
          const uint32_t w0 = vw[u][0][d / 2], w1 = vw[u][1][d / 2], w2 = vw[u][2][d / 2], w3 = vw[u][3][d / 2];
          dev::codes4_to_half<TYPE>(__byte_perm(w0, w1, 0x5140), a[0][0], a[0][1]);
          dev::codes4_to_half<TYPE>(__byte_perm(w0, w1, 0x7362), a[1][0], a[1][1]);
          dev::codes4_to_half<TYPE>(__byte_perm(w2, w3, 0x5140), a[0][2], a[0][3]);
          dev::codes4_to_half<TYPE>(__byte_perm(w2, w3, 0x7362), a[1][2], a[1][3]);
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int t = 0; t < NT; ++t) mma16816<CODES>(o[d + x][t], a[x][0], a[x][1], a[x][2], a[x][3], pb[t][0], pb[t][1]);
        }
      }
    }
    load_v(jn);
  }
  if (CODES) {  // O in units of m, as l is
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float f = m2[t][e & 1] == -INFINITY ? 0.f : ex2(m2[t][e & 1] - m[t][e & 1]);
#pragma unroll
        for (int d = 0; d < DT; ++d) o[d][t][e] *= f;
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

// Add the splits of a row, and report index values out of range.  PER warps of
// the CTA share a row, each its splits in order, joined in order: one where
// there are few splits, four where a warp alone would wait for one load after
// the other.
template <int D, int PER>
__global__ void __launch_bounds__(32 * kRowWarps) attn_combine_kernel(const __grid_constant__ AttnParams p) {
  constexpr int VPL = D / 32;
  __shared__ float s_o[PER > 1 ? kRowWarps : 1][D];
  __shared__ float s_l[PER > 1 ? kRowWarps : 1];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int b = blockIdx.z, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const AttnSeq s = attn_seq(p, b);
  if (blockIdx.x == 0) {  // the first kernel cleared the status word; what it skipped is reported here
    bool bad = s.bad;
    const int pages = (s.len + (1 << p.shift) - 1) >> p.shift;
    for (int i = threadIdx.x; i < pages; i += 32 * kRowWarps) bad |= (uint32_t)__ldg(p.table + b * p.ld_table + i) >= (uint32_t)p.n_pages;
    if (bad) attn_report(p.status);
  }
  const int row = blockIdx.x * (kRowWarps / PER) + warp / PER;  // (token, head)
  if (s.bad || row >= s.n_q * p.n_heads) return;                // PER > 1: the whole CTA
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
#pragma unroll 4
  for (int i = warp % PER; i < n; i += PER) {
    const float2 ml = p.part_ml[pr + i * stride];
    const float* src = p.part_o + (pr + i * stride) * D + lane * VPL;
    float v[VPL];
#pragma unroll
    for (int k = 0; k < VPL; ++k) v[k] = src[k];
    const bool none = ml.x == -INFINITY && ml.y == 0.f;  // the row sees nothing of this split
    const float f = exp2f(ml.x - ref);
    ll += none ? 0.f : f * ml.y;
#pragma unroll
    for (int k = 0; k < VPL; ++k) acc[k] += none ? 0.f : f * v[k];
  }
  if (PER > 1) {
#pragma unroll
    for (int k = 0; k < VPL; ++k) s_o[warp][lane * VPL + k] = acc[k];
    if (lane == 0) s_l[warp] = ll;
    __syncthreads();
    if (warp > 0) return;
    ll = 0.f;
#pragma unroll
    for (int k = 0; k < VPL; ++k) acc[k] = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      ll += s_l[i];
#pragma unroll
      for (int k = 0; k < VPL; ++k) acc[k] += s_o[i][lane * VPL + k];
    }
  }
  finish_row<D>(p, s, b, head, tok, acc, ll);
}

// Longest sequence: the kernels add a split or a step to a key's number in 32 bits.
constexpr int kMaxKeys = 1 << 30;

int check_attn(int n_heads, int n_kv_heads, int head_dim, int T, int B, int max_q, int max_kv, float scale) {
  if (n_heads < 1 || n_kv_heads < 1 || n_heads % n_kv_heads)
    return fail(WAL_ERR_SHAPE, "n_heads must be a positive multiple of the K/V heads");
  if (head_dim != 64 && head_dim != 128) return fail(WAL_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
  if (n_heads / n_kv_heads > 128 || n_kv_heads > 1024) return fail(WAL_ERR_UNSUPPORTED, "at most 128 q heads per K/V head and 1024 K/V heads");
  if (T < 0 || B < 1 || B > 65535 || max_q < 1 || max_kv < 1)
    return fail(WAL_ERR_SHAPE, "T >= 0, 1 <= B <= 65535 and the length bounds >= 1");
  if ((int64_t)max_q * (n_heads / n_kv_heads) > 0x7FFFFF00) return fail(WAL_ERR_UNSUPPORTED, "max_q * group must be below 2^31 - 256");
  if (((int64_t)T * n_heads / kTcAttnRows + (int64_t)B * n_kv_heads) > 0x7FFFFFFF / 128) return fail(WAL_ERR_UNSUPPORTED, "T * n_heads and B * n_kv_heads must stay below 2^32 and 2^24");
  if (max_kv > kMaxKeys) return fail(WAL_ERR_UNSUPPORTED, "at most 2^30 tokens a sequence");
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

// Tiles of 16 keys a step: bf16 takes one, its K and V being twice as wide, and
// fits three CTAs on an SM (25 sequences, 16384 keys: 133 us against 136 with two
// tiles and two CTAs); codes take two and fit two CTAs (int8, 32768 keys: 181 us,
// 189 squeezed into three, 203 with one tile).
template <int D, int TYPE>
void launch_decode(const AttnParams& p, const dim3& grid, cudaStream_t s) {
  constexpr int MT = TYPE == WAL_KV_BF16 ? 1 : 2;
  if (p.max_q * p.group <= 8)
    attn_decode_kernel<D, TYPE, 1, MT><<<grid, 32 * kDecWarps, 0, s>>>(p);
  else
    attn_decode_kernel<D, TYPE, 2, MT><<<grid, 32 * kDecWarps, 0, s>>>(p);
}

int launch_combine(const AttnParams& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  const bool shared = p.n_split > 6;
  const int rows = shared ? 1 : kRowWarps;  // of a CTA
  cfg.gridDim = dim3((unsigned)(((int64_t)p.max_q * p.n_heads + rows - 1) / rows), 1, (unsigned)p.B);
  cfg.blockDim = dim3(32 * kRowWarps);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e;
  if (p.head_dim == 64)
    e = shared ? cudaLaunchKernelEx(&cfg, attn_combine_kernel<64, 4>, p) : cudaLaunchKernelEx(&cfg, attn_combine_kernel<64, 1>, p);
  else
    e = shared ? cudaLaunchKernelEx(&cfg, attn_combine_kernel<128, 4>, p) : cudaLaunchKernelEx(&cfg, attn_combine_kernel<128, 1>, p);
  return launched(e, "attn_combine_kernel");
}

constexpr int kDecMany = 12, kDecFew = 4;  // decode pieces an SM
constexpr int kDecRowBytes = 128 << 10;  // K and V of a piece for each of its query rows, with more than kDecFew
constexpr int kPlanSms = 148;  // SMs the splits are planned for: a constant, so that a workspace size holds on any device

// How the keys are split.
// Decode: a CTA holds a third to a half of an SM.  Four pieces an SM keep it busy
// and cost the least beside the keys themselves (Q, the warps' join, the partial
// results of each query row); ragged lengths even out with up to twelve, which is
// worth it while a piece has 128 KB of K and V for each of its rows.  Measured with
// four an SM, this rule and twelve: 25 ragged sequences of up to 32768 int8 keys,
// 8 heads for 32, 220, 179 and 179 us; 4 equal ones 67, 67 and 79.  With 1 MB in the
// place of 128 KB a row, this rule: 25 of up to 16384 keys 116 and 100 us, 16 heads
// of 64 each with 4 tokens over up to 8192 keys 93 and 71; the one that lost, 2 equal
// bf16 sequences of 100000 keys, 138 and 154.
// Tensor-core kernel: the split with the least estimated time, in steps of 128
// keys (about 1.8 us).  A piece costs three steps more than it has; pieces that
// more than fill the SMs leave about 1.2 pieces' time unused at the end, the
// more so as only bounds of the lengths are known here; a split writes and
// reads fp32 partial results at about 5.7 TB/s, and adds a launch.  Measured,
// without and with the split it takes: two sequences of up to 1024 tokens over
// up to 16384 keys 223 and 125 us (109 with three instead of two); 2 x 2048 over
// 4096 (none) 189, with three 333.  All of these are bf16 pages and heads of 128:
// 8-bit pages, whose steps are longer, and heads of 64 are planned by the same
// numbers.
void plan_split(const wal_kv_cache& c, int n_heads, int T, int B, int max_q, int max_kv, int* n_split, int* split_keys) {
  *n_split = 1;
  *split_keys = max_kv;
  if (T == 0) return;
  const int group = n_heads / c.n_heads;
  const int64_t rows = (int64_t)std::max(1, std::min(max_q, T)) * group;
  const bool tc = rows > kDecMaxRows;
  int64_t pieces = (int64_t)B * c.n_heads;  // without a split: one a (sequence, K/V head), or
  if (tc)                                   // as many row tiles as T rows of B sequences can have
    pieces = c.n_heads * std::min<int64_t>(B * ((rows + kTcAttnRows - 1) / kTcAttnRows), (int64_t)T * group / kTcAttnRows + B);
  const int64_t tiles = ((int64_t)max_kv + 127) / 128;
  int64_t best = 1;
  if (tc) {
    double best_cost = 0;
    for (int64_t s = 1; s <= 128 && s <= (tiles + 1) / 2; ++s) {
      const double r = (double)(pieces * s) / kPlanSms, steps = (double)((tiles + s - 1) / s) + 3;
      double cost = (r <= 1 ? 1 : r + 1.2) * steps;
      if (s > 1) cost += 3 + (double)T * n_heads * c.head_dim * 4 * s * 2 / (5.7e6 * 1.8);
      if (s == 1 || cost < best_cost) {
        best = s;
        best_cost = cost;
      }
    }
  } else {
    const int key_bytes = 2 * c.head_dim * (c.type == WAL_KV_BF16 ? 2 : 1);
    auto even = [&](int n) { return (max_kv * pieces + n * kPlanSms - 1) / (n * kPlanSms); };
    const int64_t keys = std::max(even(kDecMany), std::min<int64_t>(even(kDecFew), rows * kDecRowBytes / key_bytes));
    best = std::max<int64_t>(1, tiles / std::max<int64_t>(1, (keys + 127) / 128));
  }
  const int64_t keys = (tiles + best - 1) / best * 128;
  *split_keys = (int)std::min<int64_t>(keys, 0x7FFFFF80);
  *n_split = (int)((max_kv + keys - 1) / keys);
}

// Set by wal_debug_wait_polls: the limit of the device waits of later calls; below 0, the usual one.
std::atomic<int> g_wait_polls{-1};

int launch_attn(AttnParams& p, cudaStream_t stream) {
  const int polls = g_wait_polls.load();
  p.polls = polls < 0 ? (int)ptx::kSpinLimit : polls;
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

extern "C" int wal_debug_wait_polls(int polls) { return g_wait_polls.exchange(polls < 0 ? -1 : polls); }

extern "C" size_t wal_attn_paged_workspace_bytes(const wal_kv_cache* cache, int n_heads, int T, int B, int max_q,
                                                 int max_kv) {
  if (check_cache(cache) != WAL_OK) return 0;
  if (check_attn(n_heads, cache->n_heads, cache->head_dim, T, B, max_q, max_kv, 1.f) != WAL_OK) return 0;
  int n_split, split_keys;
  plan_split(*cache, n_heads, T, B, max_q, max_kv, &n_split, &split_keys);
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
  plan_split(*cache, n_heads, T, B, max_q, max_kv, &p.n_split, &p.split_keys);
  if ((ws || p.n_split > 1) && (!ws || ws_bytes < attn_ws_bytes(p.n_split, T, n_heads, cache->head_dim)))
    return fail(WAL_ERR_WORKSPACE, "workspace too small");
  if ((st = current_device(&dev))) return st;
  p.clear = p.n_split > 1;
  p.status = status_word(ws);
  if (T > 0 && O == Q) return fail(WAL_ERR_ARG, "O must not be Q: rows are read again after others are written");
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
  int st = check_attn(n_heads, n_kv_heads, head_dim, T, B, max_len, std::max(1, std::min(max_len, T)), scale);
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
  if (O == Q || O == K || O == V) return fail(WAL_ERR_ARG, "O must not be Q, K or V: their rows are read after others are written");
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
