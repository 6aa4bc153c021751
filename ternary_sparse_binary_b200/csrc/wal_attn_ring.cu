// Attention of few query rows where they do not see every key of their sequence: a
// window with first keys that stay visible, a shared prefix, what is behind it.
//
// Products, types and running statistics are those of the single-token kernel
// (wal_attn.cu): keys are the M side of both products, S^T = K Q^T and O^T += V^T P^T.
// Keys come to the warps another way: each warp has a ring in shared memory that its
// own asynchronous copies fill, kStages steps of 16 * MT keys ahead, so that an SM has
// many times the bytes in flight that fit in registers, and no two warps wait for one
// another.  Keys that no row sees are not read; their places hold zeros.
//
// Bound by bytes over bf16 (25 slots, window of 4096, 32 q heads of 128 on 8, up to 16384
// keys: 58.5 us, 0.95 of the copy rate) and by latency over codes (int8: 44.6 us, 0.73):
// registers allow 12 warps an SM, whose steps of 32 keys take 2 us of conversions,
// products and exponentials that wait for one another.  Steps of 16 keys and four CTAs an
// SM were slower (47.3 us), two chains of products a tile the same (45.2).
//
// Rows of the ring are swizzled so that the fragments' loads, eight lanes or sixteen at
// a time, fall into different banks.  Rows of 128 bytes or more: the 16-byte chunk's
// low bits XOR the row's; a fragment's rows g and g + 1 are four keys apart (row g of a
// tile stands for key fold(g)), so that the eight lanes that read K in one go, four
// neighbouring chunks of two rows, have eight different ones, as have those that read V,
// one chunk of four key pairs and its neighbour's.  Rows of 64 bytes: two lie in a line,
// and a line's chunks XOR twice its number.
#include "wal_attn_dec.cuh"
#include "wal_ptx.cuh"

namespace wal {

namespace {

using ptx::smem_u32;

template <int D, int TYPE, int NT>
struct RingCfg {
  static constexpr bool codes = TYPE != WAL_KV_BF16;
  static constexpr int row = D * (codes ? 1 : 2);            // bytes of a key
  static constexpr int MT = codes ? 2 : 1;                   // tiles of 16 keys a step
  static constexpr int keys = 16 * MT;
  static constexpr int scales = codes ? 2 * keys * 4 : 0;
  static constexpr int step = 2 * keys * row + scales;       // K, V, their scales
  static constexpr int stages = D == 64 ? 3 : 2;
  static constexpr int ring = stages * step;                 // of a warp
  static constexpr int join = 8 * NT * (D + 4) * 4;          // a warp's sums, over its ring at the end
  static constexpr int warp = ring > join ? ring : join;
  static constexpr int smem = kDecWarps * warp;
  static constexpr int ctas = NT > 1 ? 2 : D == 64 ? 4 : 3;  // of an SM; the split of the keys counts on it
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// Zeros where the source is not there.
__device__ __forceinline__ void copy16_if(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4_if(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(there ? 4 : 0) : "memory");
}

// Place of a 16-byte chunk of a row in a tile of rows of ROW bytes.
template <int ROW>
__device__ __forceinline__ uint32_t place(int row, int chunk) {
  if (ROW == 64) {
    const int line = row >> 1;
    return (uint32_t)(line * 128 + ((((row & 1) << 2 | chunk) ^ ((line << 1) & 7)) << 4));
  }
  return (uint32_t)(row * ROW + ((chunk ^ (row & 7)) << 4));
}
// Key of a tile that row g of its fragments stands for (g < 8; g + 8 likewise).
template <int ROW>
__device__ __forceinline__ int fold(int g) { return ROW == 64 ? g : g ^ ((g & 1) << 2); }

template <int D, int TYPE, int NT>
__device__ __forceinline__ void attn_ring(const AttnParams& p, uint8_t* smem) {
  using C = RingCfg<D, TYPE, NT>;
  constexpr bool CODES = C::codes;
  constexpr int MT = C::MT, ROW = C::row, STEP = C::keys, CH = ROW / 16;
  constexpr int W = D * (CODES ? 1 : 2) / 16;   // 32-bit words of K per lane and key (of 4 lanes)
  constexpr int NW = D * (CODES ? 1 : 2) / 32;  // words of V per lane and key (of 8 lanes)
  constexpr int DT = D / 16;
  __shared__ float2 s_ml[kDecWarps][8 * NT];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int b = blockIdx.z, h = blockIdx.y, split = blockIdx.x;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const AttnSeq s = attn_seq<true, true>(p, b);
  if (p.clear) {
    if (split == 0 && h == 0 && b == 0 && threadIdx.x == 0 && !p.part_first) *p.status = 0;
  } else if (s.bad && h == 0 && threadIdx.x == 0 && p.status) {
    attn_report(p.status);
  }
  if (s.bad) return;
  const int rows = s.n_q * p.group;
  if (rows == 0) return;
  const int first = attn_limit<true>(p, s, 0), last = attn_limit<true>(p, s, s.n_q - 1);
  const AttnSpan span = attn_span(p, s, first, last);
  const int k0 = split * p.split_keys, k1 = min(span.n, k0 + p.split_keys);
  const int whole_from = span.low - span.delta;  // some row sees every place from here on
  if (k0 >= k1 && split > 0) return;  // split 0 also answers for a sequence without keys

  const uint32_t ring = smem_u32(smem) + (uint32_t)warp * C::warp;
  // The cache rows of a step's tiles, each of which lies in one page (with runs of 32
  // keys or more, each pair of them); a step ahead of its copies, which would wait for
  // the table otherwise.
  int64_t base[MT];
  auto find = [&](int j0) {
#pragma unroll
    for (int u = 0; u < MT; ++u)
      if ((u & 1) && p.gran >= 32)
        base[u] = base[u - (u & 1)] + 16;
      else
        base[u] = j0 + 16 * u < k1 ? attn_page_row(p, s.tab, h, attn_key(j0 + 16 * u, p.sinks_pad, span.delta)) : 0;
  };
  // A lane copies the chunk `ch` of rows r0, r0 + kRows, ...; r0 has no bit of kRows' multiples.
  constexpr int kRows = 32 / CH, kCopies = 16 / kRows;
  const int r0 = lane / CH, ch = lane % CH, from = r0 * ROW + 16 * ch;
  auto issue = [&](int j0, int slot) {
    const uint32_t dst = ring + (uint32_t)slot * C::step;
    const bool whole = j0 + STEP <= k1 && j0 >= whole_from;  // some row sees every key of it
    if (j0 < k1) {
#pragma unroll
      for (int u = 0; u < MT; ++u) {
        const int64_t at = base[u] * ROW + from;
        const char *ks = static_cast<const char*>(p.k) + at, *vs = static_cast<const char*>(p.v) + at;
        const uint32_t to = dst + (uint32_t)(16 * u) * ROW;
        if (whole) {
#pragma unroll
          for (int i = 0; i < kCopies; ++i) {
            copy16(to + place<ROW>(r0 | (i * kRows), ch), ks + i * kRows * ROW);
            copy16(to + STEP * ROW + place<ROW>(r0 | (i * kRows), ch), vs + i * kRows * ROW);
          }
        } else {  // zeros for the others, whose slots lie in the same page
          const int v0 = j0 + 16 * u, key0 = attn_key(v0, p.sinks_pad, span.delta);
#pragma unroll
          for (int i = 0; i < kCopies; ++i) {
            const int r = r0 | (i * kRows);
            const bool there = v0 + r < k1 && (key0 + r >= span.low || key0 + r < p.sinks);
            copy16_if(to + place<ROW>(r, ch), ks + i * kRows * ROW, there);
            copy16_if(to + STEP * ROW + place<ROW>(r, ch), vs + i * kRows * ROW, there);
          }
        }
        if (CODES) {  // K's scales, then V's
          const int r = lane & 15, v0 = j0 + 16 * u, key = attn_key(v0, p.sinks_pad, span.delta) + r;
          copy4_if(dst + 2 * STEP * ROW + (uint32_t)((lane >> 4) * STEP + 16 * u + r) * 4, (lane >> 4 ? p.vs : p.ks) + base[u] + r,
                   v0 + r < k1 && (key >= span.low || key < p.sinks));
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  constexpr int kNext = kDecWarps * STEP;
  int j0 = k0 + warp * STEP;
#pragma unroll
  for (int i = 0; i < C::stages; ++i) {
    find(j0 + i * kNext);
    issue(j0 + i * kNext, i);
  }
  find(j0 + C::stages * kNext);

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
      lim[t][e] = r < rows ? attn_limit<true>(p, s, r / p.group) : s.len;
      m[t][e] = m2[t][e] = -INFINITY;
      l[t][e] = 0.f;
    }
  // places that every row sees end at lim_min and, but for the first keys, begin at low_max
  const int lim_min = min(k1, first - span.delta), low_max = attn_low(p, s, last) - span.delta;
  float o[DT][NT][4];
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[d][t][e] = 0.f;

  const int gk = fold<ROW>(g);  // this lane's keys of K: gk and gk + 8 of a tile; of V: kv[e] + {0, 8}
  const int kv[2] = {fold<ROW>(2 * c), fold<ROW>(2 * c + 1)};
  int slot = 0;
#pragma unroll 1
  for (; j0 < k1; j0 += kNext) {
    asm volatile("cp.async.wait_group %0;" ::"n"(C::stages - 1) : "memory");
    __syncwarp();
    const uint32_t kb = ring + (uint32_t)slot * C::step, vb = kb + STEP * ROW, sb = vb + STEP * ROW;
    // S^T = K Q^T
    float sc[MT][NT][4];
#pragma unroll
    for (int u = 0; u < MT; ++u) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[u][t][e] = 0.f;
#pragma unroll
      for (int i = 0; i < W / 4; ++i) {
        const uint4 x = ptx::lds128(kb + (uint32_t)(16 * u) * ROW + place<ROW>(gk, 4 * i + c));
        const uint4 y = ptx::lds128(kb + (uint32_t)(16 * u) * ROW + place<ROW>(gk + 8, 4 * i + c));
        const uint32_t kx[4] = {x.x, x.y, x.z, x.w}, ky[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int d = 0; d < (CODES ? 4 : 2); ++d) {
          uint32_t a[4];
          if (CODES) {
            dev::codes4_to_half<TYPE>(kx[d], a[0], a[2]);
            dev::codes4_to_half<TYPE>(ky[d], a[1], a[3]);
          } else {
            a[0] = kx[(2 * d) & 3]; a[1] = ky[(2 * d) & 3]; a[2] = kx[(2 * d + 1) & 3]; a[3] = ky[(2 * d + 1) & 3];
          }
          const int f = (CODES ? 4 : 2) * i + d;
#pragma unroll
          for (int t = 0; t < NT; ++t) mma16816<CODES>(sc[u][t], a[0], a[1], a[2], a[3], q[t][f][0], q[t][f][1]);
        }
      }
    }
    // scores in log2 units, and (codes) what V's scale adds to them
    float lv[MT][2], vs[MT][2];
#pragma unroll
    for (int u = 0; u < MT; ++u)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint32_t at = sb + (uint32_t)(16 * u + gk + 8 * r) * 4;
        const float ks = CODES ? __uint_as_float(ptx::lds32(at)) : 1.f;
        vs[u][r] = CODES ? __uint_as_float(ptx::lds32(at + STEP * 4)) : 1.f;
        lv[u][r] = CODES ? lg2(fabsf(vs[u][r])) : 0.f;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float2 f = make_float2(mult[t][0], mult[t][1]);
          if (CODES) f = ptx::mul2(f, make_float2(ks, ks));
          const float2 x = ptx::mul2(make_float2(sc[u][t][2 * r], sc[u][t][2 * r + 1]), f);
          sc[u][t][2 * r] = x.x;
          sc[u][t][2 * r + 1] = x.y;
        }
      }
    if (j0 + STEP > lim_min || j0 < low_max) {  // keys a row does not see get -inf
#pragma unroll
      for (int u = 0; u < MT; ++u) {
        const int v0 = j0 + 16 * u + gk, key0 = attn_key(j0 + 16 * u, p.sinks_pad, span.delta) + gk;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = key0 + 8 * (e >> 1), up = lim[t][e & 1];
            if (v0 + 8 * (e >> 1) >= k1 || j >= up || (j < attn_low(p, s, up) && j >= p.sinks)) sc[u][t][e] = -INFINITY;
          }
      }
    }

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
      const uint32_t vt = vb + (uint32_t)(16 * u) * ROW;
#pragma unroll
      for (int i = 0; i < (NW + 3) / 4; ++i) {  // 16 bytes (of rows of 64 bytes: 8) of four keys
        uint32_t v[4][4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = kv[e & 1] + 8 * (e >> 1);
          if (NW >= 4) {
            const uint4 x = ptx::lds128(vt + place<ROW>(r, 8 * i + g));
            v[e][0] = x.x; v[e][1] = x.y; v[e][2] = x.z; v[e][3] = x.w;
          } else {
            const uint2 x = ptx::lds64(vt + place<ROW>(r, g >> 1) + 8 * (g & 1));
            v[e][0] = x.x; v[e][1] = x.y;
          }
        }
#pragma unroll
        for (int k = 0; k < (NW >= 4 ? 4 : 2); ++k) {
          if (!CODES) {  // word k: columns 64 i + 8 g + 2 k + {0, 1}
            const uint32_t a0 = __byte_perm(v[0][k], v[1][k], 0x5410), a1 = __byte_perm(v[0][k], v[1][k], 0x7632);
            const uint32_t a2 = __byte_perm(v[2][k], v[3][k], 0x5410), a3 = __byte_perm(v[2][k], v[3][k], 0x7632);
#pragma unroll
            for (int t = 0; t < NT; ++t) mma16816<CODES>(o[(4 * i + k) % DT][t], a0, a1, a2, a3, pb[t][0], pb[t][1]);
          } else {  // word k: columns (D / 8) g + 4 k + {0 .. 3}
            uint32_t a[2][4];
            dev::codes4_to_half<TYPE>(__byte_perm(v[0][k], v[1][k], 0x5140), a[0][0], a[0][1]);
            dev::codes4_to_half<TYPE>(__byte_perm(v[0][k], v[1][k], 0x7362), a[1][0], a[1][1]);
            dev::codes4_to_half<TYPE>(__byte_perm(v[2][k], v[3][k], 0x5140), a[0][2], a[0][3]);
            dev::codes4_to_half<TYPE>(__byte_perm(v[2][k], v[3][k], 0x7362), a[1][2], a[1][3]);
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
              for (int t = 0; t < NT; ++t) mma16816<CODES>(o[(2 * k + x) % DT][t], a[x][0], a[x][1], a[x][2], a[x][3], pb[t][0], pb[t][1]);
          }
        }
      }
    }
    __syncwarp();
    issue(j0 + C::stages * kNext, slot);  // where this step lay
    find(j0 + (C::stages + 1) * kNext);
    slot = slot + 1 == C::stages ? 0 : slot + 1;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
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

  // join the warps: each leaves its rows where its ring was, then a warp takes a row
  __syncwarp();
  float* mine = reinterpret_cast<float*>(smem + warp * C::warp);
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
      for (int e = 0; e < 4; ++e) mine[(8 * t + 2 * c + (e & 1)) * (D + 4) + col + (e >> 1)] = o[d][t][e];
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
      const float* from = reinterpret_cast<const float*>(smem + w * C::warp) + r * (D + 4) + lane * VPL;
#pragma unroll
      for (int i = 0; i < VPL; ++i) acc[i] += f * from[i];
    }
    const int tok = r / p.group, head = h * p.group + r % p.group;
    if (p.n_split > 1 || p.phase) {
      const int64_t pr = (int64_t)(p.part_first + split) * p.T * p.n_heads + attn_part_row(p, s, tok, head);
      float* dst = p.part_o + pr * D + lane * VPL;
      if (VPL == 4)
        *reinterpret_cast<float4*>(dst) = make_float4(acc[0], acc[1], acc[VPL - 2], acc[VPL - 1]);
      else
        *reinterpret_cast<float2*>(dst) = make_float2(acc[0], acc[1]);
      if (lane == 0) p.part_ml[pr] = make_float2(mm, ll);
    } else {
      finish_row<D, true>(p, s, s.tab, head, tok, acc, ll);
    }
  }
}

template <int D, int TYPE, int NT>
__global__ void __launch_bounds__(32 * kDecWarps, RingCfg<D, TYPE, NT>::ctas) attn_ring_kernel(const __grid_constant__ AttnParams p) {
  extern __shared__ __align__(128) uint8_t ring_smem[];
  attn_ring<D, TYPE, NT>(p, ring_smem);
  // The second launch of a shared call starts beside the first.  Its first CTA waits for
  // that, so that what comes after the second comes after both.
  if (p.phase == kOwn && threadIdx.x < 32 && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) attn_groups_end(p);
}

template <int D, int TYPE, int NT>
cudaError_t launch_one(const AttnParams& p, cudaStream_t stream) {
  using C = RingCfg<D, TYPE, NT>;
  cudaError_t e = cudaFuncSetAttribute(attn_ring_kernel<D, TYPE, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.n_split, (unsigned)p.n_kv_heads, (unsigned)p.B);
  cfg.blockDim = dim3(32 * kDecWarps);
  cfg.dynamicSmemBytes = C::smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  if (p.part_first) {  // beside the prefix's launch
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
  return cudaLaunchKernelEx(&cfg, attn_ring_kernel<D, TYPE, NT>, p);
}
template <int D, int TYPE>
cudaError_t launch_rows(const AttnParams& p, cudaStream_t stream) {
  return p.max_q * p.group <= 8 ? launch_one<D, TYPE, 1>(p, stream) : launch_one<D, TYPE, 2>(p, stream);
}

}  // namespace

int launch_attn_ring(const AttnParams& p, cudaStream_t stream) {
  const bool wide = p.head_dim == 128;
  cudaError_t e;
  switch (p.type) {
    case WAL_KV_BF16: e = wide ? launch_rows<128, WAL_KV_BF16>(p, stream) : launch_rows<64, WAL_KV_BF16>(p, stream); break;
    case WAL_KV_INT8: e = wide ? launch_rows<128, WAL_KV_INT8>(p, stream) : launch_rows<64, WAL_KV_INT8>(p, stream); break;
    default: e = wide ? launch_rows<128, WAL_KV_E4M3>(p, stream) : launch_rows<64, WAL_KV_E4M3>(p, stream); break;
  }
  if (e != cudaSuccess) return fail(WAL_ERR_CUDA, std::string("attn_ring_kernel launch: ") + cudaGetErrorString(e));
  return WAL_OK;
}

}  // namespace wal
