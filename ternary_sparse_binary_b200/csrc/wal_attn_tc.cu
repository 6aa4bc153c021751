// Attention of many query rows: tcgen05, over packed prompts or the paged cache.
//
// A CTA owns 256 query rows of one K/V head (rows are (token, head of the
// group), token-major, so the heads that share K and V share its tiles) as two
// tiles of 128, and walks the keys in tiles of 128:
//   S_t = Q_t K^T          128 x 128, K-major operands from shared memory
//   P_t = 2^(S_t - m)      in registers, one row a thread, back to tensor
//                          memory as bf16 over S_t's first half
//   O_t += P_t V           A from tensor memory, V as it lies (MN-major)
// While one tile's softmax runs on the CUDA cores, the tensor core works on the
// other's products.  384 threads:
//   warps 0-3, 4-7   softmax, rescaling and output of tile 0 and 1
//   warp 8           issues the MMAs (lane 0)
//   warp 9           bf16 K/V: TMA boxes of whole pages (or packed rows) into a
//                    ring of K and V tiles in the 128-byte swizzle
//   warps 9-11       8-bit K/V: plain loads, codes widened to bf16 (exact) and
//                    stored in the same layout; the key's scales go through a
//                    small ring of their own and meet S and P in fp32
// The MMAs of one thread run in order, so S_t of the next keys may overwrite
// P_t once P_t V has been issued, and a softmax that sees its S_t finished knows
// that its O_t is too.
//
// The maximum is lazy: m follows the row's running maximum only when that has
// grown by more than 2^8, since weights up to 2^8 and sums of them keep their
// relative precision in bf16 and fp32; O is then rescaled in tensor memory,
// which after the first tiles hardly ever happens.  Weights are rounded to bf16
// for the second product (2^-8 of a weight, averaged over the keys), scores, m,
// l and O are fp32.
//
// Keys past a row's limit get the score -inf.  V rows past the last key of the
// CTA are zeroed, since 0 * NaN would spread what lies there; a key that only
// some rows see may still do that to the others, and such a row, NaN at the
// end, is done again from its own keys (attend_row).
//
// All waits are bounded; one that gives up records WAL_ERR_TIMEOUT, and its
// role stops, waits for its copies or MMAs in flight and leaves.
#include "wal_attn.h"
#include "wal_ptx.cuh"

#include <cuda.h>

#include <mutex>

namespace wal {

using namespace ptx;

namespace {

constexpr int kThreads = 384;
constexpr int kTile = 128;      // query rows of a tile, keys of a step
constexpr int kConv = 96;       // converter threads of an 8-bit cache
constexpr int kScaleRing = 4;
constexpr float kLazy = 8.f;    // growth of the maximum, in log2, that O is rescaled for

template <int D, int TYPE>
struct Cfg {
  static constexpr uint32_t tile_bytes = kTile * D * 2;
  static constexpr int slots = D == 64 ? 8 : TYPE == WAL_KV_BF16 ? 5 : 4;
  static constexpr uint32_t scale_off = (2 + slots) * tile_bytes;
  static constexpr uint32_t bar_off = scale_off + (TYPE == WAL_KV_BF16 ? 0 : kScaleRing * 2 * kTile * 4);
  static constexpr uint32_t smem = bar_off + 512 + 1024;  // barriers, slack for the alignment
};

// Instruction descriptor: A and B bf16, D fp32, M x N; B MN-major if asked.
__device__ __forceinline__ constexpr uint32_t idesc_bf16(uint32_t M, uint32_t N, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((b_mn ? 1u : 0u) << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
}
// MN-major operand in the 128-byte swizzle: rows of 64 elements along MN, one
// row per k, groups of eight rows 1024 bytes apart, the next 64 elements along
// MN `mn_stride` bytes on.
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr, uint32_t mn_stride) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(mn_stride >> 4) << 16) | ((uint64_t)(1024u >> 4) << 32) |
         ((uint64_t)1u << 46) | ((uint64_t)2u << 61);
}
// D[tmem] (+)= A[tmem] * B[smem]^T
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t* u = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
        "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]), "=r"(u[16]),
        "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]),
        "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float* v) {
  const uint32_t* u = reinterpret_cast<const uint32_t*>(v);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]),
      "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15]), "r"(u[16]), "r"(u[17]), "r"(u[18]),
      "r"(u[19]), "r"(u[20]), "r"(u[21]), "r"(u[22]), "r"(u[23]), "r"(u[24]), "r"(u[25]), "r"(u[26]), "r"(u[27]),
      "r"(u[28]), "r"(u[29]), "r"(u[30]), "r"(u[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&u)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(taddr),
      "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]),
      "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
      " fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n add.rn.f32x2 d, a, b;\n"
      " mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mul.rn.f32x2 d, a, b;\n"
      " mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

struct Bars {
  uint32_t base;
  __device__ uint32_t full(int s) const { return base + 8u * s; }
  __device__ uint32_t empty(int s) const { return base + 64u + 8u * s; }
  __device__ uint32_t q_full(int t) const { return base + 128u + 8u * t; }
  __device__ uint32_t s_full(int t) const { return base + 144u + 8u * t; }
  __device__ uint32_t p_full(int t) const { return base + 160u + 8u * t; }
  __device__ uint32_t o_done(int t) const { return base + 176u + 8u * t; }
  __device__ uint32_t sc_full(int i) const { return base + 192u + 8u * i; }
  __device__ uint32_t sc_empty(int i) const { return base + 224u + 8u * i; }
  __device__ uint32_t v_tail() const { return base + 256u; }
  __device__ uint32_t drained() const { return base + 264u; }
  __device__ uint32_t tmem_slot() const { return base + 272u; }
};

// What a CTA works on.
struct Work {
  int b, h, split;
  int r0, rows;      // query rows [r0, r0 + rows) of the sequence's head
  int k0, k1, n;     // keys [k0, k1), n tiles
  int n_t[2];        // key tiles that query tile 0, 1 takes
};

// ---------------------------------------------------------------------------
// bf16 K/V tiles by TMA (one warp)
// ---------------------------------------------------------------------------
template <int D>
__device__ __forceinline__ void load_tiles_tma(const AttnParams& p, const AttnSeq& s, const Work& w, const CUtensorMap* km,
                                               const CUtensorMap* vm, uint32_t ring, const Bars& bars) {
  using C = Cfg<D, WAL_KV_BF16>;
  const int lane = threadIdx.x & 31;
  int item = 0;
  bool ok = true, tail = false;
  for (int j = 0; j < w.n && ok; ++j) {
    const int kb = w.k0 + kTile * j, cnt = min(kTile, w.k1 - kb);
    // this tile's boxes: lane i's page (paged) or the packed rows
    int boxes = 1, box_rows = kTile, page = 0;
    if (p.table) {
      box_rows = min(kTile, 1 << p.shift);
      boxes = (cnt + box_rows - 1) / box_rows;
      if (lane < boxes) {
        page = __ldg(p.table + w.b * p.ld_table + ((kb + lane * box_rows) >> p.shift));
        if ((uint32_t)page >= (uint32_t)p.n_pages) {
          atomicExch(p.status, (int32_t)WAL_ERR_ARG);
          page = 0;
        }
      }
    }
    for (int kv = 0; kv < 2; ++kv, ++item) {
      const int slot = item % C::slots;
      if (item >= C::slots) ok = mbar_wait(bars.empty(slot), ((item / C::slots) & 1) ^ 1, p.status);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tail = kv == 1 && cnt < kTile;
      const uint32_t dst = ring + (uint32_t)slot * C::tile_bytes, bar = tail ? bars.v_tail() : bars.full(slot);
      if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(boxes * box_rows) * D * 2);
      __syncwarp();
      const int x0 = p.table ? 0 : w.h * D, z0 = p.table ? w.h : 0;
      const int y0 = p.table ? kb & ((1 << p.shift) - 1) : s.q0 + kb;
      for (int i = 0; i < boxes; ++i) {
        const int pg = __shfl_sync(0xffffffffu, page, i);
        if (lane == 0)
#pragma unroll
          for (int a = 0; a < D / 64; ++a)
            tma_4d(dst + a * 16384u + (uint32_t)(i * box_rows) * 128u, kv ? vm : km, x0 + 64 * a, y0, z0, pg, bar);
      }
      if (tail) {  // the last V tile: zero the rows that hold no key of this CTA
        ok = __all_sync(0xffffffffu, mbar_wait(bar, 0, p.status));
        if (!ok) break;
        for (int i = lane; i < (kTile - cnt) * (D / 8); i += 32) {
          const int r = cnt + i / (D / 8), ch = i % (D / 8);
          sts128(dst + (ch >> 3) * 16384u + sw128(r, ch & 7), make_uint4(0, 0, 0, 0));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars.full(slot));
      }
    }
  }
  // nothing of this warp's stays in flight, whatever the MMA thread waited for
  if (!ok && tail) mbar_drain(bars.v_tail(), 0, p.status);
  for (int i = max(0, item - C::slots); i < item; ++i)
    mbar_drain(bars.full(i % C::slots), (i / C::slots) & 1, p.status);
}

// ---------------------------------------------------------------------------
// 8-bit K/V tiles through registers (three warps)
// ---------------------------------------------------------------------------
template <int D, int TYPE>
__device__ __forceinline__ void load_tiles_codes(const AttnParams& p, const Work& w, float sl, uint32_t ring, float* scales,
                                                 const Bars& bars) {
  using C = Cfg<D, TYPE>;
  constexpr int kPer = D / 16;                                // 16-code pieces of a row
  constexpr int kN = (kTile * kPer + kConv - 1) / kConv;      // pieces of a thread
  const int tid = threadIdx.x - (kThreads - kConv);
  const int items = 2 * w.n;
  uint4 cur[kN];
  auto fetch = [&](int item, uint4(&d)[kN]) {
    const int kb = w.k0 + kTile * (item >> 1), cnt = min(kTile, w.k1 - kb);
    const uint8_t* src = static_cast<const uint8_t*>((item & 1) ? p.v : p.k);
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int e = tid + kConv * i, key = e / kPer, part = e % kPer;
      d[i] = make_uint4(0, 0, 0, 0);
      if (e < kTile * kPer && key < cnt)
        d[i] = __ldg(reinterpret_cast<const uint4*>(src + attn_page_row(p, w.b, w.h, kb + key) * D) + part);
    }
  };
  if (items) fetch(0, cur);
  bool ok = true;
  for (int item = 0; item < items; ++item) {
    uint4 nxt[kN];
    if (item + 1 < items) fetch(item + 1, nxt);
    const int j = item >> 1, slot = item % C::slots;
    if (!(item & 1)) {  // the scales of this tile's keys
      const int kb = w.k0 + kTile * j;
      float* sc = scales + (j % kScaleRing) * 2 * kTile;
      if (j >= kScaleRing) ok = mbar_wait(bars.sc_empty(j % kScaleRing), ((j / kScaleRing) & 1) ^ 1, p.status);
      if (!ok) break;
      for (int i = tid; i < 2 * kTile; i += kConv) {
        const int key = kb + (i & (kTile - 1));
        float v = 0.f;
        if (key < w.k1) {
          const int64_t row = attn_page_row(p, w.b, w.h, key);
          v = i < kTile ? __ldg(p.ks + row) * sl : __ldg(p.vs + row);
        }
        sc[i] = v;
      }
      mbar_arrive(bars.sc_full(j % kScaleRing));
    }
    if (item >= C::slots) ok = mbar_wait(bars.empty(slot), ((item / C::slots) & 1) ^ 1, p.status);
    if (!ok) break;
    const uint32_t dst = ring + (uint32_t)slot * C::tile_bytes;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int e = tid + kConv * i, key = e / kPer, part = e % kPer;
      if (e < kTile * kPer) {
        const uint32_t a = dst + (part >> 2) * 16384u;
        uint4 x, y;
        dev::codes4_to_bf16<TYPE>(cur[i].x, x.x, x.y);
        dev::codes4_to_bf16<TYPE>(cur[i].y, x.z, x.w);
        dev::codes4_to_bf16<TYPE>(cur[i].z, y.x, y.y);
        dev::codes4_to_bf16<TYPE>(cur[i].w, y.z, y.w);
        sts128(a + sw128(key, 2 * (part & 3)), x);
        sts128(a + sw128(key, 2 * (part & 3) + 1), y);
      }
    }
    fence_proxy_async_smem();
    mbar_arrive(bars.full(slot));
#pragma unroll
    for (int i = 0; i < kN; ++i) cur[i] = nxt[i];
  }
}

// ---------------------------------------------------------------------------
// MMA issue (one thread)
// ---------------------------------------------------------------------------
template <int D, int TYPE>
__device__ __forceinline__ void issue_mmas(const AttnParams& p, const Work& w, uint32_t q_smem, uint32_t ring, uint32_t tmem,
                                           const Bars& bars) {
  using C = Cfg<D, TYPE>;
  constexpr uint32_t id_s = idesc_bf16(128, 128, false), id_o = idesc_bf16(128, D, true);
  auto scores = [&](int t, int item) {
    const uint32_t a = q_smem + t * C::tile_bytes, b = ring + (uint32_t)(item % C::slots) * C::tile_bytes;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      const uint32_t off = (k >> 2) * 16384u + (k & 3) * 32u;
      mma_f16(tmem + 128u * t, sdesc_sw128(a + off), sdesc_sw128(b + off), id_s, k > 0);
    }
    mma_commit(bars.s_full(t));
  };
  bool ok = true;
  for (int t = 0; t < 2 && ok; ++t)
    if (w.n_t[t] > 0) ok = mbar_wait(bars.q_full(t), 0, p.status);
  ok = ok && mbar_wait(bars.full(0), 0, p.status);
  if (ok) {
    tc_fence_after();
    for (int t = 0; t < 2; ++t)
      if (w.n_t[t] > 0) scores(t, 0);
    mma_commit(bars.empty(0));
  }
  for (int j = 0; j < w.n && ok; ++j) {
    const int vi = 2 * j + 1, ki = 2 * j + 2;
    ok = mbar_wait(bars.full(vi % C::slots), (vi / C::slots) & 1, p.status);
    if (ok && j + 1 < w.n) ok = mbar_wait(bars.full(ki % C::slots), (ki / C::slots) & 1, p.status);
    for (int t = 0; t < 2 && ok; ++t) {
      if (j >= w.n_t[t]) continue;
      ok = mbar_wait(bars.p_full(t), j & 1, p.status);
      if (!ok) break;
      tc_fence_after();
      const uint32_t b = ring + (uint32_t)(vi % C::slots) * C::tile_bytes;
#pragma unroll
      for (int k = 0; k < kTile / 16; ++k)
        mma_f16_ts(tmem + 256u + (uint32_t)D * t, tmem + 128u * t + 8u * k, sdesc_mn_sw128(b + 2048u * k, 16384u), id_o,
                   j > 0 || k > 0);
      if (j + 1 < w.n_t[t])
        scores(t, ki);
      else
        mma_commit(bars.o_done(t));
    }
    if (!ok) break;
    mma_commit(bars.empty(vi % C::slots));
    if (j + 1 < w.n) mma_commit(bars.empty(ki % C::slots));
  }
  mma_commit(bars.drained());
  mbar_drain(bars.drained(), 0, p.status);
}

// ---------------------------------------------------------------------------
// softmax and output of one query tile (four warps, a row a thread)
// ---------------------------------------------------------------------------
template <int D, int TYPE>
__device__ __forceinline__ void softmax_tile(const AttnParams& p, const AttnSeq& s, const Work& w, int t, float sl,
                                             uint32_t q_smem, const float* scales, uint32_t tmem, const Bars& bars) {
  using C = Cfg<D, TYPE>;
  const int tid = threadIdx.x & 127, warp = tid >> 5;
  const int n = w.n_t[t], rows_all = s.n_q * p.group;

  // Q into shared memory.  A negative scale is a sign on Q, a scale of zero
  // makes it zero: the scores below are then multiplied by sl > 0.
  {
    const uint32_t keep = p.scale_log2 == 0.f ? 0u : ~0u, flip = p.scale_log2 < 0.f ? 0x80008000u : 0u;
    const uint32_t dst = q_smem + t * C::tile_bytes;
    for (int i = tid; i < kTile * (D / 8); i += 128) {
      const int r = i / (D / 8), ch = i % (D / 8), row = w.r0 + kTile * t + r;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (row < rows_all) {
        const int tok = row / p.group, head = w.h * p.group + row - tok * p.group;
        v = __ldg(reinterpret_cast<const uint4*>(p.Q + (s.q0 + tok) * p.ldq + head * D) + ch);
        v = make_uint4((v.x & keep) ^ flip, (v.y & keep) ^ flip, (v.z & keep) ^ flip, (v.w & keep) ^ flip);
      }
      sts128(dst + (ch >> 3) * 16384u + sw128(r, ch & 7), v);
    }
    fence_proxy_async_smem();
    mbar_arrive(bars.q_full(t));
  }

  const int row = w.r0 + kTile * t + tid;
  const bool live = row < rows_all;
  const int tok = live ? row / p.group : 0, head = w.h * p.group + (live ? row - tok * p.group : 0);
  const int lim = live ? min(w.k1, attn_limit(s, tok)) : w.k1;
  const int lim0 = __shfl_sync(0xffffffffu, lim, 0);  // the warp's smallest: limits grow with the row
  const uint32_t lanes = (uint32_t)(32 * warp) << 16;
  const uint32_t t_s = tmem + 128u * t + lanes, t_o = tmem + 256u + (uint32_t)D * t + lanes;
  float m = -INFINITY, l = 0.f;
  bool ok = true;
  for (int j = 0; j < n; ++j) {
    const int kb = w.k0 + kTile * j;
    const float* sc = scales + (j % kScaleRing) * 2 * kTile;
    ok = mbar_wait(bars.s_full(t), j & 1, p.status);
    if (TYPE != WAL_KV_BF16) ok = ok && mbar_wait(bars.sc_full(j % kScaleRing), (j / kScaleRing) & 1, p.status);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) break;
    tc_fence_after();
    float x[kTile];
#pragma unroll
    for (int i = 0; i < 4; ++i) tmem_ld32(t_s + 32u * i, x + 32 * i);
    tmem_ld_wait();
    if (TYPE != WAL_KV_BF16) {
#pragma unroll
      for (int i = 0; i < kTile; i += 2) {
        const float2 y = mul2(make_float2(x[i], x[i + 1]), *reinterpret_cast<const float2*>(sc + i));
        x[i] = y.x;
        x[i + 1] = y.y;
      }
    }
    if (kb + kTile > lim0) {
      const int c = lim - kb;
#pragma unroll
      for (int i = 0; i < kTile; ++i) x[i] = i < c ? x[i] : -INFINITY;
    }
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < kTile; i += 4) mx = fmaxf(mx, fmaxf(fmaxf(x[i], x[i + 1]), fmaxf(x[i + 2], x[i + 3])));
    if (TYPE == WAL_KV_BF16) mx *= sl;
    const bool grow = mx > m + kLazy || (m == -INFINITY && mx > m);
    if (__any_sync(0xffffffffu, grow)) {
      const float mn = grow ? mx : m;
      const float f = grow ? ex2(m - mn) : 1.f;  // 0 for a row that had no key yet
      m = mn;
      l *= f;
      if (j > 0) {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          float o[32];
          tmem_ld32(t_o + 32u * i, o);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] *= f;
          tmem_st32(t_o + 32u * i, o);
        }
      }
    }
    const float ref = m == -INFINITY ? 0.f : -m;
    const float2 ref2 = make_float2(ref, ref), sl2 = TYPE == WAL_KV_BF16 ? make_float2(sl, sl) : make_float2(1.f, 1.f);
    float2 sum = make_float2(0.f, 0.f), sum_b = sum;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t pk[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const int e = 32 * i + 2 * k;
        float2 y = make_float2(x[e], x[e + 1]);
        y = TYPE == WAL_KV_BF16 ? fma2(y, sl2, ref2) : add2(y, ref2);
        y.x = ex2(y.x);
        y.y = ex2(y.y);
        if (k & 1) sum_b = add2(sum_b, y); else sum = add2(sum, y);
        if (TYPE != WAL_KV_BF16) y = mul2(y, *reinterpret_cast<const float2*>(sc + kTile + e));
        pk[k] = dev::float2_to_bf16x2(y.x, y.y);
      }
      tmem_st16(t_s + 16u * i, pk);
    }
    sum = add2(sum, sum_b);
    l += sum.x + sum.y;
    tmem_st_wait();
    tc_fence_before();
    mbar_arrive(bars.p_full(t));
    if (TYPE != WAL_KV_BF16) mbar_arrive(bars.sc_empty(j % kScaleRing));
  }

  // output: the row's sums, or its share of them
  if (n > 0) ok = __all_sync(0xffffffffu, ok && mbar_wait(bars.o_done(t), 0, p.status));
  if (!ok) return;
  tc_fence_after();
  const bool partial = p.n_split > 1;
  const float inv = lim == 0 ? 0.f : 1.f / l;
  bool nan = false;
  const int64_t pr = (int64_t)w.split * p.T * p.n_heads + attn_part_row(p, s, tok, head);
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    float o[32];
    if (n > 0) {
      tmem_ld32(t_o + 32u * i, o);
      tmem_ld_wait();
    } else {
#pragma unroll
      for (int k = 0; k < 32; ++k) o[k] = 0.f;
    }
    if (live && partial) {
      float4* dst = reinterpret_cast<float4*>(p.part_o + pr * D + 32 * i);
#pragma unroll
      for (int k = 0; k < 8; ++k) dst[k] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
    } else if (live) {
      uint32_t u[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const float a = lim == 0 ? 0.f : o[2 * k] * inv, b = lim == 0 ? 0.f : o[2 * k + 1] * inv;
        nan |= a != a || b != b;
        u[k] = dev::float2_to_bf16x2(a, b);
      }
      uint4* dst = reinterpret_cast<uint4*>(p.O + (s.q0 + tok) * p.ldo + head * D + 32 * i);
#pragma unroll
      for (int k = 0; k < 4; ++k) dst[k] = make_uint4(u[4 * k], u[4 * k + 1], u[4 * k + 2], u[4 * k + 3]);
    }
    __syncwarp();
  }
  if (partial) {
    if (live) p.part_ml[pr] = make_float2(m, l);
    return;
  }
  // a key that the row does not see may have made it NaN
  uint32_t again = __ballot_sync(0xffffffffu, live && nan && lim < w.k1);
  while (again) {
    const int src = __ffs(again) - 1;
    again &= again - 1;
    attend_row<D>(p, s, w.b, __shfl_sync(0xffffffffu, head, src), __shfl_sync(0xffffffffu, tok, src));
  }
}

template <int D, int TYPE>
__global__ void __launch_bounds__(kThreads, 1)
attn_tc_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap km, const __grid_constant__ CUtensorMap vm) {
  using C = Cfg<D, TYPE>;
  extern __shared__ uint8_t smem_raw[];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  Work w;
  w.b = blockIdx.z;
  w.h = blockIdx.y;
  w.split = blockIdx.x % p.n_split;
  const int tile = (int)(gridDim.x / p.n_split) - 1 - (int)(blockIdx.x / p.n_split);  // longest rows of keys first
  const AttnSeq s = attn_seq(p, w.b);
  if (s.bad) {
    if (blockIdx.x == 0 && w.h == 0 && threadIdx.x == 0) atomicExch(p.status, (int32_t)WAL_ERR_ARG);
    return;
  }
  const int rows_all = s.n_q * p.group;
  w.r0 = tile * kTcAttnRows;
  w.rows = min(kTcAttnRows, rows_all - w.r0);
  if (w.rows <= 0) return;
  w.k0 = w.split * p.split_keys;
  w.k1 = min(min(s.len, attn_limit(s, (w.r0 + w.rows - 1) / p.group)), w.k0 + p.split_keys);
  w.n = w.k1 > w.k0 ? (w.k1 - w.k0 + kTile - 1) / kTile : 0;
  if (w.n == 0) {  // none of the rows sees a key of this split
    for (int i = threadIdx.x; i < w.rows * (D / 8); i += kThreads) {
      const int row = w.r0 + i / (D / 8), ch = i % (D / 8), tok = row / p.group, head = w.h * p.group + row - tok * p.group;
      if (p.n_split > 1) {
        if (ch == 0)
          p.part_ml[(int64_t)w.split * p.T * p.n_heads + attn_part_row(p, s, tok, head)] = make_float2(-INFINITY, 0.f);
      } else {
        reinterpret_cast<uint4*>(p.O + (s.q0 + tok) * p.ldo + head * D)[ch] = make_uint4(0, 0, 0, 0);
      }
    }
    return;
  }
  w.n_t[1] = w.rows > kTile ? w.n : 0;
  w.n_t[0] = w.n;
  if (TYPE == WAL_KV_BF16 && w.rows > kTile) {  // the first tile's rows may see fewer keys
    const int end = min(w.k1, attn_limit(s, (w.r0 + kTile - 1) / p.group));
    w.n_t[0] = end > w.k0 ? (end - w.k0 + kTile - 1) / kTile : 0;
  }

  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  float* scales = reinterpret_cast<float*>(smem_raw + (base - smem_u32(smem_raw)) + C::scale_off);
  const uint32_t ring = base + 2 * C::tile_bytes;
  const Bars bars = {base + C::bar_off};
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::slots; ++i) {
      mbar_init(bars.full(i), TYPE == WAL_KV_BF16 ? 1 : kConv);
      mbar_init(bars.empty(i), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(bars.q_full(t), 128);
      mbar_init(bars.s_full(t), 1);
      mbar_init(bars.p_full(t), 128);
      mbar_init(bars.o_done(t), 1);
    }
    for (int i = 0; i < kScaleRing; ++i) {
      mbar_init(bars.sc_full(i), kConv);
      mbar_init(bars.sc_empty(i), w.rows > kTile ? 256 : 128);
    }
    mbar_init(bars.v_tail(), 1);
    mbar_init(bars.drained(), 1);
    mbar_init_fence();
  }
  if (warp == 8) {
    tmem_alloc(bars.tmem_slot(), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = lds32(bars.tmem_slot());
  const float sl = p.scale_log2 == 0.f ? 1.f : fabsf(p.scale_log2);

  if (warp < 8) {
    if (warp < 4 || w.rows > kTile) softmax_tile<D, TYPE>(p, s, w, warp >> 2, sl, base, scales, tmem, bars);
  } else if (warp == 8) {
    if ((threadIdx.x & 31) == 0) issue_mmas<D, TYPE>(p, w, base, ring, tmem, bars);
    __syncwarp();
  } else if (TYPE == WAL_KV_BF16) {
    if (warp == 9) load_tiles_tma<D>(p, s, w, &km, &vm, ring, bars);
  } else {
    load_tiles_codes<D, TYPE>(p, w, sl, ring, scales, bars);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static EncodeFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult res = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &res) == cudaSuccess &&
        res == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeFn>(f);
  });
  return fn;
}

// K or V as (column, row, head, page): boxes of 64 columns and up to 128 rows.
int make_map(CUtensorMap* map, const AttnParams& p, const void* base, int64_t ld) {
  const EncodeFn enc = encode_fn();
  if (!enc) return fail(WAL_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
  const cuuint64_t D = (cuuint64_t)p.head_dim, H = (cuuint64_t)p.n_kv_heads;
  cuuint64_t dims[4] = {H * D, (cuuint64_t)p.T, 1, 1};  // packed rows: the head is part of the column
  cuuint64_t strides[3] = {(cuuint64_t)ld * 2, (cuuint64_t)ld * 2, (cuuint64_t)ld * 2};
  cuuint32_t box[4] = {64, kTile, 1, 1}, step[4] = {1, 1, 1, 1};
  if (p.table) {
    const cuuint64_t page = (cuuint64_t)1 << p.shift;
    dims[0] = D;
    dims[1] = page;
    dims[2] = H;
    dims[3] = (cuuint64_t)p.n_pages;
    strides[0] = D * 2;
    strides[1] = page * D * 2;
    strides[2] = H * page * D * 2;
    if (page < kTile) box[1] = (cuuint32_t)page;
  }
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, step,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(WAL_ERR_CUDA, "cuTensorMapEncodeTiled failed with " + std::to_string((int)r));
  return WAL_OK;
}

template <int D, int TYPE>
int launch_one(const AttnParams& p, const CUtensorMap& km, const CUtensorMap& vm, cudaStream_t stream) {
  // the attribute is per device; setting it again is cheap and needs no state
  cudaError_t e = cudaFuncSetAttribute(attn_tc_kernel<D, TYPE>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg<D, TYPE>::smem);
  if (e == cudaSuccess) {
    const int64_t tiles = ((int64_t)p.max_q * p.group + kTcAttnRows - 1) / kTcAttnRows;
    const dim3 grid((unsigned)(tiles * p.n_split), (unsigned)p.n_kv_heads, (unsigned)p.B);
    attn_tc_kernel<D, TYPE><<<grid, kThreads, Cfg<D, TYPE>::smem, stream>>>(p, km, vm);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return fail(WAL_ERR_CUDA, std::string("attn_tc_kernel launch: ") + cudaGetErrorString(e));
  return WAL_OK;
}

}  // namespace

int launch_attn_tc(const AttnParams& p, cudaStream_t stream) {
  CUtensorMap km = {}, vm = {};
  const bool wide = p.head_dim == 128;
  if (p.type == WAL_KV_BF16) {
    int st = make_map(&km, p, p.k, p.ldk);
    if (st || (st = make_map(&vm, p, p.v, p.ldv))) return st;
    return wide ? launch_one<128, WAL_KV_BF16>(p, km, vm, stream) : launch_one<64, WAL_KV_BF16>(p, km, vm, stream);
  }
  if (p.type == WAL_KV_INT8)
    return wide ? launch_one<128, WAL_KV_INT8>(p, km, vm, stream) : launch_one<64, WAL_KV_INT8>(p, km, vm, stream);
  return wide ? launch_one<128, WAL_KV_E4M3>(p, km, vm, stream) : launch_one<64, WAL_KV_E4M3>(p, km, vm, stream);
}

}  // namespace wal
