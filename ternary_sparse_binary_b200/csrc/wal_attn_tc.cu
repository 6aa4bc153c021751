// Attention of many query rows: tcgen05, over packed prompts or the paged cache.
//
// A piece of work is 256 query rows of one K/V head (rows are (token, head of
// the group), token-major, so the heads that share K and V share its tiles) as
// two tiles of 128, and a range of keys, in tiles of 128:
//   S_t = Q_t K^T          128 x 128, K-major operands from shared memory
//   P_t = 2^(S_t - m)      in registers, one row a thread, back to tensor
//                          memory as bf16 over S_t's first half
//   O_t += P_t V           A from tensor memory, V as it lies (MN-major)
// While one tile's softmax runs on the CUDA cores, the tensor core works on the
// other's products.  A piece with one tile of rows gives both halves of the CTA
// that tile and every other key tile each.  CTAs are persistent: each role walks
// the CTA's pieces by itself, so the loads and the first products of a piece run
// under the end of the one before.
//   warps 0-3, 4-7   softmax, rescaling and output of half 0 and 1
//   warp 8           issues the MMAs
//   warp 9           K/V by TMA, boxes of whole pages or packed rows: bf16 tiles
//                    into a ring in the 128-byte swizzle, 8-bit codes and their
//                    scales into a ring as they lie
//   warps 10, 11     Q
//   warps 12-15      (8-bit) codes to bf16 tiles, exact; scales go to a ring of
//                    their own and meet S and P in fp32
// The MMAs of one thread run in order, so S_t of the next keys may overwrite
// P_t once P_t V has been issued, and a softmax that sees its S_t finished knows
// that its O_t is too.
//
// Bound by the chain of a step, softmax of one tile beside the products of the other:
// about 3200 cycles where the MMAs take 2048.  A prompt of 8192 tokens, 32 q heads of
// 128 on 8: 429 us, 1280 TFLOP/s of what the mask leaves.  One warp issues all MMAs:
// two of them made the halves fall in step (552 us against 507 then); 16 softmax
// warps, two to a row, were slower too (592).
//
// The maximum is lazy: m follows the row's running maximum only when that has
// grown by more than 2^16, since weights up to 2^16 and sums of them keep their
// relative precision in bf16 and fp32; O is then rescaled in tensor memory,
// which after the first tiles hardly ever happens.  Weights are rounded to bf16
// for the second product (2^-8 of a weight, averaged over the keys), scores, m,
// l and O are fp32.
//
// Keys past a row's limit get the score -inf.  V rows past the last key of the
// CTA are zeroed, since 0 * NaN would spread what lies there; a key that only
// some rows see may still do that to the others, and such a row, NaN at the
// end though its sum of weights is not, is done again from its own keys if a V
// behind its last key is to blame (attn_last_nonfinite, attend_row).
//
// All waits are bounded; one that gives up records WAL_ERR_TIMEOUT, and its
// role stops, waits for its copies or MMAs in flight and leaves.  What the others
// wait for then does not come, so that they give up too, the softmax warps last:
// they make the rows that they have no result for NaN.
#include "wal_attn.h"
#include "wal_ptx.cuh"

#include <cuda.h>

#include <mutex>

namespace wal {

using namespace ptx;

namespace {

constexpr int kTile = 128;      // query rows of a tile, keys of a step
constexpr int kScaleRing = 4;   // key tiles whose scales are held at once
constexpr int kQThreads = 64;   // threads that load Q
constexpr float kLazy = 16.f;   // growth of the maximum, in log2, that O is rescaled for
constexpr int kGrid = 148;      // CTAs of a launch at most; they wait for nobody, so any number is right

// Shared memory and registers.  Launched registers are shared out again by
// setmaxnreg: 384 threads of 168 as 256 x 208 + 128 x 88, 512 threads of 128 as
// 256 x 176 + 256 x 80.
template <int D, int TYPE>
struct Cfg {
  static constexpr bool codes = TYPE != WAL_KV_BF16;
  static constexpr int threads = codes ? 512 : 384;
  static constexpr int soft_regs = codes ? 176 : 208, other_regs = codes ? 80 : 88;
  static constexpr uint32_t tile = kTile * D * 2;                    // a Q, K or V tile in bf16
  static constexpr int slots = D == 64 ? (codes ? 6 : 8) : (codes ? 3 : 5);
  static constexpr uint32_t raw = codes ? kTile * D + kTile * 4 : 0;  // a tile as it lies in the cache, and its scales
  static constexpr int raws = D == 64 ? 6 : 3;
  static constexpr uint32_t ring_off = 2 * tile;
  static constexpr uint32_t raw_off = ring_off + slots * tile;
  static constexpr uint32_t scale_off = raw_off + (codes ? raws * raw : 0);
  static constexpr uint32_t ml_off = scale_off + (codes ? kScaleRing * 2 * kTile * 4 : 0);  // half 1's m and l of each row
  static constexpr uint32_t bar_off = ml_off + kTile * 8;
  static constexpr uint32_t smem = bar_off + 512 + 1024;             // barriers, slack for the alignment
  static_assert(smem <= 232448, "above the shared memory of an SM");
};

// Instruction descriptor: A and B bf16, D fp32, M x N; B MN-major if asked.
__device__ __forceinline__ constexpr uint32_t idesc_bf16(uint32_t M, uint32_t N, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((b_mn ? 1u : 0u) << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
}
// Shared-memory descriptors in the 128-byte swizzle, as two words: the start
// address in 16-byte units (and, for V, the byte offset of the next 64 columns),
// and what all tiles share: groups of eight rows 1024 bytes apart, version 1,
// the swizzle.  Q and K are K-major; V is MN-major: rows of 64 elements along
// the columns, one row per key, the next 64 columns 16 KB on.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t kDescK = 1u << 16, kDescV = (16384u >> 4) << 16;
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t offset_bits) { return ((saddr & 0x3FFFFu) >> 4) | offset_bits; }
// D[tmem] (+)= A[smem] * B[smem]^T, and A[tmem] * B[smem]^T
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.b32 p, %4, 0;\n mov.b64 a, {%1, %5};\n mov.b64 b, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 b;\n setp.ne.b32 p, %4, 0;\n mov.b64 b, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kDescHi)
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
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&u)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(taddr),
      "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]),
      "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// mbar_wait with its loop rolled: the kernel has many waits, and its code must
// stay small (see softmax_rows).
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, const AttnParams& p) {
#pragma unroll 1
  for (int it = 0; it < p.polls; ++it)
    if (mbar_try_wait(bar, parity)) return true;
  if (p.status) atomicExch(p.status, (int32_t)WAL_ERR_TIMEOUT);
  return false;
}
// 32 bytes to a 32-byte aligned address: a whole sector, where two 16-byte
// stores of lanes with rows of their own would send two halves.
__device__ __forceinline__ void stg256(void* dst, const uint32_t* u) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]),
               "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
               : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {  // NaN if one of them is
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
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
  __device__ uint32_t full(int s) const { return base + 8u * s; }               // K/V tile ready for the MMAs
  __device__ uint32_t empty(int s) const { return base + 64u + 8u * s; }
  __device__ uint32_t raw_full(int s) const { return base + 128u + 8u * s; }    // codes ready for the converters
  __device__ uint32_t raw_empty(int s) const { return base + 176u + 8u * s; }
  __device__ uint32_t sc_full(int i) const { return base + 224u + 8u * i; }     // scales ready for the softmax
  __device__ uint32_t sc_empty(int i) const { return base + 256u + 8u * i; }
  __device__ uint32_t q_full(int t) const { return base + 288u + 8u * t; }
  __device__ uint32_t q_empty(int t) const { return base + 304u + 8u * t; }
  __device__ uint32_t s_full(int t) const { return base + 320u + 8u * t; }      // scores in tensor memory
  __device__ uint32_t p_half(int t) const { return base + 416u + 8u * t; }      // weights in tensor memory: the first 64 keys',
  __device__ uint32_t p_full(int t) const { return base + 336u + 8u * t; }      // and the others'
  __device__ uint32_t o_done(int t) const { return base + 352u + 8u * t; }      // the last product of a piece
  __device__ uint32_t join() const { return base + 456u; }                // dual: half 1's sums are there
  __device__ uint32_t o1_free() const { return base + 448u; }                   // dual: and have been joined
  __device__ uint32_t v_tail() const { return base + 384u; }
  __device__ uint32_t drained() const { return base + 392u; }
  __device__ uint32_t tmem_slot() const { return base + 400u; }
};

// A piece.  With more than one tile of rows, query tile t walks n_t[t] key
// tiles.  With one (dual), both halves of the CTA walk its keys, half t the key
// tiles t, t + 2, ..., and their sums are joined at the end.
struct Work {
  int b, h, split;
  int r0, rows;      // query rows [r0, r0 + rows) of the sequence's head
  int k0, k1, n;     // keys [k0, k1), n tiles
  int n0, n1;        // key tiles of half 0 and 1
  bool dual;
  __device__ int n_t(int t) const { return t ? n1 : n0; }
  __device__ bool has_q(int t) const { return t ? n1 > 0 && !dual : n0 > 0; }
  __device__ int tile_of(int t, int k) const { return dual ? 2 * k + t : k; }
};

// The pieces of a launch: (query tile pair, sequence, split of its keys, K/V
// head), without those that have no rows, the tile pairs that see most keys
// first.  The CTAs take one each, then one each in the opposite order, and so
// on, so that they get about the same.  Each role walks its CTA's pieces by
// itself, whole warps at a time: a lane looks at a sequence, and the search for
// a piece goes on where the last one ended.
template <int TYPE>
struct Walk {
  const AttnParams& p;
  int tile, at;            // tile pair, and the next piece's place among those from there on
  int stride, back;        // pieces to the next one, and to the one after that
  AttnSeq mine;            // this lane's sequence, and how many tile pairs and splits it has
  int tiles, splits, held; // (the first lane's sequence)
  int each, same;          // of `tile`: pieces of one head, -1 if not counted yet, and the last pair with the same ones
  int down, b0, before;    // where the search stands: the tile pair, the sequences, the pieces before them
  __device__ __forceinline__ Walk(const AttnParams& p_, int most) : p(p_), tile(most - 1), at(blockIdx.x), held(-1), each(-1) {
    stride = 2 * ((int)gridDim.x - (int)blockIdx.x) - 1;
    back = 2 * (int)blockIdx.x + 1;
  }
  __device__ __forceinline__ void look(int first) {  // at 32 sequences
    if (first == held) return;
    held = first;
    const int b = first + (threadIdx.x & 31);
    tiles = 0;
    splits = 1;
    if (b >= p.B) return;
    mine = attn_seq(p, b);
    tiles = (mine.n_q * p.group + kTcAttnRows - 1) / kTcAttnRows;
    if (p.n_split > 1) splits = max(1, (mine.len + p.split_keys - 1) / p.split_keys);
  }
  // The next piece.
  __device__ __forceinline__ bool next(Work& w, AttnSeq& s) {
#pragma unroll 1
    while (tile >= 0) {
      if (each < 0) {
        each = same = 0;
        down = -1;
#pragma unroll 1
        for (int b1 = 0; b1 < p.B; b1 += 32) {
          look(b1);
          each += __reduce_add_sync(0xffffffffu, tiles > tile ? splits : 0);
          same = max(same, __reduce_max_sync(0xffffffffu, tiles > tile ? 0 : tiles));
        }
      }
      const int per = each * p.n_kv_heads, pairs = tile - same + 1;
      if (at >= per * pairs) {
        at -= per * pairs;
        tile = same - 1;
        each = -1;
        continue;
      }
      if (at / per != down) {
        down = at / per;
        b0 = before = 0;
      }
      const int place = at - down * per;
      const int of = place / p.n_kv_heads;  // of `each`
      w.h = place - of * p.n_kv_heads;
#pragma unroll 1
      for (; b0 < p.B; b0 += 32) {  // the sequence with the of-th piece
        look(b0);
        const int v = tiles > tile ? splits : 0;
        int sum = v;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
          const int up = __shfl_up_sync(0xffffffffu, sum, o);
          if ((int)(threadIdx.x & 31) >= o) sum += up;
        }
        const int mask = __ballot_sync(0xffffffffu, before + sum > of);
        if (mask) {
          const int src = __ffs(mask) - 1;
          w.b = b0 + src;
          w.split = of - before - __shfl_sync(0xffffffffu, sum - v, src);
          s.q0 = __shfl_sync(0xffffffffu, mine.q0, src);
          s.n_q = __shfl_sync(0xffffffffu, mine.n_q, src);
          s.len = __shfl_sync(0xffffffffu, mine.len, src);
          s.bad = false;
          break;
        }
        before += __shfl_sync(0xffffffffu, sum, 31);
      }
      if (b0 >= p.B) return false;  // the index arrays were changed meanwhile
      w.r0 = (tile - down) * kTcAttnRows;
      at += stride;
      const int other = stride;
      stride = back;
      back = other;
      w.rows = min(kTcAttnRows, s.n_q * p.group - w.r0);
      w.k0 = w.split * p.split_keys;
      w.k1 = min(min(s.len, attn_limit(s, (w.r0 + w.rows - 1) / p.group)), w.k0 + p.split_keys);
      w.n = w.k1 > w.k0 ? (w.k1 - w.k0 + kTile - 1) / kTile : 0;
      w.dual = w.rows <= kTile && w.n > 1;
      if (w.dual) {
        w.n0 = (w.n + 1) / 2;
        w.n1 = w.n / 2;
      } else {
        w.n0 = w.n;
        w.n1 = w.rows > kTile ? w.n : 0;
        if (TYPE == WAL_KV_BF16 && w.rows > kTile) {  // the first tile's rows may see fewer keys
          const int end = min(w.k1, attn_limit(s, (w.r0 + kTile - 1) / p.group));
          w.n0 = end > w.k0 ? (end - w.k0 + kTile - 1) / kTile : 0;
        }
      }
      return true;
    }
    return false;
  }
};

// ---------------------------------------------------------------------------
// K/V tiles by TMA (one warp): bf16 tiles as the MMAs want them, or codes and
// scales for the converters
// ---------------------------------------------------------------------------
template <int D, int TYPE>
__device__ __forceinline__ void load_tiles(const AttnParams& p, int most, const CUtensorMap* km, const CUtensorMap* vm,
                                           uint32_t base, const Bars& bars) {
  using C = Cfg<D, TYPE>;
  constexpr int kSlots = C::codes ? C::raws : C::slots;
  constexpr uint32_t kBytes = C::codes ? C::raw : C::tile;
  const uint32_t ring = base + (C::codes ? C::raw_off : C::ring_off);
  const int lane = threadIdx.x & 31;
  auto full = [&](int s) { return C::codes ? bars.raw_full(s) : bars.full(s); };
  auto empty = [&](int s) { return C::codes ? bars.raw_empty(s) : bars.empty(s); };
  uint32_t item = 0, tails = 0;
  bool ok = true, tail = false;
  Walk<TYPE> walk(p, most);
  Work w;
  AttnSeq s;
#pragma unroll 1
  while (ok && walk.next(w, s)) {
#pragma unroll 1
    for (int j = 0; j < w.n && ok; ++j) {
      const int kb = w.k0 + kTile * j, cnt = min(kTile, w.k1 - kb);
      // this tile's boxes: lane i's page (paged) or the packed rows
      int boxes = 1, box_rows = kTile, page = 0;
      if (p.table) {
        box_rows = min(kTile, 1 << p.shift);
        boxes = (cnt + box_rows - 1) / box_rows;
        if (lane < boxes) page = attn_page(p, w.b, kb + lane * box_rows);
      }
      const int x0 = p.table ? 0 : w.h * D, z0 = p.table ? w.h : 0;
      const int y0 = p.table ? kb & ((1 << p.shift) - 1) : s.q0 + kb;
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv, ++item) {
        const int slot = item % kSlots;
        if (item >= kSlots) ok = bar_wait(empty(slot), ((item / kSlots) & 1) ^ 1, p);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tail = !C::codes && kv == 1 && cnt < kTile;
        const uint32_t dst = ring + (uint32_t)slot * kBytes, bar = tail ? bars.v_tail() : full(slot);
        const uint32_t row_bytes = C::codes ? D + 4 : D * 2;
        if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(boxes * box_rows) * row_bytes);
        __syncwarp();
        if (lane < boxes) {  // a lane for each page
          if (C::codes) {
            tma_4d(dst + (uint32_t)(lane * box_rows) * D, kv ? vm : km, 0, y0, z0, page, bar);
            const float* sc = (kv ? p.vs : p.ks) + ((((int64_t)page * p.n_kv_heads + w.h) << p.shift) + y0);
            bulk_g2s(dst + kTile * D + (uint32_t)(lane * box_rows) * 4u, sc, (uint32_t)box_rows * 4u, bar);
          } else {
#pragma unroll
            for (int a = 0; a < D / 64; ++a)
              tma_4d(dst + a * 16384u + (uint32_t)(lane * box_rows) * 128u, kv ? vm : km, x0 + 64 * a, y0, z0, page, bar);
          }
        }
        __syncwarp();
        if (tail) {  // the piece's last V tile: zero the rows that hold no key of it
          ok = __all_sync(0xffffffffu, bar_wait(bar, tails & 1, p));
          if (!ok) break;
          ++tails;
          tail = false;
#pragma unroll 1
          for (int r8 = lane; r8 < (kTile - cnt) * (D / 8); r8 += 32) {
            const int r = cnt + r8 / (D / 8), ch = r8 % (D / 8);
            sts128(dst + (ch >> 3) * 16384u + sw128(r, ch & 7), make_uint4(0, 0, 0, 0));
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bars.full(slot));
        }
      }
    }
  }
  // nothing of this warp's stays in flight, whatever its readers waited for
  if (!ok && tail) mbar_drain(bars.v_tail(), tails & 1, p.status);
#pragma unroll 1
  for (uint32_t i = item > kSlots ? item - kSlots : 0; i < item; ++i) mbar_drain(full(i % kSlots), (i / kSlots) & 1, p.status);
}

// ---------------------------------------------------------------------------
// codes to bf16 tiles (four warps)
// ---------------------------------------------------------------------------
template <int D, int TYPE>
__device__ __forceinline__ void convert_tiles(const AttnParams& p, int most, uint32_t base, const Bars& bars) {
  using C = Cfg<D, TYPE>;
  const int tid = threadIdx.x & 127;
  uint32_t item = 0, tiles = 0;
  Walk<TYPE> walk(p, most);
  Work w;
  AttnSeq s;
#pragma unroll 1
  while (walk.next(w, s)) {
#pragma unroll 1
    for (int j = 0; j < w.n; ++j, ++tiles) {
      const int cnt = min(kTile, w.k1 - w.k0 - kTile * j);
      const int si = tiles % kScaleRing;
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv, ++item) {
        const int rs = item % C::raws, slot = item % C::slots;
        bool ok = bar_wait(bars.raw_full(rs), (item / C::raws) & 1, p);
        if (ok && kv == 0 && tiles >= kScaleRing) ok = bar_wait(bars.sc_empty(si), ((tiles / kScaleRing) & 1) ^ 1, p);
        if (ok && item >= C::slots) ok = bar_wait(bars.empty(slot), ((item / C::slots) & 1) ^ 1, p);
        if (!__all_sync(0xffffffffu, ok)) return;
        const uint32_t src = base + C::raw_off + (uint32_t)rs * C::raw, dst = base + C::ring_off + (uint32_t)slot * C::tile;
        // keys that are not there get codes and scales of zero
        sts32(base + C::scale_off + (uint32_t)(si * 2 + kv) * (kTile * 4) + 4u * tid,
              tid < cnt ? lds32(src + kTile * D + 4u * tid) : 0u);
#pragma unroll 4
        for (int q = 0; q < D / 16; ++q) {
          // 16 codes: piece `part` (of 64 columns' four) of `atom` in `row`.  Eight
          // lanes read 128 bytes in different banks and write chunks that are.
          const int e = q * 128 + tid, part = e & 3;
          int row, atom;
          if (D == 128) {
            row = 2 * (e >> 4) + ((e >> 2) & 1);
            atom = ((e >> 2) ^ (e >> 3)) & 1;
          } else {
            row = e >> 2;
            atom = 0;
          }
          uint4 v = lds128(src + (uint32_t)row * D + atom * 64u + part * 16u);
          if (row >= cnt) v = make_uint4(0, 0, 0, 0);
          uint4 x, y;
          dev::codes4_to_bf16<TYPE>(v.x, x.x, x.y);
          dev::codes4_to_bf16<TYPE>(v.y, x.z, x.w);
          dev::codes4_to_bf16<TYPE>(v.z, y.x, y.y);
          dev::codes4_to_bf16<TYPE>(v.w, y.z, y.w);
          const uint32_t a = dst + atom * 16384u;
          sts128(a + sw128(row, 2 * part), x);
          sts128(a + sw128(row, 2 * part + 1), y);
        }
        mbar_arrive(bars.raw_empty(rs));
        if (kv == 1) mbar_arrive(bars.sc_full(si));
        fence_proxy_async_smem();
        mbar_arrive(bars.full(slot));
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Q tiles (two warps)
// ---------------------------------------------------------------------------
// 16-byte asynchronous copies, all of a tile in flight at once: a row may be any
// (token, head), so no box fits every group.
template <int D, int TYPE>
__device__ __forceinline__ void load_q(const AttnParams& p, int most, uint32_t base, const Bars& bars) {
  using C = Cfg<D, TYPE>;
  constexpr int kChunks = D / 8, kStep = kQThreads / kChunks;  // 16-byte chunks of a row, rows between a thread's copies
  const int tid = threadIdx.x & (kQThreads - 1);               // of warps 10, 11
  const int ch = tid % kChunks, r_first = tid / kChunks;
  const int step_tok = kStep / p.group, step_head = kStep % p.group;
  uint32_t uses0 = 0, uses1 = 0;
  Walk<TYPE> walk(p, most);
  Work w;
  AttnSeq s;
#pragma unroll 1
  while (walk.next(w, s)) {
    const bool both = w.has_q(0) && w.has_q(1);
#pragma unroll 1
    for (int t = 0; t < 2; ++t) {  // both tiles' copies, then what is left to do for each
      if (!w.has_q(t)) continue;
      uint32_t& uses = t ? uses1 : uses0;
      if (!__all_sync(0xffffffffu, uses == 0 || bar_wait(bars.q_empty(t), (uses - 1) & 1, p))) {
        asm volatile("cp.async.wait_all;" ::: "memory");
        return;
      }
      ++uses;
      const uint32_t dst = base + t * C::tile + (ch >> 3) * 16384u;
      int row = w.r0 + kTile * t + r_first, tok = row / p.group, rem = row - tok * p.group;
      const uint16_t* q = p.Q + s.q0 * p.ldq + (int64_t)w.h * p.group * D + 8 * ch;
#pragma unroll 4
      for (int r = r_first; r < kTile; r += kStep) {
        const bool there = kTile * t + r < w.rows;  // other rows are zero
        const uint16_t* src = there ? q + tok * p.ldq + rem * D : p.Q;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + sw128(r, ch & 7)), "l"(src), "r"(there ? 16 : 0)
                     : "memory");
        tok += step_tok;
        rem += step_head;
        if (rem >= p.group) {
          rem -= p.group;
          ++tok;
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
#pragma unroll 1
    for (int t = 0; t < 2; ++t) {
      if (!w.has_q(t)) continue;
      if (both && t == 0)
        asm volatile("cp.async.wait_group 1;" ::: "memory");
      else
        asm volatile("cp.async.wait_group 0;" ::: "memory");
      // A negative scale is a sign on Q, a scale of zero makes it zero: the
      // scores are then multiplied by sl > 0.
      if (p.scale_log2 <= 0.f) {
        const uint32_t keep = p.scale_log2 == 0.f ? 0u : ~0u, flip = p.scale_log2 < 0.f ? 0x80008000u : 0u;
        const uint32_t dst = base + t * C::tile + (ch >> 3) * 16384u;
#pragma unroll 1
        for (int r = r_first; r < kTile; r += kStep) {
          const uint4 v = lds128(dst + sw128(r, ch & 7));
          sts128(dst + sw128(r, ch & 7), make_uint4((v.x & keep) ^ flip, (v.y & keep) ^ flip, (v.z & keep) ^ flip, (v.w & keep) ^ flip));
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(bars.q_full(t));
    }
  }
}

// ---------------------------------------------------------------------------
// MMA issue (one warp; the same elected lane issues everything)
// ---------------------------------------------------------------------------
// The whole warp walks the loop: with one lane alone in it the operands are not
// known to be uniform, and an MMA took about 200 cycles to issue instead of the
// 64 that it runs.
template <int D, int TYPE>
__device__ __forceinline__ void issue_mmas(const AttnParams& p, int most, uint32_t base, uint32_t tmem, const Bars& bars) {
  using C = Cfg<D, TYPE>;
  constexpr uint32_t id_s = idesc_bf16(128, 128, false), id_o = idesc_bf16(128, D, true);
  const uint32_t q_lo = desc_lo(base, kDescK), k_lo = desc_lo(base + C::ring_off, kDescK), v_lo = desc_lo(base + C::ring_off, kDescV);
  // Ring position of a K or V tile.
  struct Pos {
    uint32_t slot, parity;
    __device__ void next() {
      if (++slot == C::slots) {
        slot = 0;
        parity ^= 1;
      }
    }
    __device__ void next2() {
      next();
      next();
    }
  };
  auto wait = [&](uint32_t bar, uint32_t parity) { return bar_wait(bar, parity, p); };
  auto kv_wait = [&](const Pos& at) { return bar_wait(bars.full(at.slot), at.parity, p); };
  auto all = [&](bool ok) { return (bool)__all_sync(0xffffffffu, ok); };
  // the functions below run in the elected lane
  auto scores = [&](int t, int qt, uint32_t slot) {  // S_t = Q_qt K^T
    const uint32_t a = q_lo + qt * (C::tile >> 4), b = k_lo + slot * (C::tile >> 4), d = tmem + 128u * t;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      const uint32_t off = ((k >> 2) * 16384u + (k & 3) * 32u) >> 4;
      mma_ss(d, a + off, b + off, id_s, k > 0);
    }
    mma_commit(bars.s_full(t));
  };
  auto weigh = [&](int t, int half, uint32_t slot, bool more) {  // O_t (+)= P_t V over the first or last 64 keys
    const uint32_t a = tmem + 128u * t + 32u * half, b = v_lo + slot * (C::tile >> 4) + half * (8192u >> 4), d = tmem + 256u + (uint32_t)D * t;
#pragma unroll
    for (int k = 0; k < 4; ++k) mma_ts(d, a + 8u * k, b + k * (2048u >> 4), id_o, more || k > 0);
  };
  Pos pos = {0, 0};                                  // the piece's next K tile
  uint32_t quse0 = 0, quse1 = 0, ph0 = 0, ph1 = 0;  // parities: of the Q tiles' uses, of the halves' weights
  bool ok = true;
  Walk<TYPE> walk(p, most);
  Work w;
  AttnSeq s;
#pragma unroll 1
  while (ok && walk.next(w, s)) {
    if (w.n == 0) continue;
    if (w.has_q(0)) {
      ok = wait(bars.q_full(0), quse0);
      quse0 ^= 1;
    }
    if (ok && w.has_q(1)) {
      ok = wait(bars.q_full(1), quse1);
      quse1 ^= 1;
    }
    const int ahead = w.dual ? 2 : 1;  // K tiles that S runs ahead of the weights
    Pos v = pos;                        // V_j
    v.next();
    // the first scores of both halves: of one K tile, or (dual) of two
#pragma unroll 1
    for (int t = 0; t < 2; ++t) {
      if (w.n_t(t) == 0) continue;
      ok = all(ok && kv_wait(pos));
      if (!ok) break;
      tc_fence_after();
      const bool last = w.dual || t == 1 || w.n1 == 0;  // of the K tile's readers
      if (elect_one()) {
        scores(t, w.dual ? 0 : t, pos.slot);
        if (w.dual ? t == 1 && w.n == 2 : w.n_t(t) == 1) mma_commit(bars.q_empty(w.dual ? 0 : t));
        if (last) mma_commit(bars.empty(pos.slot));
      }
      __syncwarp();
      if (last) pos.next2();
    }
#pragma unroll 1
    for (int j = 0; j < w.n && ok; ++j) {
      const bool more_k = j + ahead < w.n;  // `pos` is there
#pragma unroll 1
      for (int t = w.dual ? j & 1 : 0; t < 2; ++t) {
        if (!w.dual && j >= w.n_t(t)) continue;
        const uint32_t ph = t ? ph1 : ph0;
        ok = all(kv_wait(v) && wait(bars.p_half(t), ph));
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) weigh(t, 0, v.slot, j >= ahead);
        __syncwarp();
        const bool again = j + ahead < (w.dual ? w.n : w.n_t(t));  // this half has another tile
        const bool last = w.dual || t == 1 || w.n1 == 0;            // of the step's products
        ok = all(wait(bars.p_full(t), ph));
        if (!ok) break;
        if (t) ph1 ^= 1; else ph0 ^= 1;
        tc_fence_after();
        if (elect_one()) {
          weigh(t, 1, v.slot, true);
          if (last) mma_commit(bars.empty(v.slot));
          if (!again) mma_commit(bars.o_done(t));
        }
        __syncwarp();
        if (again) {  // while the tensor core weighs; in a short ring this tile takes the place of V's
          ok = all(kv_wait(pos));
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            scores(t, w.dual ? 0 : t, pos.slot);
            if (j + ahead + 1 == (w.dual ? w.n : w.n_t(t))) mma_commit(bars.q_empty(w.dual ? 0 : t));
            if (last) mma_commit(bars.empty(pos.slot));
          }
          __syncwarp();
        }
        if (w.dual) break;
      }
      v.next2();
      if (more_k) pos.next2();
    }
  }
  if (elect_one()) mma_commit(bars.drained());
  __syncwarp();
  mbar_drain(bars.drained(), 0, p.status);
}

// ---------------------------------------------------------------------------
// rows beside a non-finite value, and rows without a result
// ---------------------------------------------------------------------------
// Rows of half t that a key which they do not see has made NaN.  This comes after
// the CTA's last piece, when nobody waits for this warp; a call of its own, so
// that its code and registers stay out of the loop of softmax_rows.
template <int D, int TYPE>
__device__ __noinline__ void redo_rows(const AttnParams& p, int most, int t) {
  const int tid = threadIdx.x & 127;
  Walk<TYPE> walk(p, most);
  Work w;
  AttnSeq s;
#pragma unroll 1
  while (walk.next(w, s)) {
    const int row = w.r0 + (w.dual ? 0 : kTile * t) + tid;
    const bool live = row < w.r0 + w.rows && !(w.dual && t == 1);
    const int tok = live ? row / p.group : 0, head = w.h * p.group + (live ? row - tok * p.group : 0);
    if (!__any_sync(0xffffffffu, live)) continue;
    const int last = attn_last_nonfinite<D>(p, s, w.b, w.h, __shfl_sync(0xffffffffu, attn_limit(s, tok), 0), w.k1);
    bool nan = false;
    if (live && attn_limit(s, tok) <= last) {
      const uint4* o = reinterpret_cast<const uint4*>(p.O + (s.q0 + tok) * p.ldo + head * D);
#pragma unroll 2
      for (int i = 0; i < D / 8; ++i) {
        const uint4 o8 = o[i];
        const uint32_t u[4] = {o8.x, o8.y, o8.z, o8.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) nan |= (u[k] & 0x7FFFu) > 0x7F80u || ((u[k] >> 16) & 0x7FFFu) > 0x7F80u;
      }
    }
    uint32_t again = __ballot_sync(0xffffffffu, nan);
#pragma unroll 1
    while (again) {
      const int src = __ffs(again) - 1;
      again &= again - 1;
      attend_row<D>(p, s, w.b, __shfl_sync(0xffffffffu, head, src), __shfl_sync(0xffffffffu, tok, src));
    }
  }
}

// Rows of half t in the CTA's pieces after the first `done`, which a wait that gave
// up has cut off: NaN, so that the loss shows even if nobody reads the status word.
template <int D, int TYPE>
__device__ __noinline__ void lose_rows(const AttnParams& p, int most, int t, uint32_t done) {
  const int tid = threadIdx.x & 127;
  Walk<TYPE> walk(p, most);
  Work w;
  AttnSeq s;
#pragma unroll 1
  for (uint32_t i = 0; walk.next(w, s); ++i) {
    const int row = w.r0 + (w.dual ? 0 : kTile * t) + tid;
    if (i >= done && row < w.r0 + w.rows && !(w.dual && t == 1)) {
      const int tok = row / p.group, head = w.h * p.group + row - tok * p.group;
      const float nan = __int_as_float(0x7FC00000);
      if (p.n_split > 1) {
        p.part_ml[(int64_t)w.split * p.T * p.n_heads + attn_part_row(p, s, tok, head)] = make_float2(nan, nan);
      } else {
        uint4* o = reinterpret_cast<uint4*>(p.O + (s.q0 + tok) * p.ldo + head * D);
#pragma unroll 1
        for (int k = 0; k < D / 8; ++k) o[k] = make_uint4(0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u);
      }
    }
    __syncwarp();
  }
}

// ---------------------------------------------------------------------------
// softmax and output (four warps for a half of the CTA, a row a thread)
// ---------------------------------------------------------------------------
// The loops over steps and pieces are kept rolled here and in the other roles:
// the schedulers' instruction caches are small, and code that is fetched anew
// in every step costs the MMA warp, which runs each of its instructions once a
// step, several times what the instructions do.
template <int D, int TYPE>
__device__ __forceinline__ void softmax_rows(const AttnParams& p, int most, int t, float sl, uint32_t base,
                                             uint32_t tmem, const Bars& bars) {
  using C = Cfg<D, TYPE>;
  const int tid = threadIdx.x & 127;
  const bool lead = (tid & 31) == 0;
  const uint32_t lanes = (uint32_t)(tid & 96) << 16;
  const uint32_t t_s = tmem + 128u * t + lanes, t_o = tmem + 256u + (uint32_t)D * t + lanes;
  const float2 sl2 = make_float2(sl, sl);
  const bool sectors = (((uintptr_t)p.O | (uintptr_t)(p.ldo * 2)) & 31) == 0;  // every row of O starts on 32 bytes
  uint32_t steps = 0, pieces = 0, duals = 0, tiles = 0;
  uint32_t begun = 0;
  bool redo = false, lost = false;
  auto wait = [&](uint32_t bar, uint32_t parity) { return (bool)__all_sync(0xffffffffu, bar_wait(bar, parity, p)); };
  auto arrive = [&](uint32_t bar) {  // for the warp
    tc_fence_before();
    __syncwarp();
    if (lead) mbar_arrive(bar);
  };
  Walk<TYPE> walk(p, most);
  Work w;
  AttnSeq s;
#pragma unroll 1
  while (walk.next(w, s)) {
    ++begun;
    const int row = w.r0 + (w.dual ? 0 : kTile * t) + tid;
    const int n = w.n_t(t);
    const int lim = row < w.r0 + w.rows ? min(w.k1, attn_limit(s, row / p.group)) : w.k1;
    const int lim0 = __shfl_sync(0xffffffffu, lim, 0);  // the warp's smallest: limits grow with the row
    float m = -INFINITY, l = 0.f;
#pragma unroll 1
    for (int k = 0; k < n; ++k, ++steps) {
      const int kb = w.k0 + kTile * w.tile_of(t, k);
      const uint32_t ti = tiles + w.tile_of(t, k);
      const uint32_t sc = base + C::scale_off + (ti % kScaleRing) * (2 * kTile * 4);  // K's scales of the tile, then V's
      lost = !wait(bars.s_full(t), steps & 1) || (C::codes && !wait(bars.sc_full(ti % kScaleRing), (ti / kScaleRing) & 1));
      if (lost) break;
      tc_fence_after();
      float x[kTile];
#pragma unroll
      for (int q = 0; q < 4; ++q) tmem_ld32(t_s + 32u * q, x + 32 * q);
      tmem_ld_wait();
      const int seen = lim - kb;  // this row's keys in the tile
      const bool masked = kb + kTile > lim0;
      // scores of n keys from the q-th on: the keys' K scales, and -inf for keys
      // that the row does not see
      auto prepare = [&](float* v, int q, int n) {
        if (C::codes) {
#pragma unroll
          for (int e = 0; e < n; e += 4) {
            const uint4 k4 = lds128(sc + 4u * (q + e));
            const float2 y = mul2(make_float2(v[e], v[e + 1]), make_float2(__uint_as_float(k4.x), __uint_as_float(k4.y)));
            const float2 z = mul2(make_float2(v[e + 2], v[e + 3]), make_float2(__uint_as_float(k4.z), __uint_as_float(k4.w)));
            v[e] = y.x; v[e + 1] = y.y;
            v[e + 2] = z.x; v[e + 3] = z.y;
          }
        }
        if (masked) {
#pragma unroll
          for (int e = 0; e < n; ++e) v[e] = q + e < seen ? v[e] : -INFINITY;
        }
      };
      prepare(x, 0, kTile);
      // weights of 32 keys, as bf16 pairs, and their sums
      float2 sum[2];
      auto weights = [&](int q, const float* v, float ref, uint32_t(&pk)[16]) {
        const float2 ref2 = make_float2(ref, ref);
        uint4 v4;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float2 y = fma2(make_float2(v[2 * e], v[2 * e + 1]), sl2, ref2);
          y.x = ex2(y.x);
          y.y = ex2(y.y);
          sum[e & 1] = add2(sum[e & 1], y);
          if (C::codes) {
            if (!(e & 1)) v4 = lds128(sc + kTile * 4 + 4u * (32 * q + 2 * e));
            y = mul2(y, (e & 1) ? make_float2(__uint_as_float(v4.z), __uint_as_float(v4.w))
                                : make_float2(__uint_as_float(v4.x), __uint_as_float(v4.y)));
          }
          pk[e] = dev::float2_to_bf16x2(y.x, y.y);
        }
      };
      float mx[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) mx[q] = max3(x[2 * q], x[2 * q + 1], x[2 * q]);
#pragma unroll
      for (int q = 8; q < kTile; q += 8)
#pragma unroll
        for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], x[q + 2 * e], x[q + 2 * e + 1]);
      const float top = max3(max3(mx[0], mx[1], mx[2]), mx[3], mx[3]) * sl;
      const bool grow = !(top <= m + kLazy);
      if (__any_sync(0xffffffffu, grow)) {
        // a NaN or +inf among the scores makes the row NaN
        const float mn = !grow ? m : top < INFINITY ? top : __int_as_float(0x7FC00000);
        const float f = grow ? ex2(m - mn) : 1.f;  // 0 for a row that had no key yet
        m = mn;
        l *= f;
        if (k > 0) {
#pragma unroll 1
          for (int q = 0; q < D / 16; ++q) {
            uint32_t o[16];
            tmem_ld16(t_o + 16u * q, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st16(t_o + 16u * q, o);
          }
        }
      }
      const float ref = m == -INFINITY ? 0.f : -m;
      sum[0] = sum[1] = make_float2(0.f, 0.f);
      uint32_t pa[16], pb[16];
      {
        weights(0, x, ref, pa);
        tmem_st16(t_s, pa);
        weights(1, x + 32, ref, pb);
        tmem_st16(t_s + 16u, pb);
        tmem_st_wait();
        arrive(bars.p_half(t));
        weights(2, x + 64, ref, pa);
        tmem_st16(t_s + 32u, pa);
        weights(3, x + 96, ref, pb);
        tmem_st16(t_s + 48u, pb);
        tmem_st_wait();
        arrive(bars.p_full(t));
      }
      sum[0] = add2(sum[0], sum[1]);
      l += sum[0].x + sum[0].y;
      if (C::codes && lead) {  // eight arrivals free the scales: one of a warp, two where one half alone reads them
        mbar_arrive(bars.sc_empty(ti % kScaleRing));
        if (w.dual || w.rows <= kTile) mbar_arrive(bars.sc_empty(ti % kScaleRing));
      }
    }
    if (lost) break;
    tiles += w.n;

    // output: the row's sums over its keys, or its share of them.  A dual
    // piece's rows are half 0's to write.
    const bool live = row < w.r0 + w.rows && !(w.dual && t == 1);
    float f = 1.f, f1 = 0.f;  // factors of this half's and the other half's sums
    if (n > 0) {
      lost = !wait(bars.o_done(t), pieces++ & 1);
      if (lost) break;
      tc_fence_after();
    }
    if (w.dual) {
      const uint32_t ml = base + C::ml_off + 8u * tid;
      if (t == 1) {  // half 0 takes it from here
        sts64(ml, make_uint2(__float_as_uint(m), __float_as_uint(l)));
        arrive(bars.join());
        lost = !wait(bars.o1_free(), duals++ & 1);
        if (lost) break;
        continue;
      }
      lost = !wait(bars.join(), duals++ & 1);
      if (lost) break;
      tc_fence_after();
      const uint2 u = lds64(ml);
      const float m1 = __uint_as_float(u.x), l1 = __uint_as_float(u.y), mm = fmaxf(m, m1), ref = mm == -INFINITY ? 0.f : mm;
      f = ex2(m - ref);
      f1 = ex2(m1 - ref);
      m = mm;
      l = l * f + l1 * f1;
    }
    const int tok = live ? row / p.group : 0, head = w.h * p.group + (live ? row - tok * p.group : 0);
    const bool partial = p.n_split > 1;
    const float inv = lim == 0 ? 0.f : 1.f / l;
    bool nan = false;
    const int64_t pr = (int64_t)w.split * p.T * p.n_heads + attn_part_row(p, s, tok, head);
#pragma unroll 1
    for (int q = 0; q < D / 32; ++q) {
      float o[32];
      if (n > 0) {
        tmem_ld32(t_o + 32u * q, o);
        tmem_ld_wait();
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = 0.f;
      }
      if (w.dual) {
        float o1[32];
        tmem_ld32(t_o + (uint32_t)D + 32u * q, o1);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = o[e] * f + o1[e] * f1;
      }
      if (live && partial) {
#pragma unroll
        for (int e = 0; e < 4; ++e) stg256(p.part_o + pr * D + 32 * q + 8 * e, reinterpret_cast<const uint32_t*>(o) + 8 * e);
      } else if (live) {
        uint32_t u[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float a = lim == 0 ? 0.f : o[2 * e] * inv, b = lim == 0 ? 0.f : o[2 * e + 1] * inv;
          nan |= a != a || b != b;
          u[e] = dev::float2_to_bf16x2(a, b);
        }
        uint16_t* dst = p.O + (s.q0 + tok) * p.ldo + head * D + 32 * q;
        if (sectors) {
          stg256(dst, u);
          stg256(dst + 16, u + 8);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            reinterpret_cast<uint4*>(dst)[e] = make_uint4(u[4 * e], u[4 * e + 1], u[4 * e + 2], u[4 * e + 3]);
        }
      }
      __syncwarp();
    }
    if (w.dual) arrive(bars.o1_free());
    if (partial) {
      if (live) p.part_ml[pr] = make_float2(m, l);
      continue;
    }
    redo |= __any_sync(0xffffffffu, live && nan && l == l && lim < w.k1);
  }
  if (redo) redo_rows<D, TYPE>(p, most, t);
  if (lost) lose_rows<D, TYPE>(p, most, t, begun - 1);
}

template <int D, int TYPE>
__global__ void __launch_bounds__(Cfg<D, TYPE>::threads, 1)
attn_tc_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap km, const __grid_constant__ CUtensorMap vm) {
  using C = Cfg<D, TYPE>;
  extern __shared__ uint8_t smem_raw[];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - smem_u32(smem_raw));
  const Bars bars = {base + C::bar_off};
  int* shape = reinterpret_cast<int*>(gbase + C::bar_off + 404);  // most tile pairs of a sequence, any out of range
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0);
  if (threadIdx.x == 0) {
#pragma unroll 1
    for (int i = 0; i < C::slots; ++i) {
      mbar_init(bars.full(i), C::codes ? 128 : 1);
      mbar_init(bars.empty(i), 1);
    }
    if (C::codes) {
      for (int i = 0; i < C::raws; ++i) {
        mbar_init(bars.raw_full(i), 1);
        mbar_init(bars.raw_empty(i), 128);
      }
      for (int i = 0; i < kScaleRing; ++i) {
        mbar_init(bars.sc_full(i), 128);
        mbar_init(bars.sc_empty(i), 8);
      }
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(bars.q_full(t), kQThreads);
      mbar_init(bars.q_empty(t), 1);
      mbar_init(bars.s_full(t), 1);
      mbar_init(bars.p_full(t), 4);
      mbar_init(bars.p_half(t), 4);
      mbar_init(bars.o_done(t), 1);
    }
    mbar_init(bars.join(), 4);
    mbar_init(bars.o1_free(), 4);
    mbar_init(bars.v_tail(), 1);
    mbar_init(bars.drained(), 1);
    mbar_init_fence();
    shape[0] = shape[1] = 0;
  }
  if (warp == 8) {
    tmem_alloc(bars.tmem_slot(), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, lds32(bars.tmem_slot()), 0);
  // how far the pieces reach, and which sequences are out of range
  {
    int tiles = 0, bad = 0;
#pragma unroll 1
    for (int b = threadIdx.x; b < p.B; b += C::threads) {
      const AttnSeq s = attn_seq(p, b);
      bad |= s.bad;
      tiles = max(tiles, (s.n_q * p.group + kTcAttnRows - 1) / kTcAttnRows);
    }
    atomicMax(&shape[0], tiles);
    if (bad) shape[1] = 1;
  }
  __syncthreads();
  const int most = shape[0];
  if (blockIdx.x == 0 && threadIdx.x == 0 && p.status) {
    if (p.clear) *p.status = p.n_split == 1 && shape[1] ? (int32_t)WAL_ERR_ARG : 0;
    else if (shape[1]) attn_report(p.status);
  }
  const float sl = p.scale_log2 == 0.f ? 1.f : fabsf(p.scale_log2);

  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::soft_regs));
    softmax_rows<D, TYPE>(p, most, warp >> 2, sl, base, tmem, bars);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::other_regs));
    if (warp == 8) {
      issue_mmas<D, TYPE>(p, most, base, tmem, bars);
    } else if (warp == 9) {
      load_tiles<D, TYPE>(p, most, &km, &vm, base, bars);
    } else if (warp < 12) {
      load_q<D, TYPE>(p, most, base, bars);
    } else {
      convert_tiles<D, TYPE>(p, most, base, bars);
    }
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

// K or V as (column, row, head, page): boxes of up to 128 rows, and of 64 bf16
// columns in the 128-byte swizzle or of whole rows of codes.
int make_map(CUtensorMap* map, const AttnParams& p, const void* base, int64_t ld) {
  const EncodeFn enc = encode_fn();
  if (!enc) return fail(WAL_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
  const bool codes = p.type != WAL_KV_BF16;
  const cuuint64_t D = (cuuint64_t)p.head_dim, H = (cuuint64_t)p.n_kv_heads, size = codes ? 1 : 2;
  cuuint64_t dims[4] = {H * D, (cuuint64_t)p.T, 1, 1};  // packed rows: the head is part of the column
  cuuint64_t strides[3] = {(cuuint64_t)ld * 2, (cuuint64_t)ld * 2, (cuuint64_t)ld * 2};
  cuuint32_t box[4] = {codes ? (cuuint32_t)D : 64, kTile, 1, 1}, step[4] = {1, 1, 1, 1};
  if (p.table) {
    const cuuint64_t page = (cuuint64_t)1 << p.shift;
    dims[0] = D;
    dims[1] = page;
    dims[2] = H;
    dims[3] = (cuuint64_t)p.n_pages;
    strides[0] = D * size;
    strides[1] = page * D * size;
    strides[2] = H * page * D * size;
    if (page < kTile) box[1] = (cuuint32_t)page;
  }
  const CUresult r = enc(map, codes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims,
                         strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, codes ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(WAL_ERR_CUDA, "cuTensorMapEncodeTiled failed with " + std::to_string((int)r));
  return WAL_OK;
}

template <int D, int TYPE>
int launch_one(const AttnParams& p, cudaStream_t stream) {
  CUtensorMap km = {}, vm = {};
  int st = make_map(&km, p, p.k, p.ldk);
  if (st || (st = make_map(&vm, p, p.v, p.ldv))) return st;
  // the attribute is per device; setting it again is cheap and needs no state
  cudaError_t e = cudaFuncSetAttribute(attn_tc_kernel<D, TYPE>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg<D, TYPE>::smem);
  if (e == cudaSuccess) {
    const int64_t tiles = ((int64_t)p.max_q * p.group + kTcAttnRows - 1) / kTcAttnRows;
    const int64_t pieces = tiles * p.n_split * p.n_kv_heads * p.B;
    attn_tc_kernel<D, TYPE><<<(unsigned)(pieces < kGrid ? pieces : kGrid), Cfg<D, TYPE>::threads, Cfg<D, TYPE>::smem, stream>>>(p, km, vm);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return fail(WAL_ERR_CUDA, std::string("attn_tc_kernel launch: ") + cudaGetErrorString(e));
  return WAL_OK;
}

}  // namespace

int launch_attn_tc(const AttnParams& p, cudaStream_t stream) {
  const bool wide = p.head_dim == 128;
  switch (p.type) {
    case WAL_KV_BF16: return wide ? launch_one<128, WAL_KV_BF16>(p, stream) : launch_one<64, WAL_KV_BF16>(p, stream);
    case WAL_KV_INT8: return wide ? launch_one<128, WAL_KV_INT8>(p, stream) : launch_one<64, WAL_KV_INT8>(p, stream);
    default: return wide ? launch_one<128, WAL_KV_E4M3>(p, stream) : launch_one<64, WAL_KV_E4M3>(p, stream);
  }
}

}  // namespace wal
