// Internal interface of the attention kernels (wal_attn.cu, wal_attn_tc.cu).
#pragma once

#include "wal_kv.h"

namespace wal {

// Parameters of one attention call.  A sequence's query rows are counted as
// (token, head of the group), token-major: row r of K/V head h is new token
// r / group and q head h * group + r % group.
struct AttnParams {
  const uint16_t* Q;
  uint16_t* O;
  const void* k;             // cache pages, or packed rows when table is NULL
  const void* v;
  const float* ks;           // scales of an 8-bit cache
  const float* vs;
  const int32_t* q_start;
  const int32_t* kv_len;     // NULL for a prompt: as many keys as queries
  const int32_t* table;
  int64_t ldq, ldo, ldk, ldv, ld_table;
  int n_heads, n_kv_heads, group, head_dim, type;
  int shift, n_pages;        // log2(page_size)
  int T, B, max_q, max_kv;
  float scale_log2;          // scale * log2(e)
  int polls;                 // of a device wait before it gives up
  int32_t* status;           // NULL: nothing is recorded
  // A call that splits its keys clears the status word in its first kernel and
  // reports index values in its second, a prompt does both in its one kernel,
  // another call after a memset.
  bool clear;
  // keys split over CTAs: split s holds keys [s * split_keys, (s + 1) * split_keys)
  int n_split, split_keys;
  float* part_o;             // n_split > 1: [n_split][T * n_heads][head_dim], sums of w v
  float2* part_ml;           // [n_split][T * n_heads]: {m, l}, m in units of log2
  // The general kernels (GEN): a window, or a shared prefix, whose keys one launch
  // takes (kPrefix, its "sequences" being the groups) and what is behind it another
  // (kOwn), each leaving partial results, the second from split part_first on.
  bool gen, tc;              // tc: the tensor-core kernel
  int window, sinks;         // a row sees its last `window` keys and the first `sinks`
  int gran;                  // keys of a piece are looked up in runs of this many, aligned where there are pages
  int sinks_pad;             // the first keys' runs
  int piece_toks;            // new tokens of a piece of the tensor-core kernel at most
  int phase;
  int part_first, prefix_keys;  // kOwn: the prefix has part_first splits at most, of prefix_keys keys
  const int32_t* group_start;
  const int32_t* prefix_len;
  int n_groups, n_seqs, max_prefix, max_own;
};
enum { kAll = 0, kPrefix = 1, kOwn = 2 };  // phase
constexpr int kNoWindow = 1 << 30;

// The tensor-core kernel (wal_attn_tc.cu).
constexpr int kTcAttnRows = 256;  // query rows of one CTA there
int launch_attn_tc(const AttnParams& p, cudaStream_t stream);
// The general kernel of few query rows (wal_attn_ring.cu).
int launch_attn_ring(const AttnParams& p, cudaStream_t stream);

// An index value out of range: recorded, unless something is already (a wait that gave up).
__device__ __forceinline__ void attn_report(int32_t* status) { atomicCAS(status, 0, (int32_t)WAL_ERR_ARG); }

// Sequence b as its index arrays give it; n_q = 0 where they are out of range.
struct AttnSeq {
  int q0, n_q, len;
  bool bad;
  int tab;       // GEN: its row of the page table,
  int lo, head;  // how many keys it shares (kOwn takes those from there on), and the table row of these
};
// Group g of a shared call: its sequences [first, last), their rows [q0, q1), the keys they share; false if out of range.
struct AttnGroup {
  int first, last, q0, q1, keys;
};
__device__ __forceinline__ bool attn_group(const AttnParams& p, int g, AttnGroup& r) {
  r.first = p.group_start[g];
  r.last = p.group_start[g + 1];
  r.keys = p.prefix_len[g];
  if (r.first < 0 || r.last < r.first || r.last > p.n_seqs || r.keys < 0 || r.keys > p.max_prefix) return false;
  r.q0 = p.q_start[r.first];
  r.q1 = p.q_start[r.last];
  return r.q0 >= 0 && r.q1 >= r.q0 && r.q1 <= p.T;
}
// WARP: the lanes of a warp ask for one sequence and look for its group together.  Loads
// come before the checks of what others gave, so that they wait for one another as little
// as they can.
template <bool GEN = false, bool WARP = false>
__device__ __forceinline__ AttnSeq attn_seq(const AttnParams& p, int b) {
  AttnSeq s = {0, 0, 0, true};
  if (GEN) {
    s.tab = s.head = b;
    s.lo = 0;
    if (p.phase == kPrefix) {
      AttnGroup g;
      if (!attn_group(p, b, g)) return s;
      s.tab = g.first;
      s.q0 = g.q0;
      s.n_q = g.keys ? g.q1 - g.q0 : 0;
      s.len = g.keys;
      s.bad = false;
      return s;
    }
  }
  const int q0 = p.q_start[b], q1 = p.q_start[b + 1];
  int len = p.kv_len ? p.kv_len[b] : 0;
  int g = 0;
  if (GEN && p.phase == kOwn) {  // the last group that starts at b or before
    int end = p.n_groups;
    if (WARP) {
      const int lane = threadIdx.x & 31;
      for (int size = end; size > 1;) {
        const int step = (size + 31) >> 5, i = g + lane * step;
        const int at = p.group_start[min(i, p.n_groups - 1)];
        // the first probe is taken for granted: `first` tells below
        const uint32_t below = __ballot_sync(0xffffffffu, lane * step < size && i < p.n_groups && at <= b) | 1u;
        g += (31 - __clz(below)) * step;
        size = step;
      }
    } else {
      while (end - g > 1) {
        const int mid = (g + end) >> 1;
        if (p.group_start[mid] <= b) g = mid; else end = mid;
      }
    }
  }
  if (!p.kv_len) len = q1 - q0;
  const bool fits = q0 >= 0 && q1 >= q0 && q1 <= p.T && q1 - q0 <= p.max_q && len >= 0 && len <= p.max_kv;
  if (GEN && p.phase == kOwn) {
    AttnGroup r;
    const int first = p.group_start[g];
    const bool sound = attn_group(p, g, r);
    if (!fits) return s;
    if (first <= b && b < r.last) {  // behind the last group, a sequence shares nothing whatever that group holds
      if (!sound || q0 < r.q0 || q1 > r.q1) return s;
      s.lo = r.keys;
      s.head = r.first;
    }
    // Without shared keys, tokens before the first key see nothing, as elsewhere.  A
    // sequence without new tokens may hold less than its group shares.
    if ((s.lo && q1 > q0 && len - (q1 - q0) < s.lo) || len - s.lo > p.max_own) {
      s.lo = 0;
      return s;
    }
  }
  if (!fits) return s;
  s.q0 = q0;
  s.n_q = q1 - q0;
  s.len = len;
  s.bad = false;
  return s;
}
// Where the starts of a shared call's groups fall, it is open whose a sequence is: all of
// them are left out then.  The two launches may take a sequence for any group's, within
// all bounds, and leave partial results of two groups in one row; nobody reads them, as the
// joining kernel finds this word, which the second launch's first CTA leaves at its end
// (one warp does: the first launch, which cleared the status word, is waited for).  It also
// reports groups that are out of range, which may have no sequence to report them.
constexpr int kGroupsFall = 32;  // place of the word behind the status word
__device__ __forceinline__ void attn_groups_end(const AttnParams& p) {
  const int lane = threadIdx.x & 31;
  int fall = 0, bad = 0;
#pragma unroll 2
  for (int i = lane; i < p.n_groups; i += 32) {
    AttnGroup g;
    bad |= !attn_group(p, i, g);
    fall |= g.last < g.first;
  }
  fall = __any_sync(0xffffffffu, fall);
  bad = __any_sync(0xffffffffu, bad);
  if (p.part_first) asm volatile("griddepcontrol.wait;" ::: "memory");
  if (lane) return;
  p.status[kGroupsFall] = fall;
  if (bad) attn_report(p.status);
}
// Keys that new token i sees: the first attn_limit(s, i) of the sequence.
__device__ __forceinline__ int attn_limit(const AttnSeq& s, int i) { return max(0, s.len - s.n_q + i + 1); }
// GEN: it sees keys j below that with j >= attn_low or j < sinks (and, in a shared call, the shared ones).
template <bool GEN>
__device__ __forceinline__ int attn_limit(const AttnParams& p, const AttnSeq& s, int i) {
  return GEN && p.phase == kPrefix ? s.len : attn_limit(s, i);
}
__device__ __forceinline__ int attn_low(const AttnParams& p, const AttnSeq& s, int limit) { return max(s.lo, limit - p.window); }

// The keys of a piece whose rows have limits from `first` to `last`, counted
// without the gap between the first keys and the window: place v is key v below
// sinks_pad and key v + delta from there on.  Keys [low, ..) and [0, sinks) count, the
// other places up to n are there for the alignment.  With a gap (delta > 0), every row
// of the piece sees all of the first keys.
struct AttnSpan {
  int low, delta, n;
};
__device__ __forceinline__ AttnSpan attn_span(const AttnParams& p, const AttnSeq& s, int first, int last) {
  AttnSpan a;
  a.low = attn_low(p, s, first);
  const int before = a.low - p.sinks_pad;
  a.delta = before > 0 ? before & -p.gran : 0;
  a.n = max(0, last - a.delta);
  return a;
}
__device__ __forceinline__ int attn_key(int v, int sinks_pad, int delta) { return v < sinks_pad ? v : v + delta; }
// Splits that the keys of a sequence have in this launch (of one that has rows).  Of the
// tensor-core kernel's pieces this is a bound: those beyond a piece's keys are empty.
__device__ __forceinline__ int attn_splits(const AttnParams& p, const AttnSeq& s) {
  if (p.n_split == 1) return 1;
  int n;
  if (p.tc) {
    const int64_t most = (int64_t)p.window + p.piece_toks + p.sinks_pad + p.gran;
    n = (int)min((int64_t)(s.len - (s.lo & -p.gran)), most);
  } else {
    n = attn_span(p, s, attn_limit<true>(p, s, 0), attn_limit<true>(p, s, s.n_q - 1)).n;
  }
  return max(1, (n + p.split_keys - 1) / p.split_keys);
}

// Page of key j; an id out of range is recorded and page 0 read in its place.
__device__ __forceinline__ int attn_page(const AttnParams& p, int b, int j) {
  const int page = __ldg(p.table + b * p.ld_table + (j >> p.shift));
  if ((uint32_t)page < (uint32_t)p.n_pages) return page;
  if (!p.clear && p.status) attn_report(p.status);
  return 0;
}
// Row of key j in the cache (in units of head_dim elements).
__device__ __forceinline__ int64_t attn_page_row(const AttnParams& p, int b, int h, int j) {
  return (((int64_t)attn_page(p, b, j) * p.n_kv_heads + h) << p.shift) + (j & ((1 << p.shift) - 1));
}

// Row of a query in the partial results.
__device__ __forceinline__ int64_t attn_part_row(const AttnParams& p, const AttnSeq& s, int tok, int head) {
  return (int64_t)(s.q0 + tok) * p.n_heads + head;
}

// A key that a row does not see has the weight 0 there, but the row's piece
// multiplies it with V all the same, and 0 * NaN or 0 * inf is NaN.  Such a row
// is done again by attend_row; a row that is NaN by a key it sees, by its own Q
// or by its sum of weights (hidden keys add exactly 0 to that) is right as it
// is.  The keys in question are few: a piece's keys end at the limit of its last
// row, and its rows are those of one multiple of kTcAttnRows (the decode
// kernel's are fewer than that altogether).
__device__ __forceinline__ int attn_reach(const AttnParams& p, const AttnSeq& s, int row) {
  return attn_limit(s, min(row | (kTcAttnRows - 1), s.n_q * p.group - 1) / p.group);
}
// With a window, the keys below the row's own that other rows of its piece see hide there too: from here on.
__device__ __forceinline__ int attn_from(const AttnParams& p, const AttnSeq& s, int row) {
  return attn_low(p, s, attn_limit(s, (row & ~(kTcAttnRows - 1)) / p.group));
}
// The last of the keys [from, to) whose V, or V scale, is not finite; -1 without
// one.  By a warp, a key a lane.
template <int D>
__device__ __noinline__ int attn_last_nonfinite(const AttnParams& p, const AttnSeq& s, int b, int h, int from, int to) {
  const bool codes = p.table && p.type != WAL_KV_BF16;
  int last = -1;
#pragma unroll 1
  for (int j = from + (int)(threadIdx.x & 31); j < to; j += 32) {
    const int64_t row = p.table ? attn_page_row(p, b, h, j) : 0;
    const char* v = static_cast<const char*>(p.v);
    if (!p.table)
      v += ((s.q0 + j) * p.ldv + h * D) * 2;
    else
      v += row * (codes ? D : 2 * D);
    // the largest magnitude of the row's halves or, in e4m3, bytes; int8 codes are all finite
    uint32_t top = 0;
    if (!codes || p.type == WAL_KV_E4M3) {
      const uint32_t mask = codes ? 0x7F7F7F7Fu : 0x7FFF7FFFu;
#pragma unroll 4
      for (int i = 0; i < (codes ? D / 16 : D / 8); ++i) {
        const uint4 u = __ldg(reinterpret_cast<const uint4*>(v) + i);
        const uint32_t x = codes ? __vmaxu4(__vmaxu4(u.x & mask, u.y & mask), __vmaxu4(u.z & mask, u.w & mask))
                                 : __vmaxu2(__vmaxu2(u.x & mask, u.y & mask), __vmaxu2(u.z & mask, u.w & mask));
        top = codes ? __vmaxu4(top, x) : __vmaxu2(top, x);
      }
    }
    bool bad;
    if (codes)
      bad = !(fabsf(p.vs[row]) < INFINITY) || __vcmpeq4(top, 0x7F7F7F7Fu) != 0;
    else
      bad = (top & 0xFFFFu) >= 0x7F80u || (top >> 16) >= 0x7F80u;
    if (bad) last = j;
  }
  return __reduce_max_sync(0xffffffffu, last);
}

// One row by one warp, in fp32: lane i holds columns [i * VPL, (i + 1) * VPL).
// Only visible keys are touched, and a non-finite one among them acts as in the
// formula: a NaN or +inf score, or scores that are all -inf, give NaN; so does
// a NaN in V, or an infinity there under the weight 0; under another weight the
// infinity stays one.  Nothing can change a row of NaN, so it ends there.  Slow,
// a key after the other (0.5 us each): a prompt of 8192, 32 q heads of 128 on 8, whose
// last V is NaN takes 137 ms (0.44 without it), all for the rows of the last pieces.
template <int D, bool GEN = false>
__device__ __noinline__ void attend_row(const AttnParams& p, const AttnSeq& s, int b, int head, int tok) {
  constexpr int VPL = D / 32;
  const int lane = threadIdx.x & 31, h = head / p.group;
  const int lim = attn_limit(s, tok), low = GEN ? lim - p.window : 0;
  const int own = b;
  float q[VPL], acc[VPL];
  const uint16_t* qr = p.Q + (s.q0 + tok) * p.ldq + head * D + lane * VPL;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    q[i] = __uint_as_float((uint32_t)qr[i] << 16);
    acc[i] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
#pragma unroll 1
  for (int j = 0; j < lim; ++j) {
    if (GEN && j >= p.sinks && j < low) j = low;
    if (GEN) b = j < s.lo ? s.head : own;
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
    if ((j & 15) == 0) {
      bool dead = true;
#pragma unroll
      for (int i = 0; i < VPL; ++i) dead &= acc[i] != acc[i];
      if (__all_sync(0xffffffffu, dead || l != l)) break;
    }
  }
  uint16_t* o = p.O + (s.q0 + tok) * p.ldo + head * D + lane * VPL;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const float y = lim == 0 ? 0.f : acc[i] / l;
    o[i] = (uint16_t)(dev::float2_to_bf16x2(y, 0.f) & 0xFFFFu);
  }
}

}  // namespace wal
