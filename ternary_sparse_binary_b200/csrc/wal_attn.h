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
  int32_t* status;
};

// Sequence b as its index arrays give it; n_q = 0 where they are out of range.
struct AttnSeq {
  int q0, n_q, len;
  bool bad;
};
__device__ __forceinline__ AttnSeq attn_seq(const AttnParams& p, int b) {
  const int q0 = p.q_start[b], q1 = p.q_start[b + 1];
  AttnSeq s = {0, 0, 0, true};
  if (q0 < 0 || q1 < q0 || q1 > p.T || q1 - q0 > p.max_q) return s;
  const int len = p.kv_len ? p.kv_len[b] : q1 - q0;
  if (len < 0 || len > p.max_kv) return s;
  s.q0 = q0;
  s.n_q = q1 - q0;
  s.len = len;
  s.bad = false;
  return s;
}
// Keys that new token i sees: the first attn_limit(s, i) of the sequence.
__device__ __forceinline__ int attn_limit(const AttnSeq& s, int i) { return max(0, s.len - s.n_q + i + 1); }

// Row of key j (in units of head_dim elements) in the cache; a page id out of
// range is recorded and page 0 read in its place.
__device__ __forceinline__ int64_t attn_page_row(const AttnParams& p, int b, int h, int j) {
  int page = __ldg(p.table + b * p.ld_table + (j >> p.shift));
  if ((uint32_t)page >= (uint32_t)p.n_pages) {
    atomicExch(p.status, (int32_t)WAL_ERR_ARG);
    page = 0;
  }
  return (((int64_t)page * p.n_kv_heads + h) << p.shift) + (j & ((1 << p.shift) - 1));
}

}  // namespace wal
