// The plan of a serving step, from the requests' lengths: pages taken from and
// given back to a free list, the page table, and the place of every new token.
//
// Sequences take pages and rows in order, so everything is a prefix sum over them.
// It moves a few bytes for each sequence and row and is bound by the chain of its
// loads and barriers.  One CTA does a small step, a cluster of eight a large one:
// each CTA sums its share of the sequences, the totals go round over distributed
// shared memory, and then pages and rows are dealt out evenly, each finding its
// sequence by bisection of the sums.
#include "wal_kv.h"

#include <algorithm>
#include <cooperative_groups.h>

namespace wal {

namespace {

namespace cg = cooperative_groups;

constexpr int kCluster = 8;
constexpr int kMaxThreads = 1024;
constexpr uint32_t kMost = 0x7FFFFFFFu;  // sums stop here; what they are compared with is below

struct PlanParams {
  const int32_t* n_new;
  const int32_t* kv_len;
  int32_t* kv_len_out;
  int32_t* table;
  int32_t* free_pages;
  const int32_t* n_free;
  int32_t* n_free_out;
  int32_t* q_start;
  int32_t* positions;
  int32_t* slots;
  int32_t* status;  // NULL: nothing is recorded
  int64_t ld_table;
  int B, T, shift, n_pages, max_kv;
  int per;         // sequences of a CTA
  bool starts;     // q_start fits in shared memory
};

// What a sequence asks for: rows, pages to take, pages to give back.  One whose
// values are out of range asks for nothing.
struct Ask {
  uint32_t rows, take, give;
  int len, n_new;
  bool bad;
};
__device__ __forceinline__ uint32_t pages_of(int n, int shift) { return ((uint32_t)n + (1u << shift) - 1) >> shift; }
__device__ __forceinline__ Ask ask(const PlanParams& p, int b) {
  Ask a = {};
  a.len = p.kv_len[b];
  a.n_new = p.n_new[b];
  const int64_t after = (int64_t)a.len + a.n_new;
  a.bad = a.len < 0 || a.len > p.max_kv || after < 0 || after > p.max_kv;
  if (a.bad) {
    a.n_new = 0;
    return a;
  }
  const uint32_t had = pages_of(a.len, p.shift), has = pages_of((int)after, p.shift);
  a.rows = (uint32_t)max(a.n_new, 0);
  a.take = has > had ? has - had : 0;
  a.give = had > has ? had - has : 0;
  return a;
}

struct Sums {
  uint32_t v[3];  // rows, pages to take, pages to give back
};
__device__ __forceinline__ uint32_t add(uint32_t a, uint32_t b) { return min(a + b, kMost); }

// The last place i of sums[0 .. n) (not falling, the first is 0) with sums[i] <= v.
__device__ __forceinline__ int find(const uint32_t* sums, int n, uint32_t v) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sums[mid] <= v)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

template <int C>
__global__ void __launch_bounds__(kMaxThreads) plan_kernel(const __grid_constant__ PlanParams p) {
  extern __shared__ uint32_t dyn[];
  __shared__ Sums s_warp[32], s_total, s_in;
  __shared__ int s_bad;
  uint32_t *s_rows = dyn, *s_take = dyn + p.per, *s_give = dyn + 2 * p.per, *s_len = dyn + 3 * p.per, *s_start = dyn + 4 * p.per;
  const cg::cluster_group cluster = cg::this_cluster();
  auto barrier = [&] {
    if (C > 1)
      cluster.sync();
    else
      __syncthreads();
  };
  auto of = [&](auto* v, int rank) { return C > 1 ? cluster.map_shared_rank(v, rank) : v; };
  const int rank = C > 1 ? (int)cluster.block_rank() : 0;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, n_warps = blockDim.x >> 5;
  const int lo = min(p.B, rank * p.per), mine = min(p.B, lo + p.per) - lo;
  if (tid == 0) {
    s_bad = 0;
    s_in = {};
  }
  const int n_free = *p.n_free;
  bool bad = false;

  // sums over this CTA's sequences: what comes before each of them
  Sums carry = {};
  for (int i0 = 0; i0 < mine; i0 += blockDim.x) {
    const int i = i0 + tid;
    Ask a = {};
    if (i < mine) {
      a = ask(p, lo + i);
      bad |= a.bad;
    }
    const Sums own = {{a.rows, a.take, a.give}};
    Sums sum = own;
#pragma unroll
    for (int o = 1; o < 32; o *= 2)
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const uint32_t up = __shfl_up_sync(0xffffffffu, sum.v[k], o);
        if (lane >= o) sum.v[k] = add(sum.v[k], up);
      }
    if (lane == 31) s_warp[warp] = sum;
    __syncthreads();
    Sums before = carry, all = carry;
    for (int w = 0; w < n_warps; ++w)
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        if (w == warp) before.v[k] = all.v[k];
        all.v[k] = add(all.v[k], s_warp[w].v[k]);
      }
    carry = all;
    // what comes before is the inclusive sum of the lane below
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const uint32_t up = __shfl_up_sync(0xffffffffu, sum.v[k], 1);
      before.v[k] = add(before.v[k], lane ? up : 0);
    }
    if (i < mine) {
      s_rows[i] = before.v[0];
      s_take[i] = before.v[1];
      s_give[i] = before.v[2];
      s_len[i] = (uint32_t)a.len;
    }
    __syncthreads();
  }
  if (tid == 0) s_total = carry;
  barrier();
  Sums base = {}, total = {};
#pragma unroll
  for (int r = 0; r < C; ++r) {
    const Sums t = *of(&s_total, r);
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      if (r == rank) base.v[k] = total.v[k];
      total.v[k] = add(total.v[k], t.v[k]);
    }
  }
  // who goes in: all, or the sequences before the first that finds too little
  const bool sound = n_free >= 0 && n_free <= p.n_pages && total.v[2] <= (uint32_t)(p.n_pages - n_free);
  const uint32_t held = sound ? (uint32_t)n_free + total.v[2] : 0;
  uint32_t rows = total.v[0], take = total.v[1];
  if (!sound || rows > (uint32_t)p.T || take > held) {
    bad = true;
    uint32_t most_rows = 0, most_take = 0;
    if (sound)
      for (int i = tid; i < mine; i += blockDim.x) {
        const Ask a = ask(p, lo + i);
        const uint32_t r = add(add(base.v[0], s_rows[i]), a.rows), t = add(add(base.v[1], s_take[i]), a.take);
        if (r <= (uint32_t)p.T && t <= held) {
          most_rows = max(most_rows, r);
          most_take = max(most_take, t);
        }
      }
    atomicMax(&s_in.v[0], most_rows);
    atomicMax(&s_in.v[1], most_take);
    barrier();
    rows = take = 0;
#pragma unroll
    for (int r = 0; r < C; ++r) {
      const Sums t = *of(&s_in, r);
      rows = max(rows, t.v[0]);
      take = max(take, t.v[1]);
    }
  }
  // Sequences that go in are those whose rows end at `rows` at most.  Starts and lengths, and given pages on top of the list
  const uint32_t give = sound ? carry.v[2] : 0;
  for (int i = tid; i < mine; i += blockDim.x) {
    const uint32_t start = add(base.v[0], s_rows[i]);
    const int b = lo + i, m = p.n_new[b];
    const uint32_t want = i + 1 < mine ? s_rows[i + 1] - s_rows[i] : carry.v[0] - s_rows[i];
    const bool trim = m < 0 && sound && (int64_t)s_len[i] + m >= 0 && (int)s_len[i] >= 0 && (int)s_len[i] <= p.max_kv;
    const int len = (int)s_len[i];
    int after = trim ? len + m : len;
    if (want && start < rows && want <= rows - start) after = len + (int)want;
    p.kv_len_out[b] = after;
    const uint32_t s = min(start, rows);
    p.q_start[b] = (int)s;
    if (p.starts) for (int r = 0; r < C; ++r) of(s_start, r)[b] = s;
  }
  if (rank == C - 1 && tid == 0) p.q_start[p.B] = (int)rows;
  for (uint32_t k = tid; k < give; k += blockDim.x) {
    const int i = find(s_give, mine, k);
    const uint32_t end = i + 1 < mine ? s_give[i + 1] : carry.v[2];
    const uint32_t at = pages_of((int)s_len[i], p.shift) - (end - k);
    const int page = p.table[(lo + i) * p.ld_table + at];
    bad |= (uint32_t)page >= (uint32_t)p.n_pages;
    p.free_pages[(uint32_t)n_free + base.v[2] + k] = page;
  }
  if (total.v[2]) barrier();
  // taken pages, from the top of the list
  const uint32_t taken = take > base.v[1] ? min(take - base.v[1], carry.v[1]) : 0;
  for (uint32_t k = tid; k < taken; k += blockDim.x) {
    const int i = find(s_take, mine, k);
    const int page = __ldcg(p.free_pages + (held - 1 - base.v[1] - k));
    bad |= (uint32_t)page >= (uint32_t)p.n_pages;
    p.table[(lo + i) * p.ld_table + pages_of((int)s_len[i], p.shift) + (k - s_take[i])] = page;
  }
  barrier();
  // rows
  for (int t = rank * blockDim.x + tid; t < p.T; t += C * blockDim.x) {
    int pos = 0, slot = -1;
    if ((uint32_t)t < rows) {
      int b;
      uint32_t start, end;
      if (p.starts) {
        b = find(s_start, p.B, (uint32_t)t);
        start = s_start[b];
        end = b + 1 < p.B ? s_start[b + 1] : rows;
      } else {
        int l = 0, h = p.B;
        while (h - l > 1) {
          const int mid = (l + h) >> 1;
          if (__ldcg(p.q_start + mid) <= t) l = mid; else h = mid;
        }
        b = l;
        start = (uint32_t)__ldcg(p.q_start + b);
        end = (uint32_t)__ldcg(p.q_start + b + 1);
      }
      pos = __ldcg(p.kv_len_out + b) - (int)(end - start) + (t - (int)start);
      const int page = __ldcg(p.table + b * p.ld_table + (pos >> p.shift));
      if ((uint32_t)page < (uint32_t)p.n_pages)
        slot = (page << p.shift) + (pos & ((1 << p.shift) - 1));
      else
        bad = true;
    }
    p.positions[t] = pos;
    p.slots[t] = slot;
  }
  if (bad) atomicOr(of(&s_bad, 0), 1);
  barrier();
  if (rank == 0 && tid == 0) {
    *p.n_free_out = sound ? (int)(held - take) : n_free;
    if (p.status) *p.status = s_bad ? (int32_t)WAL_ERR_ARG : 0;
  }
}

constexpr int kSmall = 1024;    // sequences, and
constexpr int kSmallRows = 8192;  // rows of a step that one CTA does
constexpr int kStarts = 24576;  // sequences whose starts fit in shared memory beside the sums

}  // namespace
}  // namespace wal

using namespace wal;

extern "C" int wal_kv_plan(const wal_kv_cache* cache, const int32_t* n_new, const int32_t* kv_len, int B, int32_t* table, int ld_table,
                           int max_kv, int32_t* free_pages, const int32_t* n_free, int T, int32_t* q_start, int32_t* positions,
                           int32_t* slots, int32_t* kv_len_out, int32_t* n_free_out, void* ws, size_t ws_bytes, wal_stream_t stream) {
  int st = check_cache(cache);
  if (st) return st;
  if (B < 1 || B > 65535 || T < 0 || max_kv < 1) return fail(WAL_ERR_SHAPE, "1 <= B <= 65535, T >= 0 and max_kv >= 1");
  if (T == 0x7FFFFFFF) return fail(WAL_ERR_UNSUPPORTED, "T must be below 2^31 - 1");
  if (max_kv > 1 << 30) return fail(WAL_ERR_UNSUPPORTED, "at most 2^30 tokens a sequence");
  for (const void* a : {(const void*)n_new, (const void*)kv_len, (const void*)table, (const void*)free_pages, (const void*)n_free,
                        (const void*)q_start, (const void*)kv_len_out, (const void*)n_free_out})
    if (!a || misaligned(a, 4)) return fail(WAL_ERR_ARG, "every array is required, 4-byte aligned");
  if ((T > 0 && (!positions || !slots)) || misaligned(positions, 4) || misaligned(slots, 4))
    return fail(WAL_ERR_ARG, "positions and slots are required, 4-byte aligned");
  if (kv_len_out == n_new || n_free == kv_len_out || n_free_out == n_new || n_free_out == kv_len)
    return fail(WAL_ERR_ARG, "only kv_len and n_free may be written in place");
  if ((int64_t)ld_table * cache->page_size < max_kv) return fail(WAL_ERR_ARG, "ld_table pages must cover max_kv tokens");
  if (ws && ws_bytes < kStatusWs) return fail(WAL_ERR_WORKSPACE, "a workspace has at least 512 bytes");
  int dev = 0;
  if ((st = current_device(&dev))) return st;
  PlanParams p = {};
  p.n_new = n_new; p.kv_len = kv_len; p.kv_len_out = kv_len_out;
  p.table = table; p.ld_table = ld_table;
  p.free_pages = free_pages; p.n_free = n_free; p.n_free_out = n_free_out;
  p.q_start = q_start; p.positions = positions; p.slots = slots;
  p.status = status_word(ws);
  p.B = B; p.T = T; p.max_kv = max_kv;
  p.shift = log2_of(cache->page_size); p.n_pages = cache->n_pages;
  p.starts = B <= kStarts;
  const bool small = B <= kSmall && T <= kSmallRows;
  p.per = small ? B : (B + kCluster - 1) / kCluster;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(small ? 1 : kCluster);
  const int most = std::min(kMaxThreads, (std::max(B, T) + 31) / 32 * 32);
  cfg.blockDim = dim3(small ? most : kMaxThreads);
  cfg.dynamicSmemBytes = (size_t)4 * (4 * p.per + (p.starts ? B : 0));
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {(unsigned)kCluster, 1, 1};
  cudaError_t e;
  if (small) {
    e = cudaLaunchKernelEx(&cfg, plan_kernel<1>, p);
  } else {
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaFuncSetAttribute(plan_kernel<kCluster>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)cfg.dynamicSmemBytes);
    if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, plan_kernel<kCluster>, p);
  }
  if (e != cudaSuccess) return fail(WAL_ERR_CUDA, std::string("plan_kernel launch: ") + cudaGetErrorString(e));
  return WAL_OK;
}
