// The plan of a serving step, from the requests' lengths: pages taken from and
// given back to a free list, the page table, and the place of every new token.
//
// Sequences take pages and rows in order, so everything is a prefix sum over them.
// It moves a few bytes for each sequence and row and is bound by the chain of its
// loads and barriers: 2.9 us of a graph for 25 sequences of a token each, 15.4 for 1500
// with 70000 rows and 8000 pages taken or given back.  One CTA does a small step, a
// cluster of eight a large one (of sixteen: 13.6 us, but not every device has it): each
// CTA sums its share of the sequences, the totals go round over distributed shared
// memory, and then pages and rows are dealt out evenly to warps, which find their
// sequences in the sums.
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
  bool starts;     // every sequence's place fits in shared memory
  bool wide;       // positions and slots are 16-byte aligned
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

// The sums up to and with each lane's.
__device__ __forceinline__ Sums warp_sums(Sums s, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o *= 2)
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const uint32_t up = __shfl_up_sync(0xffffffffu, s.v[k], o);
      if (lane >= o) s.v[k] = add(s.v[k], up);
    }
  return s;
}

// For each of a lane's four values the last place i of [0, n) with at(i) <= v[e]; at does
// not fall, and at(0) is 0.  The warp's values lie between `first` and `last`: it looks
// for the places of these two with a probe a lane, then each lane bisects between them,
// all in the same steps.  No load is behind a branch: a step is one latency.
constexpr int kDeal = 4;
template <typename At>
__device__ __forceinline__ void find(int n, uint32_t first, uint32_t last, int lane, const uint32_t (&v)[kDeal], int (&place)[kDeal], At at) {
  int lo = 0, hi = 0;
  for (int size = n; size > 1;) {
    const int step = (size + 31) >> 5, i = lo + lane * step, j = hi + lane * step;
    const uint32_t ai = at(min(i, n - 1)), aj = at(min(j, n - 1));
    lo += (__popc(__ballot_sync(0xffffffffu, lane * step < size && i < n && ai <= first)) - 1) * step;
    hi += (__popc(__ballot_sync(0xffffffffu, lane * step < size && j < n && aj <= last)) - 1) * step;
    size = step;
  }
  int w = lo, x = lo, y = lo, z = lo;
#pragma unroll 1
  for (int step = hi > lo ? 1 << (31 - __clz(hi - lo)) : 0; step > 0; step >>= 1) {
    const uint32_t aw = at(min(w + step, hi)), ax = at(min(x + step, hi)), ay = at(min(y + step, hi)), az = at(min(z + step, hi));
    if (w + step <= hi && aw <= v[0]) w += step;
    if (x + step <= hi && ax <= v[1]) x += step;
    if (y + step <= hi && ay <= v[2]) y += step;
    if (z + step <= hi && az <= v[3]) z += step;
  }
  place[0] = w;
  place[1] = x;
  place[2] = y;
  place[3] = z;
}

// Where a sequence's rows begin, and what makes a row's number its position.
struct Place {
  uint32_t start;
  int to_position;
};

template <int C>
__global__ void __launch_bounds__(kMaxThreads) plan_kernel(const __grid_constant__ PlanParams p) {
  extern __shared__ __align__(8) uint32_t dyn[];
  __shared__ Sums s_warp[32], s_total[C], s_in;
  __shared__ int s_bad;
  Place* s_place = reinterpret_cast<Place*>(dyn);  // of every sequence
  uint32_t* s_rows = dyn + (p.starts ? 2 * p.B : 0);  // of this CTA's
  uint32_t *s_take = s_rows + p.per, *s_give = s_take + p.per, *s_len = s_give + p.per, *s_new = s_len + p.per;
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
  if (C > 1) cluster.barrier_arrive();
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
    const Sums sum = warp_sums({{a.rows, a.take, a.give}}, lane);
    if (lane == 31) s_warp[warp] = sum;
    __syncthreads();
    const Sums warps = warp_sums(lane < n_warps ? s_warp[lane] : Sums{}, lane);
    // what comes before: the chunks before, the warps below, the lanes below
    Sums before;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const uint32_t below = __shfl_sync(0xffffffffu, warps.v[k], (warp - 1) & 31), up = __shfl_up_sync(0xffffffffu, sum.v[k], 1);
      before.v[k] = add(add(carry.v[k], warp ? below : 0), lane ? up : 0);
      carry.v[k] = add(carry.v[k], __shfl_sync(0xffffffffu, warps.v[k], 31));
    }
    if (i < mine) {
      s_rows[i] = before.v[0];
      s_take[i] = before.v[1];
      s_give[i] = before.v[2];
      s_len[i] = (uint32_t)a.len;
      s_new[i] = (uint32_t)a.n_new;
    }
    __syncthreads();
  }
  Sums base = {}, total = carry;
  if (C > 1) {  // the CTAs' totals go round
    cluster.barrier_wait();
    if (tid < C) *of(s_total + rank, tid) = carry;
    barrier();
    const Sums sum = warp_sums(lane < C ? s_total[lane] : Sums{}, lane);
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const uint32_t below = __shfl_sync(0xffffffffu, sum.v[k], (rank - 1) & 31);
      base.v[k] = rank ? below : 0;
      total.v[k] = __shfl_sync(0xffffffffu, sum.v[k], 31);
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
    const int b = lo + i, len = (int)s_len[i], m = (int)s_new[i];  // 0 new tokens where a value is out of range
    int after = m < 0 && sound ? len + m : len;
    if (m > 0 && start < rows && (uint32_t)m <= rows - start) after = len + m;
    p.kv_len_out[b] = after;
    const uint32_t s = min(start, rows);
    p.q_start[b] = (int)s;
    if (p.starts) {
      const Place place = {s, len - (int)s};
      for (int r = 0; r < C; ++r) of(s_place, r)[b] = place;
    }
  }
  if (rank == C - 1 && tid == 0) p.q_start[p.B] = (int)rows;
  // Pages of this CTA's sequences, a run of 32 * kDeal a warp
  auto deal = [&](const uint32_t* sums, uint32_t n, auto load, auto store) {
    for (uint32_t k0 = warp * 32 * kDeal; k0 < n; k0 += n_warps * 32 * kDeal) {
      uint32_t k[kDeal];
      int i[kDeal], page[kDeal];
#pragma unroll
      for (int e = 0; e < kDeal; ++e) k[e] = min(k0 + 32 * e + lane, n - 1);
      find(mine, k0, min(k0 + 32 * kDeal, n) - 1, lane, k, i, [&](int j) { return sums[j]; });
#pragma unroll
      for (int e = 0; e < kDeal; ++e) page[e] = load(k[e], i[e], k[e] - sums[i[e]]);
#pragma unroll
      for (int e = 0; e < kDeal; ++e) {
        if (k0 + 32 * e + lane >= n) continue;
        bad |= (uint32_t)page[e] >= (uint32_t)p.n_pages;
        store(k[e], i[e], k[e] - sums[i[e]], page[e]);
      }
    }
  };
  // a sequence's entry of the table: `nth` of those behind its pages after (given) or before (taken)
  auto entry = [&](int i, int len, uint32_t nth) { return p.table + (lo + i) * p.ld_table + (pages_of(len, p.shift) + nth); };
  deal(s_give, give, [&](uint32_t, int i, uint32_t nth) { return *entry(i, (int)(s_len[i] + s_new[i]), nth); },
       [&](uint32_t k, int, uint32_t, int page) { p.free_pages[(uint32_t)n_free + base.v[2] + k] = page; });
  if (total.v[2]) barrier();
  // taken from the top of the list
  const uint32_t taken = take > base.v[1] ? min(take - base.v[1], carry.v[1]) : 0;
  deal(s_take, taken, [&](uint32_t k, int, uint32_t) { return __ldcg(p.free_pages + (held - 1 - base.v[1] - k)); },
       [&](uint32_t, int i, uint32_t nth, int page) { *entry(i, (int)s_len[i], nth) = page; });
  barrier();
  // rows, likewise over all CTAs, four neighbours a lane
  for (int64_t t0 = (int64_t)(rank * n_warps + warp) * 32 * kDeal; t0 < p.T; t0 += C * n_warps * 32 * kDeal) {
    const int64_t t = t0 + kDeal * lane;
    int pos[kDeal], slot[kDeal], b[kDeal];
    uint32_t v[kDeal];
#pragma unroll
    for (int e = 0; e < kDeal; ++e) {
      v[e] = min((uint32_t)t + e, rows - 1);
      pos[e] = 0;
      slot[e] = -1;
    }
    if (t0 < rows) {
      const uint32_t last = min((uint32_t)t0 + 32 * kDeal, rows) - 1;
      if (p.starts)
        find(p.B, (uint32_t)t0, last, lane, v, b, [&](int j) { return s_place[j].start; });
      else
        find(p.B, (uint32_t)t0, last, lane, v, b, [&](int j) { return (uint32_t)__ldcg(p.q_start + j); });
#pragma unroll
      for (int e = 0; e < kDeal; ++e) {
        const int at = (int)v[e] + (p.starts ? s_place[b[e]].to_position : __ldcg(p.kv_len_out + b[e]) - __ldcg(p.q_start + b[e] + 1));
        const int page = __ldcg(p.table + b[e] * p.ld_table + (at >> p.shift));
        const bool there = (uint32_t)t + e < rows;
        pos[e] = there ? at : 0;
        slot[e] = there ? page : -1;
      }
#pragma unroll
      for (int e = 0; e < kDeal; ++e) {
        if ((uint32_t)t + e >= rows) continue;
        if ((uint32_t)slot[e] < (uint32_t)p.n_pages) {
          slot[e] = (slot[e] << p.shift) + (pos[e] & ((1 << p.shift) - 1));
        } else {
          slot[e] = -1;
          bad = true;
        }
      }
    }
    if (p.wide && t + kDeal <= p.T) {
      *reinterpret_cast<int4*>(p.positions + t) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      *reinterpret_cast<int4*>(p.slots + t) = make_int4(slot[0], slot[1], slot[2], slot[3]);
    } else {
#pragma unroll
      for (int e = 0; e < kDeal; ++e)
        if (t + e < p.T) {
          p.positions[t + e] = pos[e];
          p.slots[t + e] = slot[e];
        }
    }
  }
  if (bad) atomicOr(of(&s_bad, 0), 1);
  barrier();
  if (rank == 0 && tid == 0) {
    *p.n_free_out = sound ? (int)(held - take) : n_free;
    if (p.status) *p.status = s_bad ? (int32_t)WAL_ERR_ARG : 0;
  }
}

// A step that one CTA does: 256 sequences and 3439 rows 8.3 us against 9.9 of the
// cluster, 100 and 6359 8.2 against 9.3; 1000 and 3781 rows, with many pages given back,
// 15.6 against 12.7.
constexpr int kSmall = 512;       // sequences
constexpr int kSmallRows = 8192;  // rows
constexpr int kStarts = 16384;  // sequences whose places fit in shared memory beside the sums
constexpr int kMostSeqs = 65535;
constexpr int plan_smem(int B, int per) { return 4 * (5 * per + (B <= kStarts ? 2 * B : 0)); }
// The limit that is set is the same for every call: two threads may set it at once.
constexpr int kPlanSmem = std::max(plan_smem(kStarts, kStarts / kCluster), plan_smem(kMostSeqs, (kMostSeqs + kCluster - 1) / kCluster));
static_assert(kPlanSmem <= 230000 && plan_smem(kSmall, kSmall) <= 48 << 10, "above the shared memory of an SM, or of a launch without the attribute");

}  // namespace
}  // namespace wal

using namespace wal;

extern "C" int wal_kv_plan(const wal_kv_cache* cache, const int32_t* n_new, const int32_t* kv_len, int B, int32_t* table, int ld_table,
                           int max_kv, int32_t* free_pages, const int32_t* n_free, int T, int32_t* q_start, int32_t* positions,
                           int32_t* slots, int32_t* kv_len_out, int32_t* n_free_out, void* ws, size_t ws_bytes, wal_stream_t stream) {
  int st = check_cache(cache);
  if (st) return st;
  if (B < 1 || B > kMostSeqs || T < 0 || max_kv < 1) return fail(WAL_ERR_SHAPE, "1 <= B <= 65535, T >= 0 and max_kv >= 1");
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
  p.wide = !misaligned(positions, 16) && !misaligned(slots, 16);
  const bool small = B <= kSmall && T <= kSmallRows;
  p.per = small ? B : (B + kCluster - 1) / kCluster;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(small ? 1 : kCluster);
  const int most = std::min(kMaxThreads, (std::max(B, T) + 31) / 32 * 32);
  cfg.blockDim = dim3(small ? most : kMaxThreads);
  cfg.dynamicSmemBytes = (size_t)plan_smem(B, p.per);
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
    e = cudaFuncSetAttribute(plan_kernel<kCluster>, cudaFuncAttributeMaxDynamicSharedMemorySize, kPlanSmem);
    if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, plan_kernel<kCluster>, p);
  }
  if (e != cudaSuccess) return fail(WAL_ERR_CUDA, std::string("plan_kernel launch: ") + cudaGetErrorString(e));
  return WAL_OK;
}
