// Interface of the tensor-core kernel over the paged cache (paged_attn_tc.cu).
#pragma once

#include <cuda.h>

#include "paged.cuh"

namespace mtp {

constexpr int kPagedMaxCtas = 160;  // CTAs (SMs) that the workspace has places for
constexpr int kPagedTcRows = 256;  // packed query rows of a block at most

// One item of the plan: tokens t0 .. of sequence b at kv head h, `count` key tiles
// behind `first` tiles of the line (count 0: a gap).
struct alignas(16) PagedItem {
  int b, h, t0, count;
  int row0, n, ctx, pad;
  long long first, pad2;
};

// Where a CTA's share starts, in one piece: its first item (number i), the tiles
// [.., end) of the line that it takes up to, and the tiles of a share.
struct alignas(16) PagedStart {
  PagedItem item;
  long long end, per;
  int i, pad[3];
};

struct PagedTcParams {
  CUtensorMap mk, mv;  // the pools as [n_pages * Hkv * page, Dh] bf16
  CUtensorMap mq;      // the queries as [n_rows, Hq, Dh], boxes of a group's tokens x G x 64
  PagedArgs a;
  int *blocks;        // [B + 1] blocks of the sequences before b
  PagedStart *start;  // [CTAs]
  PagedItem *items;   // the line's items
  int item_cost;      // tiles that an item counts for besides its own
  int n_items;        // places of the line
  int shares;         // CTAs (or pairs) of the call
  int small;          // no plan was made: plan_share
  int rope;           // (latent attention) elements of the shared key part, 32 or 64
};

// A share's first items, copied into shared memory: a step to the next item costs two
// round trips of L2 otherwise, with every warp waiting.
constexpr int kNearItems = 16;

// Walks a share's items in the plan's order, one segment at a time; the interface
// of PagedWalk.  On the line an item is item_cost tiles, which stand for what a
// segment costs besides its tiles (queries, first scores, output), then its tiles.
template <int TK, bool NEAR = false>
struct PlanWalk {
  const PagedTcParams &sp;
  const PagedArgs &p;
  long long first, end, per;  // where the item and the share's end lie on the line
  int i, b, h, t0;
  PagedSeq s;
  PagedRange r;
  int i0, i1;
  const PagedItem *near;  // items base .. base + kNearItems - 1
  int base;

  __device__ __forceinline__ explicit PlanWalk(const PagedTcParams &x, int share, const PagedItem *copies = nullptr)
      : sp(x), p(x.a), i0(0), i1(0), near(copies) {
    const PagedStart *st = &sp.start[share];
    const longlong2 e = __ldcg(reinterpret_cast<const longlong2 *>(&st->end));
    i = base = __ldcg(&st->i);
    load(&st->item);
    end = e.x;
    per = e.y;
    const long long at = per * (long long)share - first - sp.item_cost;
    if (at + first + sp.item_cost >= end) return;  // no share
    i0 = at > 0 ? (int)at : 0;
    cut();
  }
  // From a start in shared memory (plan_share).
  __device__ __forceinline__ PlanWalk(const PagedTcParams &x, int share, const PagedStart &st, const PagedItem *copies)
      : sp(x), p(x.a), i0(0), i1(0), near(copies) {
    i = base = st.i;
    take(st.item);
    end = st.end;
    per = st.per;
    const long long at = per * (long long)share - first - sp.item_cost;
    if (at + first + sp.item_cost >= end) return;  // no share
    i0 = at > 0 ? (int)at : 0;
    cut();
  }
  __device__ __forceinline__ void load(const PagedItem *it) {
    const int4 x = __ldcg(reinterpret_cast<const int4 *>(&it->b));
    const int4 y = __ldcg(reinterpret_cast<const int4 *>(&it->row0));
    first = __ldcg(&it->first);
    b = x.x;
    h = x.y;
    t0 = x.z;
    s.row0 = y.x;
    s.n = y.y;
    s.ctx = y.z;
    r = paged_range<TK>(p, s, t0, t1());
  }
  __device__ __forceinline__ int t1() const { return min(s.n, t0 + p.tpb); }
  __device__ __forceinline__ bool valid() const { return i0 < i1; }
  __device__ __forceinline__ bool starts() const { return i0 == 0; }
  __device__ __forceinline__ bool ends() const { return i1 == r.count; }
  __device__ __forceinline__ int last_cta() const { return (int)((first + sp.item_cost + r.count - 1) / per); }
  __device__ __forceinline__ void cut() {
    const long long left = end - first - sp.item_cost;
    i1 = left >= r.count ? r.count : left > 0 ? (int)left : 0;
  }
  __device__ __forceinline__ void next() {
    i0 = i1 = 0;
    if (first + sp.item_cost + r.count >= end) return;
    if (NEAR) {
      for (++i; i < base + kNearItems; ++i)
        if (near[i - base].count != 0) {
          take(near[i - base]);
          cut();
          return;
        }
      --i;
    }
    do ++i;
    while ((!NEAR || i < sp.n_items) && __ldcg(&sp.items[i].count) == 0);  // the line goes on: an item follows
    if (NEAR && i >= sp.n_items) return;  // (only if the workspace was overwritten meanwhile)
    load(&sp.items[i]);
    cut();
  }
  __device__ __forceinline__ void take(const PagedItem &it) {
    first = it.first;
    b = it.b;
    h = it.h;
    t0 = it.t0;
    s.row0 = it.row0;
    s.n = it.n;
    s.ctx = it.ctx;
    r = paged_range<TK>(p, s, t0, t1());
  }
  // Executed by the whole CTA (a barrier follows): the copies of share's first items.
  __device__ __forceinline__ static void copy_near(const PagedTcParams &sp, int share, PagedItem *copies) {
    constexpr int kQuads = sizeof(PagedItem) / 16;
    const int k = threadIdx.x / kQuads, e = threadIdx.x % kQuads, at = __ldcg(&sp.start[share].i) + k;
    if (k < kNearItems && at < sp.n_items)
      reinterpret_cast<int4 *>(copies + k)[e] = __ldcg(reinterpret_cast<const int4 *>(sp.items + at) + e);
  }
};

// Inclusive scan over the block's threads; returns the block's sum.
template <int THREADS>
__device__ __forceinline__ long long block_scan(long long v, long long *incl, long long *scratch) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();  // scratch is free again
  if (lane == 31) scratch[warp] = v;
  __syncthreads();
  long long w = lane < THREADS / 32 ? scratch[lane] : 0;  // every warp scans the warps' sums
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += u;
  }
  const long long before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
  *incl = v + (warp > 0 ? before : 0);
  return __shfl_sync(0xffffffffu, w, 31);
}

// The plan of a call with no more items than shares (as far as the host knows), where each
// is a place of its own: every CTA makes it for itself, which takes it about 1.8 us behind
// the wait and not the 5 us of a kernel before it, the start of the next, and the reading
// of its share.
constexpr int kSmallPlan = kPagedMaxCtas;
struct SmallPlan {
  PagedSeq seq[kSmallPlan];
  int blocks[kSmallPlan + 1];
  long long scratch[32];
  PagedItem items[kSmallPlan];
  PagedStart start;
};

// Executed by the whole CTA (THREADS of them, kSmallPlan at least); leaves the share's start
// in plan->start and its first items in near.  The caller's barrier comes before `plan`'s
// memory serves anything else.
template <int TK, int THREADS>
__device__ __forceinline__ void plan_share(const PagedTcParams &sp, int shares, int share, SmallPlan *plan, PagedItem *near) {
  static_assert(THREADS >= kSmallPlan, "a thread an item");
  const PagedArgs &p = sp.a;
  const int tid = threadIdx.x;
  bool back = false;
  long long v = 0, incl;  // blocks in the upper 16 bits, places on the line below
  if (tid < p.B) {
    const PagedSeq s = paged_seq(p, tid, blockIdx.x == 0, &back);
    long long u;
    const long long c = paged_cost<TK>(p, s, &u);
    const int nb = paged_blocks(p, s.n);
    plan->seq[tid] = s;
    v = (long long)nb << 48 | (c + (long long)nb * sp.item_cost) * p.Hkv;
  }
  const long long sum = block_scan<THREADS>(v, &incl, plan->scratch);
  if (tid < p.B) plan->blocks[tid] = (int)((incl - v) >> 48);
  // (the barrier also publishes the blocks)
  const bool none = __syncthreads_or(back);
  const int N = none ? 0 : min((int)(sum >> 48) * p.Hkv, kSmallPlan);
  const long long total = none ? 0 : sum & ((1ll << 48) - 1);
  const long long per = max((long long)sp.a.min_tiles, (total + shares - 1) / shares);
  PagedItem it{};
  if (tid < N) {
    int lo = 0, hi = p.B;  // blocks[lo] * Hkv <= tid < blocks[hi] * Hkv
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (plan->blocks[mid] * p.Hkv <= tid) lo = mid;
      else hi = mid;
    }
    const PagedSeq s = plan->seq[lo];
    const int nb = paged_blocks(p, s.n), off = tid - plan->blocks[lo] * p.Hkv;
    it.b = lo;
    it.h = off / nb;
    it.t0 = (off % nb) * p.tpb;
    it.count = paged_range<TK>(p, s, it.t0, min(s.n, it.t0 + p.tpb)).count;
    it.row0 = s.row0;
    it.n = s.n;
    it.ctx = s.ctx;
  }
  const int len = tid < N ? sp.item_cost + it.count : 0;
  block_scan<THREADS>(len, &incl, plan->scratch);
  it.first = incl - len;
  if (tid < kSmallPlan) plan->items[tid] = it;
  __syncthreads();
  const long long at = per * share, end = min(total, at + per);
  auto item_at = [&](long long x) {  // the last item that starts at or before x
    int lo = 0, hi = max(N, 1);
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (plan->items[mid].first <= x) lo = mid;
      else hi = mid;
    }
    return lo;
  };
  const int lo = item_at(min(at, max(total - 1, 0ll)));
  if (tid == 0) {
    plan->start.item = plan->items[lo];
    plan->start.end = at < total ? end : 0;
    plan->start.per = per;
    plan->start.i = lo;
  }
  if (tid < kNearItems) {
    PagedItem none_left{};
    near[tid] = lo + tid < N ? plan->items[lo + tid] : none_left;
  }
  // more items in one share than near holds: they go where the walk looks for them
  if (at < total && item_at(end - 1) >= lo + kNearItems && tid >= lo + kNearItems && tid < N) sp.items[tid] = it;
  __syncthreads();
}

// Queries as a 3-D map, boxes of `tokens` x G x 64 elements, 128-byte swizzle (tc.cu).
bool make_query_map(CUtensorMap *m, const void *q, int Dh, int Hq, int n_rows, long long ldq, int G, int tokens);
// Rows of `width` elements, ld apart, boxes of box_rows x 64, 128-byte swizzle (tc.cu).
bool make_rows_map(CUtensorMap *m, const void *base, uint64_t width, uint64_t rows, uint64_t ld, uint32_t box_rows);
// [d2, d1, d0] with strides s2, s1 (elements), boxes of b2 x b1 x 64 (tc.cu).
bool make_heads_map(CUtensorMap *m, const void *base, uint64_t d0, uint64_t d1, uint64_t d2, uint64_t s1, uint64_t s2,
                    uint32_t b1, uint32_t b2);
cudaError_t paged_tc_set_attributes();
// tpb: tokens of a block
bool paged_tc_items_ok(int B, int n_rows, int tpb, int Hkv);  // the plan counts items in 31 bits
size_t paged_tc_plan_bytes(int B, int n_rows, int tpb, int Hkv);
void paged_tc_bind_plan(PagedTcParams &sp, char *base);
// Whether every CTA makes the plan for itself.  (Of the places of the line, kPagedMaxCtas
// are for gaps.)
inline void paged_small_plan(PagedTcParams &sp, int shares) {
  sp.shares = shares;
  sp.small = sp.n_items - kPagedMaxCtas <= shares;
}
// The plan of shares for `ctas` CTAs (or pairs), with tiles of TK keys (32, 64 or 128).
template <int TK>
cudaError_t launch_paged_plan(const PagedTcParams &sp, int ctas, cudaStream_t s, bool pdl);
cudaError_t launch_paged_attn_tc(const PagedTcParams &sp, int ctas, cudaStream_t s, bool pdl);

}  // namespace mtp
