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
// The plan of shares for `ctas` CTAs (or pairs), with tiles of TK keys (32, 64 or 128).
template <int TK>
cudaError_t launch_paged_plan(const PagedTcParams &sp, int ctas, cudaStream_t s, bool pdl);
cudaError_t launch_paged_attn_tc(const PagedTcParams &sp, int ctas, cudaStream_t s, bool pdl);

}  // namespace mtp
