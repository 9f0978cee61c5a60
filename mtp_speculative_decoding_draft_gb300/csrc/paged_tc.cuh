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
};

// Queries as a 3-D map, boxes of `tokens` x G x 64 elements, 128-byte swizzle (tc.cu).
bool make_query_map(CUtensorMap *m, const void *q, int Dh, int Hq, int n_rows, long long ldq, int G, int tokens);
cudaError_t paged_tc_set_attributes();
bool paged_tc_items_ok(int B, int n_rows, int G, int Hkv);  // the plan counts items in 31 bits
size_t paged_tc_plan_bytes(int B, int n_rows, int G, int Hkv);
void paged_tc_bind_plan(PagedTcParams &sp, char *base);
cudaError_t launch_paged_attn_tc(const PagedTcParams &sp, int ctas, cudaStream_t s, bool pdl);

}  // namespace mtp
