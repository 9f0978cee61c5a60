// Interface of the tensor-core kernel over the paged cache (paged_attn_tc.cu).
#pragma once

#include <cuda.h>

#include "paged.cuh"

namespace mtp {

constexpr int kPagedTcRows = 256;  // packed query rows of a block at most

struct PagedTcParams {
  CUtensorMap mk, mv;  // the pools as [n_pages * Hkv * page, Dh] bf16
  CUtensorMap mq;      // the queries as [n_rows, Hq, Dh], boxes of a group's tokens x G x 64
  PagedArgs a;
};

// Queries as a 3-D map, boxes of `tokens` x G x 64 elements, 128-byte swizzle (tc.cu).
bool make_query_map(CUtensorMap *m, const void *q, int Dh, int Hq, int n_rows, long long ldq, int G, int tokens);
cudaError_t paged_tc_set_attributes();
cudaError_t launch_paged_attn_tc(const PagedTcParams &sp, int ctas, cudaStream_t s, bool pdl);

}  // namespace mtp
