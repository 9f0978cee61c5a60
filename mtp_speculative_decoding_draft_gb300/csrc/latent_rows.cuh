// Attention of one (row, head) a warp, the softmax online: what the latent
// kernels begin with.
#pragma once

#include "latent.cuh"

namespace mtp {

// KEY(j, e): element e of key j;  VAL(j, e): element e of value j
template <int DK, int DV, class Key, class Val>
__device__ __forceinline__ void attend_row(const PagedArgs &p, const PagedSeq &s, int row, int h, const uint16_t *q, int dk,
                                           int dv, Key key, Val val) {
  const int lane = threadIdx.x & 31;
  float x[DK / 32], o[DV / 32];
#pragma unroll
  for (int e = 0; e < DK / 32; ++e) x[e] = lane + 32 * e < dk ? bf16_lo(q[lane + 32 * e]) : 0.f;
#pragma unroll
  for (int e = 0; e < DV / 32; ++e) o[e] = 0.f;
  const int t = row - s.row0, pos = s.ctx + t, hi = min(pos + 1, p.cap);
  const int lo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < hi; ++j) {
    if (j < lo && j >= p.sinks) {
      j = lo - 1;
      continue;
    }
    float d = 0.f;
#pragma unroll
    for (int e = 0; e < DK / 32; ++e)
      if (lane + 32 * e < dk) d = fmaf(x[e], bf16_lo(key(j, lane + 32 * e)), d);
    d = warp_sum(d) * p.scale_log2;
    const float n = fmaxf(m, d), f = m == -INFINITY ? 0.f : exp2f(m - n), w = d == -INFINITY ? 0.f : exp2f(d - n);
    l = l * f + w;
#pragma unroll
    for (int e = 0; e < DV / 32; ++e)
      if (lane + 32 * e < dv) o[e] = fmaf(w, bf16_lo(val(j, lane + 32 * e)), o[e] * f);
    m = n;
  }
  // keys that the row sees past the cache (a sink ahead of a window) end with hi
  for (int e = 0; e < DV / 32; ++e)
    if (lane + 32 * e < dv)
      static_cast<__nv_bfloat16 *>(p.out)[(long long)row * p.ldo + h * dv + lane + 32 * e] =
          __float2bfloat16_rn(o[e] * paged_inverse(l));
  if (lane == 0 && p.lse) p.lse[(size_t)row * p.Hq + h] = paged_lse(m, l);
}

// The sequence of a row; false if it has none, or if the row starts decrease.
// Executed by all threads of the block.
__device__ __forceinline__ bool find_row(const PagedArgs &p, int row, int *b, PagedSeq *s) {
  bool back = false;
  for (int i = threadIdx.x; i < p.B; i += blockDim.x) paged_seq(p, i, blockIdx.x == 0, &back);
  if (__syncthreads_or(back)) return false;
  *b = starts_upto(p.row_start, p.B, row, threadIdx.x & 31) - 1;
  if (*b < 0) return false;
  *s = paged_seq(p, *b, false);
  return row >= s->row0 && row < s->row0 + s->n;
}

}  // namespace mtp
