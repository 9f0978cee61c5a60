// The kernel that joins the partial states of the tensor-core attention kernels
// (paged_attn_tc.cu) in key order.
#pragma once

#include "paged.cuh"

namespace mtp {

// The workspace of `ctas` CTAs' partial states, two blocks of `rows` rows each.
inline size_t up256(size_t x) { return (x + 255) / 256 * 256; }

inline size_t region_bytes(int ctas, int rows, int Dh) {
  return up256((size_t)ctas * sizeof(PagedDesc)) + up256((size_t)ctas * 2 * rows * 2 * 4) +
         up256((size_t)ctas * 2 * rows * Dh * 4);
}

inline void bind_region(PagedArgs &a, char *base, int ctas, int rows) {
  a.desc = reinterpret_cast<PagedDesc *>(base);
  base += up256((size_t)ctas * sizeof(PagedDesc));
  a.part_ml = reinterpret_cast<float *>(base);
  base += up256((size_t)ctas * 2 * rows * 2 * 4);
  a.part_o = reinterpret_cast<float *>(base);
}

// Joins the partial states of a tensor-core kernel's items, of ROWS rows a block.  Its
// blocks start under the attention kernels (one fits beside their CTAs,
// more as those leave); each reads every CTA's description at once, and the warps
// share the rows.
constexpr int kCombineThreads = 256;
constexpr int kMaxDescs = 256;  // CTAs at most

template <int DH, int ROWS>
__global__ void __launch_bounds__(kCombineThreads, 6)
    paged_combine_tc_kernel(const __grid_constant__ PagedArgs p, int ctas) {
  trace_start(kTkPagedCombine);
  constexpr int PER = DH / 32, kBatch = 2, NW = kCombineThreads / 32;
  // a lane's elements: vectors of VEC, 32 VEC apart
  constexpr int VEC = PER < 4 ? PER : 4;
  auto place = [](int lane, int e) { return e / VEC * (32 * VEC) + lane * VEC + e % VEC; };
  __shared__ PagedDesc desc[kMaxDescs];
  __shared__ int before[kMaxDescs + 1], sums[NW];
  __shared__ float part[NW][DH + 2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dep_wait();
  trace_dep(kTkPagedCombine);
  grid_dep_launch();
  // ---- descriptions, and how many rows lie before each
  int rows[kMaxDescs / kCombineThreads], mine = 0;
#pragma unroll
  for (int e = 0; e < kMaxDescs / kCombineThreads; ++e) {
    const int i = tid * (kMaxDescs / kCombineThreads) + e;
    int4 d = make_int4(0, 0, 0, 0);
    if (i < ctas) d = __ldcg(reinterpret_cast<const int4 *>(p.desc + i));
    *reinterpret_cast<int4 *>(&desc[i]) = d;
    rows[e] = d.y;
    mine += d.y;
  }
  int inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) sums[warp] = inc;
  __syncthreads();
  int off = inc - mine;
  for (int w = 0; w < warp; ++w) off += sums[w];
#pragma unroll
  for (int e = 0; e < kMaxDescs / kCombineThreads; ++e) {
    before[tid * (kMaxDescs / kCombineThreads) + e] = off;
    off += rows[e];
  }
  if (tid == kCombineThreads - 1) before[kMaxDescs] = off;
  __syncthreads();

  // ---- rows over warps: with few rows, up to all eight warps of a block take
  // every wpr-th state of one row
  const int total = before[kMaxDescs], blocks = gridDim.x;
  int wpr = NW;
  while (wpr > 1 && (long long)total * wpr > (long long)blocks * NW) wpr >>= 1;
  const int rpb = NW / wpr, q = warp % wpr;
  for (int g0 = blockIdx.x * rpb; g0 < total; g0 += blocks * rpb) {
    const int g = g0 + warp / wpr;
    const bool mine = g < total;
    int lo = 0, hi = kMaxDescs;  // before[lo] <= g < before[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (before[mid] <= min(g, total - 1)) lo = mid;
      else hi = mid;
    }
    const PagedDesc d = desc[lo];
    const int r = g - before[lo], nseg = mine ? d.last_cta - lo + 1 : 0, my = nseg > q ? (nseg - q + wpr - 1) / wpr : 0;
    // this warp's i-th state of the row
    auto seg = [&](int i) {
      const int c = q + i * wpr;
      return ((size_t)(lo + c) * 2 + (c == 0 ? 1 : 0)) * ROWS + r;
    };
    auto stats = [&](int i) { return __ldcg(reinterpret_cast<const float2 *>(p.part_ml + seg(i) * 2)); };
    float v[kBatch][PER];
    auto fetch = [&](int i0) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (i0 + i < my) {
          const float *x = p.part_o + seg(i0 + i) * DH + lane * VEC;
          if (PER >= 4) {
#pragma unroll
            for (int e = 0; e < PER / 4; ++e) {
              const float4 y = __ldcg(reinterpret_cast<const float4 *>(x) + 32 * e);
              v[i][4 * e] = y.x;
              v[i][(4 * e + 1) % PER] = y.y;
              v[i][(4 * e + 2) % PER] = y.z;
              v[i][(4 * e + 3) % PER] = y.w;
            }
          } else if (PER == 2) {
            const float2 y = __ldcg(reinterpret_cast<const float2 *>(x));
            v[i][0] = y.x;
            v[i][1 % PER] = y.y;
          } else {
            v[i][0] = __ldcg(x);
          }
        }
    };
    float2 x = lane < my ? stats(lane) : make_float2(-INFINITY, 0.f);
    fetch(0);  // with the statistics
    float M = x.x;
    for (int i = lane + 32; i < my; i += 32) M = fmaxf(M, stats(i).x);
    M = warp_max(M);
    float S = 0.f, a[PER];
#pragma unroll
    for (int e = 0; e < PER; ++e) a[e] = 0.f;
    for (int i0 = 0; i0 < my; i0 += 32) {
      if (i0 > 0) x = i0 + lane < my ? stats(i0 + lane) : make_float2(-INFINITY, 0.f);
      const float f = x.x == -INFINITY ? 0.f : exp2f(x.x - M);
      S += warp_sum(x.y * f);
      for (int j = 0; j < 32 && i0 + j < my; j += kBatch) {
        if (i0 + j > 0) fetch(i0 + j);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const float w = __shfl_sync(0xffffffffu, f, j + i);
          if (i0 + j + i < my)
#pragma unroll
            for (int e = 0; e < PER; ++e) a[e] = fmaf(v[i][e], w, a[e]);
        }
      }
    }
    if (wpr > 1) {  // uniform over the block
      float *mem = part[warp];
#pragma unroll
      for (int e = 0; e < PER; ++e) mem[place(lane, e)] = a[e];
      if (lane == 0) {
        mem[DH] = M;
        mem[DH + 1] = S;
      }
      __syncthreads();
      if (q == 0) {
        float N = M;
        for (int w = 1; w < wpr; ++w) N = fmaxf(N, part[warp + w][DH]);
        S = 0.f;
#pragma unroll
        for (int e = 0; e < PER; ++e) a[e] = 0.f;
        for (int w = 0; w < wpr; ++w) {
          const float *y = part[warp + w];
          const float f = y[DH] == -INFINITY ? 0.f : exp2f(y[DH] - N);
          S = fmaf(y[DH + 1], f, S);
#pragma unroll
          for (int e = 0; e < PER; ++e) a[e] = fmaf(y[place(lane, e)], f, a[e]);
        }
        M = N;
      }
      __syncthreads();
    }
    const float inv = paged_inverse(S);
    const int row = d.row0 + r / p.G, hq = d.h * p.G + r % p.G;
    if (mine && q == 0 && in_bounds(row < p.n_rows, p.status)) {
      __nv_bfloat16 *at = static_cast<__nv_bfloat16 *>(p.out) + (long long)row * p.ldo + hq * DH;
#pragma unroll
      for (int e = 0; e < PER; e += VEC) {
        if constexpr (VEC == 4) {
          const __nv_bfloat162 w[2] = {__floats2bfloat162_rn(a[e] * inv, a[e + 1] * inv),
                                       __floats2bfloat162_rn(a[e + 2] * inv, a[e + 3] * inv)};
          *reinterpret_cast<uint2 *>(at + place(lane, e)) = *reinterpret_cast<const uint2 *>(w);
        } else {
#pragma unroll
          for (int j = 0; j < VEC; ++j) at[place(lane, e + j)] = __float2bfloat16_rn(a[e + j] * inv);
        }
      }
      if (lane == 0 && p.lse) p.lse[(size_t)row * p.Hq + hq] = paged_lse(M, S);
    }
  }
  trace_end(kTkPagedCombine);
}

}  // namespace mtp
