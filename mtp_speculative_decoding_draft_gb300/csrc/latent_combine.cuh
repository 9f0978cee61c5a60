// Partial states of the latent attention kernels: how they lie, and the kernel that joins
// them in key order.
//
// A state of a block of ROWS rows x DH elements lies as [DH / 4][ROWS] quads of four
// elements: the thread that holds a row stores its quads as they come, next to those of
// the rows beside it.  (Row by row, the rows had to be exchanged between the lanes first: 64
// shuffles for 32 elements, and a state took 3 us to write.)
#pragma once

#include "paged_combine.cuh"
#include "paged_tc.cuh"
#include "tcgen05_ops.cuh"

namespace mtp {

// Runs f(c, columns 32 c .. 32 c + 31 of this thread's lane) for c = 0 .. C - 1.  (Not
// unrolled, nor with the next columns' load under each: run once a segment, the code comes
// from memory each time, and twice the code cost prompts of a few tiles 8%.)
template <int C, class F>
__device__ __forceinline__ void each_columns(uint32_t taddr, F f) {
#pragma unroll 1
  for (int c = 0; c < C; ++c) {
    uint32_t a[32];
    tmem_ld32_async(taddr + 32 * c, a);
    tmem_wait_ld();
    pin32(a);
    f(c, a);
  }
}

// Scales them by a factor.
template <int C>
__device__ __forceinline__ void rescale_columns(uint32_t taddr, float f) {
  each_columns<C>(taddr, [&](int c, uint32_t (&o)[32]) {
#pragma unroll
    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
    tmem_st32(taddr + 32 * c, o);
  });
}

// Writes a row's output, or its part of a state, from tensor memory: C x 32 elements, the
// first of them element e0 of the row.
//   row_out: where the row's element 0 goes (bf16; null: nowhere), if `whole`
//   state, row: the block's state and the row in it (row < 0: nowhere), otherwise
template <int C, int ROWS>
__device__ __forceinline__ void write_row(uint32_t taddr, int e0, bool whole, uint16_t *row_out, float inv, float *state,
                                          int row, int lane) {
  if (!whole) {
    each_columns<C>(taddr, [&](int c, uint32_t (&o)[32]) {
      if (row >= 0) {
        uint4 *q = reinterpret_cast<uint4 *>(state) + (size_t)(e0 / 4 + 8 * c) * ROWS + row;
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e * ROWS] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
      }
    });
    return;
  }
  // four lanes exchange their quads, so that each row's 64 bytes leave side by side
  uint4 *to[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    to[i] = reinterpret_cast<uint4 *>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(row_out), (lane & ~3) + i));
  each_columns<C>(taddr, [&](int c, uint32_t (&o)[32]) {
    uint4 v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint32_t y[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        y[j] = pack2(__uint_as_float(o[8 * e + 2 * j]) * inv, __uint_as_float(o[8 * e + 2 * j + 1]) * inv);
      v[e] = make_uint4(y[0], y[1], y[2], y[3]);
    }
    transpose_quads<4>(v, lane);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (to[i]) to[i][e0 / 8 + 4 * c + (lane & 3)] = v[i];
  });
}

constexpr int kLatentCombineThreads = 256;

// One group of 32 rows of a split item.
struct CombineGroup {
  PagedDesc d;
  int lo, r0, nseg;  // its first share, first row, states
  // state i: the first lies in its share's second place, the others in the first
  __device__ __forceinline__ size_t state(int i) const { return (size_t)(lo + i) * 2 + (i == 0 ? 1 : 0); }
};

// The shares' descriptions and how many groups of rows lie before each.
struct CombineTable {
  PagedDesc desc[kMaxDescs];
  int before[kMaxDescs + 1], sums[kLatentCombineThreads / 32];

  // Executed by the whole block; returns the number of groups.
  __device__ __forceinline__ int fill(const PagedArgs &p, int shares) {
    static_assert(kLatentCombineThreads == kMaxDescs, "a description a thread");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int4 dd = make_int4(0, 0, 0, 0);
    if (tid < shares) dd = __ldcg(reinterpret_cast<const int4 *>(p.desc + tid));
    *reinterpret_cast<int4 *>(&desc[tid]) = dd;
    const int mine = (dd.y + 31) / 32;
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
    before[tid] = off;
    if (tid == kMaxDescs - 1) before[kMaxDescs] = off + mine;
    __syncthreads();
    return before[kMaxDescs];
  }
  __device__ __forceinline__ CombineGroup find(int g) const {
    int lo = 0, hi = kMaxDescs;  // before[lo] <= g < before[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (before[mid] <= g) lo = mid;
      else hi = mid;
    }
    return {desc[lo], lo, (g - before[lo]) * 32, desc[lo].last_cta - lo + 1};
  }
};

// Joins states i0, i0 + step, .. of row r, elements e0 .. e0 + CW - 1, into (M, S, a); kBatch
// states' statistics and elements are requested together, the running maximum rescaled for.
template <int DH, int ROWS, int CW, int kBatch>
__device__ __forceinline__ void join_states(const PagedArgs &p, const CombineGroup &g, int r, int e0, int first, int step,
                                            float &M, float &S, float (&a)[CW]) {
  constexpr int CQ = CW / 4;
  M = -INFINITY;
  S = 0.f;
#pragma unroll
  for (int e = 0; e < CW; ++e) a[e] = 0.f;
  for (int i0 = first; i0 < g.nseg; i0 += kBatch * step) {
    float2 x[kBatch];
    float4 v[kBatch][CQ];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      x[i] = make_float2(-INFINITY, 0.f);
      const int j = i0 + i * step;
      if (j < g.nseg) {
        const size_t at = g.state(j);
        x[i] = __ldcg(reinterpret_cast<const float2 *>(p.part_ml) + at * ROWS + r);
#pragma unroll
        for (int e = 0; e < CQ; ++e)
          v[i][e] = __ldcg(reinterpret_cast<const float4 *>(p.part_o) + (at * (DH / 4) + e0 / 4 + e) * ROWS + r);
      }
    }
    float N = M;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) N = fmaxf(N, x[i].x);
    const float f0 = M == -INFINITY ? 0.f : exp2f(M - N);
    M = N;
    S *= f0;
#pragma unroll
    for (int e = 0; e < CW; ++e) a[e] *= f0;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (i0 + i * step >= g.nseg) break;
      const float f = x[i].x == -INFINITY ? 0.f : exp2f(x[i].x - M);
      S = fmaf(x[i].y, f, S);
#pragma unroll
      for (int e = 0; e < CQ; ++e) {
        a[4 * e] = fmaf(v[i][e].x, f, a[4 * e]);
        a[4 * e + 1] = fmaf(v[i][e].y, f, a[4 * e + 1]);
        a[4 * e + 2] = fmaf(v[i][e].z, f, a[4 * e + 2]);
        a[4 * e + 3] = fmaf(v[i][e].w, f, a[4 * e + 3]);
      }
    }
  }
}

// Where row r's output goes (null: nowhere), and its log-sum, by the warp that has its first elements.
// PARTS: an item is one of so many parts (of DH elements) of its heads' outputs.
template <int DH, int PARTS>
__device__ __forceinline__ uint16_t *joined_row(const PagedArgs &p, const CombineGroup &g, int r, float M, float S, bool first) {
  const int row = g.d.row0 + r / p.G, hq = g.d.h / PARTS * p.G + r % p.G, part = g.d.h % PARTS;
  // (a block of heads may hold fewer than G at the end)
  if (r >= g.d.rows || hq >= p.Hq || !in_bounds(row < p.n_rows, p.status)) return nullptr;
  if (first && part == 0 && p.lse) p.lse[(size_t)row * p.Hq + hq] = paged_lse(M, S);
  return static_cast<uint16_t *>(p.out) + (long long)row * p.ldo + (hq * PARTS + part) * DH;
}

// Items cut into a few states: a warp joins 32 rows x 8 elements, a lane a row, two states
// requested together (four: 23.4 us against 24.5 where items lie in four, 55.7 against 53.1 where in two).
template <int DH, int ROWS, int PARTS>
__global__ void __launch_bounds__(kLatentCombineThreads, 4)
    latent_combine_kernel(const __grid_constant__ PagedArgs p, int shares) {
  trace_start(kTkPagedCombine);
  constexpr int NW = kLatentCombineThreads / 32, CW = 8, CU = DH / CW;
  __shared__ CombineTable table;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dep_wait();
  trace_dep(kTkPagedCombine);
  grid_dep_launch();
  const int units = table.fill(p, shares) * CU;
  for (int u = blockIdx.x * NW + warp; u < units; u += gridDim.x * NW) {
    const int c = u % CU;
    const CombineGroup g = table.find(u / CU);
    const int r = g.r0 + lane;
    float M, S, a[CW];
    if (r >= g.d.rows) continue;
    join_states<DH, ROWS, CW, 2>(p, g, r, CW * c, 0, 1, M, S, a);
    const float inv = paged_inverse(S);
    if (uint16_t *to = joined_row<DH, PARTS>(p, g, r, M, S, c == 0)) {
      uint32_t y[CW / 2];
#pragma unroll
      for (int j = 0; j < CW / 2; ++j) y[j] = pack2(a[2 * j] * inv, a[2 * j + 1] * inv);
      *reinterpret_cast<uint4 *>(to + CW * c) = make_uint4(y[0], y[1], y[2], y[3]);
    }
  }
  trace_end(kTkPagedCombine);
}

// Few items cut into many states: a block joins 32 rows x 16 elements, each of its warps
// every eighth state, three requested together (one user's 20 states in one round).
template <int DH, int ROWS, int PARTS>
__global__ void __launch_bounds__(kLatentCombineThreads, 2)
    latent_combine_many_kernel(const __grid_constant__ PagedArgs p, int shares) {
  trace_start(kTkPagedCombine);
  constexpr int NW = kLatentCombineThreads / 32, CW = 16, CU = DH / CW;
  __shared__ CombineTable table;
  __shared__ float part[NW][CW][33], stat[NW][2][32];  // [warp][element][row]; maximum, sum
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dep_wait();
  trace_dep(kTkPagedCombine);
  grid_dep_launch();
  const int units = table.fill(p, shares) * CU;
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const int c = u % CU;
    const CombineGroup g = table.find(u / CU);
    float M, S, a[CW];
    join_states<DH, ROWS, CW, 3>(p, g, min(g.r0 + lane, g.d.rows - 1), CW * c, warp, NW, M, S, a);
#pragma unroll
    for (int e = 0; e < CW; ++e) part[warp][e][lane] = a[e];
    stat[warp][0][lane] = M;
    stat[warp][1][lane] = S;
    __syncthreads();
    // ---- eight threads a row, two elements each
    const int y = tid >> 3, e = 2 * (tid & 7);
    float N = -INFINITY, T = 0.f, b0 = 0.f, b1 = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) N = fmaxf(N, stat[w][0][y]);
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float m = stat[w][0][y], f = m == -INFINITY ? 0.f : exp2f(m - N);
      T = fmaf(stat[w][1][y], f, T);
      b0 = fmaf(part[w][e][y], f, b0);
      b1 = fmaf(part[w][e + 1][y], f, b1);
    }
    const float inv = paged_inverse(T);
    if (uint16_t *to = joined_row<DH, PARTS>(p, g, g.r0 + y, N, T, c == 0 && e == 0))
      *reinterpret_cast<uint32_t *>(to + CW * c + e) = pack2(b0 * inv, b1 * inv);
    __syncthreads();
  }
  trace_end(kTkPagedCombine);
}

template <int DH, int ROWS, int PARTS>
cudaError_t launch_latent_combine(const PagedTcParams &sp, int shares, int sms, cudaStream_t s, bool pdl) {
  static_assert(kPagedMaxCtas <= kMaxDescs, "a description a share");
  cudaLaunchConfig_t cfg{};
  // More than eight shares an item: by blocks.  us (by blocks / by warps), R 512: one row of 16 heads,
  // 4 of 4096 keys 14.8 / 20.4, 8 of 2048 14.5 / 16.6, 16 of 2048 19.6 / 18.7; one of 128 heads, 16 of
  // 2048 35.6 / 28.0.  (Of the places of the line, kPagedMaxCtas are for gaps.)  The host does not
  // know an item's shares: one sequence of 131072 keys (16 heads) takes 45 us, among 20 of 512 keys,
  // where the long one's states are joined by warps, 68 (the short alone 15).
  const bool many = 8 * (sp.n_items - kPagedMaxCtas) < shares;
  // what is resident at once: with four blocks an SM of the first kind a call of two keys took 10.0
  // us, with two 9.1; with two of the second kind 16 x 4 rows of 128 heads took 60.7, with four 55.2
  cfg.gridDim = dim3((many ? 2 : 4) * sms);
  cfg.blockDim = dim3(kLatentCombineThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  note_launch();
  return many ? cudaLaunchKernelEx(&cfg, latent_combine_many_kernel<DH, ROWS, PARTS>, sp.a, shares)
              : cudaLaunchKernelEx(&cfg, latent_combine_kernel<DH, ROWS, PARTS>, sp.a, shares);
}

}  // namespace mtp
