// A product a head: y[n, h, :] = W[h] x[n, h, :], from an array of rows or from the
// pages of a latent cache (then the rows are the cached positions of the sequences
// and every head reads the same one).
#include "internal.h"
#include "latent.cuh"

namespace mtp {

namespace {

constexpr int kThreads = 256;

}  // namespace

__global__ void __launch_bounds__(kThreads) latent_heads_kernel(const __grid_constant__ LatentHeadsArgs p) {
  trace_start(kTkLatentHeads);
  grid_dep_wait();
  trace_dep(kTkLatentHeads);
  grid_dep_launch();
  const int row = blockIdx.x, h = blockIdx.y, lane = threadIdx.x & 31;
  const uint16_t *x = p.x + (long long)row * p.ldx + h * p.hsx;
  if (p.pages) {
    bool bad = false;
    if (row == 0 && h == 0)
      for (int i = threadIdx.x; i < p.B; i += kThreads) {
        const int s = __ldcg(&p.key_start[i]), e = __ldcg(&p.key_start[i + 1]);
        bad |= s < 0 || e < s || e > p.n_rows;
      }
    if (bad) set_status(p.status, kStatusBadRows);
    const int b = starts_upto(p.key_start, p.B, row, lane) - 1;
    if (b < 0) return;
    const int s = __ldcg(&p.key_start[b]), e = __ldcg(&p.key_start[b + 1]), j = row - s;
    if (row >= e || s < 0) return;
    if (j >= p.cap) {
      set_status(p.status, kStatusBadCtx);
      return;
    }
    int page = __ldg(&p.page_table[(size_t)b * p.max_pages + (j >> p.page_shift)]);
    if (page < 0 || page >= p.n_pages) {
      set_status(p.status, kStatusBadPage);
      page = 0;
    }
    x = p.pages + ((size_t)page * p.page + (j & (p.page - 1))) * (size_t)(p.K + p.Dr);
    if (h == 0 && threadIdx.x < p.Dr) p.k_rope[(long long)row * p.ldkr + threadIdx.x] = x[p.K + threadIdx.x];
  }
  for (int n = threadIdx.x; n < p.N; n += kThreads) {
    float acc = 0.f;
    for (int k = 0; k < p.K; ++k) {
      const uint16_t *w = p.w + h * p.hsw + (p.transposed ? k * p.ldw + n : n * p.ldw + k);
      acc = fmaf(bf16_lo(x[k]), bf16_lo(*w), acc);
    }
    reinterpret_cast<__nv_bfloat16 *>(p.y)[(long long)row * p.ldy + h * p.hsy + n] = __float2bfloat16_rn(acc);
  }
  trace_end(kTkLatentHeads);
}

cudaError_t launch_latent_heads(const LatentHeadsArgs &a, int, cudaStream_t s, bool pdl) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(a.n_rows, a.H);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  note_launch();
  return cudaLaunchKernelEx(&cfg, latent_heads_kernel, a);
}

MTP_TRACE_COLLECTOR(latent_heads)

}  // namespace mtp
