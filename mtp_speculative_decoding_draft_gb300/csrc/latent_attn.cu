// Absorbed latent attention over a paged cache.
#include "internal.h"
#include "latent_rows.cuh"

namespace mtp {

__global__ void __launch_bounds__(128) latent_attn_kernel(const __grid_constant__ LatentAttnArgs la) {
  const PagedArgs &p = la.a;
  trace_start(kTkLatentAttn);
  grid_dep_wait();
  trace_dep(kTkLatentAttn);
  grid_dep_launch();
  const int row = blockIdx.x, w = p.Dh + la.Dr;
  int b;
  PagedSeq s;
  if (!find_row(p, row, &b, &s)) return;
  for (int h = threadIdx.x >> 5; h < p.Hq; h += 4) {
    int j_at = -1;
    const uint16_t *src = nullptr;
    auto get = [&](int j, int e) {
      if (j != j_at) {
        src = la.pages + ((size_t)paged_page(p, b, j) * p.page + (j & (p.page - 1))) * w;
        j_at = j;
      }
      return (uint32_t)src[e];
    };
    attend_row<576, 512>(p, s, row, h, p.q + (long long)row * p.ldq + h * w, w, p.Dh, get, get);
  }
  trace_end(kTkLatentAttn);
}

bool latent_attn_items_ok(int, int, int) { return true; }
size_t latent_attn_scratch_bytes(int, int, int, int) { return 256; }

cudaError_t launch_latent_attn(const LatentAttnArgs &la, void *, int, cudaStream_t s, bool) {
  note_launch();
  latent_attn_kernel<<<la.a.n_rows, 128, 0, s>>>(la);
  return cudaGetLastError();
}

cudaError_t latent_set_attributes() { return cudaSuccess; }

MTP_TRACE_COLLECTOR(latent_attn)

}  // namespace mtp
