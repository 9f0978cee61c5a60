// Attention of a prompt's rows over keys and values of each head.
#include "internal.h"
#include "latent_rows.cuh"

namespace mtp {

__global__ void __launch_bounds__(128) latent_prefill_kernel(const __grid_constant__ LatentPrefillArgs lp) {
  const PagedArgs &p = lp.a;
  trace_start(kTkLatentPrefill);
  grid_dep_wait();
  trace_dep(kTkLatentPrefill);
  grid_dep_launch();
  const int row = blockIdx.x;
  int b;
  PagedSeq s;
  if (!find_row(p, row, &b, &s)) return;
  const int first = __ldcg(&lp.key_start[b]);
  if (first < 0 || (long long)first + s.ctx + s.n > lp.n_keys) {
    set_status(p.status, kStatusBadCtx);
    return;
  }
  const int w = lp.Dn + lp.Dv, dk = lp.Dn + lp.Dr;
  for (int h = threadIdx.x >> 5; h < p.Hq; h += 4) {
    auto key = [&](int j, int e) {
      const long long r = first + j;
      return (uint32_t)(e < lp.Dn ? lp.kv[r * lp.ldkv + h * w + e] : lp.k_rope[r * lp.ldkr + e - lp.Dn]);
    };
    auto val = [&](int j, int e) { return (uint32_t)lp.kv[(long long)(first + j) * lp.ldkv + h * w + lp.Dn + e]; };
    attend_row<192, 128>(p, s, row, h, p.q + (long long)row * p.ldq + h * dk, dk, lp.Dv, key, val);
  }
  trace_end(kTkLatentPrefill);
}

bool latent_prefill_items_ok(int, int, int) { return true; }
size_t latent_prefill_scratch_bytes(int, int, int, int) { return 256; }

cudaError_t launch_latent_prefill(const LatentPrefillArgs &lp, void *, int, cudaStream_t s, bool) {
  note_launch();
  latent_prefill_kernel<<<lp.a.n_rows, 128, 0, s>>>(lp);
  return cudaGetLastError();
}

MTP_TRACE_COLLECTOR(latent_prefill)

}  // namespace mtp
