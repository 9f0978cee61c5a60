// The new rows of a latent cache: norm of the latents, rotary positions, and the
// write into the pages.
//
// Row i of sequence b sits at position pos = ctx_len[b] + i.  Its cache row is
//   [ c * rsqrt(mean(c^2) + eps) * gain , turn(k) ]
// with c its R latent elements and k its Dr key elements; each head's rotary query
// part turns alike.  Pair t of the first rot elements, (x0, x1), turns by
// pos * f_t (the table and the angle's arithmetic are cache_append.cu's):
//   (x0, x1) -> scale (x0 cos - x1 sin, x1 cos + x0 sin)
//
// Bound by the bytes of the queries (each row read and written once): 8190 rows of 40 heads
// take 25 us, 102 MB at 61% of the copy rate (in graphs of 20, where a part of them stays in L2,
// 21.9); the rest is each warp's chain of position, page entry and store.  Four rows of 128
// heads in such a graph: 2.6 us, a launch.
// A warp takes one unit: the first unit of a row is its latent, held in registers between
// the sum of squares and the product with the gain; the others are runs of 32 x U items (an
// item: the two vectors of VEC elements that rotate together) of the heads, the key counting
// as one head more.
#include "internal.h"
#include "latent.cuh"

namespace mtp {

namespace {

constexpr int kAppWarps = 8;
constexpr unsigned kFull = 0xffffffffu;

template <int VEC>
struct Bf;
template <>
struct Bf<8> {
  typedef uint4 T;
};
template <>
struct Bf<4> {
  typedef uint2 T;
};

template <int VEC>
__device__ __forceinline__ void unpack(const typename Bf<VEC>::T &v, float (&x)[VEC]) {
  const uint32_t *w = reinterpret_cast<const uint32_t *>(&v);
#pragma unroll
  for (int i = 0; i < VEC / 2; ++i) {
    x[2 * i] = bf16_lo(w[i]);
    x[2 * i + 1] = bf16_hi(w[i]);
  }
}

template <int VEC>
__device__ __forceinline__ typename Bf<VEC>::T pack(const float (&x)[VEC]) {
  typename Bf<VEC>::T v;
  uint32_t *w = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
  for (int i = 0; i < VEC / 2; ++i) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&t);
  }
  return v;
}

}  // namespace

template <int VEC, int U>
__global__ void __launch_bounds__(32 * kAppWarps, U == 1 ? 1 : 5) latent_append_kernel(const __grid_constant__ LatentAppendArgs p) {
  trace_start(kTkLatentAppend);
  using T = typename Bf<VEC>::T;
  __shared__ float2 cs_all[kAppWarps][32];  // rot / 2 <= 32
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float2 *cs = cs_all[warp];
  const int ips = __ffs(p.Dr / (2 * VEC)) - 1, iph = 1 << ips;  // items of a head
  const int rph = p.rot / (2 * VEC);                            // of them, rotated
  const int q_items = p.q ? p.Hq * iph : 0, items = q_items + iph;
  const int upr = 1 + (items + 32 * U - 1) / (32 * U);
  const unsigned unit = blockIdx.x * kAppWarps + warp;
  const int row = (int)(unit / (unsigned)upr), u0 = (int)(unit - (unsigned)row * (unsigned)upr);
  const int first = (u0 - 1) * 32 * U;
  const bool half = p.layout == 0, latent = u0 == 0;
  grid_dep_wait();
  trace_dep(kTkLatentAppend);
  grid_dep_launch();
  if (blockIdx.x == 0) {  // once per call: are the row starts in order and inside the rows?
    bool bad = false;
    for (int i = threadIdx.x; i < p.B; i += 32 * kAppWarps) {
      const int x = __ldcg(&p.row_start[i]), y = __ldcg(&p.row_start[i + 1]);
      bad |= x < 0 || y < x || y > p.n_rows;
    }
    if (bad) set_status(p.status, kStatusBadRows);
  }
  if (row >= p.n_rows) {
    trace_end(kTkLatentAppend);
    return;
  }

  // ---- the unit's loads need no position
  T a[U], c[U];
  int head[U], e0[U], e1[U];
  bool rot[U];
  uint4 lat[2], gain[2];
  if (latent) {
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int e = (n * 32 + lane) * 8;
      lat[n] = gain[n] = make_uint4(0u, 0u, 0u, 0u);
      if (e < p.R) {
        lat[n] = __ldcs(reinterpret_cast<const uint4 *>(p.kv + (long long)row * p.ldkv + e));
        if (p.gain) gain[n] = __ldg(reinterpret_cast<const uint4 *>(p.gain + e));
      }
    }
  } else {
#pragma unroll
    for (int n = 0; n < U; ++n) {
      const int it = first + n * 32 + lane;
      head[n] = it >= items ? -1 : it < q_items ? it >> ips : p.Hq;  // Hq: the key
      const int u = it & (iph - 1);
      rot[n] = u < rph;
      e0[n] = rot[n] && half ? u * VEC : 2 * u * VEC;
      e1[n] = rot[n] && half ? e0[n] + p.rot / 2 : e0[n] + VEC;
      if (head[n] >= 0) {
        const uint16_t *src = head[n] == p.Hq ? p.kv + (long long)row * p.ldkv + p.R
                                              : p.q + (long long)row * p.ldq + head[n] * p.hsq;
        a[n] = __ldcs(reinterpret_cast<const T *>(src + e0[n]));
        c[n] = __ldcs(reinterpret_cast<const T *>(src + e1[n]));
      }
    }
  }

  // ---- the row's sequence: the last one that starts at or before it.  For up to 32
  // sequences a lane has one's numbers in hand.
  bool real = false;
  int b, s0 = row, s1 = row, c0 = 0, pos = 0, page = -1;  // c0: the context as given
  if (p.B <= 32) {
    const int mine = min(lane, p.B - 1);
    const int x0 = __ldcg(&p.row_start[mine]), x1 = __ldcg(&p.row_start[mine + 1]), x2 = __ldcg(&p.ctx_len[mine]);
    b = __popc(__ballot_sync(kFull, lane < p.B && x0 <= row)) - 1;
    s0 = __shfl_sync(kFull, x0, max(b, 0));
    s1 = __shfl_sync(kFull, x1, max(b, 0));
    c0 = __shfl_sync(kFull, x2, max(b, 0));
  } else {
    b = starts_upto(p.row_start, p.B, row, lane) - 1;
    if (b >= 0) {
      s0 = __ldcg(&p.row_start[b]);
      s1 = __ldcg(&p.row_start[b + 1]);
      c0 = __ldcg(&p.ctx_len[b]);
    }
  }
  if (b >= 0) {
    real = row < s1 && s0 >= 0 && row >= s0;
    if (real) {
      // a negative context places no row, whatever is added to it
      const long long at = (long long)c0 + (row - s0);
      const bool placed = c0 >= 0 && at < p.cap;
      pos = (int)min(max(at, 0ll), (long long)p.cap);  // of a row that is not placed: for its rotation only
      if (lane == 0 && !placed) set_status(p.status, kStatusBadCtx);
      if (placed) {
        page = __ldg(&p.page_table[(size_t)b * p.max_pages + (pos >> p.page_shift)]);
        if (page < 0 || page >= p.n_pages) {
          if (lane == 0) set_status(p.status, kStatusBadPage);
          page = -1;
        }
      }
    }
  }
  if (!real) {
    trace_end(kTkLatentAppend);
    return;
  }
  uint16_t *slot = p.pages + ((size_t)max(page, 0) * p.page + (pos & (p.page - 1))) * (size_t)(p.R + p.Dr);

  if (latent) {
    float x[2][8];
    float ss = 0.f;
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      unpack<8>(lat[n], x[n]);
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(x[n][i], x[n][i], ss);
    }
    if (p.gain) {
      ss = warp_sum(ss);
      const float inv = 1.f / sqrtf(ss / (float)p.R + p.eps);
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        float g[8];
        unpack<8>(gain[n], g);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[n][i] = x[n][i] * inv * g[i];
        lat[n] = pack<8>(x[n]);
      }
    }
    if (page >= 0)
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int e = (n * 32 + lane) * 8;
        if (e < p.R) *reinterpret_cast<uint4 *>(slot + e) = lat[n];
      }
    trace_end(kTkLatentAppend);
    return;
  }
  for (int t = lane; t < p.rot / 2; t += 32) {
    const unsigned long long f = (unsigned long long)(unsigned)pos * __ldg(&p.turns[t]);
    // the top 32 bits as a signed fraction of a half turn: [-1, 1)
    const float x = (float)(int)(f >> 32) * 4.656612873077393e-10f;
    float sn, co;
    sincospif(x, &sn, &co);
    cs[t] = make_float2(co * p.scale, sn * p.scale);
  }
  __syncwarp();
#pragma unroll
  for (int n = 0; n < U; ++n) {
    if (head[n] < 0) continue;
    float x[VEC], y[VEC];
    unpack<VEC>(a[n], x);
    unpack<VEC>(c[n], y);
    if (rot[n] && half) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float2 f = cs[e0[n] + i];
        const float x0 = x[i], x1 = y[i];
        x[i] = x0 * f.x - x1 * f.y;
        y[i] = x1 * f.x + x0 * f.y;
      }
    } else if (rot[n]) {
#pragma unroll
      for (int i = 0; i < VEC / 2; ++i) {
        const float2 f = cs[e0[n] / 2 + i], g = cs[e1[n] / 2 + i];
        const float x0 = x[2 * i], x1 = x[2 * i + 1], y0 = y[2 * i], y1 = y[2 * i + 1];
        x[2 * i] = x0 * f.x - x1 * f.y;
        x[2 * i + 1] = x1 * f.x + x0 * f.y;
        y[2 * i] = y0 * g.x - y1 * g.y;
        y[2 * i + 1] = y1 * g.x + y0 * g.y;
      }
    }
    uint16_t *dst;
    if (head[n] == p.Hq) {
      if (page < 0) continue;
      dst = slot + p.R;
    } else {
      dst = p.q_out + (long long)row * p.ldqo + head[n] * p.hsqo;
    }
    *reinterpret_cast<T *>(dst + e0[n]) = pack<VEC>(x);
    *reinterpret_cast<T *>(dst + e1[n]) = pack<VEC>(y);
  }
  trace_end(kTkLatentAppend);
}

namespace {

template <int VEC, int U>
cudaError_t launch_append(const LatentAppendArgs &a, int items, cudaStream_t s, bool pdl) {
  const long long units = (long long)a.n_rows * (1 + (items + 32 * U - 1) / (32 * U));
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((units + kAppWarps - 1) / kAppWarps));
  cfg.blockDim = dim3(32 * kAppWarps);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  note_launch();
  return cudaLaunchKernelEx(&cfg, latent_append_kernel<VEC, U>, a);
}

}  // namespace

cudaError_t launch_latent_append(const LatentAppendArgs &a, int sms, cudaStream_t s, bool pdl) {
  // 16-byte accesses need the pairs' halves in whole vectors
  const bool wide = a.rot % 16 == 0;
  const int items = ((a.q ? a.Hq : 0) + 1) * a.Dr / (wide ? 16 : 8);
  // One item a lane until each SM has a block's worth of items (38912 on 152), two from there on.
  // us (one / two, Dr 64): 4 rows of 128 heads 2.4 / 2.7, 256 of 16 3.3 / 3.4, 512 of 16 (34816 items)
  // 3.1 / 3.1, 256 of 40 (41984) 4.6 / 3.8 and 3.0 / 2.9 (64 sequences, one), 256 of 128 10.5 / 6.7,
  // 1024 of 16 5.3 / 4.9, 8190 of 16 21.7 / 18.0, of 40 37.0 / 25.2, of 128 93.0 / 62.5;
  // 1024 of 40 with 24 elements that rotate 9.0 / 6.9.
  if ((long long)a.n_rows * items < 256ll * sms)
    return wide ? launch_append<8, 1>(a, items, s, pdl) : launch_append<4, 1>(a, items, s, pdl);
  return wide ? launch_append<8, 2>(a, items, s, pdl) : launch_append<4, 2>(a, items, s, pdl);
}

MTP_TRACE_COLLECTOR(latent_append)

}  // namespace mtp
