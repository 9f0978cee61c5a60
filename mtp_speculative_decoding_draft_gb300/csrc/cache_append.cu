// Rotary positions and the write into the pages of a paged K/V cache.
//
// Row i of sequence b sits at position pos = ctx_len[b] + i.  Pair t of a
// head's first rot dims, (x0, x1), turns by pos * f_t:
//   (x0, x1) -> scale (x0 cos - x1 sin, x1 cos + x0 sin)
// with pairs (t, t + rot/2) or (2t, 2t + 1).  Queries go to q_out, keys and
// values to their page slots.
//
// The angle.  pos * f_t in fp32 loses the angle at far positions (2^-24 of
// 10^5 radians is 0.006).  The table holds f_t in turns as a 0.64 fixed-point
// fraction, so that pos * table mod 2^64 is the angle's fraction of a turn
// exactly to pos * 2^-65 turns: one 64-bit integer product, no wide floating
// point.  sincospif of that fraction is accurate to fp32.
//
// The kernel is bound by its bytes (each row read and written once).  A CTA
// takes one row at a time: every thread first issues the loads of its items
// (pairs of VEC elements that rotate together), then rot/2 threads compute the
// row's sines and cosines once for all heads, and after a barrier the items are
// rotated and stored.
#include "internal.h"
#include "paged.cuh"

namespace mtp {

namespace {

constexpr int kAppThreads = 384;
constexpr int kAppItems = 2;  // items a thread holds at a time

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

template <int VEC>
__global__ void __launch_bounds__(kAppThreads) cache_append_kernel(const __grid_constant__ AppendArgs p) {
  trace_start(kTkAppend);
  using T = typename Bf<VEC>::T;
  __shared__ float2 cs[64];  // rot / 2 <= 64
  const int tid = threadIdx.x;
  grid_dep_wait();
  trace_dep(kTkAppend);
  grid_dep_launch();
  const int iph = p.Dh / (2 * VEC);                 // items of a head
  const int rph = p.rot / (2 * VEC);                // of them, rotated
  const int q_items = p.q ? p.Hq * iph : 0, kv_items = p.Hkv * iph;
  const int items = q_items + 2 * kv_items;
  const bool half = p.layout == 0;

  for (int row = blockIdx.x; row < p.n_rows; row += gridDim.x) {
    // ---- the first items' loads need no position
    T a[kAppItems], c[kAppItems];
    auto locate = [&](int it, const uint16_t *&src, int &which, int &head, int &e0, int &e1, bool &rot) {
      which = it < q_items ? 0 : it < q_items + kv_items ? 1 : 2;
      const int i = which == 0 ? it : which == 1 ? it - q_items : it - q_items - kv_items;
      head = i / iph;
      const int u = i - head * iph;
      rot = which < 2 && u < rph;
      if (rot && half) {
        e0 = u * VEC;
        e1 = e0 + p.rot / 2;
      } else {
        e0 = 2 * u * VEC;
        e1 = e0 + VEC;
      }
      const void *base = which == 0 ? p.q : which == 1 ? p.k : p.v;
      const long long ld = which == 0 ? p.ldq : which == 1 ? p.ldk : p.ldv;
      src = static_cast<const uint16_t *>(base) + (long long)row * ld + head * p.Dh;
    };
    auto load = [&](int it0) {
#pragma unroll
      for (int n = 0; n < kAppItems; ++n) {
        const int it = it0 + n * kAppThreads;
        if (it < items) {
          const uint16_t *src;
          int which, head, e0, e1;
          bool rot;
          locate(it, src, which, head, e0, e1, rot);
          a[n] = __ldcg(reinterpret_cast<const T *>(src + e0));
          c[n] = __ldcg(reinterpret_cast<const T *>(src + e1));
        }
      }
    };
    const bool f32q = p.q_f32 != 0;
    if (!f32q) load(tid);

    // ---- the row's sequence: the last one that starts at or before the row
    int below = 0;
    for (int b0 = 0; b0 < p.B; b0 += kAppThreads) {
      const int b = b0 + tid;
      below += __syncthreads_count(b < p.B && __ldcg(&p.row_start[b]) <= row);
    }
    // sequences that start at the same row are empty but the last of them
    const int b = below - 1;
    int pos = 0, page = -1;
    bool real = b >= 0 && row < __ldcg(&p.row_start[b + 1]);
    if (real) {
      const int s0 = __ldcg(&p.row_start[b]), c0 = __ldcg(&p.ctx_len[b]);
      const int ctx = min(max(c0, 0), p.cap);
      real = s0 >= 0;
      pos = ctx + row - s0;
      if (tid == 0 && (c0 != ctx || pos >= p.cap)) set_status(p.status, kStatusBadCtx);
      if (pos < p.cap) {
        page = __ldg(&p.page_table[(size_t)b * p.max_pages + (pos >> p.page_shift)]);
        if (page < 0 || page >= p.n_pages) {
          if (tid == 0) set_status(p.status, kStatusBadPage);
          page = -1;
        }
      }
    }
    if (row == blockIdx.x && blockIdx.x == 0) {  // once per call: are the row starts in order and inside the rows?
      bool bad = false;
      for (int i = tid; i < p.B; i += kAppThreads) {
        const int x = __ldcg(&p.row_start[i]), y = __ldcg(&p.row_start[i + 1]);
        bad |= x < 0 || y < x || y > p.n_rows;
      }
      if (bad) set_status(p.status, kStatusBadRows);
    }
    if (real && tid < p.rot / 2) {
      const unsigned long long t = (unsigned long long)(unsigned)pos * p.turns[tid];
      // the top 32 bits as a signed fraction of a half turn: [-1, 1)
      const float x = (float)((long long)t >> 32) * 4.656612873077393e-10f;
      float sn, co;
      sincospif(x, &sn, &co);
      cs[tid] = make_float2(co * p.scale, sn * p.scale);
    }
    __syncthreads();
    if (real) {
      for (int it0 = tid; it0 < items; it0 += kAppItems * kAppThreads) {
        if (it0 != tid && !f32q) load(it0);
#pragma unroll
        for (int n = 0; n < kAppItems; ++n) {
          const int it = it0 + n * kAppThreads;
          if (it >= items) continue;
          const uint16_t *src;
          int which, head, e0, e1;
          bool rot;
          locate(it, src, which, head, e0, e1, rot);
          float x[VEC], y[VEC];
          if (f32q && which == 0) {  // fp32 queries, rounded once after the rotation
            const float *qs = static_cast<const float *>(p.q) + (long long)row * p.ldq + head * p.Dh;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
              x[i] = __ldcg(qs + e0 + i);
              y[i] = __ldcg(qs + e1 + i);
            }
          } else {
            if (f32q) {
              a[n] = __ldcg(reinterpret_cast<const T *>(src + e0));
              c[n] = __ldcg(reinterpret_cast<const T *>(src + e1));
            }
            unpack<VEC>(a[n], x);
            unpack<VEC>(c[n], y);
          }
          if (rot && half) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
              const float2 f = cs[e0 + i];
              const float x0 = x[i], x1 = y[i];
              x[i] = x0 * f.x - x1 * f.y;
              y[i] = x1 * f.x + x0 * f.y;
            }
          } else if (rot) {
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) {
              const float2 f = cs[e0 / 2 + i], g = cs[e1 / 2 + i];
              const float x0 = x[2 * i], x1 = x[2 * i + 1], y0 = y[2 * i], y1 = y[2 * i + 1];
              x[2 * i] = x0 * f.x - x1 * f.y;
              x[2 * i + 1] = x1 * f.x + x0 * f.y;
              y[2 * i] = y0 * g.x - y1 * g.y;
              y[2 * i + 1] = y1 * g.x + y0 * g.y;
            }
          }
          uint16_t *dst;
          if (which == 0) {
            dst = static_cast<uint16_t *>(p.q_out) + (long long)row * p.ldqo + head * p.Dh;
          } else {
            if (page < 0) continue;
            dst = (which == 1 ? p.k_pages : p.v_pages) +
                  (((size_t)page * p.Hkv + head) * p.page + (pos & (p.page - 1))) * p.Dh;
          }
          *reinterpret_cast<T *>(dst + e0) = pack<VEC>(x);
          *reinterpret_cast<T *>(dst + e1) = pack<VEC>(y);
        }
      }
    }
    __syncthreads();  // the sines are the next row's
  }
  trace_end(kTkAppend);
}

cudaError_t launch_cache_append(const AppendArgs &a, cudaStream_t s, bool pdl) {
  cudaLaunchConfig_t cfg{};
  const int grid = a.n_rows < 152 * 40 ? a.n_rows : 152 * 40;
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kAppThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  note_launch();
  // 16-byte accesses need the pairs' halves in whole vectors
  if (a.rot % 16 == 0) return cudaLaunchKernelEx(&cfg, cache_append_kernel<8>, a);
  return cudaLaunchKernelEx(&cfg, cache_append_kernel<4>, a);
}

MTP_TRACE_COLLECTOR(cache_append)

}  // namespace mtp
