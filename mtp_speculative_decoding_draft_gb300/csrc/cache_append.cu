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
// The kernel is bound by its bytes (each row read and written once).  A warp
// takes one unit, a run of 32 x U items of one row (an item: the two vectors of
// VEC elements that rotate together), with no barrier between warps: it issues
// its items' loads first, finds the row's sequence and position under them,
// computes the row's rot/2 sines and cosines two a lane into its own corner of
// shared memory, then rotates and stores.  Recomputing the sines for each unit of
// a row costs less than a block-wide barrier a row: 8190 rows of 40 + 16 heads of
// 128 took 96 us with a block a row, 43 us this way (5.45 TB/s, 80% of the copy
// rate; what is left is the chain position -> page -> store of each warp).
#include "internal.h"
#include "paged.cuh"

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
__global__ void __launch_bounds__(32 * kAppWarps, U == 1 ? 1 : 5) cache_append_kernel(const __grid_constant__ AppendArgs p) {
  trace_start(kTkAppend);
  using T = typename Bf<VEC>::T;
  __shared__ float2 cs_all[kAppWarps][64];  // rot / 2 <= 64
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float2 *cs = cs_all[warp];
  const int ips = __ffs(p.Dh / (2 * VEC)) - 1, iph = 1 << ips;  // items of a head
  const int rph = p.rot / (2 * VEC);                // of them, rotated
  const int q_items = p.q ? p.Hq * iph : 0, kv_items = p.Hkv * iph;
  const int items = q_items + 2 * kv_items, upr = (items + 32 * U - 1) / (32 * U);
  const unsigned unit = blockIdx.x * kAppWarps + warp;
  const int row = (int)(unit / (unsigned)upr), first = (int)(unit - (unsigned)row * (unsigned)upr) * 32 * U;
  const bool half = p.layout == 0;
  grid_dep_wait();
  trace_dep(kTkAppend);
  grid_dep_launch();
  if (blockIdx.x == 0 && p.row_start) {  // once per call: are the row starts in order and inside the rows?
    bool bad = false;
    for (int i = threadIdx.x; i < p.B; i += 32 * kAppWarps) {
      const int x = __ldcg(&p.row_start[i]), y = __ldcg(&p.row_start[i + 1]);
      bad |= x < 0 || y < x || y > p.n_rows;
    }
    if (bad) set_status(p.status, kStatusBadRows);
  }
  if (row >= p.n_rows) {
    trace_end(kTkAppend);
    return;
  }

  // ---- the items' loads need no position
  T a[U], c[U];
  int which[U], head[U], e0[U], e1[U];
  bool rot[U];
#pragma unroll
  for (int n = 0; n < U; ++n) {
    const int it = first + n * 32 + lane;
    which[n] = it >= items ? -1 : it < q_items ? 0 : it < q_items + kv_items ? 1 : 2;
    const int i = which[n] == 1 ? it - q_items : which[n] == 2 ? it - q_items - kv_items : it;
    head[n] = i >> ips;
    const int u = i & (iph - 1);
    rot[n] = which[n] < 2 && u < rph;
    e0[n] = rot[n] && half ? u * VEC : 2 * u * VEC;
    e1[n] = rot[n] && half ? e0[n] + p.rot / 2 : e0[n] + VEC;
    if (which[n] >= 0 && !(p.q_f32 && which[n] == 0)) {
      const void *base = which[n] == 0 ? p.q : which[n] == 1 ? p.k : p.v;
      const long long ld = which[n] == 0 ? p.ldq : which[n] == 1 ? p.ldk : p.ldv;
      const uint16_t *src = static_cast<const uint16_t *>(base) + (long long)row * ld +
                            head[n] * (which[n] == 0 ? p.Dh : which[n] == 1 ? p.khs : p.vhs);
      a[n] = __ldcs(reinterpret_cast<const T *>(src + e0[n]));
      c[n] = __ldcs(reinterpret_cast<const T *>(src + e1[n]));
    }
  }

  // ---- the row's sequence: the last one that starts at or before it (those that
  // start at the same row are empty but the last of them).  For up to 32 sequences
  // a lane has one's numbers in hand, and the search costs no second round trip.
  bool real = false;
  int b, s0 = row, s1 = row + 1, c0 = 0, pos = 0, page = -1;  // c0: the context as given
  if (!p.row_start) {
    b = row;
    c0 = __ldcg(&p.ctx_len[b]);
  } else if (p.B <= 32) {
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
      const long long at = (long long)c0 + p.ctx_add + (row - s0);
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
    trace_end(kTkAppend);
    return;
  }
  if (first < q_items + kv_items) {  // not values only
    for (int t = lane; t < p.rot / 2; t += 32) {
      const unsigned long long f = (unsigned long long)(unsigned)pos * __ldg(&p.turns[t]);
      // the top 32 bits as a signed fraction of a half turn: [-1, 1)
      const float x = (float)(int)(f >> 32) * 4.656612873077393e-10f;
      float sn, co;
      sincospif(x, &sn, &co);
      cs[t] = make_float2(co * p.scale, sn * p.scale);
    }
    __syncwarp();
  }
#pragma unroll
  for (int n = 0; n < U; ++n) {
    if (which[n] < 0) continue;
    float x[VEC], y[VEC];
    if (p.q_f32 && which[n] == 0) {  // fp32 queries, rounded once, after the rotation
      const float *qs = static_cast<const float *>(p.q) + (long long)row * p.ldq + head[n] * p.Dh;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        x[i] = __ldcg(qs + e0[n] + i);
        y[i] = __ldcg(qs + e1[n] + i);
      }
    } else {
      unpack<VEC>(a[n], x);
      unpack<VEC>(c[n], y);
    }
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
    if (which[n] == 0) {
      dst = static_cast<uint16_t *>(p.q_out) + (long long)row * p.ldqo + head[n] * p.Dh;
    } else {
      if (page < 0) continue;
      dst = (which[n] == 1 ? p.k_pages : p.v_pages) +
            (((size_t)page * p.Hkv + head[n]) * p.page + (pos & (p.page - 1))) * p.Dh;
    }
    *reinterpret_cast<T *>(dst + e0[n]) = pack<VEC>(x);
    *reinterpret_cast<T *>(dst + e1[n]) = pack<VEC>(y);
  }
  trace_end(kTkAppend);
}

namespace {

template <int VEC, int U>
cudaError_t launch_append(const AppendArgs &a, int items, cudaStream_t s, bool pdl) {
  const long long units = (long long)a.n_rows * ((items + 32 * U - 1) / (32 * U));
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
  return cudaLaunchKernelEx(&cfg, cache_append_kernel<VEC, U>, a);
}

}  // namespace

cudaError_t launch_cache_append(const AppendArgs &a, cudaStream_t s, bool pdl) {
  // 16-byte accesses need the pairs' halves in whole vectors
  const bool wide = a.rot % 16 == 0;
  const int items = (a.Hq + 2 * a.Hkv) * a.Dh / (wide ? 16 : 8);
  // Few rows: an item a lane, more warps, the shortest chain; many rows: two items a
  // lane at five blocks an SM.  In graphs of 20 calls (us, one item / two): 64 rows of
  // 32 + 16 heads of 128 3.1 / 3.5, 256 rows 8.0 / 5.3, 1000 rows 19.2 / 12.1; 256 rows
  // of 14 + 4 heads of 64 3.2 / 3.7, 1024 rows 6.6 / 4.7; 8190 rows of 40 + 16 heads of
  // 128 63 / 43 (four items at three blocks 46, at five, spilling, 60).
  if ((long long)a.n_rows * items < 152ll * 256)
    return wide ? launch_append<8, 1>(a, items, s, pdl) : launch_append<4, 1>(a, items, s, pdl);
  return wide ? launch_append<8, 2>(a, items, s, pdl) : launch_append<4, 2>(a, items, s, pdl);
}

MTP_TRACE_COLLECTOR(cache_append)

}  // namespace mtp
