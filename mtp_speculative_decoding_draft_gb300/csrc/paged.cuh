// Shared by the kernels over the paged K/V cache (cache_append.cu,
// paged_attn.cu, paged_attn_tc.cu): the call's arguments, the visible key range
// of a block of query rows, and the division of a ragged batch over the CTAs.
//
// A sequence's new rows are cut into blocks of whole tokens; with the group's G
// query heads packed beside each token, a block has tokens x G query rows that
// all read the same K/V head.  An item is one (sequence, kv head, block); its
// work is the key tiles that some row of it sees.  The tiles of all items, in
// item order, form one line that is cut into equal shares, one per CTA: every
// CTA streams the same number of tiles whatever the lengths are.  An item that
// crosses a cut leaves fp32 partial states (running maximum, sum, output) in
// the workspace, which a second kernel joins in key order.
#pragma once

#include <cuda.h>

#include "common.cuh"

namespace mtp {

// trace kinds: the MTP_TK_* values of the public header
constexpr int kTkPagedAttn = 60, kTkPagedAttnTc = 61, kTkPagedCombine = 62, kTkAppend = 63, kTkPagedPlan = 65;
// status bits (mirror MTP_STATUS_*)
constexpr int kStatusBadRows = 32;
constexpr int kStatusBadPage = 64;

// What a CTA leaves for the combine kernel: the item that starts in it and does
// not end in it (none: rows = 0).
struct alignas(16) PagedDesc {
  int row0;      // first query row (of q) of the block
  int rows;      // packed rows of the block (tokens x G)
  int h;         // kv head
  int last_cta;  // the CTA in which the item ends
};

struct PagedArgs {
  int B, Hq, Hkv, G, Dh;
  int page, page_shift, n_pages, max_pages, cap;  // cap = max_pages * page
  int n_rows;
  const int *row_start;   // [B + 1]; null: one row a sequence
  const int *ctx_len;     // [B], ctx_add more positions each
  int ctx_add;
  const int *page_table;  // [B, max_pages]
  const uint16_t *q;      // bf16 rows of Hq * Dh, ldq elements apart
  long long ldq, ldo;
  void *out;              // bf16 (or fp32) rows, ldo elements apart
  int out_f32;            // (streaming kernel only)
  float *lse;             // [n_rows, Hq] or null
  float scale_log2;       // softmax scale * log2(e)
  int window, sinks;      // window 0: every earlier key
  int *status;
  int tpb;                // tokens per block
  int min_tiles;          // tiles of a run when items are cut one by one; least tiles of a share otherwise
  PagedDesc *desc;        // [CTAs]
  float *part_o;          // [CTAs][2][block rows][Dh]
  float *part_ml;         // [CTAs][2][block rows][2]
};

struct PagedSeq {
  int row0, n, ctx;
};

// Sequence b's rows and context, clamped to the buffers; flags what was out of range, and
// sets *back if the rows end before they start.
__device__ __forceinline__ PagedSeq paged_seq(const PagedArgs &p, int b, bool flag, bool *back = nullptr) {
  const int a = p.row_start ? __ldcg(&p.row_start[b]) : b, e = p.row_start ? __ldcg(&p.row_start[b + 1]) : b + 1;
  const int c = min(__ldcg(&p.ctx_len[b]), 0x7fffffff - p.ctx_add) + p.ctx_add;  // past the cache either way
  PagedSeq s;
  s.row0 = min(max(a, 0), p.n_rows);
  s.n = min(max(e, s.row0), p.n_rows) - s.row0;
  s.ctx = min(max(c, 0), p.cap);
  if (back) *back |= e < a;
  if (flag) {
    if (s.row0 != a || s.row0 + s.n != e) set_status(p.status, kStatusBadRows);
    if (s.ctx != c || (long long)s.ctx + s.n > p.cap) set_status(p.status, kStatusBadCtx);
  }
  return s;
}

// Keys that some row of tokens [t0, t1) sees: [0, sink_end) and [lo, hi); in
// tiles of TK keys: the first ns tiles, then tiles ft ..; count in all (at least
// one, so that a block that sees nothing is still written).
struct PagedRange {
  int lo, hi, sink_end, ns, ft, count;
  __device__ __forceinline__ int tile(int i) const { return i < ns ? i : ft + (i - ns); }
  __device__ __forceinline__ bool any(int k0, int k1) const {  // some key of [k0, k1) is visible
    return (k0 < hi && k1 > lo && lo < hi) || k0 < sink_end;
  }
  __device__ __forceinline__ bool sees(int j) const { return (j < hi && j >= lo) || j < sink_end; }
};

template <int TK>
__device__ __forceinline__ PagedRange paged_range(const PagedArgs &p, const PagedSeq &s, int t0, int t1) {
  PagedRange r;
  r.hi = min(s.ctx + t1, p.cap);
  r.lo = p.window > 0 ? max(0, s.ctx + t0 - p.window + 1) : 0;
  r.sink_end = p.window > 0 ? min(min(p.sinks, r.lo), p.cap) : 0;
  r.ns = (r.sink_end + TK - 1) / TK;
  r.ft = r.lo / TK;
  const int end = (r.hi + TK - 1) / TK;
  if (r.ft <= r.ns) {
    r.ns = 0;
    r.ft = 0;
    r.count = end;
    if (r.sink_end > 0) r.count = max(end, (r.sink_end + TK - 1) / TK);
  } else {
    r.count = r.ns + max(0, end - r.ft);
  }
  if (r.count < 1) r.count = 1;
  return r;
}

__device__ __forceinline__ int paged_blocks(const PagedArgs &p, int n) { return (n + p.tpb - 1) / p.tpb; }

__device__ __forceinline__ int paged_units(const PagedArgs &p, int count) {
  return (count + p.min_tiles - 1) / p.min_tiles;
}

// Tiles of one kv head of a sequence, and the CTAs they take when every item is
// cut by itself into runs of min_tiles.
template <int TK>
__device__ __forceinline__ long long paged_cost(const PagedArgs &p, const PagedSeq &s, long long *units) {
  *units = 0;
  long long c = 0;
  for (int t0 = 0; t0 < s.n; t0 += p.tpb) {
    const int n = paged_range<TK>(p, s, t0, min(s.n, t0 + p.tpb)).count;
    c += n;
    *units += paged_units(p, n);
  }
  return c;
}

// This CTA's share: tiles [start, end) of the line, found in sequence b behind
// `off` of its tiles.  When the items cut one by one into runs of min_tiles fit
// the CTAs (cut set), a share is one such run, number `off` of sequence b: a
// small batch is not divided evenly for its own sake, and no CTA has the tail of
// one item and the head of the next.
struct PagedShare {
  long long start, end, per, off;
  long long head;  // tiles (or runs) of one kv head of sequence b
  int b;
  PagedSeq s;
  bool cut;
};

// Row starts that decrease may count rows twice: no bound on the blocks would hold and
// two CTAs could write one row, so that nothing of such a call is attended.
//
// Executed by all NT threads of the CTA; scratch: 2 NT / 32 + 5 long longs of shared memory.
template <int TK, int NT>
__device__ PagedShare paged_plan(const PagedArgs &p, long long *scratch) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int NW = NT / 32;
  long long *found = scratch + 2 * NW;
  // the first NT sequences stay in registers: most batches are read once
  PagedSeq first_s = {0, 0, 0};
  long long first = 0, first_u = 0, mine = 0, mine_u = 0;
  bool back = false;
  for (int b = tid; b < p.B; b += NT) {
    long long u;
    const PagedSeq s = paged_seq(p, b, blockIdx.x == 0, &back);
    const long long c = paged_cost<TK>(p, s, &u);
    if (b < NT) {
      first_s = s;
      first = c;
      first_u = u;
    }
    mine += c * p.Hkv;
    mine_u += u * p.Hkv;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    mine += __shfl_xor_sync(0xffffffffu, mine, o);
    mine_u += __shfl_xor_sync(0xffffffffu, mine_u, o);
  }
  const bool none = __syncthreads_or(back);
  if (lane == 0) {
    scratch[warp] = none ? 0 : mine;
    scratch[NW + warp] = none ? 0 : mine_u;
  }
  __syncthreads();
  long long total = 0, units = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    total += scratch[w];
    units += scratch[NW + w];
  }
  PagedShare sh;
  const long long nc = gridDim.x;
  sh.cut = units <= nc;
  if (sh.cut) total = units;
  sh.per = sh.cut ? 1 : (total + nc - 1) / nc;
  sh.start = min(total, sh.per * (long long)blockIdx.x);
  sh.end = min(total, sh.start + sh.per);
  sh.b = 0;
  sh.off = 0;
  if (sh.start >= sh.end) return sh;  // uniform over the CTA
  long long acc = 0;
  for (int base = 0; base < p.B; base += NT) {
    const int b = base + tid;
    PagedSeq s = first_s;
    long long head = sh.cut ? first_u : first;
    if (base > 0) {
      long long u = 0;
      head = 0;
      if (b < p.B) {
        s = paged_seq(p, b, false);
        head = paged_cost<TK>(p, s, &u);
        if (sh.cut) head = u;
      }
    }
    const long long c = head * p.Hkv;
    long long inc = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    __syncthreads();  // scratch is free again
    if (tid == 0) found[0] = -1;
    if (lane == 31) scratch[warp] = inc;
    __syncthreads();
    long long before = acc;
    for (int w = 0; w < warp; ++w) before += scratch[w];
    const long long lo = before + inc - c;
    if (c > 0 && sh.start >= lo && sh.start < lo + c) {
      found[0] = (long long)b << 32 | (unsigned)s.row0;
      found[1] = sh.start - lo;
      found[2] = head;
      found[3] = (long long)s.n << 32 | (unsigned)s.ctx;
    }
#pragma unroll
    for (int w = 0; w < NW; ++w) acc += scratch[w];
    __syncthreads();
    if (found[0] >= 0) {
      sh.b = (int)(found[0] >> 32);
      sh.s.row0 = (int)(unsigned)found[0];
      sh.off = found[1];
      sh.head = found[2];
      sh.s.n = (int)(found[3] >> 32);
      sh.s.ctx = (int)(unsigned)found[3];
      break;
    }
  }
  return sh;
}

// Walks the items of a share, one segment (an item's tiles [i0, i1)) at a time.
// Every thread that uses one walks alike.
template <int TK>
struct PagedWalk {
  const PagedArgs &p;
  long long pos, end, per;
  int b, h, t0;
  PagedSeq s;
  PagedRange r;
  int i0, i1;
  int last;  // the CTA in which the item ends

  __device__ __forceinline__ PagedWalk(const PagedArgs &pa, const PagedShare &sh)
      : p(pa), pos(sh.start), end(sh.end), per(sh.per), b(sh.b), h(0), t0(0), i0(0), i1(0), last(0) {
    if (pos >= end) return;
    s = sh.s;
    h = (int)(sh.off / sh.head);
    long long rem = sh.off - h * sh.head;
    for (;;) {
      r = paged_range<TK>(p, s, t0, t1());
      const int n = sh.cut ? paged_units(p, r.count) : r.count;
      if (rem < n) break;
      rem -= n;
      t0 += p.tpb;
    }
    if (sh.cut) {
      const int n = paged_units(p, r.count);  // the item's runs, alike to a tile
      i0 = (int)((long long)rem * r.count / n);
      i1 = (int)((long long)(rem + 1) * r.count / n);
      last = (int)blockIdx.x - (int)rem + n - 1;
      pos = 0;
      end = i1 - i0;
    } else {
      i0 = (int)rem;
      cut();
    }
  }
  __device__ __forceinline__ int t1() const { return min(s.n, t0 + p.tpb); }
  __device__ __forceinline__ bool valid() const { return pos < end; }
  __device__ __forceinline__ bool starts() const { return i0 == 0; }
  __device__ __forceinline__ bool ends() const { return i1 == r.count; }
  __device__ __forceinline__ void cut() {
    const long long left = end - pos;
    i1 = (long long)(r.count - i0) <= left ? r.count : i0 + (int)left;
    last = (int)((pos - i0 + r.count - 1) / per);
  }
  __device__ __forceinline__ void next() {
    pos += i1 - i0;
    if (pos >= end) return;
    i0 = 0;
    t0 += p.tpb;
    if (t0 >= s.n) {
      t0 = 0;
      if (++h == p.Hkv) {
        h = 0;
        long long u;
        do {
          s = paged_seq(p, ++b, false);
        } while (b + 1 < p.B && paged_cost<TK>(p, s, &u) == 0);
      }
    }
    r = paged_range<TK>(p, s, t0, t1());
    cut();
  }
};

// The page of key position j of sequence b: a table entry outside the pool is
// flagged and page 0 read in its place.
__device__ __forceinline__ int paged_page(const PagedArgs &p, int b, int j) {
  const int id = __ldg(&p.page_table[(size_t)b * p.max_pages + (j >> p.page_shift)]);
  if (id < 0 || id >= p.n_pages) {
    set_status(p.status, kStatusBadPage);
    return 0;
  }
  return id;
}

// A row's normalisation and log-sum from its sum S of weights over 2^M: zeros and -inf
// for a row that saw no key.  A NaN that it saw is in S and stays one in both: -inf
// would tell a caller who joins pieces by their log-sums to leave the piece out.
__device__ __forceinline__ float paged_inverse(float S) { return S == 0.f ? 0.f : 1.f / S; }
__device__ __forceinline__ float paged_lse(float M, float S) {
  return S == 0.f ? -INFINITY : (M + log2f(S)) * 0.6931471805599453f;
}

// Host side.

// A 2-D map over a pool of K or V pages as [rows, Dh] bf16, boxes of box_rows
// rows by at most 64 elements (tc.cu); false if the driver cannot encode it.
bool make_page_map(CUtensorMap *m, const void *base, int Dh, uint64_t rows, uint32_t box_rows);
bool paged_attn_items_ok(int B, int Hkv, int n_rows, int G);
size_t paged_attn_scratch_bytes(int B, int Hkv, int n_rows, int max_rows, int G, int Dh);
cudaError_t paged_set_attributes();
cudaError_t launch_paged_attn(const PagedArgs &a, const void *k_pages, const void *v_pages, int max_rows, void *scratch,
                              int sms, cudaStream_t s, bool pdl);

struct AppendArgs {
  int B, Hq, Hkv, Dh, page, page_shift, n_pages, max_pages, cap, n_rows;
  int rot, layout;              // rot 0: no rotation
  const unsigned long long *turns;  // [rot / 2] turns a position, 0.64 fixed point
  float scale;
  const int *row_start, *ctx_len, *page_table;  // row_start null: one row a sequence
  int ctx_add;                  // positions past ctx_len
  const void *q, *k, *v;        // bf16
  long long ldq, ldk, ldv, ldqo;
  long long khs, vhs;           // elements between heads of k and v
  void *q_out;
  uint16_t *k_pages, *v_pages;
  int *status;
  int q_f32;                    // q is fp32 (rounded to bf16 once, after the rotation)
};
cudaError_t launch_cache_append(const AppendArgs &a, cudaStream_t s, bool pdl);

}  // namespace mtp
