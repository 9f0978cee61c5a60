// Attention of a chunk of new tokens over a paged K/V cache: the streaming
// kernel (few query rows per K/V head) and the kernel that joins partial items.
//
//   o = sum_j softmax_j(scale q.k_j) v_j over the keys j that the row sees
//
// For the k + 1 candidate rows of a verification the work is bound by the
// cache's bytes: every visible K/V row is read once, and the group's query
// rows (tokens x G, up to 64 a block; 32 with heads of 128) share it.  Each CTA takes an equal share
// of the line of 64-key tiles (paged.cuh).  A producer warp brings the pages'
// pieces of a tile by TMA into a three-stage ring; four compute warps hold
// their rows' states in registers:
//   S = Q K^T   mma.m16n8k16 (bf16 operands, fp32 accumulators)
//   online softmax on the accumulator fragments, base 2; the running maximum
//               moves only when a row's maximum grew by more than 2^8, so the
//               accumulators are seldom rescaled
//   O += P V    with P in bf16, as an operand beside bf16 values has to be; the
//               row's sum takes the unrounded weights in fp32.  Blocks of 16
//               packed rows, whose matrix pipe waits for bytes, carry P in two
//               terms, what the first rounding left as a second operand (2^-16 of
//               a weight is lost, not 2^-8): 64 x 4 rows over 1024-8192 keys 198.3
//               -> 199.8 us, 4 rows over 4096 13.3 -> 13.6, and outputs as far from
//               64 bits as their own rounding (0.0017 against 0.0023 in all).
//               Wider blocks keep one term: a second costs 32 x 30 rows over 16384
//               3.5%, blocks of 64 rows of heads of 64 16%
// Warps split a tile by rows (16 each) and what is left of them by keys, and
// merge through shared memory at the end of a segment.  Two CTAs an SM, 96 KB of
// tiles in flight each: 32 sequences of 6 rows over 16384 keys run at 6.6 TB/s,
// 97-98% of the copy rate; at 16 packed rows the tensor pipe is at 23%, so that the
// warp-level product is no limit at these row counts.
#include "internal.h"
#include "paged_combine.cuh"
#include "paged_tc.cuh"

namespace mtp {

namespace {

constexpr int kTK = 64;      // keys per tile
constexpr int kStages = 3;
constexpr int kCW = 4;       // compute warps
constexpr int kThreads = 32 * (kCW + 1);
constexpr unsigned kFull = 0xffffffffu;

template <int DH, int RG>
struct Lay {
  static constexpr int RB = 16 * RG;                   // packed query rows of a block
  static constexpr int KG = kCW / RG;                  // key groups
  static constexpr int KW = kTK / KG;                  // keys of a warp per tile
  static constexpr int TERMS = RG == 1 ? 2 : 1;        // bf16 terms of a weight
  static constexpr int NB = DH >= 64 ? DH / 64 : 1;    // boxes across a head
  static constexpr int PITCH = DH >= 64 ? 128 : 64;    // bytes of a row in a box
  static constexpr int BOX = kTK * PITCH;
  static constexpr int STAGE = 2 * NB * BOX;           // K boxes, then V boxes
  static constexpr int RING = kStages * STAGE;
  static constexpr int QB = RB * DH * 2;
  static constexpr int SD = RB <= 32 ? 32 : 16;        // head dims merged at a time
  static constexpr int WLD = SD + 4;
  static constexpr int MRG = KG * RB * WLD * 4;        // warps' output slices
  static constexpr int ML = (KG * RB * 2 + 2 * RB) * 4;
  static constexpr int U = QB > MRG + ML ? QB : MRG + ML;  // queries, then the merge
  static constexpr int TAIL = 2 * kStages * 8 + 16 * 8;
  static constexpr size_t SMEM = (size_t)RING + U + TAIL;
};

__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}

__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}

// Byte offset of (row r, 16-byte chunk c of the head) in `rows`-row boxes with
// the 128-byte swizzle (64-byte for heads of 32).
template <int DH>
__device__ __forceinline__ uint32_t at(int r, int c, int rows) {
  if (DH == 32) return (uint32_t)(r * 64 + (((c ^ (r >> 1)) & 3) << 4));
  return (uint32_t)((c >> 3) * rows * 128 + r * 128 + (((c ^ r) & 7) << 4));
}

struct StreamParams {
  CUtensorMap mk, mv;  // the pools as [n_pages * Hkv * page, Dh] bf16
  PagedArgs a;
};

}  // namespace

template <int DH, int RG>
__global__ void __launch_bounds__(kThreads, 2) paged_attn_kernel(const __grid_constant__ StreamParams sp) {
  trace_start(kTkPagedAttn);
  using L = Lay<DH, RG>;
  constexpr int RB = L::RB, NB = L::NB, KS = DH / 16, ND = DH / 8, NT = L::KW / 8;
  constexpr int VX = L::TERMS;  // V fragments in hand: the terms' products of one accumulator lie 2 VX apart
  const PagedArgs &p = sp.a;
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char *ring = smem;
  unsigned char *ubuf = smem + L::RING;
  uint64_t *full = reinterpret_cast<uint64_t *>(ubuf + L::U);
  uint64_t *empty = full + kStages;
  long long *scratch = reinterpret_cast<long long *>(empty + kStages);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kCW);
    }
    fence_barrier_init();
  }
  grid_dep_wait();
  trace_dep(kTkPagedAttn);
  grid_dep_launch();
  const PagedShare sh = paged_plan<kTK, kThreads>(p, scratch);  // its barriers publish the mbarriers
  trace_mark(kTkPagedAttn, 0);  // share known
  if (tid == 0) p.desc[blockIdx.x].rows = 0;
  if (sh.start >= sh.end) {
    trace_end(kTkPagedAttn);
    return;
  }
  __syncthreads();

  bool ok = true;
  PagedWalk<kTK> w(p, sh);
  int it = 0;
  if (warp == kCW) {
    // ------------------------------------------------ producer
    const int prow = min(p.page, kTK);            // rows of a piece: a page, or a tile of it
    const int npc = (kTK / prow) * NB * 2;        // pieces of a tile (at most 16)
    const int pc = lane / (2 * NB), hb = (lane % (2 * NB)) % NB, isv = (lane % (2 * NB)) / NB;
    int issued = 0;
    for (; w.valid() && ok; w.next()) {
      // the piece of this lane in tile i: whether a row sees it, and its row of the pool
      auto locate = [&](int i, bool &need, int &y) {
        const int k0 = w.r.tile(i) * kTK + pc * prow;
        need = lane < npc && w.r.any(k0, k0 + prow);
        y = need ? (paged_page(p, w.b, k0) * p.Hkv + w.h) * p.page + (k0 & (p.page - 1)) : 0;
      };
      bool need, need_next = false;
      int y, y_next = 0;
      locate(w.i0, need, y);
      for (int i = w.i0; i < w.i1 && ok; ++i, ++it, need = need_next, y = y_next) {
        const int s = it % kStages;
        if (i + 1 < w.i1) locate(i + 1, need_next, y_next);  // its table entry loads under this tile's wait
        if (it >= kStages) ok = mbar_wait(&empty[s], (uint32_t)((it / kStages) - 1) & 1u, p.status);
        ok = __all_sync(kFull, ok);
        if (!ok) break;
        const int cnt = __popc(__ballot_sync(kFull, need));
        if (lane == 0) mbar_arrive_expect_tx(&full[s], (uint32_t)(cnt * prow * L::PITCH));
        __syncwarp();
        if (need) {
          unsigned char *dst = ring + (size_t)s * L::STAGE + (isv * NB + hb) * L::BOX + pc * prow * L::PITCH;
          const CUtensorMap *m = isv ? &sp.mv : &sp.mk;
          asm volatile(
              "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
              "[%4];" ::"r"(smem_u32(dst)),
              "l"(reinterpret_cast<uint64_t>(m)), "r"(64 * hb), "r"(y), "r"(smem_u32(&full[s]))
              : "memory");
        }
        issued = it + 1;
      }
    }
    if (!ok)  // let copies still in flight land before the CTA exits
      for (int i = max(0, issued - kStages); i < issued; ++i)
        if (!mbar_wait(&full[i % kStages], (uint32_t)(i / kStages) & 1u, p.status)) break;
    trace_end(kTkPagedAttn);
    return;
  }

  // ------------------------------------------------ compute warps
  const int kg = warp % L::KG, rg = warp / L::KG;
  const int gq = lane >> 2, tq = lane & 3;
  const uint32_t qb = smem_u32(ubuf);
  const int arow = (lane & 7) + 8 * ((lane >> 3) & 1), acol = lane >> 4;
  float *wst = reinterpret_cast<float *>(ubuf);
  float *ml = reinterpret_cast<float *>(ubuf + L::MRG);  // [KG][RB][2]
  float *rowm = ml + L::KG * RB * 2, *rowl = rowm + RB;

  for (; w.valid(); w.next()) {
    const int t1 = w.t1(), ntok = t1 - w.t0, rows = ntok * p.G;
    const int row0 = w.s.row0 + w.t0;
    // ---- the block's queries: row (token, head of the group), zero past the last
    for (int idx = tid; idx < RB * (DH / 8); idx += 32 * kCW) {
      const int r = idx / (DH / 8), c = idx % (DH / 8);
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (r < rows)
        v = __ldcg(reinterpret_cast<const uint4 *>(p.q + (long long)(row0 + r / p.G) * p.ldq +
                                                   (w.h * p.G + r % p.G) * DH + c * 8));
      *reinterpret_cast<uint4 *>(ubuf + at<DH>(r, c, RB)) = v;
    }
    named_sync(1, 32 * kCW);
    trace_mark(kTkPagedAttn, 1);  // queries staged
    uint32_t qf[KS][4];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) ldsm4(qb + at<DH>(rg * 16 + arow, 2 * ks + acol, RB), qf[ks]);

    // what this lane's rows see: positions [rlo, rhi) and the sinks below them
    int rhi[2], rlo[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int pos = w.s.ctx + w.t0 + min((rg * 16 + gq + 8 * e) / p.G, ntok - 1);
      rhi[e] = min(pos + 1, p.cap);
      rlo[e] = p.window > 0 ? max(0, pos - p.window + 1) : 0;
    }
    const int all_hi = min(w.s.ctx + w.t0 + 1, p.cap);                              // every row sees below this ..
    const int all_lo = p.window > 0 ? max(0, w.s.ctx + t1 - 1 - p.window + 1) : 0;  // .. from this on

    float o[ND][4], m[2], l[2];
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
#pragma unroll
    for (int n = 0; n < ND; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;

    for (int i = w.i0; i < w.i1; ++i, ++it) {
      const int s = it % kStages;
      if (ok) ok = mbar_wait(&full[s], (uint32_t)(it / kStages) & 1u, p.status);
      ok = __all_sync(kFull, ok);
      const int R0 = kg * L::KW;                 // this warp's keys of the tile
      const int key0 = w.r.tile(i) * kTK + R0;
      if (ok && w.r.any(key0, key0 + L::KW)) {
        const uint32_t kb = smem_u32(ring + (size_t)s * L::STAGE), vb = kb + NB * L::BOX;
        const bool whole = key0 + L::KW <= all_hi && (key0 >= all_lo || key0 + L::KW <= min(p.sinks, all_hi));
        float sc[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ks += 2) {
          uint32_t kf[NT][4];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            ldsm4(kb + at<DH>(R0 + 8 * nt + (lane & 7), 2 * (ks + (lane >> 4)) + ((lane >> 3) & 1), kTK), kf[nt]);
#pragma unroll
          for (int kx = 0; kx < 2; ++kx)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma(sc[nt], qf[ks + kx], kf[nt][2 * kx], kf[nt][2 * kx + 1]);
        }
        float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float a = sc[nt][e] * p.scale_log2, b = sc[nt][2 + e] * p.scale_log2;
            if (!whole) {
              const int j = key0 + 8 * nt + 2 * tq + e;
              if (!(j < rhi[0] && (j >= rlo[0] || j < p.sinks))) a = -INFINITY;
              if (!(j < rhi[1] && (j >= rlo[1] || j < p.sinks))) b = -INFINITY;
            }
            sc[nt][e] = a;
            sc[nt][2 + e] = b;
            x0 = fmaxf(x0, a);
            x1 = fmaxf(x1, b);
          }
        x0 = fmaxf(x0, __shfl_xor_sync(kFull, x0, 1));
        x1 = fmaxf(x1, __shfl_xor_sync(kFull, x1, 1));
        x0 = fmaxf(x0, __shfl_xor_sync(kFull, x0, 2));
        x1 = fmaxf(x1, __shfl_xor_sync(kFull, x1, 2));
        // the maximum in use moves only when it has to
        if (__any_sync(kFull, x0 > m[0] + 8.f || x1 > m[1] + 8.f)) {
          const float n0 = fmaxf(m[0], x0), n1 = fmaxf(m[1], x1);
          const float f0 = n0 == m[0] ? 1.f : exp2f(m[0] - n0), f1 = n1 == m[1] ? 1.f : exp2f(m[1] - n1);
          m[0] = n0;
          m[1] = n1;
          l[0] *= f0;
          l[1] *= f1;
#pragma unroll
          for (int n = 0; n < ND; ++n) {
            o[n][0] *= f0;
            o[n][1] *= f0;
            o[n][2] *= f1;
            o[n][3] *= f1;
          }
        }
        const float u0 = m[0] == -INFINITY ? 0.f : m[0], u1 = m[1] == -INFINITY ? 0.f : m[1];
        uint32_t pa[NT / 2][4], pr[NT / 2][4];  // bf16 weights, and with two terms what the rounding left of them
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float a = ex2_approx(sc[nt][0] - u0), b = ex2_approx(sc[nt][1] - u0);
          const float c = ex2_approx(sc[nt][2] - u1), d = ex2_approx(sc[nt][3] - u1);
          l[0] += a + b;  // this lane's columns; the quad's sums meet at the end
          l[1] += c + d;
          const uint32_t ab = pack2(a, b), cd = pack2(c, d);
          pa[nt >> 1][2 * (nt & 1)] = ab;
          pa[nt >> 1][2 * (nt & 1) + 1] = cd;
          if (L::TERMS == 2) {
            pr[nt >> 1][2 * (nt & 1)] = pack2(a - bf16_lo(ab), b - bf16_hi(ab));
            pr[nt >> 1][2 * (nt & 1) + 1] = pack2(c - bf16_lo(cd), d - bf16_hi(cd));
          }
        }
        // ---- O += P V.  Rows of V that no row of the block sees (past the
        // last key, before the window, never loaded) may hold anything, NaN
        // too: their fragments are cleared.
#pragma unroll
        for (int kk = 0; kk < NT / 2; ++kk) {
          uint32_t z0 = 0xffffffffu, z1 = 0xffffffffu;
          if (!whole) {
            const int j = key0 + 16 * kk + 2 * tq;
            z0 = (w.r.sees(j) ? 0xffffu : 0u) | (w.r.sees(j + 1) ? 0xffff0000u : 0u);
            z1 = (w.r.sees(j + 8) ? 0xffffu : 0u) | (w.r.sees(j + 9) ? 0xffff0000u : 0u);
          }
#pragma unroll
          for (int n = 0; n < ND; n += 2 * VX) {
            uint32_t v[VX][4];
#pragma unroll
            for (int x = 0; x < VX; ++x) {
              ldsm4t(vb + at<DH>(R0 + 16 * kk + (lane & 7) + 8 * ((lane >> 3) & 1), n + 2 * x + (lane >> 4), kTK), v[x]);
              if (!whole) {
                v[x][0] &= z0;
                v[x][1] &= z1;
                v[x][2] &= z0;
                v[x][3] &= z1;
              }
            }
#pragma unroll
            for (int x = 0; x < 2 * VX; ++x) mma(o[n + x], pa[kk], v[x >> 1][2 * (x & 1)], v[x >> 1][2 * (x & 1) + 1]);
            if (L::TERMS == 2)
#pragma unroll
              for (int x = 0; x < 2 * VX; ++x) mma(o[n + x], pr[kk], v[x >> 1][2 * (x & 1)], v[x >> 1][2 * (x & 1) + 1]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
    }

    trace_mark(kTkPagedAttn, 2);  // last tile done
    // ---- merge the key groups; write the output, or this segment's state
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] += __shfl_xor_sync(kFull, l[e], 1);
      l[e] += __shfl_xor_sync(kFull, l[e], 2);
    }
    named_sync(1, 32 * kCW);  // every warp is done with the queries
    if (tq == 0) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float *x = ml + (kg * RB + rg * 16 + gq + 8 * e) * 2;
        x[0] = m[e];
        x[1] = l[e];
      }
    }
    named_sync(1, 32 * kCW);
    const bool whole_item = w.starts() && w.ends();
    const int slot = w.starts() ? 1 : 0;
    for (int r = tid; r < rows; r += 32 * kCW) {
      float M = -INFINITY, S = 0.f;
#pragma unroll
      for (int g = 0; g < L::KG; ++g) M = fmaxf(M, ml[(g * RB + r) * 2]);
#pragma unroll
      for (int g = 0; g < L::KG; ++g) {
        float *x = ml + (g * RB + r) * 2;
        const float f = x[0] == -INFINITY ? 0.f : exp2f(x[0] - M);
        S = fmaf(x[1], f, S);
        x[0] = f;  // from here on the group's weight
      }
      rowm[r] = M;
      rowl[r] = paged_inverse(S);
      if (whole_item) {
        if (p.lse)
          p.lse[(size_t)(row0 + r / p.G) * p.Hq + w.h * p.G + r % p.G] = paged_lse(M, S);
      } else {
        float *x = p.part_ml + (((size_t)blockIdx.x * 2 + slot) * RB + r) * 2;
        x[0] = M;
        x[1] = S;
      }
    }
#pragma unroll
    for (int d0 = 0; d0 < DH; d0 += L::SD) {
      named_sync(1, 32 * kCW);
#pragma unroll
      for (int n = d0 / 8; n < (d0 + L::SD) / 8; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          *reinterpret_cast<float2 *>(wst + (kg * RB + rg * 16 + gq + 8 * e) * L::WLD + 8 * n - d0 + 2 * tq) =
              make_float2(o[n][2 * e], o[n][2 * e + 1]);
      named_sync(1, 32 * kCW);
      for (int idx = tid; idx < rows * (L::SD / 4); idx += 32 * kCW) {
        const int r = idx / (L::SD / 4), c = 4 * (idx % (L::SD / 4));
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int g = 0; g < L::KG; ++g) {
          const float f = ml[(g * RB + r) * 2];
          const float4 v = *reinterpret_cast<const float4 *>(wst + (g * RB + r) * L::WLD + c);
          a.x = fmaf(v.x, f, a.x);
          a.y = fmaf(v.y, f, a.y);
          a.z = fmaf(v.z, f, a.z);
          a.w = fmaf(v.w, f, a.w);
        }
        if (whole_item) {
          const float f = rowl[r];
          const long long off = (long long)(row0 + r / p.G) * p.ldo + (w.h * p.G + r % p.G) * DH + d0 + c;
          if (in_bounds(row0 + r / p.G < p.n_rows, p.status)) {
            if (p.out_f32)
              *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + off) =
                  make_float4(a.x * f, a.y * f, a.z * f, a.w * f);
            else
              *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + off) =
                  make_uint2(pack2(a.x * f, a.y * f), pack2(a.z * f, a.w * f));
          }
        } else {
          *reinterpret_cast<float4 *>(p.part_o + (((size_t)blockIdx.x * 2 + slot) * RB + r) * DH + d0 + c) = a;
        }
      }
    }
    if (tid == 0 && w.starts() && !w.ends()) {
      PagedDesc d;
      d.row0 = row0;
      d.rows = rows;
      d.h = w.h;
      d.last_cta = w.last;
      p.desc[blockIdx.x] = d;
    }
    named_sync(1, 32 * kCW);  // the buffer is the next block's queries
  }
  trace_end(kTkPagedAttn);
}

// Joins the segments of the items that end in a later CTA than they start in, in
// key order: eight rows of the item that starts in a CTA a block, a warp a row.
constexpr int kCombineRows = 8;

template <int PER>
struct Vec;
template <>
struct Vec<1> {
  typedef float T;
};
template <>
struct Vec<2> {
  typedef float2 T;
};
template <>
struct Vec<4> {
  typedef float4 T;
};

template <int DH>
__global__ void __launch_bounds__(32 * kCombineRows)
    paged_combine_kernel(const __grid_constant__ PagedArgs p, int block_rows) {
  trace_start(kTkPagedCombine);
  grid_dep_wait();
  grid_dep_launch();
  const int per = block_rows / kCombineRows, cta = blockIdx.x / per;
  constexpr int PER = DH / 32;
  const int lane = threadIdx.x & 31;
  const PagedDesc d = p.desc[cta];
  const int r = (blockIdx.x % per) * kCombineRows + (threadIdx.x >> 5);
  if (r < d.rows) {
    const int nseg = d.last_cta - cta + 1;
    auto seg = [&](int i) { return ((size_t)(cta + i) * 2 + (i == 0 ? 1 : 0)) * block_rows + r; };
    // The statistics and the first outputs are requested together: for up to
    // kBatch segments the row takes one round trip behind its description.
    constexpr int kBatch = 8;
    using V = typename Vec<PER>::T;
    V v[kBatch];
    auto fetch = [&](int i0) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (i0 + i < nseg) v[i] = __ldcg(reinterpret_cast<const V *>(p.part_o + seg(i0 + i) * DH + lane * PER));
    };
    auto stats = [&](int i) { return __ldcg(reinterpret_cast<const float2 *>(p.part_ml + seg(i) * 2)); };
    float2 x = lane < nseg ? stats(lane) : make_float2(-INFINITY, 0.f);
    fetch(0);
    float M = x.x;
    for (int i = lane + 32; i < nseg; i += 32) M = fmaxf(M, stats(i).x);
    M = warp_max(M);
    float S = 0.f, a[PER];
#pragma unroll
    for (int e = 0; e < PER; ++e) a[e] = 0.f;
    for (int i0 = 0; i0 < nseg; i0 += 32) {
      if (i0 > 0) x = i0 + lane < nseg ? stats(i0 + lane) : make_float2(-INFINITY, 0.f);
      const float f = x.x == -INFINITY ? 0.f : exp2f(x.x - M);
      S += warp_sum(x.y * f);
#pragma unroll
      for (int half = 0; half < 32; half += kBatch) {
        if (i0 + half >= nseg) break;
        if (i0 + half > 0) fetch(i0 + half);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const float g = __shfl_sync(kFull, f, half + i);
          if (i0 + half + i < nseg) {
            const float *y = reinterpret_cast<const float *>(&v[i]);
#pragma unroll
            for (int e = 0; e < PER; ++e) a[e] = fmaf(y[e], g, a[e]);
          }
        }
      }
    }
    const float inv = paged_inverse(S);
    const int row = d.row0 + r / p.G, hq = d.h * p.G + r % p.G;
    const long long off = (long long)row * p.ldo + hq * DH + lane * PER;
    if (in_bounds(row < p.n_rows, p.status)) {
#pragma unroll
      for (int e = 0; e < PER; ++e) {
        if (p.out_f32) static_cast<float *>(p.out)[off + e] = a[e] * inv;
        else static_cast<__nv_bfloat16 *>(p.out)[off + e] = __float2bfloat16_rn(a[e] * inv);
      }
      if (lane == 0 && p.lse) p.lse[(size_t)row * p.Hq + hq] = paged_lse(M, S);
    }
  }
  trace_end(kTkPagedCombine);
}

// ---------------------------------------------------------------- host side

namespace {

constexpr int kMaxSms = kPagedMaxCtas;

// Packed rows of the widest streaming block, and so of the largest sequence that the
// streaming kernel takes where there is a tensor-core kernel (heads of 64 and 128).  In
// graphs of 20 calls (us, streaming / tensor cores), 32 / 8 heads of 128:
//   sequences x keys   16 rows      32 rows      36 rows      64 rows
//   1 x 512             9.9 / 17.5  12.1 / 17.6  17.4 / 17.6  18.4 / 17.8
//   8 x 512            11.3 / 21.4  14.0 / 21.7  20.2 / 22.4  21.9 / 22.4
//   8 x 4096             33 / 41      41 / 42      61 / 42      66 / 43
//   64 x 1024-8192      193 / 204    217 / 205    364 / 205    391 / 211
// past 32 rows the streaming block of 64 rows has no registers left and its products
// bind.  16 / 4 heads of 64:
//   1 x 512             8.3 / 15.9   9.1 / 15.9  12.1 / 16.0  12.5 / 16.0
//   8 x 4096           13.8 / 23.7  16.2 / 24.2  22.4 / 24.0  23.8 / 24.4
//   64 x 1024-8192       58 / 79      69 / 79     105 / 79     112 / 83
// where small batches would lose up to a third with the bound of heads of 128.  The
// lengths are the device's, so that the host cannot tell the two apart.
constexpr int stream_rows(int Dh) { return Dh == 128 ? 32 : 64; }

cudaLaunchConfig_t config(dim3 grid, int threads, size_t smem, cudaStream_t s, cudaLaunchAttribute *attr, bool pdl) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cfg;
}

template <int DH, int RG>
cudaError_t launch_stream(const StreamParams &sp, int ctas, cudaStream_t s, bool pdl) {
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = config(dim3(ctas), kThreads, Lay<DH, RG>::SMEM, s, attr, pdl);
  note_launch();
  return cudaLaunchKernelEx(&cfg, paged_attn_kernel<DH, RG>, sp);
}

template <int DH>
cudaError_t launch_rows(const StreamParams &sp, int rb, int ctas, cudaStream_t s, bool pdl) {
  if (rb == 16) return launch_stream<DH, 1>(sp, ctas, s, pdl);
  if constexpr (stream_rows(DH) == 64)
    if (rb == 64) return launch_stream<DH, 4>(sp, ctas, s, pdl);
  return launch_stream<DH, 2>(sp, ctas, s, pdl);
}

template <int DH>
cudaError_t launch_combine(const PagedArgs &a, int ctas, int rows, cudaStream_t s, bool pdl) {
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = config(dim3(ctas * (rows / kCombineRows)), 32 * kCombineRows, 0, s, attr, pdl);
  note_launch();
  return cudaLaunchKernelEx(&cfg, paged_combine_kernel<DH>, a, rows);
}

template <int DH, int RG>
cudaError_t set_smem() {
  return cudaFuncSetAttribute(paged_attn_kernel<DH, RG>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)Lay<DH, RG>::SMEM);
}

template <int DH>
cudaError_t set_head() {
  cudaError_t e = set_smem<DH, 1>();
  if (e == cudaSuccess) e = set_smem<DH, 2>();
  if constexpr (stream_rows(DH) == 64)
    if (e == cudaSuccess) e = set_smem<DH, 4>();
  return e;
}

}  // namespace

cudaError_t paged_set_attributes() {
  cudaError_t e = set_head<32>();
  if (e == cudaSuccess) e = set_head<64>();
  if (e == cudaSuccess) e = set_head<128>();
  if (e == cudaSuccess) e = paged_tc_set_attributes();
  return e;
}

// Packed rows of the largest sequence, as far as the host knows.
static long long packed_rows(int n_rows, int max_rows, int G) {
  return (long long)(max_rows > 0 && max_rows < n_rows ? max_rows : n_rows) * G;
}

// A call with a sequence of more packed rows than a streaming block holds goes to
// the tensor cores whole: one kernel takes any mixture.  Heads of 32, for which there is
// no such kernel (its tiles are rows of 128 bytes), stay.  A call whose largest sequence
// the host does not know (max_rows 0) is chosen for by all its rows: decoding batches
// lose 7% with heads of 128 and up to 44% with heads of 64 that way (the 16-row columns
// above), chunks taken for decoding would lose up to six times.
static bool wants_tc(long long packed, int Dh) { return packed > stream_rows(Dh) && Dh != 32; }

bool paged_attn_items_ok(int B, int Hkv, int n_rows, int G) { return paged_tc_items_ok(B, n_rows, 2 * (128 / G), Hkv); }

size_t paged_attn_scratch_bytes(int B, int Hkv, int n_rows, int max_rows, int G, int Dh) {
  if (!wants_tc(packed_rows(n_rows, max_rows, G), Dh)) return region_bytes(2 * kMaxSms, stream_rows(Dh), Dh);
  return region_bytes(kMaxSms, kPagedTcRows, Dh) + paged_tc_plan_bytes(B, n_rows, 2 * (128 / G), Hkv);
}

cudaError_t launch_paged_attn(const PagedArgs &args, const void *k_pages, const void *v_pages, int max_rows, void *scratch,
                              int sms, cudaStream_t s, bool pdl) {
  const long long packed = packed_rows(args.n_rows, max_rows, args.G);
  const uint64_t rows = (uint64_t)args.n_pages * args.Hkv * args.page;
  const int n = sms < kMaxSms ? sms : kMaxSms;
  char *base = static_cast<char *>(scratch);
  cudaError_t e;
  if (wants_tc(packed, args.Dh)) {
    if (args.out_f32) return cudaErrorInvalidValue;  // the draft's, whose rows all fit a streaming block
    PagedTcParams tp;
    tp.a = args;
    tp.a.tpb = 2 * (128 / args.G);
    tp.a.min_tiles = 2;
    bind_region(tp.a, base, n, kPagedTcRows);
    paged_tc_bind_plan(tp, base + region_bytes(kMaxSms, kPagedTcRows, args.Dh));
    if (!make_page_map(&tp.mk, k_pages, args.Dh, rows, args.page) ||
        !make_page_map(&tp.mv, v_pages, args.Dh, rows, args.page) ||
        !make_query_map(&tp.mq, args.q, args.Dh, args.Hq, args.n_rows, args.ldq, args.G, 128 / args.G))
      return cudaErrorNotSupported;
    if ((e = launch_paged_attn_tc(tp, n, s, pdl))) return e;
    static_assert(kMaxSms <= kMaxDescs, "a description a CTA");
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = config(dim3(6 * n), kCombineThreads, 0, s, attr, pdl);
    note_launch();
    return args.Dh == 64 ? cudaLaunchKernelEx(&cfg, paged_combine_tc_kernel<64, kPagedTcRows>, tp.a, n)
                         : cudaLaunchKernelEx(&cfg, paged_combine_tc_kernel<128, kPagedTcRows>, tp.a, n);
  }
  StreamParams sp;
  sp.a = args;
  const int rb = packed <= 16 ? 16 : packed <= 32 ? 32 : 64, ctas = 2 * n;
  sp.a.tpb = rb / args.G;
  // runs of 2, 4, 6 and 8 tiles (us, 32 / 8 heads of 128, 4 rows): 1 x 512 keys 9.6, 10.3,
  // 11.8, 11.8; 1 x 4096 14.2, 13.7, 14.1, 15.2; 1 x 8192 18.2, 16.3, 16.4, 17.8; 2 x 4096
  // 16.3, 14.4, 15.5, 17.0; 8 x 1024 15.8, 15.8, 14.7, 14.7; 4 x 4096 and 1 x 16384 within 7%
  sp.a.min_tiles = 4;
  bind_region(sp.a, base, ctas, rb);
  const uint32_t box = (uint32_t)(args.page < kTK ? args.page : kTK);
  if (!make_page_map(&sp.mk, k_pages, args.Dh, rows, box) || !make_page_map(&sp.mv, v_pages, args.Dh, rows, box))
    return cudaErrorNotSupported;
  if (args.Dh == 32) e = launch_rows<32>(sp, rb, ctas, s, pdl);
  else if (args.Dh == 64) e = launch_rows<64>(sp, rb, ctas, s, pdl);
  else e = launch_rows<128>(sp, rb, ctas, s, pdl);
  if (e) return e;
  if (args.Dh == 32) return launch_combine<32>(sp.a, ctas, rb, s, pdl);
  if (args.Dh == 64) return launch_combine<64>(sp.a, ctas, rb, s, pdl);
  return launch_combine<128>(sp.a, ctas, rb, s, pdl);
}

MTP_TRACE_COLLECTOR(paged_attn)

}  // namespace mtp
