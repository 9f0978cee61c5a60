// Absorbed latent attention on pairs of CTAs, for sequences of many packed rows
// (tokens x heads), where the matrix products bind.
//
// A pair (a cluster of two, tcgen05 with cta_group::2) holds a block of 256 packed rows,
// 128 a CTA, and walks tiles of 128 keys:
//   S = Q K_i^T     256 x 128 over R + Dr elements: each CTA brings 64 of the keys
//   P = 2^(S - m)   one thread a row, P back over S as bf16
//   O += P V_i      256 x 256: each CTA brings 128 of the 256 elements of V
// The output of 128 rows and 512 elements would be all of tensor memory.  So an item is
// 256 of the R elements: a latent of 512 has two items a block, and its scores are formed
// twice, 1664 instead of 1088 products a (row, key).  Paired, a product of 64 cycles reads
// 6 KB of shared memory and not 8; alone, a CTA's reads would bind before its products.
//
// In graphs of 20, 64 x 4 rows of 128 heads over 1024-8192 keys take 327-335 us (350-383 a call among
// others): 503 GFLOP so counted, 260 us at the matrix rate; without loads 250 us.  What is left
// are keys on their way: six blocks of the ring in flight are what shared memory has room for
// (with four 407 us).  R = 256: 12 ragged chunks of 40 heads 340-352 us, 79% of the rate (a call
// among others 302-365, with the contexts drawn).
//
// P is rounded to bf16 for its product: half a step a weight, 2^-8 sum p |c| at most, about what
// the output's own rounding costs (against 64 bits 0.0019 relative, with fp32 weights
// 0.0017).  The rest of P as a second bf16 term would be one product more with V, 31% more
// of what binds here (R = 256: 44-47%).
//
// S_{i+1} is issued ahead of O += P_i V_i, so that the softmax of one tile runs under the
// scores of the next.  Queries take 144 of the 227 KB of shared memory (R = 512), so keys
// and values come apart: keys through a ring of 64 x 64 blocks that the scores use up as
// they arrive, values 128 x 128 at a time.
//
// Tensor memory (512 columns): O 256 | S_0 128 | S_1 128.  Warps 0-3 are the softmax, warp 4
// brings keys, warp 5 (of the first CTA) issues the products of both, warp 6 brings queries,
// warp 7 brings values and clears rows of them that no row sees.  Barriers that the issuer
// waits for lie in the first CTA and count both; those that products complete lie in both.
// Waits are at cluster scope, but for values that a CTA brings and clears for itself (zbar).
#include "internal.h"
#include "latent.cuh"
#include "paged_tc.cuh"
#include "latent_combine.cuh"

namespace mtp {

namespace {

constexpr int kTK = 128;            // keys per tile
constexpr int kRows = 128;          // packed rows of a CTA
constexpr int kDV = 256;            // elements of an item's output
constexpr int kThreads = 256;
constexpr int kKeys = 4, kIssuer = 5, kQuery = 6, kValues = 7;
constexpr unsigned kFull = 0xffffffffu;

template <int R>
struct Lay {
  static constexpr int NB = R / 64 + 1;             // 64-element blocks of a row, the rotary one last
  static constexpr int NG = (NB + 2) / 3;           // groups of blocks of the queries
  static constexpr int VH = R / kDV;                // items a block of rows
  static constexpr int QBLK = kRows * 128, QTILE = NB * QBLK;
  static constexpr int KBLK = 64 * 128;             // a block of keys: 64 rows of 128 bytes
  static constexpr int KST = R == 512 ? 6 : 9;
  static constexpr int VGRP = kTK * 128, VTILE = 2 * VGRP;  // 64 elements of 128 values; a CTA's 128 elements
  static constexpr int VST = R == 512 ? 1 : 2;
  static constexpr size_t SMEM = (size_t)QTILE + KST * KBLK + VST * VTILE + 512 + kNearItems * sizeof(PagedItem);
  __host__ __device__ static constexpr uint32_t S(int b) { return 256u + 128u * b; }
};

}  // namespace

template <int R>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    latent_attn_pair_kernel(const __grid_constant__ PagedTcParams sp) {
  trace_start(kTkLatentAttn);
  using L = Lay<R>;
  constexpr int NB = L::NB, KST = L::KST, VST = L::VST, VH = L::VH, NG = L::NG;
  const PagedArgs &p = sp.a;
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char *qbuf = smem, *kring = smem + L::QTILE, *vring = kring + KST * L::KBLK;
  uint64_t *k_full = reinterpret_cast<uint64_t *>(vring + VST * L::VTILE);
  uint64_t *k_empty = k_full + KST, *v_full = k_empty + KST, *v_empty = v_full + VST, *zbar = v_empty + VST;
  uint64_t *q_full = zbar + VST, *q_empty = q_full + NG, *drain = q_empty + 1, *o_empty = q_empty + 2;
  uint64_t *s_full = q_empty + 3, *p_full = s_full + 2, *o_done = s_full + 4;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(s_full + 6);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster_rank(), pair = blockIdx.x >> 1;

  if (tid == 0) {
    for (int s = 0; s < KST; ++s) {
      mbar_init(&k_full[s], 2);
      mbar_init(&k_empty[s], 1);
    }
    for (int s = 0; s < VST; ++s) {
      mbar_init(&v_full[s], 2);
      mbar_init(&v_empty[s], 1);
      mbar_init(&zbar[s], 1);
    }
    for (int g = 0; g < NG; ++g) mbar_init(&q_full[g], 2);
    mbar_init(q_empty, 1);
    mbar_init(drain, 1);
    mbar_init(o_empty, 8);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&s_full[b], 1);
      mbar_init(&p_full[b], 8);
      mbar_init(&o_done[b], 1);
    }
    fence_barrier_init();
  }
  if (warp == kIssuer) tmem_alloc_pair(tmem_slot, 512);
  if (warp == kKeys && lane == 0) prefetch_map(&sp.mk);
  if (warp == kValues && lane == 0) prefetch_map(&sp.mv);
  if (warp == kQuery && lane == 0) prefetch_map(&sp.mq);
  tc_fence_before();
  cluster_sync();  // both CTAs' barriers are set up
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dep_wait();
  trace_dep(kTkLatentAttn);
  grid_dep_launch();
  PagedItem *near = reinterpret_cast<PagedItem *>(smem + L::SMEM - kNearItems * sizeof(PagedItem));
  SmallPlan *plan = reinterpret_cast<SmallPlan *>(kring);  // (before the first copy)
  if (sp.small) plan_share<kTK, kThreads>(sp, sp.shares, pair, plan, near);
  PlanWalk<kTK, true> w = sp.small ? PlanWalk<kTK, true>(sp, pair, plan->start, near) : PlanWalk<kTK, true>(sp, pair, near);
  // (no share, no segment)
  if (tid == 0 && rank == 0) p.desc[pair].rows = 0;
  if (!sp.small && w.valid()) w.copy_near(sp, pair, near);
  fence_proxy_async_smem();  // the plan's memory is the copies' next
  __syncthreads();
  const int tpg = kRows / p.G;  // tokens of a CTA
  bool ok = true;

  if (warp == kKeys) {
    // -------------------------------------------------- keys: this CTA's 64 of a tile
    const int prow = min(p.page, 64), npc = 64 / prow;
    int s = 0;
    uint32_t ph = 1;  // (the first round finds the ring empty)
    for (; w.valid() && ok; w.next()) {
      // the piece of this lane in tile i: whether a row sees it, and its row of the pool
      auto locate = [&](int i, bool &need, int &y) {
        const int k0 = w.r.tile(i) * kTK + 64 * rank + lane * prow;
        need = lane < npc && w.r.any(k0, k0 + prow);
        y = need ? paged_page(p, w.b, k0) * p.page + (k0 & (p.page - 1)) : 0;
      };
      bool need, need_next = false;
      int y, y_next = 0;
      locate(w.i0, need, y);
      for (int i = w.i0; i < w.i1 && ok; ++i, need = need_next, y = y_next) {
        if (i + 1 < w.i1) locate(i + 1, need_next, y_next);  // its table entry loads under this tile's waits
        const uint32_t bytes = (uint32_t)(__popc(__ballot_sync(kFull, need)) * prow * 128);
        for (int x = 0; x < NB; ++x) {
          ok = __all_sync(kFull, mbar_wait_cluster(&k_empty[s], ph, p.status));
          if (!ok) break;
          const uint32_t bar = dsmem_addr(&k_full[s], 0);
          if (lane == 0) expect_tx_cluster(bar, bytes);
          __syncwarp();
          if (need) tma_2d_pair(kring + s * L::KBLK + lane * prow * 128, &sp.mk, 64 * x, y, bar);
          if (++s == KST) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
    }
    // Whatever happened, both CTAs' copies have landed before either leaves: the last round
    // of the ring (with no error the issuer has waited for them, and this costs nothing).
    if (rank == 0)
      for (int j = 0; j < KST; ++j) {
        if (--s < 0) {
          s = KST - 1;
          ph ^= 1u;
        }
        // the round before the first: never filled
        if (!mbar_wait_cluster(&k_full[s], ph ^ 1u, p.status)) break;
      }
  } else if (warp == kValues) {
    // -------------------------------------------------- values: this CTA's 128 elements of a
    // tile.  Rows that no row sees (past the last key, before the window, never loaded) may
    // hold anything, NaN too, which a weight of zero would not hold back: a tile that has
    // such rows is cleared before it is handed on.
    const int prow = min(p.page, kTK), npc = kTK / prow, pc = lane >> 1, grp = lane & 1;
    int s = 0;
    uint32_t ph = 1, zph = 0;
    for (; w.valid() && ok; w.next()) {
      const int x = kDV * (w.h % VH) + 128 * rank + 64 * grp;
      for (int i = w.i0; i < w.i1 && ok; ++i) {
        const int t0 = w.r.tile(i) * kTK, k0 = t0 + pc * prow;
        const bool need = pc < npc && w.r.any(k0, k0 + prow);
        const int y = need ? paged_page(p, w.b, k0) * p.page : 0;
        const uint32_t bytes = (uint32_t)(__popc(__ballot_sync(kFull, need)) * prow * 128);
        const bool whole = (t0 + kTK <= w.r.hi && t0 >= w.r.lo) || t0 + kTK <= w.r.sink_end;
        ok = __all_sync(kFull, mbar_wait_cluster(&v_empty[s], ph, p.status));
        if (!ok) break;
        unsigned char *tile = vring + s * L::VTILE, *dst = tile + grp * L::VGRP + pc * prow * 128;
        if (whole) {
          const uint32_t bar = dsmem_addr(&v_full[s], 0);
          if (lane == 0) expect_tx_cluster(bar, bytes);
          __syncwarp();
          if (need) tma_2d_pair(dst, &sp.mv, x, y, bar);
        } else {
          if (lane == 0) mbar_arrive_expect_tx(&zbar[s], bytes);
          __syncwarp();
          if (need) tma_2d(dst, &sp.mv, x, y, &zbar[s]);
          ok = __all_sync(kFull, mbar_wait(&zbar[s], zph >> s & 1u, p.status));
          zph ^= 1u << s;
          for (int e = lane; e < kTK * 8; e += 32)
            if (!w.r.sees(t0 + (e >> 3))) {
              *reinterpret_cast<uint4 *>(tile + e * 16) = make_uint4(0u, 0u, 0u, 0u);
              *reinterpret_cast<uint4 *>(tile + L::VGRP + e * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive_remote(&v_full[s], 0);  // (a release: the zeros are for both CTAs' products)
        }
        if (++s == VST) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
    if (rank == 0)  // as above
      for (int j = 0; j < VST; ++j) {
        if (--s < 0) {
          s = VST - 1;
          ph ^= 1u;
        }
        if (!mbar_wait_cluster(&v_full[s], ph ^ 1u, p.status)) break;
      }
  } else if (warp == kQuery) {
    // -------------------------------------------------- the blocks' queries
    if (lane == 0) {
      for (int seg = 0; w.valid(); w.next(), ++seg) {
        if (seg > 0 && !mbar_wait_cluster(q_empty, (uint32_t)(seg - 1) & 1u, p.status)) break;
        const int t = w.t0 + rank * tpg;
        const bool any = t < w.t1();  // else this CTA's rows are none: whatever lies there
        for (int x = 0; x < NB; ++x) {
          const uint32_t bar = dsmem_addr(&q_full[x / 3], 0);
          if (x % 3 == 0) expect_tx_cluster(bar, any ? (uint32_t)(min(3, NB - x) * tpg * p.G * 128) : 0u);
          if (any) tma_3d_pair(qbuf + x * L::QBLK, &sp.mq, 64 * x, w.h / VH * p.G, w.s.row0 + t, bar);
        }
      }
    }
    __syncwarp();
  } else if (warp == kIssuer) {
    // -------------------------------------------------- matrix products of both CTAs
    if (rank == 0) {
      // The whole warp walks and waits, one elected lane issues (paged_attn_tc.cu).
      constexpr uint32_t id_s = idesc_bf16_f32(2 * kRows, kTK), id_o = idesc_bf16_f32(2 * kRows, kDV) | (1u << 16);
      const uint32_t tm = __shfl_sync(kFull, tmem, 0);
      const uint64_t qd = sw128_kmajor_desc(smem_u32(qbuf)), kd = sw128_kmajor_desc(smem_u32(kring)),
                     vd = sw128_mnmajor_desc(smem_u32(vring), L::VGRP);
      const bool leader = elect_one();
      // A wait that gives up flags the status; the waits after it are skipped and
      // the rest is issued on whatever is there, so that no barrier is left short.
      auto await = [&](uint64_t *bar, uint32_t parity) {
        if (ok) ok = mbar_wait_cluster(bar, parity, p.status);
      };
      int it = 0, seg = 0, ks = 0, vs = 0;  // tiles whose scores were issued; stages
      uint32_t kph = 0, vph = 0, oph = 1;
      for (; __shfl_sync(kFull, w.valid(), 0); w.next(), ++seg) {
        const int nt = __shfl_sync(kFull, w.i1 - w.i0, 0);
        for (int g = 0; g < NG; ++g) await(&q_full[g], (uint32_t)seg & 1u);
        for (int i = 0; i <= nt; ++i) {
          if (i < nt) {
            const uint32_t d = tm + L::S(it & 1);
#pragma unroll 1
            for (int x = 0; x < NB; ++x) {
              await(&k_full[ks], kph);
              tc_fence_after();
              if (leader) {
                const uint64_t q = qd + (uint64_t)(x * (L::QBLK >> 4)), kk = kd + (uint64_t)(ks * (L::KBLK >> 4));
#pragma unroll
                for (int k = 0; k < 2; ++k) mma_bf16_pair(d, q + 2 * k, kk + 2 * k, id_s, x > 0 || k > 0);
                // (the last block's second half may be zeros; 12 ragged chunks, 40 heads of 256 + 32: 361 -> 349 us)
                if (x < NB - 1 || sp.rope > 32)
#pragma unroll
                  for (int k = 2; k < 4; ++k) mma_bf16_pair(d, q + 2 * k, kk + 2 * k, id_s, 1u);
                mma_commit_pair(&k_empty[ks]);
              }
              __syncwarp();
              if (++ks == KST) {
                ks = 0;
                kph ^= 1u;
              }
            }
            if (leader) {
              mma_commit_pair(&s_full[it & 1]);
              if (i == nt - 1) mma_commit_pair(q_empty);  // the block's last scores
            }
            __syncwarp();
            ++it;
          }
          if (i > 0) {
            const int j = it - (i < nt ? 2 : 1);  // the tile before
            if (i == 1) {
              await(o_empty, oph);
              oph ^= 1u;
            }
            await(&p_full[j & 1], (uint32_t)(j >> 1) & 1u);
            await(&v_full[vs], vph);
            tc_fence_after();
            if (leader) {
              const uint64_t v = vd + (uint64_t)(vs * (L::VTILE >> 4));
#pragma unroll
              for (int k = 0; k < kTK / 16; ++k)
                mma_ts_pair(tm, tm + L::S(j & 1) + 8 * k, v + (uint64_t)(k * (2048 >> 4)), id_o, k > 0 || i > 1);
              mma_commit_pair(&v_empty[vs]);
              mma_commit_pair(&o_done[j & 1]);
            }
            __syncwarp();
            if (++vs == VST) {
              vs = 0;
              vph ^= 1u;
            }
          }
        }
      }
      if (leader) mma_commit_pair(drain);  // nothing is in flight when the tensor memory is freed
      __syncwarp();
      mbar_wait_cluster(drain, 0, p.status);
    }
  } else {
    // -------------------------------------------------- softmax: a thread a row
    const int row = tid;
    const uint32_t lanebase = (uint32_t)(warp * 32) << 16, to = tmem + lanebase;
    int it = 0;
    for (; w.valid(); w.next()) {
      const int t1 = w.t1(), tg0 = w.t0 + rank * tpg, tg1 = min(t1, tg0 + tpg);  // this CTA's tokens
      const int tok = min(tg0 + row / p.G, t1 - 1), hq = w.h / VH * p.G + row % p.G, vh = w.h % VH;
      const bool live = row < (tg1 - tg0) * p.G && hq < p.Hq;
      const int pos = w.s.ctx + tok;
      const int rhi = min(pos + 1, p.cap), rlo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
      const int all_hi = min(w.s.ctx + tg0 + 1, p.cap);
      const int all_lo = p.window > 0 ? max(0, w.s.ctx + t1 - 1 - p.window + 1) : 0;
      float m = -INFINITY, l = 0.f;
      for (int i = w.i0; i < w.i1; ++i, ++it) {
        const int k0 = w.r.tile(i) * kTK;
        const bool whole = k0 + kTK <= all_hi && (k0 >= all_lo || k0 + kTK <= min(p.sinks, all_hi));
        const uint32_t ts = tmem + lanebase + L::S(it & 1);
        if (ok) ok = mbar_wait_cluster(&s_full[it & 1], (uint32_t)(it >> 1) & 1u, p.status);
        __syncwarp();
        if (i == w.i0) trace_mark(kTkLatentAttn, 0);
        tc_fence_after();
        uint32_t s[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32_async(ts + 32 * c, s + 32 * c);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 4; ++c) pin32(s + 32 * c);
        if (!whole) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int b = k0 + 32 * c;  // the row's view of 32 keys as bits
            const uint32_t see = below(rhi - b) & (~below(rlo - b) | below(p.sinks - b));
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(see >> e & 1u)) s[32 * c + e] = 0xff800000u;
          }
        }
        float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < 128; e += 2)
          x[(e >> 1) & 3] = max3(x[(e >> 1) & 3], __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
        const float mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) * p.scale_log2;
        if (__any_sync(kFull, live && mx > m + 8.f)) {
          const float n = fmaxf(m, mx);
          const float f = n == m ? 1.f : exp2f(m - n);
          m = n;
          l *= f;
          if (i > w.i0) {
            // The product of the tile before may still be running.  (A barrier for odd and
            // one for even tiles: this tile's scores show that the product two tiles before
            // is done, so that a parity never stands for two phases that are both possible.)
            if (ok) ok = mbar_wait_cluster(&o_done[(it - 1) & 1], (uint32_t)((it - 1) >> 1) & 1u, p.status);
            __syncwarp();
            tc_fence_after();
            rescale_columns<kDV / 32>(to, f);
          }
        }
        const float u = m == -INFINITY ? 0.f : m;
        const float2 sc2 = make_float2(p.scale_log2, p.scale_log2), nu2 = make_float2(-u, -u);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t pk[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            float2 y = fma2(make_float2(__uint_as_float(s[64 * c + 2 * e]), __uint_as_float(s[64 * c + 2 * e + 1])), sc2, nu2);
            y.x = ex2_approx(y.x);
            y.y = ex2_approx(y.y);
            sum[e & 1] = add2(sum[e & 1], y);
            pk[e] = pack2(y.x, y.y);
          }
          tmem_st32(ts + 32 * c, pk);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        // P and a rescaled O are handed over, all in tensor memory.  (With a release: 64 x 4 rows of
        // 128 heads 331 -> 339 us, 12 ragged chunks of 40 heads, R 256, 345 -> 425; passed on by an idle
        // warp of the second CTA, without stores to wait for, 339 and 393.)
        if (lane == 0) mbar_arrive_cluster_relaxed(dsmem_addr(&p_full[it & 1], 0));
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      }
      // ---- the block's output, or this segment's state
      if (ok) ok = mbar_wait_cluster(&o_done[(it - 1) & 1], (uint32_t)((it - 1) >> 1) & 1u, p.status);
      __syncwarp();
      tc_fence_after();
      trace_mark(kTkLatentAttn, 1);
      const bool whole_item = w.starts() && w.ends();
      const int slot = w.starts() ? 1 : 0;
      const int qrow = w.s.row0 + tok;
      const bool mine = live && in_bounds(qrow < p.n_rows, p.status);
      const float inv = paged_inverse(l);
      const size_t block = (size_t)pair * 2 + slot;
      const int srow = rank * tpg * p.G + row;  // in the pair's block
      write_row<kDV / 32, 2 * kRows>(
          to, 0, whole_item, mine ? static_cast<uint16_t *>(p.out) + (long long)qrow * p.ldo + hq * R + vh * kDV : nullptr, inv,
          p.part_o + block * (2 * kRows) * kDV, mine ? srow : -1, lane);
      if (mine) {
        if (!whole_item) {
          reinterpret_cast<float2 *>(p.part_ml)[block * (2 * kRows) + srow] = make_float2(m, l);
        } else if (p.lse && vh == 0) {
          p.lse[(size_t)qrow * p.Hq + hq] = paged_lse(m, l);
        }
      }
      if (tid == 0 && rank == 0 && w.starts() && !w.ends()) {
        PagedDesc d;
        d.row0 = w.s.row0 + w.t0;
        d.rows = (t1 - w.t0) * p.G;
        d.h = w.h;
        d.last_cta = w.last_cta();
        p.desc[pair] = d;
      }
      trace_mark(kTkLatentAttn, 2);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_relaxed(dsmem_addr(o_empty, 0));
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();  // neither CTA leaves while the other may still signal it
  tc_fence_after();
  if (warp == kIssuer) tmem_dealloc_pair(tmem, 512);
  trace_end(kTkLatentAttn);
}

// ---------------------------------------------------------------- host side

namespace {

// Blocks of 2 x 128 rows: heads split into hb runs of G, a CTA holds 128 / G tokens of one
// run; the fewest blocks at the mean number of rows a sequence.
void block_shape(int B, int n_rows, int H, int *G, int *hb) {
  const int n = (n_rows + B - 1) / B;
  long long best = -1;
  for (int r = 1; r <= H; ++r) {
    const int g = (H + r - 1) / r, t = 2 * (kRows / g);
    if ((H + g - 1) / g != r) continue;  // fewer runs of the same size do
    const long long blocks = (long long)r * ((n + t - 1) / t);
    if (best < 0 || blocks < best) {
      best = blocks;
      *G = g;
      *hb = r;
    }
  }
}

template <int R>
cudaError_t launch(const PagedTcParams &sp, int pairs, cudaStream_t s, bool pdl) {
  cudaError_t e = sp.small ? cudaSuccess : launch_paged_plan<kTK>(sp, pairs, s, pdl);
  if (e) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2 * pairs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Lay<R>::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  note_launch();
  e = cudaLaunchKernelEx(&cfg, latent_attn_pair_kernel<R>, sp);
  if (e) return e;
  return launch_latent_combine<kDV, 2 * kRows, Lay<R>::VH>(sp, pairs, 2 * pairs, s, pdl);
}

}  // namespace

// The first choice of block_shape is one run (latent_attn_scratch_bytes), of R / kDV items.
size_t latent_pair_scratch_bytes(int B, int n_rows, int H, int R) {
  return region_bytes(kPagedMaxCtas / 2, 2 * kRows, kDV) + paged_tc_plan_bytes(B, n_rows, 2 * (kRows / H), 2 * (R / kDV));
}

cudaError_t launch_latent_attn_pair(const LatentAttnArgs &la, void *scratch, int sms, cudaStream_t s, bool pdl) {
  const int n = (sms < kPagedMaxCtas ? sms : kPagedMaxCtas) / 2, w = la.a.Dh + la.Dr;
  PagedTcParams sp{};
  PagedArgs &a = sp.a;
  a = la.a;
  int hb;
  block_shape(a.B, a.n_rows, a.Hq, &a.G, &hb);
  a.Hkv = hb * (a.Dh / kDV);
  a.tpb = 2 * (kRows / a.G);
  // shares of at least 1 / 2 / 3 tiles (us, 128 heads): 1 x 2 rows over 512 14.7 / 16.5 / 16.7, 1 x 4
  // rows over 4096 20.2 / 20.0 / 21.1, 4 x 2 rows over 2048 22.5 / 22.5 / 22.6
  a.min_tiles = 1;
  sp.item_cost = 2;
  sp.rope = la.Dr;
  char *base = static_cast<char *>(scratch);
  bind_region(a, base, n, 2 * kRows);
  paged_tc_bind_plan(sp, base + region_bytes(kPagedMaxCtas / 2, 2 * kRows, kDV));
  paged_small_plan(sp, n);
  const uint64_t rows = (uint64_t)a.n_pages * a.page;
  if (!make_rows_map(&sp.mk, la.pages, w, rows, w, a.page < 64 ? a.page : 64) ||
      !make_rows_map(&sp.mv, la.pages, w, rows, w, a.page) ||
      !make_query_map(&sp.mq, a.q, w, a.Hq, a.n_rows, a.ldq, a.G, kRows / a.G))
    return cudaErrorNotSupported;
  return a.Dh == 512 ? launch<512>(sp, n, s, pdl) : launch<256>(sp, n, s, pdl);
}

cudaError_t latent_pair_set_attributes() {
  cudaError_t e = cudaFuncSetAttribute(latent_attn_pair_kernel<512>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)Lay<512>::SMEM);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(latent_attn_pair_kernel<256>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)Lay<256>::SMEM);
  return e;
}

MTP_TRACE_COLLECTOR(latent_attn_pair)

}  // namespace mtp
