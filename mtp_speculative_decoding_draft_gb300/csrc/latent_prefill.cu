// Attention of a prompt's rows over keys and values of each head, on the tensor cores.
//
// A head's key is its Dn plain elements beside the Dr rotated ones that all heads
// share; the two lie in different arrays and meet in shared memory only, so that no
// array of whole keys is ever written.  The frame is paged_attn_tc.cu's: a CTA holds
// two groups of 128 query rows of one head that take turns on the tensor core, the
// items are dealt out by its plan,
//   S_g = Q_g K_i^T     tcgen05.mma over Dn + Dr elements (a shared part of 32 lies in
//                       a block of 64, whose other half is not multiplied)
//   P_g = 2^(S_g - m)   one thread a row, P back over S as bf16
//   O_g += P_g V_i      tcgen05.mma, P from tensor memory, V row-major (MN-major)
// Queries of 192 elements take 96 KB of shared memory, which leaves 128 for 80 KB a tile.
// Three places of two blocks (128 keys x 128 elements) go round: K_i's plain part is in
// place i mod 3, V_i where K_{i-1}'s was; the shared parts have two places of their own.
// So K_i waits for V_{i-2} and V_i for K_{i-1}, and every operand lies in one piece: with
// blocks in a common ring, whose end parted a V tile now and then, the branches between the
// products cost the issuing warp 160 cycles an instruction of 64.  The scores begin with the
// shared part, which comes earlier.
//
// Bound by the products: 4096 rows over 12288, 32 heads, take 559-604 us in graphs of 20 (611-626 a
// call among others), 80% of the matrix rate at most, reading 4 KB of queries and 4 KB of keys from
// shared memory per 64 cycles, all that it gives.  Without softmax 509 us, without loads 574.
// Fresh prompts are bound by an item's start and end (16 of 1000 rows, 16 heads: 126 us for 43 us
// of products; an item 17 us, its five tiles 7).
//
// P is rounded to bf16 for its product: half a step a weight, 2^-8 sum p |v| at most (against 64 bits
// 0.0020-0.0024 relative, with fp32 weights 0.0017, the output's own rounding).  The rest of P
// as a second bf16 term would be 40% more products (Dn = Dv = 128, Dr 64), which bind here.
//
// Tensor memory (512 columns): S_0 | S_1 | O_0 | O_1, 128 each.  Warps 0-3 and 4-7 are
// the groups' softmax, warp 8 brings keys and values, warp 9 issues the products, warp 10 brings
// queries, warp 11 clears rows of V that no row sees.
#include "internal.h"
#include "latent.cuh"
#include "paged_tc.cuh"
#include "latent_combine.cuh"

namespace mtp {

namespace {

constexpr int kTK = 128;
constexpr int kThreads = 384;
// An item's queries, first scores and output in tiles.  us with 3 / 4 / 6: 16 prompts of 1000, 16 heads
// 126 / 126 / 133, 16 of 256 29.5 / 29.3 / 26.3, 3 of 1000 under a window of 6, 128 heads 120 / 117 / 115,
// 2048 rows over 10240, 16 heads 135 / 136 / 139.
constexpr int kItemCost = 4;
constexpr int kProducer = 8, kIssuer = 9, kQuery = 10, kClear = 11;
constexpr int kBlk = 128 * 128;  // bytes of a block: 128 rows of 128 bytes
constexpr unsigned kFull = 0xffffffffu;

template <int DN, int DV>
struct Lay {
  static constexpr int KB = DN / 64 + 1, VB = DV / 64;  // blocks of a tile's keys and values
  static constexpr int QTILE = KB * kBlk;               // a group's queries
  static constexpr int PLACE = (DN > DV ? DN : DV) / 64 * kBlk;
  static constexpr size_t SMEM = (size_t)2 * QTILE + 3 * PLACE + 2 * kBlk + 512 + kNearItems * sizeof(PagedItem);
};

struct PrefillParams {
  PagedTcParams tc;  // mk: the keys' and values' rows; mv: the shared key parts; mq: the queries
  int w;             // elements of a head in a row of keys and values
  int n_keys;
  const int *key_start;
};

}  // namespace

template <int DN, int DV>
__global__ void __launch_bounds__(kThreads, 1) latent_prefill_kernel(const __grid_constant__ PrefillParams pp) {
  trace_start(kTkLatentPrefill);
  using L = Lay<DN, DV>;
  constexpr int KB = L::KB, VB = L::VB;
  const PagedTcParams &sp = pp.tc;
  const PagedArgs &p = sp.a;
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char *qbuf = smem;  // [2 groups][blocks][128][128 B]
  unsigned char *places = smem + 2 * L::QTILE, *shared = places + 3 * L::PLACE;
  // of odd and even tiles: keys and values there, read, values to clear, shared parts there
  uint64_t *k_full = reinterpret_cast<uint64_t *>(shared + 2 * kBlk), *k_empty = k_full + 2, *v_full = k_full + 4,
           *v_empty = k_full + 6, *zbar = k_full + 8, *r_full = k_full + 10;
  uint64_t *q_full = r_full + 2, *q_empty = q_full + 1, *drain = q_full + 2;
  uint64_t *s_full = q_full + 3, *p_full = s_full + 2, *o_full = s_full + 4, *o_empty = s_full + 6, *p_half = s_full + 8;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(s_full + 10);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr uint32_t kS = 0, kO = 256;  // columns of S_0 and O_0, the second group's 128 further

  if (tid == 0) {
    for (int s = 0; s < 12; ++s) mbar_init(&k_full[s], 1);
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(drain, 1);
    for (int g = 0; g < 2; ++g) {
      mbar_init(&s_full[g], 1);
      mbar_init(&p_full[g], 4);
      mbar_init(&p_half[g], 4);
      mbar_init(&o_full[g], 1);
      mbar_init(&o_empty[g], 4);
    }
    fence_barrier_init();
  }
  if (warp == kIssuer) tmem_alloc(tmem_slot, 512);
  if (warp == kProducer && lane == 0) {
    prefetch_map(&sp.mk);
    prefetch_map(&sp.mv);
  }
  if (warp == kQuery && lane == 0) prefetch_map(&sp.mq);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dep_wait();
  trace_dep(kTkLatentPrefill);
  grid_dep_launch();
  PagedItem *near = reinterpret_cast<PagedItem *>(smem + L::SMEM - kNearItems * sizeof(PagedItem));
  SmallPlan *plan = reinterpret_cast<SmallPlan *>(places);  // (before the first copy)
  if (sp.small) plan_share<kTK, kThreads>(sp, sp.shares, blockIdx.x, plan, near);
  PlanWalk<kTK, true> w = sp.small ? PlanWalk<kTK, true>(sp, blockIdx.x, plan->start, near) : PlanWalk<kTK, true>(sp, blockIdx.x, near);
  // (no share, no segment)
  if (tid == 0) p.desc[blockIdx.x].rows = 0;
  if (!sp.small && w.valid()) w.copy_near(sp, blockIdx.x, near);
  fence_proxy_async_smem();  // the plan's memory is the copies' next
  __syncthreads();
  bool ok = true;

  // registers as in paged_attn_tc.cu: 384 x 168 = 256 x 216 + 128 x 72
  if (warp >= kProducer) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == kProducer) {
      // ------------------------------------------------ tiles of keys and values
      int it = 0;
      for (; w.valid() && ok; w.next()) {
        const int first = __ldcg(&pp.key_start[w.b]);
        if (lane == 0 && w.starts() && (first < 0 || (long long)first + w.s.ctx + w.s.n > pp.n_keys))
          set_status(p.status, kStatusBadCtx);
        for (int i = w.i0; i < w.i1 && ok; ++i, ++it) {
          const int t0 = w.r.tile(i) * kTK;
          // past the keys, either way, the copies read zeros
          const int y = (int)min(max((long long)first + t0, -(1ll << 30)), 1ll << 30);
          const bool whole = (t0 + kTK <= w.r.hi && t0 >= w.r.lo) || t0 + kTK <= w.r.sink_end;
          const int odd = it & 1, place = it % 3;
          if (lane == 0) {  // (V_{it-1} has waited for the scores of tile it - 2)
            mbar_arrive_expect_tx(&r_full[odd], kBlk);
            tma_2d(shared + odd * kBlk, &sp.mv, 0, y, &r_full[odd]);
          }
          __syncwarp();
          if (it >= 2) ok = mbar_wait(&v_empty[odd], (uint32_t)((it >> 1) - 1) & 1u, p.status);
          ok = __all_sync(kFull, ok);
          if (!ok) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(&k_full[odd], (KB - 1) * kBlk);
#pragma unroll
            for (int x = 0; x < KB - 1; ++x)
              tma_2d(places + place * L::PLACE + x * kBlk, &sp.mk, w.h * pp.w + 64 * x, y, &k_full[odd]);
          }
          __syncwarp();
          if (it >= 1) ok = mbar_wait(&k_empty[odd ^ 1], (uint32_t)((it - 1) >> 1) & 1u, p.status);
          ok = __all_sync(kFull, ok);
          if (lane == 0 && ok) {
            // a tile of V with rows to clear goes to the clearing warp first
            uint64_t *bar = whole ? &v_full[odd] : &zbar[odd];
            mbar_arrive_expect_tx(bar, VB * kBlk);
#pragma unroll
            for (int x = 0; x < VB; ++x)
              tma_2d(places + (it + 2) % 3 * L::PLACE + x * kBlk, &sp.mk, w.h * pp.w + DN + 64 * x, y, bar);
          }
          __syncwarp();
        }
      }
      if (!ok)  // let copies still in flight land before the CTA exits
        for (int i = max(0, it - 2); i <= it; ++i) {
          if (!mbar_wait(&r_full[i & 1], (uint32_t)(i >> 1) & 1u, p.status)) break;
          if (!mbar_wait(&k_full[i & 1], (uint32_t)(i >> 1) & 1u, p.status)) break;
          if (i < it && !mbar_wait(&v_full[i & 1], (uint32_t)(i >> 1) & 1u, p.status)) break;
        }
    } else if (warp == kClear) {
      // ------------------------------------------------ rows of V that no row sees
      uint32_t phases = 0;  // of odd and even tiles
      int it = 0;
      for (; w.valid() && ok; w.next()) {
        for (int i = w.i0; i < w.i1 && ok; ++i, ++it) {
          const int t0 = w.r.tile(i) * kTK, odd = it & 1;
          if ((t0 + kTK <= w.r.hi && t0 >= w.r.lo) || t0 + kTK <= w.r.sink_end) continue;
          ok = __all_sync(kFull, mbar_wait(&zbar[odd], phases >> odd & 1u, p.status));
          phases ^= 1u << odd;
          unsigned char *tile = places + (it + 2) % 3 * L::PLACE;
          for (int x = lane; x < kTK * 8; x += 32)
            if (!w.r.sees(t0 + (x >> 3)))
#pragma unroll
              for (int v = 0; v < VB; ++v) *reinterpret_cast<uint4 *>(tile + v * kBlk + x * 16) = make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&v_full[odd]);
        }
      }
    } else if (warp == kQuery) {
      // ------------------------------------------------ the blocks' queries
      if (lane == 0) {
        for (int seg = 0; w.valid(); w.next(), ++seg) {
          const int ng = w.t1() - w.t0 > 128 ? 2 : 1;
          if (seg > 0 && !mbar_wait(q_empty, (uint32_t)(seg - 1) & 1u, p.status)) break;
          mbar_arrive_expect_tx(q_full, (uint32_t)(ng * KB * kBlk));
          for (int g = 0; g < ng; ++g)
            for (int x = 0; x < KB; ++x)
              tma_3d(qbuf + g * L::QTILE + x * kBlk, &sp.mq, 64 * x, w.h, w.s.row0 + w.t0 + g * 128, q_full);
        }
      }
      __syncwarp();
    } else if (warp == kIssuer) {
      // ------------------------------------------------ matrix products
      // The whole warp walks and waits, one elected lane issues (paged_attn_tc.cu).
      constexpr uint32_t id_s = idesc_bf16_f32(128, 128), id_o = idesc_bf16_f32(128, DV) | (1u << 16);
      const uint32_t tm = __shfl_sync(kFull, tmem, 0);
      const uint64_t qd = sw128_kmajor_desc(smem_u32(qbuf)), kd = sw128_kmajor_desc(smem_u32(places)),
                     rd = sw128_kmajor_desc(smem_u32(shared)), vd = sw128_mnmajor_desc(smem_u32(places), kBlk);
      const bool leader = elect_one();
      // A wait that gives up flags the status; the waits after it are skipped and
      // the rest is issued on whatever is there, so that no barrier is left short.
      auto await = [&](uint64_t *bar, uint32_t parity) {
        if (ok) ok = mbar_wait(bar, parity, p.status);
      };
      int place = 0, seg = 0;  // K_i's place; V_{i-1} is in the second before it
      uint32_t n = 0, pph[2] = {0, 0}, oph[2] = {1, 1};  // (n: tiles whose scores were issued)
      for (; __shfl_sync(kFull, w.valid(), 0); w.next(), ++seg) {
        const int ng = __shfl_sync(kFull, w.t1() - w.t0 > 128 ? 2 : 1, 0), nt = __shfl_sync(kFull, w.i1 - w.i0, 0);
        await(q_full, (uint32_t)seg & 1u);
        for (int i = 0; i <= nt; ++i) {
          const uint32_t odd = n & 1u, last = n - 1u;  // K_n, V_{n-1}
          if (i > 0) await(&v_full[odd ^ 1u], (last >> 1) & 1u);
          const int vplace = place == 2 ? 0 : place + 1;  // (n - 1 + 2) mod 3
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            if (g >= ng) break;
            if (i > 0) {
              const uint64_t v = vd + (uint64_t)(vplace * (L::PLACE >> 4));
              if (i == 1) {
                await(&o_empty[g], oph[g]);
                oph[g] ^= 1u;
              }
              await(&p_half[g], pph[g]);
              tc_fence_after();
              if (leader) {
#pragma unroll
                for (int k = 0; k < kTK / 32; ++k)
                  mma_ts(tm + kO + 128 * g, tm + kS + 128 * g + 8 * k, v + (uint64_t)(k * (2048 >> 4)), id_o, k > 0 || i > 1);
              }
              await(&p_full[g], pph[g]);
              pph[g] ^= 1u;
              tc_fence_after();
              if (leader) {
#pragma unroll
                for (int k = kTK / 32; k < kTK / 16; ++k)
                  mma_ts(tm + kO + 128 * g, tm + kS + 128 * g + 8 * k, v + (uint64_t)(k * (2048 >> 4)), id_o, 1u);
                if (i == nt) mma_commit(&o_full[g]);
                if (g == ng - 1) mma_commit(&v_empty[odd ^ 1u]);
              }
            }
            if (i < nt) {
              const uint64_t q = qd + (uint64_t)(g * (L::QTILE >> 4)), kk = kd + (uint64_t)(place * (L::PLACE >> 4)),
                             rr = rd + (uint64_t)(odd * (kBlk >> 4));
              if (g == 0) {
                await(&r_full[odd], (n >> 1) & 1u);
                tc_fence_after();
              }
              if (leader) {
#pragma unroll
                for (int k = 0; k < 2; ++k)
                  mma_bf16(tm + kS + 128 * g, q + (uint64_t)(((KB - 1) * kBlk + k * 32) >> 4), rr + 2 * k, id_s, k > 0);
                if (sp.rope > 32)  // (2048 rows over 10240, 16 heads of 128 + 32: 136 us with the zeros, 133 without)
#pragma unroll
                  for (int k = 2; k < 4; ++k)
                    mma_bf16(tm + kS + 128 * g, q + (uint64_t)(((KB - 1) * kBlk + k * 32) >> 4), rr + 2 * k, id_s, 1u);
              }
              if (g == 0) {
                await(&k_full[odd], (n >> 1) & 1u);
                tc_fence_after();
              }
              if (leader) {
#pragma unroll
                for (int x = 0; x < KB - 1; ++x)
#pragma unroll
                  for (int k = 0; k < 4; ++k) {
                    const uint64_t off = (uint64_t)((x * kBlk + k * 32) >> 4);
                    mma_bf16(tm + kS + 128 * g, q + off, kk + off, id_s, 1u);
                  }
                mma_commit(&s_full[g]);
              }
            }
          }
          if (leader) {
            if (i < nt) mma_commit(&k_empty[odd]);
            if (i == nt - 1) mma_commit(q_empty);  // the block's last scores
          }
          __syncwarp();
          if (i < nt) {
            ++n;
            place = vplace;
          }
        }
      }
      if (leader) mma_commit(drain);  // nothing of this CTA is in flight when it frees its tensor memory
      __syncwarp();
      mbar_wait(drain, 0, p.status);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    // ------------------------------------------------ softmax: a thread a row
    const int g = warp >> 2, row = tid & 127;
    const uint32_t lanebase = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanebase + kS + 128 * g, to = tmem + lanebase + kO + 128 * g;
    int ns = 0, nseg = 0;
    for (; w.valid(); w.next()) {
      const int ntok = w.t1() - w.t0;
      if (g == 1 && ntok <= 128) continue;
      const int tg0 = w.t0 + g * 128, tg1 = min(w.t1(), tg0 + 128);  // the group's rows
      const int tok = min(tg0 + row, tg1 - 1);
      const bool live = tg0 + row < tg1;
      const int pos = w.s.ctx + tok;
      const int rhi = min(pos + 1, p.cap), rlo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
      const int all_hi = min(w.s.ctx + tg0 + 1, p.cap);
      const int all_lo = p.window > 0 ? max(0, w.s.ctx + tg1 - 1 - p.window + 1) : 0;
      float m = -INFINITY, l = 0.f;
      for (int i = w.i0; i < w.i1; ++i) {
        const int k0 = w.r.tile(i) * kTK;
        const bool whole = k0 + kTK <= all_hi && (k0 >= all_lo || k0 + kTK <= min(p.sinks, all_hi));
        if (ok) ok = mbar_wait(&s_full[g], (uint32_t)(ns++) & 1u, p.status);
        __syncwarp();
        if (i == w.i0) trace_mark(kTkLatentPrefill, 0);
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
            if (__all_sync(kFull, see == 0xffffffffu)) continue;  // on the diagonal half of them
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
            rescale_columns<DV / 32>(to, f);
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
            const float2 sc = make_float2(__uint_as_float(s[64 * c + 2 * e]), __uint_as_float(s[64 * c + 2 * e + 1]));
            float2 y = fma2(sc, sc2, nu2);
            y.x = ex2_approx(y.x);
            y.y = ex2_approx(y.y);
            sum[e & 1] = add2(sum[e & 1], y);
            pk[e] = pack2(y.x, y.y);
          }
          tmem_st32(ts + 32 * c, pk);
          // the product over the first half of the keys starts under the second half's exponentials
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(c == 0 ? &p_half[g] : &p_full[g]);
        }
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      }
      // ---- the block's output, or this segment's state
      if (ok) ok = mbar_wait(&o_full[g], (uint32_t)(nseg++) & 1u, p.status);
      __syncwarp();
      tc_fence_after();
      trace_mark(kTkLatentPrefill, 1);
      const bool whole_item = w.starts() && w.ends();
      const int slot = w.starts() ? 1 : 0;
      const int qrow = w.s.row0 + tok;
      const bool mine = live && in_bounds(qrow < p.n_rows, p.status);
      const float inv = paged_inverse(l);
      const size_t block = (size_t)blockIdx.x * 2 + slot;
      write_row<DV / 32, kPagedTcRows>(
          to, 0, whole_item, mine ? static_cast<uint16_t *>(p.out) + (long long)qrow * p.ldo + w.h * DV : nullptr, inv,
          p.part_o + block * kPagedTcRows * DV, mine ? g * 128 + row : -1, lane);
      if (mine) {
        if (!whole_item) {
          reinterpret_cast<float2 *>(p.part_ml)[block * kPagedTcRows + g * 128 + row] = make_float2(m, l);
        } else if (p.lse) {
          p.lse[(size_t)qrow * p.Hq + w.h] = paged_lse(m, l);
        }
      }
      if (tid == 0 && w.starts() && !w.ends()) {
        PagedDesc d;
        d.row0 = w.s.row0 + w.t0;
        d.rows = ntok;
        d.h = w.h;
        d.last_cta = w.last_cta();
        p.desc[blockIdx.x] = d;
      }
      trace_mark(kTkLatentPrefill, 2);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_empty[g]);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kIssuer) tmem_dealloc(tmem, 512);
  trace_end(kTkLatentPrefill);
}

// ---------------------------------------------------------------- host side

namespace {

constexpr int kTpb = 2 * 128;

cudaLaunchConfig_t config(int ctas, int threads, size_t smem, cudaStream_t s, cudaLaunchAttribute *attr, bool pdl) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cfg;
}

template <int DN, int DV>
cudaError_t launch(const PrefillParams &pp, int ctas, cudaStream_t s, bool pdl) {
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = config(ctas, kThreads, Lay<DN, DV>::SMEM, s, attr, pdl);
  note_launch();
  return cudaLaunchKernelEx(&cfg, latent_prefill_kernel<DN, DV>, pp);
}

template <int DN, int DV>
cudaError_t set_smem() {
  return cudaFuncSetAttribute(latent_prefill_kernel<DN, DV>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)Lay<DN, DV>::SMEM);
}

}  // namespace

size_t latent_prefill_scratch_bytes(int B, int n_rows, int H, int Dv) {
  return region_bytes(kPagedMaxCtas, kPagedTcRows, Dv) + paged_tc_plan_bytes(B, n_rows, kTpb, H);
}

cudaError_t launch_latent_prefill(const LatentPrefillArgs &lp, void *scratch, int sms, cudaStream_t s, bool pdl) {
  const int n = sms < kPagedMaxCtas ? sms : kPagedMaxCtas;
  PrefillParams pp{};
  PagedArgs &a = pp.tc.a;
  a = lp.a;
  a.tpb = kTpb;
  a.min_tiles = 2;  // of a share (one: 16 rows over 3000 19.1 us and 19.2, 256 rows of 16 heads 15.1 and 14.5)
  pp.tc.item_cost = kItemCost;
  pp.tc.rope = lp.Dr;
  pp.w = lp.Dn + lp.Dv;
  pp.n_keys = lp.n_keys;
  pp.key_start = lp.key_start;
  char *base = static_cast<char *>(scratch);
  bind_region(a, base, n, kPagedTcRows);
  paged_tc_bind_plan(pp.tc, base + region_bytes(kPagedMaxCtas, kPagedTcRows, a.Dh));
  paged_small_plan(pp.tc, n);
  if (!make_rows_map(&pp.tc.mk, lp.kv, (uint64_t)a.Hq * pp.w, lp.n_keys, lp.ldkv, kTK) ||
      !make_rows_map(&pp.tc.mv, lp.k_rope, lp.Dr, lp.n_keys, lp.ldkr, kTK) ||
      !make_query_map(&pp.tc.mq, a.q, lp.Dn + lp.Dr, a.Hq, a.n_rows, a.ldq, 1, 128))
    return cudaErrorNotSupported;
  cudaError_t e = pp.tc.small ? cudaSuccess : launch_paged_plan<kTK>(pp.tc, n, s, pdl);
  if (e) return e;
  if (lp.Dn == 128) e = lp.Dv == 128 ? launch<128, 128>(pp, n, s, pdl) : launch<128, 64>(pp, n, s, pdl);
  else e = lp.Dv == 128 ? launch<64, 128>(pp, n, s, pdl) : launch<64, 64>(pp, n, s, pdl);
  if (e) return e;
  return lp.Dv == 128 ? launch_latent_combine<128, kPagedTcRows, 1>(pp.tc, n, n, s, pdl)
                      : launch_latent_combine<64, kPagedTcRows, 1>(pp.tc, n, n, s, pdl);
}

cudaError_t latent_prefill_set_attributes() {
  cudaError_t e = set_smem<128, 128>();
  if (e == cudaSuccess) e = set_smem<128, 64>();
  if (e == cudaSuccess) e = set_smem<64, 128>();
  if (e == cudaSuccess) e = set_smem<64, 64>();
  return e;
}

MTP_TRACE_COLLECTOR(latent_prefill)

}  // namespace mtp
