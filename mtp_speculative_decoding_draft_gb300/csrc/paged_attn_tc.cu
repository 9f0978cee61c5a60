// Attention of a chunk of new tokens over a paged K/V cache: the tensor-core
// kernel, for calls with a sequence of more packed rows (tokens x G) than the
// streaming kernel's block.
//
// Bound by the two matrix products and by the exponentials between them.  A CTA
// holds a block of two groups of 128 packed query rows of one K/V head; the
// groups take turns on the tensor core, so that one group's softmax runs under
// the other group's products:
//   S_g = Q_g K_i^T     tcgen05.mma, both operands in shared memory by TMA
//   P_g = 2^(S_g - m)   one thread a row: S from tensor memory, the maximum and
//                       the sum in registers, P back over S as bf16 (the sum takes
//                       the unrounded weights; a second term would be a third
//                       product where the first two are the bound: half as much again)
//   O_g += P_g V_i      tcgen05.mma, P from tensor memory, V as it lies in its
//                       pages (row-major keys: the MN-major form of operand B)
// S_g i+1 is issued behind O_g += P_g V_i, so when a group's scores arrive its
// accumulator is at rest, and the group's own threads rescale it: only when a
// row's maximum grew by more than 2^8.  4096 rows over 12288 keys, 32 / 8 heads of
// 128: 580 us by itself (pages in L2 or not), 620 us timed in turn with a plain form;
// 1660 and 1550 TFLOP/s, 89 and 83% of the library's rate for one large product.  A
// tile takes about 2900 cycles, of which both groups' products take 2048: the chain
// of a group, 1100 cycles from its scores to its weights and 1550 until its next
// scores, is what is left.  A segment costs about 9000 cycles beside its tiles: 4500
// for the output, 2500 for the walk to the next, the rest for its first scores and
// last product.
//
// Tensor memory (512 columns): S_0 | S_1 | O_0 | O_1, 128 each; P_g lies in the
// first half of S_g.  Warps 0-3 and 4-7 are the groups' softmax, warp 8 brings
// pages by TMA into a ring of K and V tiles, warp 9 issues the products, warp 10
// brings the next block's queries as soon as the last scores are done, warp 11
// clears rows of V.
#include "internal.h"
#include "paged.cuh"
#include "paged_tc.cuh"
#include "tcgen05_ops.cuh"

// The order of the line (paged.cuh): with equal contiguous shares each CTA walks
// the blocks of a few K/V heads one after another, and all heads of the batch are
// read at the same time; past L2's size every block reads its keys from DRAM
// again (24 ragged sequences of 315 MB of keys: 455 us).  The plan deals the items
// out like cards instead, item t * CTAs + c to CTA c's t-th place, so that the
// blocks of one K/V head run side by side.
namespace mtp {

namespace {

constexpr int kTK = 128;          // keys per tile
constexpr int kThreads = 384;     // three warpgroups: the registers move between whole ones
// Tiles that a segment costs besides its own, 0 / 3 / 6 / 12 (us): 4 x 2048 rows from
// nothing 155-163 / 138-141 / 140-144 / 146-149, 24 x 512 over 3584 538 / 528 / 526 / 527, 16 x
// 128 over 512 54 / 50 / 44 / 44, 40 rows over 8192 30.6 / 26.4 / 26.4 / 26.9; 24 ragged
// chunks 312-317 with each
constexpr int kItemCost = 6;
constexpr int kProducer = 8, kIssuer = 9, kQuery = 10, kClear = 11;
constexpr unsigned kFull = 0xffffffffu;

template <int DH>
struct Lay {
  static constexpr int NB = DH / 64;               // 64-dim halves of a head
  static constexpr int HALF = 128 * 128;           // bytes of a half: 128 rows of 128 bytes
  static constexpr int TILE = NB * HALF;           // a K or V tile, or a group's queries
  static constexpr int STAGES = DH == 128 ? 5 : 8;
  static constexpr int RING = STAGES * TILE;
  static constexpr size_t SMEM = (size_t)2 * TILE + RING + 512;
  __host__ __device__ static constexpr uint32_t S(int g) { return 128u * g; }
  __host__ __device__ static constexpr uint32_t O(int g) { return 256u + 128u * g; }
};

constexpr int kPlanThreads = 512;

}  // namespace

// One CTA: the items of the batch, their order, and where each share starts.  One item may
// hold the starts of many shares (one user's few blocks over all CTAs), so that the shares
// look for their items and not the other way round: a thread that wrote 19 starts in turn
// took 2.2 of a plan's 4.9 us.
template <int TK>
__global__ void __launch_bounds__(kPlanThreads)
    paged_tc_plan_kernel(const __grid_constant__ PagedTcParams sp, int ctas) {
  trace_start(kTkPagedPlan);
  constexpr int kNear = 1024;  // sequences that are kept in shared memory
  __shared__ long long scratch[kPlanThreads / 32];
  __shared__ int near_blocks[kNear + 1];
  __shared__ PagedSeq near_seq[kNear];
  __shared__ PagedItem round_items[kPlanThreads];
  const PagedArgs &p = sp.a;
  const int tid = threadIdx.x;
  const bool near = p.B <= kNear;
  grid_dep_wait();
  trace_dep(kTkPagedPlan);
  grid_dep_launch();
  // ---- blocks of each sequence, and all tiles
  long long nblk = 0, total = 0, incl;
  bool back = false;
  for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    long long c = 0, u;
    int nb = 0;
    if (b < p.B) {
      const PagedSeq s = paged_seq(p, b, true, &back);
      c = paged_cost<TK>(p, s, &u);
      nb = paged_blocks(p, s.n);
      if (near) near_seq[b] = s;
    }
    const long long sum = block_scan<kPlanThreads>(nb, &incl, scratch);
    if (b < p.B) {
      const int before = (int)(nblk + incl - nb);
      if (near) near_blocks[b] = before;
      else sp.blocks[b] = before;
    }
    nblk += sum;
    total += block_scan<kPlanThreads>((c + (long long)nb * sp.item_cost) * p.Hkv, &incl, scratch);
  }
  if (tid == 0) {
    if (near) near_blocks[p.B] = (int)nblk;
    else sp.blocks[p.B] = (int)nblk;
  }
  // (the barrier also publishes the blocks)  The list has room for the blocks of
  // disjoint rows: row starts that decrease leave no items, and no share any tiles
  if (__syncthreads_or(back)) nblk = total = 0;
  // items fit 31 bits (the host checks), so that places and sequences divide in 32
  const unsigned N = (unsigned)(nblk * p.Hkv), q = (N + ctas - 1) / ctas, places = q * ctas;
  const long long per = max((long long)p.min_tiles, (total + ctas - 1) / ctas);
  // shares without tiles
  for (int c = tid; c < ctas; c += kPlanThreads)
    if (c * per >= total) {
      sp.start[c].end = 0;
      sp.start[c].per = per;
    }
  auto first_item = [&](int b) { return (unsigned)(near ? near_blocks[b] : __ldcg(&sp.blocks[b])) * p.Hkv; };
  // ---- items, dealt out: place i = c * q + t holds item t * CTAs + c
  long long before = 0;
  for (unsigned base = 0; base < places; base += kPlanThreads) {
    const unsigned i = base + tid, m = i < places ? (i % q) * ctas + i / q : N;
    PagedItem it{};
    if (m < N) {
      // the sequence: the last whose first item is not past m
      int lo = 0, hi = p.B;  // first_item(lo) <= m < first_item(hi)
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (first_item(mid) <= m) lo = mid;
        else hi = mid;
      }
      const PagedSeq s = near ? near_seq[lo] : paged_seq(p, lo, false);
      const int nb = paged_blocks(p, s.n), off = (int)(m - first_item(lo));
      it.b = lo;
      it.h = off / nb;
      it.t0 = (off % nb) * p.tpb;
      it.count = paged_range<TK>(p, s, it.t0, min(s.n, it.t0 + p.tpb)).count;
      it.row0 = s.row0;
      it.n = s.n;
      it.ctx = s.ctx;
    }
    const int len = it.count > 0 ? sp.item_cost + it.count : 0;  // on the line
    const long long sum = block_scan<kPlanThreads>(len, &incl, scratch);
    it.first = before + incl - len;
    round_items[tid] = it;
    if (i < places) sp.items[i] = it;
    __syncthreads();
    // ---- the shares that start inside this round's items
    for (int c = tid; c < ctas; c += kPlanThreads) {
      const long long at = c * per;
      if (at < before || at >= before + sum) continue;
      int lo = 0, hi = kPlanThreads;  // the last item that starts at or before it (gaps start where their next item does)
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (round_items[mid].first <= at) lo = mid;
        else hi = mid;
      }
      PagedStart st{};
      st.item = round_items[lo];
      st.end = min(total, at + per);
      st.per = per;
      st.i = (int)(base + lo);
      sp.start[c] = st;
    }
    before += sum;
    __syncthreads();  // the round's items are read
  }
  trace_end(kTkPagedPlan);
}

template <int DH>
__global__ void __launch_bounds__(kThreads, 1) paged_attn_tc_kernel(const __grid_constant__ PagedTcParams sp) {
  trace_start(kTkPagedAttnTc);
  using L = Lay<DH>;
  constexpr int NB = L::NB, ST = L::STAGES;
  const PagedArgs &p = sp.a;
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char *qbuf = smem;                      // [2 groups][halves][128][128 B]
  unsigned char *ring = smem + 2 * L::TILE;
  uint64_t *bars = reinterpret_cast<uint64_t *>(ring + L::RING);
  uint64_t *full = bars, *empty = bars + ST, *zbar = bars + 2 * ST;  // ring
  uint64_t *q_full = bars + 3 * ST, *q_empty = q_full + 1, *drain = q_full + 2;
  uint64_t *s_full = q_full + 3, *p_full = s_full + 2, *o_full = s_full + 4, *o_empty = s_full + 6,
           *p_half = s_full + 8;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(s_full + 10);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < ST; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&zbar[s], 1);
    }
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
  grid_dep_wait();
  trace_dep(kTkPagedAttnTc);
  grid_dep_launch();
  PlanWalk<kTK> w(sp, blockIdx.x);
  if (tid == 0) p.desc[blockIdx.x].rows = 0;
  if (!w.valid()) {  // the same for the whole CTA
    trace_end(kTkPagedAttnTc);
    return;
  }
  if (warp == kIssuer) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const int tpg = 128 / p.G, rpg = tpg * p.G;      // tokens and packed rows of a group
  bool ok = true;

  // The launch gives every thread 168 registers, 384 x 168 = 64512 in all; the
  // third warpgroup needs few, a softmax row in registers needs more:
  // 256 x 216 + 128 x 72 = 64512.
  if (warp >= kProducer) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == kProducer) {
      // ------------------------------------------------ pages into the ring
      const int prow = min(p.page, kTK);             // rows of a piece: one page
      const int npc = (kTK / prow) * NB;             // pieces of a tile (at most 16)
      const int pc = lane / NB, hb = lane % NB;
      int it = 0;
      for (; w.valid() && ok; w.next()) {
        // the piece of this lane in tile i: whether a row sees it, and its row of the pool
        auto locate = [&](int i, bool &need, int &y) {
          const int k0 = w.r.tile(i) * kTK + pc * prow;
          need = lane < npc && w.r.any(k0, k0 + prow);
          y = need ? (paged_page(p, w.b, k0) * p.Hkv + w.h) * p.page : 0;
        };
        bool need, need_next = false;
        int y, y_next = 0;
        locate(w.i0, need, y);
        for (int i = w.i0; i < w.i1 && ok; ++i, need = need_next, y = y_next) {
          const int t0 = w.r.tile(i) * kTK;
          if (i + 1 < w.i1) locate(i + 1, need_next, y_next);  // its table entry loads under this tile's waits
          const uint32_t bytes = (uint32_t)(__popc(__ballot_sync(kFull, need)) * prow * 128);
          const bool whole = (t0 + kTK <= w.r.hi && t0 >= w.r.lo) || t0 + kTK <= w.r.sink_end;
          for (int isv = 0; isv < 2 && ok; ++isv, ++it) {
            const int s = it % ST;
            if (it >= ST) ok = mbar_wait(&empty[s], (uint32_t)((it / ST) - 1) & 1u, p.status);
            ok = __all_sync(kFull, ok);
            if (!ok) break;
            // a V tile with rows to clear goes to the clearing warp first
            uint64_t *bar = isv && !whole ? &zbar[s] : &full[s];
            unsigned char *dst = ring + (size_t)s * L::TILE;
            if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
            __syncwarp();
            if (need) tma_2d(dst + hb * L::HALF + pc * prow * 128, isv ? &sp.mv : &sp.mk, 64 * hb, y, bar);
          }
        }
      }
      if (!ok)  // let copies still in flight land before the CTA exits
        for (int i = max(0, it - ST); i < it; ++i)
          if (!mbar_wait(&full[i % ST], (uint32_t)(i / ST) & 1u, p.status)) break;
    } else if (warp == kClear) {
      // ------------------------------------------------ rows of V that no row sees
      // (past the last key, before the window, never loaded) may hold anything,
      // NaN too: in a tile that has such rows they are cleared before the tile is
      // handed on
      uint32_t phases = 0;  // a bit a stage
      int it = 1;
      for (; w.valid() && ok; w.next()) {
        for (int i = w.i0; i < w.i1 && ok; ++i, it += 2) {
          const int t0 = w.r.tile(i) * kTK, s = it % ST;
          if ((t0 + kTK <= w.r.hi && t0 >= w.r.lo) || t0 + kTK <= w.r.sink_end) continue;
          ok = __all_sync(kFull, mbar_wait(&zbar[s], phases >> s & 1u, p.status));
          phases ^= 1u << s;
          unsigned char *tile = ring + (size_t)s * L::TILE;
          for (int x = lane; x < kTK * 8; x += 32)
            if (!w.r.sees(t0 + (x >> 3)))
#pragma unroll
              for (int hb = 0; hb < NB; ++hb)
                *reinterpret_cast<uint4 *>(tile + hb * L::HALF + x * 16) = make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&full[s]);
        }
      }
    } else if (warp == kQuery) {
      // ------------------------------------------------ the blocks' queries
      if (lane == 0) {
        for (int seg = 0; w.valid(); w.next(), ++seg) {
          const int ng = w.t1() - w.t0 > tpg ? 2 : 1;
          if (seg > 0 && !mbar_wait(q_empty, (uint32_t)(seg - 1) & 1u, p.status)) break;
          mbar_arrive_expect_tx(q_full, (uint32_t)(ng * NB * rpg * 128));
          for (int g = 0; g < ng; ++g)
            for (int x = 0; x < NB; ++x)
              tma_3d(qbuf + g * L::TILE + x * L::HALF, &sp.mq, 64 * x, w.h * p.G, w.s.row0 + w.t0 + g * tpg, q_full);
        }
      }
      __syncwarp();
    } else if (warp == kIssuer) {
      // ------------------------------------------------ matrix products
      // The whole warp walks and waits, one elected lane issues.  Loop bounds,
      // addresses and the tensor-memory base are warp-uniform by construction
      // (shuffles and votes), so that the operands sit in uniform registers: an
      // issue loop under `lane == 0` took about 125 cycles an instruction, twice
      // what the instruction itself takes.
      constexpr uint32_t id_s = idesc_bf16_f32(128, 128), id_o = idesc_bf16_f32(128, DH) | (1u << 16);
      const uint32_t tm = __shfl_sync(kFull, tmem, 0);
      const uint64_t qd = sw128_kmajor_desc(smem_u32(qbuf)), kd = sw128_kmajor_desc(smem_u32(ring)),
                     vd = sw128_mnmajor_desc(smem_u32(ring), L::HALF);
      const bool leader = elect_one();
      // A wait that gives up flags the status; the waits after it are skipped and
      // the rest is issued on whatever is there, so that no barrier is left short.
      auto await = [&](uint64_t *bar, uint32_t parity) {
        if (ok) ok = mbar_wait(bar, parity, p.status);
      };
      int ks = 0, vs = 0, seg = 0;  // stages of K_i and V_{i-1}
      uint32_t kph = 0, vph = 0, pph[2] = {0, 0}, oph[2] = {1, 1};
      for (; __shfl_sync(kFull, w.valid(), 0); w.next(), ++seg) {
        const int ng = __shfl_sync(kFull, w.t1() - w.t0 > tpg ? 2 : 1, 0), nt = __shfl_sync(kFull, w.i1 - w.i0, 0);
        await(q_full, (uint32_t)seg & 1u);
        for (int i = 0; i <= nt; ++i) {
          if (i < nt) await(&full[ks], kph);
          if (i > 0) await(&full[vs], vph);
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            if (g >= ng) break;
            if (i > 0) {
              const uint64_t v = vd + (uint64_t)(vs * (L::TILE >> 4));
              if (i == 1) {
                await(&o_empty[g], oph[g]);
                oph[g] ^= 1u;
              }
              await(&p_half[g], pph[g]);
              tc_fence_after();
              if (leader) {
#pragma unroll
                for (int k = 0; k < kTK / 32; ++k)
                  mma_ts(tm + L::O(g), tm + L::S(g) + 8 * k, v + (uint64_t)(k * (2048 >> 4)), id_o, k > 0 || i > 1);
              }
              await(&p_full[g], pph[g]);
              pph[g] ^= 1u;
              tc_fence_after();
              if (leader) {
#pragma unroll
                for (int k = kTK / 32; k < kTK / 16; ++k)
                  mma_ts(tm + L::O(g), tm + L::S(g) + 8 * k, v + (uint64_t)(k * (2048 >> 4)), id_o, 1u);
                if (i == nt) mma_commit(&o_full[g]);
              }
            }
            if (i < nt && leader) {
              const uint64_t q = qd + (uint64_t)(g * (L::TILE >> 4)), kk = kd + (uint64_t)(ks * (L::TILE >> 4));
#pragma unroll
              for (int k = 0; k < DH / 16; ++k) {
                const uint64_t off = (uint64_t)(((k >> 2) * L::HALF + (k & 3) * 32) >> 4);
                mma_bf16(tm + L::S(g), q + off, kk + off, id_s, k > 0);
              }
              mma_commit(&s_full[g]);
            }
          }
          if (leader) {
            if (i > 0) mma_commit(&empty[vs]);
            if (i < nt) mma_commit(&empty[ks]);
            if (i == nt - 1) mma_commit(q_empty);  // the block's last scores
          }
          __syncwarp();
          // V_i lies behind K_i, K_{i+1} behind V_i
          vs = ks + 1 == ST ? 0 : ks + 1;
          vph = ks + 1 == ST ? kph ^ 1u : kph;
          if (i < nt) {
            ks += 2;
            if (ks >= ST) {
              ks -= ST;
              kph ^= 1u;
            }
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
    const uint32_t ts = tmem + lanebase + L::S(g), to = tmem + lanebase + L::O(g);
    int ns = 0, nseg = 0;
    for (; w.valid(); w.next()) {
      const int ntok = w.t1() - w.t0;
      if (g == 1 && ntok <= tpg) continue;
      const int tg0 = w.t0 + g * tpg, tg1 = min(w.t1(), tg0 + tpg);  // the group's tokens
      const int tok = min(tg0 + row / p.G, tg1 - 1);
      const bool live = row < (tg1 - tg0) * p.G;
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
#pragma unroll 1
            for (int c = 0; c < DH / 32; ++c) {
              uint32_t o[32];
              tmem_ld32_async(to + 32 * c, o);
              tmem_wait_ld();
              pin32(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st32(to + 32 * c, o);
            }
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
      const bool whole_item = w.starts() && w.ends();
      const int slot = w.starts() ? 1 : 0;
      const int qrow = w.s.row0 + tok, hq = w.h * p.G + row % p.G;
      const bool mine = live && in_bounds(qrow < p.n_rows, p.status);
      const float inv = paged_inverse(l);
      const size_t pr = ((size_t)blockIdx.x * 2 + slot) * kPagedTcRows + g * rpg + row;
      // not unrolled: run once a segment, the code comes from memory each time
#pragma unroll 1
      for (int c = 0; c < DH / 32; ++c) {
        uint32_t o[32];
        tmem_ld32_async(to + 32 * c, o);
        tmem_wait_ld();
        pin32(o);
        // O of a row without keys was multiplied by zero weights only: still zero
        if (!whole_item) {
          uint4 v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          store_quads<8>(v, mine ? p.part_o + pr * DH + 32 * c : nullptr, lane);
        } else {
          uint16_t *d = static_cast<uint16_t *>(p.out) + (long long)qrow * p.ldo + hq * DH + 32 * c;
          uint4 v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              w[j] = pack2(__uint_as_float(o[8 * e + 2 * j]) * inv, __uint_as_float(o[8 * e + 2 * j + 1]) * inv);
            v[e] = make_uint4(w[0], w[1], w[2], w[3]);
          }
          store_quads<4>(v, mine ? d : nullptr, lane);
        }
      }
      if (mine) {
        if (!whole_item) {
          p.part_ml[pr * 2] = m;
          p.part_ml[pr * 2 + 1] = l;
        } else if (p.lse) {
          p.lse[(size_t)qrow * p.Hq + hq] = paged_lse(m, l);
        }
      }
      if (tid == 0 && w.starts() && !w.ends()) {
        PagedDesc d;
        d.row0 = w.s.row0 + w.t0;
        d.rows = ntok * p.G;
        d.h = w.h;
        d.last_cta = w.last_cta();
        p.desc[blockIdx.x] = d;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_empty[g]);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kIssuer) tmem_dealloc(tmem, 512);
  trace_end(kTkPagedAttnTc);
}

// ---------------------------------------------------------------- host side

cudaError_t paged_tc_set_attributes() {
  cudaError_t e = cudaFuncSetAttribute(paged_attn_tc_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)Lay<128>::SMEM);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(paged_attn_tc_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Lay<64>::SMEM);
  return e;
}

// Items at most: one more block a sequence than its rows fill (the sequences' rows
// are disjoint: row starts that decrease leave no items), a place's round of CTAs for
// the gaps.
static size_t plan_items(int B, int n_rows, int tpb, int Hkv) {
  return ((size_t)n_rows / tpb + B) * Hkv + kPagedMaxCtas;
}

bool paged_tc_items_ok(int B, int n_rows, int tpb, int Hkv) {
  return plan_items(B, n_rows, tpb, Hkv) < (1ull << 31) - (1 << 20);
}

static size_t up256(size_t x) { return (x + 255) / 256 * 256; }

size_t paged_tc_plan_bytes(int B, int n_rows, int tpb, int Hkv) {
  return up256((size_t)kPagedMaxCtas * sizeof(PagedStart)) + up256(((size_t)B + 1) * 4) +
         up256(plan_items(B, n_rows, tpb, Hkv) * sizeof(PagedItem));
}

void paged_tc_bind_plan(PagedTcParams &sp, char *base) {
  sp.n_items = (int)plan_items(sp.a.B, sp.a.n_rows, sp.a.tpb, sp.a.Hkv);
  sp.start = reinterpret_cast<PagedStart *>(base);
  base += up256((size_t)kPagedMaxCtas * sizeof(PagedStart));
  sp.blocks = reinterpret_cast<int *>(base);
  base += up256(((size_t)sp.a.B + 1) * 4);
  sp.items = reinterpret_cast<PagedItem *>(base);
}

static cudaLaunchConfig_t config(int ctas, int threads, size_t smem, cudaStream_t s, cudaLaunchAttribute *attr, bool pdl) {
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

template <int TK>
cudaError_t launch_paged_plan(const PagedTcParams &sp, int ctas, cudaStream_t s, bool pdl) {
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = config(1, kPlanThreads, 0, s, attr, pdl);
  note_launch();
  return cudaLaunchKernelEx(&cfg, paged_tc_plan_kernel<TK>, sp, ctas);
}
template cudaError_t launch_paged_plan<32>(const PagedTcParams &, int, cudaStream_t, bool);
template cudaError_t launch_paged_plan<64>(const PagedTcParams &, int, cudaStream_t, bool);
template cudaError_t launch_paged_plan<128>(const PagedTcParams &, int, cudaStream_t, bool);

cudaError_t launch_paged_attn_tc(const PagedTcParams &params, int ctas, cudaStream_t s, bool pdl) {
  PagedTcParams sp = params;
  sp.item_cost = kItemCost;
  cudaError_t e = launch_paged_plan<kTK>(sp, ctas, s, pdl);
  if (e) return e;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg =
      config(ctas, kThreads, sp.a.Dh == 128 ? Lay<128>::SMEM : Lay<64>::SMEM, s, attr, pdl);
  note_launch();
  return sp.a.Dh == 128 ? cudaLaunchKernelEx(&cfg, paged_attn_tc_kernel<128>, sp)
                        : cudaLaunchKernelEx(&cfg, paged_attn_tc_kernel<64>, sp);
}

MTP_TRACE_COLLECTOR(paged_attn_tc)

}  // namespace mtp
