// Absorbed latent attention over a paged cache, on the tensor cores.
//
// Every head of a row reads the same cached row: R + Dr elements as key, the first R
// as value.  A block is 64 packed rows (tokens x heads); with more heads than that, a
// block holds part of a token's heads.  Its items are cut and dealt out by the plan of
// paged_attn_tc.cu, a CTA an SM, tiles of 32 or 64 keys:
//   S = Q K_i^T     64 rows, over R + 64 elements (zeros from Dr on: the cache's bytes bind);
//                   both operands in shared memory by TMA
//   P = 2^(S - m)   two threads a row, half of the keys each
//   O += P V_i      V_i the first R elements of K_i as they lie in shared memory
//                   (row-major keys: the MN-major form of operand B)
// O of 64 rows fills half of tensor memory only if its 128 lanes are used: lane l < 16
// of each 32 holds a row's first R/2 elements, lane l + 16 its other half.  The two
// halves are two products of 128 rows with K doubled, [P; 0] V(first half) + [0; P]
// V(second half): P lies twice in tensor memory, zeros in the other half's lanes.  (A
// product of 64 rows runs at half the rate of one of 128, so the zeros cost nothing.)
// S of 64 rows arrives in the lanes l < 16 of each 32.
//
// Bound by the cache's bytes: 32 x 1 row of 16 heads over 16384-32749 keys (R 512) take 167-178 us, 907 MB
// at 75-80% of the copy rate; one row of 16 heads over 512 keys takes 10 us, one over 4096 13 us,
// in latencies (its plan 2, first scores 5, states and joining 4; all in graphs of 20).
//
// P is rounded to bf16 for its product: half a step a weight, 2^-8 sum p |c| at most, about what
// the output's own rounding costs (against 64 bits 0.0017 relative, as with fp32 weights).  The rest
// of P as a second bf16 term, for sequences of up to 16 packed rows, doubled that product in each
// tile's chain of scores, softmax and product: 167 -> 213 us, 64 x 1 row of 16 heads over 4096
// keys 66 -> 81 (R 256: 40 -> 58).
//
// S_{i+1} is issued ahead of O += P_i V_i, so that the softmax of one tile runs under
// the products of another.  Tensor memory (512 columns): O 256 | S_0 S_1 128 | P_0 P_1 128.
// Warps 0-3 are the softmax, warp 4 brings pages, warp 5 issues the products, warp 6 brings
// the next block's queries, warp 7 clears rows that no row sees.
#include "internal.h"
#include "latent.cuh"
#include "paged_tc.cuh"
#include "latent_combine.cuh"

namespace mtp {

namespace {

constexpr int kRows = 64;  // packed rows of a block
constexpr int kThreads = 256;
constexpr int kProducer = 4, kIssuer = 5, kQuery = 6, kClear = 7;
constexpr unsigned kFull = 0xffffffffu;

template <int R>
struct Lay {
  static constexpr int TK = R == 512 ? 32 : 64;  // keys per tile
  static constexpr int NB = R / 64 + 1;          // 64-element blocks of a row, the rotary one last
  static constexpr int BLK = TK * 128;           // bytes of a block of a tile: rows of 128 bytes
  static constexpr int TILE = NB * BLK;
  static constexpr int QBLK = kRows * 128, QTILE = NB * QBLK;
  static constexpr int STAGES = 4;
  static constexpr int NG = (NB + 2) / 3;        // groups of up to three blocks that arrive together
  static constexpr size_t SMEM = (size_t)QTILE + STAGES * TILE + 512 + kNearItems * sizeof(PagedItem);
  __host__ __device__ static constexpr uint32_t S(int b) { return 256u + TK * b; }
  __host__ __device__ static constexpr uint32_t P(int b) { return 384u + TK * b; }
};

// A thread's scores of a tile: the lanes l < 16 hold a row's, and lane l + 16 takes its
// second half from lane l.
template <int KH>
__device__ __forceinline__ void load_scores(uint32_t taddr, uint32_t (&s)[KH], int lane) {
  uint32_t t[2][32];
#pragma unroll
  for (int c = 0; c < KH / 16; ++c) tmem_ld32_async(taddr + 32 * c, t[c]);
  tmem_wait_ld();
#pragma unroll
  for (int c = 0; c < KH / 16; ++c) pin32(t[c]);
#pragma unroll
  for (int e = 0; e < KH; ++e) {
    const uint32_t v = __shfl_sync(kFull, t[(KH + e) / 32][(KH + e) % 32], lane & 15);
    s[e] = lane < 16 ? t[e / 32][e % 32] : v;
  }
}

}  // namespace

template <int R>
__global__ void __launch_bounds__(kThreads, 1) latent_attn_kernel(const __grid_constant__ PagedTcParams sp) {
  trace_start(kTkLatentAttn);
  using L = Lay<R>;
  constexpr int TK = L::TK, NB = L::NB, ST = L::STAGES, NG = L::NG;
  const PagedArgs &p = sp.a;
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char *qbuf = smem, *ring = smem + L::QTILE;
  uint64_t *full = reinterpret_cast<uint64_t *>(ring + ST * L::TILE);  // [stages][groups]
  uint64_t *empty = full + ST * NG, *zbar = empty + ST;
  uint64_t *q_full = zbar + ST, *q_empty = q_full + NG, *drain = q_empty + 1;
  uint64_t *s_full = drain + 1, *p_full = s_full + 2, *o_done = s_full + 4, *o_empty = s_full + 6;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(s_full + 7);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < ST * NG; ++s) mbar_init(&full[s], 1);
    for (int s = 0; s < ST; ++s) {
      mbar_init(&empty[s], 1);
      mbar_init(&zbar[s], 1);
    }
    for (int g = 0; g < NG; ++g) mbar_init(&q_full[g], 1);
    mbar_init(q_empty, 1);
    mbar_init(drain, 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&s_full[b], 1);
      mbar_init(&p_full[b], 4);
      mbar_init(&o_done[b], 1);
    }
    mbar_init(o_empty, 4);
    fence_barrier_init();
  }
  if (warp == kIssuer) tmem_alloc(tmem_slot, 512);
  if (warp == kProducer && lane == 0) prefetch_map(&sp.mk);
  if (warp == kQuery && lane == 0) prefetch_map(&sp.mq);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dep_wait();
  trace_dep(kTkLatentAttn);
  grid_dep_launch();
  PagedItem *near = reinterpret_cast<PagedItem *>(smem + L::SMEM - kNearItems * sizeof(PagedItem));
  SmallPlan *plan = reinterpret_cast<SmallPlan *>(ring);  // (before the first copy)
  if (sp.small) plan_share<TK, kThreads>(sp, sp.shares, blockIdx.x, plan, near);
  PlanWalk<TK, true> w = sp.small ? PlanWalk<TK, true>(sp, blockIdx.x, plan->start, near) : PlanWalk<TK, true>(sp, blockIdx.x, near);
  // (no share, no segment)
  if (tid == 0) p.desc[blockIdx.x].rows = 0;
  if (!sp.small && w.valid()) w.copy_near(sp, blockIdx.x, near);
  fence_proxy_async_smem();  // the plan's memory is the copies' next
  __syncthreads();
  bool ok = true;

  if (warp == kProducer) {
    // -------------------------------------------------- pages into the ring
    const int prow = min(p.page, TK), npc = TK / prow;  // rows and number of a tile's pieces
    int it = 0;
    for (; w.valid() && ok; w.next()) {
      // the piece of this lane in tile i: whether a row sees it, and its row of the pool
      auto locate = [&](int i, bool &need, int &y) {
        const int k0 = w.r.tile(i) * TK + lane * prow;
        need = lane < npc && w.r.any(k0, k0 + prow);
        y = need ? paged_page(p, w.b, k0) * p.page + (k0 & (p.page - 1)) : 0;
      };
      bool need, need_next = false;
      int y, y_next = 0;
      locate(w.i0, need, y);
      for (int i = w.i0; i < w.i1 && ok; ++i, ++it, need = need_next, y = y_next) {
        const int t0 = w.r.tile(i) * TK, s = it % ST;
        if (i + 1 < w.i1) locate(i + 1, need_next, y_next);  // its table entry loads under this tile's waits
        const uint32_t bytes = (uint32_t)(__popc(__ballot_sync(kFull, need)) * prow * 128);
        const bool whole = (t0 + TK <= w.r.hi && t0 >= w.r.lo) || t0 + TK <= w.r.sink_end;
        if (it >= ST) ok = mbar_wait(&empty[s], (uint32_t)((it / ST) - 1) & 1u, p.status);
        ok = __all_sync(kFull, ok);
        if (!ok) break;
        // a tile with rows to clear goes to the clearing warp first
        if (lane == 0) {
          if (whole)
            for (int g = 0; g < NG; ++g) mbar_arrive_expect_tx(&full[s * NG + g], (uint32_t)min(3, NB - 3 * g) * bytes);
          else
            mbar_arrive_expect_tx(&zbar[s], NB * bytes);
        }
        __syncwarp();
        if (need) {
          unsigned char *dst = ring + (size_t)s * L::TILE + lane * prow * 128;
#pragma unroll
          for (int x = 0; x < NB; ++x)
            tma_2d(dst + x * L::BLK, &sp.mk, 64 * x, y, whole ? &full[s * NG + x / 3] : &zbar[s]);
        }
      }
    }
    if (!ok)  // let copies still in flight land before the CTA exits
      for (int i = max(0, it - ST); i < it; ++i)
        for (int g = 0; g < NG; ++g)
          if (!mbar_wait(&full[(i % ST) * NG + g], (uint32_t)(i / ST) & 1u, p.status)) break;
  } else if (warp == kClear) {
    // -------------------------------------------------- rows that no row sees (past the
    // last key, before the window, never loaded) may hold anything, NaN too, which a
    // weight of zero would not hold back: they are cleared before a tile is handed on
    uint32_t phases = 0;  // a bit a stage
    int it = 0;
    for (; w.valid() && ok; w.next()) {
      for (int i = w.i0; i < w.i1 && ok; ++i, ++it) {
        const int t0 = w.r.tile(i) * TK, s = it % ST;
        if ((t0 + TK <= w.r.hi && t0 >= w.r.lo) || t0 + TK <= w.r.sink_end) continue;
        ok = __all_sync(kFull, mbar_wait(&zbar[s], phases >> s & 1u, p.status));
        phases ^= 1u << s;
        unsigned char *tile = ring + (size_t)s * L::TILE;
        for (int x = lane; x < TK * 8; x += 32)
          if (!w.r.sees(t0 + (x >> 3)))
#pragma unroll
            for (int hb = 0; hb < NB; ++hb)
              *reinterpret_cast<uint4 *>(tile + hb * L::BLK + x * 16) = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane < NG) mbar_arrive(&full[s * NG + lane]);
      }
    }
  } else if (warp == kQuery) {
    // -------------------------------------------------- the blocks' queries
    if (lane == 0) {
      for (int seg = 0; w.valid(); w.next(), ++seg) {
        if (seg > 0 && !mbar_wait(q_empty, (uint32_t)(seg - 1) & 1u, p.status)) break;
        for (int x = 0; x < NB; ++x) {
          if (x % 3 == 0) mbar_arrive_expect_tx(&q_full[x / 3], (uint32_t)(min(3, NB - x) * p.tpb * p.G * 128));
          tma_3d(qbuf + x * L::QBLK, &sp.mq, 64 * x, w.h * p.G, w.s.row0 + w.t0, &q_full[x / 3]);
        }
      }
    }
    __syncwarp();
  } else if (warp == kIssuer) {
    // -------------------------------------------------- matrix products
    // The whole warp walks and waits, one elected lane issues (paged_attn_tc.cu).
    constexpr uint32_t id_s = idesc_bf16_f32(64, TK), id_o = idesc_bf16_f32(128, R / 2) | (1u << 16);
    const uint32_t tm = __shfl_sync(kFull, tmem, 0);
    const uint64_t qd = sw128_kmajor_desc(smem_u32(qbuf)), kd = sw128_kmajor_desc(smem_u32(ring)),
                   vd = sw128_mnmajor_desc(smem_u32(ring), L::BLK);
    const bool leader = elect_one();
    // A wait that gives up flags the status; the waits after it are skipped and
    // the rest is issued on whatever is there, so that no barrier is left short.
    auto await = [&](uint64_t *bar, uint32_t parity) {
      if (ok) ok = mbar_wait(bar, parity, p.status);
    };
    int it = 0, seg = 0;  // tiles whose scores were issued
    uint32_t oph = 1;
    for (; __shfl_sync(kFull, w.valid(), 0); w.next(), ++seg) {
      const int nt = __shfl_sync(kFull, w.i1 - w.i0, 0);
      for (int g = 0; g < NG; ++g) await(&q_full[g], (uint32_t)seg & 1u);
      for (int i = 0; i <= nt; ++i) {
        if (i < nt) {
          const int s = it % ST;
          const uint32_t ph = (uint32_t)(it / ST) & 1u, d = tm + L::S(it & 1);
          const uint64_t kk = kd + (uint64_t)(s * (L::TILE >> 4));
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            await(&full[s * NG + g], ph);
            tc_fence_after();
            if (leader) {
#pragma unroll
              for (int x = 3 * g; x < 3 * g + 3 && x < NB; ++x)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  mma_bf16(d, qd + (uint64_t)((x * L::QBLK + k * 32) >> 4), kk + (uint64_t)((x * L::BLK + k * 32) >> 4), id_s,
                           x > 0 || k > 0);
                }
            }
          }
          if (leader) {
            mma_commit(&s_full[it & 1]);
            if (i == nt - 1) mma_commit(q_empty);  // the block's last scores
          }
          __syncwarp();
          ++it;
        }
        if (i > 0) {
          const int j = it - (i < nt ? 2 : 1), s = j % ST;  // the tile before
          if (i == 1) {
            await(o_empty, oph);
            oph ^= 1u;
          }
          await(&p_full[j & 1], (uint32_t)(j >> 1) & 1u);
          tc_fence_after();
          if (leader) {
            const uint64_t v = vd + (uint64_t)(s * (L::TILE >> 4));
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int k = 0; k < TK / 16; ++k)
                mma_ts(tm, tm + L::P(j & 1) + TK / 2 * h + 8 * k, v + (uint64_t)((h * (R / 128) * L::BLK + k * 2048) >> 4), id_o,
                       h > 0 || k > 0 || i > 1);
            mma_commit(&empty[s]);
            mma_commit(&o_done[j & 1]);
          }
          __syncwarp();
        }
      }
    }
    if (leader) mma_commit(drain);  // nothing of this CTA is in flight when it frees its tensor memory
    __syncwarp();
    mbar_wait(drain, 0, p.status);
  } else {
    // -------------------------------------------------- softmax: two threads a row, half of the keys each
    const uint32_t lanebase = (uint32_t)(warp * 32) << 16;
    const uint32_t to = tmem + lanebase;
    const int row = 16 * warp + (lane & 15), half = lane >> 4;
    constexpr int KH = TK / 2;  // keys of a thread
    int it = 0;
    for (; w.valid(); w.next()) {
      const int ntok = w.t1() - w.t0;
      const int tok = w.t0 + min(row / p.G, ntok - 1), hq = w.h * p.G + row % p.G;
      const bool live = row < ntok * p.G && hq < p.Hq;
      const int pos = w.s.ctx + tok;
      const int rhi = min(pos + 1, p.cap), rlo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
      const int all_hi = min(w.s.ctx + w.t0 + 1, p.cap);
      const int all_lo = p.window > 0 ? max(0, w.s.ctx + w.t1() - 1 - p.window + 1) : 0;
      float m = -INFINITY, l = 0.f;  // of the row; the sum of this thread's keys
      for (int i = w.i0; i < w.i1; ++i, ++it) {
        const int k0 = w.r.tile(i) * TK;
        const bool whole = k0 + TK <= all_hi && (k0 >= all_lo || k0 + TK <= min(p.sinks, all_hi));
        if (ok) ok = mbar_wait(&s_full[it & 1], (uint32_t)(it >> 1) & 1u, p.status);
        __syncwarp();
        if (i == w.i0) trace_mark(kTkLatentAttn, 0);
        tc_fence_after();
        uint32_t s[KH];
        load_scores<KH>(tmem + lanebase + L::S(it & 1), s, lane);
        if (!whole) {
          const int b = k0 + KH * half;  // the row's view of its keys as bits
          const uint32_t see = below(rhi - b) & (~below(rlo - b) | below(p.sinks - b));
#pragma unroll
          for (int e = 0; e < KH; ++e)
            if (!(see >> e & 1u)) s[e] = 0xff800000u;
        }
        float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < KH; e += 2)
          x[(e >> 1) & 3] = max3(x[(e >> 1) & 3], __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
        float mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
        mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 16)) * p.scale_log2;
        if (__any_sync(kFull, live && mx > m + 8.f)) {
          const float n = fmaxf(m, mx);
          const float f = n == m ? 1.f : exp2f(m - n);
          m = n;
          l *= f;
          if (i > w.i0) {
            // The product of the tile before may still be running.  (A barrier for odd and
            // one for even tiles: this tile's scores show that the product two tiles before
            // is done, so that a parity never stands for two phases that are both possible.)
            if (ok) ok = mbar_wait(&o_done[(it - 1) & 1], (uint32_t)((it - 1) >> 1) & 1u, p.status);
            __syncwarp();
            tc_fence_after();
            rescale_columns<R / 64>(to, f);
          }
        }
        const float u = m == -INFINITY ? 0.f : m;
        const float2 sc2 = make_float2(p.scale_log2, p.scale_log2), nu2 = make_float2(-u, -u);
        float2 sum = make_float2(0.f, 0.f);
        uint32_t pk[KH];  // the row's weights, in key order
#pragma unroll
        for (int e = 0; e < KH / 2; ++e) {
          float2 y = fma2(make_float2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), sc2, nu2);
          y.x = ex2_approx(y.x);
          y.y = ex2_approx(y.y);
          sum = add2(sum, y);
          const uint32_t mine = pack2(y.x, y.y), other = __shfl_xor_sync(kFull, mine, 16);
          pk[e] = half ? other : mine;
          pk[KH / 2 + e] = half ? mine : other;
        }
        l += sum.x + sum.y;
        // [P; 0], then [0; P]
#pragma unroll
        for (int c = 0; c < TK / 32; ++c) {
          uint32_t z[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) z[e] = ((32 * c + e) / KH == half) ? pk[(32 * c + e) % KH] : 0u;
          tmem_st32(tmem + lanebase + L::P(it & 1) + 32 * c, z);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[it & 1]);
      }
      // ---- the block's output, or this segment's state
      l += __shfl_xor_sync(kFull, l, 16);
      if (ok) ok = mbar_wait(&o_done[(it - 1) & 1], (uint32_t)((it - 1) >> 1) & 1u, p.status);
      __syncwarp();
      tc_fence_after();
      trace_mark(kTkLatentAttn, 1);
      const bool whole_item = w.starts() && w.ends();
      const int slot = w.starts() ? 1 : 0;
      const int qrow = w.s.row0 + tok;
      const bool mine = live && in_bounds(qrow < p.n_rows, p.status);
      const float inv = paged_inverse(l);
      const size_t block = (size_t)blockIdx.x * 2 + slot;
      write_row<R / 64, kRows>(to, half * (R / 2), whole_item,
                               mine ? static_cast<uint16_t *>(p.out) + (long long)qrow * p.ldo + hq * R : nullptr, inv,
                               p.part_o + block * kRows * R, mine ? row : -1, lane);
      if (mine && half == 0) {
        if (!whole_item) {
          reinterpret_cast<float2 *>(p.part_ml)[block * kRows + row] = make_float2(m, l);
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
      trace_mark(kTkLatentAttn, 2);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_empty);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kIssuer) tmem_dealloc(tmem, 512);
  trace_end(kTkLatentAttn);
}

// ---------------------------------------------------------------- host side

namespace {

// Blocks of at most 64 rows: the heads of a token are split into hb runs of G, a block
// holds 64 / G tokens of one run.  Chosen for the fewest blocks at the mean number of
// rows a sequence, all that the host knows: 40 heads and chunks take two runs of 20 (three
// tokens a block) and not one of 40 (one token).
void block_shape(int B, int n_rows, int H, int *G, int *hb) {
  const int n = (n_rows + B - 1) / B;
  long long best = -1;
  for (int r = (H + kRows - 1) / kRows; r <= H; ++r) {
    const int g = (H + r - 1) / r, t = kRows / g;
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
cudaError_t launch(const PagedTcParams &sp, int ctas, cudaStream_t s, bool pdl) {
  cudaError_t e = sp.small ? cudaSuccess : launch_paged_plan<Lay<R>::TK>(sp, ctas, s, pdl);
  if (e) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Lay<R>::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  note_launch();
  e = cudaLaunchKernelEx(&cfg, latent_attn_kernel<R>, sp);
  if (e) return e;
  return launch_latent_combine<R, kRows, 1>(sp, ctas, ctas, s, pdl);
}

}  // namespace

// More packed rows than two blocks of 64 hold, at the mean number of rows a sequence, go to
// pairs of CTAs.  The mean is all that the host knows, and rows past the last sequence count: 64
// sequences of one row of 16 heads over 4096 keys take 66 us, in arrays of 1024 rows 150;
// beside a chunk of 512 rows 227, the chunk alone 79.  us (64-row blocks / pairs), R 512, every
// sequence alike:
//             4 of 4096 keys   16 of 2048    48 of 1024    64 of 4096
//   1 x 128   21.4 / 24.6      28.0 / 30.2   43.5 / 47.9   130 / 161
//   4 x 40    25.8 / 24.6      35.3 / 32.2   55.3 / 49.1   181 / 164
//   4 x 128   39.9 / 30.7      75.9 / 57.3   109 / 87      440 / 311
// R 256, 1 x 128: 15.7 / 16.3, 19.0 / 21.6, 26.1 / 26.5, 65 / 60; 4 x 40: 17.5 / 17.2, 22.6 / 21.4,
// 32.6 / 30.1, 88 / 61.  (One sequence: within 2 us.)
static bool wants_pair(int B, int n_rows, int H) { return (long long)((n_rows + B - 1) / B) * H > 128; }

// Enough for every call of at most B sequences and n_rows rows, whichever kernel and blocks its
// mean takes: a program sizes its workspace once, and sequences finish.  Items: of N rows in B
// sequences, n = ceil(N / B) at the mean, block_shape takes runs r of t tokens a block with
// r ceil(n / t) <= r0 ceil(n / t0), r0 and t0 its first choice.  So
//   r (N / t + B) <= 2 B r ceil(n / t) <= 2 r0 B ceil(n / t0) <= 2 r0 (N / t0 + B).
size_t latent_attn_scratch_bytes(int B, int n_rows, int H, int R) {
  const int r0 = (H + kRows - 1) / kRows, G = (H + r0 - 1) / r0;
  const long long most = (long long)B * (128 / H);  // rows that stay with this kernel
  const size_t here = region_bytes(kPagedMaxCtas, kRows, R) +
                      paged_tc_plan_bytes(B, most < n_rows ? (int)most : n_rows, kRows / G, 2 * r0);
  if (!wants_pair(1, n_rows, H)) return here;  // (no call of fewer rows does)
  const size_t pairs = latent_pair_scratch_bytes(B, n_rows, H, R);
  return here > pairs ? here : pairs;
}

cudaError_t launch_latent_attn(const LatentAttnArgs &la, void *scratch, int sms, cudaStream_t s, bool pdl) {
  if (wants_pair(la.a.B, la.a.n_rows, la.a.Hq)) return launch_latent_attn_pair(la, scratch, sms, s, pdl);
  const int n = sms < kPagedMaxCtas ? sms : kPagedMaxCtas, w = la.a.Dh + la.Dr;
  PagedTcParams sp{};
  PagedArgs &a = sp.a;
  a = la.a;
  block_shape(a.B, a.n_rows, a.Hq, &a.G, &a.Hkv);
  a.tpb = kRows / a.G;
  const int tk = a.Dh == 512 ? Lay<512>::TK : Lay<256>::TK;
  // shares of at least 64 / 128 / 256 keys (us, one row of 16 heads, R 512): one sequence of 512
  // keys 10.4 / 12.1 / 15.4, of 4096 12.8 / 13.3 / 16.0; 4 of 2048 13.0 / 13.8 / 16.7; R 256 (128 and
  // 256): 10.1 / 11.2, 11.4 / 11.8, 11.2 / 12.2
  a.min_tiles = 2;
  sp.item_cost = 128 / tk;
  char *base = static_cast<char *>(scratch);
  bind_region(a, base, n, kRows);
  paged_tc_bind_plan(sp, base + region_bytes(kPagedMaxCtas, kRows, a.Dh));
  paged_small_plan(sp, n);
  if (!make_rows_map(&sp.mk, la.pages, w, (uint64_t)a.n_pages * a.page, w, a.page < tk ? a.page : tk) ||
      !make_query_map(&sp.mq, a.q, w, a.Hq, a.n_rows, a.ldq, a.G, a.tpb))
    return cudaErrorNotSupported;
  return a.Dh == 512 ? launch<512>(sp, n, s, pdl) : launch<256>(sp, n, s, pdl);
}

cudaError_t latent_set_attributes() {
  cudaError_t e =
      cudaFuncSetAttribute(latent_attn_kernel<512>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Lay<512>::SMEM);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(latent_attn_kernel<256>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Lay<256>::SMEM);
  if (e == cudaSuccess) e = latent_pair_set_attributes();
  if (e == cudaSuccess) e = latent_prefill_set_attributes();
  if (e == cudaSuccess) e = latent_heads_set_attributes();
  return e;
}

MTP_TRACE_COLLECTOR(latent_attn)

}  // namespace mtp
