// A product a head on the tensor cores: y[n, h, :] = W[h] x[n, h, :], from an array of
// rows or from the pages of a latent cache (then the rows are the first positions of
// the sequences and every head reads the same ones).
//
// Pairs of CTAs walk tiles of 2 x 128 rows x NT outputs of a head, the row tiles of one
// weight tile next to each other so that the weights come from memory once.  A pair's
// product (cta_group::2) reads each CTA's rows and half of the weight tile: alone, a CTA
// would bring 48 KB and read 48 KB of shared memory for every 512 cycles of products, at
// 128 bytes a cycle 768; in pairs it is 32 and 32 KB.  With one tile of rows there is no
// pair to make, and CTAs walk alone.  x and W arrive by TMA in blocks of 64 along K, W as
// it lies: rows along K ([N, K], the K-major form of the operand) or along N ([K, N], the
// MN-major one).  Two accumulators in tensor memory: a tile's output is written under the
// next one's products.
//
// Cached rows are the same for every head, so a pair keeps its 256 rows (K up to 512: 128 KB
// a CTA) and walks the heads over them; only weights, from L2, pass through the ring.  In graphs
// of 20, 8 ragged prompts of 16 heads: 23 us against 26 with rows brought for each head; 12288
// keys of 128 heads are the same 287 us both ways (308-316 a call among others).  Those are 207 us
// when nothing is stored (412 GFLOP, 2.0 PFLOP/s; the library's product, which the floors
// count with, reaches 1.93) and 238 us when the stores stay in L2: the rest is 805 MB of output
// on their way to memory, which a plain fill of that size writes in 200 us.
//
// Tiles of cached rows never cross a sequence, since page pieces start on whole pages.
// The number of tiles is the device's to know: each CTA sums up the sequences' tiles
// at its start (a run of sequences a thread) and searches that table for each tile.
#include "internal.h"
#include "latent.cuh"
#include "paged_tc.cuh"
#include "tcgen05_ops.cuh"

namespace mtp {

namespace {

constexpr int kThreads = 320;  // warps 0-7 write outputs, 8 brings blocks, 9 issues the products
constexpr int kProducer = 8, kIssuer = 9, kOutThreads = 256;
constexpr int kABytes = 128 * 128;  // of a stage: 64 of K
constexpr unsigned kFull = 0xffffffffu;

constexpr int kKeptBlocks = 8;  // blocks of 64 of kept rows: K up to 512

template <bool PAIR, bool KEEP>
struct Lay {
  static constexpr int WBYTES = (PAIR ? 128 : 256) * 128;        // of a stage: a CTA's part of the weights
  static constexpr int STAGE = (KEEP ? 0 : kABytes) + WBYTES;    // and its rows, unless they are kept
  static constexpr int STAGES = KEEP ? 5 : PAIR ? 6 : 4;
  static constexpr int KEPT = KEEP ? kKeptBlocks * kABytes : 0;
  static constexpr size_t SMEM = (size_t)KEPT + STAGES * STAGE + 256;
};

struct HeadsParams {
  CUtensorMap mx, mw;
  LatentHeadsArgs a;
  int NT, n_tiles, m_tiles;  // outputs of a tile; tiles along N and (from an array) along the rows
  int kbs, pieces;           // blocks of 64 along K; pieces of a transposed weight block
};

// A tile of rows: of sequence b (from pages), or of the array.
struct RowTile {
  int b, j0, row0, rows;  // sequence, first position, first output row, rows
};

// The sequences' row tiles before each thread's run of sequences, and the first kNear
// tiles themselves: looked up through the row starts, a tile's place took two round trips
// of the producer, which its ring (four stages, in pairs six, with kept rows five) does not cover.
constexpr int kNear = 1024;
struct TileTable {
  int before[kThreads + 1];
  int sums[kThreads / 32];
  RowTile near[kNear];
};

// Rows of sequence b that are expanded; flags what is out of range, and sets *back if the
// rows end before they start.
__device__ __forceinline__ int seq_rows(const LatentHeadsArgs &p, int b, int *start, bool flag, bool *back = nullptr) {
  const int s = __ldcg(&p.key_start[b]), e = __ldcg(&p.key_start[b + 1]);
  *start = s;
  if (back) *back |= e < s;
  if (s < 0 || e < s || e > p.n_rows) {
    if (flag) set_status(p.status, kStatusBadRows);
    return 0;
  }
  if (e - s > p.cap && flag) set_status(p.status, kStatusBadCtx);
  return min(e - s, p.cap);
}

__device__ __forceinline__ RowTile find_tile(const LatentHeadsArgs &p, const TileTable &t, int m) {
  RowTile r;
  if (!p.pages) {
    r.b = 0;
    r.j0 = 0;
    r.row0 = m * 128;
    r.rows = max(0, min(128, p.n_rows - r.row0));
    return r;
  }
  if (m >= t.before[kThreads]) return {0, 0, 0, 0};  // the second of a last, odd pair
  if (m < kNear) return t.near[m];
  int lo = 0, hi = kThreads;  // before[lo] <= m < before[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (t.before[mid] <= m) lo = mid;
    else hi = mid;
  }
  const int per = (p.B + kThreads - 1) / kThreads;
  int left = m - t.before[lo];
  for (int b = lo * per;; ++b) {
    int s;
    const int n = seq_rows(p, b, &s, false), k = (n + 127) / 128;
    if (left < k) {
      r.b = b;
      r.j0 = left * 128;
      r.row0 = s + r.j0;
      r.rows = min(128, n - r.j0);
      return r;
    }
    left -= k;
  }
}

__device__ __forceinline__ int page_entry(const LatentHeadsArgs &p, int b, int j) {
  return __ldg(&p.page_table[(size_t)b * p.max_pages + (j >> p.page_shift)]);
}

// The page of a table's entry; page 0 for one outside the pool.
__device__ __forceinline__ int page_of(const LatentHeadsArgs &p, int id) {
  if (id < 0 || id >= p.n_pages) {
    set_status(p.status, kStatusBadPage);
    return 0;
  }
  return id;
}

}  // namespace

// KEEP (rows from pages, in pairs): every head multiplies the same rows, which stay in shared
// memory while the pair walks the heads; only weights pass through the ring.
template <bool TRANS, bool PAIR, bool KEEP>
__global__ void __launch_bounds__(kThreads, 1) latent_heads_kernel(const __grid_constant__ HeadsParams hp) {
  trace_start(kTkLatentHeads);
  using L = Lay<PAIR, KEEP>;
  constexpr int kStages = L::STAGES, kStageBytes = L::STAGE, CTAS = PAIR ? 2 : 1;
  const LatentHeadsArgs &p = hp.a;
  const uint32_t rank = PAIR ? cluster_rank() : 0;
  const unsigned walker = blockIdx.x / CTAS, walkers = gridDim.x / CTAS;
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char *ring = smem + L::KEPT;
  uint64_t *full = reinterpret_cast<uint64_t *>(ring + kStages * kStageBytes);
  uint64_t *empty = full + kStages, *done = empty + kStages, *tfree = done + 2, *drain = tfree + 2, *kept = drain + 1,
           *kept_free = kept + kKeptBlocks;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(kept_free + 1);
  __shared__ TileTable table;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], CTAS);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&done[b], 1);
      mbar_init(&tfree[b], CTAS * kOutThreads / 32);
    }
    mbar_init(drain, 1);
    for (int x = 0; x < kKeptBlocks; ++x) mbar_init(&kept[x], CTAS);
    mbar_init(kept_free, 1);
    fence_barrier_init();
  }
  if (warp == kIssuer) {
    if constexpr (PAIR) tmem_alloc_pair(tmem_slot, 512);
    else tmem_alloc(tmem_slot, 512);
  }
  if (warp == kProducer && lane == 0) {
    prefetch_map(&hp.mx);
    prefetch_map(&hp.mw);
  }
  tc_fence_before();
  if constexpr (PAIR) cluster_sync();  // the barriers of both CTAs are set up
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dep_wait();
  trace_dep(kTkLatentHeads);
  grid_dep_launch();
  int m_tiles = hp.m_tiles;
  if (p.pages) {
    const int per = (p.B + kThreads - 1) / kThreads;
    int mine = 0;
    bool back = false;
    for (int b = tid * per; b < min(p.B, (tid + 1) * per); ++b) {
      int s;
      mine += (seq_rows(p, b, &s, blockIdx.x == 0, &back) + 127) / 128;
    }
    // Starts that decrease may count rows twice: two CTAs could write one row, and the tiles'
    // number would have no bound (n_keys / 128 + B otherwise).  Nothing of such a call is expanded.
    const bool none = __syncthreads_or(back);
    if (none) mine = 0;
    int inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kFull, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) table.sums[warp] = inc;
    __syncthreads();
    int before = inc - mine;
    for (int v = 0; v < warp; ++v) before += table.sums[v];
    table.before[tid] = before;
    if (tid == kThreads - 1) table.before[kThreads] = before + mine;
    for (int b = tid * per; !none && b < min(p.B, (tid + 1) * per) && before < kNear; ++b) {
      int s;
      const int n = seq_rows(p, b, &s, false);
      for (int j = 0; j < n && before < kNear; j += 128) table.near[before++] = {b, j, s + j, min(128, n - j)};
    }
  }
  if (p.pages) {
    __syncthreads();
    m_tiles = table.before[kThreads];
  }
  m_tiles = (m_tiles + CTAS - 1) / CTAS;  // of all the walker's rows
  trace_mark(kTkLatentHeads, 0);
  // Items: a tile of rows and a tile of a head's outputs.  Row tiles next to each other share
  // their weights; kept rows are walked head by head, a run of items a walker.
  const int hns = p.H * hp.n_tiles;
  const long long items = (long long)hns * m_tiles;
  const long long u0 = KEEP ? items * walker / walkers : walker, u1 = KEEP ? items * (walker + 1) / walkers : items,
                  du = KEEP ? 1 : walkers;
  auto row_tile = [&](long long u) { return (int)(KEEP ? u / hns : u % m_tiles); };
  auto head_tile = [&](long long u) { return (int)(KEEP ? u % hns : u / m_tiles); };
  bool ok = true;

  if (warp == kProducer) {
    const int prow = p.pages ? min(p.page, 128) : 128, npc = 128 / prow;
    const uint32_t bbytes = TRANS ? (uint32_t)hp.pieces * 64 * 128 : (uint32_t)(hp.NT / CTAS) * 128;
    uint32_t i = 0;
    // a tile's rows and this lane's entry of the page table, one tile ahead
    RowTile r, r_next;
    int id = 0, id_next = 0;
    auto locate = [&](long long u, RowTile &t, int &e) {
      t = find_tile(p, table, row_tile(u) * CTAS + rank);
      if (p.pages && lane < npc && lane * prow < t.rows) e = page_entry(p, t.b, t.j0 + lane * prow);
    };
    int at = -1, nkept = 0;  // the kept row tile, and how many there were
    if (u0 < u1) locate(u0, r_next, id_next);
    for (long long u = u0; u < u1 && ok; u += du) {
      const int hn = head_tile(u), h = hn / hp.n_tiles, n0 = (hn % hp.n_tiles) * hp.NT;
      r = r_next;
      id = id_next;
      const bool need = lane < npc && lane * prow < r.rows;
      const int y = p.pages && need ? page_of(p, id) * p.page : 0;
      const uint32_t abytes = (uint32_t)(__popc(__ballot_sync(kFull, need)) * prow * 128);
      if (u + du < u1 && (!KEEP || row_tile(u + du) != row_tile(u))) locate(u + du, r_next, id_next);
      const bool bring = KEEP && row_tile(u) != at;
      if (bring) {
        at = row_tile(u);
        if (nkept > 0) ok = __all_sync(kFull, mbar_wait_cluster(kept_free, (uint32_t)(nkept - 1) & 1u, p.status));
        ++nkept;
      }
      for (int kb = 0; kb < hp.kbs && ok; ++kb, ++i) {
        const int s = (int)(i % kStages);
        if (i >= (uint32_t)kStages) ok = mbar_wait_cluster(&empty[s], ((i / kStages) - 1u) & 1u, p.status);
        ok = __all_sync(kFull, ok);
        if (!ok) break;
        unsigned char *st = ring + s * kStageBytes;
        if constexpr (KEEP) {
          const uint32_t bar = dsmem_addr(&full[s], 0);
          if (bring) {
            const uint32_t kbar = dsmem_addr(&kept[kb], 0);
            if (lane == 0) expect_tx_cluster(kbar, abytes);
            __syncwarp();
            if (need) tma_2d_pair(smem + kb * kABytes + lane * prow * 128, &hp.mx, kb * 64, y, kbar);
          }
          if (lane == 0) {
            expect_tx_cluster(bar, bbytes);
            tma_3d_pair(st, &hp.mw, kb * 64, n0 + rank * (hp.NT / 2), h, bar);
          }
          __syncwarp();
        } else if constexpr (PAIR) {
          // both CTAs' copies complete on the first one's barrier, each CTA adding its bytes
          const uint32_t bar = dsmem_addr(&full[s], 0);
          if (lane == 0) {
            expect_tx_cluster(bar, abytes + bbytes);
            if (TRANS)
              for (int x = 0; x < hp.pieces; ++x)
                tma_3d_pair(st + kABytes + x * 64 * 128, &hp.mw, n0 + 64 * (rank * hp.pieces + x), kb * 64, h, bar);
            else
              tma_3d_pair(st + kABytes, &hp.mw, kb * 64, n0 + rank * (hp.NT / 2), h, bar);
          }
          __syncwarp();
          if (need) {
            if (p.pages) tma_2d_pair(st + lane * prow * 128, &hp.mx, kb * 64, y, bar);
            else tma_3d_pair(st, &hp.mx, kb * 64, h, r.row0, bar);
          }
        } else {
          if (lane == 0) {
            mbar_arrive_expect_tx(&full[s], abytes + bbytes);
            if (TRANS)
              for (int x = 0; x < hp.pieces; ++x)
                tma_3d(st + kABytes + x * 64 * 128, &hp.mw, n0 + 64 * x, kb * 64, h, &full[s]);
            else
              tma_3d(st + kABytes, &hp.mw, kb * 64, n0, h, &full[s]);
          }
          __syncwarp();
          if (need) {
            if (p.pages) tma_2d(st + lane * prow * 128, &hp.mx, kb * 64, y, &full[s]);
            else tma_3d(st, &hp.mx, kb * 64, h, r.row0, &full[s]);
          }
        }
      }
    }
    if (!ok && rank == 0)  // let copies still in flight land before the CTAs exit
      for (uint32_t q = i > (uint32_t)kStages ? i - kStages : 0u; q < i; ++q)
        if (!mbar_wait_cluster(&full[q % kStages], (q / kStages) & 1u, p.status)) break;
    if (!ok && rank == 0 && nkept > 0)
      for (int x = 0; x < hp.kbs; ++x)
        if (!mbar_wait_cluster(&kept[x], (uint32_t)(nkept - 1) & 1u, p.status)) break;
  } else if (warp == kIssuer) {
    if (rank == 0) {
      const uint32_t idesc = idesc_bf16_f32(128 * CTAS, 256) - ((uint32_t)(256 - hp.NT) >> 3 << 17) + (TRANS ? 1u << 16 : 0u);
      const bool leader = elect_one();
      const unsigned char *weights = ring + (KEEP ? 0 : kABytes);
      const uint64_t ad = sw128_kmajor_desc(smem_u32(smem)),
                     bd = TRANS ? sw128_mnmajor_desc(smem_u32(weights), 64 * 128) : sw128_kmajor_desc(smem_u32(weights));
      auto commit = [](uint64_t *bar) {
        if constexpr (PAIR) mma_commit_pair(bar);
        else mma_commit(bar);
      };
      uint32_t i = 0, n = 0;
      int at = -1, nkept = 0;
      for (long long u = u0; u < u1 && ok; u += du, ++n) {
        const uint32_t buf = n & 1u;
        const bool brought = KEEP && row_tile(u) != at;
        if (brought) {
          at = row_tile(u);
          ++nkept;
        }
        const bool last = KEEP && (u + 1 == u1 || row_tile(u + 1) != at);
        if (n >= 2) ok = mbar_wait_cluster(&tfree[buf], ((n >> 1) - 1u) & 1u, p.status);
        ok = __all_sync(kFull, ok);
        if (!ok) break;
        for (int kb = 0; kb < hp.kbs && ok; ++kb, ++i) {
          const int s = (int)(i % kStages);
          ok = mbar_wait_cluster(&full[s], (i / kStages) & 1u, p.status);
          if (brought && ok) ok = mbar_wait_cluster(&kept[kb], (uint32_t)(nkept - 1) & 1u, p.status);
          ok = __all_sync(kFull, ok);
          if (!ok) break;
          tc_fence_after();
          if (leader) {
            const uint64_t so = (uint64_t)(s * (kStageBytes >> 4));
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint64_t x = ad + (KEEP ? (uint64_t)(kb * (kABytes >> 4)) : so) + 2 * k, y = bd + so + (TRANS ? 128 : 2) * k;
              if constexpr (PAIR) mma_bf16_pair(tmem + 256 * buf, x, y, idesc, (kb | k) != 0);
              else mma_bf16(tmem + 256 * buf, x, y, idesc, (kb | k) != 0);
            }
            commit(&empty[s]);
            if (kb == hp.kbs - 1) {
              commit(&done[buf]);
              if (last) commit(kept_free);
            }
          }
          __syncwarp();
        }
      }
      if (leader) commit(drain);  // nothing is in flight when the tensor memory is freed
      __syncwarp();
    }
    mbar_sleep_wait(drain, 0, p.status);  // (a pair's second CTA waits here from the start)
  } else {
    // a thread a row: the warp's lanes of tensor memory, every other 64 outputs
    const int q = warp & 3;
    const uint32_t lanebase = (uint32_t)(q * 32) << 16;
    uint32_t n = 0;
    RowTile r{};
    int at = -1;
    for (long long u = u0; u < u1; u += du, ++n) {
      const int hn = head_tile(u), h = hn / hp.n_tiles, n0 = (hn % hp.n_tiles) * hp.NT;
      if (!KEEP || row_tile(u) != at) r = find_tile(p, table, (at = row_tile(u)) * CTAS + rank);
      const uint32_t buf = n & 1u;
      const int row = q * 32 + lane;
      const bool real = row < r.rows;
      if (p.pages && hn == 0 && warp < 4 && real) {
        // the shared key part of the tile's positions
        const int j = r.j0 + row;
        const uint4 *src = reinterpret_cast<const uint4 *>(
            p.pages + ((size_t)page_of(p, page_entry(p, r.b, j)) * p.page + (j & (p.page - 1))) * (size_t)(p.K + p.Dr) + p.K);
        uint4 *dst = reinterpret_cast<uint4 *>(p.k_rope + (long long)(r.row0 + row) * p.ldkr);
        for (int e = 0; e < p.Dr / 8; ++e) dst[e] = __ldg(src + e);
      }
      ok = __all_sync(kFull, ok && mbar_wait_cluster(&done[buf], (n >> 1) & 1u, p.status));
      if (!ok) break;
      tc_fence_after();
      if (n == 0) trace_mark(kTkLatentHeads, 1);
      uint16_t *y = p.y + (long long)(r.row0 + row) * p.ldy + h * p.hsy + n0;
      const int cols = min(hp.NT, p.N - n0);
      for (int c = 64 * (warp >> 2); c < cols; c += 128) {
        uint32_t o[64];
        tmem_ld32_async(tmem + lanebase + 256 * buf + c, o);
        tmem_ld32_async(tmem + lanebase + 256 * buf + c + 32, o + 32);
        tmem_wait_ld();
        pin32(o);
        pin32(o + 32);
        uint4 v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          uint32_t x[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) x[j] = pack2(__uint_as_float(o[8 * e + 2 * j]), __uint_as_float(o[8 * e + 2 * j + 1]));
          v[e] = make_uint4(x[0], x[1], x[2], x[3]);
        }
        store_quads<8>(v, real ? y + c : nullptr, lane, (cols - c) / 8);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        // (the reads of tensor memory are complete: there is nothing to release)
        if constexpr (PAIR) mbar_arrive_cluster_relaxed(dsmem_addr(&tfree[buf], 0));
        else mbar_arrive(&tfree[buf]);
      }
    }
  }
  trace_mark(kTkLatentHeads, 2);
  tc_fence_before();
  if constexpr (PAIR) cluster_sync();  // neither CTA leaves while the other may still signal it
  else __syncthreads();
  tc_fence_after();
  if (warp == kIssuer) {
    if constexpr (PAIR) tmem_dealloc_pair(tmem, 512);
    else tmem_dealloc(tmem, 512);
  }
  trace_end(kTkLatentHeads);
}

// ---------------------------------------------------------------- host side

namespace {

template <bool TRANS, bool PAIR, bool KEEP>
cudaError_t launch(const HeadsParams &hp, long long walkers, cudaStream_t s, bool pdl) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)walkers * (PAIR ? 2 : 1));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Lay<PAIR, KEEP>::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (PAIR) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = 2;
    attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
    ++n;
  }
  if (pdl) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  note_launch();
  return cudaLaunchKernelEx(&cfg, latent_heads_kernel<TRANS, PAIR, KEEP>, hp);
}

template <bool TRANS, bool PAIR, bool KEEP>
cudaError_t set_smem() {
  return cudaFuncSetAttribute(latent_heads_kernel<TRANS, PAIR, KEEP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)Lay<PAIR, KEEP>::SMEM);
}

}  // namespace

cudaError_t launch_latent_heads(const LatentHeadsArgs &a, int sms, cudaStream_t s, bool pdl) {
  HeadsParams hp{};
  hp.a = a;
  hp.kbs = (a.K + 63) / 64;
  hp.m_tiles = (a.n_rows + 127) / 128;
  const bool pair = hp.m_tiles > 1;
  // a CTA of a pair holds half of a weight tile: whole pieces of 64
  hp.NT = a.N > (pair ? 128 : 255) ? 256 : pair ? 128 : (a.N + 15) / 16 * 16;
  hp.n_tiles = (a.N + hp.NT - 1) / hp.NT;
  const int nt = pair ? hp.NT / 2 : hp.NT;  // outputs whose weights a CTA brings
  hp.pieces = (nt + 63) / 64;
  const bool x_ok = a.pages ? make_rows_map(&hp.mx, a.pages, a.K + a.Dr, (uint64_t)a.n_pages * a.page, a.K + a.Dr, a.page)
                            : make_heads_map(&hp.mx, a.x, a.K, a.H, a.n_rows, a.hsx, a.ldx, 1, 128);
  const bool w_ok = a.transposed ? make_heads_map(&hp.mw, a.w, a.N, a.K, a.H, a.ldw, a.hsw, 64, 1)
                                 : make_heads_map(&hp.mw, a.w, a.K, a.N, a.H, a.ldw, a.hsw, nt, 1);
  if (!x_ok || !w_ok) return cudaErrorNotSupported;
  // from pages the device knows how many tiles there are: one more a sequence at most
  const long long tiles = a.pages ? (long long)hp.m_tiles + a.B : hp.m_tiles, most = (long long)a.H * hp.n_tiles * tiles;
  const int places = pair ? sms / 2 : sms;
  const long long walkers = most < places ? most : places;
  if (a.transposed)
    return pair ? launch<true, true, false>(hp, walkers, s, pdl) : launch<true, false, false>(hp, walkers, s, pdl);
  if (a.pages && pair) return launch<false, true, true>(hp, walkers, s, pdl);
  return pair ? launch<false, true, false>(hp, walkers, s, pdl) : launch<false, false, false>(hp, walkers, s, pdl);
}

cudaError_t latent_heads_set_attributes() {
  cudaError_t e = set_smem<true, true, false>();
  if (e == cudaSuccess) e = set_smem<true, false, false>();
  if (e == cudaSuccess) e = set_smem<false, true, false>();
  if (e == cudaSuccess) e = set_smem<false, true, true>();
  if (e == cudaSuccess) e = set_smem<false, false, false>();
  return e;
}

MTP_TRACE_COLLECTOR(latent_heads)

}  // namespace mtp
