// Rules on the target's logits before verification: penalties for repeated
// tokens, biases and a grammar mask, at every candidate position of a sequence.
//
// Position j of sequence b follows the history and the drafts 0 .. j-1.  With
// c = how often token v occurs in the generated part of the history and in
// those drafts, and seen = c > 0 or v occurs in the prompt:
//   x = l(v);  seen: x = x > 0 ? x / rep : x * rep
//   x -= freq * c;  c > 0: x -= pres;  x += bias(v);  v masked: x = -inf
//
// Bound by the logits' bytes.  Few tokens have a count or a bias, so a CTA, which
// owns one range of the vocabulary for all k + 1 rows of a sequence, scans the
// sequence's history once (4 bytes a token, from L2 after the first CTA) into
// counters in shared memory and keeps a list of the tokens it touched.  Each
// row's part comes in and goes out by bulk copies through a ring in shared
// memory, the first ones under the scan; there the listed logits are recomputed and
// then the masked ones overwritten.  The counters never go to memory, no state is
// kept from step to step, and no global atomics are needed.  At 256 sequences of
// 6 rows of 151936: looking every token up in the counters while streaming
// through registers took 515 us (38 instructions a logit), rewriting the listed
// tokens in global memory behind the stream 450 us.  In place, only what a rule
// changes is read and written.
#include "common.cuh"
#include "internal.h"
#include "logits.cuh"

namespace mtp {

namespace {

// a counter's word: occurrences in the low bits, and why else the token is listed
constexpr uint32_t kPrompt = 1u << 31, kBias = 1u << 30, kDraft = 1u << 29, kCount = kDraft - 1u;
constexpr unsigned kFull = 0xffffffffu;

// Six CTAs an SM: ranges of 4096 (three CTAs) and rings of four rows measured
// slower at 256 sequences of 6 rows of 151936 (446 and 444 us against 344),
// ranges of 1024 scan the history too often (494 us).
constexpr int NT = 256;           // threads
constexpr int VPT = 2;            // vectors of four logits a thread looks at per row
constexpr int CH = VPT * 4 * NT;  // tokens of a range
constexpr int kRing = 2;          // rows in shared memory at a time

}  // namespace

namespace {

// One range of one sequence: counters, the list of touched tokens, biases.
struct Range {
  uint32_t *cnt;    // [CH]
  uint16_t *list;   // [CH] offsets of the touched tokens
  float *bias;      // [CH] (only with biases)
  int *drafts;      // [8]
  int *listed;
  int b, c0, c1;
  float rep, freq, pres;

  // Executed by all NT threads; ends with a barrier.
  __device__ __forceinline__ void build(const LogitArgs &p) {
    const int tid = threadIdx.x;
    for (int i = tid; i < CH / 4; i += NT) {
      reinterpret_cast<uint4 *>(cnt)[i] = make_uint4(0u, 0u, 0u, 0u);
      if (p.bias_tok) reinterpret_cast<float4 *>(bias)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (tid == 0) *listed = 0;
    rep = p.rep ? __ldcg(&p.rep[b]) : 1.f;
    freq = p.freq ? __ldcg(&p.freq[b]) : 0.f;
    pres = p.pres ? __ldcg(&p.pres[b]) : 0.f;
    __syncthreads();
    // the first to touch a counter puts the token on the list
    auto touched = [&](uint32_t old, int o) {
      if (old == 0u) list[atomicAdd(listed, 1)] = (uint16_t)o;
    };
    if (p.history) {
      const int n = min(max(__ldcg(&p.hist_len[b]), 0), p.hist_cap);
      const int np = p.prompt_len ? min(max(__ldcg(&p.prompt_len[b]), 0), n) : 0;
      const int *h = p.history + (size_t)b * p.hist_cap;
      auto occurs = [&](int i, int t) {
        if (t >= c0 && t < c1) {
          uint32_t *c = &cnt[t - c0];
          touched(i < np ? atomicOr(c, kPrompt) : atomicAdd(c, 1u), t - c0);
        }
      };
      const int n4 = p.hist_cap % 4 == 0 ? n / 4 : 0;  // rows that start on 16 bytes are read in vectors
      for (int i0 = tid; i0 < n4; i0 += 4 * NT) {
        int4 t[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          t[u] = i0 + u * NT < n4 ? __ldcg(reinterpret_cast<const int4 *>(h) + i0 + u * NT) : make_int4(-1, -1, -1, -1);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int i = 4 * (i0 + u * NT);
          occurs(i, t[u].x);
          occurs(i + 1, t[u].y);
          occurs(i + 2, t[u].z);
          occurs(i + 3, t[u].w);
        }
      }
      for (int i = 4 * n4 + tid; i < n; i += NT) occurs(i, __ldcg(&h[i]));
    }
    if (tid < p.k && p.draft_tok) {
      const int t = __ldcg(&p.draft_tok[b * p.k + tid]);
      drafts[tid] = t;
      if (t >= c0 && t < c1) touched(atomicOr(&cnt[t - c0], kDraft), t - c0);
    }
    if (p.bias_tok && tid >= NT - 32) {
      // one warp, in list order: a token that is listed twice gets the sum, always alike
      const int lane = tid & 31, n = min(max(__ldcg(&p.bias_len[b]), 0), p.bias_cap);
      const int *tk = p.bias_tok + (size_t)b * p.bias_cap;
      const float *tv = p.bias_val + (size_t)b * p.bias_cap;
      for (int i0 = 0; i0 < n; i0 += 32) {
        const int i = i0 + lane;
        const int t = i < n ? __ldcg(&tk[i]) : -1;
        const float v = i < n ? __ldcg(&tv[i]) : 0.f;
        const bool mine = t >= c0 && t < c1;
        const unsigned peers = __match_any_sync(kFull, mine ? t : -1 - lane);
        const int lead = __ffs(peers) - 1;
        float sum = mine && lane == lead ? bias[t - c0] + v : 0.f;
        if (__any_sync(kFull, lane != lead)) {
#pragma unroll 1
          for (int l = 1; l < 32; ++l) {
            const float x = __shfl_sync(kFull, v, l);
            if (lane == lead && l != lead && (peers >> l & 1u)) sum += x;
          }
        }
        if (mine && lane == lead) {
          bias[t - c0] = sum;
          touched(atomicOr(&cnt[t - c0], kBias), t - c0);
        }
        __syncwarp();
      }
    }
    __syncthreads();
  }

  // Penalties and bias of the touched token at offset o, at position j.
  __device__ __forceinline__ float rule(float x, int o, int j) const {
    const uint32_t c = cnt[o];
    uint32_t n = c & kCount;
    if (c & kDraft)
      for (int d = 0; d < j; ++d) n += drafts[d] == c0 + o;
    if (n || (c & kPrompt)) x = x > 0.f ? __fdiv_rn(x, rep) : x * rep;
    if (n) x = x - freq * (float)n - pres;
    if (c & kBias) x += bias[o];
    return x;
  }
};

// The mask's bits of tokens t .. t + 3 (bits 0 .. 3).
__device__ __forceinline__ uint32_t mask4(const uint32_t *mask, int t) {
  uint32_t m = __ldg(&mask[t >> 5]) >> (t & 31);
  if ((t & 31) > 28) m |= __ldg(&mask[(t >> 5) + 1]) << (32 - (t & 31));
  return m & 0xfu;
}

__device__ __forceinline__ bool mask1(const uint32_t *mask, int t) { return __ldg(&mask[t >> 5]) >> (t & 31) & 1u; }

// -inf into the masked ones of four logits.
__device__ __forceinline__ void cover(float *x, uint32_t m) {
  if (m == 0xfu) return;
  if (m == 0u) {
    *reinterpret_cast<float4 *>(x) = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (!(m >> e & 1u)) x[e] = -INFINITY;
}


// Bulk copy shared memory -> global; 16-byte aligned, a multiple of 16 bytes.
__device__ __forceinline__ void bulk_s2g(void *dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// The same in shared memory: a whole vector read and written has no bank conflicts.
__device__ __forceinline__ void cover_shared(float *x, uint32_t m) {
  if (m == 0xfu) return;
  float4 v = *reinterpret_cast<const float4 *>(x);
  if (!(m & 1u)) v.x = -INFINITY;
  if (!(m & 2u)) v.y = -INFINITY;
  if (!(m & 4u)) v.z = -INFINITY;
  if (!(m & 8u)) v.w = -INFINITY;
  *reinterpret_cast<float4 *>(x) = v;
}

// Rows [j0, j1) of a range by plain loads and stores.
__device__ __noinline__ void plain_rows(const LogitArgs &p, const Range r, int j0, int j1) {
  const int words = (p.V + 31) / 32;
  for (int j = j0; j < j1; ++j) {
    const size_t row = (size_t)r.b * (p.k + 1) + j;
    const uint32_t *mask = p.mask ? p.mask + row * words : nullptr;
    for (int t = r.c0 + threadIdx.x; t < r.c1; t += NT)
      p.out[row * p.V + t] =
          !mask || mask1(mask, t) ? r.rule(__ldcg(p.logits + row * p.V + t), t - r.c0, j) : -INFINITY;
  }
}

constexpr int range_bytes(bool bias) { return CH * (bias ? 10 : 6); }

}  // namespace

// STALL: for the self-test alone, the second row of every CTA is announced and never
// brought, so that its wait runs out.
template <bool STALL>
__global__ void __launch_bounds__(NT) adjust_logits_kernel(const __grid_constant__ LogitArgs p) {
  trace_start(kTkLogits);
  extern __shared__ __align__(128) unsigned char smem[];
  float *ring = reinterpret_cast<float *>(smem);  // [kRing][CH]
  __shared__ int listed, drafts[8], stalled;
  __shared__ __align__(8) uint64_t full[kRing];
  const int tid = threadIdx.x, ranges = (p.V + CH - 1) / CH, words = (p.V + 31) / 32;
  Range r;
  r.cnt = reinterpret_cast<uint32_t *>(ring + kRing * CH);
  r.bias = reinterpret_cast<float *>(r.cnt + CH);
  r.list = reinterpret_cast<uint16_t *>(r.cnt + CH + (p.bias_tok ? CH : 0));
  r.drafts = drafts;
  r.listed = &listed;
  r.b = blockIdx.x / ranges;
  r.c0 = (blockIdx.x % ranges) * CH;
  r.c1 = min(p.V, r.c0 + CH);
  const int n = r.c1 - r.c0;
  // rows of V % 4 != 0 start off a 16-byte boundary: the copies start at the first
  // aligned token and take whole vectors, the few tokens beside them go one by one
  const size_t base0 = (size_t)r.b * (p.k + 1) * p.V + r.c0;
  const unsigned off0 = (unsigned)(base0 & 3), offv = (unsigned)p.V & 3u;
  auto row_base = [&](int j) { return base0 + (size_t)j * p.V; };
  auto row_lead = [&](int j) { return min(n, (int)((4u - ((off0 + j * offv) & 3u)) & 3u)); };
  if (tid == 0) {
    for (int s = 0; s < kRing; ++s) mbar_init(&full[s], 1);
    stalled = p.k + 1;
    fence_barrier_init();
  }
  grid_dep_wait();
  trace_dep(kTkLogits);
  grid_dep_launch();
  const int j0 = blockIdx.y * p.rows, j1 = min(p.k + 1, j0 + p.rows);  // the CTA's rows
  auto bring = [&](int j) {  // thread 0
    const int lead = row_lead(j), nv = (n - lead) / 4;
    const int s = (j - j0) % kRing;
    mbar_arrive_expect_tx(&full[s], STALL && j == j0 + 1 ? 16u : (uint32_t)nv * 16u);
    if (nv && !(STALL && j == j0 + 1)) bulk_g2s(ring + s * CH, p.logits + row_base(j) + lead, (uint32_t)nv * 16u, &full[s]);
  };
  if (tid == 0)
    for (int j = j0; j < j1 && j < j0 + kRing; ++j) bring(j);
  uint32_t next_mask[VPT];
  auto fetch_mask = [&](int j) {
    const int lead = row_lead(j), nv = (n - lead) / 4;
    const uint32_t *mask = p.mask + ((size_t)r.b * (p.k + 1) + j) * words;
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
      const int i = tid + u * NT, t = r.c0 + lead + 4 * i;
      next_mask[u] = 0xfu;
      if (i < nv) next_mask[u] = offv | off0 ? mask4(mask, t) : __ldg(&mask[t >> 5]) >> (t & 31) & 0xfu;
    }
  };
  if (p.mask) fetch_mask(j0);
  r.build(p);

  const int n_list = listed;
  int missed = j1;  // the first row whose load this thread has given up on
  for (int j = j0; j < j1; ++j) {
    const int lead = row_lead(j), nv = (n - lead) / 4, s = (j - j0) % kRing;
    float *row = ring + s * CH;
    const uint32_t *mask = p.mask ? p.mask + ((size_t)r.b * (p.k + 1) + j) * words : nullptr;
    uint32_t m[VPT];
#pragma unroll
    for (int u = 0; u < VPT; ++u) m[u] = next_mask[u];
    if (p.mask && j + 1 < j1) fetch_mask(j + 1);
    if (missed == j1 && !mbar_wait(&full[s], (uint32_t)((j - j0) / kRing) & 1u, nullptr)) {
      missed = j;
      atomicMin(&stalled, j);
    }
    for (int i = tid; i < n_list; i += NT) {
      const int o = r.list[i], at = o - lead;
      if (at >= 0 && at < 4 * nv) row[at] = r.rule(row[at], o, j);
    }
    if (p.mask) {  // the mask last: it wins over every other rule
      if (n_list) __syncthreads();
#pragma unroll
      for (int u = 0; u < VPT; ++u)
        if (tid + u * NT < nv) cover_shared(row + 4 * (tid + u * NT), m[u]);
    }
    // the tokens before the first vector and behind the last
    const int tail = lead + 4 * nv, singles = lead + (n - tail);
    if (tid < singles) {
      const int o = tid < lead ? tid : tail + tid - lead;
      p.out[row_base(j) + o] =
          !mask || mask1(mask, r.c0 + o) ? r.rule(__ldcg(p.logits + row_base(j) + o), o, j) : -INFINITY;
    }
    fence_proxy_async_smem();
    __syncthreads();
    if (tid == 0 && missed == j1) {
      if (nv) bulk_s2g(p.out + row_base(j) + lead, row, (uint32_t)nv * 16u);
      bulk_commit();
      // the row kRing ahead takes this row's place once the copy out has read it
      if (j + kRing < j1) {
        bulk_wait_read();
        bring(j + kRing);
      }
    }
  }
  if (tid == 0) bulk_wait_all();
  // A load that did not land within the wait limit: the rows from there on may have
  // been copied out as they were, and are written again.  What thread 0 has brought
  // since has the limit once more to land before the CTA exits.
  if (const int from = stalled; from < j1) {
    if (tid == 0)
      for (int j = missed; j < j1 && j < missed + kRing; ++j)
        mbar_wait(&full[(j - j0) % kRing], (uint32_t)((j - j0) / kRing) & 1u, nullptr);
    __syncthreads();
    plain_rows(p, r, from, j1);
  }
  trace_end(kTkLogits);
}

// In place: the masked logits are overwritten, then the touched ones recomputed.
__global__ void __launch_bounds__(NT) adjust_logits_in_place_kernel(const __grid_constant__ LogitArgs p) {
  trace_start(kTkLogits);
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int listed, drafts[8];
  const int tid = threadIdx.x, ranges = (p.V + CH - 1) / CH, words = (p.V + 31) / 32;
  Range r;
  r.cnt = reinterpret_cast<uint32_t *>(smem);
  r.bias = reinterpret_cast<float *>(r.cnt + CH);
  r.list = reinterpret_cast<uint16_t *>(r.cnt + CH + (p.bias_tok ? CH : 0));
  r.drafts = drafts;
  r.listed = &listed;
  r.b = blockIdx.x / ranges;
  r.c0 = (blockIdx.x % ranges) * CH;
  r.c1 = min(p.V, r.c0 + CH);
  const int n = r.c1 - r.c0;
  grid_dep_wait();
  trace_dep(kTkLogits);
  grid_dep_launch();
  r.build(p);
  const int j0 = blockIdx.y * p.rows, j1 = min(p.k + 1, j0 + p.rows);
  for (int j = j0; j < j1; ++j) {
    const size_t base = ((size_t)r.b * (p.k + 1) + j) * p.V + r.c0;
    const uint32_t *mask = p.mask ? p.mask + ((size_t)r.b * (p.k + 1) + j) * words : nullptr;
    float *row = p.out + base;
    if (mask) {
      const int lead = min(n, (int)((4 - (base & 3)) & 3)), nv = (n - lead) / 4, tail = lead + 4 * nv;
      uint32_t m[VPT];
#pragma unroll
      for (int u = 0; u < VPT; ++u) m[u] = tid + u * NT < nv ? mask4(mask, r.c0 + lead + 4 * (tid + u * NT)) : 0xfu;
#pragma unroll
      for (int u = 0; u < VPT; ++u)
        if (tid + u * NT < nv) cover(row + lead + 4 * (tid + u * NT), m[u]);
      if (tid < lead + (n - tail)) {
        const int o = tid < lead ? tid : tail + tid - lead;
        if (!mask1(mask, r.c0 + o)) row[o] = -INFINITY;
      }
    }
    for (int i = tid; i < listed; i += NT) {
      const int o = r.list[i];
      if (mask && !mask1(mask, r.c0 + o)) continue;
      row[o] = r.rule(row[o], o, j);
    }
  }
  trace_end(kTkLogits);
}

cudaError_t logits_set_attributes() {
  cudaError_t e = cudaFuncSetAttribute(adjust_logits_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       range_bytes(true) + kRing * CH * 4);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(adjust_logits_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             range_bytes(true) + kRing * CH * 4);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(adjust_logits_in_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             range_bytes(true));
  return e;
}

cudaError_t launch_adjust_logits(const LogitArgs &args, int sms, cudaStream_t s, bool pdl, bool stall) {
  LogitArgs a = args;
  const bool in_place = a.logits == a.out;
  const long long ranges = (long long)a.B * ((a.V + CH - 1) / CH);
  // One scan of the history serves all rows of a range; with few ranges the rows
  // go to CTAs of their own instead, each with its scan (us, one row a CTA / all): 4 rows
  // of 151936, 1 sequence 7.3 / 11.5, 2 10.1 / 11.7, 4 13.4 / 12.6, 5 14.1 / 13.3, 8 18.6 / 15.9;
  // 6 rows of 32000, 8 sequences 9.7 / 15.5, 16 15.3 / 16.0, 19 16.6 / 16.2, 24 20.0 / 17.2.
  a.rows = stall || ranges >= 2 * sms ? a.k + 1 : 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)ranges, (unsigned)((a.k + a.rows) / a.rows));
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = range_bytes(a.bias_tok != nullptr) + (in_place ? 0 : kRing * CH * 4);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  note_launch();
  if (in_place) return cudaLaunchKernelEx(&cfg, adjust_logits_in_place_kernel, a);
  return stall ? cudaLaunchKernelEx(&cfg, adjust_logits_kernel<true>, a)
               : cudaLaunchKernelEx(&cfg, adjust_logits_kernel<false>, a);
}

MTP_TRACE_COLLECTOR(logits)

}  // namespace mtp
