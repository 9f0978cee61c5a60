// Rules on the target's logits before verification: penalties for repeated
// tokens, biases and a grammar mask, at every candidate position of a sequence.
//
// Position j of sequence b follows the history and the drafts 0 .. j-1.  With
// c = how often token v occurs in the generated part of the history and in
// those drafts, and seen = c > 0 or v occurs in the prompt:
//   x = l(v);  seen: x = x > 0 ? x / rep : x * rep
//   x -= freq * c;  c > 0: x -= pres;  x += bias(v);  v masked: x = -inf
//
// Bound by the logits' bytes.  A CTA owns one range of the vocabulary for all
// k + 1 rows of a sequence: it scans the sequence's history once (4 bytes a
// token, from L2 after the first CTA) into counters in shared memory, adds the
// biases of its range, then streams its part of each row, adding draft j's
// count between rows j and j + 1.  So the counters never go to memory, no
// state is kept from step to step, and no global atomics are needed.  A bit a
// token says which have a count or a bias, so that all others pay for the mask
// alone.  In place, only what a rule changes is read and written.
#include <stdlib.h>

#include "common.cuh"
#include "internal.h"
#include "logits.cuh"

namespace mtp {

namespace {

constexpr uint32_t kPrompt = 0x80000000u;  // the token occurs in the prompt; the low bits count
constexpr unsigned kFull = 0xffffffffu;

}  // namespace

// VPT: vectors of four logits a thread holds per row; the range is VPT * 4 * NT tokens.
template <int NT, int VPT, bool IN_PLACE>
__global__ void __launch_bounds__(NT) adjust_logits_kernel(const __grid_constant__ LogitArgs p) {
  trace_start(kTkLogits);
  constexpr int CH = VPT * 4 * NT;
  extern __shared__ __align__(16) unsigned char smem[];
  uint32_t *dirty = reinterpret_cast<uint32_t *>(smem);       // [CH / 32 + 1] tokens with a count or a bias
  uint32_t *cnt = dirty + CH / 32 + 4;                        // [CH]
  float *bias = reinterpret_cast<float *>(cnt + CH);          // [CH]
  const int tid = threadIdx.x, ranges = (p.V + CH - 1) / CH, b = blockIdx.x / ranges;
  const int c0 = (blockIdx.x % ranges) * CH, c1 = min(p.V, c0 + CH);
  grid_dep_wait();
  trace_dep(kTkLogits);
  grid_dep_launch();

  // rows of V % 4 != 0 start off a 16-byte boundary: the vectors start at the
  // first aligned token, the few tokens beside them go one by one
  const int words = (p.V + 31) / 32;
  auto row_base = [&](int j) { return ((size_t)b * (p.k + 1) + j) * p.V; };
  auto row_lead = [&](size_t base) { return min(c1 - c0, (int)((4 - ((base + c0) & 3)) & 3)); };
  auto row_mask = [&](int j) { return p.mask + ((size_t)b * (p.k + 1) + j) * words; };
  auto allowed4 = [&](const uint32_t *mask, int t) {  // the bits of tokens t .. t + 3
    uint32_t m = __ldg(&mask[t >> 5]) >> (t & 31);
    if ((t & 31) > 28) m |= __ldg(&mask[(t >> 5) + 1]) << (32 - (t & 31));
    return m & 0xfu;
  };
  float4 nx[VPT];
  uint32_t nm[VPT];
  auto fetch = [&](int j) {
    const size_t base = row_base(j);
    const int lead = row_lead(base), nv = (c1 - c0 - lead) / 4;
    const float4 *s4 = reinterpret_cast<const float4 *>(p.logits + base + c0 + lead);
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
      const int i = tid + u * NT;
      nm[u] = 0xfu;
      if (i < nv) {
        if (!IN_PLACE) nx[u] = __ldcs(s4 + i);
        if (p.mask) nm[u] = allowed4(row_mask(j), c0 + lead + 4 * i);
      }
    }
  };
  fetch(0);  // under the history's scan

  // ---- counters and biases of the range
  for (int i = tid; i < CH / 4; i += NT) {
    reinterpret_cast<uint4 *>(cnt)[i] = make_uint4(0u, 0u, 0u, 0u);
    if (p.bias_tok) reinterpret_cast<float4 *>(bias)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  for (int i = tid; i < CH / 32 + 4; i += NT) dirty[i] = 0u;
  __syncthreads();
  auto mark = [&](int o) { atomicOr(&dirty[o >> 5], 1u << (o & 31)); };
  if (p.history) {
    const int n = min(max(__ldcg(&p.hist_len[b]), 0), p.hist_cap);
    const int np = p.prompt_len ? min(max(__ldcg(&p.prompt_len[b]), 0), n) : 0;
    const int *h = p.history + (size_t)b * p.hist_cap;
    for (int i0 = tid; i0 < n; i0 += 8 * NT) {
      int t[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) t[u] = i0 + u * NT < n ? __ldcg(&h[i0 + u * NT]) : -1;
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (t[u] >= c0 && t[u] < c1) {
          if (i0 + u * NT < np) atomicOr(&cnt[t[u] - c0], kPrompt);
          else atomicAdd(&cnt[t[u] - c0], 1u);
          mark(t[u] - c0);
        }
    }
  }
  if (p.bias_tok && tid < 32) {
    // one warp, in list order: a token that is listed twice gets the sum, always alike
    const int n = min(max(__ldcg(&p.bias_len[b]), 0), p.bias_cap);
    const int *tk = p.bias_tok + (size_t)b * p.bias_cap;
    const float *tv = p.bias_val + (size_t)b * p.bias_cap;
    for (int i0 = 0; i0 < n; i0 += 32) {
      const int i = i0 + tid;
      const int t = i < n ? __ldcg(&tk[i]) : -1;
      const float v = i < n ? __ldcg(&tv[i]) : 0.f;
      const bool mine = t >= c0 && t < c1;
      const unsigned peers = __match_any_sync(kFull, mine ? t : -1 - tid);
      const int lead = __ffs(peers) - 1;
      float sum = mine && tid == lead ? bias[t - c0] + v : 0.f;
      if (__any_sync(kFull, tid != lead)) {
#pragma unroll 1
        for (int l = 1; l < 32; ++l) {
          const float x = __shfl_sync(kFull, v, l);
          if (tid == lead && l != lead && (peers >> l & 1u)) sum += x;
        }
      }
      if (mine && tid == lead) {
        bias[t - c0] = sum;
        mark(t - c0);
      }
      __syncwarp();
    }
  }
  const float rep = p.rep ? __ldcg(&p.rep[b]) : 1.f, freq = p.freq ? __ldcg(&p.freq[b]) : 0.f,
              pres = p.pres ? __ldcg(&p.pres[b]) : 0.f;
  __syncthreads();

  // penalties and bias of the token at offset o of the range
  auto rule = [&](float x, int o) {
    const uint32_t c = cnt[o];
    if (c) {
      x = x > 0.f ? __fdiv_rn(x, rep) : x * rep;
      const uint32_t n = c & ~kPrompt;
      if (n) x = x - freq * (float)n - pres;
    }
    if (p.bias_tok) x += bias[o];
    return x;
  };

  for (int j = 0; j <= p.k; ++j) {
    const size_t base = row_base(j);
    const float *src = p.logits + base;
    float *dst = p.out + base;
    const int lead = row_lead(base), nv = (c1 - c0 - lead) / 4;
    float4 x[VPT];
    uint32_t m[VPT];
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
      x[u] = nx[u];
      m[u] = nm[u];
    }
    if (j < p.k) fetch(j + 1);  // the next row's loads run under this row's rules and stores
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
      const int i = tid + u * NT;
      if (i >= nv) continue;
      const int o = lead + 4 * i;
      uint32_t d = dirty[o >> 5] >> (o & 31);  // most tokens have no rule but the mask
      if (lead && (o & 31) > 28) d |= dirty[(o >> 5) + 1] << (32 - (o & 31));
      d &= 0xfu;
      float4 *at = reinterpret_cast<float4 *>(dst + c0 + o);
      if (IN_PLACE) {
        if (m[u] == 0xfu && !d) continue;
        x[u] = m[u] ? *at : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      if (d) {
        if (d & 1u) x[u].x = rule(x[u].x, o);
        if (d & 2u) x[u].y = rule(x[u].y, o + 1);
        if (d & 4u) x[u].z = rule(x[u].z, o + 2);
        if (d & 8u) x[u].w = rule(x[u].w, o + 3);
      }
      if (!(m[u] & 1u)) x[u].x = -INFINITY;
      if (!(m[u] & 2u)) x[u].y = -INFINITY;
      if (!(m[u] & 4u)) x[u].z = -INFINITY;
      if (!(m[u] & 8u)) x[u].w = -INFINITY;
      __stcs(at, x[u]);
    }
    // the tokens before the first vector and behind the last
    const int tail = lead + 4 * nv, singles = lead + (c1 - c0 - tail);
    if (tid < singles) {
      const int o = tid < lead ? tid : tail + tid - lead, t = c0 + o;
      const bool allowed = !p.mask || (__ldg(&row_mask(j)[t >> 5]) >> (t & 31) & 1u);
      const float y = rule(src[t], o);
      dst[t] = allowed ? y : -INFINITY;
    }
    if (j < p.k && p.draft_tok) {
      const int t = __ldcg(&p.draft_tok[b * p.k + j]);
      __syncthreads();  // every thread has read the counters of row j
      if (tid == 0 && t >= c0 && t < c1) {
        cnt[t - c0] += 1u;
        mark(t - c0);
      }
      __syncthreads();
    }
  }
  trace_end(kTkLogits);
}

namespace {

template <int NT, int VPT, bool IN_PLACE>
cudaError_t launch_one(const LogitArgs &a, cudaStream_t s, bool pdl) {
  constexpr int CH = VPT * 4 * NT;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(a.V + CH - 1) / CH * (unsigned)a.B);
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = (CH / 32 + 4 + CH * (a.bias_tok ? 2 : 1)) * 4;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  note_launch();
  return cudaLaunchKernelEx(&cfg, adjust_logits_kernel<NT, VPT, IN_PLACE>, a);
}

template <int NT, int VPT>
cudaError_t launch_width(const LogitArgs &a, cudaStream_t s, bool pdl) {
  return a.logits == a.out ? launch_one<NT, VPT, true>(a, s, pdl) : launch_one<NT, VPT, false>(a, s, pdl);
}

template <int NT, int VPT>
cudaError_t set_smem() {
  constexpr int CH = VPT * 4 * NT, bytes = (CH / 32 + 4 + 2 * CH) * 4;
  cudaError_t e = cudaFuncSetAttribute(adjust_logits_kernel<NT, VPT, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(adjust_logits_kernel<NT, VPT, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  return e;
}

}  // namespace

cudaError_t logits_set_attributes() {
  cudaError_t e = set_smem<256, 1>();
  if (e == cudaSuccess) e = set_smem<512, 1>();
  if (e == cudaSuccess) e = set_smem<512, 2>();
  if (e == cudaSuccess) e = set_smem<512, 4>();
  return e;
}

cudaError_t launch_adjust_logits(const LogitArgs &a, int sms, cudaStream_t s, bool pdl) {
  // the widest range (fewest scans of the history) that still fills the GPU
  // several times over; a single sequence takes the narrowest
  auto ctas = [&](int ch) { return (long long)a.B * ((a.V + ch - 1) / ch); };
  int width = 0;
  if (const char *v = getenv("MTP_LG")) width = atoi(v);
  if (width == 8192 || (!width && ctas(8192) >= 4 * sms)) return launch_width<512, 4>(a, s, pdl);
  if (width == 4096 || (!width && ctas(4096) >= 4 * sms)) return launch_width<512, 2>(a, s, pdl);
  if (width == 2048 || (!width && ctas(2048) >= 2 * sms)) return launch_width<512, 1>(a, s, pdl);
  return launch_width<256, 1>(a, s, pdl);
}

MTP_TRACE_COLLECTOR(logits)

}  // namespace mtp
