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
// state is kept from step to step, and no global atomics are needed.  In place,
// only what a rule changes is read and written.
#include "common.cuh"
#include "internal.h"
#include "logits.cuh"

namespace mtp {

namespace {

constexpr int kLgThreads = 256;
constexpr uint32_t kPrompt = 0x80000000u;  // the token occurs in the prompt; the low bits count
constexpr unsigned kFull = 0xffffffffu;

}  // namespace

// VPT: vectors of four logits a thread holds per row; the range is VPT * 1024 tokens.
template <int VPT, bool IN_PLACE>
__global__ void __launch_bounds__(kLgThreads) adjust_logits_kernel(const __grid_constant__ LogitArgs p) {
  trace_start(kTkLogits);
  constexpr int CH = VPT * 4 * kLgThreads;
  extern __shared__ __align__(16) unsigned char smem[];
  uint32_t *cnt = reinterpret_cast<uint32_t *>(smem);  // [CH + 4]
  float *bias = reinterpret_cast<float *>(smem + (CH + 4) * 4);
  const int tid = threadIdx.x, ranges = (p.V + CH - 1) / CH, b = blockIdx.x / ranges;
  const int c0 = (blockIdx.x % ranges) * CH, c1 = min(p.V, c0 + CH);
  grid_dep_wait();
  trace_dep(kTkLogits);
  grid_dep_launch();

  // ---- counters and biases of the range
  for (int i = tid; i < (CH + 4) / 4; i += kLgThreads) {
    reinterpret_cast<uint4 *>(cnt)[i] = make_uint4(0u, 0u, 0u, 0u);
    if (p.bias_tok) reinterpret_cast<float4 *>(bias)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __syncthreads();
  if (p.history) {
    const int n = min(max(__ldcg(&p.hist_len[b]), 0), p.hist_cap);
    const int np = p.prompt_len ? min(max(__ldcg(&p.prompt_len[b]), 0), n) : 0;
    const int *h = p.history + (size_t)b * p.hist_cap;
    for (int i0 = tid; i0 < n; i0 += 8 * kLgThreads) {
      int t[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) t[u] = i0 + u * kLgThreads < n ? __ldcg(&h[i0 + u * kLgThreads]) : -1;
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (t[u] >= c0 && t[u] < c1) {
          if (i0 + u * kLgThreads < np) atomicOr(&cnt[t[u] - c0], kPrompt);
          else atomicAdd(&cnt[t[u] - c0], 1u);
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
      unsigned peers = __match_any_sync(kFull, mine ? t : -1 - tid);
      const int lead = __ffs(peers) - 1;
      float sum = mine && tid == lead ? bias[t - c0] : 0.f;
#pragma unroll 1
      for (int l = 0; l < 32; ++l) {
        const float x = __shfl_sync(kFull, v, l);
        if (tid == lead && (peers >> l & 1u)) sum += x;
      }
      if (mine && tid == lead) bias[t - c0] = sum;
      __syncwarp();
    }
  }
  const float rep = p.rep ? __ldcg(&p.rep[b]) : 1.f, freq = p.freq ? __ldcg(&p.freq[b]) : 0.f,
              pres = p.pres ? __ldcg(&p.pres[b]) : 0.f;
  __syncthreads();

  const int words = (p.V + 31) / 32;
  auto rule = [&](float x, uint32_t c, float bv, bool allowed) {
    if (c) {
      x = x > 0.f ? __fdiv_rn(x, rep) : x * rep;
      const uint32_t n = c & ~kPrompt;
      if (n) x = x - freq * (float)n - pres;
    }
    if (p.bias_tok) x += bv;
    return allowed ? x : -INFINITY;
  };

  for (int j = 0; j <= p.k; ++j) {
    const size_t base = ((size_t)b * (p.k + 1) + j) * p.V;
    const float *src = p.logits + base;
    float *dst = p.out + base;
    const uint32_t *mask = p.mask ? p.mask + ((size_t)b * (p.k + 1) + j) * words : nullptr;
    // rows of V % 4 != 0 start off a 16-byte boundary: the vectors start at the
    // first aligned token, the few tokens beside them go one by one
    const int lead = min(c1 - c0, (int)((4 - ((base + c0) & 3)) & 3));
    const int nv = (c1 - c0 - lead) / 4;
    float4 x[VPT];
    if (!IN_PLACE) {
#pragma unroll
      for (int u = 0; u < VPT; ++u) {
        const int i = tid + u * kLgThreads;
        if (i < nv) x[u] = __ldcs(reinterpret_cast<const float4 *>(src + c0 + lead) + i);
      }
    }
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
      const int i = tid + u * kLgThreads;
      if (i < nv) {
        const int o = lead + 4 * i, t = c0 + o;
        uint32_t bits = 0xfu;
        if (mask) {
          bits = __ldg(&mask[t >> 5]) >> (t & 31);
          if ((t & 31) > 28) bits |= __ldg(&mask[(t >> 5) + 1]) << (32 - (t & 31));
        }
        uint32_t n[4];
        float bv[4] = {0.f, 0.f, 0.f, 0.f};
        if (lead == 0) {
          const uint4 v = *reinterpret_cast<const uint4 *>(cnt + o);
          n[0] = v.x; n[1] = v.y; n[2] = v.z; n[3] = v.w;
          if (p.bias_tok) {
            const float4 w = *reinterpret_cast<const float4 *>(bias + o);
            bv[0] = w.x; bv[1] = w.y; bv[2] = w.z; bv[3] = w.w;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            n[e] = cnt[o + e];
            if (p.bias_tok) bv[e] = bias[o + e];
          }
        }
        const bool touched = (bits & 0xfu) != 0xfu || (n[0] | n[1] | n[2] | n[3]) || bv[0] != 0.f || bv[1] != 0.f ||
                             bv[2] != 0.f || bv[3] != 0.f;
        if (IN_PLACE) {
          if (!touched) continue;
          x[u] = (bits & 0xfu) ? reinterpret_cast<const float4 *>(src + c0 + lead)[i] : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        if (touched) {
          x[u].x = rule(x[u].x, n[0], bv[0], bits & 1u);
          x[u].y = rule(x[u].y, n[1], bv[1], bits & 2u);
          x[u].z = rule(x[u].z, n[2], bv[2], bits & 4u);
          x[u].w = rule(x[u].w, n[3], bv[3], bits & 8u);
        }
        __stcs(reinterpret_cast<float4 *>(dst + c0 + lead) + i, x[u]);
      }
    }
    // the tokens before the first vector and behind the last
    const int tail = lead + 4 * nv, singles = lead + (c1 - c0 - tail);
    if (tid < singles) {
      const int o = tid < lead ? tid : tail + tid - lead, t = c0 + o;
      const bool allowed = !mask || (__ldg(&mask[t >> 5]) >> (t & 31) & 1u);
      dst[t] = rule(src[t], cnt[o], p.bias_tok ? bias[o] : 0.f, allowed);
    }
    if (j < p.k && p.draft_tok) {
      const int t = __ldcg(&p.draft_tok[b * p.k + j]);
      __syncthreads();  // every thread has read the counters of row j
      if (tid == 0 && t >= c0 && t < c1) cnt[t - c0] += 1u;
      __syncthreads();
    }
  }
  trace_end(kTkLogits);
}

namespace {

template <int VPT, bool IN_PLACE>
cudaError_t launch_one(const LogitArgs &a, cudaStream_t s, bool pdl) {
  constexpr int CH = VPT * 4 * kLgThreads;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(a.V + CH - 1) / CH * (unsigned)a.B);
  cfg.blockDim = dim3(kLgThreads);
  cfg.dynamicSmemBytes = (CH + 4) * 4 * (a.bias_tok ? 2 : 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  note_launch();
  return cudaLaunchKernelEx(&cfg, adjust_logits_kernel<VPT, IN_PLACE>, a);
}

template <int VPT>
cudaError_t launch_vpt(const LogitArgs &a, cudaStream_t s, bool pdl) {
  return a.logits == a.out ? launch_one<VPT, true>(a, s, pdl) : launch_one<VPT, false>(a, s, pdl);
}

template <int VPT>
cudaError_t set_smem() {
  const int bytes = (VPT * 4 * kLgThreads + 4) * 8;
  cudaError_t e = cudaFuncSetAttribute(adjust_logits_kernel<VPT, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(adjust_logits_kernel<VPT, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  return e;
}

}  // namespace

cudaError_t logits_set_attributes() {
  cudaError_t e = set_smem<1>();
  if (e == cudaSuccess) e = set_smem<2>();
  if (e == cudaSuccess) e = set_smem<4>();
  if (e == cudaSuccess) e = set_smem<8>();
  return e;
}

cudaError_t launch_adjust_logits(const LogitArgs &a, int sms, cudaStream_t s, bool pdl) {
  // the widest range (fewest scans of the history) that still fills the GPU twice
  auto ctas = [&](int vpt) { return (long long)a.B * ((a.V + vpt * 1024 - 1) / (vpt * 1024)); };
  if (ctas(8) >= 2 * sms) return launch_vpt<8>(a, s, pdl);
  if (ctas(4) >= 2 * sms) return launch_vpt<4>(a, s, pdl);
  if (ctas(2) >= 2 * sms) return launch_vpt<2>(a, s, pdl);
  return launch_vpt<1>(a, s, pdl);
}

MTP_TRACE_COLLECTOR(logits)

}  // namespace mtp
