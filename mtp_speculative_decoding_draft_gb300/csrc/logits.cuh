// Arguments of the rules on the target's logits (logits.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace mtp {

constexpr int kTkLogits = 64;  // trace kind: MTP_TK_LOGITS

struct LogitArgs {
  int B, k, V;
  const int *history;     // [B, hist_cap] or null
  int hist_cap;
  const int *prompt_len;  // [B] or null (0)
  const int *hist_len;    // [B]
  const float *rep, *freq, *pres;  // [B] or null
  const int *bias_tok;    // [B, bias_cap] or null
  const float *bias_val;
  const int *bias_len;    // [B]
  int bias_cap;
  const uint32_t *mask;   // [B, k + 1, ceil(V / 32)] or null
  const float *logits;    // [B, k + 1, V]
  float *out;             // the same, or logits itself
  const int *draft_tok;   // [B, k] or null
  int rows;               // rows of a CTA (set by the launch)
};
cudaError_t logits_set_attributes();
// stall: the self-test's kernel, in which the second row of every CTA never arrives
cudaError_t launch_adjust_logits(const LogitArgs &a, int sms, cudaStream_t s, bool pdl, bool stall);

}  // namespace mtp
