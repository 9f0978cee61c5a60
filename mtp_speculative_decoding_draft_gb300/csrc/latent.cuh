// Shared by the latent-attention kernels: the calls' arguments.
//
// A target with latent attention keeps, of each token, one vector of R elements
// (the latent) and one rotated key part of Dr elements, in a row of R + Dr in
// the pages of a cache.  Absorbed, the row is the key of every head and its first
// R elements are the value; expanded, each head has keys and values of its own,
// formed from the latent.
#pragma once

#include "paged.cuh"

namespace mtp {

// trace kinds: the MTP_TK_* values of the public header
constexpr int kTkLatentAppend = 70, kTkLatentHeads = 71, kTkLatentAttn = 72, kTkLatentPrefill = 73;

struct LatentAppendArgs {
  int B, Hq, R, Dr, page, page_shift, n_pages, max_pages, cap, n_rows;
  int rot, layout;  // rot 0: no rotation
  const unsigned long long *turns;
  float scale, eps;
  const int *row_start, *ctx_len, *page_table;
  const uint16_t *kv, *gain, *q;  // gain null: the latents are copied; q null: keys only
  uint16_t *q_out, *pages;
  long long ldkv, ldq, hsq, ldqo, hsqo;
  int *status;
};
cudaError_t launch_latent_append(const LatentAppendArgs &a, int sms, cudaStream_t s, bool pdl);

// y[n, h, :] = W[h] x[n, h, :], or, with pages, of the rows of a cache's sequences
// (x shared by the heads).
struct LatentHeadsArgs {
  int n_rows, H, K, N, transposed;
  const uint16_t *x, *w;  // W[h] is [N, K], or [K, N] where transposed
  uint16_t *y;
  long long ldx, hsx, ldw, hsw, ldy, hsy;
  int *status;
  // rows from the pages of a cache (pages null: from x)
  const uint16_t *pages;
  int B, Dr, page, page_shift, n_pages, max_pages, cap;
  const int *key_start, *page_table;
  uint16_t *k_rope;
  long long ldkr;
};
cudaError_t launch_latent_heads(const LatentHeadsArgs &a, int sms, cudaStream_t s, bool pdl);

// Absorbed attention: PagedArgs with Hq = G heads, Dh the latent's size, q rows of Hq * (Dh + rope).
struct LatentAttnArgs {
  PagedArgs a;
  int Dr;
  const uint16_t *pages;
};
size_t latent_attn_scratch_bytes(int B, int n_rows, int H, int R);
cudaError_t launch_latent_attn(const LatentAttnArgs &la, void *scratch, int sms, cudaStream_t s, bool pdl);

// Attention over keys and values of each head: PagedArgs with Hkv = Hq, G = 1.
struct LatentPrefillArgs {
  PagedArgs a;
  int Dn, Dr, Dv, n_keys;
  const int *key_start;
  const uint16_t *kv, *k_rope;
  long long ldkv, ldkr;
};
size_t latent_prefill_scratch_bytes(int B, int n_rows, int H, int Dv);
cudaError_t launch_latent_prefill(const LatentPrefillArgs &lp, void *scratch, int sms, cudaStream_t s, bool pdl);

// The same on pairs of CTAs (latent_attn_pair.cu).
size_t latent_pair_scratch_bytes(int B, int n_rows, int H, int R);
cudaError_t launch_latent_attn_pair(const LatentAttnArgs &la, void *scratch, int sms, cudaStream_t s, bool pdl);
cudaError_t latent_pair_set_attributes();

cudaError_t latent_set_attributes();
cudaError_t latent_prefill_set_attributes();
cudaError_t latent_heads_set_attributes();

}  // namespace mtp
