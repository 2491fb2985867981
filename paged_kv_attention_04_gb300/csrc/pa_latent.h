// Internal declarations of the latent-attention calls.
#pragma once

#include "pa_internal.h"

namespace pa {

constexpr int kLatentRope = 64;       // numbers of the shared key part
constexpr int kLatentMaxHeads = 256;
constexpr int kLatentMaxCtas = 152;  // of the bf16 kernel: workspaces are sized for them

struct LatentWriteArgs {
  const void *c, *k;
  long long c_stride, k_stride;
  const void* weight;
  float eps;
  const void* q;  // null: the cache alone
  long long q_stride, q_head_stride;
  const pa_rope* rope;
  const int64_t* slots;
  int num_tokens;
  void* q_out;
  long long qo_stride, qo_head_stride;
  void* cache;
  int32_t* status;
};
cudaError_t launch_latent_write(const LatentWriteArgs& a, const pa_latent_layout& L, cudaStream_t stream);
cudaError_t launch_latent_read(const void* cache, const int64_t* slots, int num_tokens, void* c,
                               void* k, const pa_latent_layout& L, int32_t* status,
                               cudaStream_t stream);

// One step of attention over a latent cache.
struct LatentParams {
  const void* q;      // [T][H][R + 64]
  const void* cache;  // [NB][16][R + 64]
  const int32_t* block_tables;
  const int32_t* seq_lens;
  const int32_t* qsl;
  void* out;  // [T][H][R]
  int max_blocks_per_seq, num_seqs, num_tokens, max_query_len, max_seq_len, num_heads, num_blocks;
  float scale_log2;  // softmax scale x log2(e)
  int splits;        // fp32: pieces of every request's keys
  float* part_acc;   // partial sums, and per row {maximum, sum}
  float* part_ml;
  int4* recs;  // bf16: per CTA and slot, what piece it holds
  int32_t* status;
};

// One step of attention over expanded keys and values.
struct ExpandedParams {
  const void *q, *k, *kr, *v;
  const int32_t* qsl;
  const int32_t* kvsl;
  void* out;
  int num_seqs, num_tokens, num_kv_tokens, max_query_len, max_kv_len, num_heads;
  long long q_stride, q_head_stride, k_stride, k_head_stride, kr_stride, v_stride, v_head_stride;
  float scale_log2;
  int32_t* status;
  // bf16: partial states of units cut in pieces, and per CTA a record; null: units are not cut
  float4* part_acc;   // [slot][D / 4][rows of a unit]
  float2* part_ml;    // [slot][rows]: maximum, sum
  int4* recs;
};

// fp32: CUDA cores.
cudaError_t launch_latent_cc(const LatentParams& p, int latent_size, cudaStream_t stream);
cudaError_t launch_expanded_cc(const ExpandedParams& p, int head_size, cudaStream_t stream);
// Rows of partial states that the bf16 kernel may leave.
size_t latent_tc_partial_rows(int num_heads, int max_query_len);
// bf16: tensor cores (tcgen05).
cudaError_t launch_latent_tc(const LatentParams& p, int latent_size, int num_sms, cudaStream_t stream);
// Rows of partial states that its units may leave; 0 where cutting them is of no use.
size_t expanded_tc_partial_rows(int num_heads, int num_tokens, int max_kv_len);
cudaError_t launch_expanded_tc(const ExpandedParams& p, int head_size, int num_sms, cudaStream_t stream);

}  // namespace pa
