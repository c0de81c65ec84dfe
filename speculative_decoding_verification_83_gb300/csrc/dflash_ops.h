// dflash_ops.h -- parameters and launchers of the operators around the
// verification step: the paged key/value append (dflash_kvappend.cu), the
// attention over the paged cache (dflash_attention.cu) and the drafter's
// distillation loss (dflash_distill.cu). The entry points and their argument
// checks are in dflash_ops_abi.cu.
#pragma once

#include <cstddef>
#include <cstdint>

namespace dflash {

// SMs the calling thread's current context may use (dflash_abi.cu).
int context_sms(int dev);

constexpr int kOpsMaxB = 2048;

// The requests of a packed batch: request b's new tokens are q_start[b] ..
// q_start[b + 1] - 1, or b * q_per ... when q_start is null.
struct PackedTokens {
  const int32_t* q_start;
  int tokens, B, q_per;
};

// A paged cache as the kernels address it: all strides in 16-byte units.
struct PagedView {
  unsigned char *k, *v;
  const int32_t* table;
  long long table_stride;
  uint32_t page_s, head_s, slot_s;
  int num_pages, page_size, page_shift;  // page_shift: log2(page_size), or -1
  int max_pages, kv_heads;
  const float *k_scale, *v_scale;  // e4m3 caches: stored value = value / scale (null: 1)
};

struct AppendParams {
  PagedView c;
  PackedTokens tk;
  const unsigned char *k, *v, *q;  // 16-bit values
  unsigned char* q_out;
  long long k_ts, k_hs, v_ts, v_hs, q_ts, q_hs, qo_ts, qo_hs;  // token and head strides in elements
  int q_heads;
  const int32_t* lens;
  const unsigned long long* phases;  // turns per token, 64-bit fixed point
  int rot, interleaved;
  int norm;                            // keys and queries are normed first,
  const void *q_weight, *k_weight;     // with weights [head_dim] (null: 1)
  int weight_f32;                      // in fp32, or in the tokens' type
  float eps;
  uint32_t* status;
};
int launch_kv_append(const AppendParams& p, int dtype, int cache_dtype, int head_dim, void* stream);

struct AttnParams {
  PagedView c;
  PackedTokens tk;
  const unsigned char* q;
  unsigned char* out;
  float* lse;
  long long q_ts, q_hs, o_ts, o_hs;  // in elements
  int G;                             // query heads per key/value head
  const int32_t* lens;
  float scale;
  int causal;
  unsigned char* ws;
  uint32_t* status;
};
size_t attention_workspace(int head_dim);
int launch_attention(const AttnParams& p, int dtype, int cache_dtype, int head_dim, int sms, void* stream);

struct DistillParams {
  const unsigned char* z;  // student logits
  long long z_stride;      // in elements
  int rows, V, K;
  const int32_t* ids;
  const float* teacher;
  const float* weight;    // per row, or null
  const float* upstream;  // per row, upstream_stride apart, or null (backward only)
  long long upstream_stride;
  float inv_t;
  float* loss;
  float* lse;  // [rows, 2] statistics; forward: written (or null); backward: read. s < 0: about the largest logit
  unsigned char* grad;
  long long grad_stride;
  uint32_t* status;
};
constexpr int kMaxTeacher = 256;
constexpr int kMaxDistillRows = 1 << 27;  // times 8 CTAs, below 2^31
int launch_distill_loss(const DistillParams& p, int dtype, int sms, void* stream);
int launch_distill_grad(const DistillParams& p, int dtype, void* stream);
int launch_distill_loss_grad(const DistillParams& p, int dtype, int sms, void* stream);

}  // namespace dflash
