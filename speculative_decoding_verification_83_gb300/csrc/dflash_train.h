// dflash_train.h -- parameters and launchers of the operators that train a
// drafter and serve its prompts: the norms of queries and keys with rotation
// (dflash_norm.cu), attention over packed sequences (dflash_packed*.cu) and the
// cross entropy through the vocabulary projection (dflash_entropy.cu). The entry
// points and their argument checks are in dflash_train_abi.cu.
#pragma once

#include <vector_types.h>

#include <cstddef>
#include <cstdint>

namespace dflash {

// A [tokens, heads, head_dim] array of 16-bit values: strides in elements.
struct HeadRows {
  unsigned char* p;
  long long ts, hs;
};

struct NormParams {
  HeadRows q, k;                 // the values; p null: none
  HeadRows qo, ko;               // forward: the results; backward: the values' gradients
  HeadRows dq, dk;               // backward: the results' gradients
  const void *q_weight, *k_weight;  // [head_dim], or null: 1
  void *gq_weight, *gk_weight;      // backward: their gradients, or null
  int weight_f32;                // else in the tokens' type
  int tokens, q_heads, k_heads;  // 0 heads: none
  float eps;
  const int32_t* positions;
  const unsigned long long* phases;
  int rot, interleaved;
  float* partial;                // backward: [kNormBlocks][2][head_dim]
};
constexpr int kNormBlocks = 304;  // of the backward pass, at most: two for each of 152 SMs
inline size_t norm_workspace(int head_dim) { return (size_t)kNormBlocks * 2 * head_dim * sizeof(float); }
int launch_norm(const NormParams& p, int dtype, int head_dim, void* stream);
int launch_norm_grad(const NormParams& p, int dtype, int head_dim, void* stream);

// Cross entropy of h W^T (bf16): h [rows, K], W [V, K].
struct EntropyParams {
  const unsigned char *h, *w;
  long long h_stride, w_stride;  // elements between rows
  int rows, V, K;
  const int32_t* labels;
  const float* weight;  // per row, or null
  float* loss;
  float2* stats;        // per row: the largest logit m and the sum of e^(z - m)
  const float* upstream;
  long long upstream_stride;
  unsigned char *dh, *dw;  // contiguous, or null
  unsigned char* ws;
  uint32_t* status;
};
constexpr int kMaxEntropyRows = 1 << 20, kMaxEntropyV = 1 << 24, kMaxEntropyK = 1 << 16;  // tiles are counted in 32 bits
size_t entropy_workspace(int rows, int V, int K, bool backward);
int launch_entropy(const EntropyParams& p, int sms, void* stream);
int launch_entropy_grad(const EntropyParams& p, int sms, void* stream);


// Attention over packed sequences: sequence b's queries are rows q_start[b] ..
// q_start[b + 1] - 1, its keys and values rows kv_start[b] .. kv_start[b + 1] - 1.
struct PackedParams {
  HeadRows q, k, v, o;
  int8_t* low;               // [q_tokens, q_heads, head_dim] or null: what the outputs' rounding left, see out_low
  float* lse;                // [q_tokens, q_heads]
  HeadRows d_o, dq, dk, dv;  // backward
  // backward: by head, stat_pitch rows of -lse log2 e (-inf for a row that sees nothing), then of -delta, delta = sum of d_o o
  float* row_stats;
  int stat_pitch;
  const int32_t *q_start, *kv_start;
  int B, q_tokens, kv_tokens, q_heads, kv_heads, G;
  float scale;
  int causal;
  int fill;  // rows of no sequence are set to 0
  unsigned char* ws;
  uint32_t* status;
};
constexpr int kMaxPackedTokens = 1 << 24, kMaxPackedHeads = 1024;  // units of work are counted in 32 bits
size_t packed_workspace(int B, int q_tokens, int kv_tokens, int q_heads, int kv_heads, int head_dim, bool backward);
int launch_packed(const PackedParams& p, int dtype, int head_dim, int sms, void* stream);
int launch_packed_grad(const PackedParams& p, int head_dim, int sms, void* stream);  // bf16

}  // namespace dflash
