// dflash_train_abi.cu -- the extern "C" entry points of the operators that train
// a drafter and serve its prompts (norms with rotation, attention over packed
// sequences, cross entropy through the vocabulary projection): argument checks
// and launches. Nothing is allocated here and no exception leaves a call.

#include <cuda_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include <nvtx3/nvToolsExt.h>

#include "../../include/dflash_verify.h"
#include "dflash_internal.h"
#include "dflash_ops.h"
#include "dflash_train.h"

using namespace dflash;

namespace {

int fail(int code, const char* fmt, ...) {
  char msg[400];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof msg, fmt, ap);
  va_end(ap);
  set_last_error(msg);
  return code;
}
int launched(int e, const char* what) {
  if (e == 0) return DFLASH_OK;
  return fail(DFLASH_ERR_CUDA, "launching %s: %s", what, cudaGetErrorString((cudaError_t)e));
}

struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

bool aligned(const void* p, size_t a) { return (uintptr_t)p % a == 0; }

int sms_here(int* sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail(DFLASH_ERR_CUDA, "no CUDA device: %s", cudaGetErrorString(e));
  *sms = context_sms(dev);
  if (*sms < 1) return fail(DFLASH_ERR_CUDA, "no SMs available to the context");
  return DFLASH_OK;
}

// A [tokens, heads, head_dim] array of 16-bit values and its strides; an extent of
// one is never stepped over, whatever its stride says.
int bind_rows(const void* p, const int64_t* strides, int tokens, int heads, int dim, const char* name, HeadRows* out) {
  if (!p) return fail(DFLASH_ERR_INVALID_ARG, "null %s", name);
  if (!aligned(p, 16)) return fail(DFLASH_ERR_INVALID_ARG, "%s must be 16-byte aligned", name);
  const int64_t ts = tokens > 1 ? strides[0] : (int64_t)heads * dim, hs = heads > 1 ? strides[1] : dim;
  if (ts % 8 || hs % 8 || ts < dim || hs < dim || ts >= 1ll << 36 || hs >= 1ll << 36)
    return fail(DFLASH_ERR_INVALID_ARG,
                "%s: strides %lld and %lld must be multiples of 16 bytes, at least head_dim=%d and below 2^36 values", name,
                (long long)ts, (long long)hs, dim);
  out->p = static_cast<unsigned char*>(const_cast<void*>(p));
  out->ts = ts;
  out->hs = hs;
  return DFLASH_OK;
}

int check_workspace(const void* ws, size_t have, size_t need) {
  if (!ws || have < need)
    return fail(DFLASH_ERR_INVALID_ARG, "workspace of %zu bytes is smaller than the %zu needed", ws ? have : (size_t)0, need);
  if (!aligned(ws, 256)) return fail(DFLASH_ERR_INVALID_ARG, "the workspace must be 256-byte aligned");
  return DFLASH_OK;
}

// ---- norms with rotation
int bind_norm(int dtype, int tokens, int q_heads, int k_heads, int head_dim, const void* q_weight, const void* k_weight,
              int weight_dtype, float eps, const int32_t* positions, const uint64_t* phases, int rot_dim, int interleaved,
              NormParams* p) {
  memset(p, 0, sizeof *p);
  if (dtype != DFLASH_BF16 && dtype != DFLASH_F16)
    return fail(DFLASH_ERR_INVALID_ARG, "dtype=%d is neither bf16 nor f16", dtype);
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return fail(DFLASH_ERR_UNSUPPORTED, "head_dim=%d is not 64, 128 or 256", head_dim);
  if (tokens < 0) return fail(DFLASH_ERR_INVALID_ARG, "tokens=%d must not be negative", tokens);
  if (q_heads < 0 || k_heads < 0 || q_heads + (long long)k_heads < 1)
    return fail(DFLASH_ERR_INVALID_ARG, "q_heads=%d and k_heads=%d must not be negative, and not both 0", q_heads, k_heads);
  if (tokens > 1 << 30) return fail(DFLASH_ERR_UNSUPPORTED, "tokens=%d is more than 2^30", tokens);
  // a block's rows (4 tokens) are counted in 32 bits
  if (q_heads + (long long)k_heads > 1 << 20)
    return fail(DFLASH_ERR_UNSUPPORTED, "%lld heads are more than a token may have", q_heads + (long long)k_heads);
  if (weight_dtype != dtype && weight_dtype != DFLASH_F32)
    return fail(DFLASH_ERR_INVALID_ARG, "weight_dtype=%d is neither the tokens' dtype=%d nor fp32", weight_dtype, dtype);
  if (!aligned(q_weight, 16) || !aligned(k_weight, 16))
    return fail(DFLASH_ERR_INVALID_ARG, "the norms' weights must be 16-byte aligned");
  if (!(eps >= 0.0f) || std::isinf(eps))
    return fail(DFLASH_ERR_INVALID_ARG, "eps=%g must be finite and not negative", (double)eps);
  if (rot_dim < 0 || rot_dim > head_dim || rot_dim % 16)
    return fail(DFLASH_ERR_UNSUPPORTED, "rot_dim=%d must be a multiple of 16 in [0, head_dim=%d]", rot_dim, head_dim);
  if (rot_dim && tokens && (!phases || !positions))
    return fail(DFLASH_ERR_INVALID_ARG, "null phases or positions with rot_dim=%d", rot_dim);
  p->q_weight = q_weight;
  p->k_weight = k_weight;
  p->weight_f32 = weight_dtype == DFLASH_F32;
  p->tokens = tokens;
  p->q_heads = q_heads;
  p->k_heads = k_heads;
  p->eps = eps;
  p->positions = positions;
  p->phases = reinterpret_cast<const unsigned long long*>(phases);
  p->rot = rot_dim;
  p->interleaved = interleaved != 0;
  return DFLASH_OK;
}

// ---- packed sequences
int bind_packed(const dflash_packed_batch* c, PackedParams* p) {
  memset(p, 0, sizeof *p);
  if (!c || !c->q_start || !c->kv_start) return fail(DFLASH_ERR_INVALID_ARG, "null pointer in the batch");
  if (c->dtype != DFLASH_BF16 && c->dtype != DFLASH_F16)
    return fail(DFLASH_ERR_INVALID_ARG, "dtype=%d is neither bf16 nor f16", c->dtype);
  if (c->head_dim != 64 && c->head_dim != 128)
    return fail(DFLASH_ERR_UNSUPPORTED, "head_dim=%d is not 64 or 128", c->head_dim);
  if (c->batch < 1 || c->batch > kOpsMaxB)
    return fail(DFLASH_ERR_INVALID_ARG, "batch=%d outside [1, %d]", c->batch, kOpsMaxB);
  if (c->q_tokens < 0 || c->kv_tokens < 0 || c->q_tokens > kMaxPackedTokens || c->kv_tokens > kMaxPackedTokens)
    return fail(DFLASH_ERR_INVALID_ARG, "q_tokens=%d and kv_tokens=%d outside [0, %d]", c->q_tokens, c->kv_tokens,
                kMaxPackedTokens);
  if (c->kv_heads < 1 || c->q_heads < 1 || c->q_heads % c->kv_heads)
    return fail(DFLASH_ERR_INVALID_ARG, "q_heads=%d must be a positive multiple of kv_heads=%d", c->q_heads, c->kv_heads);
  if (c->q_heads > kMaxPackedHeads)
    return fail(DFLASH_ERR_UNSUPPORTED, "q_heads=%d is more than %d", c->q_heads, kMaxPackedHeads);
  if (!(c->scale > 0.0f) || std::isinf(c->scale))
    return fail(DFLASH_ERR_INVALID_ARG, "scale=%g must be positive and finite", (double)c->scale);
  p->q_start = c->q_start;
  p->kv_start = c->kv_start;
  p->B = c->batch;
  p->q_tokens = c->q_tokens;
  p->kv_tokens = c->kv_tokens;
  p->q_heads = c->q_heads;
  p->kv_heads = c->kv_heads;
  p->G = c->q_heads / c->kv_heads;
  p->scale = c->scale;
  p->causal = c->causal != 0;
  return DFLASH_OK;
}
size_t packed_bytes(const dflash_packed_batch* c, bool backward) {
  return packed_workspace(c->batch, c->q_tokens, c->kv_tokens, c->q_heads, c->kv_heads, c->head_dim, backward);
}

// ---- cross entropy
int check_entropy(const void* h, int64_t h_stride, const void* w, int64_t w_stride, int rows, int V, int K,
                  const int32_t* labels) {
  if (rows < 0 || rows > kMaxEntropyRows)
    return fail(DFLASH_ERR_INVALID_ARG, "rows=%d outside [0, %d]", rows, kMaxEntropyRows);
  if (V < 1 || V > kMaxEntropyV) return fail(DFLASH_ERR_INVALID_ARG, "V=%d outside [1, %d]", V, kMaxEntropyV);
  if (K < 8 || K % 8 || K > kMaxEntropyK)
    return fail(DFLASH_ERR_UNSUPPORTED, "K=%d must be a multiple of 8 in [8, %d]", K, kMaxEntropyK);
  if (!w || (rows && (!h || !labels))) return fail(DFLASH_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned(h, 16) || !aligned(w, 16))
    return fail(DFLASH_ERR_INVALID_ARG, "the hidden states and the projection must be 16-byte aligned");
  if ((rows > 1 && (h_stride < K || h_stride % 8 || h_stride >= 1ll << 36)) ||
      (V > 1 && (w_stride < K || w_stride % 8 || w_stride >= 1ll << 36)))
    return fail(DFLASH_ERR_INVALID_ARG, "row strides must be multiples of 16 bytes, at least K=%d and below 2^36 values", K);
  return DFLASH_OK;
}

}  // namespace

extern "C" {

int dflash_norm_rotate(const void* q, const void* k, void* q_out, void* k_out, int dtype, int tokens, int q_heads,
                       int k_heads, int head_dim, const int64_t* strides, const void* q_weight, const void* k_weight,
                       int weight_dtype, float eps, const int32_t* positions, const uint64_t* phases, int rot_dim,
                       int interleaved, void* stream) {
  NvtxRange nvtx_range("dflash_norm_rotate");
  NormParams p;
  int rc = bind_norm(dtype, tokens, q_heads, k_heads, head_dim, q_weight, k_weight, weight_dtype, eps, positions, phases,
                     rot_dim, interleaved, &p);
  if (rc) return rc;
  if (tokens == 0) return DFLASH_OK;
  if (!strides) return fail(DFLASH_ERR_INVALID_ARG, "null strides");
  if (q_heads && ((rc = bind_rows(q, strides, tokens, q_heads, head_dim, "q", &p.q)) ||
                  (rc = bind_rows(q_out, strides + 4, tokens, q_heads, head_dim, "q_out", &p.qo))))
    return rc;
  if (k_heads && ((rc = bind_rows(k, strides + 2, tokens, k_heads, head_dim, "k", &p.k)) ||
                  (rc = bind_rows(k_out, strides + 6, tokens, k_heads, head_dim, "k_out", &p.ko))))
    return rc;
  return launched(launch_norm(p, dtype, head_dim, stream), "the norm with rotation");
}

size_t dflash_norm_workspace_bytes(int head_dim) {
  return head_dim == 64 || head_dim == 128 || head_dim == 256 ? norm_workspace(head_dim) : 0;
}

int dflash_norm_rotate_grad(const void* q, const void* k, const void* dq_out, const void* dk_out, void* dq, void* dk,
                            int dtype, int tokens, int q_heads, int k_heads, int head_dim, const int64_t* strides,
                            const void* q_weight, const void* k_weight, void* dq_weight, void* dk_weight, int weight_dtype,
                            float eps, const int32_t* positions, const uint64_t* phases, int rot_dim, int interleaved,
                            void* workspace, size_t workspace_bytes, void* stream) {
  NvtxRange nvtx_range("dflash_norm_rotate_grad");
  NormParams p;
  int rc = bind_norm(dtype, tokens, q_heads, k_heads, head_dim, q_weight, k_weight, weight_dtype, eps, positions, phases,
                     rot_dim, interleaved, &p);
  if (rc) return rc;
  if (!strides && tokens) return fail(DFLASH_ERR_INVALID_ARG, "null strides");
  if ((rc = check_workspace(workspace, workspace_bytes, norm_workspace(head_dim)))) return rc;
  if (tokens && q_heads &&
      ((rc = bind_rows(q, strides, tokens, q_heads, head_dim, "q", &p.q)) ||
       (rc = bind_rows(dq_out, strides + 4, tokens, q_heads, head_dim, "dq_out", &p.dq)) ||
       (rc = bind_rows(dq, strides + 8, tokens, q_heads, head_dim, "dq", &p.qo))))
    return rc;
  if (tokens && k_heads &&
      ((rc = bind_rows(k, strides + 2, tokens, k_heads, head_dim, "k", &p.k)) ||
       (rc = bind_rows(dk_out, strides + 6, tokens, k_heads, head_dim, "dk_out", &p.dk)) ||
       (rc = bind_rows(dk, strides + 10, tokens, k_heads, head_dim, "dk", &p.ko))))
    return rc;
  if (tokens == 0) p.rot = 0;  // (the weights' gradients are 0, without positions and phases)
  p.gq_weight = dq_weight;
  p.gk_weight = dk_weight;
  p.partial = static_cast<float*>(workspace);
  return launched(launch_norm_grad(p, dtype, head_dim, stream), "the gradient of the norm with rotation");
}

size_t dflash_packed_workspace_bytes(const dflash_packed_batch* batch, int backward) {
  PackedParams p;
  return bind_packed(batch, &p) ? 0 : packed_bytes(batch, backward != 0);
}

int dflash_packed_attention(const dflash_packed_batch* batch, const void* q, const void* k, const void* v, void* out,
                            const int64_t* strides, float* lse, int8_t* out_low, int fill, void* workspace,
                            size_t workspace_bytes, uint32_t* status, void* stream) {
  NvtxRange nvtx_range("dflash_packed_attention");
  PackedParams p;
  int rc = bind_packed(batch, &p);
  if (rc) return rc;
  if (p.q_tokens == 0) return DFLASH_OK;
  if (!strides) return fail(DFLASH_ERR_INVALID_ARG, "null strides");
  const int d = batch->head_dim;
  if ((rc = bind_rows(q, strides, p.q_tokens, p.q_heads, d, "q", &p.q)) ||
      (rc = bind_rows(out, strides + 6, p.q_tokens, p.q_heads, d, "out", &p.o)))
    return rc;
  if (p.kv_tokens && ((rc = bind_rows(k, strides + 2, p.kv_tokens, p.kv_heads, d, "k", &p.k)) ||
                      (rc = bind_rows(v, strides + 4, p.kv_tokens, p.kv_heads, d, "v", &p.v))))
    return rc;
  if (out_low && (batch->dtype != DFLASH_BF16 || !aligned(out_low, 16)))
    return fail(DFLASH_ERR_INVALID_ARG, "out_low is for bf16 and must be 16-byte aligned");
  if ((rc = check_workspace(workspace, workspace_bytes, packed_bytes(batch, false)))) return rc;
  p.lse = lse;
  p.low = out_low;
  p.fill = fill != 0;
  p.ws = static_cast<unsigned char*>(workspace);
  p.status = status;
  int sms = 0;
  if ((rc = sms_here(&sms))) return rc;
  return launched(launch_packed(p, batch->dtype, d, sms, stream), "the packed attention");
}

int dflash_packed_attention_grad(const dflash_packed_batch* batch, const void* q, const void* k, const void* v,
                                 const void* out, const float* lse, const int8_t* out_low, const void* dout, void* dq,
                                 void* dk, void* dv, const int64_t* strides, int fill, void* workspace,
                                 size_t workspace_bytes, uint32_t* status, void* stream) {
  NvtxRange nvtx_range("dflash_packed_attention_grad");
  PackedParams p;
  int rc = bind_packed(batch, &p);
  if (rc) return rc;
  if (batch->dtype != DFLASH_BF16) return fail(DFLASH_ERR_UNSUPPORTED, "the packed attention's gradient is bf16 only");
  if (p.q_tokens == 0 && p.kv_tokens == 0) return DFLASH_OK;
  if (!strides) return fail(DFLASH_ERR_INVALID_ARG, "null strides");
  const int d = batch->head_dim;
  if (p.q_tokens && ((rc = bind_rows(q, strides, p.q_tokens, p.q_heads, d, "q", &p.q)) ||
                     (rc = bind_rows(out, strides + 6, p.q_tokens, p.q_heads, d, "out", &p.o)) ||
                     (rc = bind_rows(dout, strides + 8, p.q_tokens, p.q_heads, d, "dout", &p.d_o)) ||
                     (rc = bind_rows(dq, strides + 10, p.q_tokens, p.q_heads, d, "dq", &p.dq))))
    return rc;
  if (p.kv_tokens && ((rc = bind_rows(k, strides + 2, p.kv_tokens, p.kv_heads, d, "k", &p.k)) ||
                      (rc = bind_rows(v, strides + 4, p.kv_tokens, p.kv_heads, d, "v", &p.v)) ||
                      (rc = bind_rows(dk, strides + 12, p.kv_tokens, p.kv_heads, d, "dk", &p.dk)) ||
                      (rc = bind_rows(dv, strides + 14, p.kv_tokens, p.kv_heads, d, "dv", &p.dv))))
    return rc;
  if (p.q_tokens && !lse) return fail(DFLASH_ERR_INVALID_ARG, "null lse");
  if ((rc = check_workspace(workspace, workspace_bytes, packed_bytes(batch, true)))) return rc;
  if (!aligned(out_low, 16)) return fail(DFLASH_ERR_INVALID_ARG, "out_low must be 16-byte aligned");
  p.lse = const_cast<float*>(lse);
  p.low = const_cast<int8_t*>(out_low);
  p.fill = fill != 0;
  p.ws = static_cast<unsigned char*>(workspace);
  p.status = status;
  int sms = 0;
  if ((rc = sms_here(&sms))) return rc;
  return launched(launch_packed_grad(p, d, sms, stream), "the packed attention's gradient");
}

size_t dflash_linear_entropy_workspace_bytes(int rows, int V, int K, int backward) {
  if (rows < 1 || rows > kMaxEntropyRows || V < 1 || V > kMaxEntropyV || K < 8 || K % 8 || K > kMaxEntropyK) return 0;
  return entropy_workspace(rows, V, K, backward != 0);
}

int dflash_linear_entropy(const void* h, int64_t h_stride, const void* w, int64_t w_stride, int rows, int V, int K,
                          const int32_t* labels, const float* row_weight, float* loss, float* row_stats, void* workspace,
                          size_t workspace_bytes, uint32_t* status, void* stream) {
  NvtxRange nvtx_range("dflash_linear_entropy");
  int rc = check_entropy(h, h_stride, w, w_stride, rows, V, K, labels);
  if (rc) return rc;
  if (rows == 0) return DFLASH_OK;
  if (!loss) return fail(DFLASH_ERR_INVALID_ARG, "null loss");
  if (!aligned(row_stats, 8)) return fail(DFLASH_ERR_INVALID_ARG, "row_stats must be 8-byte aligned");
  if ((rc = check_workspace(workspace, workspace_bytes, entropy_workspace(rows, V, K, false)))) return rc;
  EntropyParams p;
  memset(&p, 0, sizeof p);
  p.h = static_cast<const unsigned char*>(h);
  p.w = static_cast<const unsigned char*>(w);
  p.h_stride = rows > 1 ? h_stride : K;
  p.w_stride = V > 1 ? w_stride : K;
  p.rows = rows;
  p.V = V;
  p.K = K;
  p.labels = labels;
  p.weight = row_weight;
  p.loss = loss;
  p.stats = reinterpret_cast<float2*>(row_stats);
  p.ws = static_cast<unsigned char*>(workspace);
  p.status = status;
  int sms = 0;
  if ((rc = sms_here(&sms))) return rc;
  return launched(launch_entropy(p, sms, stream), "the cross entropy");
}

int dflash_linear_entropy_grad(const void* h, int64_t h_stride, const void* w, int64_t w_stride, int rows, int V, int K,
                               const int32_t* labels, const float* row_weight, const float* row_stats,
                               const float* upstream, int64_t upstream_stride, void* dh, void* dw, void* workspace,
                               size_t workspace_bytes, uint32_t* status, void* stream) {
  NvtxRange nvtx_range("dflash_linear_entropy_grad");
  int rc = check_entropy(h, h_stride, w, w_stride, rows, V, K, labels);
  if (rc) return rc;
  if (rows == 0) return fail(DFLASH_ERR_INVALID_ARG, "no rows: the gradient of the projection is 0");
  if (!row_stats || !aligned(row_stats, 8)) return fail(DFLASH_ERR_INVALID_ARG, "row_stats is null or not 8-byte aligned");
  if (!aligned(dh, 16) || !aligned(dw, 16)) return fail(DFLASH_ERR_INVALID_ARG, "the gradients must be 16-byte aligned");
  if (upstream_stride < 0) return fail(DFLASH_ERR_INVALID_ARG, "upstream_stride must not be negative");
  if (!dh && !dw) return DFLASH_OK;
  if ((rc = check_workspace(workspace, workspace_bytes, entropy_workspace(rows, V, K, true)))) return rc;
  EntropyParams p;
  memset(&p, 0, sizeof p);
  p.h = static_cast<const unsigned char*>(h);
  p.w = static_cast<const unsigned char*>(w);
  p.h_stride = rows > 1 ? h_stride : K;
  p.w_stride = V > 1 ? w_stride : K;
  p.rows = rows;
  p.V = V;
  p.K = K;
  p.labels = labels;
  p.weight = row_weight;
  p.stats = reinterpret_cast<float2*>(const_cast<float*>(row_stats));
  p.upstream = upstream;
  p.upstream_stride = upstream_stride;
  p.dh = static_cast<unsigned char*>(dh);
  p.dw = static_cast<unsigned char*>(dw);
  p.ws = static_cast<unsigned char*>(workspace);
  p.status = status;
  int sms = 0;
  if ((rc = sms_here(&sms))) return rc;
  return launched(launch_entropy_grad(p, sms, stream), "the cross entropy's gradients");
}

}  // extern "C"
