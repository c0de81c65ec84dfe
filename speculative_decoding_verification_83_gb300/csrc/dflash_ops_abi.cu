// dflash_ops_abi.cu -- the extern "C" entry points of the operators around the
// verification step (paged key/value append, attention over the paged cache,
// the drafter's distillation loss): argument checks and launches. Nothing is
// allocated here and no exception leaves a call.

#include <cuda_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include <nvtx3/nvToolsExt.h>

#include "../../include/dflash_verify.h"
#include "dflash_internal.h"
#include "dflash_ops.h"

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

// The cache's description, checked, with its strides in 16-byte units.
int bind_cache(const dflash_paged_cache* c, int dtype, PagedView* out) {
  if (!c || !c->k || !c->v || !c->page_table) return fail(DFLASH_ERR_INVALID_ARG, "null pointer in the cache");
  if (dtype != DFLASH_BF16 && dtype != DFLASH_F16)
    return fail(DFLASH_ERR_INVALID_ARG, "dtype=%d is neither bf16 nor f16", dtype);
  if (c->dtype != dtype && c->dtype != DFLASH_E4M3)
    return fail(DFLASH_ERR_INVALID_ARG, "the cache's dtype=%d is neither the tokens' dtype=%d nor e4m3", c->dtype, dtype);
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
    return fail(DFLASH_ERR_UNSUPPORTED, "head_dim=%d is not 64, 128 or 256", c->head_dim);
  if (c->batch < 1 || c->batch > kOpsMaxB)
    return fail(DFLASH_ERR_INVALID_ARG, "batch=%d outside [1, %d]", c->batch, kOpsMaxB);
  if (c->num_pages < 1 || c->page_size < 1 || c->max_pages < 1 || c->kv_heads < 1)
    return fail(DFLASH_ERR_INVALID_ARG, "num_pages=%d, page_size=%d, max_pages=%d and kv_heads=%d must be positive",
                c->num_pages, c->page_size, c->max_pages, c->kv_heads);
  if (!aligned(c->k, 16) || !aligned(c->v, 16))
    return fail(DFLASH_ERR_INVALID_ARG, "the caches must be 16-byte aligned");
  const long long es = c->dtype == DFLASH_E4M3 ? 1 : 2;
  const int64_t st[3] = {c->page_stride, c->head_stride, c->slot_stride};
  const int64_t ext[3] = {c->num_pages - 1, c->kv_heads - 1, c->page_size - 1};
  double span = 0.0;
  for (int i = 0; i < 3; ++i) {
    if (st[i] < 0 || st[i] * es % 16 != 0)
      return fail(DFLASH_ERR_INVALID_ARG, "cache stride %lld must be a multiple of 16 bytes and not negative",
                  (long long)st[i]);
    span += (double)st[i] * (double)es * (double)ext[i];
  }
  // rows are addressed in 16-byte units of 32 bits
  if (span / 16.0 >= 4294967295.0)
    return fail(DFLASH_ERR_UNSUPPORTED, "the cache spans 64 GiB or more");
  // the table's row stride may exceed its width; the width times the page
  // size bounds the positions
  if (c->table_stride < 0) return fail(DFLASH_ERR_INVALID_ARG, "table_stride must not be negative");
  out->k = static_cast<unsigned char*>(c->k);
  out->v = static_cast<unsigned char*>(c->v);
  out->table = c->page_table;
  out->table_stride = c->table_stride;
  out->page_s = (uint32_t)(st[0] * es / 16);
  out->head_s = (uint32_t)(st[1] * es / 16);
  out->slot_s = (uint32_t)(st[2] * es / 16);
  out->num_pages = c->num_pages;
  out->page_size = c->page_size;
  out->page_shift = -1;
  if ((c->page_size & (c->page_size - 1)) == 0)
    for (int i = 0; i < 31; ++i)
      if (c->page_size == (1 << i)) out->page_shift = i;
  out->max_pages = c->max_pages;
  out->kv_heads = c->kv_heads;
  out->k_scale = c->dtype == DFLASH_E4M3 ? c->k_scale : nullptr;
  out->v_scale = c->dtype == DFLASH_E4M3 ? c->v_scale : nullptr;
  return DFLASH_OK;
}

int bind_tokens(const dflash_paged_cache* c, const int32_t* q_start, int tokens, PackedTokens* out) {
  if (tokens < 0) return fail(DFLASH_ERR_INVALID_ARG, "tokens=%d must not be negative", tokens);
  if (!q_start && tokens % c->batch != 0)
    return fail(DFLASH_ERR_INVALID_ARG, "%d tokens do not divide evenly over %d requests: q_start is needed", tokens,
                c->batch);
  out->q_start = q_start;
  out->tokens = tokens;
  out->B = c->batch;
  out->q_per = tokens / c->batch;
  return DFLASH_OK;
}

// token and head strides of a [tokens, heads, head_dim] array of 16-bit values
int check_rows(const void* p, int64_t token_stride, int64_t head_stride, const char* name) {
  if (!p) return fail(DFLASH_ERR_INVALID_ARG, "null %s", name);
  if (!aligned(p, 16)) return fail(DFLASH_ERR_INVALID_ARG, "%s must be 16-byte aligned", name);
  if (token_stride % 8 || head_stride % 8 || token_stride < 0 || head_stride < 0)
    return fail(DFLASH_ERR_INVALID_ARG, "%s: strides must be multiples of 16 bytes and not negative", name);
  return DFLASH_OK;
}

int check_distill(const void* student, int64_t stride, int rows, int V, int dtype, const int32_t* ids,
                  const float* teacher, int K, float temperature) {
  if (rows != 0 && (!student || !ids || !teacher)) return fail(DFLASH_ERR_INVALID_ARG, "null pointer argument");
  if (rows < 0 || rows > kMaxDistillRows)
    return fail(DFLASH_ERR_INVALID_ARG, "rows=%d outside [0, %d]", rows, kMaxDistillRows);
  if (V < 1) return fail(DFLASH_ERR_INVALID_ARG, "V=%d must be >= 1", V);
  if (K < 1 || K > kMaxTeacher) return fail(DFLASH_ERR_INVALID_ARG, "K=%d outside [1, %d]", K, kMaxTeacher);
  if (dtype != DFLASH_BF16 && dtype != DFLASH_F32)
    return fail(DFLASH_ERR_INVALID_ARG, "dtype=%d is neither bf16 nor fp32", dtype);
  if (stride < 0) return fail(DFLASH_ERR_INVALID_ARG, "the row stride must not be negative");
  if (!(temperature > 0.0f) || std::isinf(temperature))
    return fail(DFLASH_ERR_INVALID_ARG, "temperature=%g must be positive and finite", (double)temperature);
  if (std::isinf(1.4426950408889634f * (1.0f / temperature)))  // the exponents' scale
    return fail(DFLASH_ERR_INVALID_ARG, "temperature=%g is too small: 1 / (T ln 2) must be finite", (double)temperature);
  if (!aligned(student, dtype == DFLASH_BF16 ? 2 : 4))
    return fail(DFLASH_ERR_INVALID_ARG, "student logits are not aligned to their type");
  return DFLASH_OK;
}

int sms_here(int* sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail(DFLASH_ERR_CUDA, "no CUDA device: %s", cudaGetErrorString(e));
  *sms = context_sms(dev);
  if (*sms < 1) return fail(DFLASH_ERR_CUDA, "no SMs available to the context");
  return DFLASH_OK;
}

}  // namespace

extern "C" {

int dflash_kv_append(const dflash_paged_cache* cache, const void* k, const void* v, const void* q, void* q_out,
                     int dtype, int tokens, int q_heads, const int64_t* strides, const int32_t* cached_lens,
                     const int32_t* q_start, const uint64_t* phases, int rot_dim, int interleaved, uint32_t* status,
                     void* stream) {
  NvtxRange nvtx_range("dflash_kv_append");
  AppendParams p;
  memset(&p, 0, sizeof p);
  int rc = bind_cache(cache, dtype, &p.c);
  if (rc || (rc = bind_tokens(cache, q_start, tokens, &p.tk))) return rc;
  if (!strides || !cached_lens) return fail(DFLASH_ERR_INVALID_ARG, "null pointer argument");
  if ((q == nullptr) != (q_out == nullptr))
    return fail(DFLASH_ERR_INVALID_ARG, "q and q_out are given together or not at all");
  if (q && q_heads < 1) return fail(DFLASH_ERR_INVALID_ARG, "q_heads=%d must be positive", q_heads);
  // pieces of 16 values of a token's heads: a grid's second extent times a block's
  if ((2LL * cache->kv_heads + (q ? q_heads : 0)) * (cache->head_dim / 16) > 65535LL * 256)
    return fail(DFLASH_ERR_UNSUPPORTED, "%d query and %d key/value heads of %d are more than a token may have",
                q ? q_heads : 0, cache->kv_heads, cache->head_dim);
  if (rot_dim < 0 || rot_dim > cache->head_dim || rot_dim % 16)
    return fail(DFLASH_ERR_UNSUPPORTED, "rot_dim=%d must be a multiple of 16 in [0, head_dim=%d]", rot_dim,
                cache->head_dim);
  if (rot_dim && !phases) return fail(DFLASH_ERR_INVALID_ARG, "null phases with rot_dim=%d", rot_dim);
  if (tokens == 0) return DFLASH_OK;
  if ((rc = check_rows(k, strides[0], strides[1], "k")) || (rc = check_rows(v, strides[2], strides[3], "v")) ||
      (q && ((rc = check_rows(q, strides[4], strides[5], "q")) ||
             (rc = check_rows(q_out, strides[6], strides[7], "q_out")))))
    return rc;
  p.k = static_cast<const unsigned char*>(k);
  p.v = static_cast<const unsigned char*>(v);
  p.q = static_cast<const unsigned char*>(q);
  p.q_out = static_cast<unsigned char*>(q_out);
  p.k_ts = strides[0];
  p.k_hs = strides[1];
  p.v_ts = strides[2];
  p.v_hs = strides[3];
  p.q_ts = strides[4];
  p.q_hs = strides[5];
  p.qo_ts = strides[6];
  p.qo_hs = strides[7];
  p.q_heads = q ? q_heads : 0;
  p.lens = cached_lens;
  p.phases = reinterpret_cast<const unsigned long long*>(phases);
  p.rot = rot_dim;
  p.interleaved = interleaved != 0;
  p.status = status;
  return launched(launch_kv_append(p, dtype, cache->dtype, cache->head_dim, stream), "the key/value append");
}

size_t dflash_attention_workspace_bytes(int batch, int head_dim) {
  if (batch < 1 || batch > kOpsMaxB || (head_dim != 64 && head_dim != 128 && head_dim != 256)) return 0;
  return attention_workspace(head_dim);
}

int dflash_paged_attention(const dflash_paged_cache* cache, const void* q, void* out, float* lse, int dtype,
                           int tokens, int q_heads, const int64_t* strides, const int32_t* kv_lens,
                           const int32_t* q_start, float scale, int causal, void* workspace, size_t workspace_bytes,
                           uint32_t* status, void* stream) {
  NvtxRange nvtx_range("dflash_paged_attention");
  AttnParams p;
  memset(&p, 0, sizeof p);
  int rc = bind_cache(cache, dtype, &p.c);
  if (rc || (rc = bind_tokens(cache, q_start, tokens, &p.tk))) return rc;
  if (!strides || !kv_lens) return fail(DFLASH_ERR_INVALID_ARG, "null pointer argument");
  if (q_heads < 1 || q_heads % cache->kv_heads)
    return fail(DFLASH_ERR_INVALID_ARG, "q_heads=%d must be a positive multiple of kv_heads=%d", q_heads,
                cache->kv_heads);
  if (!(scale > 0.0f) || std::isinf(scale))
    return fail(DFLASH_ERR_INVALID_ARG, "scale=%g must be positive and finite", (double)scale);
  if ((long long)tokens * q_heads > 0x7fffffffLL)
    return fail(DFLASH_ERR_UNSUPPORTED, "%d tokens of %d heads are more than 2^31 - 1 rows", tokens, q_heads);
  if (tokens == 0) return DFLASH_OK;
  if ((rc = check_rows(q, strides[0], strides[1], "q")) || (rc = check_rows(out, strides[2], strides[3], "out")))
    return rc;
  const size_t need = attention_workspace(cache->head_dim);
  if (!workspace || workspace_bytes < need)
    return fail(DFLASH_ERR_INVALID_ARG, "workspace of %zu bytes is smaller than the %zu needed",
                workspace ? workspace_bytes : (size_t)0, need);
  if (!aligned(workspace, 256)) return fail(DFLASH_ERR_INVALID_ARG, "the workspace must be 256-byte aligned");
  p.q = static_cast<const unsigned char*>(q);
  p.out = static_cast<unsigned char*>(out);
  p.lse = lse;
  p.q_ts = strides[0];
  p.q_hs = strides[1];
  p.o_ts = strides[2];
  p.o_hs = strides[3];
  p.G = q_heads / cache->kv_heads;
  p.lens = kv_lens;
  p.scale = scale;
  p.causal = causal != 0;
  p.ws = static_cast<unsigned char*>(workspace);
  p.status = status;
  int sms = 0;
  if ((rc = sms_here(&sms))) return rc;
  return launched(launch_attention(p, dtype, cache->dtype, cache->head_dim, sms, stream), "the paged attention");
}

int dflash_distill_loss(const void* student, int64_t row_stride, int rows, int V, int dtype,
                        const int32_t* teacher_ids, const float* teacher_logits, int K, float temperature,
                        const float* row_weight, float* loss, float* lse, uint32_t* status, void* stream) {
  NvtxRange nvtx_range("dflash_distill_loss");
  int rc = check_distill(student, row_stride, rows, V, dtype, teacher_ids, teacher_logits, K, temperature);
  if (rc) return rc;
  if (rows == 0) return DFLASH_OK;
  if (!loss) return fail(DFLASH_ERR_INVALID_ARG, "null loss");
  DistillParams p;
  memset(&p, 0, sizeof p);
  p.z = static_cast<const unsigned char*>(student);
  p.z_stride = row_stride;
  p.rows = rows;
  p.V = V;
  p.K = K;
  p.ids = teacher_ids;
  p.teacher = teacher_logits;
  p.weight = row_weight;
  p.inv_t = 1.0f / temperature;
  p.loss = loss;
  p.lse = lse;
  p.status = status;
  int sms = 0;
  if ((rc = sms_here(&sms))) return rc;
  return launched(launch_distill_loss(p, dtype, sms, stream), "the distillation loss");
}

int dflash_distill_grad(const void* student, int64_t row_stride, int rows, int V, int dtype,
                        const int32_t* teacher_ids, const float* teacher_logits, int K, float temperature,
                        const float* row_weight, const float* lse, const float* upstream,
                        int64_t upstream_stride, void* grad, int64_t grad_stride, void* stream) {
  NvtxRange nvtx_range("dflash_distill_grad");
  int rc = check_distill(student, row_stride, rows, V, dtype, teacher_ids, teacher_logits, K, temperature);
  if (rc) return rc;
  if (rows == 0) return DFLASH_OK;
  if (!lse || !grad) return fail(DFLASH_ERR_INVALID_ARG, "null pointer argument");
  if (upstream_stride < 0) return fail(DFLASH_ERR_INVALID_ARG, "upstream_stride must not be negative");
  if (!aligned(grad, dtype == DFLASH_BF16 ? 2 : 4) || grad_stride < V)
    return fail(DFLASH_ERR_INVALID_ARG, "the gradient's rows must be aligned to their type and at least V apart");
  DistillParams p;
  memset(&p, 0, sizeof p);
  p.z = static_cast<const unsigned char*>(student);
  p.z_stride = row_stride;
  p.rows = rows;
  p.V = V;
  p.K = K;
  p.ids = teacher_ids;
  p.teacher = teacher_logits;
  p.weight = row_weight;
  p.upstream = upstream;
  p.upstream_stride = upstream_stride;
  p.inv_t = 1.0f / temperature;
  p.lse = const_cast<float*>(lse);
  p.grad = static_cast<unsigned char*>(grad);
  p.grad_stride = grad_stride;
  return launched(launch_distill_grad(p, dtype, stream), "the distillation gradient");
}

int dflash_distill_loss_grad(const void* student, int64_t row_stride, int rows, int V, int dtype,
                             const int32_t* teacher_ids, const float* teacher_logits, int K, float temperature,
                             const float* row_weight, float* loss, void* grad, int64_t grad_stride, uint32_t* status,
                             void* stream) {
  NvtxRange nvtx_range("dflash_distill_loss_grad");
  int rc = check_distill(student, row_stride, rows, V, dtype, teacher_ids, teacher_logits, K, temperature);
  if (rc) return rc;
  if (rows == 0) return DFLASH_OK;
  if (!loss || !grad) return fail(DFLASH_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned(grad, dtype == DFLASH_BF16 ? 2 : 4) || grad_stride < V)
    return fail(DFLASH_ERR_INVALID_ARG, "the gradient's rows must be aligned to their type and at least V apart");
  DistillParams p;
  memset(&p, 0, sizeof p);
  p.z = static_cast<const unsigned char*>(student);
  p.z_stride = row_stride;
  p.rows = rows;
  p.V = V;
  p.K = K;
  p.ids = teacher_ids;
  p.teacher = teacher_logits;
  p.weight = row_weight;
  p.inv_t = 1.0f / temperature;
  p.loss = loss;
  p.grad = static_cast<unsigned char*>(grad);
  p.grad_stride = grad_stride;
  p.status = status;
  int sms = 0;
  if ((rc = sms_here(&sms))) return rc;
  return launched(launch_distill_loss_grad(p, dtype, sms, stream), "the distillation loss and gradient");
}

}  // extern "C"
