// C ABI of a decoder layer's attention (declared in include/w4a16.h): norms and rotation of the heads, the paged cache in
// 8 bits, attention over it and over packed prompts. As in abi.cu, every check runs before anything is enqueued.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>

#include "internal.h"
#include "w4a16.h"

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int64_t kMaxDim = 0x7FFFFFFF;

bool type16(int32_t dtype) { return dtype == W4_DTYPE_F16 || dtype == W4_DTYPE_BF16; }

int num_sms_current_device() {
  static int cache[64] = {0};
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  std::lock_guard<std::mutex> lk(mu);
  if (dev < 64 && cache[dev] > 0) return cache[dev];
  int sms = 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (dev < 64) cache[dev] = sms;
  return sms;
}

int status_of(cudaError_t e) { return e == cudaSuccess ? W4_OK : W4_ERR_CUDA; }

// Rows of `heads` heads, ld values apart, that start on 16-byte boundaries.
int check_rows(int64_t ld, int64_t heads, int64_t head_dim) {
  if (ld < heads * head_dim) return W4_ERR_INVALID_ARG;
  return ld % 8 != 0 || ld > kMaxDim ? W4_ERR_UNSUPPORTED_SHAPE : W4_OK;
}

int check_cache(int64_t pages, int32_t batch, int32_t max_pages, int32_t heads, int32_t head_dim, int32_t page) {
  if (pages < 1 || batch < 0 || max_pages < 1 || heads < 1 || head_dim < 1 || page < 1) return W4_ERR_INVALID_ARG;
  if (head_dim % 16 != 0 || head_dim > w4::kKvMaxDim || page % 16 != 0 || page > w4::kKvMaxPage || pages > kMaxDim ||
      heads > 32767 || static_cast<int64_t>(max_pages) * page > kMaxDim - 1024)
    return W4_ERR_UNSUPPORTED_SHAPE;
  return W4_OK;
}

int check_kv_attention_sizes(int32_t batch, int32_t n, int32_t q_heads, int32_t k_heads, int32_t head_dim) {
  if (batch < 0 || n < 1 || q_heads < 1 || k_heads < 1 || q_heads % k_heads != 0 || head_dim < 1) return W4_ERR_INVALID_ARG;
  if (head_dim % 16 != 0 || head_dim > w4::kKvMaxDim || n > w4::kKvMaxQueries || q_heads > 65535) return W4_ERR_UNSUPPORTED_SHAPE;
  // items: 16 query rows of a sequence and key head each
  const int64_t tiles = w4::cdiv(static_cast<int64_t>(n) * (q_heads / k_heads), 16) * k_heads;
  return batch * tiles > (int64_t{1} << 24) ? W4_ERR_UNSUPPORTED_SHAPE : W4_OK;
}

}  // namespace

extern "C" {

int w4_qk_norm_rope(const w4_rope_args *a, void *stream) {
  if (!a || a->T < 0 || a->q_heads < 1 || a->k_heads < 0 || a->head_dim < 1 || a->rot < 0 || a->rot > a->head_dim)
    return W4_ERR_INVALID_ARG;
  if (!type16(a->dtype) || (a->interleaved != 0 && a->interleaved != 1) || !(a->eps >= 0.0f) || std::isinf(a->eps))
    return W4_ERR_INVALID_ARG;
  if (a->head_dim % 8 != 0 || a->head_dim > 256 || a->rot % 16 != 0 || a->T > kMaxDim || a->q_heads > 65535 || a->k_heads > 65535)
    return W4_ERR_UNSUPPORTED_SHAPE;
  const int32_t sections[4] = {a->section0, a->section1, a->section2, a->section3};
  int end = 0;
  w4::RopeArgs r;
  for (int i = 0; i < 4; ++i) {
    if (sections[i] < 0 || sections[i] > a->rot / 2 || (i >= a->axes && sections[i] != 0)) return W4_ERR_INVALID_ARG;
    end += sections[i];
    r.section_end[i] = end;
  }
  if (a->axes < (a->rot > 0 ? 1 : 0) || a->axes > (a->rot > 0 ? 4 : 0) || end != a->rot / 2) return W4_ERR_INVALID_ARG;
  if (a->rot == 0 && !a->q_weight_dev && !a->k_weight_dev) return W4_ERR_INVALID_ARG;
  int rc = check_rows(a->ldq, a->q_heads, a->head_dim);
  if (rc == W4_OK) rc = check_rows(a->ldqo, a->q_heads, a->head_dim);
  if (rc == W4_OK && a->k_heads) rc = check_rows(a->ldk, a->k_heads, a->head_dim);
  if (rc == W4_OK && a->k_heads) rc = check_rows(a->ldko, a->k_heads, a->head_dim);
  if (rc != W4_OK) return rc;
  // in place means the same rows
  if ((a->q_dev == a->q_out_dev && a->q_dev && a->ldq != a->ldqo) ||
      (a->k_heads && a->k_dev == a->k_out_dev && a->k_dev && a->ldk != a->ldko))
    return W4_ERR_INVALID_ARG;
  if (a->T == 0) return W4_OK;
  if (!a->q_dev || !a->q_out_dev || (a->k_heads && (!a->k_dev || !a->k_out_dev)) ||
      (a->rot && (!a->positions_dev || !a->freqs_dev)))
    return W4_ERR_INVALID_ARG;
  if (!aligned(a->q_dev, 16) || !aligned(a->q_out_dev, 16) || (a->k_heads && (!aligned(a->k_dev, 16) || !aligned(a->k_out_dev, 16))) ||
      !aligned(a->positions_dev, 4) || !aligned(a->freqs_dev, 4) || !aligned(a->q_weight_dev, 16) || !aligned(a->k_weight_dev, 16))
    return W4_ERR_MISALIGNED;
  r.q = a->q_dev;
  r.k = a->k_dev;
  r.q_out = a->q_out_dev;
  r.k_out = a->k_out_dev;
  r.positions = a->positions_dev;
  r.freqs = a->freqs_dev;
  r.q_weight = a->q_weight_dev;
  r.k_weight = a->k_weight_dev;
  r.T = a->T;
  r.ldq = a->ldq;
  r.ldk = a->ldk;
  r.ldqo = a->ldqo;
  r.ldko = a->ldko;
  r.q_heads = a->q_heads;
  r.k_heads = a->k_heads;
  r.head_dim = a->head_dim;
  r.rot = a->rot;
  r.interleaved = a->interleaved != 0;
  r.dtype = a->dtype;
  r.eps = a->eps;
  return status_of(w4::launch_rope(r, num_sms_current_device(), static_cast<cudaStream_t>(stream)));
}

int w4_kv_append(const w4_kv_append_args *a, void *stream) {
  if (!a || a->T < 0 || !type16(a->dtype)) return W4_ERR_INVALID_ARG;
  int rc = check_cache(a->pages, a->batch, a->max_pages, a->heads, a->head_dim, a->page);
  if (rc == W4_OK) rc = check_rows(a->ldk, a->heads, a->head_dim);
  if (rc == W4_OK) rc = check_rows(a->ldv, a->heads, a->head_dim);
  if (rc != W4_OK) return rc;
  if (a->T > kMaxDim - 1024) return W4_ERR_UNSUPPORTED_SHAPE;
  if (a->T == 0 || a->batch == 0) return W4_OK;
  if (!a->k_dev || !a->v_dev || !a->k_cache_dev || !a->v_cache_dev || !a->k_scale_dev || !a->v_scale_dev || !a->table_dev ||
      !a->cu_dev || !a->lens_dev)
    return W4_ERR_INVALID_ARG;
  if (!aligned(a->k_dev, 16) || !aligned(a->v_dev, 16) || !aligned(a->k_cache_dev, 16) || !aligned(a->v_cache_dev, 16) ||
      !aligned(a->k_scale_dev, 4) || !aligned(a->v_scale_dev, 4) || !aligned(a->table_dev, 4) || !aligned(a->cu_dev, 4) ||
      !aligned(a->lens_dev, 4))
    return W4_ERR_MISALIGNED;
  w4::KvAppendArgs k;
  k.k = a->k_dev;
  k.v = a->v_dev;
  k.k_cache = a->k_cache_dev;
  k.v_cache = a->v_cache_dev;
  k.k_scale = a->k_scale_dev;
  k.v_scale = a->v_scale_dev;
  k.table = a->table_dev;
  k.cu = a->cu_dev;
  k.lens = a->lens_dev;
  k.T = a->T;
  k.ldk = a->ldk;
  k.ldv = a->ldv;
  k.pages = a->pages;
  k.batch = a->batch;
  k.max_pages = a->max_pages;
  k.heads = a->heads;
  k.head_dim = a->head_dim;
  k.page = a->page;
  k.dtype = a->dtype;
  return status_of(w4::launch_kv_append(k, num_sms_current_device(), static_cast<cudaStream_t>(stream)));
}

size_t w4_kv_attention_workspace_bytes(int32_t batch, int32_t n, int32_t q_heads, int32_t k_heads, int32_t head_dim) {
  if (check_kv_attention_sizes(batch, n, q_heads, k_heads, head_dim) != W4_OK) return 0;
  return w4::kv_attention_workspace_bytes(n, q_heads, k_heads, head_dim, num_sms_current_device());
}

int w4_kv_attention(const w4_kv_attention_args *a, void *workspace_dev, size_t workspace_bytes, void *stream) {
  if (!a || !type16(a->dtype)) return W4_ERR_INVALID_ARG;
  if (!(a->scale > 0.0f) || std::isinf(a->scale)) return W4_ERR_INVALID_ARG;
  int rc = check_kv_attention_sizes(a->batch, a->n, a->q_heads, a->k_heads, a->head_dim);
  if (rc == W4_OK) rc = check_cache(a->pages, a->batch, a->max_pages, a->k_heads, a->head_dim, a->page);
  if (rc == W4_OK) rc = check_rows(a->ldq, a->q_heads, a->head_dim);
  if (rc == W4_OK) rc = check_rows(a->ldo, a->q_heads, a->head_dim);
  if (rc != W4_OK) return rc;
  // tiles (16 keys of 16 query rows) and what beginning an item costs are counted in 32 bits
  const int64_t items = static_cast<int64_t>(a->batch) * a->k_heads * w4::cdiv(static_cast<int64_t>(a->n) * (a->q_heads / a->k_heads), 16);
  if (items * (w4::cdiv(static_cast<int64_t>(a->max_pages) * a->page, 16) + 16) > (int64_t{1} << 30)) return W4_ERR_UNSUPPORTED_SHAPE;
  if (a->batch == 0) return W4_OK;
  if (!a->q_dev || !a->k_cache_dev || !a->v_cache_dev || !a->k_scale_dev || !a->v_scale_dev || !a->table_dev || !a->lens_dev ||
      !a->out_dev || !workspace_dev)
    return W4_ERR_INVALID_ARG;
  if (!aligned(a->q_dev, 16) || !aligned(a->k_cache_dev, 16) || !aligned(a->v_cache_dev, 16) || !aligned(a->out_dev, 16) ||
      !aligned(a->k_scale_dev, 4) || !aligned(a->v_scale_dev, 4) || !aligned(a->table_dev, 4) || !aligned(a->lens_dev, 4) ||
      !aligned(workspace_dev, 256))
    return W4_ERR_MISALIGNED;
  const int sms = num_sms_current_device();
  if (workspace_bytes < w4::kv_attention_workspace_bytes(a->n, a->q_heads, a->k_heads, a->head_dim, sms))
    return W4_ERR_WORKSPACE_TOO_SMALL;
  w4::KvAttentionArgs k;
  k.q = a->q_dev;
  k.k_cache = a->k_cache_dev;
  k.v_cache = a->v_cache_dev;
  k.k_scale = a->k_scale_dev;
  k.v_scale = a->v_scale_dev;
  k.table = a->table_dev;
  k.lens = a->lens_dev;
  k.out = a->out_dev;
  k.ldq = a->ldq;
  k.ldo = a->ldo;
  k.pages = a->pages;
  k.batch = a->batch;
  k.n = a->n;
  k.max_pages = a->max_pages;
  k.q_heads = a->q_heads;
  k.k_heads = a->k_heads;
  k.head_dim = a->head_dim;
  k.page = a->page;
  k.dtype = a->dtype;
  k.scale = a->scale;
  return status_of(w4::launch_kv_attention(k, workspace_dev, sms, static_cast<cudaStream_t>(stream)));
}

namespace {

int check_prompt_sizes(int64_t T, int32_t batch, int32_t q_heads) {
  if (T < 0 || batch < 0 || q_heads < 1) return W4_ERR_INVALID_ARG;
  if (T > (1 << 30) || q_heads > 65535 || (w4::cdiv(T, 128) + batch) * q_heads > kMaxDim) return W4_ERR_UNSUPPORTED_SHAPE;
  return W4_OK;
}

}  // namespace

size_t w4_prompt_attention_workspace_bytes(int64_t T, int32_t batch, int32_t q_heads) {
  if (check_prompt_sizes(T, batch, q_heads) != W4_OK) return 0;
  return w4::kPromptWorkspaceBytes;
}

int w4_prompt_attention(const w4_prompt_attention_args *a, void *workspace_dev, size_t workspace_bytes, void *stream) {
  return w4_prompt_attention_opts(a, workspace_dev, workspace_bytes, nullptr, stream);
}

int w4_prompt_attention_opts(const w4_prompt_attention_args *a, void *workspace_dev, size_t workspace_bytes,
                             const w4a16_options *opts, void *stream) {
  if (!a || !type16(a->dtype) || a->k_heads < 1 || a->head_dim < 1) return W4_ERR_INVALID_ARG;
  if (opts && (opts->kernel || opts->block_n || opts->ctas || opts->schedule || opts->cluster || opts->dtype || opts->reserved ||
               (opts->flags & ~W4_FLAG_TEST_TIMEOUT)))
    return W4_ERR_INVALID_ARG;
  if (!(a->scale > 0.0f) || std::isinf(a->scale)) return W4_ERR_INVALID_ARG;
  int rc = check_prompt_sizes(a->T, a->batch, a->q_heads);
  if (rc != W4_OK) return rc;
  if (a->q_heads % a->k_heads != 0) return W4_ERR_INVALID_ARG;
  if (a->head_dim % 8 != 0 || a->head_dim > 128) return W4_ERR_UNSUPPORTED_SHAPE;
  rc = check_rows(a->ldq, a->q_heads, a->head_dim);
  if (rc == W4_OK) rc = check_rows(a->ldk, a->k_heads, a->head_dim);
  if (rc == W4_OK) rc = check_rows(a->ldv, a->k_heads, a->head_dim);
  if (rc == W4_OK) rc = check_rows(a->ldo, a->q_heads, a->head_dim);
  if (rc != W4_OK) return rc;
  if (a->T == 0 || a->batch == 0) return W4_OK;
  if (!a->q_dev || !a->k_dev || !a->v_dev || !a->cu_dev || !a->out_dev || !workspace_dev) return W4_ERR_INVALID_ARG;
  if (!aligned(a->q_dev, 16) || !aligned(a->k_dev, 16) || !aligned(a->v_dev, 16) || !aligned(a->out_dev, 16) ||
      !aligned(a->cu_dev, 4) || !aligned(workspace_dev, 256))
    return W4_ERR_MISALIGNED;
  if (workspace_bytes < w4::kPromptWorkspaceBytes) return W4_ERR_WORKSPACE_TOO_SMALL;
  w4::PromptArgs p;
  p.q = a->q_dev;
  p.k = a->k_dev;
  p.v = a->v_dev;
  p.cu = a->cu_dev;
  p.out = a->out_dev;
  p.T = a->T;
  p.ldq = a->ldq;
  p.ldk = a->ldk;
  p.ldv = a->ldv;
  p.ldo = a->ldo;
  p.batch = a->batch;
  p.q_heads = a->q_heads;
  p.k_heads = a->k_heads;
  p.head_dim = a->head_dim;
  p.dtype = a->dtype;
  p.scale = a->scale;
  p.wait_limit = opts ? opts->wait_limit_cycles : 0;
  p.test_timeout = opts && (opts->flags & W4_FLAG_TEST_TIMEOUT) != 0;
  return status_of(w4::launch_prompt_attention(p, workspace_dev, num_sms_current_device(), static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
