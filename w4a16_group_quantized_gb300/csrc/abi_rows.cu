// C ABI of the operators whose weights are chosen row by row (declared in include/w4a16.h): the router, the experts'
// products and the low-rank adapters. As in abi.cu, every check runs before anything is enqueued.
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

int check_experts_sizes(int64_t T, int64_t K, int64_t I, int32_t experts, int32_t k, int32_t g) {
  if (T < 0 || K < 1 || I < 1 || experts < 1 || k < 1 || k > experts || g < 1 || g % 8 != 0) return W4_ERR_INVALID_ARG;
  if (K % 8 != 0 || I % 8 != 0 || experts > w4::kRowsMaxKeys || k > w4::kRouteMaxK) return W4_ERR_UNSUPPORTED_SHAPE;
  if (T > kMaxDim || K > kMaxDim / 2 || I > kMaxDim / 4 || T * k > kMaxDim) return W4_ERR_UNSUPPORTED_SHAPE;
  if (T * K > (int64_t{1} << 40) || T * I > (int64_t{1} << 40)) return W4_ERR_UNSUPPORTED_SHAPE;
  // a launch's blocks: 32 weight rows of one tile of rows each
  const int64_t rows = K > 2 * I ? K : 2 * I;
  if (w4::max_row_tiles(T * k, experts, 8) * w4::cdiv(rows, 32) > kMaxDim) return W4_ERR_UNSUPPORTED_SHAPE;
  return W4_OK;
}

int check_lora_sizes(int64_t T, int64_t K, int64_t N, int32_t adapters, int32_t rank) {
  if (T < 0 || K < 1 || N < 1 || adapters < 1 || rank < 1) return W4_ERR_INVALID_ARG;
  if (K % 8 != 0 || rank % 8 != 0 || rank > w4::kLoraMaxRank || adapters > w4::kRowsMaxKeys)
    return W4_ERR_UNSUPPORTED_SHAPE;
  // 2^28: a turn past the end of a loop over K or N still fits 32 bits
  if (T > kMaxDim || K > (1 << 28) || N > (1 << 28)) return W4_ERR_UNSUPPORTED_SHAPE;
  return W4_OK;
}

}  // namespace

extern "C" {

int w4_route(const void *logits_dev, int64_t T, int32_t experts, int64_t ld, const float *bias_dev,
             const w4_route_options *opts, float *weights_dev, int32_t *ids_dev, void *stream) {
  if (!opts || T < 0 || experts < 1 || ld < experts) return W4_ERR_INVALID_ARG;
  if ((opts->sigmoid != 0 && opts->sigmoid != 1) || (opts->renormalize != 0 && opts->renormalize != 1))
    return W4_ERR_INVALID_ARG;
  if (!type16(opts->dtype) && opts->dtype != W4_DTYPE_F32) return W4_ERR_INVALID_ARG;
  w4::RouteParams o;
  o.k = opts->k;
  o.groups = opts->groups == 0 ? 1 : opts->groups;
  o.top_groups = opts->top_groups == 0 ? o.groups : opts->top_groups;
  o.group_top = opts->group_top == 0 ? 1 : opts->group_top;
  o.sigmoid = opts->sigmoid != 0;
  o.renormalize = opts->renormalize != 0;
  o.scale = opts->scale;
  if (o.k < 1 || o.groups < 1 || experts % o.groups != 0 || o.top_groups < 1 || o.top_groups > o.groups ||
      o.group_top < 1 || o.group_top > 2 || std::isnan(o.scale))
    return W4_ERR_INVALID_ARG;
  const int size = experts / o.groups;
  if (o.k > o.top_groups * size || (o.groups > 1 && o.group_top > size)) return W4_ERR_INVALID_ARG;
  if (experts > w4::kRouteMaxExperts || o.k > w4::kRouteMaxK || o.groups > 32 || T > kMaxDim)
    return W4_ERR_UNSUPPORTED_SHAPE;
  if (T == 0) return W4_OK;
  if (!logits_dev || !weights_dev || !ids_dev) return W4_ERR_INVALID_ARG;
  if (!aligned(logits_dev, opts->dtype == W4_DTYPE_F32 ? 4 : 2) || (bias_dev && !aligned(bias_dev, 4)) ||
      !aligned(weights_dev, 4) || !aligned(ids_dev, 4))
    return W4_ERR_MISALIGNED;
  o.group_mul = ((1u << 22) + static_cast<uint32_t>(size) - 1u) / static_cast<uint32_t>(size);
  return status_of(w4::launch_route(logits_dev, opts->dtype, T, experts, ld, bias_dev, o, weights_dev, ids_dev,
                                    static_cast<cudaStream_t>(stream)));
}

size_t w4_lora_workspace_bytes(int64_t T, int64_t K, int64_t N, int32_t adapters, int32_t rank) {
  if (check_lora_sizes(T, K, N, adapters, rank) != W4_OK) return 0;
  return w4::lora_workspace_bytes(T > 0 ? T : 1, N, K, adapters, rank, num_sms_current_device());
}

int w4_lora_add(const w4_lora_args *a, void *workspace_dev, size_t workspace_bytes, void *stream) {
  if (!a) return W4_ERR_INVALID_ARG;
  const int rc = check_lora_sizes(a->T, a->K, a->N, a->adapters, a->rank);
  if (rc != W4_OK) return rc;
  if (!type16(a->dtype) || a->reserved != 0 || a->ldx < a->K || a->ldy < a->N || (a->base_dev && a->ldbase < a->N))
    return W4_ERR_INVALID_ARG;
  if (a->ldx % 8 != 0) return W4_ERR_UNSUPPORTED_SHAPE;  // rows of x start on 16-byte boundaries
  // in place means the same rows
  if (a->base_dev == a->y_dev && a->base_dev && a->ldbase != a->ldy) return W4_ERR_INVALID_ARG;
  if (a->T == 0) return W4_OK;
  if (!a->x_dev || !a->A_dev || !a->B_dev || !a->adapter_dev || !a->y_dev || !workspace_dev) return W4_ERR_INVALID_ARG;
  if (!aligned(a->x_dev, 16) || !aligned(a->A_dev, 16) || !aligned(a->B_dev, 16) || !aligned(a->adapter_dev, 4) ||
      !aligned(a->y_dev, 2) || (a->base_dev && !aligned(a->base_dev, 2)) ||
      (a->scaling_dev && !aligned(a->scaling_dev, 4)) || (a->ranks_dev && !aligned(a->ranks_dev, 4)) ||
      !aligned(workspace_dev, 256))
    return W4_ERR_MISALIGNED;
  const int sms = num_sms_current_device();
  if (workspace_bytes < w4::lora_workspace_bytes(a->T, a->N, a->K, a->adapters, a->rank, sms))
    return W4_ERR_WORKSPACE_TOO_SMALL;
  w4::LoraArgs l;
  l.base = a->base_dev;
  l.x = a->x_dev;
  l.A = a->A_dev;
  l.B = a->B_dev;
  l.adapter = a->adapter_dev;
  l.scaling = a->scaling_dev;
  l.ranks = a->ranks_dev;
  l.y = a->y_dev;
  l.T = a->T;
  l.N = a->N;
  l.K = a->K;
  l.ldx = a->ldx;
  l.ldbase = a->ldbase;
  l.ldy = a->ldy;
  l.adapters = a->adapters;
  l.rank = a->rank;
  l.dtype = a->dtype;
  return status_of(w4::launch_lora(l, workspace_dev, sms, static_cast<cudaStream_t>(stream)));
}

size_t w4a16_experts_workspace_bytes(int64_t T, int64_t K, int64_t I, int32_t experts, int32_t k, int32_t g) {
  if (check_experts_sizes(T, K, I, experts, k, g) != W4_OK) return 0;
  return w4::experts_workspace_bytes(T > 0 ? T : 1, K, I, experts, k, g);
}

int w4a16_experts(const w4a16_experts_args *a, void *workspace_dev, size_t workspace_bytes, void *stream) {
  return w4a16_experts_opts(a, workspace_dev, workspace_bytes, nullptr, stream);
}

int w4a16_experts_opts(const w4a16_experts_args *a, void *workspace_dev, size_t workspace_bytes, const w4a16_options *opts,
                       void *stream) {
  if (!a) return W4_ERR_INVALID_ARG;
  if (opts && (opts->kernel || opts->block_n || opts->ctas || opts->schedule || opts->cluster || opts->dtype || opts->reserved ||
               (opts->flags & ~W4_FLAG_TEST_TIMEOUT)))
    return W4_ERR_INVALID_ARG;
  const int rc = check_experts_sizes(a->T, a->K, a->I, a->experts, a->k, a->g);
  if (rc != W4_OK) return rc;
  if (!type16(a->dtype)) return W4_ERR_INVALID_ARG;
  if (a->T == 0) return W4_OK;
  if (!a->x_dev || !a->gate_up_dev || !a->down_dev || !a->ids_dev || !a->weights_dev || !a->y_dev || !workspace_dev)
    return W4_ERR_INVALID_ARG;
  if (!aligned(a->x_dev, 16) || !aligned(a->gate_up_dev, 16) || !aligned(a->down_dev, 16) || !aligned(a->ids_dev, 4) ||
      !aligned(a->weights_dev, 4) || !aligned(a->y_dev, 16) || !aligned(workspace_dev, 256))
    return W4_ERR_MISALIGNED;
  const int sms = num_sms_current_device();
  if (workspace_bytes < w4::experts_workspace_bytes(a->T, a->K, a->I, a->experts, a->k, a->g))
    return W4_ERR_WORKSPACE_TOO_SMALL;
  w4::ExpertsArgs e;
  e.x = a->x_dev;
  e.gate_up = a->gate_up_dev;
  e.down = a->down_dev;
  e.ids = a->ids_dev;
  e.weights = a->weights_dev;
  e.y = a->y_dev;
  e.T = a->T;
  e.K = a->K;
  e.I = a->I;
  e.experts = a->experts;
  e.k = a->k;
  e.g = a->g;
  e.dtype = a->dtype;
  e.wait_limit = opts ? opts->wait_limit_cycles : 0;
  e.test_timeout = opts && (opts->flags & W4_FLAG_TEST_TIMEOUT) != 0;
  return status_of(w4::launch_experts(e, workspace_dev, sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
