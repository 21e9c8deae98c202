// w4_route: the experts of each token and their weights, from the router's scores.
//
// For each row l of E logits: s_i = e^(l_i - max l) / sum e^(l - max l), or 1 / (1 + e^-l_i); c_i = s_i + b_i.
// The row keeps its `top_groups` best groups of E / groups consecutive experts (a group is worth the sum of
// its `group_top` best c) and chooses the k best c in them, the lowest index first among equals; its weights are
// s at the chosen experts, divided by their sum if asked (also where they vanish in 32 bits), times `scale`.
// Without a bias the chosen experts are found by the logits themselves, which order the scores and do not round
// (32-bit scores of unlike logits may be equal).
//
// One warp per row: lane i holds PER consecutive experts as 32-bit keys whose unsigned order is that of the values, so
// that each choice is a warp-wide integer reduction (the largest key) and a vote (the lowest lane that has it). Groups
// that are a power of two of whole lanes are all ranked at once, by exchanges between their lanes; others one
// after another. The rows are independent and short (512 bytes at E = 256): latency bounds a decode step, and the
// issue of the k choices a large prefill. Measured: 64 rows of 256 experts (8 groups, sigmoid, bias, k = 8) 6.3 us, 16384
// rows 25 us (9.6 us and 44 with the groups one after another).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "gemm_common.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace w4 {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kRouteWarps = 4;  // rows per block

template <int DT>
__device__ __forceinline__ float load_logit(const void *p, int64_t i) {
  if (DT == kDtypeF32) return static_cast<const float *>(p)[i];
  if (DT == kDtypeBf16) return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(p)[i]) << 16);
  return __half2float(static_cast<const __half *>(p)[i]);
}

// A lane's PER consecutive logits, in as few loads as 16 bytes each allow.
template <int DT, int PER>
__device__ __forceinline__ void load_logits(const void *p, int64_t i, float (&l)[PER]) {
  constexpr int kSize = DT == kDtypeF32 ? 4 : 2, kBytes = PER * kSize;
  constexpr int kWords = (kBytes + 3) / 4;
  uint32_t w[kWords];
  const char *at = static_cast<const char *>(p) + i * kSize;
  if constexpr (kBytes >= 16) {
#pragma unroll
    for (int j = 0; j < kBytes / 16; ++j) {
      const uint4 v = reinterpret_cast<const uint4 *>(at)[j];
      w[4 * j] = v.x, w[4 * j + 1] = v.y, w[4 * j + 2] = v.z, w[4 * j + 3] = v.w;
    }
  } else if constexpr (kBytes == 8) {
    const uint2 v = *reinterpret_cast<const uint2 *>(at);
    w[0] = v.x, w[1] = v.y;
  } else if constexpr (kBytes == 4) {
    w[0] = *reinterpret_cast<const uint32_t *>(at);
  } else {
    w[0] = *reinterpret_cast<const uint16_t *>(at);
  }
#pragma unroll
  for (int j = 0; j < PER; ++j)
    l[j] = DT == kDtypeF32 ? __uint_as_float(w[j * kSize / 4])
                           : detail::scale_f32<DT == kDtypeF32 ? kDtypeF16 : DT>(w[j * kSize / 4] >> (16 * (j & 1)) & 0xffffu);
}

// Unsigned key with the order of the value (-0 and 0 alike; every key of a value is above 0, which marks
// experts that cannot be chosen any more).
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7fffffffu) : ~key);
}

// A masked logit (-inf; a NaN counts as one) as -inf.
__device__ __forceinline__ float masked(float l) { return isnan(l) ? -INFINITY : l; }

__device__ __forceinline__ float sigmoid(float l) { return 1.0f / (1.0f + expf(-l)); }

// e^(l - max), 1 at the maximum also where that is infinite, 0 at a masked place.
__device__ __forceinline__ float exp_below(float l, float top) {
  return l == -INFINITY ? 0.0f : l == top ? 1.0f : expf(l - top);
}

template <int DT, int PER>
__global__ void __launch_bounds__(32 * kRouteWarps)
    route_kernel(const void *logits, int64_t T, int E, int64_t ld, const float *bias, RouteParams o,
                 float *weights, int32_t *ids) {
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kRouteWarps + (threadIdx.x >> 5);
  griddep_wait();
  if (row >= T) return;
  const int64_t at = row * ld;

  float l[PER];
  float top = -INFINITY;
  if (o.wide) {
    load_logits<DT, PER>(logits, at + lane * PER, l);
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) l[i] = lane * PER + i < E ? load_logit<DT>(logits, at + lane * PER + i) : -INFINITY;
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    l[i] = masked(l[i]);
    top = fmaxf(top, l[i]);
  }
  float sum = 1.0f;
  if (!o.sigmoid) {
    top = value_of(__reduce_max_sync(kFull, key_of(top)));
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) sum += exp_below(l[i], top);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(kFull, sum, d);
    sum = fmaxf(sum, 1e-37f);  // every expert masked: scores of zero
  }

  uint32_t key[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane * PER + i;
    float c = l[i];
    if (bias && e < E && c != -INFINITY) c = (o.sigmoid ? sigmoid(c) : exp_below(c, top) / sum) + bias[e];
    key[i] = e < E ? key_of(isnan(c) ? -INFINITY : c) : 0u;
  }

  if (o.groups > 1) {
    // lane j keeps what group j is worth; a place's group by a multiplication (e < 1024, exact)
    uint32_t worth = 0u;
    const int lanes = o.group_lanes;  // of a group, a power of two; 0: groups that end inside a lane
    // the sum of two is one of scores, which the logits' own order cannot give
    const bool by_score = o.group_top == 2 && !bias;
    auto merged = [&](uint32_t first, uint32_t second) {
      return o.group_top == 2 ? key_of(value_of(first) + value_of(second)) : first;
    };
    if (lanes > 0) {
      uint32_t first = 0u, second = 0u;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const uint32_t v = by_score && key[i] != 0u ? key_of(o.sigmoid ? sigmoid(l[i]) : exp_below(l[i], top) / sum) : key[i];
        second = max(second, min(first, v));
        first = max(first, v);
      }
      for (int d = 1; d < lanes; d <<= 1) {
        const uint32_t f = __shfl_xor_sync(kFull, first, d), s = __shfl_xor_sync(kFull, second, d);
        second = max(max(second, s), min(first, f));
        first = max(first, f);
      }
      worth = __shfl_sync(kFull, merged(first, second), (lane * lanes) & 31);
      if (lane >= o.groups) worth = 0u;
    } else {
      for (int j = 0; j < o.groups; ++j) {
        uint32_t first = 0u, second = 0u;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int e = lane * PER + i;
          if (e >= E || static_cast<int>((e * o.group_mul) >> 22) != j) continue;
          const uint32_t v = by_score ? key_of(o.sigmoid ? sigmoid(l[i]) : exp_below(l[i], top) / sum) : key[i];
          second = max(second, min(first, v));
          first = max(first, v);
        }
        const uint32_t best = __reduce_max_sync(kFull, first);
        uint32_t next = 0u;
        if (o.group_top == 2) {
          const int has = __ffs(__ballot_sync(kFull, first == best)) - 1;  // one lane gives its best up
          next = __reduce_max_sync(kFull, lane == has ? second : first);
        }
        const uint32_t w = merged(best, next);
        if (lane == j) worth = w;
      }
    }
    uint32_t kept = 0u;
    for (int j = 0; j < o.top_groups; ++j) {
      const uint32_t best = __reduce_max_sync(kFull, worth);
      const int has = __ffs(__ballot_sync(kFull, worth == best)) - 1;
      kept |= 1u << has;
      if (lane == has) worth = 0u;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = lane * PER + i;
      if (e < E && !((kept >> ((e * o.group_mul) >> 22)) & 1u)) key[i] = 0u;
    }
  }

  int mine = 0;  // lane j: the j-th choice
  for (int j = 0; j < o.k; ++j) {
    uint32_t mine_best = 0u;
#pragma unroll
    for (int i = 0; i < PER; ++i) mine_best = max(mine_best, key[i]);
    const uint32_t best = __reduce_max_sync(kFull, mine_best);
    // the lowest lane that has it holds the lowest such places; the first of its own is the choice
    const int has = __ffs(__ballot_sync(kFull, mine_best == best)) - 1;
    int place = 0;
#pragma unroll
    for (int i = PER - 1; i >= 0; --i)
      if (key[i] == best) place = i;
    if (lane == has) {
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (i == place) key[i] = 0u;
    }
    place = __shfl_sync(kFull, place, has) + has * PER;
    if (lane == j) mine = place;
  }

  float w = 0.0f;
  if (lane < o.k) {
    const float c = masked(load_logit<DT>(logits, at + mine));
    w = o.sigmoid ? sigmoid(c) : exp_below(c, top) / sum;
  }
  if (o.renormalize) {
    float all = w;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) all += __shfl_xor_sync(kFull, all, d);
    if (all < 1e-30f) {
      // The chosen scores leave the range of 32 bits, but their quotients do not: below 1e-30 / 32 both kinds of score are
      // e^l times what all experts share, so the weights are e^(l - m) over their sum, m the largest chosen logit.
      const float c = lane < o.k ? masked(load_logit<DT>(logits, at + mine)) : -INFINITY;
      const float m = value_of(__reduce_max_sync(kFull, key_of(c)));
      w = exp_below(c, m);
      all = w;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) all += __shfl_xor_sync(kFull, all, d);
    }
    w = all > 0.0f ? w / all : 0.0f;  // no expert left: weights of 0
  }
  if (lane < o.k) {
    weights[row * o.k + lane] = w * o.scale;
    ids[row * o.k + lane] = mine;
  }
}

template <int DT>
cudaError_t launch_dt(const void *logits, int64_t T, int E, int64_t ld, const float *bias, RouteParams o,
                      float *weights, int32_t *ids, cudaStream_t stream) {
  int per = 1;
  while (per * 32 < E) per *= 2;
  const int size = E / o.groups, lanes = size % per == 0 ? size / per : 0;
  const int bytes = DT == kDtypeF32 ? 4 : 2;
  o.wide = E == 32 * per && ld * bytes % 16 == 0 && reinterpret_cast<uintptr_t>(logits) % 16 == 0;
  o.group_lanes = lanes > 0 && (lanes & (lanes - 1)) == 0 ? lanes : 0;
  auto kern = per <= 1   ? route_kernel<DT, 1>
              : per <= 2 ? route_kernel<DT, 2>
              : per <= 4 ? route_kernel<DT, 4>
              : per <= 8 ? route_kernel<DT, 8>
              : per <= 16 ? route_kernel<DT, 16>
                          : route_kernel<DT, 32>;
  return detail::launch_programmatic(kern, static_cast<int>(cdiv(T, kRouteWarps)), 32 * kRouteWarps, 0, stream, logits,
                                     T, E, ld, bias, o, weights, ids);
}

}  // namespace

cudaError_t launch_route(const void *logits, int dtype, int64_t T, int E, int64_t ld, const float *bias,
                         const RouteParams &o, float *weights, int32_t *ids, cudaStream_t stream) {
  switch (dtype) {
    case kDtypeF16: return launch_dt<kDtypeF16>(logits, T, E, ld, bias, o, weights, ids, stream);
    case kDtypeBf16: return launch_dt<kDtypeBf16>(logits, T, E, ld, bias, o, weights, ids, stream);
    default: return launch_dt<kDtypeF32>(logits, T, E, ld, bias, o, weights, ids, stream);
  }
}

}  // namespace w4
