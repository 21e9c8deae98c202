// w4_prompt_attention: causal attention over packed prompts.
//
// out[t, h] = sum_p w_p v_p / sum_p w_p, w_p = exp(scale * q . k_p) over the rows p <= t of t's sequence, with the running
// maximum m and sum l of a softmax: s = q . k * scale * log2 e, w = 2^(s - m), O = O * 2^(m_old - m) + w v.
#include <atomic>

#include "gemm_common.cuh"
#include "internal.h"
#include "mma.cuh"
#include "ptx.cuh"

namespace w4 {
namespace {

using namespace detail;

constexpr uint32_t kAll = 0xffffffffu;

struct PromptParams {
  const uint16_t *q, *k, *v;
  const int32_t *cu;
  uint16_t *out;
  int64_t ldq, ldk, ldv, ldo;
  int T, batch, q_heads, r, head_dim;
  float scale;  // times log2 e
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// One row by one warp in fp32: 32 keys at a time, a key a lane for the products with q, four of the head's values a lane for
// the sums.
template <int DT>
__device__ __noinline__ void one_row(const PromptParams &p, int begin, int row, int h) {
  const int lane = threadIdx.x % 32;
  const uint16_t *q = p.q + row * p.ldq + static_cast<int64_t>(h) * p.head_dim;
  const uint16_t *k = p.k + static_cast<int64_t>(h / p.r) * p.head_dim;
  const uint16_t *v = p.v + static_cast<int64_t>(h / p.r) * p.head_dim;
  float m = -INFINITY, l = 0.0f, o[4] = {};
  for (int key0 = begin; key0 <= row; key0 += 32) {
    const int key = key0 + lane;
    float s = -INFINITY;
    if (key <= row) {
      s = 0.0f;
      for (int d = 0; d < p.head_dim; ++d) s = fmaf(value_f32<DT>(q[d]), value_f32<DT>(k[key * p.ldk + d]), s);
      s *= p.scale;
    }
    float top = s;
#pragma unroll
    for (int i = 16; i > 0; i /= 2) top = fmaxf(top, __shfl_xor_sync(kAll, top, i));
    const float now = fmaxf(m, top);
    const float alpha = now == m ? 1.0f : ex2(m - now);
    m = now;
    const float w = key <= row ? ex2(s - now) : 0.0f;
    l = l * alpha + w;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] *= alpha;
    const int count = min(32, row - key0 + 1);
    for (int j = 0; j < count; ++j) {
      const float wj = __shfl_sync(kAll, w, j);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (4 * lane + e < p.head_dim) o[e] = fmaf(wj, value_f32<DT>(v[(key0 + j) * p.ldv + 4 * lane + e]), o[e]);
    }
  }
#pragma unroll
  for (int i = 16; i > 0; i /= 2) l += __shfl_xor_sync(kAll, l, i);
  uint16_t *out = p.out + row * p.ldo + static_cast<int64_t>(h) * p.head_dim;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (4 * lane + e < p.head_dim) out[4 * lane + e] = out_bits<DT>(o[e] / l);
}

template <int DT>
__global__ void __launch_bounds__(256) prompt_rows_kernel(const __grid_constant__ PromptParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 8 + threadIdx.x / 32;
  const int row = static_cast<int>(i / p.q_heads), h = static_cast<int>(i % p.q_heads);
  if (row >= p.T) return;
  for (int b = 0; b < p.batch; ++b) {
    const int begin = max(p.cu[b], 0), end = min(p.cu[b + 1], p.T);
    if (row >= begin && row < end) {
      one_row<DT>(p, begin, row, h);
      return;
    }
  }
}

}  // namespace

size_t prompt_attention_workspace_bytes(int64_t, int, int) { return 256; }

cudaError_t launch_prompt_attention(const PromptArgs &a, void *, int, cudaStream_t stream) {
  PromptParams p;
  p.q = static_cast<const uint16_t *>(a.q);
  p.k = static_cast<const uint16_t *>(a.k);
  p.v = static_cast<const uint16_t *>(a.v);
  p.cu = a.cu;
  p.out = static_cast<uint16_t *>(a.out);
  p.ldq = a.ldq;
  p.ldk = a.ldk;
  p.ldv = a.ldv;
  p.ldo = a.ldo;
  p.T = static_cast<int>(a.T);
  p.batch = a.batch;
  p.q_heads = a.q_heads;
  p.r = a.q_heads / a.k_heads;
  p.head_dim = a.head_dim;
  p.scale = a.scale * 1.4426950408889634f;
  const int blocks = static_cast<int>(cdiv(a.T * a.q_heads, 8));
  return a.dtype == kDtypeBf16 ? launch_programmatic(prompt_rows_kernel<kDtypeBf16>, blocks, 256, 0, stream, p)
                               : launch_programmatic(prompt_rows_kernel<kDtypeF16>, blocks, 256, 0, stream, p);
}

}  // namespace w4
