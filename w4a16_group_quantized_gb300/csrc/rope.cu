// w4_qk_norm_rope: the norm of each head of queries and keys and the rotation of its values by the row's position, in one
// pass over both.
//
// For a head x: u = x * rsqrt(mean(x^2) + eps) * weight; for each pair (i, j) of the first `rot` values
// (y_i, y_j) = (u_i cos a - u_j sin a, u_j cos a + u_i sin a) with the angle a = position * freq_i.
//
// A position may be far (a = 10^6 and more), and 32 bits would lose the angle: what matters is position * freq / 2 pi modulo
// 1. A block forms freq / 2 pi modulo 1 once, in 64 bits, as a 64-bit fraction of a turn; the product with the
// position in wrapping integer arithmetic is the turn, exact to position * 2^-64 and the fraction's own rounding.
//
// A lane holds 8 consecutive values (16 bytes) of a head, a power of two of lanes a head; the sum of squares and the pairs'
// other halves (the same place of another lane, unless neighbours are paired) go by shuffles, so that a value is read and
// written once and a call may run in place. Sines and cosines of a row are made once a block and shared by its heads.
// Bound by memory for many rows, by latency for few.
#include "gemm_common.cuh"
#include "internal.h"
#include "mma.cuh"
#include "ptx.cuh"

namespace w4 {
namespace {

using namespace detail;

constexpr int kRopeThreads = 256;
constexpr uint32_t kAll = 0xffffffffu;

struct RopeParams {
  const uint16_t *q, *k;
  uint16_t *q_out, *k_out;
  const int32_t *positions;
  const float *freqs;
  const uint16_t *q_weight, *k_weight;
  int64_t T, ldq, ldk, ldqo, ldko;
  int q_heads, heads, head_dim, half;
  int section_end[4];
  int interleaved;
  float eps;
  int rows;        // of a block
  int head_step;   // heads of a block in a pass
  int head_parts;  // blocks that share a row's heads
};

template <int DT>
__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = value_f32<DT>(w[i] & 0xffffu);
    f[2 * i + 1] = value_f32<DT>(w[i] >> 16);
  }
}

// LG: lanes a head.
template <int DT, int LG>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  extern __shared__ float2 turn[];  // [rows][half]: cosine, sine
  griddep_launch_dependents();
  griddep_wait();
  const int64_t row0 = static_cast<int64_t>(blockIdx.x / p.head_parts) * p.rows;
  const int part = blockIdx.x % p.head_parts;
  const int rows = static_cast<int>(min(static_cast<int64_t>(p.rows), p.T - row0));
  // thread i % half's frequency, for the rows i / half, ...
  for (int i = threadIdx.x; i < p.half * rows; i += kRopeThreads) {
    const int f = i % p.half, r = i / p.half;
    const double turns = static_cast<double>(p.freqs[f]) * 0.15915494309189533577;  // 1 / 2 pi
    const long long fraction = __double2ll_rn((turns - rint(turns)) * 18446744073709551616.0);
    const int axis = (f >= p.section_end[0]) + (f >= p.section_end[1]) + (f >= p.section_end[2]);
    const int32_t pos = p.positions[axis * p.T + row0 + r];
    const long long at = static_cast<long long>(static_cast<unsigned long long>(fraction) * static_cast<unsigned long long>(static_cast<long long>(pos)));
    float2 cs;
    sincospif(__ll2float_rn(at) * 0x1p-63f, &cs.y, &cs.x);  // half turns
    turn[i] = cs;
  }
  __syncthreads();

  const int lane = threadIdx.x % LG;
  const int group = threadIdx.x / LG;
  const bool inside = 8 * lane < p.head_dim;
  const float inv_dim = 1.0f / static_cast<float>(p.head_dim);
  const int heads_here = p.head_step * p.head_parts;  // heads between a group's
  // where this lane's values lie in the rotation: all of a lane's are on one side (half is a multiple of 8)
  const bool turned = 8 * lane < 2 * p.half;
  const bool upper = 8 * lane >= p.half;
  const int other = upper ? lane - p.half / 8 : lane + p.half / 8;
  for (int r = 0; r < rows; ++r) {
    const int64_t row = row0 + r;
    for (int h = part * p.head_step + group; h - group < p.heads; h += heads_here) {
      const bool live = inside && h < p.heads;
      const bool of_q = h < p.q_heads;
      const uint16_t *weight = of_q ? p.q_weight : p.k_weight;
      const int hh = of_q ? h : h - p.q_heads;
      uint4 raw = make_uint4(0, 0, 0, 0);
      if (live) raw = *reinterpret_cast<const uint4 *>((of_q ? p.q + row * p.ldq : p.k + row * p.ldk) + hh * p.head_dim + 8 * lane);
      float x[8];
      unpack8<DT>(raw, x);
      if (p.q_weight || p.k_weight) {  // (the same for the whole warp)
        float sum = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = fmaf(x[e], x[e], sum);
#pragma unroll
        for (int s = LG / 2; s > 0; s /= 2) sum += __shfl_xor_sync(kAll, sum, s, LG);
        if (weight) {
          float w[8];
          uint4 wr = make_uint4(0, 0, 0, 0);
          if (live) wr = *reinterpret_cast<const uint4 *>(weight + 8 * lane);
          unpack8<DT>(wr, w);
          const float scale = rsqrtf(fmaf(sum, inv_dim, p.eps));
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = x[e] * scale * w[e];
        }
      }
      if (p.half) {
        const float2 *cs = turn + r * p.half;
        if (p.interleaved) {
          if (turned) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 c = cs[4 * lane + e];
              const float a = x[2 * e], b = x[2 * e + 1];
              x[2 * e] = a * c.x - b * c.y;
              x[2 * e + 1] = fmaf(b, c.x, a * c.y);
            }
          }
        } else {
          float y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = __shfl_sync(kAll, x[e], other, LG);
          if (turned) {
            const float2 *mine = cs + 8 * (upper ? other : lane);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float2 c = mine[e];
              x[e] = upper ? fmaf(x[e], c.x, y[e] * c.y) : x[e] * c.x - y[e] * c.y;
            }
          }
        }
      }
      if (live)
        *reinterpret_cast<uint4 *>((of_q ? p.q_out + row * p.ldqo : p.k_out + row * p.ldko) + hh * p.head_dim + 8 * lane) =
            make_uint4(out_bits2<DT>(x[0], x[1]), out_bits2<DT>(x[2], x[3]), out_bits2<DT>(x[4], x[5]), out_bits2<DT>(x[6], x[7]));
    }
  }
}

template <int DT>
cudaError_t launch_dim(RopeParams p, int num_sms, cudaStream_t stream) {
  int lg = 1;
  while (8 * lg < p.head_dim) lg *= 2;
  p.head_step = kRopeThreads / lg;
  const int passes = static_cast<int>(cdiv(p.heads, p.head_step));
  // few rows: a row's heads go to blocks of their own; many: a block takes a few rows
  p.head_parts = 1;
  while (p.head_parts < passes && p.T * p.head_parts < 4 * num_sms) p.head_parts *= 2;
  p.rows = 1;
  while (p.rows < 8 && p.T > static_cast<int64_t>(16) * num_sms * p.rows) p.rows *= 2;
  const int64_t blocks = cdiv(p.T, p.rows) * p.head_parts;
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
  const int smem = p.rows * p.half * static_cast<int>(sizeof(float2));
  auto go = [&](auto kern) { return launch_programmatic(kern, static_cast<int>(blocks), kRopeThreads, smem, stream, p); };
  switch (lg) {
    case 1: return go(rope_kernel<DT, 1>);
    case 2: return go(rope_kernel<DT, 2>);
    case 4: return go(rope_kernel<DT, 4>);
    case 8: return go(rope_kernel<DT, 8>);
    case 16: return go(rope_kernel<DT, 16>);
    default: return go(rope_kernel<DT, 32>);
  }
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &a, int num_sms, cudaStream_t stream) {
  RopeParams p;
  p.q = static_cast<const uint16_t *>(a.q);
  p.k = static_cast<const uint16_t *>(a.k);
  p.q_out = static_cast<uint16_t *>(a.q_out);
  p.k_out = static_cast<uint16_t *>(a.k_out);
  p.positions = a.positions;
  p.freqs = a.freqs;
  p.q_weight = static_cast<const uint16_t *>(a.q_weight);
  p.k_weight = static_cast<const uint16_t *>(a.k_weight);
  p.T = a.T;
  p.ldq = a.ldq;
  p.ldk = a.ldk;
  p.ldqo = a.ldqo;
  p.ldko = a.ldko;
  p.q_heads = a.q_heads;
  p.heads = a.q_heads + a.k_heads;
  p.head_dim = a.head_dim;
  p.half = a.rot / 2;
  for (int i = 0; i < 4; ++i) p.section_end[i] = a.section_end[i];
  p.interleaved = a.interleaved;
  p.eps = a.eps;
  return a.dtype == kDtypeBf16 ? launch_dim<kDtypeBf16>(p, num_sms, stream) : launch_dim<kDtypeF16>(p, num_sms, stream);
}

}  // namespace w4
