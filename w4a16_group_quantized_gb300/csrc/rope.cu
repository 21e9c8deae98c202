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
// A lane holds 8 values of a head, a power of two of lanes a head: four pairs' both halves (values 4 i .. 4 i + 3 and those
// half the rotation further, or 8 neighbours where neighbours are paired), or 8 neighbours past the rotation. So a pair is
// turned within a lane, and the sines and cosines that a lane needs are the same for all heads of a row: they stay in
// registers. Only the sum of squares goes by shuffles. A value is read and written once, by the same lane, and a call may run in
// place. Sines and cosines of a block's rows are made once and shared through shared memory, as are the weights in fp32.
// Bound by memory for many rows, by latency for few. What keeps it from being bound by instructions is that all that differs
// between calls but not within one (neighbours paired or not, norms or not) is a template's: chosen by the lane it was 307
// instructions for 8 values, and 181 us for 16384 rows of 72 heads of 128.
#include <type_traits>

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
__device__ __forceinline__ void unpack8(const uint2 &lo, const uint2 &hi, float (&f)[8]) {
  const uint32_t w[4] = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = value_f32<DT>(w[i] & 0xffffu);
    f[2 * i + 1] = value_f32<DT>(w[i] >> 16);
  }
}

// LG: lanes a head. PAIRED: neighbours are paired.
template <int DT, int LG, bool NORM, bool PAIRED>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  float *weights = reinterpret_cast<float *>(smem);                         // [q, k][LG][8] in the lanes' order
  float *cosines = weights + (NORM ? 16 * LG : 0), *sines = cosines + p.rows * p.half;  // [rows][half] each
  long long *fractions = reinterpret_cast<long long *>(sines + p.rows * p.half);        // [half], of a turn a position
  griddep_launch_dependents();
  griddep_wait();
  const int64_t row0 = static_cast<int64_t>(blockIdx.x / p.head_parts) * p.rows;
  const int part = blockIdx.x % p.head_parts;
  const int rows = static_cast<int>(min(static_cast<int64_t>(p.rows), p.T - row0));
  const int lane = threadIdx.x % LG;
  const int group = threadIdx.x / LG;
  // the lane's values: four from at0, four from at1
  const bool inside = 8 * lane < p.head_dim, turned = 8 * lane < 2 * p.half;
  const bool apart = turned && !PAIRED;
  const int at0 = apart ? 4 * lane : 8 * lane, at1 = apart ? p.half + 4 * lane : 8 * lane + 4;
  if (NORM && threadIdx.x < 2 * LG) {
    const uint16_t *w = threadIdx.x < LG ? p.q_weight : p.k_weight;
    uint2 lo = make_uint2(0, 0), hi = lo;
    if (w && inside) lo = *reinterpret_cast<const uint2 *>(w + at0), hi = *reinterpret_cast<const uint2 *>(w + at1);
    float f[8];
    unpack8<DT>(lo, hi, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) weights[8 * threadIdx.x + e] = f[e];
  }
  for (int f = threadIdx.x; f < p.half; f += kRopeThreads) {
    const double turns = static_cast<double>(p.freqs[f]) * 0.15915494309189533577;  // 1 / 2 pi
    fractions[f] = __double2ll_rn((turns - rint(turns)) * 18446744073709551616.0);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.half * rows; i += kRopeThreads) {
    const int r = i / p.half, f = i - r * p.half;
    const int axis = (f >= p.section_end[0]) + (f >= p.section_end[1]) + (f >= p.section_end[2]);
    const long long pos = p.positions[axis * p.T + row0 + r];
    const long long at = static_cast<long long>(static_cast<unsigned long long>(fractions[f]) * static_cast<unsigned long long>(pos));
    sincospif(__ll2float_rn(at) * 0x1p-63f, &sines[i], &cosines[i]);  // half turns
  }
  __syncthreads();

  const float inv_dim = 1.0f / static_cast<float>(p.head_dim);
  const int step = p.head_step * p.head_parts;  // heads between a group's
  const int first = part * p.head_step + group;
  for (int r = 0; r < rows; ++r) {
    const int64_t row = row0 + r;
    const uint16_t *qx = p.q + row * p.ldq, *kx = p.k + row * p.ldk - p.q_heads * p.head_dim;
    uint16_t *qy = p.q_out + row * p.ldqo, *ky = p.k_out + row * p.ldko - p.q_heads * p.head_dim;
    float c[4], s[4];
    if (turned) {
      const float4 c4 = *reinterpret_cast<const float4 *>(cosines + r * p.half + 4 * lane);
      const float4 s4 = *reinterpret_cast<const float4 *>(sines + r * p.half + 4 * lane);
      c[0] = c4.x, c[1] = c4.y, c[2] = c4.z, c[3] = c4.w;
      s[0] = s4.x, s[1] = s4.y, s[2] = s4.z, s[3] = s4.w;
    }
    auto load = [&](int h, uint2 *lo, uint2 *hi) {
      *lo = *hi = make_uint2(0, 0);
      if (inside && h < p.heads) {
        const uint16_t *x = (h < p.q_heads ? qx : kx) + h * p.head_dim;
        *lo = *reinterpret_cast<const uint2 *>(x + at0);
        *hi = *reinterpret_cast<const uint2 *>(x + at1);
      }
    };
    // the next head's while one is worked on (a lane writes only what it has read: in place too)
    uint2 lo, hi, next_lo, next_hi;
    load(first, &next_lo, &next_hi);
    for (int h = first; h - group < p.heads; h += step) {
      lo = next_lo, hi = next_hi;
      load(h + step, &next_lo, &next_hi);
      float x[8];
      unpack8<DT>(lo, hi, x);
      const bool of_q = h < p.q_heads;
      if (NORM) {
        float sum = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = fmaf(x[e], x[e], sum);
#pragma unroll
        for (int i = LG / 2; i > 0; i /= 2) sum += __shfl_xor_sync(kAll, sum, i, LG);
        if (of_q ? p.q_weight != nullptr : p.k_weight != nullptr) {
          const float scale = rsqrtf(fmaf(sum, inv_dim, p.eps));
          const float4 *w = reinterpret_cast<const float4 *>(weights + (of_q ? 0 : 8 * LG) + 8 * lane);
          const float4 w0 = w[0], w1 = w[1];
          const float f[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = x[e] * scale * f[e];
        }
      }
      if (turned) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = PAIRED ? 2 * e : e, j = PAIRED ? 2 * e + 1 : 4 + e;
          const float a = x[i], b = x[j];
          x[i] = a * c[e] - b * s[e];
          x[j] = fmaf(b, c[e], a * s[e]);
        }
      }
      if (inside && h < p.heads) {
        uint16_t *y = (of_q ? qy : ky) + h * p.head_dim;
        *reinterpret_cast<uint2 *>(y + at0) = make_uint2(out_bits2<DT>(x[0], x[1]), out_bits2<DT>(x[2], x[3]));
        *reinterpret_cast<uint2 *>(y + at1) = make_uint2(out_bits2<DT>(x[4], x[5]), out_bits2<DT>(x[6], x[7]));
      }
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
  const bool norm = p.q_weight || p.k_weight;
  const int smem = (norm ? 16 * lg * static_cast<int>(sizeof(float)) : 0) + p.half * (p.rows * 2 * static_cast<int>(sizeof(float)) + static_cast<int>(sizeof(long long)));
  auto go = [&](auto kern) { return launch_programmatic(kern, static_cast<int>(blocks), kRopeThreads, smem, stream, p); };
  auto pick = [&](auto n, auto paired) {
    constexpr bool N = decltype(n)::value, P = decltype(paired)::value;
    switch (lg) {
      case 1: return go(rope_kernel<DT, 1, N, P>);
      case 2: return go(rope_kernel<DT, 2, N, P>);
      case 4: return go(rope_kernel<DT, 4, N, P>);
      case 8: return go(rope_kernel<DT, 8, N, P>);
      case 16: return go(rope_kernel<DT, 16, N, P>);
      default: return go(rope_kernel<DT, 32, N, P>);
    }
  };
  if (norm) return p.interleaved ? pick(std::true_type{}, std::true_type{}) : pick(std::true_type{}, std::false_type{});
  return p.interleaved ? pick(std::false_type{}, std::true_type{}) : pick(std::false_type{}, std::false_type{});
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
