// w4_qk_norm_rope: the norm of each head of queries and keys and the rotation of its values by the row's position, in one
// pass over both.
//
// For a head x: u = x * rsqrt(mean(x^2) + eps) * weight; for each pair (i, j) of the first `rot` values
// (y_i, y_j) = (u_i cos a - u_j sin a, u_j cos a + u_i sin a) with the angle a = position * freq_i.
//
// A position may be far (a = 10^6 and more), and 32 bits would lose the angle: what matters is position * freq / 2 pi modulo
// 1. A block forms freq / 2 pi modulo 1 once, as a 64-bit fraction of a turn; the product with the position in wrapping
// integer arithmetic is the turn, exact to position * 2^-64 and the fraction's own rounding.
//
// A lane holds 8 values of a head, a power of two of lanes a head: four pairs' both halves (values 4 i .. 4 i + 3 and those
// half the rotation further, or 8 neighbours where neighbours are paired), or 8 neighbours past the rotation. So a pair is
// turned within a lane, and only the sum of squares goes by shuffles. A value is read and written once, by the same lane, and a
// call may run in place. A block makes the sines and cosines of its rows once, in shared memory; then a lane stays with
// a head for all of the block's rows, four rows' loads at a time: its weights stay in registers, and from row to row one
// offset moves.
// Bound by memory for many rows, by latency for few; for many rows it was bound by instructions until all that differs between
// calls but not within one (neighbours paired or not, norms or not) became a template's, and the rows the inner loop (16384
// rows of 72 heads of 128 with norms: 307 instructions for 8 values, 181 us; 181 and 125 us with heads inside; now 100 us, 6.0
// TB/s, 0.88 of a copy's rate: two waves of blocks, the second one two thirds full). 96 rows of 72 heads: 3.6 us; one of 64: 1.8.
#include <algorithm>
#include <type_traits>

#include "gemm_common.cuh"
#include "internal.h"
#include "mma.cuh"
#include "ptx.cuh"

namespace w4 {
namespace {

using namespace detail;

constexpr int kRopeThreads = 128;
constexpr int kBatch = 4;  // rows whose loads are on their way together
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
  int head_step;   // heads of a block in a turn
  int q_turned;    // q's heads in whole turns
  int head_parts;  // blocks that share a row's heads
};

// Two fp32 values side by side.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

template <int DT>
__device__ __forceinline__ uint64_t unpack2(uint32_t w) {
  if (DT == kDtypeBf16) return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return pair(value_f32<DT>(w & 0xffffu), value_f32<DT>(w >> 16));
}
template <int DT>
__device__ __forceinline__ uint32_t pack2(uint64_t v) {
  const float2 f = unpair(v);
  uint32_t d;
  if (DT == kDtypeBf16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(f.y), "f"(f.x));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(f.y), "f"(f.x));
  return d;
}

// freq / 2 pi modulo 1 in units of 2^-64: freq is m * 2^(e - 150) with integers m and e, and m * (2^64 / 2 pi) a product of 24 by 62
// bits. Off by freq * 2^-64 and the last unit. (64-bit floating point would do, but each of its instructions takes
// some 40 cycles here.)
__device__ __forceinline__ uint64_t fraction_of_turn(float freq) {
  constexpr uint64_t kInvTwoPi = 0x28BE60DB9391054Aull;  // 2^64 / 2 pi
  const uint32_t bits = __float_as_uint(freq), e = bits >> 23 & 255u;
  const uint64_t m = (bits & 0x7FFFFFu) | (e ? 0x800000u : 0u);
  const int down = 150 - static_cast<int>(e ? e : 1u);  // the product's places below 2^-64
  const uint64_t lo = m * kInvTwoPi, hi = __umul64hi(m, kInvTwoPi);
  uint64_t f = 0;
  if (down <= 0)
    f = down > -64 ? lo << -down : 0;
  else if (down < 64)
    f = lo >> down | hi << (64 - down);
  else if (down < 128)
    f = hi >> (down - 64);
  return bits >> 31 ? 0 - f : f;
}

// LG: lanes a head. PAIRED: neighbours are paired.
template <int DT, int LG, bool NORM, bool PAIRED>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  float *cosines = reinterpret_cast<float *>(smem), *sines = cosines + p.rows * p.half;  // [rows][half] each
  uint64_t *fractions = reinterpret_cast<uint64_t *>(sines + p.rows * p.half);          // [half], of a turn a position
  griddep_launch_dependents();
  griddep_wait();
  const int64_t row0 = static_cast<int64_t>(blockIdx.x / p.head_parts) * p.rows;
  const int part = blockIdx.x % p.head_parts;
  const int rows = static_cast<int>(min(static_cast<int64_t>(p.rows), p.T - row0));
  auto position = [&](int i, int *f) {
    const int r = i / p.half;
    *f = i - r * p.half;
    const int axis = (*f >= p.section_end[0]) + (*f >= p.section_end[1]) + (*f >= p.section_end[2]);
    return p.positions[axis * p.T + row0 + r];
  };
  int f, pos = 0;
  if (static_cast<int>(threadIdx.x) < p.half * rows) pos = position(threadIdx.x, &f);  // (beside the frequencies)
  for (int i = threadIdx.x; i < p.half; i += kRopeThreads) fractions[i] = fraction_of_turn(p.freqs[i]);
  __syncthreads();
  for (int i = threadIdx.x; i < p.half * rows; i += kRopeThreads) {
    if (i >= kRopeThreads) pos = position(i, &f);
    const uint64_t at = fractions[f] * static_cast<uint64_t>(static_cast<int64_t>(pos));
    // as half turns; the two halves by themselves, as a conversion of 64 bits would go through the slow pipe
    const float half_turns = fmaf(static_cast<float>(static_cast<int32_t>(at >> 32)), 0x1p-31f, static_cast<float>(static_cast<uint32_t>(at)) * 0x1p-63f);
    sincospif(half_turns, &sines[i], &cosines[i]);
  }
  __syncthreads();

  const int lane = threadIdx.x % LG;
  const int group = threadIdx.x / LG;
  // the lane's values: four from at0, four from at1
  const bool inside = 8 * lane < p.head_dim, turned = 8 * lane < 2 * p.half;
  const bool apart = turned && !PAIRED;
  const int at0 = apart ? 4 * lane : 8 * lane, at1 = apart ? p.half + 4 * lane : 8 * lane + 4;
  const float inv_dim = 1.0f / static_cast<float>(p.head_dim);
  // q's heads, then k's, a head a group and turn
  for (int base = part * p.head_step; base < p.q_turned + p.heads - p.q_heads; base += p.head_step * p.head_parts) {
    const bool of_q = base < p.q_turned;  // (q's turns are whole ones: q_turned is a multiple of head_step)
    const int h = of_q ? base + group : base - p.q_turned + group;
    const bool live = inside && h < (of_q ? p.q_heads : p.heads - p.q_heads);
    const int64_t ld = of_q ? p.ldq : p.ldk, ldo = of_q ? p.ldqo : p.ldko;
    const char *x = reinterpret_cast<const char *>((of_q ? p.q : p.k) + row0 * ld);
    char *y = reinterpret_cast<char *>((of_q ? p.q_out : p.k_out) + row0 * ldo);
    const uint32_t hop = static_cast<uint32_t>(2 * ld), hop_out = static_cast<uint32_t>(2 * ldo);  // (a block's rows span less than 2^31 bytes)
    uint32_t at = 2u * (h * p.head_dim + at0), at_out = at;
    const uint32_t apart_by = 2u * (at1 - at0);
    const uint16_t *weight = of_q ? p.q_weight : p.k_weight;
    uint64_t w[4] = {};
    if (NORM && weight && live) {
      const uint2 lo = *reinterpret_cast<const uint2 *>(weight + at0), hi = *reinterpret_cast<const uint2 *>(weight + at1);
      w[0] = unpack2<DT>(lo.x), w[1] = unpack2<DT>(lo.y), w[2] = unpack2<DT>(hi.x), w[3] = unpack2<DT>(hi.y);
    }
    const float *cs = cosines + 4 * lane, *sn = sines + 4 * lane;
    for (int r = 0; r < rows; r += kBatch) {
      uint2 lo[kBatch], hi[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        lo[i] = hi[i] = make_uint2(0, 0);
        if (live && r + i < rows) {
          lo[i] = *reinterpret_cast<const uint2 *>(x + at);
          hi[i] = *reinterpret_cast<const uint2 *>(x + at + apart_by);
        }
        at += hop;
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (r + i >= rows) break;
        uint64_t v[4] = {unpack2<DT>(lo[i].x), unpack2<DT>(lo[i].y), unpack2<DT>(hi[i].x), unpack2<DT>(hi[i].y)};
        if (NORM && weight) {
          const float2 sums = unpair(fma2(v[3], v[3], fma2(v[2], v[2], fma2(v[1], v[1], mul2(v[0], v[0])))));
          float sum = sums.x + sums.y;
#pragma unroll
          for (int e = LG / 2; e > 0; e /= 2) sum += __shfl_xor_sync(kAll, sum, e, LG);
          const float scale = rsqrtf(fmaf(sum, inv_dim, p.eps));
          const uint64_t scale2 = pair(scale, scale);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = mul2(mul2(v[e], scale2), w[e]);
        }
        if (turned) {
          const ulonglong2 c = *reinterpret_cast<const ulonglong2 *>(cs), s = *reinterpret_cast<const ulonglong2 *>(sn);
          if (PAIRED) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 ab = unpair(v[e]), cc = unpair(e < 2 ? c.x : c.y), ss = unpair(e < 2 ? s.x : s.y);
              const float ce = e % 2 ? cc.y : cc.x, se = e % 2 ? ss.y : ss.x;
              v[e] = pair(ab.x * ce - ab.y * se, fmaf(ab.y, ce, ab.x * se));
            }
          } else {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint64_t a = v[e], b = v[2 + e], ce = e ? c.y : c.x, se = e ? s.y : s.x;
              v[e] = sub2(mul2(a, ce), mul2(b, se));
              v[2 + e] = fma2(b, ce, mul2(a, se));
            }
          }
        }
        cs += p.half, sn += p.half;
        if (live) {
          *reinterpret_cast<uint2 *>(y + at_out) = make_uint2(pack2<DT>(v[0]), pack2<DT>(v[1]));
          *reinterpret_cast<uint2 *>(y + at_out + apart_by) = make_uint2(pack2<DT>(v[2]), pack2<DT>(v[3]));
        }
        at_out += hop_out;
      }
    }
  }
}

template <int DT>
cudaError_t launch_dim(RopeParams p, int num_sms, cudaStream_t stream) {
  int lg = 1;
  while (8 * lg < p.head_dim) lg *= 2;
  p.head_step = kRopeThreads / lg;
  const int q_turns = static_cast<int>(cdiv(p.q_heads, p.head_step)), turns = q_turns + static_cast<int>(cdiv(p.heads - p.q_heads, p.head_step));
  p.q_turned = q_turns * p.head_step;
  // few rows: a row's heads go to blocks of their own; many: a block takes a few rows (whose offsets fit 32 bits)
  p.head_parts = 1;
  while (p.head_parts < turns && p.T * p.head_parts < 4 * num_sms) p.head_parts *= 2;
  const int64_t widest = std::max(std::max(p.ldq, p.ldqo), std::max(p.ldk, p.ldko));
  p.rows = 1;
  while (p.rows < 8 && p.T > static_cast<int64_t>(16) * num_sms * p.rows && 4 * p.rows * widest < (int64_t{1} << 30)) p.rows *= 2;
  const int64_t blocks = cdiv(p.T, p.rows) * p.head_parts;
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
  const bool norm = p.q_weight || p.k_weight;
  const int smem = p.half * (p.rows * 2 * static_cast<int>(sizeof(float)) + static_cast<int>(sizeof(uint64_t)));
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
