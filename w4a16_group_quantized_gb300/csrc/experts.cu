// w4a16_experts: y[t] = sum_j weights[t, j] * down_e (silu(gate_e x_t) * up_e x_t), e = ids[t, j], with each expert's
// weights in 4-bit groups, w = (q - z) s.
//
// The pairs (token, choice) are sorted by expert (rows.cu) and cut into tiles of one expert; a first product makes
// h = silu(gate) * up of each pair, rounded once to the 16-bit type (the second product's operand), a second one the
// expert's output in 32 bits, and a last pass adds a token's outputs with their weights, in the order of its choices.
//
// The products here run on register-operand tensor-core instructions, for few rows per expert: the weights of the
// chosen experts are read once and that bounds them. Codes go from global memory straight to the registers that the
// products read (8 bytes a lane: the tile layout deals a lane 16 consecutive codes of a row), with no barrier between
// the loads; a block's warps split K, so that a slab of 32 weight rows starts all its loads at once, and add their
// sums in shared memory in a fixed order.
//
// Codes become operands without arithmetic: a code's four bits under the exponent of 16 are 16 + q in either type.
// A product with ones gives X = sum x over the same k, and (q - z) x sums to sum (16 + q) x - (16 + z) X, exactly in
// the operands and in 32 bits in the sums; a group's sum is multiplied by its 32-bit s. So no weight is rounded.
#include "experts.cuh"
#include "gemm_common.cuh"
#include "internal.h"
#include "mma.cuh"
#include "ptx.cuh"

namespace w4 {
namespace {

using namespace detail;

constexpr int kWarps = 8;      // they split K
constexpr int kSlabRows = 32;  // weight rows of a block
constexpr int kTmemRows = 12;  // rows an expert has on average from which the tensor-memory kernel runs

// Eight codes -> four pairs (k, k + 1) of 16 + q: each code's bits moved to the top of the fraction that 16 leaves
// (fp16: a step of 2^-6 at 16, bits 6 to 9; bf16: 2^-3, bits 3 to 6).
template <int DT>
__device__ __forceinline__ void operands(uint32_t w, uint32_t *o) {
  if (DT == kDtypeBf16) {
    o[0] = lop3_and_or(w << 3, 0x00780078u, 0x41804180u);
    o[1] = lop3_and_or(w >> 1, 0x00780078u, 0x41804180u);
    o[2] = lop3_and_or(w >> 5, 0x00780078u, 0x41804180u);
    o[3] = lop3_and_or(w >> 9, 0x00780078u, 0x41804180u);
  } else {
    o[0] = lop3_and_or(w << 6, 0x03C003C0u, 0x4C004C00u);
    o[1] = lop3_and_or(w << 2, 0x03C003C0u, 0x4C004C00u);
    o[2] = lop3_and_or(w >> 2, 0x03C003C0u, 0x4C004C00u);
    o[3] = lop3_and_or(w >> 6, 0x03C003C0u, 0x4C004C00u);
  }
}

// A block: 32 weight rows of one expert x one tile of up to 8 NT rows of `in`. GATED: rows 2 j and 2 j + 1 are gate
// and up j. WHOLE: g is a multiple of 64, so that a block of 64 k lies in one group; else a k block's groups take
// turns, each with the other groups' x as zeros.
template <int DT, int NT, bool GATED, bool WHOLE>
__global__ void __launch_bounds__(32 * kWarps, NT == 1 ? 2 : 1) experts_kernel(const Products p) {
  griddep_launch_dependents();
  griddep_wait();
  const int tile = blockIdx.x / p.slabs;
  const int n0 = (blockIdx.x - tile * p.slabs) * kSlabRows;
  if (tile >= *p.plan.ntiles) return;
  const RowTile rt = p.plan.tiles[tile];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;

  const uint16_t *xr[NT];
  bool has[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    has[n] = n * 8 + g < rt.rows;
    const int pos = rt.row0 + n * 8 + g;
    const int64_t row = !has[n] ? 0 : GATED ? p.plan.perm[pos] / p.choices : pos;
    xr[n] = p.in + row * p.K + 16 * t;
  }
  const uint8_t *expert = p.codes + rt.key * p.expert_bytes;
  const int wt = n0 / kTN, r0 = n0 % kTN;
  // lane t's 16 codes of row r in a 4 KB tile: k = 16 t ..: half t / 2, bytes 8 (t % 2) of the row's 16
  const uint8_t *codes =
      expert + static_cast<int64_t>(wt) * p.KB * kTileBytes + (t >> 1) * 2048 + (r0 + g) * 16 + 8 * (t & 1);
  const uint8_t *meta = expert + p.meta + static_cast<int64_t>(wt) * p.G * kRecBytes;

  const int kb0 = p.KB * warp / kWarps, kb1 = p.KB * (warp + 1) / kWarps;
  constexpr uint32_t kOne = DT == kDtypeBf16 ? 0x3F803F80u : 0x3C003C00u;
  float sum[2][NT][4] = {};  // rows g, g + 8 (and 16, 24): what is done
  constexpr int U = NT == 1 ? 4 : 2;
  for (int kb = kb0; kb < kb1; kb += U) {
    uint2 c[U][4];
    uint4 x[U][NT][2];
    uint32_t rec[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = kb + u < kb1;
      const uint8_t *cb = codes + static_cast<int64_t>(kb + u) * kTileBytes;
#pragma unroll
      for (int i = 0; i < 4; ++i) c[u][i] = in ? __ldg(reinterpret_cast<const uint2 *>(cb + i * 128)) : make_uint2(0u, 0u);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int k = (kb + u) * kTK + 8 * i;  // K is a multiple of 8
          x[u][n][i] = in && has[n] && k + 16 * t < p.K ? __ldg(reinterpret_cast<const uint4 *>(xr[n] + k))
                                                         : make_uint4(0u, 0u, 0u, 0u);
        }
      if (WHOLE) {  // lane l: row l's scale, and its zero in the upper half
        const uint8_t *m = meta + static_cast<int64_t>(p.gdiv.div((kb + u) * kTK)) * kRecBytes;
        rec[u] = in ? *reinterpret_cast<const uint16_t *>(m + 2 * (r0 + lane)) |
                          static_cast<uint32_t>((m[256 + (r0 + lane) / 2] >> (4 * (lane & 1))) & 15) << 16
                    : 0u;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (kb + u >= kb1) break;
      uint32_t a[4][8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        operands<DT>(c[u][i].x, a[i]);
        operands<DT>(c[u][i].y, a[i] + 4);
      }
      const int k0 = (kb + u) * kTK;
      const int j0 = WHOLE ? 0 : p.gdiv.div(k0), j1 = WHOLE ? 0 : p.gdiv.div(min(k0 + kTK, p.K) - 1);
      for (int j = j0; j <= j1; ++j) {
        uint32_t r = WHOLE ? rec[u] : 0u;
        bool first = true, second = true;  // whether the lane's two words of codes lie in group j
        if (!WHOLE) {
          const uint8_t *m = meta + static_cast<int64_t>(j) * kRecBytes;
          r = *reinterpret_cast<const uint16_t *>(m + 2 * (r0 + lane)) |
              static_cast<uint32_t>((m[256 + (r0 + lane) / 2] >> (4 * (lane & 1))) & 15) << 16;
          first = p.gdiv.div(k0 + 16 * t) == j;
          second = p.gdiv.div(k0 + 16 * t + 8) == j;
        }
        float s[4], zb[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t v = __shfl_sync(0xffffffffu, r, i * 8 + g);
          s[i] = scale_f32<DT>(v & 0xffffu);
          zb[i] = static_cast<float>(16 + static_cast<int>(v >> 16));
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          uint32_t b[8] = {x[u][n][0].x, x[u][n][0].y, x[u][n][0].z, x[u][n][0].w,
                           x[u][n][1].x, x[u][n][1].y, x[u][n][1].z, x[u][n][1].w};
          if (!WHOLE) {
#pragma unroll
            for (int i = 0; i < 8; ++i) b[i] = (i < 4 ? first : second) ? b[i] : 0u;
          }
          float d0[4] = {}, d1[4] = {}, ones[4] = {};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            mma_16816<DT>(d0, a[0][2 * q], a[1][2 * q], a[0][2 * q + 1], a[1][2 * q + 1], b[2 * q], b[2 * q + 1]);
            mma_16816<DT>(d1, a[2][2 * q], a[3][2 * q], a[2][2 * q + 1], a[3][2 * q + 1], b[2 * q], b[2 * q + 1]);
            mma_16816<DT>(ones, kOne, kOne, kOne, kOne, b[2 * q], b[2 * q + 1]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {  // i / 2: row g or g + 8; i % 2: column 2 t + i % 2
            sum[0][n][i] += s[i / 2] * (d0[i] - zb[i / 2] * ones[i]);
            sum[1][n][i] += s[2 + i / 2] * (d1[i] - zb[2 + i / 2] * ones[i]);
          }
        }
      }
    }
  }

  // [warp][column][row], a column's rows one bank off the next column's
  constexpr int kLd = kSlabRows + 4;
  __shared__ float red[kWarps][8 * NT][kLd];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[warp][n * 8 + 2 * t + (i & 1)][m * 16 + (i >> 1) * 8 + g] = sum[m][n][i];
  __syncthreads();
  if (GATED) {
    for (int i = threadIdx.x; i < 8 * NT * 16; i += 32 * kWarps) {
      const int col = i / 16, j = i % 16;
      if (col >= rt.rows || n0 + 2 * j >= p.N) continue;
      float gate = 0.0f, up = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        gate += red[w][col][2 * j];
        up += red[w][col][2 * j + 1];
      }
      static_cast<uint16_t *>(p.out)[static_cast<int64_t>(rt.row0 + col) * (p.N / 2) + n0 / 2 + j] =
          out_bits<DT>(silu_mul(gate, up));
    }
  } else {
    for (int i = threadIdx.x; i < 8 * NT * 32; i += 32 * kWarps) {
      const int col = i / 32, r = i % 32;
      if (col >= rt.rows || n0 + r >= p.N) continue;
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += red[w][col][r];
      static_cast<float *>(p.out)[static_cast<int64_t>(rt.row0 + col) * p.N + n0 + r] = v;
    }
  }
}

// y[t] = sum over the token's choices of weight * output, in their order; a dropped choice adds nothing.
template <int DT>
__global__ void __launch_bounds__(256)
    combine_kernel(const float *__restrict__ part, const int32_t *__restrict__ inverse, const float *__restrict__ weights,
                   int64_t T, int K, int choices, uint16_t *__restrict__ y) {
  griddep_launch_dependents();
  griddep_wait();
  const int per_row = K / 8;  // K is a multiple of 8
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= T * per_row) return;
  const int64_t t = i / per_row;
  const int c = static_cast<int>(i - t * per_row) * 8;
  float s[8] = {};
  for (int j = 0; j < choices; ++j) {
    const int pos = inverse[t * choices + j];
    if (pos < 0) continue;
    const float w = weights[t * choices + j];
    const float4 a = __ldg(reinterpret_cast<const float4 *>(part + static_cast<int64_t>(pos) * K + c));
    const float4 b = __ldg(reinterpret_cast<const float4 *>(part + static_cast<int64_t>(pos) * K + c + 4));
    s[0] += w * a.x;
    s[1] += w * a.y;
    s[2] += w * a.z;
    s[3] += w * a.w;
    s[4] += w * b.x;
    s[5] += w * b.y;
    s[6] += w * b.z;
    s[7] += w * b.w;
  }
  *reinterpret_cast<uint4 *>(y + t * K + c) = make_uint4(out_bits2<DT>(s[0], s[1]), out_bits2<DT>(s[2], s[3]),
                                                         out_bits2<DT>(s[4], s[5]), out_bits2<DT>(s[6], s[7]));
}

// The workspace: [error word][ntiles][outputs in 32 bits][h][perm][inverse][tiles].
struct ExpertsPlan {
  bool tmem;
  int tile, max_tiles;
  size_t part, h, perm, inverse, tiles, bytes;
};

ExpertsPlan experts_plan(int64_t T, int64_t K, int64_t I, int experts, int k, int g) {
  ExpertsPlan p;
  const int64_t pairs = T * k;
  // rows per tile: as many as an expert has on average, from the widths that the kernels have
  const int64_t mean = pairs / experts;
  p.tmem = mean >= kTmemRows && experts_tmem_takes(g);
  p.tile = p.tmem ? (mean <= 48 || g % 64 != 0 ? 64 : 128) : mean <= 8 ? 8 : mean <= 16 ? 16 : 32;
  p.max_tiles = static_cast<int>(max_row_tiles(pairs, experts, p.tile));
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  p.part = 256;
  p.h = p.part + up(static_cast<size_t>(pairs) * K * 4);
  p.perm = p.h + up(static_cast<size_t>(pairs) * I * 2);
  p.inverse = p.perm + up(static_cast<size_t>(pairs) * 4);
  p.tiles = p.inverse + up(static_cast<size_t>(pairs) * 4);
  p.bytes = p.tiles + up(static_cast<size_t>(p.max_tiles) * sizeof(RowTile));
  return p;
}

template <int DT, bool GATED>
cudaError_t launch_products(const Products &p, const ExpertsPlan &plan, int num_sms, cudaStream_t stream) {
  if (plan.tmem) return launch_experts_tmem(p, DT, GATED, plan.tile, num_sms, stream);
  const bool whole = p.g % kTK == 0;
  auto kern = plan.tile == 8    ? (whole ? experts_kernel<DT, 1, GATED, true> : experts_kernel<DT, 1, GATED, false>)
              : plan.tile == 16 ? (whole ? experts_kernel<DT, 2, GATED, true> : experts_kernel<DT, 2, GATED, false>)
                                : (whole ? experts_kernel<DT, 4, GATED, true> : experts_kernel<DT, 4, GATED, false>);
  return launch_programmatic(kern, p.slabs * plan.max_tiles, 32 * kWarps, 0, stream, p);
}

template <int DT>
cudaError_t launch_dt(const ExpertsArgs &a, uint8_t *ws, const ExpertsPlan &plan, int num_sms, cudaStream_t stream) {
  RowPlan rows;
  rows.perm = reinterpret_cast<int32_t *>(ws + plan.perm);
  rows.inverse = reinterpret_cast<int32_t *>(ws + plan.inverse);
  rows.tiles = reinterpret_cast<RowTile *>(ws + plan.tiles);
  rows.ntiles = reinterpret_cast<int32_t *>(ws + 4);
  rows.err = reinterpret_cast<uint32_t *>(ws);
  cudaError_t e = launch_row_plan(a.ids, a.T * a.k, a.experts, plan.tile, false, rows, stream);
  if (e != cudaSuccess) return e;
  auto products = [&](const void *in, int64_t in_rows, const void *packed, int64_t N, int64_t K, void *out) {
    Products p;
    p.in_rows = in_rows;
    p.in = static_cast<const uint16_t *>(in);
    p.codes = static_cast<const uint8_t *>(packed);
    p.K = static_cast<int>(K);
    p.N = static_cast<int>(N);
    p.G = static_cast<int>(cdiv(K, a.g));
    p.KB = static_cast<int>(cdiv(K, kTK));
    p.g = a.g;
    p.meta = cdiv(N, kTN) * p.KB * kTileBytes;
    p.expert_bytes = p.meta + cdiv(N, kTN) * p.G * kRecBytes;
    p.out = out;
    p.plan = rows;
    p.err = rows.err;
    p.slabs = static_cast<int>(cdiv(N, plan.tmem ? kTN : kSlabRows));
    p.choices = a.k;
    p.gdiv = make_fastdiv(static_cast<uint32_t>(a.g));
    return p;
  };
  e = launch_products<DT, true>(products(a.x, a.T, a.gate_up, 2 * a.I, a.K, ws + plan.h), plan, num_sms, stream);
  if (e != cudaSuccess) return e;
  e = launch_products<DT, false>(products(ws + plan.h, a.T * a.k, a.down, a.K, a.I, ws + plan.part), plan, num_sms, stream);
  if (e != cudaSuccess) return e;
  return launch_programmatic(combine_kernel<DT>, static_cast<int>(cdiv(a.T * (a.K / 8), 256)), 256, 0, stream,
                             reinterpret_cast<const float *>(ws + plan.part), static_cast<const int32_t *>(rows.inverse), a.weights,
                             a.T, static_cast<int>(a.K), a.k, static_cast<uint16_t *>(a.y));
}

}  // namespace

size_t experts_workspace_bytes(int64_t T, int64_t K, int64_t I, int experts, int k, int g, int num_sms) {
  (void)num_sms;
  return experts_plan(T, K, I, experts, k, g).bytes;
}

cudaError_t launch_experts(const ExpertsArgs &a, void *workspace, int num_sms, cudaStream_t stream) {
  const ExpertsPlan plan = experts_plan(a.T, a.K, a.I, a.experts, a.k, a.g);
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  return a.dtype == kDtypeBf16 ? launch_dt<kDtypeBf16>(a, ws, plan, num_sms, stream)
                               : launch_dt<kDtypeF16>(a, ws, plan, num_sms, stream);
}

}  // namespace w4
