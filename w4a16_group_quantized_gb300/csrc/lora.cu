// w4_lora_add: y = base + scaling[a] * B[a] . (A[a] . x) for each row x with its own adapter a, beside a projection that
// all rows share.
//
// Two kernels, v = A x and y = base + scaling B v, with v in 32 bits between them. A row's 2 r (K + N) products go with
// its 2 K + 4 N bytes of x, base and y, and an adapter's 2 r (K + N) bytes of weights with all its rows: at ranks up to
// 64 every case is bound by memory, or, for a few rows, by the latency of its launches. So operands go from global
// memory straight to the registers of the tensor-core products, 16 bytes a lane: a lane's k are consecutive (mma.cuh),
// and for the outputs' sake so are the four pairs of columns n that a lane holds of four products.
//
// Rows stand by adapter (rows.cu), cut into tiles of up to 32; up to kDirectRows rows go without a sort, one row to a
// tile (rows of one adapter then read its weights again, from L2).
//
// v stands in the second product as the sum of two 16-bit values, its rounding and what that left, which keeps about
// twice the type's bits for one more product each (they are not what bounds the kernel). For fp16 a row of v is first
// divided by a power of two, so that no v overflows the type.
#include "gemm_common.cuh"
#include "internal.h"
#include "mma.cuh"
#include "ptx.cuh"

namespace w4 {
namespace {

using namespace detail;

constexpr int kWarps = 8;
constexpr int kDirectRows = 32;

struct Tiles {
  RowPlan plan;
  const int32_t *adapter;  // direct: row i is tile i
  int direct;
  int T;
};

// The block's tile: its adapter (-1: none) and rows; false past the last.
__device__ __forceinline__ bool get_tile(const Tiles &ts, int i, int adapters, int *key, int *row0, int *rows) {
  if (ts.direct) {
    const int k = ts.adapter[i];
    *key = k >= 0 && k < adapters ? k : -1;
    *row0 = i;
    *rows = 1;
    return true;
  }
  if (i >= *ts.plan.ntiles) return false;
  const RowTile t = ts.plan.tiles[i];
  *key = t.key < adapters ? t.key : -1;
  *row0 = t.row0;
  *rows = t.rows;
  return true;
}

__device__ __forceinline__ int64_t row_at(const Tiles &ts, int pos) { return ts.direct ? pos : ts.plan.perm[pos]; }

__device__ __forceinline__ uint4 ldg16(const uint16_t *p) { return __ldg(reinterpret_cast<const uint4 *>(p)); }

// v[split][position][rank] = A[a] . x over the split's part of K. A block holds a tile of 16 MT rows and NB * 8 ranks;
// its warps take 32 U of K in turn and add their sums in shared memory, in a fixed order.
template <int DT, int MT, int NB, int U>
__global__ void __launch_bounds__(32 * kWarps)
    lora_shrink_kernel(const Tiles ts, const LoraArgs a, float *__restrict__ v) {
  griddep_launch_dependents();
  griddep_wait();
  int key, row0, rows;
  if (!get_tile(ts, blockIdx.x, a.adapters, &key, &row0, &rows) || key < 0) return;
  const int rank = a.ranks ? min(max(a.ranks[key], 0), a.rank) : a.rank;
  const int r0 = blockIdx.z * NB * 8;
  if (r0 >= rank) return;  // (the second kernel reads no v at or past the adapter's rank)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int K = static_cast<int>(a.K);

  const uint16_t *xr[2 * MT];
  bool has[2 * MT];
#pragma unroll
  for (int m = 0; m < 2 * MT; ++m) {
    has[m] = m * 8 + g < rows;
    xr[m] = static_cast<const uint16_t *>(a.x) + (has[m] ? row_at(ts, row0 + m * 8 + g) * a.ldx : 0);
  }
  const uint16_t *ar = static_cast<const uint16_t *>(a.A) + (static_cast<int64_t>(key) * a.rank + r0 + g) * K;
  bool live[NB];
#pragma unroll
  for (int n = 0; n < NB; ++n) live[n] = r0 + n * 8 + g < rank;

  float acc[MT][NB][4] = {};
  const int chunk = 32 * U;
  const int step = chunk * kWarps * gridDim.y;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (int k0 = (blockIdx.y * kWarps + warp) * chunk; k0 < K; k0 += step) {
    uint4 xa[U][2 * MT], wb[U][NB];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * 32 + t * 8;  // K is a multiple of 8: eight values lie inside or outside together
      const bool in = k < K;
#pragma unroll
      for (int m = 0; m < 2 * MT; ++m) xa[u][m] = in && has[m] ? ldg16(xr[m] + k) : zero;
#pragma unroll
      for (int n = 0; n < NB; ++n) wb[u][n] = in && live[n] ? ldg16(ar + static_cast<int64_t>(n) * 8 * K + k) : zero;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          mma_16816<DT>(acc[m][n], xa[u][2 * m].x, xa[u][2 * m + 1].x, xa[u][2 * m].y, xa[u][2 * m + 1].y, wb[u][n].x,
                        wb[u][n].y);
          mma_16816<DT>(acc[m][n], xa[u][2 * m].z, xa[u][2 * m + 1].z, xa[u][2 * m].w, xa[u][2 * m + 1].w, wb[u][n].z,
                        wb[u][n].w);
        }
  }

  // the upper half of the warps gives its sums to the lower half until one warp has them all
  __shared__ float red[kWarps / 2][MT * NB * 4][32];
#pragma unroll
  for (int half = kWarps / 2; half > 0; half >>= 1) {
    if (warp >= half && warp < 2 * half) {
#pragma unroll
      for (int i = 0; i < MT * NB * 4; ++i) red[warp - half][i][lane] = acc[i / (NB * 4)][i / 4 % NB][i % 4];
    }
    __syncthreads();
    if (warp < half) {
#pragma unroll
      for (int i = 0; i < MT * NB * 4; ++i) acc[i / (NB * 4)][i / 4 % NB][i % 4] += red[warp][i][lane];
    }
    __syncthreads();
  }
  if (warp != 0) return;
  float *vs = v + static_cast<int64_t>(blockIdx.y) * ts.T * a.rank;
#pragma unroll
  for (int m = 0; m < 2 * MT; ++m) {
    if (!has[m]) continue;
    float *row = vs + static_cast<int64_t>(row0 + m * 8 + g) * a.rank + r0 + 2 * t;
#pragma unroll
    for (int n = 0; n < NB; ++n)
      if (r0 + n * 8 < a.rank)
        *reinterpret_cast<float2 *>(row + n * 8) = make_float2(acc[m / 2][n][2 * (m & 1)], acc[m / 2][n][2 * (m & 1) + 1]);
  }
}

// Two values as the type's nearest (hi) and what that leaves (lo), each as a pair of 16-bit values. What an infinity
// leaves is nothing (not the NaN of its difference to itself).
template <int DT>
__device__ __forceinline__ void split_pair(float p, float q, uint32_t *hi, uint32_t *lo) {
  *hi = out_bits2<DT>(p, q);
  const float ph = value_f32<DT>(*hi & 0xffffu), qh = value_f32<DT>(*hi >> 16);
  *lo = out_bits2<DT>(isinf(ph) ? 0.0f : p - ph, isinf(qh) ? 0.0f : q - qh);
}

// Four values of B's row from rank place k on, as pairs; what lies at or past the adapter's rank is zero and not read.
__device__ __forceinline__ uint2 load_b4(const uint16_t *row, int k, int rank) {
  if (k + 4 <= rank) return __ldg(reinterpret_cast<const uint2 *>(row + k));
  uint32_t e[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) e[i] = k + i < rank ? row[k + i] : 0u;
  return make_uint2(e[0] | e[1] << 16, e[2] | e[3] << 16);
}

// y = base + scaling * B[a] . v for a tile of 16 MT rows. A warp takes 32 columns of y at a time: four products whose
// columns are dealt so that lane t holds the eight from 8 t on.
template <int DT, int MT, int KB>
__global__ void __launch_bounds__(32 * kWarps)
    lora_expand_kernel(const Tiles ts, const LoraArgs a, const float *__restrict__ v, int splits, int vec) {
  griddep_launch_dependents();
  griddep_wait();
  int key, row0, rows;
  if (!get_tile(ts, blockIdx.x, a.adapters, &key, &row0, &rows)) return;
  if (key < 0 && a.base == a.y) return;  // rows without an adapter, in place
  const int rank = key < 0 ? 0 : a.ranks ? min(max(a.ranks[key], 0), a.rank) : a.rank;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int N = static_cast<int>(a.N);
  const float scale = key >= 0 && a.scaling ? a.scaling[key] : 1.0f;

  int64_t yr[2 * MT], br[2 * MT];  // the rows' first values in y and base
  bool has[2 * MT];
  float mul[2 * MT];
  uint32_t hi[MT][KB][4], lo[MT][KB][4];
#pragma unroll
  for (int m = 0; m < 2 * MT; ++m) {
    has[m] = m * 8 + g < rows;
    const int64_t row = has[m] ? row_at(ts, row0 + m * 8 + g) : 0;
    yr[m] = row * a.ldy;
    br[m] = row * a.ldbase;
    float4 p[KB];
    float top = 0.0f;
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      p[b] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      const int k = b * 16 + t * 4;
      if (has[m] && k < rank) {
        for (int s = 0; s < splits; ++s) {
          const float4 q = __ldg(reinterpret_cast<const float4 *>(
              v + (static_cast<int64_t>(s) * ts.T + row0 + m * 8 + g) * a.rank + k));
          p[b].x += q.x;
          p[b].y += q.y;
          p[b].z += q.z;
          p[b].w += q.w;
        }
        // v past the adapter's rank is zero, whatever stands there
        if (k + 1 >= rank) p[b].y = 0.0f;
        if (k + 2 >= rank) p[b].z = 0.0f;
        if (k + 3 >= rank) p[b].w = 0.0f;
      }
      top = fmaxf(top, fmaxf(fmaxf(fabsf(p[b].x), fabsf(p[b].y)), fmaxf(fabsf(p[b].z), fabsf(p[b].w))));
    }
    mul[m] = scale;
    float down = 1.0f;
    if (DT == kDtypeF16) {
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // 2^e <= top < 2^(e + 1), e kept where 2^e and 2^-e are normal: the row divided by 2^e has its largest in [1, 2)
      const int e = min(max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -100), 100);
      if (top > 0.0f && top < INFINITY) {
        down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        mul[m] = scale * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
      }
    }
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      split_pair<DT>(p[b].x * down, p[b].y * down, &hi[m / 2][b][m & 1], &lo[m / 2][b][m & 1]);
      split_pair<DT>(p[b].z * down, p[b].w * down, &hi[m / 2][b][2 + (m & 1)], &lo[m / 2][b][2 + (m & 1)]);
    }
  }

  const uint16_t *B = static_cast<const uint16_t *>(a.B) + static_cast<int64_t>(max(key, 0)) * N * a.rank;
  const uint16_t *base = static_cast<const uint16_t *>(a.base);
  uint16_t *y = static_cast<uint16_t *>(a.y);
  for (int n0 = (blockIdx.y * kWarps + warp) * 32; n0 < N; n0 += gridDim.y * kWarps * 32) {
    uint2 w[4][KB];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + 8 * (g >> 1) + 2 * j + (g & 1);  // product j's column g
#pragma unroll
      for (int b = 0; b < KB; ++b) {
        const int k = b * 16 + t * 4;
        w[j][b] = n < N && k < rank ? load_b4(B + static_cast<int64_t>(n) * a.rank, k, rank) : make_uint2(0u, 0u);
      }
    }
    const int n = n0 + 8 * t;
    const bool wide = vec && n + 8 <= N;
    uint4 old[2 * MT];
#pragma unroll
    for (int m = 0; m < 2 * MT; ++m) {
      old[m] = make_uint4(0u, 0u, 0u, 0u);
      if (!base || !has[m] || n >= N) continue;
      if (wide) {
        old[m] = *reinterpret_cast<const uint4 *>(base + br[m] + n);
      } else {
        uint32_t e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = n + i < N ? base[br[m] + n + i] : 0u;
        old[m] = make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
      }
    }
    float acc[MT][4][4] = {};
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int b = 0; b < KB; ++b) {
          mma_16816<DT>(acc[m][j], lo[m][b][0], lo[m][b][1], lo[m][b][2], lo[m][b][3], w[j][b].x, w[j][b].y);
          mma_16816<DT>(acc[m][j], hi[m][b][0], hi[m][b][1], hi[m][b][2], hi[m][b][3], w[j][b].x, w[j][b].y);
        }
#pragma unroll
    for (int m = 0; m < 2 * MT; ++m) {
      if (!has[m] || n >= N) continue;
      uint32_t out[4] = {old[m].x, old[m].y, old[m].z, old[m].w};
      if (key >= 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          out[j] = out_bits2<DT>(value_f32<DT>(out[j] & 0xffffu) + mul[m] * acc[m / 2][j][2 * (m & 1)],
                                 value_f32<DT>(out[j] >> 16) + mul[m] * acc[m / 2][j][2 * (m & 1) + 1]);
      }
      if (wide) {
        *reinterpret_cast<uint4 *>(y + yr[m] + n) = make_uint4(out[0], out[1], out[2], out[3]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (n + i < N) y[yr[m] + n + i] = static_cast<uint16_t>(out[i / 2] >> (16 * (i & 1)));
      }
    }
  }
}

// The launch's shape, and the workspace's: [v][perm][tiles][ntiles].
struct LoraPlan {
  bool direct;
  int tile, max_tiles, splits;
  size_t perm, tiles, ntiles, bytes;
};

LoraPlan lora_plan(int64_t T, int64_t N, int64_t K, int adapters, int rank, int num_sms) {
  LoraPlan p;
  p.direct = T <= kDirectRows;
  p.tile = rank > 64 ? 16 : 32;
  p.max_tiles = static_cast<int>(p.direct ? T : max_row_tiles(T, adapters, p.tile));
  // few tiles: the blocks of one tile split K, no finer than one turn of a block's warps (32 K values each)
  const int64_t turns = cdiv(K, 32 * kWarps);
  const int64_t want = cdiv(2 * num_sms, p.max_tiles < 1 ? 1 : p.max_tiles);
  p.splits = static_cast<int>(want < turns ? (want < 8 ? want : 8) : (turns < 8 ? turns : 8));
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  p.perm = up(static_cast<size_t>(p.splits) * T * rank * 4);
  p.tiles = p.perm + (p.direct ? 0 : up(static_cast<size_t>(T) * 4));
  p.ntiles = p.tiles + (p.direct ? 0 : up(static_cast<size_t>(p.max_tiles) * sizeof(RowTile)));
  p.bytes = p.ntiles + 256;
  return p;
}

template <int DT, int MT>
cudaError_t launch_mt(const Tiles &ts, const LoraArgs &a, const LoraPlan &p, float *v, int num_sms, cudaStream_t stream) {
  auto shrink = a.rank <= 8    ? lora_shrink_kernel<DT, MT, 1, 4>
                : a.rank <= 16 ? lora_shrink_kernel<DT, MT, 2, 4>
                : a.rank <= 32 ? lora_shrink_kernel<DT, MT, 4, 2>
                               : lora_shrink_kernel<DT, MT, 8, 1>;
  const int vec = a.ldy % 8 == 0 && reinterpret_cast<uintptr_t>(a.y) % 16 == 0 &&
                  (!a.base || (a.ldbase % 8 == 0 && reinterpret_cast<uintptr_t>(a.base) % 16 == 0));
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = stream;
  cfg.blockDim = dim3(32 * kWarps);
  cfg.gridDim = dim3(p.max_tiles, p.splits, a.rank > 64 ? 2 : 1);
  cudaError_t e = cudaLaunchKernelEx(&cfg, shrink, ts, a, v);
  if (e != cudaSuccess) return e;
  // columns: enough blocks for the device, no more than one turn of a block's warps each
  const int64_t turns = cdiv(a.N, 32 * kWarps);
  const int64_t want = cdiv(4 * num_sms, p.max_tiles);
  cfg.gridDim = dim3(p.max_tiles, static_cast<unsigned>(turns < want ? turns : want), 1);
  auto expand = a.rank <= 16   ? lora_expand_kernel<DT, MT, 1>
                : a.rank <= 32 ? lora_expand_kernel<DT, MT, 2>
                : a.rank <= 64 ? lora_expand_kernel<DT, MT, 4>
                               : lora_expand_kernel<DT, 1, 8>;
  e = cudaLaunchKernelEx(&cfg, expand, ts, a, static_cast<const float *>(v), p.splits, vec);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace

size_t lora_workspace_bytes(int64_t T, int64_t N, int64_t K, int adapters, int rank, int num_sms) {
  return lora_plan(T, N, K, adapters, rank, num_sms).bytes;
}

cudaError_t launch_lora(const LoraArgs &a, void *workspace, int num_sms, cudaStream_t stream) {
  const LoraPlan p = lora_plan(a.T, a.N, a.K, a.adapters, a.rank, num_sms);
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  Tiles ts = {};
  ts.adapter = a.adapter;
  ts.direct = p.direct;
  ts.T = static_cast<int>(a.T);
  if (!p.direct) {
    ts.plan.perm = reinterpret_cast<int32_t *>(ws + p.perm);
    ts.plan.tiles = reinterpret_cast<RowTile *>(ws + p.tiles);
    ts.plan.ntiles = reinterpret_cast<int32_t *>(ws + p.ntiles);
    const cudaError_t e = launch_row_plan(a.adapter, a.T, a.adapters, p.tile, true, ts.plan, stream);
    if (e != cudaSuccess) return e;
  }
  float *v = reinterpret_cast<float *>(ws);
  const bool small = p.direct || p.tile == 16;
  if (a.dtype == kDtypeBf16)
    return small ? launch_mt<kDtypeBf16, 1>(ts, a, p, v, num_sms, stream)
                 : launch_mt<kDtypeBf16, 2>(ts, a, p, v, num_sms, stream);
  return small ? launch_mt<kDtypeF16, 1>(ts, a, p, v, num_sms, stream)
               : launch_mt<kDtypeF16, 2>(ts, a, p, v, num_sms, stream);
}

}  // namespace w4
