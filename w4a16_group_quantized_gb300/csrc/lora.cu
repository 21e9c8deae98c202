// w4_lora_add: y = base + scaling[a] * B[a] . (A[a] . x) for each row x with its own adapter a, beside a projection that
// all rows share.
//
// Two kernels, v = A x and y = base + scaling B v, with v in 32 bits between them. A row's 2 r (K + N) products go with
// its 2 K + 4 N bytes of x, base and y, and an adapter's 2 r (K + N) bytes of weights with all its rows: at ranks up to
// 64 memory is the floor of every case. What bounds them is, for a few rows, the latency of the launches and of each block's
// first loads, and for many that too few bytes are in flight (8192 rows: DRAM 41% busy in the first kernel, whose warps hold
// one chunk of loads each and wait for it, 50% in the second). The first kernel's operands go
// from global memory straight to the registers of the tensor-core products, 16 bytes a lane: a lane's k are consecutive
// (mma.cuh). In the second, so are the four pairs of columns n that a lane holds of four products.
//
// Rows stand by adapter (rows.cu), in tiles of 16 (of 32 or 64, which read an adapter's weights less, 12 - 40% slower
// at 64 to 1024 rows an adapter); up to kDirectRows rows go without a sort, one row to a tile (rows of one adapter then
// read its weights again, from L2). Without and with the sort, us, 4096 -> 4096 at rank 16 and 4096 -> 12288 at rank 64: 32 rows
// of one adapter 8.6 / 10.0 and 14.5 / 15.4, of 32 adapters 8.5 / 12.1 and 14.7 / 18.2; 64 rows of one 11.0 / 10.7 and 15.3 / 15.4.
//
// v stands in the second product as the sum of two 16-bit values, its rounding and what that left, which keeps about
// twice the type's bits for one more product each (they are not what bounds the kernel). For fp16 a row of v is first
// divided by a power of two, so that no v overflows the type.
//
// Measured: 8192 rows, 8192 -> 10240, rank 32: 122 us, 3.9 TB/s of x, base and y (0.58 of a copy's); 96 rows of 30
// adapters, 4096 -> 12288, ranks 16 to 64: 11 + 15 us and 5 for the sort; 1501 rows, 4000 -> 4099, rank 24: 9 + 19 and 6.
#include <atomic>

#include "gemm_common.cuh"
#include "internal.h"
#include "mma.cuh"
#include "ptx.cuh"

namespace w4 {
namespace {

using namespace detail;

constexpr int kWarps = 8;
constexpr int kTileRows = 16;
constexpr int kDirectRows = 32;

struct Tiles {
  RowPlan plan;
  const int32_t *adapter;  // direct: row i is tile i
  int direct;
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
  const RowTile t = ts.plan.tiles[i];  // (read beside the count: the list has room for every block)
  if (i >= *ts.plan.ntiles) return false;
  *key = t.key < adapters ? t.key : -1;
  *row0 = t.row0;
  *rows = t.rows;
  return true;
}

__device__ __forceinline__ int64_t row_at(const Tiles &ts, int pos) { return ts.direct ? pos : ts.plan.perm[pos]; }

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ uint4 ldg16(const uint16_t *p) { return *reinterpret_cast<const uint4 *>(p); }

// v[position][rank] = A[a] . x. A block holds a tile of 16 rows and NB * 8 ranks; its warps take 32 U of K in turn and add
// their sums in shared memory, in a fixed order. Where tiles are few the blocks of a cluster split K and add theirs through
// distributed shared memory, each a part of the tile, in the order of their ranks.
template <int DT, int NB, int U>
__global__ void __launch_bounds__(32 * kWarps, 2) lora_shrink_kernel(const Tiles ts, const LoraArgs a, float *v) {
  griddep_launch_dependents();
  griddep_wait();
  int key, row0, rows;
  if (!get_tile(ts, blockIdx.x, a.adapters, &key, &row0, &rows) || key < 0) return;
  const int rank = a.ranks ? min(max(a.ranks[key], 0), a.rank) : a.rank;
  const int n0 = blockIdx.z * NB * 8;
  if (n0 >= rank) return;  // (the second kernel reads no v at or past the adapter's rank)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int K = static_cast<int>(a.K);

  const uint16_t *xr[2];
  bool has[2];
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    has[m] = m * 8 + g < rows;
    xr[m] = static_cast<const uint16_t *>(a.x) + (has[m] ? row_at(ts, row0 + m * 8 + g) * a.ldx : 0);
  }
  const uint16_t *ar = static_cast<const uint16_t *>(a.A) + (static_cast<int64_t>(key) * a.rank + n0 + g) * K;
  bool live[NB];
#pragma unroll
  for (int n = 0; n < NB; ++n) live[n] = n0 + n * 8 + g < rank;

  float acc[NB][4] = {};
  const int chunk = 32 * U;
  const int step = chunk * kWarps * gridDim.y;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (int k0 = (blockIdx.y * kWarps + warp) * chunk; k0 < K; k0 += step) {
    uint4 xa[U][2], wb[U][NB];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * 32 + t * 8;  // K is a multiple of 8: eight values lie inside or outside together
      const bool in = k < K;
#pragma unroll
      for (int m = 0; m < 2; ++m) xa[u][m] = in && has[m] ? ldg16(xr[m] + k) : zero;
#pragma unroll
      for (int n = 0; n < NB; ++n) wb[u][n] = in && live[n] ? ldg16(ar + static_cast<int64_t>(n) * 8 * K + k) : zero;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        mma_16816<DT>(acc[n], xa[u][0].x, xa[u][1].x, xa[u][0].y, xa[u][1].y, wb[u][n].x, wb[u][n].y);
        mma_16816<DT>(acc[n], xa[u][0].z, xa[u][1].z, xa[u][0].w, xa[u][1].w, wb[u][n].z, wb[u][n].w);
      }
  }

  // the upper half of the warps gives its sums to the lower half until one warp has them all
  __shared__ float red[kWarps / 2][NB * 4][32];
#pragma unroll
  for (int half = kWarps / 2; half > 0; half >>= 1) {
    if (warp >= half && warp < 2 * half) {
#pragma unroll
      for (int i = 0; i < NB * 4; ++i) red[warp - half][i][lane] = acc[i / 4][i % 4];
    }
    __syncthreads();
    if (warp < half) {
#pragma unroll
      for (int i = 0; i < NB * 4; ++i) acc[i / 4][i % 4] += red[warp][i][lane];
    }
    __syncthreads();
  }
  const int C = gridDim.y;  // blocks of the cluster
  if (C == 1) {
    if (warp != 0) return;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      if (!has[m]) continue;
      float *row = v + static_cast<int64_t>(row0 + m * 8 + g) * a.rank + n0 + 2 * t;
#pragma unroll
      for (int n = 0; n < NB; ++n)
        if (n0 + n * 8 < a.rank) *reinterpret_cast<float2 *>(row + n * 8) = make_float2(acc[n][2 * m], acc[n][2 * m + 1]);
    }
    return;
  }
  float *part = &red[0][0][0];  // [row of the tile][NB * 8]
  static_assert(16 * NB * 8 <= kWarps / 2 * NB * 4 * 32, "the tile's sums fit");
  if (warp == 0) {
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int n = 0; n < NB; ++n)
        *reinterpret_cast<float2 *>(part + (m * 8 + g) * NB * 8 + n * 8 + 2 * t) = make_float2(acc[n][2 * m], acc[n][2 * m + 1]);
  }
  cluster_sync_all();
  for (int i = threadIdx.x + 32 * kWarps * blockIdx.y; i < rows * NB * 8; i += 32 * kWarps * C) {
    const int n = n0 + i % (NB * 8);
    if (n >= a.rank) continue;
    float sum = 0.0f;
    for (int c = 0; c < C; ++c) sum += ld_cluster_f32(mapa_shared(smem_u32(part + i), c));
    v[static_cast<int64_t>(row0 + i / (NB * 8)) * a.rank + n] = sum;
  }
  cluster_sync_all();  // no block leaves while another reads its sums
}

// Two values as the type's nearest (hi) and what that leaves (lo), each as a pair of 16-bit values. What an infinity
// leaves is nothing (not the NaN of its difference to itself).
template <int DT>
__device__ __forceinline__ void split_pair(float p, float q, uint32_t *hi, uint32_t *lo) {
  *hi = out_bits2<DT>(p, q);
  const float ph = value_f32<DT>(*hi & 0xffffu), qh = value_f32<DT>(*hi >> 16);
  *lo = out_bits2<DT>(isinf(ph) ? 0.0f : p - ph, isinf(qh) ? 0.0f : q - qh);
}

// stretches of base that a warp has in flight (8192 x 10240: 2 132 us, 3 147, 4 188: more reads ahead of the writes to
// other rows cost the memory more than they hide)
constexpr int kAhead = 2;
constexpr int kAheadB = 2;  // stretches of B

// Asynchronous copy of BYTES (8 or 16), of which the first `have` are read and the rest is zero.
template <int BYTES>
__device__ __forceinline__ void copy_ahead(uint32_t to, const void *from, uint32_t have) {
  if (BYTES == 16)
    cp_async16_zfill(to, from, have);
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(to), "l"(from), "r"(have) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Shared memory of an expand block. Both kernels: v; each warp's ring of B's stretches, every lane its own part. Rows of 16-byte
// pieces (wide): the rows' operands, factors and offsets, each warp's ring of base's stretches. Else: each warp's sums.
template <int KB, bool WIDE>
struct Expand {
  static constexpr int kLd = KB * 16 + 4;
  static constexpr int P = KB == 1 ? 1 : KB / 2;  // loads of B a product: 8 bytes a lane at ranks up to 16, else 16
  static constexpr int kLoad = KB == 1 ? 8 : 16;
  static constexpr int kWords = kLoad / 4;
  static constexpr int kStageB = 4 * P * 32 * kLoad;
  static constexpr int kLdSums = 66;
  static constexpr int kV = 16 * kLd * 4;
  static constexpr int kStageBase = 2 * 32 * 16;
  static constexpr int kWarp = kAheadB * kStageB + (WIDE ? kAhead * kStageBase : 16 * kLdSums * 4);
  static constexpr int kWarp0 = WIDE ? 0 : kV;  // wide: once the operands are made the rings take v's place
  static constexpr int kRings = kWarp0 + kWarps * kWarp;
  static constexpr int kFrags = kRings > kV ? kRings : kV;                      // [KB][hi, lo][lane] 16 bytes
  static constexpr int kOffsets = kFrags + (WIDE ? KB * 2 * 32 * 16 : 0);  // [row] offset in y, in base; else addresses
  static constexpr int kFactors = kOffsets + 16 * 16;                      // [row] factor of the sums, divisor's inverse; else flags
  static constexpr int kBytes = kFactors + 16 * 8;
  // that an SM's 228 KB hold, each with 1 KB of the system's (rows that are not wide: by their registers)
  static constexpr int kBlocks = !WIDE ? (KB <= 4 ? 2 : 1) : kBytes > 113 * 1024 ? 1 : kBytes > 75 * 1024 ? 2 : 3;
};

// The tile's v to shared memory; zero past the rows and past the adapter's rank, whatever stands there.
template <int KB, int LD>
__device__ __forceinline__ void load_v(float (*vs)[LD], const float *v, int row0, int rows, int rank, int rank_all) {
  for (int i = threadIdx.x; i < 16 * KB * 4; i += 32 * kWarps) {
    const int r = i / (KB * 4), k = i % (KB * 4) * 4;
    float4 p = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (r < rows && k < rank) {
      p = *reinterpret_cast<const float4 *>(v + (static_cast<int64_t>(row0) + r) * rank_all + k);
      if (k + 1 >= rank) p.y = 0.0f;
      if (k + 2 >= rank) p.z = 0.0f;
      if (k + 3 >= rank) p.w = 0.0f;
    }
    *reinterpret_cast<float4 *>(&vs[r][k]) = p;
  }
}

// What a row of v is multiplied by (down) before its operands are made, and its sums after (mul).
template <int DT>
__device__ __forceinline__ void row_factors(float top, float scale, float *down, float *mul) {
  *down = 1.0f;
  *mul = scale;
  if (DT == kDtypeF16 && top > 0.0f && top < INFINITY) {
    // 2^e <= top < 2^(e + 1), e kept where 2^e and 2^-e are normal: the row divided by 2^e has its largest in [1, 2)
    const int e = min(max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -100), 100);
    *down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    *mul = scale * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
  }
}

// A lane's four k of product b: a half of its load of B.
template <int KB>
__device__ __forceinline__ int k_of(int b, int t) {
  return KB == 1 ? 4 * t : 32 * (b / 2) + 8 * t + 4 * (b % 2);
}

// Copies a stretch of 32 columns of B ahead: the lane's part of four products, whose columns are dealt so that lane t then
// holds the eight columns of y from 8 t on.
template <typename E>
__device__ __forceinline__ void fetch_b(uint32_t to, const uint16_t *B, int n0, int N, int rank, int rank_all, const void *any) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int n = n0 + 8 * (g >> 1) + 2 * j + (g & 1);  // product j's column g
#pragma unroll
    for (int q = 0; q < E::P; ++q) {
      const int k = q * (E::kLoad * 2) + t * (E::kLoad / 2);
      const int have = n < N ? min(max(2 * (rank - k), 0), E::kLoad) : 0;
      copy_ahead<E::kLoad>(to + ((j * E::P + q) * 32 + lane) * E::kLoad,
                           have ? B + static_cast<int64_t>(n) * rank_all + k : any, have);
    }
  }
}

template <typename E>
__device__ __forceinline__ void load_b(uint32_t (&w)[E::P][E::kWords], uint32_t stage, int j) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int q = 0; q < E::P; ++q) {
    const uint32_t at = stage + ((j * E::P + q) * 32 + lane) * E::kLoad;
    if (E::kLoad == 16) {
      const uint4 v4 = lds128(at);
      w[q][0] = v4.x, w[q][1] = v4.y, w[q][2 % E::kWords] = v4.z, w[q][3 % E::kWords] = v4.w;
    } else {
      asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[q][0]), "=r"(w[q][1]) : "r"(at) : "memory");
    }
  }
}

// Product b of one column tile: lo before hi, so that the small terms are added first.
template <int DT, int KB, typename E>
__device__ __forceinline__ void product(float (&acc)[4], const uint32_t (&w)[E::P][E::kWords], int b, uint4 hi, uint4 lo) {
  const uint32_t b0 = w[KB == 1 ? 0 : b / 2][KB == 1 ? 0 : 2 * (b % 2)];
  const uint32_t b1 = w[KB == 1 ? 0 : b / 2][KB == 1 ? 1 : 2 * (b % 2) + 1];
  mma_16816<DT>(acc, lo.x, lo.y, lo.z, lo.w, b0, b1);
  mma_16816<DT>(acc, hi.x, hi.y, hi.z, hi.w, b0, b1);
}

// y = base + scaling * B[a] . v for a tile of 16 rows whose rows of y and base are 16-byte aligned. A warp takes every
// eighth stretch of 32 columns; B's and base's next stretches are copied ahead to shared memory (as loads to registers
// too few bytes were in flight: this kernel took 95 us for 8192 x 10240 at rank 32 instead of 74).
template <int DT, int KB>
__global__ void __launch_bounds__(32 * kWarps, Expand<KB, true>::kBlocks)
    lora_expand_wide_kernel(const Tiles ts, const LoraArgs a, const float *v) {
  using E = Expand<KB, true>;
  extern __shared__ __align__(16) uint8_t smem[];
  float(*vs)[E::kLd] = reinterpret_cast<float(*)[E::kLd]>(smem);
  uint4 *frags = reinterpret_cast<uint4 *>(smem + E::kFrags);
  int64_t(*offsets)[2] = reinterpret_cast<int64_t(*)[2]>(smem + E::kOffsets);
  float(*factors)[2] = reinterpret_cast<float(*)[2]>(smem + E::kFactors);
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

  if (threadIdx.x < 16) {
    const int64_t row = static_cast<int>(threadIdx.x) < rows ? row_at(ts, row0 + threadIdx.x) : 0;
    offsets[threadIdx.x][0] = row * a.ldy;
    offsets[threadIdx.x][1] = row * a.ldbase;
  }
  load_v<KB>(vs, v, row0, rows, rank, a.rank);
  __syncthreads();
  if (threadIdx.x < 16) {
    float top = 0.0f;
    if (DT == kDtypeF16)
      for (int k = 0; k < KB * 16; ++k) top = fmaxf(top, fabsf(vs[threadIdx.x][k]));
    row_factors<DT>(top, scale, &factors[threadIdx.x][1], &factors[threadIdx.x][0]);
  }
  __syncthreads();
  if (warp < KB) {
    const int b = warp;
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const int r = m * 8 + g;
      const float down = factors[r][1];
      const float4 p = *reinterpret_cast<const float4 *>(&vs[r][k_of<KB>(b, t)]);
      split_pair<DT>(p.x * down, p.y * down, &hi[m], &lo[m]);
      split_pair<DT>(p.z * down, p.w * down, &hi[2 + m], &lo[2 + m]);
    }
    frags[(b * 2 + 0) * 32 + lane] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    frags[(b * 2 + 1) * 32 + lane] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
  __syncthreads();

  const uint16_t *B = static_cast<const uint16_t *>(a.B) + static_cast<int64_t>(max(key, 0)) * N * a.rank;
  const uint16_t *base = static_cast<const uint16_t *>(a.base);
  uint16_t *y = static_cast<uint16_t *>(a.y);
  uint8_t *mine = smem + E::kWarp0 + warp * E::kWarp;
  const uint32_t b_ring = smem_u32(mine);
  uint4 *const ahead = reinterpret_cast<uint4 *>(mine + kAheadB * E::kStageB) + lane;
  auto fetch = [&](int n0, int slot) {
    const int n = n0 + 8 * t;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const int r = m * 8 + g;
      const int bytes = base && r < rows && n < N ? min(2 * (N - n), 16) : 0;
      cp_async16_zfill(smem_u32(ahead + (slot * 2 + m) * 32), bytes ? base + offsets[r][1] + n : a.B, bytes);
    }
  };
  const int first = (blockIdx.y * kWarps + warp) * 32, step = gridDim.y * kWarps * 32;
  static_assert(kAhead >= kAheadB, "base's copies lead");
  // the groups of copies in order: base's first stretches, then with each of B's the base kAhead - kAheadB after it
#pragma unroll
  for (int i = 0; i < kAhead - kAheadB; ++i) fetch(first + i * step, i);
#pragma unroll
  for (int i = 0; i < kAheadB - 1; ++i) {
    fetch_b<E>(b_ring + i * E::kStageB, B, first + i * step, N, rank, a.rank, a.B);
    fetch(first + (i + kAhead - kAheadB) * step, i + kAhead - kAheadB);
    copies_commit();
  }
  int slot = 0, slot_b = 0;
  for (int n0 = first; n0 < N; n0 += step) {
    fetch_b<E>(b_ring + (slot_b + kAheadB - 1) % kAheadB * E::kStageB, B, n0 + (kAheadB - 1) * step, N, rank, a.rank, a.B);
    fetch(n0 + (kAhead - 1) * step, (slot + kAhead - 1) % kAhead);
    copies_commit();
    copies_wait<kAheadB - 1>();
    const int n = n0 + 8 * t;
    float acc[4][4] = {};
    if (key >= 0) {
      uint32_t w[4][E::P][E::kWords];
#pragma unroll
      for (int j = 0; j < 4; ++j) load_b<E>(w[j], b_ring + slot_b * E::kStageB, j);
#pragma unroll
      for (int b = 0; b < KB; ++b) {
        const uint4 hi = frags[(b * 2 + 0) * 32 + lane], lo = frags[(b * 2 + 1) * 32 + lane];
#pragma unroll
        for (int j = 0; j < 4; ++j) product<DT, KB, E>(acc[j], w[j], b, hi, lo);
      }
    }
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const int r = m * 8 + g;
      if (r >= rows || n >= N) continue;
      const uint4 old = ahead[(slot * 2 + m) * 32];
      uint32_t out[4] = {old.x, old.y, old.z, old.w};
      if (key >= 0) {
        const float mul = factors[r][0];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          out[j] = out_bits2<DT>(value_f32<DT>(out[j] & 0xffffu) + mul * acc[j][2 * m],
                                 value_f32<DT>(out[j] >> 16) + mul * acc[j][2 * m + 1]);
      }
      uint16_t *to = y + offsets[r][0] + n;
      if (n + 8 <= N) {
        *reinterpret_cast<uint4 *>(to) = make_uint4(out[0], out[1], out[2], out[3]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (n + i < N) to[i] = static_cast<uint16_t>(out[i / 2] >> (16 * (i & 1)));
      }
    }
    slot = (slot + 1) % kAhead;
    slot_b = (slot_b + 1) % kAheadB;
  }
  copies_wait<0>();
}

// The same for rows that are not 16-byte aligned (of odd length, say): a warp takes every eighth stretch of 64 columns, whose
// sums go through shared memory, so that the warp reads and writes consecutive columns of a row, in pairs from the row's
// first 4-byte boundary. In a row that starts off that boundary lane 0 has the stretch's last column and its first instead
// of a pair. (1501 x 4099 at rank 24: 19 us; with every value's place worked out in the loop 35.)
template <int DT, int KB>
__global__ void __launch_bounds__(32 * kWarps, Expand<KB, false>::kBlocks)
    lora_expand_kernel(const Tiles ts, const LoraArgs a, const float *v) {
  using E = Expand<KB, false>;
  extern __shared__ __align__(16) uint8_t smem[];
  float(*vs)[E::kLd] = reinterpret_cast<float(*)[E::kLd]>(smem);
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

  const uint16_t *base = static_cast<const uint16_t *>(a.base);
  // the rows' first pairs in y and in base (the value before the row for one off the boundary), and how they lie
  struct Row {
    uint16_t *y;
    const uint16_t *base;
  };
  Row *const row_of = reinterpret_cast<Row *>(smem + E::kOffsets);
  int *const lies = reinterpret_cast<int *>(smem + E::kFactors);
  constexpr int kOff = 1, kPairs = 2, kLive = 4, kBase = 8;
  if (threadIdx.x < 16) {
    const bool live = static_cast<int>(threadIdx.x) < rows;
    const int64_t row = live ? row_at(ts, row0 + threadIdx.x) : 0;
    uint16_t *yp = static_cast<uint16_t *>(a.y) + row * a.ldy;
    const int off = (reinterpret_cast<uintptr_t>(yp) >> 1) & 1;
    const uint16_t *bp = base ? base + row * a.ldbase - off : nullptr;
    row_of[threadIdx.x] = Row{yp - off, bp};
    lies[threadIdx.x] = (off ? kOff : 0) | ((reinterpret_cast<uintptr_t>(bp) & 3) == 0 ? kPairs : 0) | (live ? kLive : 0) |
                        (base && live ? kBase : 0);
  }
  load_v<KB>(vs, v, row0, rows, rank, a.rank);
  __syncthreads();

  float mul[2];
  uint32_t hi[KB][4], lo[KB][4];
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const int r = m * 8 + g;
    float top = 0.0f, down;
    if (DT == kDtypeF16) {
      for (int k = t; k < KB * 16; k += 4) top = fmaxf(top, fabsf(vs[r][k]));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    }
    row_factors<DT>(top, scale, &down, &mul[m]);
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      const float4 p = *reinterpret_cast<const float4 *>(&vs[r][k_of<KB>(b, t)]);
      split_pair<DT>(p.x * down, p.y * down, &hi[b][m], &lo[b][m]);
      split_pair<DT>(p.z * down, p.w * down, &hi[b][2 + m], &lo[b][2 + m]);
    }
  }

  const uint16_t *B = static_cast<const uint16_t *>(a.B) + static_cast<int64_t>(max(key, 0)) * N * a.rank;
  uint8_t *mine = smem + E::kWarp0 + warp * E::kWarp;
  const uint32_t b_ring = smem_u32(mine);
  float(*sums)[E::kLdSums] = reinterpret_cast<float(*)[E::kLdSums]>(mine + kAheadB * E::kStageB);
  const int first = (blockIdx.y * kWarps + warp) * 64, step = gridDim.y * kWarps * 64;
  static_assert(kAheadB == 2, "a stretch's halves take the ring's places in turn");
  fetch_b<E>(b_ring, B, first, N, rank, a.rank, a.B);
  copies_commit();
  for (int n0 = first; n0 < N; n0 += step) {
    // base's pairs: the loads are predicated, not branched around, and joined only after the products
    const bool whole = n0 + 64 <= N;
    uint32_t both[16], low[16], high[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int how = lies[i];
      const uint16_t *bp = row_of[i].base + n0 + 2 * lane;
      const bool split = (how & kOff) && lane == 0;
      const int lo = split ? 64 : 0;  // where the lane's first value is, and its column:
      const int col = 2 * lane - (how & kOff) + lo;
      if (whole && (how & kPairs)) {
        both[i] = (how & kBase) && !split ? *reinterpret_cast<const uint32_t *>(bp) : 0u;
        low[i] = (how & kBase) && split ? bp[64] : 0u;
        high[i] = (how & kBase) && split ? bp[1] : 0u;
      } else {
        both[i] = 0u;
        low[i] = (how & kBase) && n0 + col < N ? bp[lo] : 0u;
        high[i] = (how & kBase) && n0 + 2 * lane - (how & kOff) + 1 < N ? bp[1] : 0u;
      }
    }
    __syncwarp();  // the stretch before has been read
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
      fetch_b<E>(b_ring + (1 - h) * E::kStageB, B, h == 0 ? n0 + 32 : n0 + step, N, rank, a.rank, a.B);
      copies_commit();
      copies_wait<1>();
      if (key < 0) continue;
      float acc[4][4] = {};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t w[E::P][E::kWords];
        load_b<E>(w, b_ring + h * E::kStageB, j);
#pragma unroll
        for (int b = 0; b < KB; ++b)
          product<DT, KB, E>(acc[j], w, b, make_uint4(hi[b][0], hi[b][1], hi[b][2], hi[b][3]),
                             make_uint4(lo[b][0], lo[b][1], lo[b][2], lo[b][3]));
      }
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<float2 *>(&sums[m * 8 + g][32 * h + 8 * t + 2 * j]) =
              make_float2(mul[m] * acc[j][2 * m], mul[m] * acc[j][2 * m + 1]);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int how = lies[i];
      if (!(how & kLive)) continue;
      uint16_t *yp = row_of[i].y + n0 + 2 * lane;
      const bool split = (how & kOff) && lane == 0;
      const int lo = split ? 64 : 0;
      const int col = 2 * lane - (how & kOff);  // the second value's column less one
      uint32_t out = both[i] | low[i] | high[i] << 16;
      if (key >= 0)
        out = out_bits2<DT>(value_f32<DT>(out & 0xffffu) + sums[i][col + lo], value_f32<DT>(out >> 16) + sums[i][col + 1]);
      if (whole && !split) {
        *reinterpret_cast<uint32_t *>(yp) = out;
      } else {
        if (n0 + col + lo < N) yp[lo] = static_cast<uint16_t>(out);
        if (n0 + col + 1 < N) yp[1] = static_cast<uint16_t>(out >> 16);
      }
    }
  }
  copies_wait<0>();
}

// The launch's shape, and the workspace's: [error block, left as it is, with ntiles in its second word][v][perm][tiles].
struct LoraPlan {
  bool direct;
  int max_tiles, splits;
  size_t v, perm, tiles, bytes;
};

LoraPlan lora_plan(int64_t T, int64_t N, int64_t K, int adapters, int rank, int num_sms) {
  LoraPlan p;
  p.direct = T <= kDirectRows;
  p.max_tiles = static_cast<int>(p.direct ? T : max_row_tiles(T, adapters, kTileRows));
  // few tiles: the blocks of a cluster split a tile's K, no finer than one turn of a block's warps (32 K values each)
  const int64_t turns = cdiv(K, 32 * kWarps);
  // (two blocks an SM run at a time: as many blocks as fit at once, since one more would wait for a whole turn)
  const int64_t want = 2 * num_sms / p.max_tiles;
  const int64_t splits = want < turns ? want : turns;
  p.splits = static_cast<int>(splits < 1 ? 1 : splits < 8 ? splits : 8);
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  p.v = 256;
  p.perm = p.v + up(static_cast<size_t>(T) * rank * 4);
  p.tiles = p.perm + (p.direct ? 0 : up(static_cast<size_t>(T) * 4));
  p.bytes = p.tiles + (p.direct ? 0 : up(static_cast<size_t>(p.max_tiles) * sizeof(RowTile)));
  return p;
}

template <typename... Args>
cudaError_t launch_grid(void (*kern)(Args...), dim3 grid, int cluster, int smem, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(32 * kWarps);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {1, static_cast<unsigned>(cluster), 1};
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int DT, int KB, bool WIDE>
cudaError_t launch_expand(const Tiles &ts, const LoraArgs &a, const LoraPlan &p, const float *v, int num_sms,
                          cudaStream_t stream) {
  void (*kern)(const Tiles, const LoraArgs, const float *);
  if constexpr (WIDE)
    kern = lora_expand_wide_kernel<DT, KB>;
  else
    kern = lora_expand_kernel<DT, KB>;
  constexpr int bytes = Expand<KB, WIDE>::kBytes;
  static std::atomic<uint64_t> set{0};
  const cudaError_t e = allow_smem(kern, bytes, &set);
  if (e != cudaSuccess) return e;
  // columns: as many blocks as run at a time, but three parts at least (8192 rows in one part 132 us, in three 123: the
  // parts of a tile run apart from one another) and no more than one turn of a block's warps each
  const int64_t turns = cdiv(a.N, (WIDE ? 32 : 64) * kWarps);
  int64_t parts = static_cast<int64_t>(Expand<KB, WIDE>::kBlocks) * num_sms / p.max_tiles;
  parts = parts < 3 ? 3 : parts;
  return launch_grid(kern, dim3(p.max_tiles, static_cast<unsigned>(parts < turns ? parts : turns)), 1, bytes, stream, ts, a,
                     v);
}

template <int DT>
cudaError_t launch_dt(const Tiles &ts, const LoraArgs &a, const LoraPlan &p, float *v, int num_sms, cudaStream_t stream) {
  auto shrink = a.rank <= 8    ? lora_shrink_kernel<DT, 1, 4>
                : a.rank <= 16 ? lora_shrink_kernel<DT, 2, 4>
                : a.rank <= 32 ? lora_shrink_kernel<DT, 4, 2>
                               : lora_shrink_kernel<DT, 8, 1>;
  const cudaError_t e =
      launch_grid(shrink, dim3(p.max_tiles, p.splits, a.rank > 64 ? 2 : 1), p.splits, 0, stream, ts, a, v);
  if (e != cudaSuccess) return e;
  const bool wide = a.ldy % 8 == 0 && reinterpret_cast<uintptr_t>(a.y) % 16 == 0 &&
                    (!a.base || (a.ldbase % 8 == 0 && reinterpret_cast<uintptr_t>(a.base) % 16 == 0));
  if (wide)
    return a.rank <= 16   ? launch_expand<DT, 1, true>(ts, a, p, v, num_sms, stream)
           : a.rank <= 32 ? launch_expand<DT, 2, true>(ts, a, p, v, num_sms, stream)
           : a.rank <= 64 ? launch_expand<DT, 4, true>(ts, a, p, v, num_sms, stream)
                          : launch_expand<DT, 8, true>(ts, a, p, v, num_sms, stream);
  return a.rank <= 16   ? launch_expand<DT, 1, false>(ts, a, p, v, num_sms, stream)
         : a.rank <= 32 ? launch_expand<DT, 2, false>(ts, a, p, v, num_sms, stream)
         : a.rank <= 64 ? launch_expand<DT, 4, false>(ts, a, p, v, num_sms, stream)
                        : launch_expand<DT, 8, false>(ts, a, p, v, num_sms, stream);
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
  if (!p.direct) {
    ts.plan.perm = reinterpret_cast<int32_t *>(ws + p.perm);
    ts.plan.tiles = reinterpret_cast<RowTile *>(ws + p.tiles);
    ts.plan.ntiles = reinterpret_cast<int32_t *>(ws + 4);
    const cudaError_t e = launch_row_plan(a.adapter, a.T, a.adapters, kTileRows, true, ts.plan, stream);
    if (e != cudaSuccess) return e;
  }
  float *v = reinterpret_cast<float *>(ws + p.v);
  return a.dtype == kDtypeBf16 ? launch_dt<kDtypeBf16>(ts, a, p, v, num_sms, stream)
                               : launch_dt<kDtypeF16>(ts, a, p, v, num_sms, stream);
}

}  // namespace w4
