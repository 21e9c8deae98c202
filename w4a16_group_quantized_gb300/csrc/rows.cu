// Sorting rows by a key that is chosen on the device (a token's expert, a request's adapter), so that the rows that
// share weights stand together: counts per key, their running sum, each row's place, and the list of tiles of one
// key that the kernels after it walk.
//
// The keys are a few kilobytes (a decode batch) to a few hundred, so latency bounds it: one block up to 4096 rows, above
// that a cluster of eight, each of which counts and places its part of the rows and reads the others' counts in their
// shared memory (32,768 rows of 64 keys: 60 us in one block). The rows of one key come in no fixed order within
// their part: a place decides where a row's sums are held, never what is added to what, so no result depends on it.
#include "gemm_common.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace w4 {
namespace {

constexpr int kThreads = 1024;
constexpr int kBuckets = kRowsMaxKeys + 1;  // the last: no key
constexpr int kPlanCluster = 8;

// Adds the warp's rows to their buckets' counters and returns each row's old count (its rank among the bucket's rows so
// far): one addition for a warp whose rows are all of one key (the rows of a long request), else one a row. Every lane
// of the warp calls it; bucket < 0 takes no part.
__device__ __forceinline__ int count_in(int32_t *counter, int bucket) {
  int same;
  __match_all_sync(0xffffffffu, bucket, &same);
  if (same) {
    const int lane = threadIdx.x & 31;
    int at = 0;
    if (lane == 0 && bucket >= 0) at = atomicAdd(&counter[bucket], 32);
    return __shfl_sync(0xffffffffu, at, 0) + lane;
  }
  return bucket >= 0 ? atomicAdd(&counter[bucket], 1) : 0;
}

__device__ __forceinline__ int warp_sum_to(int v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// Running sums over the block of two values per thread: the sums of the threads before this one, and of all.
__device__ __forceinline__ int2 sums_before(int2 v, int2 *warp_sums, int2 *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int2 s = make_int2(warp_sum_to(v.x), warp_sum_to(v.y));
  if (lane == 31) warp_sums[warp] = s;
  __syncthreads();
  if (warp == 0) {
    const int2 w = warp_sums[lane];
    warp_sums[lane] = make_int2(warp_sum_to(w.x), warp_sum_to(w.y));
  }
  __syncthreads();
  const int2 before = warp > 0 ? warp_sums[warp - 1] : make_int2(0, 0);
  *total = warp_sums[kThreads / 32 - 1];
  return make_int2(before.x + s.x - v.x, before.y + s.y - v.y);
}

__device__ __forceinline__ int32_t ld_cluster_s32(uint32_t addr) {
  int32_t v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

template <int C>
__global__ void __launch_bounds__(kThreads)
    row_plan_kernel(const int32_t *keys, int64_t count, int nkeys, int tile, int keyless, RowPlan plan) {
  // counts: of this block's rows; all: of every block's; begin: the next free place of a bucket for this block
  __shared__ int32_t counts[kBuckets], all[kBuckets], begin[kBuckets], tile_begin[kBuckets];
  __shared__ int2 warp_sums[kThreads / 32];
  const int tid = threadIdx.x;
  const int rank = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  griddep_launch_dependents();
  for (int b = tid; b <= nkeys; b += kThreads) counts[b] = 0;
  griddep_wait();
  __syncthreads();
  const int64_t part = (count + C * kThreads - 1) / (C * kThreads) * kThreads;
  const int64_t i_end = min(count, (rank + 1) * part);
  for (int64_t i0 = rank * part; i0 < i_end; i0 += kThreads) {
    const int64_t i = i0 + tid;
    int bucket = -1;
    if (i < i_end) {
      const int32_t key = keys[i];
      bucket = key >= 0 && key < nkeys ? key : nkeys;
    }
    count_in(counts, bucket);
  }
  if (C > 1) cluster_sync_all(); else __syncthreads();
  // per bucket: rows in the blocks before this one, and in all
  for (int b = tid; b <= nkeys; b += kThreads) {
    int before = 0, sum = 0;
    if (C == 1) {
      sum = counts[b];
    } else {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int n = ld_cluster_s32(mapa_shared(smem_u32(&counts[b]), c));
        before += c < rank ? n : 0;
        sum += n;
      }
    }
    all[b] = sum;
    begin[b] = before;
  }
  __syncthreads();
  // bucket nkeys = 1024 comes after every thread's
  const int rows = tid <= nkeys ? all[tid] : 0;
  const int tiles = tid < nkeys || (tid == nkeys && keyless) ? (rows + tile - 1) / tile : 0;
  int2 total;
  const int2 at = sums_before(make_int2(rows, tiles), warp_sums, &total);
  if (tid <= nkeys) {
    begin[tid] += at.x;
    tile_begin[tid] = at.y;
  }
  int ntiles = total.y;
  if (nkeys == kThreads) {
    if (tid == 0) {
      begin[nkeys] += total.x;
      tile_begin[nkeys] = total.y;
    }
    if (keyless) ntiles += (all[nkeys] + tile - 1) / tile;
  }
  if (rank == 0 && tid == 0) {
    *plan.ntiles = ntiles;
    if (plan.err) *plan.err = 0u;
  }
  __syncthreads();
  const int buckets = nkeys + (keyless ? 1 : 0);
  for (int i = rank * kThreads + tid; i < ntiles; i += C * kThreads) {
    int lo = 0, hi = buckets;  // the last bucket with tile_begin <= i
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (tile_begin[mid] <= i) lo = mid; else hi = mid;
    }
    // the bucket's first place: this block's next one less the rows of the blocks before it
    int first = begin[lo];
    if (C > 1)
      for (int c = 0; c < rank; ++c) first -= ld_cluster_s32(mapa_shared(smem_u32(&counts[lo]), c));
    const int in = (i - tile_begin[lo]) * tile;
    plan.tiles[i] = RowTile{lo, first + in, min(tile, all[lo] - in), 0};
  }
  // counts of every block have been read, and begin by every thread of this one, which the loop below changes
  if (C > 1) cluster_sync_all(); else __syncthreads();
  for (int64_t i0 = rank * part; i0 < i_end; i0 += kThreads) {
    const int64_t i = i0 + tid;
    int bucket = -1;
    if (i < i_end) {
      const int32_t key = keys[i];
      bucket = key >= 0 && key < nkeys ? key : nkeys;
    }
    const int place = count_in(begin, bucket);
    if (i < i_end) {
      plan.perm[place] = static_cast<int32_t>(i);
      if (plan.inverse) plan.inverse[i] = bucket < nkeys ? place : -1;
    }
  }
}

}  // namespace

cudaError_t launch_row_plan(const int32_t *keys, int64_t count, int nkeys, int tile, bool keyless, const RowPlan &plan,
                            cudaStream_t stream) {
  if (count <= 4096)
    return detail::launch_programmatic(row_plan_kernel<1>, 1, kThreads, 0, stream, keys, count, nkeys, tile,
                                       static_cast<int>(keyless), plan);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kPlanCluster);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {kPlanCluster, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, row_plan_kernel<kPlanCluster>, keys, count, nkeys, tile,
                                           static_cast<int>(keyless), plan);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace w4
