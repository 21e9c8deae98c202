// Sorting rows by a key that is chosen on the device (a token's expert, a request's adapter), so that the rows that
// share weights stand together: counts per key, their running sum, each row's place, and the list of tiles of one
// key that the kernels after it walk.
//
// One block: the keys are a few kilobytes (a decode batch) to a few hundred, so the launch itself and the latency of
// its passes over them bound it. The rows of one key come in no fixed order: a place decides where a row's sums are
// held, never what is added to what, so no result depends on it.
#include "gemm_common.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace w4 {
namespace {

constexpr int kThreads = 1024;
constexpr int kBuckets = kRowsMaxKeys + 1;  // the last: no key

// Adds the warp's rows to their buckets' counters, one addition per bucket and warp, and returns each row's old
// count (its rank among the bucket's rows so far). Every lane of the warp calls it; bucket < 0 takes no part.
__device__ __forceinline__ int count_in(int32_t *counter, int bucket) {
  const int lane = threadIdx.x & 31;
  const uint32_t same = __match_any_sync(0xffffffffu, bucket);
  const int leader = __ffs(same) - 1;
  int at = 0;
  if (lane == leader && bucket >= 0) at = atomicAdd(&counter[bucket], __popc(same));
  return __shfl_sync(0xffffffffu, at, leader) + __popc(same & ((1u << lane) - 1u));
}

// Running sum over the block of one value per thread: the sum of the values of the threads before this one.
__device__ __forceinline__ int sum_before(int v, int32_t *warp_sums, int *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, s, d);
    if (lane >= d) s += o;
  }
  __syncthreads();  // the last use of warp_sums is over
  if (lane == 31) warp_sums[warp] = s;
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    const int x = warp_sums[w];
    before += w < warp ? x : 0;
    all += x;
  }
  *total = all;
  return before + s - v;
}

__global__ void __launch_bounds__(kThreads)
    row_plan_kernel(const int32_t *__restrict__ keys, int64_t count, int nkeys, int tile, int keyless, RowPlan plan) {
  __shared__ int32_t counts[kBuckets], begin[kBuckets], tile_begin[kBuckets], warp_sums[kThreads / 32];
  const int tid = threadIdx.x;
  griddep_launch_dependents();
  for (int b = tid; b < kBuckets; b += kThreads) counts[b] = 0;
  griddep_wait();
  __syncthreads();
  for (int64_t i0 = 0; i0 < count; i0 += kThreads) {
    const int64_t i = i0 + tid;
    int bucket = -1;
    if (i < count) {
      const int32_t key = keys[i];
      bucket = key >= 0 && key < nkeys ? key : nkeys;
    }
    count_in(counts, bucket);
  }
  __syncthreads();
  int rows = 0, tiles = 0, all;
  const bool own = tid <= nkeys && tid < kThreads;  // bucket nkeys = 1024 comes after every thread's
  if (own) {
    rows = counts[tid];
    tiles = tid < nkeys || keyless ? (rows + tile - 1) / tile : 0;
  }
  const int b0 = sum_before(rows, warp_sums, &all);
  if (own) begin[tid] = b0;
  if (nkeys == kThreads && tid == 0) begin[nkeys] = all;
  const int t0 = sum_before(tiles, warp_sums, &all);
  if (own) tile_begin[tid] = t0;
  if (nkeys == kThreads && keyless) {
    if (tid == 0) tile_begin[nkeys] = all;
    all += (counts[nkeys] + tile - 1) / tile;
  }
  if (tid == 0) *plan.ntiles = all;
  if (tid == 0 && plan.err) *plan.err = 0u;
  __syncthreads();
  const int buckets = nkeys + (keyless ? 1 : 0);
  for (int i = tid; i < all; i += kThreads) {
    int lo = 0, hi = buckets;  // the last bucket with tile_begin <= i
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (tile_begin[mid] <= i) lo = mid; else hi = mid;
    }
    const int first = (i - tile_begin[lo]) * tile;
    plan.tiles[i] = RowTile{lo, begin[lo] + first, min(tile, counts[lo] - first), 0};
  }
  __syncthreads();
  for (int64_t i0 = 0; i0 < count; i0 += kThreads) {
    const int64_t i = i0 + tid;
    int bucket = -1;
    if (i < count) {
      const int32_t key = keys[i];
      bucket = key >= 0 && key < nkeys ? key : nkeys;
    }
    const int at = count_in(begin, bucket);
    if (i < count) {
      plan.perm[at] = static_cast<int32_t>(i);
      if (plan.inverse) plan.inverse[i] = bucket < nkeys ? at : -1;
    }
  }
}

}  // namespace

cudaError_t launch_row_plan(const int32_t *keys, int64_t count, int nkeys, int tile, bool keyless, const RowPlan &plan,
                            cudaStream_t stream) {
  return detail::launch_programmatic(row_plan_kernel, 1, kThreads, 0, stream, keys, count, nkeys, tile,
                                     static_cast<int>(keyless), plan);
}

}  // namespace w4
