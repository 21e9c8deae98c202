// What the two kernels of the experts' products share (experts.cu: few rows an expert; experts_tmem.cu: many).
#pragma once

#include "gemm_common.cuh"
#include "internal.h"

namespace w4 {
namespace detail {

struct Products {
  const uint16_t *in;    // gate/up: x [T, K]; down: h [pairs, K]
  const uint8_t *codes;  // expert 0's packed weights
  int64_t expert_bytes;
  int64_t meta;          // offset of the group records in them
  void *out;             // gate/up: h [pairs, N / 2], 16 bits; down: [pairs, N], 32 bits
  float *wide;           // fp16 gate/up after a sort: [pairs, N / 2], written only where h is past the type's range
  RowPlan plan;
  uint32_t *err;
  int64_t in_rows;
  int K, N, G, KB, g;
  int slabs;             // blocks (experts.cu) or weight tiles (experts_tmem.cu) of N
  int choices;           // k: pair / k is the token
  // experts.cu without a plan: tile i is pair i (gate/up) or token i with all its choices (down, whose out is then y)
  const int32_t *ids;
  const float *weights;
  int experts;
  int kw;                // warps that share a slab's K
  FastDiv gdiv;
  // experts_tmem.cu
  uint64_t wait_limit;   // cycles a wait may take before the kernel gives up
  int test_extra;        // test only: arrivals that the first barrier expects and that never come
};

// The h of sorted row pos, column j, of tile t: rounded to the type. Where that overflows, the 32-bit value goes to `wide` and the
// tile is marked (range_kernel in experts.cu then scales the row).
template <int DT>
__device__ __forceinline__ void store_h(const Products &p, float h, int64_t at, int t) {
  const uint16_t bits = out_bits<DT>(h);
  static_cast<uint16_t *>(p.out)[at] = bits;
  if (DT == kDtypeF16 && (bits & 0x7FFFu) == 0x7C00u) {
    p.wide[at] = h;
    p.plan.tiles[t].flag = 1;
  }
}

// Whether the tensor-memory kernel takes groups of g: a block of 64 k then holds at most two, 32 k each.
inline bool experts_tmem_takes(int g) { return g % 32 == 0; }

// The products with `tile` (64 or 128) rows of `in` a tile; `in` stands in the sort's order for gate/up too.
cudaError_t launch_experts_tmem(const Products &p, int dtype, bool gated, int tile, int num_sms, cudaStream_t stream);

}  // namespace detail
}  // namespace w4
