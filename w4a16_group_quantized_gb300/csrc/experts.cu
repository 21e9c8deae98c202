// w4a16_experts: y[t] = sum_j weights[t, j] * down_e (silu(gate_e x_t) * up_e x_t), e = ids[t, j], with each expert's
// weights in 4-bit groups, w = (q - z) s.
//
// The pairs (token, choice) are sorted by expert (rows.cu) and cut into tiles of one expert; a first product makes
// h = silu(gate) * up of each pair, rounded once to the 16-bit type (the second product's operand: 32 bits of it would take
// two or three products instead of one), a second one the expert's output in 32 bits, and a last pass adds a token's
// outputs with their weights, in the order of its choices. In fp16 a row of h whose largest value is past the type's range
// is divided by a power of two before the second product (range_kernel).
// Few pairs go without a sort, one row a product, which leaves columns of the products free: h then stands in two of them, as
// its rounding to bf16 and what that left (16 bits and a 32-bit exponent, whatever the type: codes are exact in either).
//
// The products here run on register-operand tensor-core instructions, for few rows per expert: the weights of the
// chosen experts are read once and that is the floor. Codes go through rings in shared memory that belong to one warp
// each, so that no barrier stands between the copies and the products; a lane reads 8 bytes of a row (the tile layout
// deals it 16 consecutive codes). Where slabs of 32 weight rows are few, a block's warps split K and add their sums
// in shared memory in a fixed order.
//
// Codes become operands without arithmetic: a code's four bits under the exponent of 16 are 16 + q in either type.
// A product with ones gives X = sum x over the same k, and (q - z) x sums to sum (16 + q) x - (16 + z) X, exactly in
// the operands and in 32 bits in the sums; a group's sum is multiplied by its 32-bit s. So no weight is rounded.
//
// Measured (8 experts, 4096 x 11008, 16 rows of 2 choices, fp16): 100 us for gate/up and 52 for down, 3.6 TB/s of
// codes; 186 instructions a kilobyte of codes keep the issue slots 62% and the shift and logic units 55% busy, memory
// 46%. One token through 8 of 64 experts of 2048 x 1024: 12 + 9 us.
#include <atomic>

#include "experts.cuh"
#include "gemm_common.cuh"
#include "internal.h"
#include "mma.cuh"
#include "ptx.cuh"

namespace w4 {
namespace {

using namespace detail;

constexpr int kSlabRows = 32;  // weight rows of a block
// Rows an expert has on average from which the tensor-memory kernel runs: the host knows no more than the average, so a batch
// that crowds into a few of many experts runs in tiles chosen for few rows (right, but its experts' weights are read by more
// tiles). Measured, this kernel / that one: 8 experts of
// 4096 x 11008: 4 rows 144 / 188 us, 8 rows 211 / 201, 16 rows 369 / 205; 64 experts of 2048 x 1024: 4 rows 74 / 79,
// 8 rows 99 / 86, 16 rows 180 / 89.
constexpr int kTmemRows = 8;

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

// How groups lie: kAny takes a 64-block's groups in turn, each with the other groups' x as zeros; kBlock: g a multiple of
// 64, one group a block; kTwo: g a multiple of 128, one group two blocks.
enum Groups { kAny, kBlock, kTwo };

// A warp's ring of stages of two blocks of 64 k: [codes: block, half of its k, row, 16 bytes][x: block, 8 rows x 128 bytes,
// 16-byte pieces swapped by row][group records: block, 32 scales and 32 zeros].
template <int NT>
struct Stage {
  static constexpr int kX = 2048, kRec = kX + 2 * NT * 1024, kBytes = kRec + 256;
  static constexpr int kCount = NT <= 2 ? 3 : 2;
  static constexpr int kRing = kCount * kBytes;
};

// A block of warps: kw of them share a slab of 32 weight rows x one tile of up to 8 NT rows of `in`, and split its K in
// steps of two blocks. GATED: rows 2 j and 2 j + 1 are gate and up j. DIRECT: no plan (see Products); down then runs over
// all choices of a token, each group's scale multiplied by the choice's weight, and its sums are y.
// Everything a warp reads it copies ahead into its own ring: as loads to registers, two blocks ahead, 8 experts of
// 4096 x 11008 took 124 + 61 us instead of 100 + 52.
template <int DT, int NT, bool GATED, Groups MODE, bool DIRECT, int NW>
__global__ void __launch_bounds__(32 * NW, NT == 1 && NW == 8 ? 2 : 1) experts_kernel(const Products p) {
  using St = Stage<NT>;
  constexpr int D = St::kCount;
  constexpr bool ALL = DIRECT && !GATED;
  constexpr int OT = ALL ? kDtypeBf16 : DT;  // the operands' type
  extern __shared__ __align__(128) uint8_t smem[];
  griddep_launch_dependents();
  griddep_wait();
  if (DIRECT && GATED && blockIdx.x == 0 && threadIdx.x == 0) *p.err = 0u;  // (else the sort clears it)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int kw = p.kw, part = warp % kw;
  const int slabs_block = NW / kw;
  const int per_tile = (p.slabs + slabs_block - 1) / slabs_block;
  const int tile = blockIdx.x / per_tile;
  const int n0 = ((blockIdx.x - tile * per_tile) * slabs_block + warp / kw) * kSlabRows;
  RowTile rt;
  int cols;           // of `in` in the tile: its rows, or a row's two halves
  int id = -1;        // ALL: lane j's are choice j's
  float weight = 0.0f;
  if (DIRECT) {
    rt = RowTile{ALL ? 0 : p.ids[tile], tile, 1, 0};
    if (!ALL && (rt.key < 0 || rt.key >= p.experts)) return;
    if (ALL && lane < p.choices) {
      id = p.ids[static_cast<int64_t>(tile) * p.choices + lane];
      weight = p.weights[static_cast<int64_t>(tile) * p.choices + lane];
      if (id >= p.experts) id = -1;
    }
  } else {
    rt = p.plan.tiles[tile];  // (read beside the count: the list has room for every block)
    if (tile >= *p.plan.ntiles) return;
  }
  cols = ALL ? 2 : rt.rows;

  // the rows that the lane copies: lane / 8 and lane / 8 + 4 of each eight, piece lane % 8 of their 128 bytes
  const uint16_t *xr[2 * NT];
#pragma unroll
  for (int n = 0; n < 2 * NT; ++n) {
    const int col = n * 4 + (lane >> 3), pos = rt.row0 + col;
    xr[n] = nullptr;
    if (col < cols) {
      const int64_t row = ALL ? static_cast<int64_t>(rt.row0) * p.choices * 2 + col
                          : DIRECT && GATED ? pos / p.choices
                          : GATED ? p.plan.perm[pos] / p.choices : pos;
      xr[n] = p.in + row * p.K + 8 * (lane & 7);
    }
  }
  const int wt = n0 / kTN, r0 = n0 % kTN;
  const int64_t codes0 = static_cast<int64_t>(wt) * p.KB * kTileBytes + (r0 + lane) * 16;
  const int64_t meta0 = p.meta + static_cast<int64_t>(wt) * p.G * kRecBytes;
  const bool live = n0 < p.N;
  const uint32_t ring = smem_u32(smem) + warp * St::kRing;
  // where the lane's pieces of x go
  const uint32_t x_to = ring + St::kX + (lane >> 3) * 128 + ((lane & 7) ^ (lane >> 3)) * 16;
  const uint32_t x_to4 = ring + St::kX + ((lane >> 3) + 4) * 128 + ((lane & 7) ^ ((lane >> 3) + 4)) * 16;
  if (cols < 8 * NT)  // rows that the tile has not are zeros
    for (int i = lane; i < D * 2 * NT * 64; i += 32) {
      const int at = i / 64, row = i % (64) / 8;
      if (at % NT * 8 + row >= cols)
        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(ring + at / (2 * NT) * St::kBytes + St::kX +
                                                                      at % (2 * NT) * 1024 + i % 64 * 16),
                     "r"(0)
                     : "memory");
    }

  // the warp's steps: of the tile's expert, or of all choices one after another
  const int steps = (p.KB + 1) / 2, all = ALL ? steps * p.choices : steps;
  const int f0 = all * part / kw, f1 = live ? all * (part + 1) / kw : f0;
  int jf = ALL ? f0 / steps : 0;  // choice and step of the next copies
  int sf = f0 - jf * steps;
  auto fill = [&](int f, int slot) {
    if (f < f1) {
      int key = rt.key;
      const int choice = jf, kb = 2 * sf++;
      if (ALL) {
        key = __shfl_sync(0xffffffffu, id, choice);
        if (sf == steps) sf = 0, ++jf;
      }
      if (key >= 0) {
        const uint8_t *expert = p.codes + key * p.expert_bytes;
        const uint32_t to = slot * St::kBytes;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if (kb + u >= p.KB) break;
          const uint8_t *cb = expert + codes0 + static_cast<int64_t>(kb + u) * kTileBytes;
          cp_async16_zfill(ring + to + u * 1024 + lane * 16, cb, 16);
          cp_async16_zfill(ring + to + u * 1024 + 512 + lane * 16, cb + 2048, 16);
          const int k = (kb + u) * kTK;
          const uint32_t bytes = k + 8 * (lane & 7) < p.K ? 16u : 0u;  // K is a multiple of 8
#pragma unroll
          for (int n = 0; n < 2 * NT; ++n)
            if (xr[n])
              cp_async16_zfill((n & 1 ? x_to4 : x_to) + to + (u * NT + n / 2) * 1024,
                               bytes ? xr[n] + (ALL ? static_cast<int64_t>(choice) * 2 * p.K : 0) + k : p.in, bytes);
          if (MODE == kBlock || (MODE == kTwo && u == 0)) {
            const uint8_t *m = expert + meta0 + static_cast<int64_t>(p.gdiv.div(k)) * kRecBytes;
            if (lane < 20)  // 32 scales and 32 zeros, 4 bytes a lane
              asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(ring + to + St::kRec + u * 128 + 4 * lane),
                           "l"(lane < 16 ? m + 2 * r0 + 4 * lane : m + 256 + r0 / 2 + 4 * (lane - 16))
                           : "memory");
          }
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // row l's scale, and its zero in the upper half, for lane l
  auto record = [&](const uint8_t *m) {
    return *reinterpret_cast<const uint16_t *>(m + 2 * (r0 + lane)) |
           static_cast<uint32_t>((m[256 + (r0 + lane) / 2] >> (4 * (lane & 1))) & 15) << 16;
  };
  auto record_at = [&](uint32_t at) { return lds16(at + 2 * lane) | ((lds8(at + 64 + lane / 2) >> (4 * (lane & 1))) & 15) << 16; };

  constexpr uint32_t kOne = OT == kDtypeBf16 ? 0x3F803F80u : 0x3C003C00u;
  float sum[2][NT][4] = {};  // rows g, g + 8 (and 16, 24): what is done
  float d0[NT][4], d1[NT][4], ones[NT][4];
  auto clear = [&] {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) d0[n][i] = d1[n][i] = ones[n][i] = 0.0f;
  };
  // adds a group's products to the sums: scale * (sum (16 + q) x - (16 + zero) sum x)
  auto close = [&](uint32_t rec, float weight) {
    float s[4], zb[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t v = __shfl_sync(0xffffffffu, rec, i * 8 + g);
      s[i] = scale_f32<DT>(v & 0xffffu);
      if (ALL) s[i] *= weight;
      zb[i] = static_cast<float>(16 + static_cast<int>(v >> 16));
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // i / 2: row g or g + 8; i % 2: column 2 t + i % 2
        sum[0][n][i] += s[i / 2] * (d0[n][i] - zb[i / 2] * ones[n][i]);
        sum[1][n][i] += s[2 + i / 2] * (d1[n][i] - zb[2 + i / 2] * ones[n][i]);
      }
  };
  // one block's products; first, second: whether the lane's two words of codes take part
  auto block = [&](const uint32_t (&a)[4][8], uint32_t x_at, bool first, bool second) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const uint4 x0 = lds128(x_at + n * 1024 + g * 128 + ((2 * t) ^ g) * 16);
      const uint4 x1 = lds128(x_at + n * 1024 + g * 128 + ((2 * t + 1) ^ g) * 16);
      uint32_t b[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
      if (MODE == kAny) {
#pragma unroll
        for (int i = 0; i < 8; ++i) b[i] = (i < 4 ? first : second) ? b[i] : 0u;
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        mma_16816<OT>(d0[n], a[0][2 * q], a[1][2 * q], a[0][2 * q + 1], a[1][2 * q + 1], b[2 * q], b[2 * q + 1]);
        mma_16816<OT>(d1[n], a[2][2 * q], a[3][2 * q], a[2][2 * q + 1], a[3][2 * q + 1], b[2 * q], b[2 * q + 1]);
        mma_16816<OT>(ones[n], kOne, kOne, kOne, kOne, b[2 * q], b[2 * q + 1]);
      }
    }
  };
  int jc = ALL ? f0 / steps : 0, sc = f0 - jc * steps;  // choice and step of the next products
  auto compute = [&](int slot) {
    const int kb = 2 * sc++;
    int key = rt.key;
    float w = 1.0f;
    if (ALL) {
      key = __shfl_sync(0xffffffffu, id, jc);
      w = __shfl_sync(0xffffffffu, weight, jc);
      if (sc == steps) sc = 0, ++jc;
      if (key < 0) return;
    }
    const uint32_t at = ring + slot * St::kBytes;
    if (MODE != kAny) clear();
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (kb + u >= p.KB) break;
      uint32_t a[4][8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // lane t's 16 codes of a row: half t / 2 of the block's k, bytes 8 (t % 2) of the row's 16
        uint32_t c0, c1;
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                     : "=r"(c0), "=r"(c1)
                     : "r"(at + u * 1024 + (t >> 1) * 512 + (8 * i + g) * 16 + 8 * (t & 1))
                     : "memory");
        operands<OT>(c0, a[i]);
        operands<OT>(c1, a[i] + 4);
      }
      const uint32_t x_at = at + St::kX + u * NT * 1024;
      if (MODE == kAny) {
        const uint8_t *meta = p.codes + key * p.expert_bytes + meta0;
        const int k0 = (kb + u) * kTK;
        const int j1 = p.gdiv.div(min(k0 + kTK, p.K) - 1);
        for (int j = p.gdiv.div(k0); j <= j1; ++j) {
          clear();
          block(a, x_at, p.gdiv.div(k0 + 16 * t) == j, p.gdiv.div(k0 + 16 * t + 8) == j);
          close(record(meta + static_cast<int64_t>(j) * kRecBytes), w);
        }
      } else {
        block(a, x_at, true, true);
        if (MODE == kBlock) {
          close(record_at(at + St::kRec + u * 128), w);
          clear();
        }
      }
    }
    if (MODE == kTwo) close(record_at(at + St::kRec), w);
  };
#pragma unroll
  for (int i = 0; i < D - 1; ++i) fill(f0 + i, i);
  int slot = 0;
  for (int f = f0; f < f1; ++f) {
    asm volatile("cp.async.wait_group %0;" ::"n"(D - 2) : "memory");
    __syncwarp();  // every lane's copies of this stage are there, and every lane is done with the stage before
    fill(f + D - 1, slot == 0 ? D - 1 : slot - 1);
    compute(slot);
    slot = slot == D - 1 ? 0 : slot + 1;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");

  // [warp][column][row], a column's rows one bank off the next column's
  constexpr int kLd = kSlabRows + 4;
  __syncthreads();  // every warp is done with its ring, which the sums take over
  float(*red)[8 * NT][kLd] = reinterpret_cast<float(*)[8 * NT][kLd]>(smem);
  static_assert(sizeof(float) * 8 * NT * kLd <= St::kRing, "the sums fit");
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[warp][n * 8 + 2 * t + (i & 1)][m * 16 + (i >> 1) * 8 + g] = sum[m][n][i];
  __syncthreads();
  // the slab's warps write its outputs: the sums of its parts of K in order
  const int w0 = warp - part, tid = part * 32 + lane, threads = 32 * kw;
  if (GATED) {
    for (int i = tid; i < rt.rows * 16; i += threads) {
      const int col = i / 16, j = i % 16;
      if (n0 + 2 * j >= p.N) continue;
      float gate = 0.0f, up = 0.0f;
      for (int w = w0; w < w0 + kw; ++w) {
        gate += red[w][col][2 * j];
        up += red[w][col][2 * j + 1];
      }
      const float h = silu_mul(gate, up);
      const int64_t row = rt.row0 + col;
      if (DIRECT) {  // (what an infinity leaves is nothing, not the NaN of its difference to itself)
        uint16_t *out = static_cast<uint16_t *>(p.out) + row * p.N + n0 / 2 + j;
        const uint16_t hi = out_bits<kDtypeBf16>(h);
        const float left = value_f32<kDtypeBf16>(hi);
        out[0] = hi;
        out[p.N / 2] = out_bits<kDtypeBf16>(isinf(left) ? 0.0f : h - left);
      } else {
        store_h<DT>(p, h, row * (p.N / 2) + n0 / 2 + j, tile);
      }
    }
  } else {
    for (int i = tid; i < rt.rows * 32; i += threads) {
      const int col = i / 32, r = i % 32;
      if (n0 + r >= p.N) continue;
      float v = 0.0f;
      for (int w = w0; w < w0 + kw; ++w) v += ALL ? red[w][1][r] + red[w][0][r] : red[w][col][r];
      const int64_t at = static_cast<int64_t>(rt.row0 + col) * p.N + n0 + r;
      if (ALL)
        static_cast<uint16_t *>(p.out)[at] = out_bits<DT>(v);
      else
        static_cast<float *>(p.out)[at] = v;
    }
  }
}

// in[pos] = x[token of the pair at pos]: the rows of gate/up in the sort's order, a warp a row. The tensor-memory kernel
// reads each of them once per 128 weight rows, a box of rows a copy.
__global__ void __launch_bounds__(256) order_kernel(const uint4 *x, const int32_t *perm, int64_t pairs,
                                                    int pieces, int choices, uint4 *in) {
  griddep_launch_dependents();
  griddep_wait();
  const int64_t pos = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (pos >= pairs) return;
  const uint4 *from = x + static_cast<int64_t>(perm[pos] / choices) * pieces;
  uint4 *to = in + pos * pieces;
  for (int i = threadIdx.x & 31; i < pieces; i += 128) {
    uint4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + 32 * j < pieces) v[j] = from[i + 32 * j];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + 32 * j < pieces) to[i + 32 * j] = v[j];
  }
}

// fp16: the rows of h in the tiles that gate/up has marked. A row with values past the type's range (infinities in h, whose 32-bit
// values stand in `wide`) is written anew divided by 2^e, which brings its largest finite one below 2^15, and its factor is 2^e; every
// other row's factor is 1. What a small value of such a row loses is below 2^-39 of its largest. A block a tile; without a marked
// tile it writes the factors alone (a call of 16 rows 156.2 us with it, 154.8 without).
__global__ void __launch_bounds__(256)
    range_kernel(const RowTile *tiles, const int32_t *ntiles, uint16_t *h, const float *wide, int cols, float *factor) {
  griddep_launch_dependents();
  griddep_wait();
  if (static_cast<int>(blockIdx.x) >= *ntiles) return;
  const RowTile rt = tiles[blockIdx.x];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (!rt.flag) {
    for (int r = threadIdx.x; r < rt.rows; r += 256) factor[rt.row0 + r] = 1.0f;
    return;
  }
  for (int r = warp; r < rt.rows; r += 8) {
    const int64_t at = static_cast<int64_t>(rt.row0 + r) * cols;
    float top = 0.0f;
    for (int j = lane; j < cols; j += 32)
      if ((h[at + j] & 0x7FFFu) == 0x7C00u && !isinf(wide[at + j])) top = fmaxf(top, fabsf(wide[at + j]));
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    const int e = top > 0.0f ? static_cast<int>(__float_as_uint(top) >> 23) - 127 - 14 : 0;  // 2^(e + 14) <= top < 2^(e + 15)
    if (lane == 0) factor[rt.row0 + r] = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
    if (e == 0) continue;
    const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    for (int j = lane; j < cols; j += 32) {
      const uint16_t bits = h[at + j];
      const float v = (bits & 0x7FFFu) == 0x7C00u ? wide[at + j] : value_f32<kDtypeF16>(bits);
      h[at + j] = out_bits<kDtypeF16>(v * down);
    }
  }
}

// y[t] = sum over the token's choices of weight * output, in their order; a dropped choice adds nothing. FACTOR: the outputs of
// rows that range_kernel has divided are multiplied by their factors.
template <int DT, bool FACTOR>
__global__ void __launch_bounds__(256)
    combine_kernel(const float *part, const int32_t *inverse, const float *weights,
                   const float *factor, int64_t T, int K, int choices, uint16_t *y) {
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
    float4 a = *reinterpret_cast<const float4 *>(part + static_cast<int64_t>(pos) * K + c);
    float4 b = *reinterpret_cast<const float4 *>(part + static_cast<int64_t>(pos) * K + c + 4);
    if (FACTOR) {
      const float f = factor[pos];
      a.x *= f, a.y *= f, a.z *= f, a.w *= f;
      b.x *= f, b.y *= f, b.z *= f, b.w *= f;
    }
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

// The workspace: [error word][ntiles][outputs in 32 bits][h][perm][inverse][tiles]. Until the second product the outputs' place
// holds what the first one needs: the rows in order (tensor memory) and, fp16, the values of h past the type's range. The second
// product and the last pass need no perm: its place then holds the rows' factors (fp16).
struct ExpertsPlan {
  bool direct;  // no sort: each pair by itself, and a token's choices added in the second product
  bool tmem;
  int tile, max_tiles;
  size_t part, wide, h, perm, inverse, tiles, bytes;
};

ExpertsPlan experts_plan(int64_t T, int64_t K, int64_t I, int experts, int k, int g) {
  ExpertsPlan p;
  const int64_t pairs = T * k;
  // rows per tile: as many as an expert has on average, from the widths that the kernels have
  const int64_t mean = pairs / experts;
  // (pairs that are few beside the experts seldom share one: 2 tokens of 8 choices among 64 experts 26 us against 33 with
  // the sort, 4 tokens 44 against 42)
  p.direct = T == 1 || pairs <= experts / 4;
  p.tmem = !p.direct && mean >= kTmemRows && experts_tmem_takes(g);
  // (tensor memory, 64 / 128 rows a tile, 64 experts of 2048 x 1024, g = 128: 32 rows an expert 108 / 114 us, 48 rows 123 /
  // 121, 96 rows 181 / 152; g = 64, whose tiles of 128 rows take 64 k a chunk: 64 rows 164 / 182, 128 rows 256 / 251)
  p.tile = p.tmem ? (mean < (g % 128 == 0 ? 48 : 128) || g % 64 != 0 ? 64 : 128) : mean <= 8 ? 8 : mean <= 16 ? 16 : 32;
  p.max_tiles = static_cast<int>(p.direct ? pairs : max_row_tiles(pairs, experts, p.tile));
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  p.part = 256;
  p.wide = p.part + (p.tmem ? up(static_cast<size_t>(pairs) * K * 2) : 0);
  const size_t outputs = p.direct ? 0 : up(static_cast<size_t>(pairs) * K * 4);
  const size_t wide_end = p.direct ? 0 : p.wide - p.part + up(static_cast<size_t>(pairs) * I * 4);
  p.h = p.part + (outputs > wide_end ? outputs : wide_end);
  p.perm = p.h + up(static_cast<size_t>(pairs) * I * (p.direct ? 4 : 2));
  p.inverse = p.perm + up(static_cast<size_t>(pairs) * 4);
  p.tiles = p.inverse + up(static_cast<size_t>(pairs) * 4);
  p.bytes = p.tiles + up(static_cast<size_t>(p.max_tiles) * sizeof(RowTile));
  return p;
}

template <int DT, int NT, bool GATED, bool DIRECT, int NW>
cudaError_t launch_few(const Products &p, int tiles, cudaStream_t stream) {
  const int mode = p.g % 128 == 0 ? kTwo : p.g % kTK == 0 ? kBlock : kAny;
  auto kern = mode == kTwo     ? experts_kernel<DT, NT, GATED, kTwo, DIRECT, NW>
              : mode == kBlock ? experts_kernel<DT, NT, GATED, kBlock, DIRECT, NW>
                               : experts_kernel<DT, NT, GATED, kAny, DIRECT, NW>;
  constexpr int bytes = NW * Stage<NT>::kRing;
  static std::atomic<uint64_t> set[3];
  const cudaError_t e = allow_smem(kern, bytes, &set[mode]);
  if (e != cudaSuccess) return e;
  return launch_programmatic(kern, static_cast<int>(cdiv(p.slabs, NW / p.kw)) * tiles, 32 * NW, bytes, stream, p);
}

template <int DT, bool GATED>
cudaError_t launch_products(Products p, const ExpertsPlan &plan, int64_t T, int num_sms, cudaStream_t stream) {
  if (plan.tmem) return launch_experts_tmem(p, DT, GATED, plan.tile, num_sms, stream);
  const int tiles = plan.direct && !GATED ? static_cast<int>(T) : plan.max_tiles;
  // K is split over as many warps as fill the device a few times over, none with fewer than two steps (gate/up of 8 experts
  // of 4096 x 11008: unsplit 100 us, over 2 warps 103, over 8 124; one token's 64 slabs need all 16)
  const int64_t slabs = static_cast<int64_t>(p.slabs) * tiles;
  const int64_t steps = cdiv(p.KB, 2) * (plan.direct && !GATED ? p.choices : 1);
  const int most = plan.direct ? 16 : 8;
  p.kw = most;
  while (p.kw > 1 && (slabs * p.kw / 2 >= 48 * num_sms || steps < 2 * p.kw)) p.kw /= 2;
  if (plan.direct)
    return launch_few<DT, 1, GATED, true, 16>(p, tiles, stream);
  return plan.tile == 8    ? launch_few<DT, 1, GATED, false, 8>(p, tiles, stream)
         : plan.tile == 16 ? launch_few<DT, 2, GATED, false, 8>(p, tiles, stream)
                           : launch_few<DT, 4, GATED, false, 8>(p, tiles, stream);
}

template <int DT>
cudaError_t launch_dt(const ExpertsArgs &a, uint8_t *ws, const ExpertsPlan &plan, int num_sms, cudaStream_t stream) {
  RowPlan rows;
  rows.perm = reinterpret_cast<int32_t *>(ws + plan.perm);
  rows.inverse = reinterpret_cast<int32_t *>(ws + plan.inverse);
  rows.tiles = reinterpret_cast<RowTile *>(ws + plan.tiles);
  rows.ntiles = reinterpret_cast<int32_t *>(ws + 4);
  rows.err = reinterpret_cast<uint32_t *>(ws);
  cudaError_t e = cudaSuccess;
  if (!plan.direct) e = launch_row_plan(a.ids, a.T * a.k, a.experts, plan.tile, false, rows, stream);
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
    p.wide = reinterpret_cast<float *>(ws + plan.wide);
    p.plan = rows;
    p.err = rows.err;
    p.slabs = static_cast<int>(cdiv(N, plan.tmem ? kTN : kSlabRows));
    p.choices = a.k;
    p.ids = a.ids;
    p.weights = a.weights;
    p.experts = a.experts;
    p.kw = 1;
    p.gdiv = make_fastdiv(static_cast<uint32_t>(a.g));
    p.wait_limit = a.wait_limit ? a.wait_limit : kWaitLimitCycles;
    p.test_extra = a.test_timeout ? 1 : 0;
    return p;
  };
  const void *in = a.x;
  int64_t in_rows = a.T;
  if (plan.tmem) {  // the outputs' place holds the rows until the second product
    in = ws + plan.part;
    in_rows = a.T * a.k;
    e = launch_programmatic(order_kernel, static_cast<int>(cdiv(in_rows, 8)), 256, 0, stream,
                            static_cast<const uint4 *>(a.x), static_cast<const int32_t *>(rows.perm), in_rows,
                            static_cast<int>(a.K / 8), a.k, reinterpret_cast<uint4 *>(ws + plan.part));
    if (e != cudaSuccess) return e;
  }
  e = launch_products<DT, true>(products(in, in_rows, a.gate_up, 2 * a.I, a.K, ws + plan.h), plan, a.T, num_sms, stream);
  if (e != cudaSuccess) return e;
  if (plan.direct)
    return launch_products<DT, false>(products(ws + plan.h, a.T * a.k, a.down, a.K, a.I, a.y), plan, a.T, num_sms, stream);
  constexpr bool kRange = DT == kDtypeF16;
  float *factor = reinterpret_cast<float *>(rows.perm);
  if (kRange) {
    e = launch_programmatic(range_kernel, plan.max_tiles, 256, 0, stream, static_cast<const RowTile *>(rows.tiles),
                            static_cast<const int32_t *>(rows.ntiles), reinterpret_cast<uint16_t *>(ws + plan.h),
                            reinterpret_cast<const float *>(ws + plan.wide), static_cast<int>(a.I), factor);
    if (e != cudaSuccess) return e;
  }
  e = launch_products<DT, false>(products(ws + plan.h, a.T * a.k, a.down, a.K, a.I, ws + plan.part), plan, a.T, num_sms, stream);
  if (e != cudaSuccess) return e;
  return launch_programmatic(combine_kernel<DT, kRange>, static_cast<int>(cdiv(a.T * (a.K / 8), 256)), 256, 0, stream,
                             reinterpret_cast<const float *>(ws + plan.part), static_cast<const int32_t *>(rows.inverse), a.weights,
                             static_cast<const float *>(factor), a.T, static_cast<int>(a.K), a.k, static_cast<uint16_t *>(a.y));
}

}  // namespace

size_t experts_workspace_bytes(int64_t T, int64_t K, int64_t I, int experts, int k, int g) {
  return experts_plan(T, K, I, experts, k, g).bytes;
}

cudaError_t launch_experts(const ExpertsArgs &a, void *workspace, int num_sms, cudaStream_t stream) {
  const ExpertsPlan plan = experts_plan(a.T, a.K, a.I, a.experts, a.k, a.g);
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  return a.dtype == kDtypeBf16 ? launch_dt<kDtypeBf16>(a, ws, plan, num_sms, stream)
                               : launch_dt<kDtypeF16>(a, ws, plan, num_sms, stream);
}

}  // namespace w4
