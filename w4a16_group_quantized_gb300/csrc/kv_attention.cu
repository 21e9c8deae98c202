// w4_kv_attention: a few query rows of each sequence over the paged cache of e4m3 codes.
//
// For a sequence and key head the n query rows of the r query heads that share it are n * r rows (row = j * r + head), taken 16
// at a time (an item). For a tile of 16 keys, which lies in one page: S = q . codes, s = S * (k scale * softmax scale *
// log2 e) + log2(v scale / unit), a row's running maximum m, w = 2^(s - m) in fp16, O += w . codes, l += (sum of w) / (v scale /
// unit): with the page's scale of the values inside the weight no product needs a scale of its own. The sum is that of the
// weights as they were rounded, by a product with ones, so that an output is an average of values. m may lag behind by 2^5 as
// a weight, so that O is rescaled a few times in an item.
// O is in units of `unit`, a warp's own: the power of two below the largest scale that its lookups, of 32 tiles each, have found
// in the item so far (O is rescaled where it grows). Scales from 2^-8 units up go into the weights, smaller ones and those that
// are not positive and finite go by a product of their own, in fp32. The weights are kept 2^10 times larger than 2^(s - m): 2^15
// at most; m is at most 2 above a row's largest exp(score) and a page's scale 2^8 below it, so that fp16's smallest step
// loses at most 2^-26 of that exp(score), whichever pages' scales stand beside each other.
//
// The products are register-operand ones (mma.sync m16n8k16, fp16 operands, fp32 sums): e4m3 codes are exact in fp16, and so
// are q's values (bf16 rows times a power of two that keeps them within fp16's range). S has the rows on its M side and the
// keys on its N side, so that its fragments are the second product's as they stand. With up to 8 rows (ROWS 8) that product is
// turned round, values on the M side, rows on the N side: half the products, half the sums.
//
// The tiles of all items in order are dealt out evenly, a stretch to each of the device's warps, so that sequences of unlike
// lengths load it evenly (an item counts kItemCost tiles more for what it costs to begin); a warp works alone, with a ring of its
// own in shared memory (cp.async, whole lines of 128 bytes, zeros past the sequence's end): no barriers. What a lane reads
// follows from the fragments: of key 8 u + lane / 4 the quarter of the head that its place in the quad has, in 16-byte
// pieces; of keys 2 t, 2 t + 1 and those plus 8 (t = lane % 4) an eighth of the head, whose codes of two neighbouring keys are
// put side by side by byte permutes. The pieces of a line are exchanged so that these reads meet no bank twice.
// Items cut between warps leave parts (O / l, m, l) in the workspace, one for a block whose warps are all within one item; a second
// launch adds them in order. Few items go to a block each instead, whose warps share the item, where that is quicker.
//
// Measured (us a call within a graph; heads of 128, one query): 128 sequences of 8192 keys, 64 / 8 heads 337 (2.15 GB: 6.4 TB/s,
// 0.94 of a copy's rate); 48 of up to 8000 29.9, four queries 50; one of 1003 keys, 32 / 32 heads 10.0, of 8000 20.6; 100 keys
// 4.5. What long batches wait for is memory; short ones some 12 us beside it: launches, the dealing (1 to 2), a first lookup
// (1.5), the first tiles of all warps at once (1.4 to 4), sums (1.8) and their adding. With four queries it is a tile's
// arithmetic, 0.9 us a warp, most of it the codes' conversion and dependent instructions (issue slots 36%, tensor pipe 26%); two tiles
// at a time, with twice as many independent ones, took as long (55), as did more sums a row or more warps with fewer registers.
#include <atomic>
#include <type_traits>

#include "e4m3.cuh"
#include "gemm_common.cuh"
#include "internal.h"
#include "mma.cuh"
#include "ptx.cuh"

namespace w4 {
namespace {

using namespace detail;

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kItemCost = 4;      // what beginning an item costs, in tiles
constexpr int kSoloTiles = 6;     // what adding parts takes, in tiles of a warp
constexpr float kLog2e = 1.4426950408889634f;
// log2 of how far a score may pass the maximum in use, of the least scale in units that goes into the weights, and of what the
// weights are raised by.
constexpr float kSlack = 5.0f, kFold = -8.0f, kRaise = 10.0f;
constexpr float kLeastUnit = -126.0f;  // log2

// How `units` are dealt out to warps: the first unit of each one's stretch is quotient * w + remainder * w / workers.
struct Deal {
  uint32_t quotient, remainder, workers;  // workers <= 2^12
  __device__ __forceinline__ int start(uint32_t w) const {
    w = min(w, workers);
    return static_cast<int>(quotient * w + remainder * w / workers);
  }
  // The warp in whose stretch a unit lies.
  __device__ __forceinline__ int holder(int unit) const {
    // (right to a warp or two)
    int w = static_cast<int>(static_cast<float>(unit) / (static_cast<float>(quotient) + static_cast<float>(remainder) / static_cast<float>(workers)));
    while (w > 0 && start(w) > unit) --w;
    while (start(w + 1) <= unit) ++w;
    return w;
  }
};

// An item that begins in a warp's stretch and ends in another's: what the second launch adds. Positions are in units: an item's are
// kItemCost ones for its beginning and one for each tile (2^30 in all at most: 64-bit divisions and conversions would cost a call
// some 2 us, by a pipe of some 40 cycles an instruction).
struct CutItem {
  int32_t b, j;        // sequence and item of it
  int32_t first, last; // the warps that hold the item's first and last tile
  int32_t warps;       // of a block that have stretches
  int32_t begin, end;  // its tiles
  Deal deal;
};

struct KvParams {
  const uint16_t *q;
  const uint8_t *k_cache, *v_cache;
  const float *k_scale, *v_scale;
  const int32_t *table, *lens;
  uint16_t *out;
  int32_t *workers;  // how many warps have a stretch
  int32_t *cut;      // [workers], or [items] by_item: whether cuts has an item
  CutItem *cuts;
  float *sums;     // [2 * warps]: O / l [rows][D], m [rows], l [rows], padded to 16 bytes, of a stretch's first and last item
  int64_t ldq, ldo, pages;
  int batch, n, max_pages, k_heads, head_dim, page, r, row_tiles, rows, items;  // items of a sequence
  int by_item;     // few items: an entry of cut and cuts for each, else for each warp
  float scale;
  FastDiv page_div, r_div, row_tiles_div;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
// Whether one of the four codes of a word is NaN (0x7F or 0xFF).
__device__ __forceinline__ bool any_nan_code(uint32_t w) { return __vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu) != 0; }

// Warps of a block, with heads of up to d values and up to `rows` rows an item: as many as have the registers, but for a few words at
// most (heads of 64, us: 128 x 8000 keys, 24 / 8 heads 205 with 12 warps, 180 with 16; 64 x 4000, four queries 83 with 8, 69 with 12, 66 with
// 16. Heads of 128: 16 spill a tile's operands, 350 -> 686; 12 for 16 rows take as long as 8).
constexpr int warps_of(int d, int rows) { return d <= 64 ? 16 : rows <= 8 ? 12 : 8; }

// D: head_dim rounded up to 64 or 128. ROWS: of an item, up to 8 or up to 16.
template <int D, int ROWS>
struct KvCfg {
  static constexpr int kWarps = warps_of(D, ROWS);
  static constexpr int kStages = 4;
  static constexpr int kPieces = D / 64;                 // 16-byte pieces of a key in a lane
  static constexpr int kVBytes = D / 8;                  // bytes of a value row in a lane
  static constexpr int kPart = 16 * D;                   // bytes of a tile's keys, and of its values
  static constexpr int kTileBytesWarp = 2 * kPart;
  static constexpr int kRing = kStages * kTileBytesWarp;
  static constexpr int kSumRow = D + 4;                  // floats of a row of a warp's sums in shared memory
  static constexpr int kSumBytes = kWarps * ROWS * kSumRow * 4;
  static constexpr int kInfo = kWarps * 64 * 16;         // what the lookups found: two times 32 tiles a warp
  static constexpr int kSmem = kInfo + (kWarps * kRing > kSumBytes ? kWarps * kRing : kSumBytes);
};

// Where piece c of key (or value row) `key` of a tile lies in shared memory. Lines of 128 bytes, eight pieces each: a key, or two of 64
// bytes. Eight lanes that read at once have, of keys, pieces t of keys g and g + 1, of values pieces g and g + 1 (or one
// of them) of keys 2 t.
template <int D>
__device__ __forceinline__ int key_place(int key, int c) {
  return D == 128 ? key * 128 + 16 * (c ^ (key & 1) << 2) : key * 64 + 16 * c;
}
template <int D>
__device__ __forceinline__ int value_place(int key, int c) {
  return D == 128 ? key * 128 + 16 * (c ^ (key >> 1 & 3) << 1) : (key >> 1) * 128 + 16 * (((key & 1) * 4 + c) ^ (key >> 1 & 3) << 1);
}

// The place of row i of item j of sequence b in q or out.
__device__ __forceinline__ int64_t row_at(const KvParams &p, int b, int j, int i, int64_t ld) {
  const int h = p.row_tiles_div.div(j), rho = (j - h * p.row_tiles) * 16 + i;
  const int token = p.r_div.div(rho);
  return (static_cast<int64_t>(b) * p.n + token) * ld + static_cast<int64_t>(h * p.r + rho - token * p.r) * p.head_dim;
}

template <int DT>
__device__ __forceinline__ uint4 eight_out(const float (&v)[8]) {
  return make_uint4(out_bits2<DT>(v[0], v[1]), out_bits2<DT>(v[2], v[3]), out_bits2<DT>(v[4], v[5]), out_bits2<DT>(v[6], v[7]));
}

// The least maximum of a row that has seen a key: all its scores may be -inf, which is not the same as seeing nothing.
constexpr float kLeastMax = -3.402823466e38f;

// 1 / l of all of a row: 0 where it saw nothing, NaN where all that it saw scores -inf.
__device__ __forceinline__ float over_sum(float l, float m) { return l != 0.0f ? 1.0f / l : m == -INFINITY ? 0.0f : NAN; }

// Parts of a row are kept as O / l, in fp32 whatever their units, with l times 2^-20: sums of O / l times that stay far from fp32's ends. 1 / l of
// a part, to a unit or two; 0 where it has no weight.
constexpr float kPartSum = 0x1p-20f;
__device__ __forceinline__ float over_part(float l) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(l));
  return l == 0.0f ? 0.0f : y;
}

// Which row the sums o[s][i] are of, and which value of it.
template <int ROWS>
__device__ __forceinline__ int row_of(int s, int i) {
  return ROWS == 16 ? threadIdx.x % 32 / 4 + 8 * (s % 2) : threadIdx.x % 4 * 2 + i;
}
template <int D, int ROWS>
__device__ __forceinline__ int value_of(int s, int i) {
  return ROWS == 16 ? (threadIdx.x % 4 * 2 + i) * (D / 8) + s / 2 : threadIdx.x % 32 / 4 * (D / 8) + s;
}

// The second product of a tile, w the weights' fragments, added to o; or, SOME, f times it to the rows lo .. hi - 1 alone.
template <int D, int ROWS, bool SOME>
__device__ __forceinline__ void add_values(float (&o)[D / 8 * (ROWS / 8)][2], const uint32_t (&v)[4][D / 32],
                                           const uint32_t (&w)[ROWS / 4], float f, int lo, int hi) {
#pragma unroll
  for (int x = 0; x < D / 32; ++x) {
    uint32_t b0[4], b1[4];  // keys 2 t, 2 t + 1 and those plus 8, values 4 x .. 4 x + 3 of the lane's
    e4m3x4_f16x4(__byte_perm(v[0][x], v[1][x], 0x5140), &b0[0], &b0[1]);
    e4m3x4_f16x4(__byte_perm(v[0][x], v[1][x], 0x7362), &b0[2], &b0[3]);
    e4m3x4_f16x4(__byte_perm(v[2][x], v[3][x], 0x5140), &b1[0], &b1[1]);
    e4m3x4_f16x4(__byte_perm(v[2][x], v[3][x], 0x7362), &b1[2], &b1[3]);
    // 16 rows: value 4 x + e of row g in set s, of row g + 8 in set s + 1, columns 2 t, 2 t + 1; 8 rows: value 4 x + e in set s, the
    // next one in set s + 1, rows 2 t, 2 t + 1
#pragma unroll
    for (int e = 0; e < 4; e += ROWS == 16 ? 1 : 2) {
      const int s = ROWS == 16 ? 2 * (4 * x + e) : 4 * x + e;
      float d[4] = {};
      if (!SOME) d[0] = o[s][0], d[1] = o[s][1], d[2] = o[s + 1][0], d[3] = o[s + 1][1];
      if (ROWS == 16)
        mma_16816<kDtypeF16>(d, w[0], w[ROWS / 4 - 2], w[1], w[ROWS / 4 - 1], b0[e], b1[e]);
      else
        mma_16816<kDtypeF16>(d, b0[e], b0[(e + 1) % 4], b1[e], b1[(e + 1) % 4], w[0], w[1]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = row_of<ROWS>(s + i / 2, i % 2);
        if (!SOME)
          o[s + i / 2][i % 2] = d[i];
        else if (row >= lo && row < hi)
          o[s + i / 2][i % 2] = fmaf(f, d[i], o[s + i / 2][i % 2]);
      }
    }
  }
}

template <int DT, int D, int ROWS>
__global__ void __launch_bounds__(32 * KvCfg<D, ROWS>::kWarps, 1) kv_attention_kernel(const __grid_constant__ KvParams p) {
  using C = KvCfg<D, ROWS>;
  constexpr int W = C::kWarps, S = C::kStages, RR = ROWS / 8;  // RR: rows of a lane in S
  constexpr int NO = D / 8 * RR;  // sets of two sums: 16 rows: rows g, g + 8 x values; 8 rows: values x rows 2 t, 2 t + 1
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int upto[32 * W];  // units of a warp's sequences up to and with the thread's
  __shared__ float row_m[W][ROWS], row_l[W][ROWS];
  const int warp = __shfl_sync(kAll, threadIdx.x / 32, 0), lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  // what the lookups found of a tile's page: k scale, log2 of the v scale in units as far as it goes into the weights, log2 of the unit, and the rest
  // of the scale (1, or what the products are to be multiplied with)
  float4 *info = reinterpret_cast<float4 *>(smem) + warp * 64;
  const uint32_t ring = smem_u32(smem + C::kInfo) + warp * C::kRing;
  griddep_launch_dependents();
  griddep_wait();

  // ------------------------------------------------- the warp's stretch of the tiles
  const int head_dim = p.head_dim;
  const bool exact = head_dim == D;
  const int most = p.max_pages * p.page;
  auto tiles_of = [&](int b) { return max((min(p.lens[b], most) + 15) / 16, 1); };  // (a sequence without keys still has an output)
  // The warp's stretch, its first tile (at: its unit) with the sequence and item, and whether all the block's tiles are of one
  // item, whose sums are then added here
  int from, to, at, block_from, block_to, one_begin;
  int b = 0, j = 0, tile = 0, tiles = 1, one_b, one_j, one_tiles, me = 0, warps = W;
  bool together, solo = p.batch * p.items <= gridDim.x;
  Deal deal = {};
  if (solo) {
    // few items: a block each, and nothing to add afterwards, unless the longest takes longer that way, by more than the adding (as
    // long as kSoloTiles tiles of a warp), than 1.2 times all of them dealt out evenly (us, whole / dealt out: one sequence of
    // 1003 keys, 32 heads 9.8 / 10.3, of 1500 12.5 / 11.0; 8 of 2000, 8 key heads 17.3 / 19.0; 16 of 1003 12.8 / 14.8)
    int longest = 0, all = 0;  // in tiles, and in 16 of them
    for (int i = lane; i < p.batch; i += 32) {
      const int t16 = tiles_of(i);
      longest = max(longest, t16);
      all += t16 / 16;
    }
    solo = static_cast<int64_t>(__reduce_max_sync(kAll, longest) - W * kSoloTiles) * (5 * gridDim.x) <=
           static_cast<int64_t>(__reduce_add_sync(kAll, all)) * (6 * 16 * p.items);
  }
  if (solo) {
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.workers = 0;
    if (blockIdx.x >= p.batch * p.items) return;
    one_b = b = blockIdx.x / p.items;
    one_j = j = blockIdx.x - b * p.items;
    one_tiles = tiles = tiles_of(b);
    one_begin = block_from = 0;
    block_to = tiles;
    at = from = tile = tiles / W * warp + tiles % W * warp / W;
    to = tiles / W * (warp + 1) + tiles % W * (warp + 1) / W;
    together = true;
  } else {
    // the units of the sequences up to and with each: for few, in each warp's lanes; else by warps, and within each by threads
    const bool few = p.batch <= 32;
    const int share = few ? 1 : (p.batch + 32 * W - 1) / (32 * W);  // sequences a thread adds up
    const int sb0 = few ? lane : threadIdx.x * share;
    const int lane_tiles = few && lane < p.batch ? tiles_of(lane) : 0;
    int sum = 0;
    for (int sb = sb0; sb < min(sb0 + share, p.batch); ++sb) sum += ((few ? lane_tiles : tiles_of(sb)) + kItemCost) * p.items;
    const int mine = sum;
#pragma unroll
    for (int i = 1; i < 32; i *= 2) {
      const int x = __shfl_up_sync(kAll, sum, i);
      if (lane >= i) sum += x;
    }
    int warp_sum = 0, warp_mine = 0;  // of the warps up to and with the lane's, and of that one
    if (!few) {
      upto[threadIdx.x] = sum;
      __syncthreads();
      warp_sum = warp_mine = lane < W ? upto[32 * lane + 31] : 0;
#pragma unroll
      for (int i = 1; i < 16; i *= 2) {
        const int x = __shfl_up_sync(kAll, warp_sum, i);
        if (lane >= i) warp_sum += x;
      }
    }
    const int total = __shfl_sync(kAll, few ? sum : warp_sum, few ? 31 : W - 1);
    // fewer warps where there is little to do (one sequence of 8000 keys, 8 key heads, us: 17.3 with stretches of 8 units at least, 15.2
    // with 4, 14.2 with 2, 14.1 with 1, which gains nothing elsewhere either and costs up to one)
    deal.workers = min(W * gridDim.x, static_cast<uint32_t>(max(total / 2, 1)));
    deal.quotient = total / deal.workers;
    deal.remainder = total - deal.quotient * deal.workers;
    // (those that there are, in all blocks alike)
    warps = static_cast<int>((deal.workers + gridDim.x - 1) / gridDim.x);
    me = warp < warps ? blockIdx.x * warps + warp : gridDim.x * W;
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.workers = static_cast<int32_t>(deal.workers);
    from = deal.start(me), to = deal.start(me + 1);
    block_from = deal.start(blockIdx.x * warps), block_to = deal.start((blockIdx.x + 1) * warps);

    // the sequence and item that a unit lies in, and the unit within the item
    auto find = [&](int unit, int *fb, int *fj, int *ftiles) {
      int rest;
      if (few) {
        *fb = __ffs(__ballot_sync(kAll, sum > unit)) - 1;
        rest = unit - __shfl_sync(kAll, sum - mine, *fb);
        *ftiles = __shfl_sync(kAll, lane_tiles, *fb);
      } else {
        const int of = __ffs(__ballot_sync(kAll, lane < W && warp_sum > unit)) - 1;
        rest = unit - __shfl_sync(kAll, warp_sum - warp_mine, of);
        const int within = upto[32 * of + lane];
        const int at = __ffs(__ballot_sync(kAll, within > rest)) - 1;
        const int before = __shfl_sync(kAll, within, max(at - 1, 0));
        rest -= at > 0 ? before : 0;
        const int lo = 32 * of + at;
        for (*fb = lo * share;; ++*fb) {
          *ftiles = tiles_of(*fb);
          const int units = (*ftiles + kItemCost) * p.items;
          if (rest < units || *fb + 1 >= p.batch) break;
          rest -= units;
        }
      }
      *fj = static_cast<uint32_t>(rest) / static_cast<uint32_t>(*ftiles + kItemCost);
      return rest - *fj * (*ftiles + kItemCost);
    };
    // (every warp finds the block's first item for itself: no more barriers)
    together = false;
    one_b = one_j = one_tiles = 0;
    one_begin = 0;
    if (block_from < block_to) {
      const int off = find(block_from, &one_b, &one_j, &one_tiles);
      one_begin = block_from - off + kItemCost;
      together = block_to > one_begin && block_to <= one_begin + one_tiles + kItemCost;
    }
    at = to;
    if (from < to) {
      int off;
      if (together) {
        b = one_b, j = one_j, tiles = one_tiles;
        off = from - one_begin + kItemCost;
      } else {
        off = find(from, &b, &j, &tiles);
      }
      tile = max(off - kItemCost, 0);
      at = from + max(kItemCost - off, 0);
      if (tile >= tiles) tile = 0, at = to;  // (what is left of the block's stretch is the next item's beginning)
    }
  }
  bool cut = false;

  // ---------------------------------------------------------------- copies
  // The tile that is copied next, and what the lookups found for up to 32 tiles of its item (sent: tiles so far)
  int cb = b, cj = j, ct = tile, ctiles = tiles, ckeys = 0, found = 0, first = 0, book = 0, next_book = 0;
  int cat = at;
  uint32_t off_lo = 0, off_hi = 0;  // this lane's tile: offset in the cache, in 16 bytes; all ones: no page
  int sent = 0;
  uint32_t infos = 0;  // the places in `info` of the tiles on their way, 8 bits each (255: no page), the next one's lowest
  // a lane copies piece lane_c of keys lane_key, lane_key + kCopyKeys, ...
  constexpr int kCopyKeys = 512 / D;
  const int lane_key = lane * 16 / D, lane_c = lane % (D / 16);
  const int lane_off = lane_key * head_dim + lane_c * 16;
  // what the scales of the last lookup become: done after its first copies have been sent
  float found_ks = 0.0f, found_vs = 0.0f;
  bool pending = false;
  float unit_found = kLeastUnit;  // of the item so far
  auto keep_scales = [&]() {
    if (!pending) return;
    pending = false;
    const float size = fabsf(found_vs);
    const bool finite = size < INFINITY;
    const int exponent = static_cast<int>(__reduce_max_sync(kAll, finite ? __float_as_uint(size) >> 23 : 0u));
    unit_found = fmaxf(unit_found, static_cast<float>(exponent - 127));
    const float in_units = log2f(size) - unit_found;
    const bool inside = in_units >= kFold && finite;
    const float rest = inside ? copysignf(1.0f, found_vs) : finite ? copysignf(ex2(in_units), found_vs) : found_vs;
    info[(book + lane) % 64] = make_float4(found_ks, inside ? in_units : 0.0f, unit_found, rest);
    __syncwarp();
  };
  auto send = [&]() {
    uint32_t place = 255;
    __syncwarp();  // the place's last tile has been read
    if (cat < to) {
      if (ct - first >= found) {  // look up the next 32 tiles of the item
        keep_scales();
        if (ct == 0 || found == 0) ckeys = min(p.lens[cb], most), unit_found = kLeastUnit;
        first = ct;
        found = min(32, ctiles - ct);
        // (places go round: when it comes to a lookup, at most S tiles of the ones before are still to be worked on)
        book = next_book;
        next_book = (book + found) % 64;
        int64_t off = -1;
        found_vs = 0.0f;
        if (lane < found) {
          const int key0 = (ct + lane) * 16;
          const int pi = p.page_div.div(key0), h = p.row_tiles_div.div(cj);
          int pg = -1;
          if (pi < p.max_pages) pg = p.table[static_cast<int64_t>(cb) * p.max_pages + pi];
          if (pg >= 0 && pg < p.pages) {
            const int64_t ph = static_cast<int64_t>(pg) * p.k_heads + h;
            found_ks = p.k_scale[ph], found_vs = p.v_scale[ph];
            off = (ph * p.page + key0 - pi * p.page) * (head_dim / 16);
          }
        }
        pending = true;
        off_lo = static_cast<uint32_t>(off);
        off_hi = static_cast<uint32_t>(off >> 32);
      }
      const uint32_t lo = __shfl_sync(kAll, off_lo, ct - first), hi = __shfl_sync(kAll, off_hi, ct - first);
      if (hi != 0xffffffffu) {
        place = static_cast<uint32_t>(book + ct - first) % 64;
        const int64_t base = static_cast<int64_t>((static_cast<uint64_t>(hi) << 32 | lo) * 16);
        const uint32_t to = ring + sent % S * C::kTileBytesWarp;
        const uint8_t *k = p.k_cache + base + lane_off, *v = p.v_cache + base + lane_off;
        const int here = ckeys - ct * 16;  // keys of the tile
        if (exact && here >= 16) {
#pragma unroll
          for (int i = 0; i < 16; i += kCopyKeys) cp_async16(to + key_place<D>(lane_key + i, lane_c), k + i * D);
#pragma unroll
          for (int i = 0; i < 16; i += kCopyKeys) cp_async16(to + C::kPart + value_place<D>(lane_key + i, lane_c), v + i * D);
        } else {
#pragma unroll
          for (int i = 0; i < 16; i += kCopyKeys) {
            const bool there = lane_key + i < here && 16 * lane_c < head_dim;
            cp_async16_zfill(to + key_place<D>(lane_key + i, lane_c), there ? k + i * head_dim : p.k_cache, there ? 16u : 0u);
            cp_async16_zfill(to + C::kPart + value_place<D>(lane_key + i, lane_c), there ? v + i * head_dim : p.v_cache,
                             there ? 16u : 0u);
          }
        }
      }
      ++cat;
      if (++ct == ctiles) {  // the next item
        ct = first = found = 0;
        cat += kItemCost;
        if (++cj == p.items) {
          cj = 0;
          if (++cb < p.batch) ctiles = tiles_of(cb);
        }
      }
    }
    infos |= place << (8 * (S - 1));
    ++sent;
    cp_commit();
  };

  // ------------------------------------------------------------ products
  uint32_t q[D / 16][2 * RR];  // a step's pairs: (row g, pair 0), (row g, pair 1) and, of 16 rows, those of row g + 8
  float o[NO][2], m[RR], l[2], mul[RR], unit = kLeastUnit;  // (l: of the rows of o; m: the maximum in use less kRaise; unit: log2 of it)
  int sees[RR], least = 0, len = 0;
  auto begin_item = [&]() {
    const int rt = j - p.row_tiles_div.div(j) * p.row_tiles;
    len = max(p.lens[b], 0);
    const int keys = min(len, most);
    least = keys;
#pragma unroll
    for (int i = 0; i < RR; ++i) {
      const int rho = rt * 16 + g + 8 * i;
      const bool live = rho < p.n * p.r;
      const int token = p.r_div.div(rho);
      sees[i] = live ? min(max(len - p.n + token + 1, 0), keys) : keys;
      least = min(least, sees[i]);
      // values (t + 4 c) * 16 .. + 15 of the row: four steps' pairs
      uint4 w[C::kPieces][2];
      float high = 0.0f;
      const uint16_t *src = p.q + row_at(p, b, j, g + 8 * i, p.ldq);
#pragma unroll
      for (int c = 0; c < C::kPieces; ++c)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int d = (t + 4 * c) * 16 + 8 * e;
          w[c][e] = live && d < head_dim ? *reinterpret_cast<const uint4 *>(src + d) : make_uint4(0, 0, 0, 0);
        }
      mul[i] = p.scale * kLog2e;
      float up = 1.0f;
      if (DT == kDtypeBf16) {
#pragma unroll
        for (int c = 0; c < C::kPieces; ++c)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t v[4] = {w[c][e].x, w[c][e].y, w[c][e].z, w[c][e].w};
#pragma unroll
            for (int x = 0; x < 4; ++x)
              high = fmaxf(high, fmaxf(fabsf(value_f32<DT>(v[x] & 0xffffu)), fabsf(value_f32<DT>(v[x] >> 16))));
          }
        high = fmaxf(high, __shfl_xor_sync(kAll, high, 1));
        high = fmaxf(high, __shfl_xor_sync(kAll, high, 2));
        // the row's largest value to [2^10, 2^11): products with codes stay far from fp32's ends, and what falls below
        // fp16's smallest step, 2^-24, is below 2^-34 of the largest
        const int e = static_cast<int>(__float_as_uint(high) >> 23);
        if (e != 0 && e != 255) up = __uint_as_float(static_cast<uint32_t>(min(max(137 - e, -126), 126) + 127) << 23);
        mul[i] /= up;
      }
#pragma unroll
      for (int c = 0; c < C::kPieces; ++c)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t v[4] = {w[c][e].x, w[c][e].y, w[c][e].z, w[c][e].w};
#pragma unroll
          for (int x = 0; x < 4; ++x) {  // step 4 c + 2 e + x / 2, pair x % 2
            uint32_t bits = v[x];
            if (DT == kDtypeBf16) bits = half2_bits(value_f32<DT>(v[x] & 0xffffu) * up, value_f32<DT>(v[x] >> 16) * up);
            q[4 * c + 2 * e + x / 2][2 * i + x % 2] = bits;
          }
        }
      m[i] = -INFINITY;
    }
    least = static_cast<int>(__reduce_min_sync(kAll, least));
    unit = kLeastUnit;
    l[0] = l[1] = 0.0f;
#pragma unroll
    for (int x = 0; x < NO; ++x) o[x][0] = o[x][1] = 0.0f;
  };
  for (int i = 0; i < S - 1; ++i) {
    infos >>= 8;
    send();
  }
  begin_item();  // (also for a warp without tiles: sums of nothing)
  keep_scales();
  for (int i = 0; at < to; ++i) {
    if (i > 0 && tile == 0) begin_item();
    infos >>= 8;
    send();  // (its place held tile i - 1, which is done)
    keep_scales();
    cp_wait<S - 1>();
    __syncwarp();  // (every lane has waited for what it copied)
    const uint32_t mine = infos & 0xffu;
    if (mine != 255u) {
      const float4 st = info[mine];
      const int key0 = tile * 16;
      const uint32_t kt = ring + i % S * C::kTileBytesWarp, vt = kt + C::kPart;
      float s[2][4] = {};
#pragma unroll
      for (int c = 0; c < C::kPieces; ++c) {
        const uint4 k0 = lds128(kt + key_place<D>(g, t + 4 * c)), k1 = lds128(kt + key_place<D>(g + 8, t + 4 * c));
        const uint32_t x[4] = {k0.x, k0.y, k0.z, k0.w}, y[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t x0, x1, y0, y1;
          e4m3x4_f16x4(x[w], &x0, &x1);
          e4m3x4_f16x4(y[w], &y0, &y1);
          const uint32_t(&f)[2 * RR] = q[4 * c + w];
          const uint32_t f2 = RR == 2 ? f[2 * RR - 2] : 0u, f3 = RR == 2 ? f[2 * RR - 1] : 0u;
          mma_16816<kDtypeF16>(s[0], f[0], f2, f[1], f3, x0, x1);
          mma_16816<kDtypeF16>(s[1], f[0], f2, f[1], f3, y0, y1);
        }
      }
      // values: words of the four keys
      uint32_t v[4][C::kVBytes / 4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if constexpr (C::kVBytes == 16) {
          const uint4 x = lds128(vt + value_place<D>(2 * t + c % 2 + c / 2 * 8, g));
          v[c][0] = x.x, v[c][1] = x.y, v[c][2] = x.z, v[c][3] = x.w;
        } else {
          asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v[c][0]), "=r"(v[c][1]) : "r"(vt + value_place<D>(2 * t + c % 2 + c / 2 * 8, g / 2) + g % 2 * 8) : "memory");
        }
      }
      const bool border = key0 + 16 > least;  // some row does not see all of the tile
      float top[RR];
#pragma unroll
      for (int r2 = 0; r2 < RR; ++r2) {
        const float f = st.x * mul[r2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int e = 2 * r2; e < 2 * r2 + 2; ++e) s[u][e] = fmaf(s[u][e], f, st.y);
      }
      if (border) {
#pragma unroll
        for (int r2 = 0; r2 < RR; ++r2)
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (key0 + 8 * u + 2 * t + e >= sees[r2]) s[u][2 * r2 + e] = -INFINITY;
      }
#pragma unroll
      for (int r2 = 0; r2 < RR; ++r2)
        top[r2] = fmaxf(fmaxf(s[0][2 * r2], s[0][2 * r2 + 1]), fmaxf(s[1][2 * r2], s[1][2 * r2 + 1]));
#pragma unroll
      for (int x = 1; x < 4; x *= 2)
#pragma unroll
        for (int r2 = 0; r2 < RR; ++r2) top[r2] = fmaxf(top[r2], __shfl_xor_sync(kAll, top[r2], x));
      // (-inf + 15 is below any score: a row's first tile sets its maximum)
      if (__any_sync(kAll, top[0] > m[0] + (kSlack + kRaise) || top[RR - 1] > m[RR - 1] + (kSlack + kRaise) || st.z != unit)) {
        const float move = ex2(unit - st.z);
        unit = st.z;
        float alpha[RR];
#pragma unroll
        for (int r2 = 0; r2 < RR; ++r2) {
          const float now = top[r2] > m[r2] + (kSlack + kRaise) ? top[r2] - kRaise : m[r2];  // (a row's own scores alone say when)
          alpha[r2] = now == m[r2] ? 1.0f : ex2(m[r2] - now);
          m[r2] = now;
        }
        const float a0 = ROWS == 16 ? alpha[0] : __shfl_sync(kAll, alpha[0], 8 * t);
        const float a1 = ROWS == 16 ? alpha[RR - 1] : __shfl_sync(kAll, alpha[0], 8 * t + 4);
        l[0] *= a0, l[1] *= a1;
        const float o0 = a0 * move, o1 = a1 * move;
#pragma unroll
        for (int x = 0; x < NO; ++x) o[x][0] *= ROWS == 16 && x % 2 ? o1 : o0, o[x][1] *= ROWS == 16 && x % 2 == 0 ? o0 : o1;
      }
#pragma unroll
      for (int r2 = 0; r2 < RR; ++r2) {
        const float base = m[r2] == -INFINITY ? 0.0f : m[r2];  // (nothing seen yet: weights of 0)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int e = 2 * r2; e < 2 * r2 + 2; ++e) s[u][e] = ex2(s[u][e] - base);
        if (key0 < sees[r2]) m[r2] = fmaxf(m[r2], kLeastMax);
      }
      uint32_t w[2 * RR];  // as q's: (row g, keys 2 t ..), (row g, those plus 8), row g + 8
#pragma unroll
      for (int r2 = 0; r2 < RR; ++r2) {
        w[2 * r2] = half2_bits(s[0][2 * r2], s[0][2 * r2 + 1]);
        w[2 * r2 + 1] = half2_bits(s[1][2 * r2], s[1][2 * r2 + 1]);
      }
      {
        // l: the sum of the weights as they were rounded, by a product with ones
        constexpr uint32_t kOnes = 0x3C003C00u;
        const float per_unit = ex2(-st.y);
        float d[4] = {};
        if (ROWS == 16)
          mma_16816<kDtypeF16>(d, w[0], w[ROWS / 4 - 2], w[1], w[ROWS / 4 - 1], kOnes, kOnes);
        else
          mma_16816<kDtypeF16>(d, kOnes, kOnes, kOnes, kOnes, w[0], w[1]);
        l[0] = fmaf(d[0], per_unit, l[0]);
        l[1] = fmaf(d[ROWS == 16 ? 2 : 1], per_unit, l[1]);
      }
      bool odd = st.w != 1.0f;
      if (border && !odd) {
        // 0 * NaN is NaN: whether the tile, of which some rows do not see all, holds NaN
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int x = 0; x < C::kVBytes / 4; ++x) odd |= any_nan_code(v[c][x]);
        odd = __any_sync(kAll, odd);
      }
      if (!odd) {
        add_values<D, ROWS, false>(o, v, w, 1.0f, 0, ROWS);
      } else {
        // the rest of the scale on the products, and where some rows do not see all, each query's rows by themselves, with zeros
        // in the place of what they do not see
        const int rt = j - p.row_tiles_div.div(j) * p.row_tiles;
#pragma unroll 1
        for (int token = 0; token < (border ? p.n : 1); ++token) {
          const int limit = border ? min(max(len - p.n + token + 1, 0), most) : key0 + 16;
          const int lo = border ? token * p.r - rt * 16 : 0, hi = border ? lo + p.r : ROWS;  // the query's rows of the item
          if (limit <= key0 || hi <= 0 || lo >= ROWS) continue;
          uint32_t y[4][C::kVBytes / 4];
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int x = 0; x < C::kVBytes / 4; ++x) y[c][x] = key0 + 2 * t + c % 2 + c / 2 * 8 >= limit ? 0u : v[c][x];
          add_values<D, ROWS, true>(o, y, w, st.w, lo, hi);
        }
      }
    }

    if ((tile + 1 == tiles || at + 1 == to) && !together) {
      // ------------------------------------------- the item's end, or the stretch's
      const int begin = at - tile, end = begin + tiles;
      const bool here = begin >= from;  // the item begins in the stretch
      const bool whole = here && end <= to;
      const int rows = min(16, p.n * p.r - (j - p.row_tiles_div.div(j) * p.row_tiles) * 16);
      if (here) {
        cut = !whole;
        const int entry = p.by_item ? b * p.items + j : me;
        if (cut && lane == 0) p.cuts[entry] = CutItem{b, j, me, deal.holder(end - 1), warps, begin, end, deal};
        if (p.by_item && lane == 0) p.cut[entry] = cut;
      }
      float *sums = p.sums + (static_cast<int64_t>(2 * me) + (here ? 1 : 0)) * p.rows * (D + 4);
      // a lane's sums of two rows: ROWS 16: rows g and g + 8 of two stretches of values, 8: rows 2 t and 2 t + 1 of one
      float mr[2];
      mr[0] = ROWS == 16 ? m[0] : __shfl_sync(kAll, m[0], 8 * t);
      mr[1] = ROWS == 16 ? m[RR - 1] : __shfl_sync(kAll, m[0], 8 * t + 4);
#pragma unroll
      for (int r2 = 0; r2 < 2; ++r2) {
        const int row = ROWS == 16 ? g + 8 * r2 : 2 * t + r2;
        if (row >= rows) continue;
        const float inv = whole ? over_sum(l[r2], mr[r2]) : over_part(l[r2]), one_unit = ex2(unit);
        uint16_t *out = p.out + row_at(p, b, j, row, p.ldo);
#pragma unroll
        for (int e = 0; e < RR; ++e)
#pragma unroll
          for (int x = 0; x < D / 8; x += 8) {
            float v8[8];
#pragma unroll
            for (int y = 0; y < 8; ++y) v8[y] = (ROWS == 16 ? o[(2 * (x + y) + r2) % NO][e] : o[(x + y) % NO][r2]) * inv * one_unit;
            const int d = ROWS == 16 ? (2 * t + e) * (D / 8) + x : g * (D / 8) + x;
            if (whole) {
              if (d < head_dim) *reinterpret_cast<uint4 *>(out + d) = eight_out<DT>(v8);
            } else {
              *reinterpret_cast<float4 *>(sums + row * D + d) = make_float4(v8[0], v8[1], v8[2], v8[3]);
              *reinterpret_cast<float4 *>(sums + row * D + d + 4) = make_float4(v8[4], v8[5], v8[6], v8[7]);
            }
          }
        if (!whole && (ROWS == 16 ? t : g) == 0) sums[p.rows * D + row] = mr[r2], sums[p.rows * (D + 1) + row] = l[r2] * kPartSum;
      }
    }
    ++at;
    if (++tile == tiles) {
      tile = 0;
      at += kItemCost;
      if (++j == p.items) {
        j = 0;
        if (++b < p.batch) tiles = tiles_of(b);
      }
    }
  }
  if (!together) {
    if (!p.by_item && lane == 0 && from < to) p.cut[me] = cut;
    return;
  }

  // ------------------------------------------- the block's tiles are of one item
  const int begin = one_begin, end = one_begin + one_tiles;
  __syncthreads();  // the rings are idle (no copies are in flight: every tile sent was waited for)
  float *sums = reinterpret_cast<float *>(smem + C::kInfo);
#pragma unroll
  for (int r2 = 0; r2 < RR; ++r2)
    if (t == 0) row_m[warp][g + 8 * r2] = m[r2];
#pragma unroll
  for (int r2 = 0; r2 < 2; ++r2)
    if ((ROWS == 16 ? t : g) == 0) row_l[warp][ROWS == 16 ? g + 8 * r2 : 2 * t + r2] = l[r2] * kPartSum;
  // (as O / l, so that parts of unlike units can be added)
  const float inv[2] = {over_part(l[0]), over_part(l[1])};
  const float one_unit = ex2(unit);
#pragma unroll
  for (int x = 0; x < NO; ++x)
#pragma unroll
    for (int i = 0; i < 2; ++i)
      sums[(warp * ROWS + row_of<ROWS>(x, i)) * C::kSumRow + value_of<D, ROWS>(x, i)] = o[x][i] * inv[ROWS == 16 ? x % 2 : i] * one_unit;
  __syncthreads();
  const bool here = begin >= block_from, whole = here && end <= block_to;
  if (lane == 0 && from < to && !solo) {
    const int entry = p.by_item ? one_b * p.items + one_j : me;
    if (p.by_item ? here && warp == 0 : true) p.cut[entry] = here && !whole && warp == 0;
    if (here && !whole && warp == 0) p.cuts[entry] = CutItem{one_b, one_j, me, deal.holder(end - 1), warps, begin, end, deal};
  }
  const int rows = min(ROWS, p.n * p.r - (one_j - p.row_tiles_div.div(one_j) * p.row_tiles) * 16);
  float *slot = p.sums + (static_cast<int64_t>(2) * blockIdx.x * warps + (here ? 1 : 0)) * p.rows * (D + 4);
  for (int i = threadIdx.x; i < rows * (D / 4); i += 32 * W) {
    const int row = i / (D / 4), d = i % (D / 4) * 4;
    float high = -INFINITY, sum_l = 0.0f, x[4] = {};
#pragma unroll
    for (int w = 0; w < W; ++w) high = fmaxf(high, row_m[w][row]);
#pragma unroll 4
    for (int w = 0; w < W; ++w) {
      const float f = row_m[w][row] == high ? row_l[w][row] : row_l[w][row] * ex2(row_m[w][row] - high);
      sum_l += f;
      const float4 y = *reinterpret_cast<const float4 *>(sums + (w * ROWS + row) * C::kSumRow + d);
      x[0] = fmaf(y.x, f, x[0]), x[1] = fmaf(y.y, f, x[1]), x[2] = fmaf(y.z, f, x[2]), x[3] = fmaf(y.w, f, x[3]);
    }
    const float over = whole ? over_sum(sum_l, high) : over_part(sum_l);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] *= over;
    if (whole) {
      if (d < head_dim)
        *reinterpret_cast<uint2 *>(p.out + row_at(p, one_b, one_j, row, p.ldo) + d) =
            make_uint2(out_bits2<DT>(x[0], x[1]), out_bits2<DT>(x[2], x[3]));
    } else {
      *reinterpret_cast<float4 *>(slot + row * D + d) = make_float4(x[0], x[1], x[2], x[3]);
      if (d == 0) slot[p.rows * D + row] = high, slot[p.rows * (D + 1) + row] = sum_l;
    }
  }
}

constexpr int kAddWarps = 8;

// The items that are cut, their parts added in order: a block for each entry of `cut`, a warp a row or, APART, a block a row, whose
// warps have every eighth part each. Which parts there are follows from the dealing: an entry is all that is read first,
// then the parts' maxima and sums with the first of their values.
template <int DT, int D, bool APART>
__global__ void __launch_bounds__(32 * kAddWarps, APART ? 3 : 8) kv_add_kernel(const __grid_constant__ KvParams p) {
  constexpr int N = D / 32;    // values of a lane
  constexpr int kAhead = APART ? 8 : 4;  // parts whose values are fetched together
  __shared__ float part_o[APART ? kAddWarps : 1][D], part_m[kAddWarps], part_l[kAddWarps];
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int workers = *p.workers, cut = p.cut[blockIdx.x];
  const CutItem it = p.cuts[blockIdx.x];
  // (entries that this call has not written hold anything)
  if (workers == 0 || (!p.by_item && static_cast<int>(blockIdx.x) >= workers) || !cut) return;
  const int rows = min(16, p.n * p.r - (it.j - p.row_tiles_div.div(it.j) * p.row_tiles) * 16);
  const int row = APART ? blockIdx.y : blockIdx.y * kAddWarps + warp;
  if (row >= rows) return;
  // the item's parts: those of its first block's warps, of its last block's, and of each block between them one; also one of a
  // block that has tiles of no other item
  const int block0 = it.first / it.warps, block1 = it.last / it.warps;
  auto one = [&](int block) {
    return it.deal.start(block * it.warps) >= it.begin - kItemCost && it.deal.start((block + 1) * it.warps) <= it.end + kItemCost;
  };
  const int end0 = min((block0 + 1) * it.warps - 1, it.last);
  const int parts0 = one(block0) ? 1 : end0 - it.first + 1, between = max(block1 - block0 - 1, 0);
  const int parts1 = block1 == block0 ? 0 : one(block1) ? 1 : it.last - block1 * it.warps + 1;
  const int parts = parts0 + between + parts1;
  // a part's sums
  auto sums_of = [&](int i) {
    const int at = i < parts0 ? it.first + i : i < parts0 + between ? (block0 + 1 + i - parts0) * it.warps : block1 * it.warps + i - parts0 - between;
    return p.sums + (2 * static_cast<int64_t>(at) + (it.deal.start(at) <= it.begin ? 1 : 0)) * p.rows * (D + 4);
  };
  const int step = APART ? kAddWarps : 1, from = APART ? warp : 0;
  float m = -INFINITY, l = 0.0f, o[N] = {};
  for (int base = from; base < parts; base += 32 * step) {
    const int here = min((parts - base + step - 1) / step, 32);  // parts of this turn, one a lane
    const float *mine = sums_of(base + min(lane, here - 1) * step);
    const uint64_t mine_at = reinterpret_cast<uint64_t>(mine + row * D);
    float high = lane < here ? mine[p.rows * D + row] : -INFINITY;
    const float l_part = lane < here ? mine[p.rows * (D + 1) + row] : 0.0f;
    const float m_part = high;
    float v[kAhead][N];
    auto fetch = [&](int first) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const float *from_part = reinterpret_cast<const float *>(__shfl_sync(kAll, mine_at, min(first + i, here - 1))) + N * lane;
        if constexpr (N == 4) {
          const float4 x = *reinterpret_cast<const float4 *>(from_part);
          v[i][0] = x.x, v[i][1] = x.y, v[i][2] = x.z, v[i][3] = x.w;
        } else {
          const float2 x = *reinterpret_cast<const float2 *>(from_part);
          v[i][0] = x.x, v[i][1] = x.y;
        }
      }
    };
    fetch(0);
#pragma unroll
    for (int i = 16; i > 0; i /= 2) high = fmaxf(high, __shfl_xor_sync(kAll, high, i));
    high = fmaxf(high, m);
    // (a maximum that is not above the one so far, -inf beside -inf among them, weighs 1 as it stands)
    const float f = lane >= here ? 0.0f : m_part == high ? l_part : l_part * ex2(m_part - high);
    const float f_old = m == high ? 1.0f : ex2(m - high);
    float l_sum = f;
#pragma unroll
    for (int i = 16; i > 0; i /= 2) l_sum += __shfl_xor_sync(kAll, l_sum, i);
    l = fmaf(l, f_old, l_sum);
#pragma unroll
    for (int x = 0; x < N; ++x) o[x] *= f_old;
    m = high;
    for (int first = 0; first < here; first += kAhead) {
      if (first > 0) fetch(first);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const float g = __shfl_sync(kAll, f, min(first + i, 31));
        if (first + i >= here) continue;
#pragma unroll
        for (int x = 0; x < N; ++x) o[x] = fmaf(v[i][x], g, o[x]);
      }
    }
  }
  if (APART) {
    if (lane == 0) part_m[warp] = m, part_l[warp] = l;
#pragma unroll
    for (int x = 0; x < N; ++x) part_o[APART ? warp : 0][N * lane + x] = o[x];
    __syncthreads();
    if (warp != 0) return;
    float high = -INFINITY;
#pragma unroll
    for (int w = 0; w < kAddWarps; ++w) high = fmaxf(high, part_m[w]);
    m = high;
    l = 0.0f;
#pragma unroll
    for (int x = 0; x < N; ++x) o[x] = 0.0f;
#pragma unroll
    for (int w = 0; w < kAddWarps; ++w) {
      const float f = part_m[w] == high ? 1.0f : ex2(part_m[w] - high);
      l = fmaf(part_l[w], f, l);
#pragma unroll
      for (int x = 0; x < N; ++x) o[x] = fmaf(part_o[APART ? w : 0][N * lane + x], f, o[x]);
    }
  }
  if (N * lane >= p.head_dim) return;
  const float inv = over_sum(l, m);
  uint16_t *out = p.out + row_at(p, it.b, it.j, row, p.ldo) + N * lane;
  if constexpr (N == 4)
    *reinterpret_cast<uint2 *>(out) = make_uint2(out_bits2<DT>(o[0] * inv, o[1] * inv), out_bits2<DT>(o[2] * inv, o[3] * inv));
  else
    *reinterpret_cast<uint32_t *>(out) = out_bits2<DT>(o[0] * inv, o[1] * inv);
}

template <int DT, int D, int ROWS>
cudaError_t launch_d(const KvParams &p, int num_sms, cudaStream_t stream) {
  using C = KvCfg<D, ROWS>;
  auto kern = kv_attention_kernel<DT, D, ROWS>;
  static std::atomic<uint64_t> set{0};
  cudaError_t e = allow_smem(kern, C::kSmem, &set);
  if (e != cudaSuccess) return e;
  e = launch_programmatic(kern, num_sms, 32 * C::kWarps, C::kSmem, stream, p);
  if (e != cudaSuccess) return e;
  // (a cache whose sequences have no more tiles than this never cuts an item)
  if (p.by_item && cdiv(static_cast<int64_t>(p.max_pages) * p.page, 16) <= C::kWarps * kSoloTiles) return cudaSuccess;
  // an entry an item, or one a warp where there are more items than blocks; a row's parts to a block's warps where they may be many, or
  // where a row is all there is
  const bool apart = p.by_item || p.rows == 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.by_item ? p.batch * p.items : num_sms * C::kWarps),
                     static_cast<unsigned>(apart ? p.rows : cdiv(p.rows, kAddWarps)));
  cfg.blockDim = dim3(32 * kAddWarps);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = apart ? cudaLaunchKernelEx(&cfg, kv_add_kernel<DT, D, true>, p) : cudaLaunchKernelEx(&cfg, kv_add_kernel<DT, D, false>, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// Where the parts begin, for so many warps in all.
size_t slots_at(int warps) { return 256 + 256 * static_cast<size_t>(cdiv(warps * (sizeof(CutItem) + sizeof(int32_t)), 256)); }

}  // namespace

// The first 256 bytes (whose first word, another call's error word, is left alone) hold the number of workers; then the cut items and their
// parts. What is enough for n queries is for fewer: 8 rows, which have more warps, take more than 9.
size_t kv_attention_workspace_bytes(int n, int q_heads, int k_heads, int head_dim, int num_sms) {
  const int64_t all = static_cast<int64_t>(n) * (q_heads / k_heads);
  const size_t d = head_dim <= 64 ? 64 : 128;
  auto of = [&](int rows) {
    const int warps = num_sms * warps_of(head_dim, rows);
    return slots_at(warps) + static_cast<size_t>(2 * warps) * rows * (d + 4) * sizeof(float);
  };
  const size_t own = of(all < 16 ? static_cast<int>(all) : 16), fewer = of(all < 8 ? static_cast<int>(all) : 8);
  return own > fewer ? own : fewer;
}

cudaError_t launch_kv_attention(const KvAttentionArgs &a, void *workspace, int num_sms, cudaStream_t stream) {
  KvParams p;
  p.q = static_cast<const uint16_t *>(a.q);
  p.k_cache = static_cast<const uint8_t *>(a.k_cache);
  p.v_cache = static_cast<const uint8_t *>(a.v_cache);
  p.k_scale = a.k_scale;
  p.v_scale = a.v_scale;
  p.table = a.table;
  p.lens = a.lens;
  p.out = static_cast<uint16_t *>(a.out);
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  p.workers = reinterpret_cast<int32_t *>(ws + 128);
  p.cuts = reinterpret_cast<CutItem *>(ws + 256);
  p.ldq = a.ldq;
  p.ldo = a.ldo;
  p.pages = a.pages;
  p.batch = a.batch;
  p.n = a.n;
  p.max_pages = a.max_pages;
  p.k_heads = a.k_heads;
  p.head_dim = a.head_dim;
  p.page = a.page;
  p.r = a.q_heads / a.k_heads;
  p.row_tiles = static_cast<int>(cdiv(static_cast<int64_t>(a.n) * p.r, 16));
  p.rows = a.n * p.r < 16 ? a.n * p.r : 16;
  const int warps = num_sms * warps_of(a.head_dim, p.rows);
  p.cut = reinterpret_cast<int32_t *>(ws + 256 + static_cast<size_t>(warps) * sizeof(CutItem));
  p.sums = reinterpret_cast<float *>(ws + slots_at(warps));
  p.items = p.row_tiles * a.k_heads;
  p.by_item = static_cast<int64_t>(p.batch) * p.items <= num_sms;
  p.scale = a.scale;
  p.page_div = make_fastdiv(static_cast<uint32_t>(a.page));
  p.r_div = make_fastdiv(static_cast<uint32_t>(p.r));
  p.row_tiles_div = make_fastdiv(static_cast<uint32_t>(p.row_tiles));
  auto go = [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    if (p.rows <= 8) return a.head_dim > 64 ? launch_d<DT, 128, 8>(p, num_sms, stream) : launch_d<DT, 64, 8>(p, num_sms, stream);
    return a.head_dim > 64 ? launch_d<DT, 128, 16>(p, num_sms, stream) : launch_d<DT, 64, 16>(p, num_sms, stream);
  };
  return a.dtype == kDtypeBf16 ? go(std::integral_constant<int, kDtypeBf16>{}) : go(std::integral_constant<int, kDtypeF16>{});
}

}  // namespace w4
