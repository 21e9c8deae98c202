// w4_kv_attention: a few query rows of each sequence over the paged cache of e4m3 codes.
//
// For a sequence and key head the n query rows of the r query heads that share it are n * r rows (row = j * r + head), taken 16
// at a time (an item) as the M side of register-operand products (mma.sync m16n8k16, fp16 operands, fp32 sums): e4m3
// codes are exact in fp16, and so are q's values (bf16 rows times a power of two that keeps them within fp16's range).
// For a tile of 16 keys, which lies in one page: S = q . codes, s = S * (k scale * softmax scale * log2 e) + log2(v scale), a
// row's running maximum m, w = 2^(s - m) in fp16, O += w . codes, l += (sum of w) / v scale: with the page's scale of the
// values inside the weight no product needs a scale of its own. m may lag behind by 2^8 as a weight, so that O is
// rescaled a few times in an item. A page whose scale is no positive number within 2^+-100 goes by a product of its own.
//
// The tiles of all items in order are dealt out evenly, a stretch to each of the device's warps, so that sequences of unlike
// lengths load it evenly; a warp works alone and a lane copies to shared memory exactly the bytes that it will read
// (cp.async, 16 bytes each, zeros past the sequence's end): no barriers. Which bytes follows from the fragments: of key 8 u +
// lane / 4 the quarter of the head that its place in the quad has, in 16-byte pieces; of keys 2 t, 2 t + 1 and those plus 8
// (t = lane % 4) an eighth of the head, whose codes of two neighbouring keys are put side by side by byte permutes.
// Items cut between warps leave sums (O, m, l) in the workspace, one for a block whose warps are all within one item; a second
// launch adds them in order.
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
constexpr int kKvWarps = 12;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.0f;    // how far a score may pass the maximum in use (log2 of the weight)
// Scales of values that go into the weights: 2^-40 to 2^40, so that a weight of one page beside another's stays a normal number
// of 32 bits (it counts in the sum l, however small its part of O).
constexpr float kScaleMin = 0x1p-40f, kScaleMax = 0x1p40f;

// An item that begins in a warp's stretch and ends in another's: what the second launch adds.
struct CutItem {
  int32_t b, j;        // sequence and item of it
  int32_t last;        // the warp that holds the item's end
  int32_t reserved;
  int64_t begin, end;  // the item's tiles in the order of all
  int64_t total, workers;
};

// The first tile of warp w's stretch.
__device__ __forceinline__ int64_t stretch_of(int64_t w, int64_t workers, int64_t total) { return min(w, workers) * total / workers; }

struct KvParams {
  const uint16_t *q;
  const uint8_t *k_cache, *v_cache;
  const float *k_scale, *v_scale;
  const int32_t *table, *lens;
  uint16_t *out;
  int32_t *cut;    // [warps of the device]: whether cuts has an item
  CutItem *cuts;
  float *sums;     // [2 * warps]: O [rows][D], m [rows], l [rows], padded to 16 bytes, of a stretch's first and last item
  int64_t ldq, ldo, pages;
  int batch, n, max_pages, q_heads, k_heads, head_dim, page, r, row_tiles, rows, items;  // items of a sequence
  float scale;
  FastDiv page_div, r_div;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
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

// D: head_dim rounded up to 64 or 128.
template <int D>
struct KvCfg {
  static constexpr int kStages = 4;
  static constexpr int kPieces = D / 64;                 // 16-byte pieces of a key in a lane
  static constexpr int kVBytes = D / 8;                  // bytes of a value row in a lane
  static constexpr int kTileBytesWarp = 32 * (32 * kPieces + 4 * kVBytes);
  static constexpr int kRing = kStages * kTileBytesWarp;
  static constexpr int kSumRow = D + 4;                  // floats of a row of a warp's sums in shared memory
  static constexpr int kSumBytes = kKvWarps * 16 * kSumRow * 4;
  static constexpr int kSmem = kKvWarps * kRing > kSumBytes ? kKvWarps * kRing : kSumBytes;
};

// What a row's sums are made of: value d of the item's row g (+ 8) is o[d % NT][2 i + e], d / NT = 2 t + e.
template <int D>
struct Sums {
  float o[D / 8][4];
  float m[2], l[2];
};

// The place of row i of item j of sequence b in q or out.
__device__ __forceinline__ int64_t row_at(const KvParams &p, int b, int j, int i, int64_t ld) {
  const int h = j / p.row_tiles, rho = (j - h * p.row_tiles) * 16 + i;
  const int token = p.r_div.div(rho);
  return (static_cast<int64_t>(b) * p.n + token) * ld + static_cast<int64_t>(h * p.r + rho - token * p.r) * p.head_dim;
}

template <int DT>
__device__ __forceinline__ uint4 eight_out(const float (&v)[8], float f) {
  return make_uint4(out_bits2<DT>(v[0] * f, v[1] * f), out_bits2<DT>(v[2] * f, v[3] * f), out_bits2<DT>(v[4] * f, v[5] * f),
                    out_bits2<DT>(v[6] * f, v[7] * f));
}

// 0 for a row that saw nothing (sum 0; where it saw something the sum is positive or NaN).
__device__ __forceinline__ float over_sum(float l) { return l == 0.0f ? 0.0f : 1.0f / l; }

template <int DT, int D, bool WHOLE>
__global__ void __launch_bounds__(32 * kKvWarps, 1) kv_attention_kernel(const __grid_constant__ KvParams p) {
  using C = KvCfg<D>;
  constexpr int NT = D / 8;  // n-tiles of the output
  constexpr int S = C::kStages;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int64_t upto[32 * kKvWarps];   // tiles of the sequences up to and with the thread's
  // of a tile's page: k scale, log2 of the part of the v scale that goes into the weights, 1 / that part, and 0 for no page, 1
  // for all of the scale in the weights, 2 else; the rest of it
  __shared__ float4 stage_of[kKvWarps][S];
  __shared__ float stage_rest[kKvWarps][S];
  __shared__ bool together_sh;
  __shared__ float row_m[kKvWarps][16], row_l[kKvWarps][16];
  const int warp = __shfl_sync(kAll, threadIdx.x / 32, 0), lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const uint32_t ring = smem_u32(smem) + warp * C::kRing;
  griddep_launch_dependents();
  griddep_wait();

  // ------------------------------------------------- the warp's stretch of the tiles
  const int head_dim = WHOLE ? D : p.head_dim;
  const int most = p.max_pages * p.page;
  auto tiles_of = [&](int b) { return max((min(p.lens[b], most) + 15) / 16, 1); };  // (a sequence without keys still has an output)
  const int share = (p.batch + 32 * kKvWarps - 1) / (32 * kKvWarps);  // sequences a thread adds up
  int64_t sum = 0;
  for (int i = 0; i < share; ++i) {
    const int b = threadIdx.x * share + i;
    if (b < p.batch) sum += static_cast<int64_t>(tiles_of(b)) * p.items;
  }
#pragma unroll
  for (int i = 1; i < 32; i *= 2) {
    const int64_t x = __shfl_up_sync(kAll, sum, i);
    if (lane >= i) sum += x;
  }
  upto[threadIdx.x] = sum;
  __syncthreads();
  int64_t before = 0;
  for (int i = 0; i < warp; ++i) before += upto[32 * i + 31];
  __syncthreads();
  upto[threadIdx.x] = sum + before;
  __syncthreads();
  const int64_t total = upto[32 * kKvWarps - 1];
  const int all_warps = kKvWarps * gridDim.x;
  // fewer warps where the tiles are few: each takes two at least
  const int64_t workers = min(static_cast<int64_t>(all_warps), max(total / 2, int64_t{1}));
  const int me = blockIdx.x * kKvWarps + warp;
  const int64_t from = stretch_of(me, workers, total), to = stretch_of(me + 1, workers, total);
  const int count = static_cast<int>(to - from);
  bool cut = false;

  // the sequence, its item and the item's tile that `from` is
  int b = 0, j = 0, tile = 0, tiles = 1;
  {
    int lo = 0, hi = 32 * kKvWarps - 1;
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (upto[mid] > from)
        hi = mid;
      else
        lo = mid + 1;
    }
    int64_t rest = from - (lo > 0 ? upto[lo - 1] : 0);
    b = lo * share;
    if (count > 0) {
      for (;; ++b) {
        tiles = tiles_of(b);
        if (rest < static_cast<int64_t>(tiles) * p.items) break;
        rest -= static_cast<int64_t>(tiles) * p.items;
      }
      j = static_cast<int>(rest / tiles);
      tile = static_cast<int>(rest - static_cast<int64_t>(j) * tiles);
    }
  }
  // whether all the warps of the block are within one item (its first warp's): their sums are then added here
  const int64_t block_from = stretch_of(static_cast<int64_t>(blockIdx.x) * kKvWarps, workers, total);
  const int64_t block_to = stretch_of((static_cast<int64_t>(blockIdx.x) + 1) * kKvWarps, workers, total);
  if (threadIdx.x == 0) together_sh = count > 0 && from - tile + tiles >= block_to;
  __syncthreads();
  const bool together = together_sh;

  // ---------------------------------------------------------------- copies
  // The tile that is copied next, and what the lookup found for 32 tiles of its item
  int cb = b, cj = j, ct = tile, ctiles = tiles, found = 0, first = 0;
  int at_page = -1;
  float at_ks = 0.0f, at_vs = 0.0f;
  const uint32_t lane_k = lane * 16, lane_v = 2 * C::kPieces * 512 + lane * C::kVBytes;
  auto send = [&](int i) {
    if (i < count) {
      const int h = cj / p.row_tiles;
      if (ct - first >= found) {  // look up the next 32 tiles of the item
        first = ct;
        found = min(32, ctiles - ct);
        at_page = -1;
        if (lane < found) {
          const int pi = p.page_div.div((ct + lane) * 16);
          int at = -1;
          if (pi < p.max_pages) at = p.table[static_cast<int64_t>(cb) * p.max_pages + pi];
          if (at >= 0 && at < p.pages) {
            at_page = at;
            at_ks = p.k_scale[static_cast<int64_t>(at) * p.k_heads + h];
            at_vs = p.v_scale[static_cast<int64_t>(at) * p.k_heads + h];
          }
        }
      }
      const int page_at = __shfl_sync(kAll, at_page, ct - first);
      if (lane == ct - first) {
        const float size = fabsf(at_vs);
        const bool plain = size >= kScaleMin && size <= kScaleMax;
        const float part = plain ? size : size > kScaleMax ? kScaleMax : kScaleMin;
        stage_of[warp][i % S] = make_float4(at_ks, log2f(part), 1.0f / part, at_page < 0 ? 0.0f : plain && at_vs > 0.0f ? 1.0f : 2.0f);
        stage_rest[warp][i % S] = plain ? copysignf(1.0f, at_vs) : at_vs / part;
      }
      __syncwarp();
      if (page_at >= 0) {
        const int key0 = ct * 16;
        const int slot0 = key0 - p.page_div.div(key0) * p.page;
        const int64_t base = ((static_cast<int64_t>(page_at) * p.k_heads + h) * p.page + slot0) * head_dim;
        const uint32_t to_k = ring + i % S * C::kTileBytesWarp + lane_k, to_v = ring + i % S * C::kTileBytesWarp + lane_v;
        const uint8_t *k = p.k_cache + base + g * head_dim + t * 16, *v = p.v_cache + base + 2 * t * head_dim + g * C::kVBytes;
        const int here = min(p.lens[cb], most) - key0;  // keys of the tile
        if (WHOLE && here >= 16) {
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int c = 0; c < C::kPieces; ++c) cp_async16(to_k + (u * C::kPieces + c) * 512, k + 8 * u * D + 64 * c);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint8_t *src = v + (c % 2 + c / 2 * 8) * D;
            if (C::kVBytes == 16)
              cp_async16(to_v + c * 512, src);
            else
              cp_async8(to_v + c * 256, src, 8);
          }
        } else {
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int c = 0; c < C::kPieces; ++c) {
              const bool there = 8 * u + g < here && (t + 4 * c) * 16 < head_dim;
              cp_async16_zfill(to_k + (u * C::kPieces + c) * 512, there ? k + 8 * u * head_dim + 64 * c : p.k_cache, there ? 16u : 0u);
            }
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int key = c % 2 + c / 2 * 8;
            const bool there = 2 * t + key < here && g * C::kVBytes < head_dim;
            const uint8_t *src = there ? v + key * head_dim : p.v_cache;
            if (C::kVBytes == 16)
              cp_async16_zfill(to_v + c * 512, src, there ? 16u : 0u);
            else
              cp_async8(to_v + c * 256, src, there ? 8u : 0u);
          }
        }
      }
      if (++ct == ctiles) {  // the next item
        ct = first = found = 0;
        if (++cj == p.items) {
          cj = 0;
          if (++cb < p.batch) ctiles = tiles_of(cb);
        }
      }
    }
    cp_commit();
  };

  // ------------------------------------------------------------ products
  uint32_t q[D / 16][4];
  Sums<D> a;
  float mul[2];
  int sees[2], least = 0, len = 0;
  auto begin_item = [&]() {
    const int h = j / p.row_tiles, rt = j - h * p.row_tiles;
    len = max(p.lens[b], 0);
    const int keys = min(len, most);
    least = keys;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
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
            q[4 * c + 2 * e + x / 2][x % 2 * 2 + i] = bits;
          }
        }
      a.m[i] = -INFINITY;
      a.l[i] = 0.0f;
    }
    least = static_cast<int>(__reduce_min_sync(kAll, least));
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
      for (int e = 0; e < 4; ++e) a.o[x][e] = 0.0f;
  };

  a.m[0] = a.m[1] = -INFINITY;
  a.l[0] = a.l[1] = 0.0f;
#pragma unroll
  for (int x = 0; x < NT; ++x)
#pragma unroll
    for (int e = 0; e < 4; ++e) a.o[x][e] = 0.0f;
  for (int i = 0; i < S - 1; ++i) send(i);
  for (int i = 0; i < count; ++i) {
    if (i == 0 || tile == 0) begin_item();
    send(i + S - 1);  // (its place held tile i - 1, which is done)
    cp_wait<S - 1>();
    const float4 st = stage_of[warp][i % S];
    if (st.w != 0.0f) {
      const int key0 = tile * 16;
      const uint32_t kt = ring + i % S * C::kTileBytesWarp + lane_k, vt = ring + i % S * C::kTileBytesWarp + lane_v;
      float s[2][4] = {};
#pragma unroll
      for (int c = 0; c < C::kPieces; ++c) {
        const uint4 k0 = lds128(kt + c * 512), k1 = lds128(kt + (C::kPieces + c) * 512);
        const uint32_t x[4] = {k0.x, k0.y, k0.z, k0.w}, y[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t x0, x1, y0, y1;
          e4m3x4_f16x4(x[w], &x0, &x1);
          e4m3x4_f16x4(y[w], &y0, &y1);
          const uint32_t(&f)[4] = q[4 * c + w];
          mma_16816<kDtypeF16>(s[0], f[0], f[1], f[2], f[3], x0, x1);
          mma_16816<kDtypeF16>(s[1], f[0], f[1], f[2], f[3], y0, y1);
        }
      }
      // values: words of the four keys
      uint32_t v[4][C::kVBytes / 4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if constexpr (C::kVBytes == 16) {
          const uint4 x = lds128(vt + c * 512);
          v[c][0] = x.x, v[c][1] = x.y, v[c][2] = x.z, v[c][3] = x.w;
        } else {
          asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v[c][0]), "=r"(v[c][1]) : "r"(vt + c * 256) : "memory");
        }
      }
      const bool border = key0 + 16 > least;  // some row does not see all of the tile
      const bool own = st.w == 2.0f;          // not all of the values' scale is in the weights
      float top[2];
#pragma unroll
      for (int r2 = 0; r2 < 2; ++r2) {
        const float f = st.x * mul[r2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int e = 2 * r2; e < 2 * r2 + 2; ++e) {
            s[u][e] = fmaf(s[u][e], f, st.y);
            if (border && key0 + 8 * u + 2 * t + e % 2 >= sees[r2]) s[u][e] = -INFINITY;
          }
        top[r2] = fmaxf(fmaxf(s[0][2 * r2], s[0][2 * r2 + 1]), fmaxf(s[1][2 * r2], s[1][2 * r2 + 1]));
      }
#pragma unroll
      for (int x = 1; x < 4; x *= 2)
#pragma unroll
        for (int r2 = 0; r2 < 2; ++r2) top[r2] = fmaxf(top[r2], __shfl_xor_sync(kAll, top[r2], x));
      // (-inf + 8 is below any score: a row's first tile sets its maximum)
      if (__any_sync(kAll, top[0] > a.m[0] + kSlack || top[1] > a.m[1] + kSlack)) {
#pragma unroll
        for (int r2 = 0; r2 < 2; ++r2) {
          const float now = fmaxf(a.m[r2], top[r2]);
          const float alpha = now == a.m[r2] ? 1.0f : ex2(a.m[r2] - now);
          a.m[r2] = now;
          a.l[r2] *= alpha;
#pragma unroll
          for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int e = 2 * r2; e < 2 * r2 + 2; ++e) a.o[x][e] *= alpha;
        }
      }
#pragma unroll
      for (int r2 = 0; r2 < 2; ++r2) {
        const float base = a.m[r2] == -INFINITY ? 0.0f : a.m[r2];  // (nothing seen yet: weights of 0)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int e = 2 * r2; e < 2 * r2 + 2; ++e) s[u][e] = ex2(s[u][e] - base);
        a.l[r2] = fmaf((s[0][2 * r2] + s[0][2 * r2 + 1]) + (s[1][2 * r2] + s[1][2 * r2 + 1]), st.z, a.l[r2]);
      }
      const uint32_t w[4] = {half2_bits(s[0][0], s[0][1]), half2_bits(s[0][2], s[0][3]), half2_bits(s[1][0], s[1][1]),
                             half2_bits(s[1][2], s[1][3])};
      bool odd = own;
      if (border && !own) {
        // 0 * NaN is NaN: whether the tile, of which some rows do not see all, holds NaN
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int x = 0; x < C::kVBytes / 4; ++x) odd |= any_nan_code(v[c][x]);
        odd = __any_sync(kAll, odd);
      }
      if (!odd) {
#pragma unroll
        for (int x = 0; x < C::kVBytes / 4; ++x) {
          uint32_t b0[4], b1[4];
          e4m3x4_f16x4(__byte_perm(v[0][x], v[1][x], 0x5140), &b0[0], &b0[1]);
          e4m3x4_f16x4(__byte_perm(v[0][x], v[1][x], 0x7362), &b0[2], &b0[3]);
          e4m3x4_f16x4(__byte_perm(v[2][x], v[3][x], 0x5140), &b1[0], &b1[1]);
          e4m3x4_f16x4(__byte_perm(v[2][x], v[3][x], 0x7362), &b1[2], &b1[3]);
#pragma unroll
          for (int e = 0; e < 4; ++e) mma_16816<kDtypeF16>(a.o[4 * x + e], w[0], w[1], w[2], w[3], b0[e], b1[e]);
        }
      } else {
        // each query's rows by themselves, with zeros in the place of what they do not see, and the rest of the scale on the
        // products
        const float f = stage_rest[warp][i % S];
        const int rt = j % p.row_tiles;
#pragma unroll 1
        for (int token = 0; token < p.n; ++token) {
          const int limit = min(max(len - p.n + token + 1, 0), most);
          const bool on0 = p.r_div.div(rt * 16 + g) == token, on1 = p.r_div.div(rt * 16 + g + 8) == token;
          if (limit <= key0 || !__any_sync(kAll, on0 || on1)) continue;
#pragma unroll
          for (int x = 0; x < C::kVBytes / 4; ++x) {
            uint32_t y[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) y[c] = key0 + 2 * t + c % 2 + c / 2 * 8 >= limit ? 0u : v[c][x];
            uint32_t b0[4], b1[4];
            e4m3x4_f16x4(__byte_perm(y[0], y[1], 0x5140), &b0[0], &b0[1]);
            e4m3x4_f16x4(__byte_perm(y[0], y[1], 0x7362), &b0[2], &b0[3]);
            e4m3x4_f16x4(__byte_perm(y[2], y[3], 0x5140), &b1[0], &b1[1]);
            e4m3x4_f16x4(__byte_perm(y[2], y[3], 0x7362), &b1[2], &b1[3]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float d[4] = {};
              mma_16816<kDtypeF16>(d, w[0], w[1], w[2], w[3], b0[e], b1[e]);
              if (on0) a.o[4 * x + e][0] = fmaf(f, d[0], a.o[4 * x + e][0]), a.o[4 * x + e][1] = fmaf(f, d[1], a.o[4 * x + e][1]);
              if (on1) a.o[4 * x + e][2] = fmaf(f, d[2], a.o[4 * x + e][2]), a.o[4 * x + e][3] = fmaf(f, d[3], a.o[4 * x + e][3]);
            }
          }
        }
      }
    }

    if (tile + 1 == tiles || i + 1 == count) {
      // ------------------------------------------- the item's end, or the stretch's
      const int64_t item = from + i - tile;  // its first tile
#pragma unroll
      for (int r2 = 0; r2 < 2; ++r2) {
        a.l[r2] += __shfl_xor_sync(kAll, a.l[r2], 1);
        a.l[r2] += __shfl_xor_sync(kAll, a.l[r2], 2);
      }
      const int rows = min(16, p.n * p.r - j % p.row_tiles * 16);
      const bool whole = item >= from && item + tiles <= to;
      if (together) break;
      if (!whole && item >= from) {
        cut = true;
        if (lane == 0)
          p.cuts[me] = CutItem{b, j, static_cast<int32_t>(((item + tiles) * workers - 1) / total), 0, item, item + tiles, total, workers};
      }
#pragma unroll
      for (int r2 = 0; r2 < 2; ++r2) {
        const int row = g + 8 * r2;
        if (row >= rows) continue;
        if (whole) {
          const float inv = over_sum(a.l[r2]);
          uint16_t *out = p.out + row_at(p, b, j, row, p.ldo);
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int x = 0; x < NT; x += 8) {
              const int d = (2 * t + e) * NT + x;
              float v8[8];
#pragma unroll
              for (int y = 0; y < 8; ++y) v8[y] = a.o[x + y][2 * r2 + e];
              if (WHOLE || d < head_dim) *reinterpret_cast<uint4 *>(out + d) = eight_out<DT>(v8, inv);
            }
        } else {
          float *sums = p.sums + (static_cast<int64_t>(2 * me) + (item >= from ? 1 : 0)) * p.rows * (D + 4);
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int x = 0; x < NT; x += 4)
              *reinterpret_cast<float4 *>(sums + row * D + (2 * t + e) * NT + x) =
                  make_float4(a.o[x][2 * r2 + e], a.o[x + 1][2 * r2 + e], a.o[x + 2][2 * r2 + e], a.o[x + 3][2 * r2 + e]);
          if (t == 0) sums[p.rows * D + row] = a.m[r2], sums[p.rows * (D + 1) + row] = a.l[r2];
        }
      }
    }
    if (++tile == tiles) {
      tile = 0;
      if (++j == p.items) {
        j = 0;
        if (++b < p.batch) tiles = tiles_of(b);
      }
    }
  }
  if (!together) {
    if (lane == 0) p.cut[me] = cut;
    return;
  }

  // ------------------------------------------- the block's warps are of one item
  // (its first warp holds the item's place: b, j, tile and tiles as its stretch began)
  __shared__ int b_sh, j_sh;
  __shared__ int64_t begin_sh, end_sh;
  if (threadIdx.x == 0) {
    b_sh = b;
    j_sh = j;
    begin_sh = from + count - 1 - tile;  // (the loop was left at the stretch's last tile)
    end_sh = begin_sh + tiles;
  }
  __syncthreads();  // the rings are idle
  float *sums = reinterpret_cast<float *>(smem);
#pragma unroll
  for (int r2 = 0; r2 < 2; ++r2) {
    float *to_row = sums + (warp * 16 + g + 8 * r2) * C::kSumRow;
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int x = 0; x < NT; x += 4)
        *reinterpret_cast<float4 *>(to_row + (2 * t + e) * NT + x) =
            make_float4(a.o[x][2 * r2 + e], a.o[x + 1][2 * r2 + e], a.o[x + 2][2 * r2 + e], a.o[x + 3][2 * r2 + e]);
    if (t == 0) row_m[warp][g + 8 * r2] = a.m[r2], row_l[warp][g + 8 * r2] = a.l[r2];
  }
  __syncthreads();
  const int64_t begin = begin_sh, end = end_sh;
  const bool whole = begin >= block_from && end <= block_to;
  if (lane == 0) {
    p.cut[me] = !whole && begin >= block_from && warp == 0;
    if (!whole && begin >= block_from && warp == 0)
      p.cuts[me] = CutItem{b_sh, j_sh, static_cast<int32_t>((end * workers - 1) / total), 0, begin, end, total, workers};
  }
  const int rows = min(16, p.n * p.r - j_sh % p.row_tiles * 16);
  float *slot = p.sums + (static_cast<int64_t>(2) * blockIdx.x * kKvWarps + (begin >= block_from ? 1 : 0)) * p.rows * (D + 4);
  for (int i = threadIdx.x; i < rows * (D / 8); i += 32 * kKvWarps) {
    const int row = i / (D / 8), d = i % (D / 8) * 8;
    float top = -INFINITY, l = 0.0f, v8[8] = {};
#pragma unroll
    for (int w = 0; w < kKvWarps; ++w) top = fmaxf(top, row_m[w][row]);
#pragma unroll 4
    for (int w = 0; w < kKvWarps; ++w) {
      const float f = row_m[w][row] == top ? 1.0f : ex2(row_m[w][row] - top);
      l = fmaf(row_l[w][row], f, l);
      const float *o = sums + (w * 16 + row) * C::kSumRow + d;
#pragma unroll
      for (int e = 0; e < 8; ++e) v8[e] = fmaf(o[e], f, v8[e]);
    }
    if (whole) {
      if (WHOLE || d < head_dim)
        *reinterpret_cast<uint4 *>(p.out + row_at(p, b_sh, j_sh, row, p.ldo) + d) = eight_out<DT>(v8, over_sum(l));
    } else {
      *reinterpret_cast<float4 *>(slot + row * D + d) = make_float4(v8[0], v8[1], v8[2], v8[3]);
      *reinterpret_cast<float4 *>(slot + row * D + d + 4) = make_float4(v8[4], v8[5], v8[6], v8[7]);
      if (d == 0) slot[p.rows * D + row] = top, slot[p.rows * (D + 1) + row] = l;
    }
  }
}

constexpr int kAddThreads = 256;

// The items that are cut, their parts added in order. A block looks at warps [x * all / gridDim.x, (x + 1) * all / gridDim.x)
// for items that begin there and adds p.add_rows rows of them; the groups of D / 4 threads take a row each or, with one row, the
// parts in turn.
template <int DT, int D>
__global__ void __launch_bounds__(kAddThreads) kv_add_kernel(const __grid_constant__ KvParams p, int all_warps, int add_rows) {
  constexpr int kLane = D / 4, kGroups = kAddThreads / kLane;
  __shared__ float4 part_o[kGroups][kLane];
  __shared__ float part_m[kGroups], part_l[kGroups];
  griddep_launch_dependents();
  griddep_wait();
  const int w0 = static_cast<int>(static_cast<int64_t>(blockIdx.x) * all_warps / gridDim.x);
  const int w1 = static_cast<int>((static_cast<int64_t>(blockIdx.x) + 1) * all_warps / gridDim.x);
  const int group = threadIdx.x / kLane, x = threadIdx.x % kLane;
  const int row = blockIdx.y * add_rows + (add_rows > 1 ? group : 0);
  const int first = add_rows > 1 ? 0 : group, step = add_rows > 1 ? 1 : kGroups;
  for (int base = w0; base < w1; base += kAddThreads) {
    // (the whole block takes the same turns)
    __shared__ uint32_t mask[kAddThreads / 32];
    const int mine = base + threadIdx.x;
    const uint32_t any = __ballot_sync(kAll, mine < w1 && p.cut[mine] != 0);
    __syncthreads();
    if (threadIdx.x % 32 == 0) mask[threadIdx.x / 32] = any;
    __syncthreads();
    for (int k = 0; k < kAddThreads / 32; ++k)
      for (uint32_t bits = mask[k]; bits; bits &= bits - 1) {
        const int w = base + 32 * k + __ffs(bits) - 1;
        const CutItem it = p.cuts[w];
        const int rows = min(16, p.n * p.r - it.j % p.row_tiles * 16);
        float m = -INFINITY, l = 0.0f;
        float4 o = make_float4(0, 0, 0, 0);
        if (row < rows && (add_rows == 1 || group < add_rows)) {
          for (int at = w + first; at <= it.last; at += step) {
            // a block within the item has one part, in its first warp's place
            const int64_t block = at / kKvWarps;
            const int64_t from = stretch_of(block * kKvWarps, it.workers, it.total);
            const bool one = from >= it.begin && stretch_of((block + 1) * kKvWarps, it.workers, it.total) <= it.end;
            if (one && at % kKvWarps != 0) continue;
            const float *slot = p.sums + (static_cast<int64_t>(2 * at) + (stretch_of(at, it.workers, it.total) <= it.begin ? 1 : 0)) * p.rows * (D + 4);
            const float pm = slot[p.rows * D + row], pl = slot[p.rows * (D + 1) + row];
            const float4 po = *reinterpret_cast<const float4 *>(slot + row * D + 4 * x);
            const float now = fmaxf(m, pm);
            const float f = m == now ? 1.0f : ex2(m - now), pf = pm == now ? 1.0f : ex2(pm - now);
            m = now;
            l = l * f + pl * pf;
            o = make_float4(o.x * f + po.x * pf, o.y * f + po.y * pf, o.z * f + po.z * pf, o.w * f + po.w * pf);
          }
        }
        if (add_rows == 1) {
          part_o[group][x] = o;
          if (x == 0) part_m[group] = m, part_l[group] = l;
          __syncthreads();
          if (group == 0) {
            for (int y = 1; y < kGroups; ++y) {
              const float pm = part_m[y], pl = part_l[y];
              const float4 po = part_o[y][x];
              const float now = fmaxf(m, pm);
              const float f = m == now ? 1.0f : ex2(m - now), pf = pm == now ? 1.0f : ex2(pm - now);
              m = now;
              l = l * f + pl * pf;
              o = make_float4(o.x * f + po.x * pf, o.y * f + po.y * pf, o.z * f + po.z * pf, o.w * f + po.w * pf);
            }
          }
          __syncthreads();
        }
        if (row < rows && (add_rows > 1 ? group < add_rows : group == 0) && 4 * x < p.head_dim) {
          const float inv = over_sum(l);
          *reinterpret_cast<uint2 *>(p.out + row_at(p, it.b, it.j, row, p.ldo) + 4 * x) =
              make_uint2(out_bits2<DT>(o.x * inv, o.y * inv), out_bits2<DT>(o.z * inv, o.w * inv));
        }
      }
  }
}

template <int DT, int D, bool WHOLE>
cudaError_t launch_d(const KvParams &p, int num_sms, cudaStream_t stream) {
  auto kern = kv_attention_kernel<DT, D, WHOLE>;
  static std::atomic<uint64_t> set{0};
  cudaError_t e = allow_smem(kern, KvCfg<D>::kSmem, &set);
  if (e != cudaSuccess) return e;
  e = launch_programmatic(kern, num_sms, 32 * kKvWarps, KvCfg<D>::kSmem, stream, p);
  if (e != cudaSuccess) return e;
  const int all = num_sms * kKvWarps;
  const int64_t items = static_cast<int64_t>(p.batch) * p.items;
  const int add_rows = items >= num_sms ? (p.rows < 4 ? 4 : kAddThreads * 4 / D) : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(items < all ? items : all), static_cast<unsigned>(cdiv(p.rows, add_rows)));
  cfg.blockDim = dim3(kAddThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kv_add_kernel<DT, D>, p, all, add_rows);
  return e != cudaSuccess ? e : cudaGetLastError();
}

size_t slots_at(int num_sms) { return 256 + 256 * static_cast<size_t>(cdiv(num_sms * kKvWarps * (sizeof(CutItem) + sizeof(int32_t)), 256)); }

}  // namespace

// The first block is left alone (its first word is another call's error word); then the cut items and their parts.
size_t kv_attention_workspace_bytes(int, int n, int q_heads, int k_heads, int head_dim, int num_sms) {
  const int64_t rows = static_cast<int64_t>(n) * (q_heads / k_heads);
  const size_t d = head_dim <= 64 ? 64 : 128;
  return slots_at(num_sms) + static_cast<size_t>(2 * num_sms * kKvWarps) * (rows < 16 ? rows : 16) * (d + 4) * sizeof(float);
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
  p.cuts = reinterpret_cast<CutItem *>(ws + 256);
  p.cut = reinterpret_cast<int32_t *>(ws + 256 + static_cast<size_t>(num_sms) * kKvWarps * sizeof(CutItem));
  p.sums = reinterpret_cast<float *>(ws + slots_at(num_sms));
  p.ldq = a.ldq;
  p.ldo = a.ldo;
  p.pages = a.pages;
  p.batch = a.batch;
  p.n = a.n;
  p.max_pages = a.max_pages;
  p.q_heads = a.q_heads;
  p.k_heads = a.k_heads;
  p.head_dim = a.head_dim;
  p.page = a.page;
  p.r = a.q_heads / a.k_heads;
  p.row_tiles = static_cast<int>(cdiv(static_cast<int64_t>(a.n) * p.r, 16));
  p.rows = a.n * p.r < 16 ? a.n * p.r : 16;
  p.items = p.row_tiles * a.k_heads;
  p.scale = a.scale;
  p.page_div = make_fastdiv(static_cast<uint32_t>(a.page));
  p.r_div = make_fastdiv(static_cast<uint32_t>(p.r));
  auto go = [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    if (a.head_dim == 128) return launch_d<DT, 128, true>(p, num_sms, stream);
    if (a.head_dim > 64) return launch_d<DT, 128, false>(p, num_sms, stream);
    if (a.head_dim == 64) return launch_d<DT, 64, true>(p, num_sms, stream);
    return launch_d<DT, 64, false>(p, num_sms, stream);
  };
  return a.dtype == kDtypeBf16 ? go(std::integral_constant<int, kDtypeBf16>{}) : go(std::integral_constant<int, kDtypeF16>{});
}

}  // namespace w4
