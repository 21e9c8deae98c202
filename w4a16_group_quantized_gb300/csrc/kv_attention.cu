// w4_kv_attention: a few query rows of each sequence over the paged cache of e4m3 codes.
//
// For a sequence and key head the n query rows of the r query heads that share it are n * r rows (row = j * r + head), taken 16
// at a time as the M side of register-operand products (mma.sync m16n8k16, fp16 operands, fp32 sums): e4m3 codes
// are exact in fp16, and so are q's values (bf16 rows times a power of two that keeps them within fp16's range).
// For a tile of 16 keys, which lies in one page: S = q . codes, s = S * (k scale * softmax scale * log2 e), running maximum m
// and sum l of a row, w = 2^(s - m) in fp16, O = O * 2^(m_old - m) + v scale * (w . codes).
//
// A warp takes every 8th tile of its item and a lane copies to shared memory exactly the bytes that it will read
// (cp.async, 16 bytes each, zeros past the sequence's end), so that no barrier is needed until the 8 warps' sums are
// added at the end. Which keys and values of a head a lane holds follows from the fragments: of key 8 u + lane / 4 the
// quarter of the head that its place in the quad has, in 16-byte pieces; of keys 2 t, 2 t + 1 and those plus 8 (t = lane % 4)
// an eighth of the head, whose codes of two neighbouring keys are put side by side by byte permutes.
#include <atomic>

#include "e4m3.cuh"
#include "gemm_common.cuh"
#include "internal.h"
#include "mma.cuh"
#include "ptx.cuh"

namespace w4 {
namespace {

using namespace detail;

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kKvWarps = 8;
constexpr float kLog2e = 1.4426950408889634f;

struct KvParams {
  const uint16_t *q;
  const uint8_t *k_cache, *v_cache;
  const float *k_scale, *v_scale;
  const int32_t *table, *lens;
  uint16_t *out;
  int64_t ldq, ldo, pages;
  int batch, n, max_pages, q_heads, k_heads, head_dim, page, r, row_tiles;
  float scale;
  FastDiv page_div, r_div;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool there) {
  cp_async16_zfill(dst, src, there ? 16u : 0u);
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void *src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(there ? 8u : 0u) : "memory");
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
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}
// Whether one of the four codes of a word is NaN (0x7F or 0xFF).
__device__ __forceinline__ bool any_nan_code(uint32_t w) { return __vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu) != 0; }

// D: head_dim rounded up to 64 or 128.
template <int D>
struct KvCfg {
  static constexpr int kStages = 3;
  static constexpr int kPieces = D / 64;                 // 16-byte pieces of a key in a lane
  static constexpr int kVBytes = D / 8;                  // bytes of a value row in a lane
  static constexpr int kTileLane = 2 * 16 * kPieces + 4 * kVBytes;  // bytes of a tile in a lane
  static constexpr int kTileBytesWarp = 32 * kTileLane;
  static constexpr int kRing = kStages * kTileBytesWarp;
  static constexpr int kQBytes = D / 16 * 32 * 16;       // q in the fragments' order
  static constexpr int kSumRow = D + 4;                  // floats of a row of a warp's sums
  static constexpr int kSumBytes = kKvWarps * 16 * kSumRow * 4;
  static constexpr int kSmem = kKvWarps * kRing + kQBytes + kSumBytes;
};

template <int DT, int D>
__global__ void __launch_bounds__(32 * kKvWarps) kv_attention_kernel(const __grid_constant__ KvParams p) {
  using C = KvCfg<D>;
  constexpr int NT = D / 8;  // n-tiles of the output
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float row_m[kKvWarps][16], row_l[kKvWarps][16];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  uint4 *qf = reinterpret_cast<uint4 *>(smem);
  float *sums = reinterpret_cast<float *>(smem + C::kQBytes);
  const uint32_t ring = smem_u32(smem + C::kQBytes + C::kSumBytes) + warp * C::kRing;
  griddep_launch_dependents();
  griddep_wait();

  const int rt = blockIdx.x % p.row_tiles;
  const int h = blockIdx.x / p.row_tiles % p.k_heads;
  const int b = blockIdx.x / p.row_tiles / p.k_heads;
  const int rows = min(16, p.n * p.r - rt * 16);
  const int len = max(p.lens[b], 0);
  const int keys = min(len, p.max_pages * p.page);
  const int tiles = (keys + 15) / 16;

  // q of row i, values d: 0 past the item's rows and the head; bf16 rows times 2^-shift
  __shared__ float row_scale[16];
  for (int i = warp; i < 16; i += kKvWarps) {
    const int rho = rt * 16 + i;
    const int j = p.r_div.div(rho);
    const uint16_t *src = p.q + (static_cast<int64_t>(b) * p.n + j) * p.ldq + static_cast<int64_t>(h * p.r + rho - j * p.r) * p.head_dim;
    float v[D / 32];
    float most = 0.0f;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) {
      const int d = lane * (D / 32) + e;
      v[e] = i < rows && d < p.head_dim ? value_f32<DT>(src[d]) : 0.0f;
      most = fmaxf(most, fabsf(v[e]));
    }
    float mul = 1.0f;
    if (DT == kDtypeBf16) {
      most = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(most)));
      // the row's largest value to [2^10, 2^11): products with codes stay far from fp32's ends, and what falls below
      // fp16's smallest step, 2^-24, is below 2^-34 of the largest
      const int e = static_cast<int>(__float_as_uint(most) >> 23 & 0xFFu);
      const int up = min(max(137 - e, -126), 126);
      mul = e == 0 || e == 255 ? 1.0f : __uint_as_float(static_cast<uint32_t>(up + 127) << 23);
    }
    if (lane == 0) row_scale[i] = p.scale * kLog2e / mul;
    // value d of row i: lane 4 (i % 8) + t of step s, where d = (t + 4 (s / 4)) * 16 + 4 (s % 4) + {0 .. 3}
#pragma unroll
    for (int e = 0; e < D / 32; ++e) {
      const int d = lane * (D / 32) + e;
      const int piece = d / 16, s = piece / 4 * 4 + d % 16 / 4;
      uint16_t *to = reinterpret_cast<uint16_t *>(qf + s * 32 + 4 * (i % 8) + piece % 4);
      to[(d % 4 / 2) * 4 + (i / 8) * 2 + d % 2] = __half_as_ushort(__float2half_rn(v[e] * mul));
    }
  }
  __syncthreads();

  // how far this lane's two rows see
  int sees[2];
  float mul[2];
  int least = keys;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int rho = rt * 16 + g + 8 * i;
    const int j = min(p.r_div.div(rho), p.n - 1);
    sees[i] = min(max(len - p.n + j + 1, 0), keys);
    mul[i] = row_scale[g + 8 * i];
    least = min(least, sees[i]);
  }
  least = static_cast<int>(__reduce_min_sync(kAll, least));

  float o[NT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.0f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};

  // lane i holds what tile 32 * batch + i of this warp needs: its page, and the page's scales
  const int mine = tiles > warp ? (tiles - warp + kKvWarps - 1) / kKvWarps : 0;
  int at_page = -1;
  float at_ks = 0.0f, at_vs = 0.0f;
  auto look_up = [&](int first) {
    const int i = first + lane;
    at_page = -1;
    if (i < mine) {
      const int pi = p.page_div.div((warp + i * kKvWarps) * 16);
      const int at = p.table[static_cast<int64_t>(b) * p.max_pages + pi];
      if (at >= 0 && at < p.pages) {
        at_page = at;
        at_ks = p.k_scale[static_cast<int64_t>(at) * p.k_heads + h];
        at_vs = p.v_scale[static_cast<int64_t>(at) * p.k_heads + h];
      }
    }
  };
  auto copy = [&](int i, int page_at) {  // tile i of this warp, to its place in the ring
    const int key0 = (warp + i * kKvWarps) * 16;
    const int slot0 = key0 - p.page_div.div(key0) * p.page;
    const int64_t base = ((static_cast<int64_t>(page_at) * p.k_heads + h) * p.page + slot0) * p.head_dim;
    const uint32_t to = ring + i % C::kStages * C::kTileBytesWarp + lane * 16;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int c = 0; c < C::kPieces; ++c) {
        const int key = 8 * u + g, at = (t + 4 * c) * 16;
        const bool there = page_at >= 0 && key0 + key < keys && at < p.head_dim;
        cp_async16(to + (u * C::kPieces + c) * 512, p.k_cache + (there ? base + key * p.head_dim + at : 0), there);
      }
    const uint32_t tv = ring + i % C::kStages * C::kTileBytesWarp + 2 * C::kPieces * 512 + lane * C::kVBytes;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int key = 2 * t + c % 2 + c / 2 * 8, at = g * C::kVBytes;
      const bool there = page_at >= 0 && key0 + key < keys && at < p.head_dim;
      const uint8_t *src = p.v_cache + (there ? base + key * p.head_dim + at : 0);
      if (C::kVBytes == 16)
        cp_async16(tv + c * 32 * C::kVBytes, src, there);
      else
        cp_async8(tv + c * 32 * C::kVBytes, src, there);
    }
  };

  look_up(0);
  // tiles i .. i + kStages - 2 are on their way while tile i is worked on; the lookup of tile i + kStages - 1 may be of the
  // next 32, whose registers replace these: what the tiles in between need is kept
  int ring_page[C::kStages];
  float ring_ks[C::kStages], ring_vs[C::kStages];
  auto send = [&](int i) {
    if (i < mine) {
      if (i > 0 && i % 32 == 0) look_up(i);
      const int pg = __shfl_sync(kAll, at_page, i % 32);
      const float ks = __shfl_sync(kAll, at_ks, i % 32), vs = __shfl_sync(kAll, at_vs, i % 32);
#pragma unroll
      for (int s = 0; s < C::kStages - 1; ++s) ring_page[s] = ring_page[s + 1], ring_ks[s] = ring_ks[s + 1], ring_vs[s] = ring_vs[s + 1];
      ring_page[C::kStages - 1] = pg, ring_ks[C::kStages - 1] = ks, ring_vs[C::kStages - 1] = vs;
      copy(i, pg);
    } else {
#pragma unroll
      for (int s = 0; s < C::kStages - 1; ++s) ring_page[s] = ring_page[s + 1], ring_ks[s] = ring_ks[s + 1], ring_vs[s] = ring_vs[s + 1];
    }
    cp_commit();
  };
#pragma unroll
  for (int s = 0; s < C::kStages - 1; ++s) send(s);
  for (int i = 0; i < mine; ++i) {
    send(i + C::kStages - 1);  // (its place held tile i - 1, which is done)
    cp_wait<C::kStages - 1>();
    const int page_at = ring_page[0];
    const float ks = ring_ks[0], vs = ring_vs[0];
    const int key0 = (warp + i * kKvWarps) * 16;
    if (page_at < 0) continue;
    const uint32_t kt = ring + i % C::kStages * C::kTileBytesWarp + lane * 16;
    const uint32_t vt = ring + i % C::kStages * C::kTileBytesWarp + 2 * C::kPieces * 512 + lane * C::kVBytes;

    float s[2][4] = {};
#pragma unroll
    for (int c = 0; c < C::kPieces; ++c) {
      const uint4 k0 = lds128(kt + c * 512), k1 = lds128(kt + (C::kPieces + c) * 512);
      const uint32_t a[4] = {k0.x, k0.y, k0.z, k0.w}, d[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint4 qa = qf[(4 * c + w) * 32 + lane];
        mma_16816<kDtypeF16>(s[0], qa.x, qa.y, qa.z, qa.w, e4m3x2_f16x2(a[w] & 0xffffu), e4m3x2_f16x2(a[w] >> 16));
        mma_16816<kDtypeF16>(s[1], qa.x, qa.y, qa.z, qa.w, e4m3x2_f16x2(d[w] & 0xffffu), e4m3x2_f16x2(d[w] >> 16));
      }
    }
    const bool border = key0 + 16 > least;  // some row does not see all of the tile
    uint32_t hidden = 0;                    // of this lane's values, bit 4 u + e
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[u][e] *= ks * mul[e / 2];
        if (border && key0 + 8 * u + 2 * t + e % 2 >= sees[e / 2]) s[u][e] = -INFINITY, hidden |= 1u << (4 * u + e);
      }
    float alpha[2];
    bool moved = false;
#pragma unroll
    for (int i2 = 0; i2 < 2; ++i2) {
      float top = fmaxf(fmaxf(s[0][2 * i2], s[0][2 * i2 + 1]), fmaxf(s[1][2 * i2], s[1][2 * i2 + 1]));
      top = fmaxf(top, __shfl_xor_sync(kAll, top, 1));
      top = fmaxf(top, __shfl_xor_sync(kAll, top, 2));
      const float now = fmaxf(m[i2], top);
      alpha[i2] = now == m[i2] ? 1.0f : ex2(m[i2] - now);
      moved |= now != m[i2];
      m[i2] = now;
      float sum = 0.0f;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // (a row that sees nothing yet: -inf - -inf)
          const float w = hidden >> (4 * u + 2 * i2 + e) & 1u ? 0.0f : ex2(s[u][2 * i2 + e] - now);
          s[u][2 * i2 + e] = w;
          sum += w;
        }
      l[i2] = fmaf(l[i2], alpha[i2], sum);
    }
    if (__any_sync(kAll, moved)) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][e] *= alpha[e / 2];
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
    bool bad = false;
    if (border) {
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int w = 0; w < C::kVBytes / 4; ++w) bad |= any_nan_code(v[c][w]);
      bad |= !(fabsf(vs) < INFINITY);
      bad = __any_sync(kAll, bad);
    }
    // 0 * NaN is NaN: where a row does not see all of the tile and the tile holds NaN, each query's rows go by
    // themselves, with zeros in the place of what they do not see
    const int turns = bad ? p.n : 1;
    for (int turn = 0; turn < turns; ++turn) {
      const int limit = bad ? min(max(len - p.n + turn + 1, 0), keys) : keys;
      if (bad && limit <= key0) continue;
      bool on[2] = {true, true};
      uint32_t a[4] = {half2_bits(s[0][0], s[0][1]), half2_bits(s[0][2], s[0][3]), half2_bits(s[1][0], s[1][1]),
                       half2_bits(s[1][2], s[1][3])};
      if (bad) {
#pragma unroll
        for (int i2 = 0; i2 < 2; ++i2) on[i2] = p.r_div.div(rt * 16 + g + 8 * i2) == turn;
        if (!on[0]) a[0] = a[2] = 0;
        if (!on[1]) a[1] = a[3] = 0;
      }
      uint32_t x[4][C::kVBytes / 4];
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int w = 0; w < C::kVBytes / 4; ++w)
          x[c][w] = bad && key0 + 2 * t + c % 2 + c / 2 * 8 >= limit ? 0u : v[c][w];
#pragma unroll
      for (int w = 0; w < C::kVBytes / 4; ++w) {
        uint32_t pair[2][2] = {{__byte_perm(x[0][w], x[1][w], 0x5140), __byte_perm(x[0][w], x[1][w], 0x7362)},
                               {__byte_perm(x[2][w], x[3][w], 0x5140), __byte_perm(x[2][w], x[3][w], 0x7362)}};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t b0 = e % 2 ? pair[0][e / 2] >> 16 : pair[0][e / 2] & 0xffffu;
          const uint32_t b1 = e % 2 ? pair[1][e / 2] >> 16 : pair[1][e / 2] & 0xffffu;
          float d[4] = {};
          mma_16816<kDtypeF16>(d, a[0], a[1], a[2], a[3], e4m3x2_f16x2(b0), e4m3x2_f16x2(b1));
#pragma unroll
          for (int f = 0; f < 4; ++f)
            if (!bad || on[f / 2]) o[4 * w + e][f] = fmaf(vs, d[f], o[4 * w + e][f]);
        }
      }
    }
  }

  // the warps' sums: value d of row g (+ 8) is o[d % NT] of the lane whose columns 2 t, 2 t + 1 are d / NT
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    l[i] += __shfl_xor_sync(kAll, l[i], 1);
    l[i] += __shfl_xor_sync(kAll, l[i], 2);
    if (t == 0) row_m[warp][g + 8 * i] = m[i], row_l[warp][g + 8 * i] = l[i];
    float *to = sums + (warp * 16 + g + 8 * i) * C::kSumRow;
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int j = 0; j < NT; j += 4)
        *reinterpret_cast<float4 *>(to + (2 * t + e) * NT + j) =
            make_float4(o[j][2 * i + e], o[j + 1][2 * i + e], o[j + 2][2 * i + e], o[j + 3][2 * i + e]);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < rows * (D / 8); i += 32 * kKvWarps) {
    const int row = i / (D / 8), d = i % (D / 8) * 8;
    if (d >= p.head_dim) continue;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kKvWarps; ++w) top = fmaxf(top, row_m[w][row]);
    float sum = 0.0f, acc[8] = {};
    for (int w = 0; w < kKvWarps; ++w) {
      const float f = row_m[w][row] == top ? 1.0f : ex2(row_m[w][row] - top);
      sum = fmaf(row_l[w][row], f, sum);
      const float *from = sums + (w * 16 + row) * C::kSumRow + d;
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = fmaf(from[e], f, acc[e]);
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    const int rho = rt * 16 + row, j = p.r_div.div(rho);
    uint4 w;
    uint32_t *ww = &w.x;
#pragma unroll
    for (int e = 0; e < 4; ++e) ww[e] = out_bits2<DT>(acc[2 * e] * inv, acc[2 * e + 1] * inv);
    *reinterpret_cast<uint4 *>(p.out + (static_cast<int64_t>(b) * p.n + j) * p.ldo +
                               static_cast<int64_t>(h * p.r + rho - j * p.r) * p.head_dim + d) = w;
  }
}

template <int DT, int D>
cudaError_t launch_d(const KvParams &p, cudaStream_t stream) {
  auto kern = kv_attention_kernel<DT, D>;
  static std::atomic<uint64_t> set{0};
  const cudaError_t e = allow_smem(kern, KvCfg<D>::kSmem, &set);
  if (e != cudaSuccess) return e;
  return launch_programmatic(kern, p.batch * p.k_heads * p.row_tiles, 32 * kKvWarps, KvCfg<D>::kSmem, stream, p);
}

}  // namespace

size_t kv_attention_workspace_bytes(int, int, int, int, int, int) { return 256; }

cudaError_t launch_kv_attention(const KvAttentionArgs &a, void *, int, cudaStream_t stream) {
  KvParams p;
  p.q = static_cast<const uint16_t *>(a.q);
  p.k_cache = static_cast<const uint8_t *>(a.k_cache);
  p.v_cache = static_cast<const uint8_t *>(a.v_cache);
  p.k_scale = a.k_scale;
  p.v_scale = a.v_scale;
  p.table = a.table;
  p.lens = a.lens;
  p.out = static_cast<uint16_t *>(a.out);
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
  p.scale = a.scale;
  p.page_div = make_fastdiv(static_cast<uint32_t>(a.page));
  p.r_div = make_fastdiv(static_cast<uint32_t>(p.r));
  if (a.head_dim <= 64)
    return a.dtype == kDtypeBf16 ? launch_d<kDtypeBf16, 64>(p, stream) : launch_d<kDtypeF16, 64>(p, stream);
  return a.dtype == kDtypeBf16 ? launch_d<kDtypeBf16, 128>(p, stream) : launch_d<kDtypeF16, 128>(p, stream);
}

}  // namespace w4
