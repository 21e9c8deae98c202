// w4_kv_append: new rows of keys and values into the paged cache of e4m3 codes with a scale for each page and head.
//
// The rows of a sequence that go into one page are a run. For each run and head: m = the largest finite |value|,
// need = the least 2^e with m <= 448 * 2^e, s = max(old scale, need) where the page goes on, else need; codes are
// e4m3(x / s), and rows that the page held are rescaled where s grew. Scales are powers of two: for a float type of 8
// bits any other scale keeps no more bits, and a page's rows survive a growing scale unchanged but for what
// falls below the type's range.
//
// A block takes a stretch of rows of one head of k or v and does the runs that begin in it, so that no plan is needed: the
// stretch is a page long for prompts and a row for a decode step. A run's values stay in registers between the search
// for the maximum and the conversion. Bound by memory for prompts; by latency (cu, lens, table, old scale, one after
// another) for a decode step.
#include "e4m3.cuh"
#include "gemm_common.cuh"
#include "internal.h"
#include "mma.cuh"
#include "ptx.cuh"

namespace w4 {
namespace {

using namespace detail;

constexpr int kAppendThreads = 128;
constexpr int kHeldPieces = 8;  // 16-byte pieces of a run that a thread keeps

struct AppendParams {
  const uint16_t *k, *v;
  uint8_t *k_cache, *v_cache;
  float *k_scale, *v_scale;
  const int32_t *table, *cu, *lens;
  int64_t T, ldk, ldv, pages;
  int batch, max_pages, heads, head_dim, page;
  int stretch;  // rows of a block
  FastDiv page_div, piece_div;
};

// The least e with m <= 448 * 2^e = 1.75 * 2^(e + 8), within [-100, 120] (m is 0 or finite and positive).
__device__ __forceinline__ int scale_exponent(float m) {
  const uint32_t bits = __float_as_uint(m);
  const int e = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return min(max(e, -100), 120);
}

__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// x / s: a product where 1 / s is exact.
__device__ __forceinline__ float over(float x, float s, float inv, bool exact) { return exact ? x * inv : __fdiv_rn(x, s); }

// The code of a value; infinities become NaN (the conversion alone would make 448 of them).
template <int DT>
__device__ __forceinline__ float finite_or_nan(uint32_t bits) {
  const float x = value_f32<DT>(bits);
  constexpr uint32_t kInf = DT == kDtypeBf16 ? 0x7F80u : 0x7C00u;
  return (bits & 0x7FFFu) >= kInf ? __uint_as_float(0x7FC00000u) : x;
}

template <int DT>
__device__ __forceinline__ void most_of(uint32_t w, float *m) {
  constexpr uint32_t kInf = DT == kDtypeBf16 ? 0x7F80u : 0x7C00u;
  const uint32_t lo = w & 0x7FFFu, hi = w >> 16 & 0x7FFFu;
  if (lo < kInf) *m = fmaxf(*m, value_f32<DT>(lo));
  if (hi < kInf) *m = fmaxf(*m, value_f32<DT>(hi));
}

template <int DT>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const __grid_constant__ AppendParams p) {
  __shared__ float most_of_warp[kAppendThreads / 32];
  griddep_launch_dependents();
  griddep_wait();
  const int h = blockIdx.y;
  const bool of_v = blockIdx.z != 0;
  const uint16_t *x = (of_v ? p.v : p.k) + static_cast<int64_t>(h) * p.head_dim;
  const int64_t ld = of_v ? p.ldv : p.ldk;
  uint8_t *cache = of_v ? p.v_cache : p.k_cache;
  float *scales = of_v ? p.v_scale : p.k_scale;
  const int pieces = p.head_dim / 8;  // 16-byte pieces of a row
  const int T = static_cast<int>(p.T);

  int row = static_cast<int>(blockIdx.x) * p.stretch;
  const int stop = min(row + p.stretch, T);
  // the last sequence that begins at or before the stretch
  int b = 0;
  for (int lo = 0, hi = p.batch - 1; lo <= hi;) {
    const int mid = (lo + hi) / 2;
    if (p.cu[mid] <= row) {
      b = mid;
      lo = mid + 1;
    } else {
      hi = mid - 1;
    }
  }
  for (; b < p.batch && row < stop; ++b) {
    const int begin = max(p.cu[b], 0), end = min(p.cu[b + 1], T);
    const int held = max(p.lens[b], 0);
    if (row < begin) row = begin;
    // the first run that begins at `row` or after it
    while (row < end && row < stop) {
      const int64_t pos = static_cast<int64_t>(held) + (row - begin);
      if (pos >= static_cast<int64_t>(p.max_pages) * p.page) {
        row = end;
        break;
      }
      const int pi = p.page_div.div(static_cast<int>(pos));
      const int off = static_cast<int>(pos) - pi * p.page;
      const int left = p.page - off;
      const int n = min(left, end - row);
      if (off != 0 && row != begin) {  // inside a run of another block
        row += n;
        continue;
      }
      const int at = p.table[static_cast<int64_t>(b) * p.max_pages + pi];
      if (at >= 0 && at < p.pages) {
        const int64_t ph = static_cast<int64_t>(at) * p.heads + h;
        uint8_t *dst = cache + ph * p.page * p.head_dim;
        const int count = n * pieces;
        uint4 keep[kHeldPieces];
        float m = 0.0f;
#pragma unroll
        for (int j = 0; j < kHeldPieces; ++j) {
          const int i = j * kAppendThreads + threadIdx.x;
          keep[j] = make_uint4(0, 0, 0, 0);
          if (i < count) {
            const int r = p.piece_div.div(i);
            keep[j] = *reinterpret_cast<const uint4 *>(x + static_cast<int64_t>(row + r) * ld + 8 * (i - r * pieces));
          }
        }
#pragma unroll
        for (int j = 0; j < kHeldPieces; ++j) {
          most_of<DT>(keep[j].x, &m);
          most_of<DT>(keep[j].y, &m);
          most_of<DT>(keep[j].z, &m);
          most_of<DT>(keep[j].w, &m);
        }
        for (int i = kHeldPieces * kAppendThreads + threadIdx.x; i < count; i += kAppendThreads) {
          const int r = p.piece_div.div(i);
          const uint4 w = *reinterpret_cast<const uint4 *>(x + static_cast<int64_t>(row + r) * ld + 8 * (i - r * pieces));
          most_of<DT>(w.x, &m);
          most_of<DT>(w.y, &m);
          most_of<DT>(w.z, &m);
          most_of<DT>(w.w, &m);
        }
        // (positive floats are ordered as their bits)
        m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
        if (threadIdx.x % 32 == 0) most_of_warp[threadIdx.x / 32] = m;
        const float old = off > 0 ? scales[ph] : 0.0f;
        __syncthreads();
        m = fmaxf(fmaxf(most_of_warp[0], most_of_warp[1]), fmaxf(most_of_warp[2], most_of_warp[3]));
        const float need = power_of_two(scale_exponent(m));
        const bool grows = !(old >= need);
        const float s = grows ? need : old;
        __syncthreads();  // everyone has read the old scale and the maxima
        const uint32_t sb = __float_as_uint(s);
        const bool exact = (sb & 0x7FFFFFu) == 0 && s >= 0x1p-126f && s <= 0x1p126f;
        const float inv = 1.0f / s;
        auto put = [&](int i, const uint4 &w) {
          const uint32_t v[4] = {w.x, w.y, w.z, w.w};
          uint32_t c[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            c[e] = f32_e4m3x2(over(finite_or_nan<DT>(v[e] & 0xffffu), s, inv, exact), over(finite_or_nan<DT>(v[e] >> 16), s, inv, exact));
          const int r = p.piece_div.div(i);
          *reinterpret_cast<uint2 *>(dst + static_cast<int64_t>(off + r) * p.head_dim + 8 * (i - r * pieces)) =
              make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
        };
#pragma unroll
        for (int j = 0; j < kHeldPieces; ++j) {
          const int i = j * kAppendThreads + threadIdx.x;
          if (i < count) put(i, keep[j]);
        }
        for (int i = kHeldPieces * kAppendThreads + threadIdx.x; i < count; i += kAppendThreads) {
          const int r = p.piece_div.div(i);
          put(i, *reinterpret_cast<const uint4 *>(x + static_cast<int64_t>(row + r) * ld + 8 * (i - r * pieces)));
        }
        if (off > 0 && grows) {
          const float f = __fdiv_rn(old, s);
          for (int i = threadIdx.x; i < off * p.head_dim / 8; i += kAppendThreads) {
            uint2 *to = reinterpret_cast<uint2 *>(dst) + i;
            const uint2 w = *to;
            const uint32_t v[2] = {w.x, w.y};
            uint32_t c[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t a = e4m3x2_f16x2(v[e] & 0xffffu), d = e4m3x2_f16x2(v[e] >> 16);
              c[e] = f32_e4m3x2(value_f32<kDtypeF16>(a & 0xffffu) * f, value_f32<kDtypeF16>(a >> 16) * f) |
                     f32_e4m3x2(value_f32<kDtypeF16>(d & 0xffffu) * f, value_f32<kDtypeF16>(d >> 16) * f) << 16;
            }
            *to = make_uint2(c[0], c[1]);
          }
        }
        if (threadIdx.x == 0) scales[ph] = s;
      }
      row += n;
    }
  }
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs &a, int num_sms, cudaStream_t stream) {
  AppendParams p;
  p.k = static_cast<const uint16_t *>(a.k);
  p.v = static_cast<const uint16_t *>(a.v);
  p.k_cache = static_cast<uint8_t *>(a.k_cache);
  p.v_cache = static_cast<uint8_t *>(a.v_cache);
  p.k_scale = a.k_scale;
  p.v_scale = a.v_scale;
  p.table = a.table;
  p.cu = a.cu;
  p.lens = a.lens;
  p.T = a.T;
  p.ldk = a.ldk;
  p.ldv = a.ldv;
  p.pages = a.pages;
  p.batch = a.batch;
  p.max_pages = a.max_pages;
  p.heads = a.heads;
  p.head_dim = a.head_dim;
  p.page = a.page;
  p.page_div = make_fastdiv(static_cast<uint32_t>(a.page));
  p.piece_div = make_fastdiv(static_cast<uint32_t>(a.head_dim / 8));
  p.stretch = 1;
  while (p.stretch < a.page && cdiv(a.T, p.stretch) * a.heads * 2 > 16 * num_sms) p.stretch *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(cdiv(a.T, p.stretch)), static_cast<unsigned>(a.heads), 2);
  cfg.blockDim = dim3(kAppendThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = a.dtype == kDtypeBf16 ? cudaLaunchKernelEx(&cfg, kv_append_kernel<kDtypeBf16>, p)
                                              : cudaLaunchKernelEx(&cfg, kv_append_kernel<kDtypeF16>, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace w4
