// w4_kv_append: new rows of keys and values into the paged cache of e4m3 codes with a scale for each page and head.
//
// The rows of a sequence that go into one page are a run. For each run and head: m = the largest finite |value|,
// need = the least 2^e with m <= 448 * 2^e, s = max(old scale, need) where the page goes on, else need; codes are
// e4m3(x / s), and rows that the page held are rescaled where s grew. Scales are powers of two: for a float type of 8
// bits any other scale keeps no more bits, and a page's rows survive a growing scale unchanged but for what
// falls below the type's range.
//
// A block takes a stretch of rows and does the runs that begin in it, so that no plan is needed: the stretch is a page long for
// prompts and a row for a decode step. What it has to know of a run (cu, lens, table) is read once for a few heads of k and v,
// and while one head's maximum is found and its values converted, which stay in registers between the two, the next
// one's are on their way. Bound by memory for prompts (16384 rows of 32 heads of 128: 68 us, 5.9 TB/s, 0.87 of a copy's rate);
// by latency (cu, lens, table, old scale, one after another) for a decode step (32 rows of 8 heads: 3.0 us).
#include <type_traits>

#include "e4m3.cuh"
#include "gemm_common.cuh"
#include "internal.h"
#include "mma.cuh"
#include "ptx.cuh"

namespace w4 {
namespace {

using namespace detail;

constexpr int kAppendThreads = 128;

struct AppendParams {
  const uint16_t *k, *v;
  uint8_t *k_cache, *v_cache;
  float *k_scale, *v_scale;
  const int32_t *table, *cu, *lens;
  int64_t T, ldk, ldv, pages;
  int batch, max_pages, heads, head_dim, page;
  int stretch;  // rows of a block
  int tasks;    // heads of k and of v that a block takes: k of heads h, h + 1, .. and v of them in turn
  FastDiv page_div, piece_div;
};

// The least e with m <= 448 * 2^e = 1.75 * 2^(e + 8), within [-100, 120] (m is 0 or finite and positive).
__device__ __forceinline__ int scale_exponent(float m) {
  const uint32_t bits = __float_as_uint(m);
  const int e = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return min(max(e, -100), 120);
}

__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

template <int DT>
constexpr uint32_t kInf = DT == kDtypeBf16 ? 0x7F80u : 0x7C00u;

// The larger sizes of two pairs of 16-bit values, as bits (which order them; infinities and NaN are above all others).
__device__ __forceinline__ uint32_t most2(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7FFF7FFFu); }
// Of those that are finite.
template <int DT>
__device__ __forceinline__ uint32_t most_finite2(uint32_t m, uint32_t w) {
  const uint32_t lo = w & 0x7FFFu, hi = w >> 16 & 0x7FFFu;
  return __vmaxu2(m, (lo < kInf<DT> ? lo : 0u) | (hi < kInf<DT> ? hi << 16 : 0u));
}

// Codes of four words' values / s, where 1 / s = inv is exact and all values are finite.
template <int DT>
__device__ __forceinline__ uint2 codes8(const uint4 &w, float inv) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
  uint32_t c[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float lo, hi;
    if (DT == kDtypeBf16) {
      lo = __uint_as_float(v[e] << 16), hi = __uint_as_float(v[e] & 0xffff0000u);
    } else {
      lo = value_f32<DT>(v[e] & 0xffffu), hi = value_f32<DT>(v[e] >> 16);
    }
    c[e] = f32_e4m3x2(lo * inv, hi * inv);
  }
  return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}
// Any values, any s: infinities become NaN (the conversion alone would make 448 of them).
template <int DT>
__device__ __noinline__ uint2 codes8_any(uint4 w, float s) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
  uint32_t c[4];
  for (int e = 0; e < 4; ++e) {
    float f[2];
    for (int i = 0; i < 2; ++i) {
      const uint32_t bits = v[e] >> (16 * i) & 0xffffu;
      f[i] = (bits & 0x7FFFu) >= kInf<DT> ? __uint_as_float(0x7FC00000u) : __fdiv_rn(value_f32<DT>(bits), s);
    }
    c[e] = f32_e4m3x2(f[0], f[1]);
  }
  return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

// A run: n rows of a sequence, from `row` on, into slots off .. of page `at`.
struct Run {
  int row, off, n, at;
};

// HELD: 16-byte pieces of a run that a thread keeps (what is more is read twice).
template <int DT, int HELD>
__device__ __forceinline__ void append_run(const AppendParams &p, const Run &run, int first, int last, uint32_t *most_of_warp) {
  const int pieces = p.head_dim / 8;  // 16-byte pieces of a row
  const int count = run.n * pieces;
  auto source = [&](int task, int i) {
    const int r = p.piece_div.div(i), h = task / 2;
    const int64_t ld = task % 2 ? p.ldv : p.ldk;
    return reinterpret_cast<const uint4 *>((task % 2 ? p.v : p.k) + (run.row + r) * ld + h * p.head_dim + 8 * (i - r * pieces));
  };
  uint4 next[HELD];
  auto load = [&](int task) {
#pragma unroll
    for (int j = 0; j < HELD; ++j) {
      const int i = j * kAppendThreads + threadIdx.x;
      next[j] = make_uint4(0, 0, 0, 0);
      if (i < count) next[j] = *source(task, i);
    }
  };
  load(first);  // (beside the table's entry)
  if (run.at < 0 || run.at >= p.pages) return;
  for (int task = first; task < last; ++task) {
    uint4 keep[HELD];
#pragma unroll
    for (int j = 0; j < HELD; ++j) keep[j] = next[j];
    const int64_t ph = static_cast<int64_t>(run.at) * p.heads + task / 2;
    float *scale = (task % 2 ? p.v_scale : p.k_scale) + ph;
    const float old = run.off > 0 ? *scale : 0.0f;
    if (task + 1 < last) load(task + 1);
    uint8_t *dst = (task % 2 ? p.v_cache : p.k_cache) + ph * p.page * p.head_dim;
    // the largest size, and whether it is finite; where it is not, the largest finite one
    uint32_t *most = most_of_warp + task % 2 * (kAppendThreads / 32);  // (a task's are read before those of the next but one are written)
    auto largest = [&](auto two) {
      uint32_t m2 = 0;
#pragma unroll
      for (int j = 0; j < HELD; ++j) m2 = two(two(two(two(m2, keep[j].x), keep[j].y), keep[j].z), keep[j].w);
      for (int i = HELD * kAppendThreads + threadIdx.x; i < count; i += kAppendThreads) {
        const uint4 w = *source(task, i);
        m2 = two(two(two(two(m2, w.x), w.y), w.z), w.w);
      }
      m2 = __reduce_max_sync(0xffffffffu, max(m2 & 0xffffu, m2 >> 16));
      if (threadIdx.x % 32 == 0) most[threadIdx.x / 32] = m2;
      __syncthreads();  // (everyone has read the old scale, too)
      return max(max(most[0], most[1]), max(most[2], most[3]));
    };
    uint32_t bits = largest([](uint32_t m, uint32_t w) { return most2(m, w); });
    const bool finite = bits < kInf<DT>;
    if (!finite) {
      __syncthreads();
      bits = largest([](uint32_t m, uint32_t w) { return most_finite2<DT>(m, w); });
    }
    const float need = power_of_two(scale_exponent(value_f32<DT>(bits)));
    const bool grows = !(old >= need);
    const float s = grows ? need : old;
    const uint32_t sb = __float_as_uint(s);
    const bool exact = finite && (sb & 0x7FFFFFu) == 0 && s >= 0x1p-126f && s <= 0x1p126f;
    const float inv = 1.0f / s;
    dst += run.off * p.head_dim;
    // (pieces of 8 codes follow one another as pieces of 8 values do)
#pragma unroll
    for (int j = 0; j < HELD; ++j) {
      const int i = j * kAppendThreads + threadIdx.x;
      if (i < count) reinterpret_cast<uint2 *>(dst)[i] = exact ? codes8<DT>(keep[j], inv) : codes8_any<DT>(keep[j], s);
    }
    for (int i = HELD * kAppendThreads + threadIdx.x; i < count; i += kAppendThreads)
      reinterpret_cast<uint2 *>(dst)[i] = exact ? codes8<DT>(*source(task, i), inv) : codes8_any<DT>(*source(task, i), s);
    dst -= run.off * p.head_dim;
    if (run.off > 0 && grows) {
      const float f = __fdiv_rn(old, s);
      for (int i = threadIdx.x; i < run.off * pieces; i += kAppendThreads) {
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
    if (threadIdx.x == 0) *scale = s;
  }
  __syncthreads();  // the maxima have been read
}

template <int DT, int HELD>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const __grid_constant__ AppendParams p) {
  __shared__ uint32_t most_of_warp[2 * (kAppendThreads / 32)];
  griddep_launch_dependents();
  griddep_wait();
  const int first = blockIdx.y * p.tasks, last = min(first + p.tasks, 2 * p.heads);
  const int T = static_cast<int>(p.T);
  int row = static_cast<int>(blockIdx.x) * p.stretch;
  const int stop = min(row + p.stretch, T);
  // the last sequence that begins at or before the stretch: each lane looks at one of 32 that cut what is left evenly
  int b = 0;
  for (int span = p.batch; span > 1;) {
    const int cut = (span + 31) / 32;
    const int at = b + static_cast<int>(threadIdx.x % 32) * cut;
    const uint32_t before = __ballot_sync(0xffffffffu, at < b + span && p.cu[at] <= row);
    const int top = before ? 31 - __clz(before) : 0;  // (cu ascends)
    const int end = b + span;
    b += top * cut;
    span = min(cut, end - b);
    if (cut == 1) break;
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
      Run run;
      run.row = row;
      run.off = static_cast<int>(pos) - pi * p.page;
      run.n = min(p.page - run.off, end - row);
      row += run.n;
      if (run.off != 0 && run.row != begin) continue;  // inside a run of another block
      run.at = p.table[static_cast<int64_t>(b) * p.max_pages + pi];
      append_run<DT, HELD>(p, run, first, last, most_of_warp);
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
  // a page's rows where there are enough of them to fill the device with blocks of a few heads each, else fewer
  p.stretch = 1;
  while (p.stretch < a.page && cdiv(a.T, p.stretch) * a.heads * 2 > 16 * num_sms) p.stretch *= 2;
  p.tasks = 1;
  while (p.tasks < 8 && cdiv(a.T, p.stretch) * cdiv(2 * a.heads, 2 * p.tasks) >= 8 * num_sms) p.tasks *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(cdiv(a.T, p.stretch)), static_cast<unsigned>(cdiv(2 * a.heads, p.tasks)));
  cfg.blockDim = dim3(kAppendThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // short pages need few registers, and more blocks are resident (21 pieces of up to 700 rows of 6 heads of 48, pages of
  // 16: 11.4 us with 8 pieces kept, 6.8 with 2; prompts into pages of 64 with heads of 128 need all 8 of them)
  const bool few = a.page * (a.head_dim / 8) <= 2 * kAppendThreads;
  auto go = [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    return few ? cudaLaunchKernelEx(&cfg, kv_append_kernel<DT, 2>, p) : cudaLaunchKernelEx(&cfg, kv_append_kernel<DT, 8>, p);
  };
  const cudaError_t e = a.dtype == kDtypeBf16 ? go(std::integral_constant<int, kDtypeBf16>{}) : go(std::integral_constant<int, kDtypeF16>{});
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace w4
