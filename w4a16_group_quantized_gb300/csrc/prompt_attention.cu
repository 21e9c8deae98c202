// w4_prompt_attention: causal attention over packed prompts, on tcgen05.
//
// out[t, h] = sum_p w_p v_p / sum_p w_p, w_p = exp(scale * q . k_p) over the rows p <= t of t's sequence, with the running
// maximum m and sum l of a softmax: s = q . k * scale * log2 e, w = 2^(s - m), O = O * 2^(m_old - m) + w v. The maximum
// need not be the newest for that: while no score is above it by more than 2^8 as a weight, O and l are left as they are and the
// weights are simply larger than 1 (in fp32 sums; as 16 bits they are rounded to the type's half step of themselves, in fp16 to
// 2^-25 of the maximum in use where that is more), so that O is rescaled a few times in a row's life instead of at
// each step. The sum that divides is that of the unrounded weights: taking the rounded ones apart again for it made 8192 rows of 64
// heads of 128 660 us instead of 602, of 64 525 instead of 484, for an error of 1.16 to 1.22 times that of 32-bit weights instead of
// 1.27 to 1.30.
//
// A block takes 128 or 256 rows of one sequence and head, as one tile or two, which share the keys and values that it copies,
// 128 rows a step. Tensor memory holds for each tile the scores S (128 x 128 fp32, one row a lane), whose columns the 16-bit
// weights P then take as the second product's A operand, and O (128 x head_dim fp32): 256 columns a tile. Blocks of one tile go
// two to an SM, where one's beginning and end run beside the other's products; blocks of two read keys and values half as
// often. With heads of 64 and many blocks a step is 64 keys, and with 128 columns a tile four blocks go to an SM. Roles (8 or 12 warps):
//   4 softmax warps a tile  a thread a row: S to registers, maximum, weights, P; at the end O / l to memory
//   1 issue warp a tile   O += P V, the first half of the keys as soon as their weights are there, then the next
//                         S = Q K^T. One tile's softmax runs beside the other's products, and one warp's waits (some 130
//                         cycles each, even when over) beside the other's: with one warp for both tiles a step took 2825
//                         cycles, 550 of them its waits
//   1 copy warp           Q, then K and V of each step through a ring
//   1 looking warp        sees the V of the block's own rows (which their first queries do not all see)
// V is used as it stands, an MN-major operand. (Blocks that go four to an SM have 64 registers a thread, and spill some 40 bytes.)
//
// Rows that a query does not see have weight 0, but 0 * NaN is NaN. The rows of V that are the block's own, of which its first queries do
// not see all, go into the product with zeros in the place of rows behind the sequence's end and of values that are not
// finite; those are added at the end, read from memory again, to the rows that do see them.
//
// Measured (bf16): 8192 rows, 64 / 8 heads of 128: 613 us in a burst, 1.79 PFLOP/s, 0.94 of the rate of large products in a burst, 680
// in longer runs, where the clock falls (0.95 of that rate there); the tensor pipe is busy 80% of the time. Heads of 64 are
// bound by the softmax instead: as many exponentials for half of the products (8192 rows 488 us, 1.13 PFLOP/s). A prompt of
// 37 rows: 5.7 to 6.5 us.
//
// Every wait is bounded (ptx.cuh).
#include <atomic>

#include "gemm_common.cuh"
#include "internal.h"
#include "mma.cuh"
#include "ptx.cuh"

namespace w4 {
namespace {

using namespace detail;

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kTile = 128;         // query rows of a tile, and keys of a step
constexpr float kSlack = 8.0f;     // how far a score may pass the maximum in use (log2 of the weight)

struct PromptParams {
  const uint16_t *q, *k, *v;
  const int32_t *cu;
  uint16_t *out;
  uint32_t *err;
  int64_t ldq, ldk, ldv, ldo;
  int T, batch, q_heads, r, head_dim;
  float scale;  // times log2 e
  uint64_t wait_limit;
  int test_extra;
};

// D: head_dim rounded up to 64 or 128. TILES: of a block. KEYS: of a step. BLOCKS: to an SM.
template <int D, int TILES, int KEYS, int BLOCKS>
struct PromptCfg {
  static constexpr int kThreads = (TILES + 1) * 128;
  static constexpr int kQHalf = kTile * 128, kKvHalf = KEYS * 128;  // 64 values of a tile's rows, of a step's
  static constexpr int kQBytes = kQHalf * (D / 64), kKvBytes = kKvHalf * (D / 64);
  static constexpr int kStages = TILES == 2 || D == 64 && KEYS == 128 ? 5 : D == 64 ? 4 : 2;
  static constexpr int kSmem = TILES * kQBytes + kStages * kKvBytes + 1024;
  static constexpr uint32_t kO = TILES * KEYS;         // O's first column; O of the second tile D further
  static constexpr uint32_t kColumns = 512 / BLOCKS >= 256 ? 512 / BLOCKS : 128;
  static_assert(kO + TILES * D <= kColumns && kColumns * BLOCKS <= 512, "tensor memory");
  static constexpr int kRegsLaunch = TILES == 2 ? 168 : BLOCKS == 2 ? 128 : 64;
  static constexpr int kRegsSoftmax = TILES == 2 ? 216 : BLOCKS == 2 ? 208 : 96;
  static constexpr int kRegsOthers = TILES == 2 ? 72 : BLOCKS == 2 ? 48 : 32;
  static_assert(TILES * kRegsSoftmax + kRegsOthers <= (TILES + 1) * kRegsLaunch, "the registers that the block was launched with");
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int R>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ void unpack2(uint64_t v, float *lo, float *hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(*lo), "=f"(*hi) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// Two weights, the lower column's first.
template <int DT>
__device__ __forceinline__ uint32_t weights2(float lo, float hi) {
  uint32_t d;
  if (DT == kDtypeBf16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// Adds what is not finite of 8 of V's values (at v) of the rows from `first` up to and with `row` to 8 values of a row of the output (a
// weight is positive): infinities stay infinities, both signs or a NaN make NaN.
template <int DT>
__device__ __noinline__ uint4 add_odd(uint4 out, const uint16_t *v, int64_t ldv, int first, int row) {
  constexpr uint32_t kInf = DT == kDtypeBf16 ? 0x7F80u : 0x7C00u;
  float f[8];
  const uint32_t w[4] = {out.x, out.y, out.z, out.w};
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = value_f32<DT>(w[e / 2] >> (16 * (e % 2)) & 0xffffu);
  for (int key = first; key <= row; ++key) {
    const uint4 x = *reinterpret_cast<const uint4 *>(v + key * ldv);
    const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t bits = y[e / 2] >> (16 * (e % 2)) & 0xffffu;
      if ((bits & kInf) == kInf) f[e] += value_f32<DT>(bits);
    }
  }
  return make_uint4(out_bits2<DT>(f[0], f[1]), out_bits2<DT>(f[2], f[3]), out_bits2<DT>(f[4], f[5]), out_bits2<DT>(f[6], f[7]));
}

// What a block works on.
struct __align__(16) Work {
  int begin, len;  // the sequence
  int row0;        // the block's first row of it
  int head;
};

// The block's part: sequences have a block a head for every `rows` rows. The blocks that see most come first, whatever their
// sequence: block m of a sequence (rows m * rows ..) comes before block m - 1 of any. Up to and with block m there are
// sum max(0, blocks - m) of them over the sequences, so that m is found by halving. One warp.
__device__ __forceinline__ bool find_work(const PromptParams &p, int rows, Work *w) {
  const int lane = threadIdx.x % 32;
  int begin, len;
  auto count = [&](int b) {
    begin = len = 0;
    if (b < p.batch) {
      begin = min(max(p.cu[b], 0), p.T);
      len = max(min(p.cu[b + 1], p.T) - begin, 0);
    }
    return (len + rows - 1) / rows;
  };
  const int first = count(lane);
  auto all_from = [&](int m) {  // blocks m and up of all sequences
    int sum = max(first - m, 0);
    for (int b = 32; b < p.batch; b += 32) sum += max(count(b + lane) - m, 0);
    return static_cast<int>(__reduce_add_sync(kAll, sum));
  };
  int at = static_cast<int>(blockIdx.x) / p.q_heads;
  w->head = blockIdx.x % p.q_heads;
  if (at >= all_from(0)) return false;
  int most = first;
  for (int b = 32; b < p.batch; b += 32) most = max(most, count(b + lane));
  most = __reduce_max_sync(kAll, most);
  int m = 0;  // the largest with all_from(m) > at
  for (int lo = 1, hi = most - 1; lo <= hi;) {
    const int mid = (lo + hi) / 2;
    if (all_from(mid) > at) {
      m = mid;
      lo = mid + 1;
    } else {
      hi = mid - 1;
    }
  }
  at -= all_from(m + 1);
  for (int b = 0; b < p.batch; b += 32) {
    const bool mine = count(b + lane) > m;
    const uint32_t has = __ballot_sync(kAll, mine);
    if (at < __popc(has)) {
      const int from = __ffs(__ballot_sync(kAll, mine && __popc(has & ((1u << lane) - 1u)) == at)) - 1;  // the at-th that has one
      w->begin = __shfl_sync(kAll, begin, from);
      w->len = __shfl_sync(kAll, len, from);
      w->row0 = m * rows;
      return true;
    }
    at -= __popc(has);
  }
  return false;
}

// After a wait that gave up, the copies in flight land within some microseconds: ten milliseconds pass before the block leaves
// its shared memory.
__device__ __forceinline__ void let_copies_land() {
  const uint64_t t0 = clock_cycles();
  while (clock_cycles() - t0 < 20ull * 1000 * 1000) __nanosleep(1000);
}

template <int DT, int D, int TILES, int KEYS, int BLOCKS>
__global__ void __launch_bounds__(PromptCfg<D, TILES, KEYS, BLOCKS>::kThreads, BLOCKS)
    prompt_attention_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                            const __grid_constant__ CUtensorMap v_map, const __grid_constant__ PromptParams p) {
  using C = PromptCfg<D, TILES, KEYS, BLOCKS>;
  constexpr int S = C::kStages, kIssue = 4 * TILES;  // the first warp that is not a softmax warp
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t q_bar[2], full_bar[S], free_bar[TILES][S], s_bar[2], p_bar[2][2], o_bar[2], last_bar[2], look_bar[2], turn_bar[2], drain_bar[2];
  __shared__ uint32_t tmem_sh, abort_sh;
  __shared__ uint32_t odd_sh[2];  // V of the tile's last step holds what is not finite
  __shared__ Work work_sh;
  __shared__ bool any_sh;
  const uint32_t smem_base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const int warp = __shfl_sync(kAll, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  volatile uint32_t *abort_flag = &abort_sh;

  if (threadIdx.x == 32) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&q_bar[i]), 1 + (i == 0 ? p.test_extra : 0));
      mbar_init(smem_u32(&s_bar[i]), 1);
      mbar_init(smem_u32(&p_bar[i][0]), 4);
      mbar_init(smem_u32(&p_bar[i][1]), 4);
      mbar_init(smem_u32(&drain_bar[i]), 1);
      mbar_init(smem_u32(&o_bar[i]), 1);
      mbar_init(smem_u32(&last_bar[i]), 1);
      mbar_init(smem_u32(&look_bar[i]), 1);
      mbar_init(smem_u32(&turn_bar[i]), 1);
      odd_sh[i] = 0;
    }
    for (int i = 0; i < S; ++i) {
      mbar_init(smem_u32(&full_bar[i]), 1);
      for (int tile = 0; tile < TILES; ++tile) mbar_init(smem_u32(&free_bar[tile][i]), 1);
    }
    abort_sh = 0;
    fence_mbar_init();
  }
  // The next grid may begin only once every block has its tensor memory: a GEMM's blocks take theirs before they wait for this grid,
  // and on a shared SM this block would wait for them and they for it.
  if (warp == kIssue) {
    tmem_alloc(smem_u32(&tmem_sh), C::kColumns);
    tmem_relinquish();
    if (lane == 0) griddep_launch_dependents();
  }
  if (warp == kIssue + 2 && elect_one()) {
    prefetch_tensormap(&q_map);
    prefetch_tensormap(&k_map);
    prefetch_tensormap(&v_map);
  }
  griddep_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.err = 0;
  if (warp == 0) {
    Work w;
    const bool any = find_work(p, TILES * kTile, &w);
    if (lane == 0) {
      work_sh = w;
      any_sh = any;
    }
  }
  tc_fence_before();
  __syncwarp();
  cta_sync_all();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(kAll, tmem_sh, 0);
  if (!any_sh) {  // (the grid is for as many blocks as there could be)
    if (warp == kIssue) tmem_dealloc(tmem, C::kColumns);
    return;
  }
  const Work w = work_sh;
  const bool two = TILES == 2 && w.len > w.row0 + kTile;  // the second tile has rows
  // steps: before the block's own rows, of the first tile, of the block
  const int looked = w.row0 / KEYS;
  const int n0 = looked + (KEYS == kTile ? 1 : min((w.len - w.row0 + KEYS - 1) / KEYS, kTile / KEYS));
  const int n = n0 + (two ? 1 : 0);
  const uint32_t ring = smem_base + TILES * C::kQBytes;
  const uint32_t full0 = smem_u32(&full_bar[0]);

  if (warp < kIssue) {
    // ------------------------------------------------------------ softmax
    regs_up<C::kRegsSoftmax>();
    const int tile = warp / 4;
    const int r = warp % 4 * 32 + lane;  // the thread's row of the tile
    const uint32_t lanes = static_cast<uint32_t>(warp % 4 * 32) << 16;
    const uint32_t s_at = tmem + lanes + tile * KEYS, o_at = tmem + lanes + C::kO + tile * D;
    const uint32_t s_full = smem_u32(&s_bar[tile]), p_full = smem_u32(&p_bar[tile][0]);
    const int steps = tile == 0 ? n0 : two ? n0 + 1 : 0;
    const int own = KEYS == kTile ? steps - 1 : looked;  // the first step with keys that not all rows of the tile see
    const uint64_t scale2 = pack2(p.scale, p.scale);
    float m = -INFINITY;
    float l = 0.0f;
    bool ok = true;
    for (int i = 0; i < steps; ++i) {
      ok = warp_wait(s_full, i & 1, abort_flag, p.err, p.wait_limit);
      if (!ok) break;
      tc_fence_after();
      constexpr int N32 = KEYS / 32;
      uint32_t s[N32][32];
#pragma unroll
      for (int c = 0; c < N32; ++c) tmem_ld_32x32b_x32(s_at + 32 * c, s[c]);
      tmem_wait_ld();
      if (i >= own) {
        const int last = KEYS == kTile ? r : r - (i - own) * KEYS;
#pragma unroll
        for (int c = 0; c < N32; ++c)
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (32 * c + j > last) s[c][j] = 0xFF800000u;  // -inf
      }
      // the first half's weights by the maximum in use, and the newest maximum beside them: for most steps the one in use stays
      auto row_top = [&]() {
        float top[N32];
#pragma unroll
        for (int c = 0; c < N32; ++c) {
          top[c] = __uint_as_float(s[c][0]);
#pragma unroll
          for (int j = 1; j + 1 < 32; j += 2) top[c] = max3(top[c], __uint_as_float(s[c][j]), __uint_as_float(s[c][j + 1]));
          top[c] = fmaxf(top[c], __uint_as_float(s[c][31]));
        }
        if constexpr (N32 == 2) return max3(top[0], top[1], m);
        else return max3(max3(top[0], top[1], top[N32 - 2]), top[N32 - 1], m);
      };
      uint64_t off2, sum[2];
      uint32_t w2[KEYS / 4];
      auto weights = [&](int half) {
#pragma unroll
        for (int j = 0; j < KEYS / 4; ++j) {
          const int c = half * (N32 / 2) + j / 16;
          const uint64_t e = fma2(pack2(__uint_as_float(s[c][2 * (j % 16)]), __uint_as_float(s[c][2 * (j % 16) + 1])), scale2, off2);
          float a, b;
          unpack2(e, &a, &b);
          a = ex2(a);
          b = ex2(b);
          sum[j & 1] = add2(sum[j & 1], pack2(a, b));
          w2[j] = weights2<DT>(a, b);
        }
      };
      auto hand_over = [&](int half) {
        if constexpr (KEYS == 128)
          tmem_st_32x32b_x32(s_at + 32 * half, w2);
        else
          tmem_st_32x32b_x16(s_at + 16 * half, w2);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + 8 * half);
      };
      // (a loop, so that the code is there once: it fills much of the instruction cache)
#pragma unroll 1
      for (;;) {
        const float off = m == -INFINITY ? 0.0f : -m * p.scale;
        off2 = pack2(off, off);
        sum[0] = sum[1] = 0ull;
        weights(0);
        const float top = row_top();
        // (a row's own scores alone say when its maximum moves: what stands beside it does not change its roundings)
        const bool passed = (top - m) * p.scale > kSlack;
        if (!__any_sync(kAll, passed)) break;
        const float now = passed ? top : m;
        if (i > 0) {
          // (the step before this one's S is complete, and with it O)
          const float alpha = now == m ? 1.0f : ex2((m - now) * p.scale);
          l *= alpha;
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            uint32_t o[16];
            tmem_ld_32x32b_x16(o_at + 16 * c, o);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
            tmem_st_32x32b_x16(o_at + 16 * c, o);
          }
        }
        m = now;
      }
      hand_over(0);
      weights(1);
      hand_over(1);
      float a, b;
      unpack2(add2(sum[0], sum[1]), &a, &b);
      l += a + b;
    }
    if (ok && steps > 0) ok = warp_wait(smem_u32(&o_bar[tile]), 0, abort_flag, p.err, p.wait_limit);
    for (int i = 0; i < (KEYS == kTile ? tile + 1 : steps - looked); ++i)
      if (ok && steps > 0) ok = warp_wait(smem_u32(&look_bar[i]), 0, abort_flag, p.err, p.wait_limit);
    if (ok && steps > 0) {
      tc_fence_after();
      // (the block's place is read again: in registers through the loop it cost the scores theirs)
      Work e;
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(e.begin), "=r"(e.len), "=r"(e.row0), "=r"(e.head)
                   : "r"(smem_u32(&work_sh))
                   : "memory");
      const int row = e.row0 + tile * kTile + r;
      // (the second tile's rows see all of the first one's last V)
      const bool odd = (*static_cast<volatile uint32_t *>(&odd_sh[0]) | *static_cast<volatile uint32_t *>(&odd_sh[KEYS == kTile ? tile : steps - looked - 1])) != 0;
      const float inv = 1.0f / l;
      // each warp's rows by way of the tile's place of Q, which is done with, so that they are stored as whole lines; the 16-byte
      // pieces of a row are exchanged against bank conflicts
      constexpr int kPieces = D / 8;
      const uint32_t place = smem_base + tile * C::kQBytes + warp % 4 * 32 * D * 2;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        tmem_ld_32x32b_x32(o_at + 32 * c, o);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            x[e] = weights2<DT>(__uint_as_float(o[8 * j + 2 * e]) * inv, __uint_as_float(o[8 * j + 2 * e + 1]) * inv);
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(place + lane * D * 2 + 16 * ((4 * c + j) ^ (lane % kPieces))),
                       "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3])
                       : "memory");
        }
      }
      __syncwarp();
      uint16_t *out = p.out + static_cast<int64_t>(e.begin + row - lane) * p.ldo + static_cast<int64_t>(e.head) * p.head_dim;
#pragma unroll 4
      for (int i = lane; i < 32 * kPieces; i += 32) {
        const int rr = i / kPieces, c = i % kPieces;
        if (row - lane + rr < e.len && 8 * c < p.head_dim) {
          uint4 x = lds128(place + rr * D * 2 + 16 * (c ^ (rr % kPieces)));
          if (odd)
            x = add_odd<DT>(x, p.v + static_cast<int64_t>(e.head / p.r) * p.head_dim + 8 * c, p.ldv, e.begin + e.row0, e.begin + row - lane + rr);
          *reinterpret_cast<uint4 *>(out + rr * p.ldo + 8 * c) = x;
        }
      }
    }
  } else {
    regs_down<C::kRegsOthers>();
    if (warp < kIssue + TILES) {
      // -------------------------------------------------------- products
      const int tile = warp - kIssue;
      const int steps = tile == 0 ? n0 : two ? n : 0;
      constexpr uint32_t qk = idesc_f16_f32(kTile, KEYS, DT == kDtypeBf16), pv = idesc_f16_f32(kTile, D, DT == kDtypeBf16, true);
      const uint32_t s_at = tmem + tile * KEYS, o_at = tmem + C::kO + tile * D;
      const uint32_t free0 = smem_u32(&free_bar[tile][0]);
      const uint32_t s_full = smem_u32(&s_bar[tile]), p_full = smem_u32(&p_bar[tile][0]);
      auto scores = [&](uint32_t stage) {
        const uint64_t a = sw128_kmajor_desc(smem_base + tile * C::kQBytes), b = sw128_kmajor_desc(ring + stage * C::kKvBytes);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_f16_ss(s_at, a + static_cast<uint64_t>(kk / 4 * (C::kQHalf >> 4) + kk % 4 * 2),
                     b + static_cast<uint64_t>(kk / 4 * (C::kKvHalf >> 4) + kk % 4 * 2), qk, kk > 0);
        mma_commit(s_full);
      };
      auto values = [&](uint32_t stage, int half, bool first) {
        const uint64_t b = sw128_mnmajor_desc(ring + stage * C::kKvBytes, C::kKvHalf);
#pragma unroll
        for (int kk = half * (KEYS / 32); kk < (half + 1) * (KEYS / 32); ++kk)
          mma_f16_ts(o_at, s_at + kk * 8, b + static_cast<uint64_t>(kk * (2048 >> 4)), pv, !first || kk > 0);
      };
      auto landed = [&](int item) {
        return warp_wait(full0 + 8 * static_cast<uint32_t>(item % S), (item / S) & 1, abort_flag, p.err, p.wait_limit);
      };
      bool ok = steps > 0 && warp_wait(smem_u32(&q_bar[tile]), 0, abort_flag, p.err, p.wait_limit) && landed(0);
      if (ok) {
        tc_fence_after();
        if (elect_one()) {
          scores(0);
          mma_commit(free0);
        }
        __syncwarp();
      }
      for (int i = 0; ok && i < steps; ++i) {
        const uint32_t vs = static_cast<uint32_t>((2 * i + 1) % S), ks = static_cast<uint32_t>((2 * i + 2) % S);
        // (the looking warp has waited for the last steps' V, and may have changed it)
        ok = i < looked ? landed(2 * i + 1) : warp_wait(smem_u32(&look_bar[i - looked]), 0, abort_flag, p.err, p.wait_limit);
        if (ok && i + 1 < steps) ok = landed(2 * i + 2);
        // the tiles' products go in turns: run together they would take twice as long each and leave the tensor pipe idle together
        if (ok && two && (tile == 0 ? i > 0 : i < n0))
          ok = warp_wait(smem_u32(&turn_bar[tile]), (tile == 0 ? i - 1 : i) & 1, abort_flag, p.err, p.wait_limit);
        if (ok) ok = warp_wait(p_full, i & 1, abort_flag, p.err, p.wait_limit);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) values(vs, 0, i == 0);
        __syncwarp();
        ok = warp_wait(p_full + 8, i & 1, abort_flag, p.err, p.wait_limit);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          values(vs, 1, false);
          mma_commit(free0 + 8 * vs);
          if (i + 1 < steps) {
            scores(ks);
            mma_commit(free0 + 8 * ks);
          } else {
            mma_commit(smem_u32(&o_bar[tile]));
          }
          if (two) mbar_arrive(smem_u32(&turn_bar[1 - tile]));
        }
        __syncwarp();
      }
      const bool aborted = __any_sync(kAll, *abort_flag != 0);
      if (aborted) {
        if (elect_one()) mma_commit(smem_u32(&drain_bar[tile]));
        __syncwarp();
        drain_wait(smem_u32(&drain_bar[tile]), 0);
      }
    } else if (warp == kIssue + 2) {
      // ---------------------------------------------------------- copies
      auto load = [&](const CUtensorMap *map, uint32_t to, int half_bytes, int head, int row, uint32_t bar) {
        mbar_arrive_expect_tx(bar, half_bytes * (D / 64));
#pragma unroll
        for (int half = 0; half < D / 64; ++half) tma_load_3d(to + half * half_bytes, map, 64 * half, head, row, bar);
      };
      const int kv_head = w.head / p.r;
      bool ok = true;
      if (elect_one()) load(&q_map, smem_base, C::kQHalf, w.head, w.begin + w.row0, smem_u32(&q_bar[0]));
      __syncwarp();
      for (int item = 0; item < 2 * n; ++item) {
        const uint32_t stage = static_cast<uint32_t>(item % S);
        if (item >= S)
          for (int tile = 0; tile < (two ? 2 : 1); ++tile)
            ok = ok && warp_wait(smem_u32(&free_bar[tile][stage]), (item / S - 1) & 1, abort_flag, p.err, p.wait_limit);
        if (!ok) break;
        if (elect_one()) {
          // the last steps' V signals barriers of its own, which have one phase: the looking warps do not follow the ring
          const uint32_t bar = item % 2 && item / 2 >= looked ? smem_u32(&last_bar[item / 2 - looked]) : full0 + 8 * stage;
          load(item % 2 ? &v_map : &k_map, ring + stage * C::kKvBytes, C::kKvHalf, kv_head, w.begin + item / 2 * KEYS, bar);
          if (item == 0 && two) load(&q_map, smem_base + C::kQBytes, C::kQHalf, w.head, w.begin + w.row0 + kTile, smem_u32(&q_bar[1]));
        }
        __syncwarp();
      }
    } else if (warp == kIssue + 3) {
      // ------------------------- V of the steps with the block's own rows (its places are not used again)
      // (this wait lasts all the block's steps, each of which has the limit; a warp that gives up within one ends it)
      const uint64_t limit = __umul64hi(p.wait_limit, n) ? ~0ull : p.wait_limit * n;
      for (int tile = 0; tile < n - looked; ++tile) {
        const int step = looked + tile;
        const uint32_t stage = static_cast<uint32_t>((2 * step + 1) % S);
        if (!warp_wait(smem_u32(&last_bar[tile]), 0, abort_flag, p.err, limit)) break;
        const int live = min(w.len - step * KEYS, KEYS);  // rows of the sequence in it
        const uint32_t at = ring + stage * C::kKvBytes;
        // an exponent of all ones: one more carries into the sign's place
        constexpr uint32_t kInf = DT == kDtypeBf16 ? 0x7F807F80u : 0x7C007C00u, kOne = DT == kDtypeBf16 ? 0x00800080u : 0x04000400u;
        uint32_t carries = 0;
        for (int h = 0; h < D / 64; ++h) {
          const uint32_t end = at + h * C::kKvHalf + live * 128, stop = at + (h + 1) * C::kKvHalf;
          uint32_t i = at + h * C::kKvHalf + 16 * lane;
#pragma unroll 8
          for (; i < end; i += 512) {
            const uint4 x = lds128(i);
            carries |= ((x.x & kInf) + kOne) | ((x.y & kInf) + kOne) | ((x.z & kInf) + kOne) | ((x.w & kInf) + kOne);
          }
          for (; i < stop; i += 512) asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(i), "r"(0u) : "memory");
        }
        const bool odd = __any_sync(kAll, (carries & 0x80008000u) != 0);
        if (odd) {
          for (int h = 0; h < D / 64; ++h)
#pragma unroll 1
            for (uint32_t i = at + h * C::kKvHalf + 16 * lane; i < at + h * C::kKvHalf + live * 128; i += 512) {
              const uint4 x = lds128(i);
              auto finite = [&](uint32_t w) {
                const uint32_t bad = ((w & kInf) + kOne) & 0x80008000u;
                return w & ~((bad >> 15) * 0xffffu);
              };
              asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(i), "r"(finite(x.x)), "r"(finite(x.y)), "r"(finite(x.z)),
                           "r"(finite(x.w))
                           : "memory");
            }
        }
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) {
          odd_sh[tile] = odd;
          mbar_arrive(smem_u32(&look_bar[tile]));
        }
      }
    }
  }

  tc_fence_before();
  __syncwarp();
  cta_sync_all();
  if (*abort_flag) let_copies_land();  // (else every copy has been waited for)
  if (warp == kIssue) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kColumns);
  }
}

template <int DT, int D, int TILES, int KEYS, int BLOCKS>
cudaError_t launch_tiles(const PromptArgs &a, const PromptParams &p, cudaStream_t stream) {
  auto kern = prompt_attention_kernel<DT, D, TILES, KEYS, BLOCKS>;
  using C = PromptCfg<D, TILES, KEYS, BLOCKS>;
  static std::atomic<uint64_t> set{0};
  const cudaError_t e = allow_smem(kern, C::kSmem, &set);
  if (e != cudaSuccess) return e;
  CUtensorMap q_map, k_map, v_map;
  const int k_heads = a.k_heads;
  if (!make_heads_map(&q_map, a.q, a.T, a.q_heads, a.head_dim, a.ldq, kTile, DT) ||
      !make_heads_map(&k_map, a.k, a.T, k_heads, a.head_dim, a.ldk, KEYS, DT) ||
      !make_heads_map(&v_map, a.v, a.T, k_heads, a.head_dim, a.ldv, KEYS, DT))
    return cudaErrorInvalidValue;
  const int64_t blocks = (a.T / (TILES * kTile) + a.batch) * a.q_heads;
  return launch_programmatic(kern, static_cast<int>(blocks), C::kThreads, C::kSmem, stream, q_map, k_map, v_map, p);
}

// One tile or two a block (bf16, us, one / two). Heads of 64: 8192 rows x 64 heads 513 / 561, nine prompts of up to 1900 rows x 24
// heads 28 / 36, four of 256 x 32 8.5 / 7.8. Heads of 128: 8192 x 64 675 / 650, 4096 x 2 x 32 213 / 200, 2048 x 32 37.9 / 37.0,
// 1000 x 8 14.4 / 18.1: two, where they are a block for each SM and prompts are long enough for whole ones (64 x 128 x 32 heads 113 / 202,
// 128 x 64 66 / 108, 256 x 64 138 / 147, up to 500 x 64 83 / 120, 300 x 40 136 / 163; 512 x 32 148 / 145, 1000 x 16 188 / 177).
// Heads of 64, steps of 128 keys and two blocks an SM / of 64 and four: a step of 64 takes nearly as long as one of 128, but more of them
// run beside each other, which pays where there are many blocks for each place. With the tiles an SM: 16 x 256 x 16 heads (3.4)
// 13.1 / 11.9, 8 x 1000 x 8 (3.3) 18.9 / 23.2, 2048 x 32 (3.4) 25.8 / 38.2, 4096 x 24 (5.1) 60.5 / 72.4, 2048 x 48 (5.1) 39.2 / 40.5, 8 x 1000 x
// 12 (5.0) 28.1 / 24.5, x 16 (6.6) 37.1 / 31.2, 16 x 256 x 32 (6.7) 26.7 / 19.6, 4096 x 32 (6.7) 76.4 / 74.6, 8192 x 16 (6.7) 127 / 138, x 24 (10.1)
// 188 / 191, twenty of up to 1000 x 16 (8.1) 42.1 / 34.1, 4096 x 64 (13.5) 146 / 139, nine of up to 1900 x 32 (16.4) 102 / 86, 8192 x 64 (27) 520 /
// 488. Taken from 6 tiles an SM on, where prompts are longer than 4096 rows on average from 12 on.
template <int DT>
cudaError_t launch_type(const PromptArgs &a, const PromptParams &p, int num_sms, cudaStream_t stream) {
  const bool lengthy = a.T > 4096 * static_cast<int64_t>(a.batch);
  if (a.head_dim <= 64)
    return cdiv(a.T, kTile) * a.q_heads < (lengthy ? 12 : 6) * num_sms ? launch_tiles<DT, 64, 1, 128, 2>(a, p, stream)
                                                                         : launch_tiles<DT, 64, 1, 64, 4>(a, p, stream);
  const bool few = cdiv(a.T, 2 * kTile) * a.q_heads < num_sms, brief = a.T < 4 * kTile * static_cast<int64_t>(a.batch);
  return few || brief ? launch_tiles<DT, 128, 1, 128, 2>(a, p, stream)
                                                    : launch_tiles<DT, 128, 2, 128, 1>(a, p, stream);
}

}  // namespace

cudaError_t launch_prompt_attention(const PromptArgs &a, void *workspace, int num_sms, cudaStream_t stream) {
  PromptParams p;
  p.q = static_cast<const uint16_t *>(a.q);
  p.k = static_cast<const uint16_t *>(a.k);
  p.v = static_cast<const uint16_t *>(a.v);
  p.cu = a.cu;
  p.out = static_cast<uint16_t *>(a.out);
  p.err = static_cast<uint32_t *>(workspace);
  p.ldq = a.ldq;
  p.ldk = a.ldk;
  p.ldv = a.ldv;
  p.ldo = a.ldo;
  p.T = static_cast<int>(a.T);
  p.batch = a.batch;
  p.q_heads = a.q_heads;
  p.r = a.q_heads / a.k_heads;
  p.head_dim = a.head_dim;
  p.scale = a.scale * 1.4426950408889634f;
  p.wait_limit = a.wait_limit ? a.wait_limit : kWaitLimitCycles;
  p.test_extra = a.test_timeout ? 1 : 0;
  return a.dtype == kDtypeBf16 ? launch_type<kDtypeBf16>(a, p, num_sms, stream) : launch_type<kDtypeF16>(a, p, num_sms, stream);
}

}  // namespace w4
