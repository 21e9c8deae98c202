// The experts' products for many rows an expert, on tcgen05 (the formulas and the few-row form: experts.cu).
//
// As in gemm.cu the weights are the MMA's M = 128 side and the rows of `in` its N side; A comes from tensor memory,
// where dequant warps store it, and B from shared memory. Unlike there, A is the integers q - z, exactly, and a
// group's sum is multiplied by its 32-bit scale outside of the tensor cores: no weight is rounded, so that the one
// 16-bit rounding between x and y is that of h. The price is that every group's sums leave tensor memory once
// (128 x 128 values per 128 k, a packed 32-bit multiply-add for two of them).
//
// A unit is one 128-row weight tile x one tile of up to BN rows of one expert; the CTAs take units in turn and walk K in
// chunks of CB blocks of 64, with no stop between units. Roles (24 or 32 warps, one CTA a SM):
//   1 row warp         copies the rows of `in`, which stand in the sort's order, with the 128-byte swizzle, one box a
//                      block (three idle warps fill up its warpgroup)
//   2 weight warps     copy the chunks' codes, and their group records, in bulk, through a ring of their own
//   2 MMA warps        take the chunks in turn, each into an accumulator of its own that the chunk starts from zero
//   8 dequant warps    two warpgroups take the chunks in turn: thread r stores row r's q - z in tensor memory and its
//                      scale in a ring in shared memory
//   8 or 16 sum warps  a warpgroup for each 32 rows of `in`: add scale * (chunk's sums) to their 32-bit registers, and
//                      write h or the output at a unit's end
// SUB = 2: a chunk's halves (64 k, or 32 for one block) lie in different groups, each with an accumulator of its own.
//
// Barriers, each waited for in every phase and in order (chunk c; S stages of rows, W of weights):
//   go[c % S]        what the chunk's MMAs need: its rows have landed, its A operand is stored, and its accumulator has
//                    been read (one barrier for the three: each wait costs an MMA warp some 200 cycles, even when over)
//   wfull[c % W], wfree[c % W]   its codes and records have landed; a dequant warpgroup has read them
//   free[c % 2][c / 2 % 2]   its MMAs are complete, for the dequant warps: the A slot is free
//   done[c % S]      its MMAs are complete, for the others: the rows' stage is free, its sums can be read
// The sum warps have read chunk c's sums before the MMAs of c + 2 or, with two accumulators an MMA warp, c + 4 start, hence
// before done of those: the scale ring's eight places (a dequant warp writes c + 8's after free of c + 4) and done's
// parity (S is at least 4, or 6 with two) are never overtaken.
// Every wait is bounded (ptx.cuh).
//
// Measured (bf16, 64 experts of 2048 x 1024, 4096 rows of 8 choices): 279 us for gate/up and 160 for down, 0.98 and 0.86
// PFLOP/s; the tensor pipe is 44% busy and the issue slots 77%: some 800 warp instructions an SM quarter and chunk of 128 x 128 x 128 (dequant 270, sums
// 270) where the products take 512 cycles.
// tcgen05 instructions are issued under elect.sync, which keeps their operands in uniform registers: by "lane 0" an
// MMA took 125 cycles to issue, so 40. Gathering x's rows here, by 16-byte asynchronous copies of 128 threads, took 1200
// cycles a chunk, and by four-row tensor copies 280 instructions of an SM quarter (gate/up 354 us): they are copied into
// order once before (24 us). Measured no faster: one MMA warp, or two with three barriers each, one ring for rows and
// weights, sum warps of 64 columns, waits that poll or sleep longer.
#include <atomic>

#include "experts.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace w4 {
namespace {

using namespace detail;

template <int BN, int CB, int SUB>
struct TCfg {
  static constexpr int kSumGroups = BN / 32;                     // warpgroups that add, 32 rows of `in` each
  static constexpr int kThreads = 4 * 128 + kSumGroups * 128;    // 768 (BN = 64) or 1024
  // BN = 128: 64 registers a thread at launch, dealt out anew by warpgroup
  static constexpr bool kDeal = BN == 128;
  static constexpr int kRegsRows = 56, kRegsIssue = 40, kRegsDequant = 64, kRegsSum = 72;
  static_assert(!kDeal || kRegsRows + kRegsIssue + 2 * kRegsDequant + kSumGroups * kRegsSum <= 64 * kThreads / 128,
                "the registers that the block was launched with");
  static constexpr int kXSub = BN * 128;  // one block of 64 k of BN rows
  static constexpr int kXBytes = CB * kXSub;
  static constexpr int kCodeBytes = CB * kTileBytes;
  static constexpr int kSubK = CB * kTK / SUB;            // k of an accumulator: a group's part of a chunk
  static constexpr int kWBytes = kCodeBytes + SUB * 384;  // codes, group records (320 bytes each)
  // two rings: rows wait for their turn in the tensor cores, codes only until a dequant warp has read them
  static constexpr int kXStages = BN == 128 ? (CB == 2 ? 4 : 8) : (CB == 2 ? 6 : 8);
  static constexpr int kWStagesRaw = (214 * 1024 - kXStages * kXBytes) / kWBytes;
  static constexpr int kWStages = kWStagesRaw > 16 ? 16 : kWStagesRaw;
  static constexpr int kScaleSlots = 8;
  static constexpr int kSmemBytes = kXStages * kXBytes + kWStages * kWBytes + 1024;
  static constexpr int kASlotCols = CB * 32;   // 128 rows x 64 16-bit values: 32 columns a block
  // accumulators of each MMA warp; a second one where tensor memory has room
  static constexpr int kDBufs = SUB * BN <= 64 ? 2 : 1;
  static constexpr int kACol0 = 2 * kDBufs * SUB * BN;  // accumulators first
  static_assert(kXStages % 2 == 0 && kXStages >= 4 && kXStages >= 2 * kDBufs, "ring of rows");
  static_assert(kACol0 + 4 * kASlotCols <= 512, "tensor memory");
  // a dequant warpgroup may meet a stage of weights that the other one had last: that chunk, c - W, is then long done (a
  // warpgroup at c has seen c - 4 done, whose MMAs waited for the sums of c - 8 at the latest, read in order)
  static_assert(kWStages >= 9, "ring of weights");
};

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
  return d;
}
__device__ __forceinline__ void unpack2(uint64_t v, float *lo, float *hi) {
  uint32_t a, b;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(v));
  *lo = __uint_as_float(a);
  *hi = __uint_as_float(b);
}

__device__ __forceinline__ void sts_f32(uint32_t addr, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

template <bool ON, int R>
__device__ __forceinline__ void regs_down() {
  if constexpr (ON) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}
template <bool ON, int R>
__device__ __forceinline__ void regs_up() {
  if constexpr (ON) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}

// The limit of the waits, in shared memory: as a value it took registers from the roles (333 rows of 60 experts, 257 us: 261).
struct SharedLimit {
  const volatile uint64_t *at;
  __device__ __forceinline__ operator uint64_t() const { return *at; }
};

// After a wait that gave up, the barriers say no more when the copies in flight have landed, which takes some
// microseconds: ten milliseconds pass before the CTA leaves its shared memory.
__device__ __forceinline__ void let_copies_land() {
  const uint64_t t0 = clock_cycles();
  while (clock_cycles() - t0 < 20ull * 1000 * 1000) __nanosleep(1000);
}

// The units of a CTA in order, the next one's tile read ahead.
struct UnitWalk {
  const Products &p;
  int u, units, step;
  RowTile next;
  __device__ __forceinline__ UnitWalk(const Products &p_, int units_) : p(p_), u(blockIdx.x), units(units_), step(gridDim.x) {
    if (u < units) next = p.plan.tiles[u / p.slabs];
  }
  __device__ __forceinline__ bool take(RowTile *tile, int *wt) {
    if (u >= units) return false;
    *tile = next;
    *wt = u % p.slabs;
    u += step;
    if (u < units) next = p.plan.tiles[u / p.slabs];
    return true;
  }
  // the index of the tile that was taken last
  __device__ __forceinline__ int taken() const { return (u - step) / p.slabs; }
};

// A place in the ring of S stages: chunk c's, with the parity of its phase.
template <int S>
struct Ring {
  uint32_t s = 0, phase = 0;
  __device__ __forceinline__ void step() {
    if (++s == S) {
      s = 0;
      phase ^= 1;
    }
  }
};

template <int DT, int BN, int CB, int SUB, bool GATED>
__global__ void __launch_bounds__(TCfg<BN, CB, SUB>::kThreads, 1)
    experts_tmem_kernel(const __grid_constant__ CUtensorMap in_map, const __grid_constant__ Products p) {
  using C = TCfg<BN, CB, SUB>;
  constexpr int S = C::kXStages, W = C::kWStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t go_bar[S], done_bar[S], wfull_bar[W], wfree_bar[W], free_bar[2][2], drain_bar[2];
  __shared__ float scales[C::kScaleSlots][SUB][kTN];
  __shared__ uint32_t tmem_sh, abort_sh;
  __shared__ uint64_t limit_sh;

  const uint32_t smem_base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  volatile uint32_t *abort_flag = &abort_sh;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      // the row warp, the chunk's dequant warps, and the sum warps of the accumulator's chunk before
      mbar_init(smem_u32(&go_bar[s]), 1 + 4 + 4 * C::kSumGroups + (s == 0 ? p.test_extra : 0));
      mbar_init(smem_u32(&done_bar[s]), 1);
    }
    for (int s = 0; s < W; ++s) {
      mbar_init(smem_u32(&wfull_bar[s]), 2);  // the weight warps
      mbar_init(smem_u32(&wfree_bar[s]), 4);
    }
    for (int e = 0; e < 2; ++e) {
      for (int a = 0; a < 2; ++a) mbar_init(smem_u32(&free_bar[e][a]), 1);
      mbar_init(smem_u32(&drain_bar[e]), 1);
    }
    abort_sh = 0;
    limit_sh = p.wait_limit;
    fence_mbar_init();
  }
  if (warp == 0 && elect_one()) prefetch_tensormap(&in_map);
  if (warp == 8) {
    tmem_alloc(smem_u32(&tmem_sh), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncwarp();
  cta_sync_all();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_sh, 0);
  if (threadIdx.x == 0) griddep_launch_dependents();
  griddep_wait();  // the plan and `in` come from the grids before this one
  const int units = *p.plan.ntiles * p.slabs;  // (the host has checked that this fits)
  const int chunks = (p.KB + CB - 1) / CB;  // of a unit
  const SharedLimit limit{&limit_sh};
  const uint32_t go0 = smem_u32(&go_bar[0]), done0 = smem_u32(&done_bar[0]);
  const uint32_t wfull0 = smem_u32(&wfull_bar[0]), wfree0 = smem_u32(&wfree_bar[0]);
  const uint32_t w_base = smem_base + S * C::kXBytes;
  const uint32_t free0 = smem_u32(&free_bar[0][0]);

  if (warp < 4) {
    // ----------------------------------------------------------------- rows
    regs_down<C::kDeal, C::kRegsRows>();
    Ring<S> at;
    uint32_t c = 0;
    bool ok = true;
    RowTile rt;
    int wt;
    for (UnitWalk w(p, units); warp == 0 && ok && w.take(&rt, &wt);) {
      for (int q = 0; q < chunks; ++q, ++c, at.step()) {
        if (c >= static_cast<uint32_t>(S)) ok = warp_wait(done0 + 8 * at.s, at.phase ^ 1, abort_flag, p.err, limit);
        if (!ok) break;
        if (elect_one()) {
          const uint32_t bar = go0 + 8 * at.s;
          const int nb = min(CB, p.KB - q * CB);
          mbar_arrive_expect_tx(bar, nb * C::kXSub);
#pragma unroll
          for (int b = 0; b < CB; ++b)
            if (b < nb) tma_load_2d(smem_base + at.s * C::kXBytes + b * C::kXSub, &in_map, (q * CB + b) * kTK, rt.row0, bar);
        }
        __syncwarp();
      }
    }
  } else if (warp < 8) {
    regs_down<C::kDeal, C::kRegsIssue>();
    if (warp < 6) {
      // ---------------------------------------------------------- MMA issue
      const int e = warp - 4;
      Ring<S> at;  // S is even: a stage's chunks are all of one warp, which so waits for each of its phases
      if (e) at.step();
      uint32_t n = 0;  // this warp's chunks so far
      int skip = e;    // chunks of the unit before its first
      bool ok = true;
      RowTile rt;
      int wt;
      for (UnitWalk w(p, units); ok && w.take(&rt, &wt);) {
        const uint32_t idesc = idesc_f16_f32(128, (rt.rows + 15) / 16 * 16, DT == kDtypeBf16);
        int q = skip;
        for (; q < chunks; q += 2, ++n) {
          const uint32_t slot = 2 * e + (n & 1);
          const uint32_t d = C::kDBufs * e + n % C::kDBufs;
          ok = warp_wait(go0 + 8 * at.s, at.phase, abort_flag, p.err, limit);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const int nb = min(CB, p.KB - q * CB);
            const uint32_t xs = smem_base + at.s * C::kXBytes;
            const uint32_t a = tmem + C::kACol0 + slot * C::kASlotCols;
#pragma unroll
            for (int b = 0; b < CB; ++b) {
              if (b >= nb) break;
              const uint64_t bdesc = sw128_kmajor_desc(xs + b * C::kXSub);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {
                const int half = (b * kTK + kk * 16) / C::kSubK;
                const bool fresh = (b * kTK + kk * 16) % C::kSubK == 0;
                mma_f16_ts(tmem + (d * SUB + half) * BN, a + b * 32 + kk * 8, bdesc + static_cast<uint64_t>(kk * 2), idesc,
                           fresh ? 0u : 1u);
              }
            }
            mma_commit(free0 + 8 * slot);
            mma_commit(done0 + 8 * at.s);
          }
          __syncwarp();
          at.step();
          at.step();
        }
        skip = q - chunks;
      }
      const bool aborted = __any_sync(0xffffffffu, *abort_flag != 0);
      if (aborted && elect_one()) {
        mma_commit(smem_u32(&drain_bar[e]));
        drain_wait(smem_u32(&drain_bar[e]), 0);
      }
    } else {
      // ------------------------------------------------- codes and records
      const bool records = warp == 7;
      const uint64_t policy = policy_evict_normal();  // an expert's other row tiles read the weights again
      Ring<W> at;
      uint32_t c = 0;
      bool ok = true;
      RowTile rt;
      int wt;
      for (UnitWalk w(p, units); ok && w.take(&rt, &wt);) {
        const uint8_t *expert = p.codes + rt.key * p.expert_bytes;
        const uint8_t *codes = expert + static_cast<int64_t>(wt) * p.KB * kTileBytes;
        const uint8_t *meta = expert + p.meta + static_cast<int64_t>(wt) * p.G * kRecBytes;
        for (int q = 0; q < chunks; ++q, ++c, at.step()) {
          if (c >= static_cast<uint32_t>(W)) ok = warp_wait(wfree0 + 8 * at.s, at.phase ^ 1, abort_flag, p.err, limit);
          if (!ok) break;
          if (elect_one()) {
            const uint32_t to = w_base + at.s * C::kWBytes;
            const uint32_t bar = wfull0 + 8 * at.s;
            if (records) {
              const int k0 = q * CB * kTK;
              const int j0 = p.gdiv.div(k0);
              const int nrec = SUB == 1 ? 1 : p.gdiv.div(min(k0 + CB * kTK, p.K) - 1) - j0 + 1;
              mbar_arrive_expect_tx(bar, nrec * kRecBytes);
              bulk_g2s(to + C::kCodeBytes, meta + static_cast<int64_t>(j0) * kRecBytes, nrec * kRecBytes, bar, policy);
            } else {
              const int nb = min(CB, p.KB - q * CB);
              mbar_arrive_expect_tx(bar, nb * kTileBytes);
              bulk_g2s(to, codes + static_cast<int64_t>(q) * CB * kTileBytes, nb * kTileBytes, bar, policy);
            }
          }
          __syncwarp();
        }
      }
    }
  } else if (warp < 16) {
    // ------------------------------------------------------------ dequant
    const int e = (warp - 8) / 4;
    const int lq = warp % 4;
    const int r = lq * 32 + lane;
    const uint32_t lane_addr = static_cast<uint32_t>(lq * 32) << 16;
    const int mine = static_cast<int>(blockIdx.x) < units ? (units - static_cast<int>(blockIdx.x) + static_cast<int>(gridDim.x) - 1) /
                                                               static_cast<int>(gridDim.x)
                                                         : 0;  // units of the CTA
    // the warpgroup's chunks: chunk q of unit i, n of them so far
    int i = 0, q = e;
    uint32_t x_at = e;  // its place in the ring of rows
    Ring<W> at;
    if (e) at.step();
    const uint32_t scale0 = smem_u32(&scales[0][0][0]) + 4 * r;
    for (uint32_t n = 0;; ++n) {
      while (q >= chunks) {
        q -= chunks;
        ++i;
      }
      if (i >= mine) break;
      if (!warp_wait(wfull0 + 8 * at.s, at.phase, abort_flag, p.err, limit)) break;
      const uint32_t slot = 2 * e + (n & 1);
      if (n >= 2 && !warp_wait(free0 + 8 * slot, (n / 2 - 1) & 1, abort_flag, p.err, limit)) break;
      const uint32_t codes = w_base + at.s * C::kWBytes + r * 16;
      const uint32_t rec = w_base + at.s * C::kWBytes + C::kCodeBytes;
      const int nb = min(CB, p.KB - q * CB);
      GroupConsts gc[SUB];
#pragma unroll
      for (int h = 0; h < SUB; ++h) {
        // the second half's record is the first's when both lie in one group (or the half lies past K)
        const int k0 = q * CB * kTK;
        const uint32_t off = h == 0 ? 0u : (p.gdiv.div(min(k0 + C::kSubK, p.K - 1)) - p.gdiv.div(k0)) * kRecBytes;
        const uint32_t bits = lds16(rec + off + 2 * r);
        gc[h] = group_consts<DT>(bits, (lds8(rec + off + 256 + r / 2) >> (4 * (r & 1))) & 0xFu);
        sts_f32(scale0 + (((2 * n + e) % C::kScaleSlots) * SUB + h) * kTN * 4, scale_f32<DT>(bits));
      }
      const uint32_t a = tmem + lane_addr + C::kACol0 + slot * C::kASlotCols;
      tc_fence_after();
#pragma unroll
      for (int b = 0; b < CB; ++b) {
        if (b >= nb) break;
        const uint4 w0 = lds128(codes + b * kTileBytes);
        const uint4 w1 = lds128(codes + b * kTileBytes + 2048);
        if (b == nb - 1) {  // the stage has been read
          __syncwarp();
          if (lane == 0) mbar_arrive(wfree0 + 8 * at.s);
        }
        uint32_t out[16];
        dequant_word_int<DT>(w0.x, gc[b * kTK / C::kSubK], out);
        dequant_word_int<DT>(w0.y, gc[b * kTK / C::kSubK], out + 4);
        dequant_word_int<DT>(w0.z, gc[b * kTK / C::kSubK], out + 8);
        dequant_word_int<DT>(w0.w, gc[b * kTK / C::kSubK], out + 12);
        tmem_st_32x32b_x16(a + b * 32, out);
        dequant_word_int<DT>(w1.x, gc[(b * kTK + 32) / C::kSubK], out);
        dequant_word_int<DT>(w1.y, gc[(b * kTK + 32) / C::kSubK], out + 4);
        dequant_word_int<DT>(w1.z, gc[(b * kTK + 32) / C::kSubK], out + 8);
        dequant_word_int<DT>(w1.w, gc[(b * kTK + 32) / C::kSubK], out + 12);
        tmem_st_32x32b_x16(a + b * 32 + 16, out);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(go0 + 8 * x_at);
      x_at = x_at + 2 >= S ? x_at + 2 - S : x_at + 2;
      q += 2;
      at.step();
      at.step();
    }
  } else {
    // ------------------------------------------------------------ sums
    regs_up<C::kDeal, C::kRegsSum>();
    constexpr int kCols = 32;  // of a warpgroup
    const int part = (warp - 16) / 4;
    const int lq = warp % 4;
    const int r = lq * 32 + lane;
    const uint32_t lane_addr = static_cast<uint32_t>(lq * 32) << 16;
    Ring<S> at;
    constexpr uint32_t kAhead = 2 * C::kDBufs;  // the accumulator's next chunk
    if (lane == 0)
      for (uint32_t i = 0; i < kAhead; ++i) mbar_arrive(go0 + 8 * i);  // the first chunks' accumulators are free
    uint32_t c = 0;
    bool ok = true;
    const uint32_t scale0 = smem_u32(&scales[0][0][0]) + 4 * r;
    RowTile rt;
    int wt;
    for (UnitWalk w(p, units); ok && w.take(&rt, &wt);) {
      const int cols = min(max(rt.rows - part * kCols, 0), kCols);  // this warpgroup's columns with a row
      uint64_t acc[kCols / 2];
#pragma unroll
      for (int i = 0; i < kCols / 2; ++i) acc[i] = 0ull;
      for (int q = 0; q < chunks; ++q, ++c, at.step()) {
        ok = warp_wait(done0 + 8 * at.s, at.phase, abort_flag, p.err, limit);
        if (!ok) break;
        tc_fence_after();
        const uint32_t buf = C::kDBufs * (c & 1) + c / 2 % C::kDBufs;
        const uint32_t next = go0 + 8 * (at.s + kAhead >= S ? at.s + kAhead - S : at.s + kAhead);
#pragma unroll
        for (int h = 0; h < SUB; ++h) {
          if (h == 1 && q * CB * kTK + C::kSubK >= p.K) break;  // its products were not of this unit's K
          const uint32_t sb = lds32(scale0 + ((c % C::kScaleSlots) * SUB + h) * kTN * 4);
          const uint64_t s2 = pack2(sb, sb);
          const uint32_t d = tmem + lane_addr + (buf * SUB + h) * BN + part * kCols;
          if (cols > 0) {
            uint32_t v0[16], v1[16];
            tmem_ld_32x32b_x16(d, v0);
            tmem_ld_32x32b_x16(d + 16, v1);
            tmem_wait_ld();
            if (h == SUB - 1 || q * CB * kTK + C::kSubK >= p.K) {  // the last read of the chunk's sums
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(next);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = fma2(s2, pack2(v0[2 * i], v0[2 * i + 1]), acc[i]);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[8 + i] = fma2(s2, pack2(v1[2 * i], v1[2 * i + 1]), acc[8 + i]);
          }
        }
        if (cols == 0) {
          __syncwarp();
          if (lane == 0) mbar_arrive(next);
        }
      }
      if (!ok) break;
      const int n = wt * kTN + r;
      const int64_t pos0 = rt.row0 + part * kCols;
      if (GATED) {
        // rows n & ~1 (even lane: gate) and n | 1 (odd lane: up): the pair swaps values, the even lane makes the
        // first half of the columns, the odd lane the second
        const int odd = lane & 1;
        const int ld = p.N / 2;
#pragma unroll
        for (int i = 0; i < kCols / 4; ++i) {
          float f[2], b[2];  // columns 2 i, 2 i + 1 of the first and the second half
          unpack2(acc[i], &f[0], &f[1]);
          unpack2(acc[i + kCols / 4], &b[0], &b[1]);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float got = __shfl_xor_sync(0xffffffffu, odd ? f[j] : b[j], 1);
            const float gate = odd ? got : f[j], up = odd ? b[j] : got;
            const int col = 2 * i + j + odd * (kCols / 2);
            if (n < p.N && col < cols) store_h<DT>(p, silu_mul(gate, up), (pos0 + col) * ld + n / 2, w.taken());
          }
        }
      } else if (n < p.N) {
        float *out = static_cast<float *>(p.out) + n;
#pragma unroll
        for (int i = 0; i < kCols / 2; ++i) {
          float f0, f1;
          unpack2(acc[i], &f0, &f1);
          if (2 * i < cols) out[(pos0 + 2 * i) * p.N] = f0;
          if (2 * i + 1 < cols) out[(pos0 + 2 * i + 1) * p.N] = f1;
        }
      }
      __syncwarp();
    }
  }

  tc_fence_before();
  __syncwarp();
  cta_sync_all();
  if (*abort_flag) let_copies_land();  // (else every copy has been waited for)
  if (warp == 8) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int DT, int BN, int CB, int SUB, bool GATED>
cudaError_t launch_one(const Products &p, int num_sms, cudaStream_t stream) {
  auto kern = experts_tmem_kernel<DT, BN, CB, SUB, GATED>;
  constexpr int bytes = TCfg<BN, CB, SUB>::kSmemBytes;
  static std::atomic<uint64_t> set{0};
  const cudaError_t e = allow_smem(kern, bytes, &set);
  if (e != cudaSuccess) return e;
  CUtensorMap in_map;
  if (!make_rows_map(&in_map, p.in, p.in_rows, p.K, BN, DT)) return cudaErrorInvalidValue;
  return launch_programmatic(kern, num_sms, TCfg<BN, CB, SUB>::kThreads, bytes, stream, in_map, p);
}

template <int DT, bool GATED>
cudaError_t launch_groups(const Products &p, int tile, int num_sms, cudaStream_t stream) {
  if (p.g % 128 == 0)
    return tile == 128 ? launch_one<DT, 128, 2, 1, GATED>(p, num_sms, stream) : launch_one<DT, 64, 2, 1, GATED>(p, num_sms, stream);
  if (p.g % 64 == 0)
    return tile == 128 ? launch_one<DT, 128, 1, 1, GATED>(p, num_sms, stream) : launch_one<DT, 64, 2, 2, GATED>(p, num_sms, stream);
  return launch_one<DT, 64, 1, 2, GATED>(p, num_sms, stream);
}

}  // namespace

namespace detail {

cudaError_t launch_experts_tmem(const Products &p, int dtype, bool gated, int tile, int num_sms, cudaStream_t stream) {
  if (dtype == kDtypeBf16)
    return gated ? launch_groups<kDtypeBf16, true>(p, tile, num_sms, stream) : launch_groups<kDtypeBf16, false>(p, tile, num_sms, stream);
  return gated ? launch_groups<kDtypeF16, true>(p, tile, num_sms, stream) : launch_groups<kDtypeF16, false>(p, tile, num_sms, stream);
}

}  // namespace detail
}  // namespace w4
