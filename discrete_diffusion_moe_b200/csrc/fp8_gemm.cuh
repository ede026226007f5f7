// fp8_gemm.cuh - the block-scaled e4m3 product on CTA pairs (tcgen05,
// cta_group::2), dense or with the rows split among groups of weights:
//
//   D[m, n] = w[m] * sum_kb sa[kb, m] * sb[n / 128, kb] * sum_{k in block kb} A[m, k] * B[n, k]
//
// Tokens (A) are the rows of the accumulator, weights (B) its columns: a
// thread of the epilogue owns one row, so the scale of a block is one number
// per thread and 128 columns, and scaling costs one fused multiply-add per
// accumulator element.  (With the weights as rows every column would need its
// own scale from shared memory.)
//
// A unit is 256 rows x kW columns of one group.  Per block of 128 k (one stage:
// 128 bytes of each row, the width of the 128-byte swizzle) four tcgen05.mma of
// M = 256, N = kW, K = 32 go into a fresh tensor-memory buffer; eight epilogue
// warps in each CTA take the block's sums out, multiply them by the scales and
// add them in registers, while the tensor cores work on the next block in
// another buffer.  fp32 throughout; one rounding at the store.
//
// What bounds it, in cycles per block of 256 x 256 (the parts timed alone): copies 486,
// MMAs 600, copies and MMAs together 790, since both use the shared memory, all with
// the epilogue 1030.  The last step is the chain MMA - commit - take out - release -
// MMA through two buffers of 256 columns, which fill the tensor memory.  8192 x 5632 x
// 2816 into bf16: 138 us with 1.9 PFLOP/s; under a steady load of such products the
// 1000 W limit takes the clock to 1.64 GHz (158 us).  With kW = 128 rows are read twice as
// often, but there are four buffers and finer units, for small or ragged work.
//
// Each CTA of a pair copies its own 128 rows of A and half of the columns of B
// (32 KB a stage at 256 columns), so a pair reads 512 rows per block.  Copies of
// few rows use a smaller box (16 or 64 rows): the rest of the tile holds old
// bytes, and only rows that are not stored depend on them.
//
// The results are turned through shared memory so that a warp stores whole
// 128-byte lines (a thread holds one row; storing from registers touched 32
// lines per instruction and took a sixth of a unit's time).
//
// Protocol of the barriers (rank 0 leads):
//   full[s]       rank 0's: both CTAs' copies of a stage have landed
//   acc_full[s]   both: the sums of the stage's block are in tensor memory and the
//                 stage is free
//   acc_empty[b]  rank 0's: the epilogue warps of both CTAs have read the buffer
//   sc_full, sc_empty[i]  each CTA's own: a slot of scales is written, is read
// All waits are bounded.  A role whose wait runs out stops: it copies, multiplies,
// commits and releases nothing more, so that no barrier gets an arrival that its phase
// does not expect and no other role takes old bytes for new ones; those that depend on it
// run out in turn, in the other CTA too.  A CTA in which a wait ran out stores NaN from
// then on, so whatever is stored as a number is the product.
#pragma once

#include "fp8_small.cuh"
#include <type_traits>

#include "gemm_pair.cuh"

namespace dg {

constexpr int kFp8MaxGroups = 1024;
constexpr int kFp8EpiWarps = 8;
// Warpgroup 0: a copying warp, two MMA warps, a scale warp; warpgroups 1 and 2:
// the epilogue.  384 threads x 168 registers at launch; warpgroup 0 gives back what
// the epilogue takes.  Spills count: with nearly all of the SM's memory used as
// shared memory a spilled register comes back from L2, and several of them in the
// loop over blocks doubled the kernel's time.  (ptxas reports 16 bytes of stack at
// kW = 256, 48 to 56 of spill stores and 108 of loads; none at 128.)
constexpr int kFp8Threads = 128 + 32 * kFp8EpiWarps;
constexpr int kFp8RegsCopy = 72, kFp8RegsEpi = 216;
static_assert(128 * kFp8RegsCopy + 32 * kFp8EpiWarps * kFp8RegsEpi <= kFp8Threads * 168, "register split");

// The waits of a product: how long each may take, the error word of a context (or
// null) that gets kDevErrTimeout when one runs out, and for failure tests what a unit
// leaves out of block `block`.
enum { kHoldNothing = 0, kHoldCopies = 1, kHoldScales = 2 };
struct Fp8Waits {
  unsigned long long limit_ns;
  int* err;
  int hold, unit, block;
};

// One lane of a converged warp.  The copies and MMAs take their descriptors from
// uniform registers; issued from a branch on the lane number the compiler moves
// them there one instruction at a time.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "selp.b32 %0, 1, 0, q;\n\t}"
      : "=r"(p));
  return p != 0;
}
// instruction descriptor of tcgen05.mma kind::f8f6f4: D fp32, A and B e4m3, both K-major
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void umma_e4m3_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ int ld_shared_flag(uint32_t addr) {
  int v;
  asm volatile("ld.volatile.shared.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_shared_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
// Whether no wait of this CTA has run out so far; the same answer for the whole warp.
__device__ __forceinline__ bool alive(uint32_t dead) { return __all_sync(0xffffffffu, !ld_shared_flag(dead)); }
// Bounded wait of one thread; false when it ran out, or another one of the CTA did
// meanwhile (the flag at shared address `dead`).
__device__ __forceinline__ bool thread_wait(uint32_t bar, uint32_t parity, uint32_t dead, const Fp8Waits& wt) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = globaltimer_ns();
  uint32_t n = 0;
#pragma unroll 1
  while (!mbar_try_wait(bar, parity)) {
    if ((++n & 255u) == 0u) {
      if (ld_shared_flag(dead)) return false;
      if (globaltimer_ns() - t0 > wt.limit_ns) {
        asm volatile("st.volatile.shared.s32 [%0], 1;" ::"r"(dead) : "memory");
        set_error(wt.err, kDevErrTimeout);
        return false;
      }
    }
  }
  return true;
}
// The same of a whole warp: after false the warp's role has to stop.
__device__ __forceinline__ bool wait_or_die(uint32_t bar, uint32_t parity, uint32_t dead, const Fp8Waits& wt) {
  return __all_sync(0xffffffffu, thread_wait(bar, parity, dead, wt));
}
// The epilogue's: it goes on, but the lane that releases buffers (`releases`) does so no
// more once its own wait ran out, and the results are marked at their store.  After a
// wait of its own that ended well the phase is complete, even if another lane has
// just given up on it.  (Leaving the loop over blocks on the warp's vote cost 5 % of
// the time of 256-column units, with more spills.)
__device__ __forceinline__ void wait_or_keep(uint32_t bar, uint32_t parity, uint32_t dead, const Fp8Waits& wt, bool& releases) {
  if (!thread_wait(bar, parity, dead, wt)) releases = false;
  __syncwarp();
}
// The same for what has to end before the CTA may leave (copies into its memory,
// MMAs that read it): a failed wait elsewhere does not cut it short.
__device__ __forceinline__ void wait_to_leave(uint32_t bar, uint32_t parity, uint32_t dead, const Fp8Waits& wt) {
  if (!mbar_wait(bar, parity, wt.err, wt.limit_ns)) asm volatile("st.volatile.shared.s32 [%0], 1;" ::"r"(dead) : "memory");
  __syncwarp();
}
// 32 lanes x 32 consecutive fp32 columns of tensor memory; the registers are
// undefined until tmem_wait32 on them
__device__ __forceinline__ void tmem_ld32_nowait(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
                 "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]),
                 "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                 "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]),
                 "+r"(r[31])
               :
               : "memory");
}
// Arrive on a pair peer's (or this CTA's) mbarrier at the default scope.  What it
// orders are tensor-memory reads, by the tcgen05 fence before it; a release at
// cluster scope would add a memory barrier to every block of every warp (8192 x
// 5632 x 2816 took 350 us with it and 205 without).
__device__ __forceinline__ void mbar_arrive_peer(uint32_t bar_cluster) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster) : "memory");
}
// tensor maps: A with boxes of 16, 64 and 128 rows, B with boxes of kW / 4 and kW / 2 rows
// and the output with boxes of 128 bytes x 32 rows (when its rows are 16-byte aligned)
struct Fp8Maps {
  CUtensorMap a[3];
  CUtensorMap b[2];
  CUtensorMap out;
};

struct Fp8Tables {
  int* first;  // [groups + 1] row tiles of the groups before g
  int* row0;   // [groups]
  int* row1;
  __device__ Fp8Tables(int* at, int groups) : first(at), row0(at + groups + 1), row1(at + 2 * groups + 1) {}
};

// The groups' rows and their prefix sums of tiles of kRows rows (one warp).
template <int kRows>
__device__ __forceinline__ void fp8_tables(const Fp8GemmParams& p, const Fp8Tables& tb, int lane) {
  int sum = 0;
  for (int base = 0; base < p.G; base += 32) {
    const int g = base + lane;
    RowRange r{0, 0};
    if (g < p.G) r = group_rows(p.off, g, p.M);
    const int t = (r.row1 - r.row0 + kRows - 1) / kRows;
    int inc = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (g < p.G) {
      tb.first[g] = sum + inc - t;
      tb.row0[g] = r.row0;
      tb.row1[g] = r.row1;
    }
    sum += __shfl_sync(0xffffffffu, inc, 31);
  }
  if (lane == 0) tb.first[p.G] = sum;
}

struct Fp8Job {
  int group, row0, row1, n0;  // the unit's rows [row0, row1) of at most kRows, first column of B
};

// Unit u of tiles of kRows rows x bn columns: n_tiles column tiles, m_tiles row
// tiles (all groups together); a group's row tiles of one column tile are
// consecutive units, which share their columns of B.
template <int kRows>
__device__ __forceinline__ Fp8Job fp8_job(const Fp8GemmParams& p, const Fp8Tables& tb, int u, int m_tiles, int n_tiles,
                                          int bn) {
  Fp8Job j;
  if (!p.off) {
    const int nt = u / m_tiles, mt = u - nt * m_tiles;
    j.group = 0;
    j.row0 = mt * kRows;
    j.row1 = min(p.M, j.row0 + kRows);
    j.n0 = nt * bn;
    return j;
  }
  int lo = 0, hi = p.G;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tb.first[mid] * n_tiles <= u) lo = mid;
    else hi = mid;
  }
  const int tiles = tb.first[lo + 1] - tb.first[lo];
  const int r = u - tb.first[lo] * n_tiles;
  const int nt = r / tiles, mt = r - nt * tiles;
  j.group = lo;
  j.row0 = tb.row0[lo] + mt * kRows;
  j.row1 = min(tb.row1[lo], j.row0 + kRows);
  j.n0 = nt * bn;
  return j;
}

template <int kW>
struct Fp8Shape {
  static constexpr int kBufs = kW >= 256 ? 2 : 4;  // tensor-memory buffers of kW columns
  // Even, so that an MMA warp, which takes every second block, comes back to the same
  // stages and has itself seen each phase of their barriers.  A wait tells only a
  // phase from the one before it: with an odd number a warp could pass on the
  // phase two back while the other warp's copy into the stage was still under way.
  static constexpr int kStages = kW >= 256 ? 4 : 6;
  static_assert(kStages % 2 == 0 && kBufs % 2 == 0, "two MMA warps in turn");
  static constexpr int kStageA = 128 * 128, kStageB = (kW / 2) * 128;
  static constexpr int kTurn = kFp8EpiWarps * 8192;  // two buffers of 32 rows x 128 bytes per warp
  static constexpr int kCols = kW / 2;               // columns of an epilogue warp
  // row and weight scales of four blocks per slot: [128][4], and [4] for either half of the columns
  static constexpr int kScaleSlots = kW >= 256 ? 4 : 2, kScaleSlot = 4 * 128 + 4 * 2;
  static constexpr int kBars = 2 * kStages + kBufs + 2 * kScaleSlots + 1;
  static constexpr int kSmem = 1024 + kStages * (kStageA + kStageB) + kTurn + kScaleSlots * kScaleSlot * 4 + kBars * 8 + 16;
  static_assert(kSmem + 13 * 1024 <= 227 * 1024, "shared memory, with the tables of the groups");
};

__device__ __forceinline__ void cp_async4(uint32_t dst, const float* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// one arrival on `bar` when this thread's copies so far have landed
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, uint32_t src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(map), "r"(src), "r"(x),
               "r"(y)
               : "memory");
}
template <int kPending>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kPending) : "memory");
}

// Stores a warp's 32 rows x kCols results (thread `lane` holds row lane in acc),
// 128 bytes of each row at a time, through its two 4 KB buffers of shared memory
// with the 128-byte swizzle (16-byte units by row): free of bank conflicts on
// both sides.  With a tensor map the copy engine does the global side while the
// warp goes on (columns from the matrix's end on are clipped); else the warp
// stores whole rows itself: rows [0, rows), columns [0, cols).  `next`: the buffer
// to use, the other one than the last pass's (of this unit or the one before).
template <class TO, int kCols>
__device__ __forceinline__ void store_turned(uint8_t* turn, const CUtensorMap* map, int x, int y, TO* out, long long ldo,
                                             const float* acc, float w, int lane, int rows, int cols, bool vec, uint32_t& next) {
  constexpr int kPer = 128 / (int)sizeof(TO);  // columns per pass
  constexpr int kPass = kCols < kPer ? kCols : kPer;
  constexpr int kUnit = 16 / (int)sizeof(TO);  // columns per 16-byte unit
#pragma unroll
  for (int c0 = 0; c0 < kCols; c0 += kPass) {
    if (c0 >= cols) break;
    uint8_t* const buf = turn + next;
    next ^= 4096u;
    if (lane == 0) bulk_wait_read<1>();  // what this buffer held has been read
    __syncwarp();
#pragma unroll
    for (int u = 0; u < kPass / kUnit; ++u) {
      uint32_t v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(TO) == 4) {
          v[i] = __float_as_uint(acc[c0 + u * kUnit + i] * w);
        } else {
          const float lo = acc[c0 + u * kUnit + 2 * i] * w, hi = acc[c0 + u * kUnit + 2 * i + 1] * w;
          if constexpr (std::is_same_v<TO, __half>) v[i] = pack_f16x2(lo, hi);
          else v[i] = pack_bf16x2(lo, hi);
        }
      }
      *reinterpret_cast<uint4*>(buf + lane * 128 + ((u ^ (lane & 7)) * 16)) = make_uint4(v[0], v[1], v[2], v[3]);
    }
    // the copy engine clips rows of whole 16-byte units only: where the matrix ends
    // inside one it wrote zeros up to the unit's end
    if (map && (c0 + kPass <= cols || cols % kUnit == 0)) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tma_store_2d(map, smem_u32(buf), x + c0, y);
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      }
    } else {
      __syncwarp();
      const int n = min(kPass, cols - c0);
      constexpr int kUnits = kPass / kUnit;
      if (vec && n == kPass) {
        const int u = lane % kUnits;
        for (int r = lane / kUnits; r < rows; r += 32 / kUnits)
          *reinterpret_cast<uint4*>(out + r * ldo + c0 + u * kUnit) =
              *reinterpret_cast<const uint4*>(buf + r * 128 + ((u ^ (r & 7)) * 16));
      } else {
        // unaligned or cut rows: element by element, eight rows in flight
        constexpr int kEach = (kPass + 31) / 32;
        for (int r0 = 0; r0 < rows; r0 += 8) {
          TO v[8][kEach];
#pragma unroll
          for (int k = 0; k < 8; ++k)
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
              const int r = r0 + k, c = (lane + 32 * e) % kPass;
              v[k][e] = *reinterpret_cast<const TO*>(buf + r * 128 + (((c / kUnit) ^ (r & 7)) * 16) + (c % kUnit) * sizeof(TO));
            }
#pragma unroll
          for (int k = 0; k < 8; ++k)
#pragma unroll
            for (int e = 0; e < kEach; ++e)
              if (r0 + k < rows && lane + 32 * e < n) out[(r0 + k) * ldo + c0 + lane + 32 * e] = v[k][e];
        }
      }
      if (lane == 0) asm volatile("cp.async.bulk.commit_group;" ::: "memory");  // keeps the count of passes
      __syncwarp();
    }
  }
}

template <int kW, class TO>
__global__ void __launch_bounds__(kFp8Threads, 1)
    fp8_pair_kernel(const __grid_constant__ Fp8Maps maps, const __grid_constant__ Fp8GemmParams p, const Fp8Waits wt) {
  using S = Fp8Shape<kW>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ int s_tabs[3 * kFp8MaxGroups + 1];
  const Fp8Tables tabs(s_tabs, kFp8MaxGroups);
  __shared__ int s_dead;
  uint8_t* const smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* const sA = smem;
  uint8_t* const sB = sA + S::kStages * S::kStageA;
  uint8_t* const s_turn = sB + S::kStages * S::kStageB;
  float* const s_scale = (float*)(s_turn + S::kTurn);
  uint64_t* const bars = (uint64_t*)(s_scale + S::kScaleSlots * S::kScaleSlot);
  uint32_t* const tmem_slot = (uint32_t*)(bars + S::kBars);
  const uint32_t full = smem_u32(bars);
  const uint32_t acc_full = full + 8 * S::kStages;
  const uint32_t acc_empty = acc_full + 8 * S::kStages;
  const uint32_t sc_full = acc_empty + 8 * S::kBufs;          // [kScaleSlots]
  const uint32_t sc_empty = sc_full + 8 * S::kScaleSlots;
  const uint32_t drain = sc_empty + 8 * S::kScaleSlots;
  const uint32_t dead = smem_u32(&s_dead);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = (int)(blockIdx.x >> 1), pairs = (int)(gridDim.x >> 1);
  const int n_tiles = (p.N + kW - 1) / kW;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(full + 8 * s, 1);
      mbar_init(acc_full + 8 * s, 1);
    }
    for (int b = 0; b < S::kBufs; ++b) mbar_init(acc_empty + 8 * b, 2 * kFp8EpiWarps);
    for (int i = 0; i < S::kScaleSlots; ++i) {
      mbar_init(sc_full + 8 * i, 32);
      mbar_init(sc_empty + 8 * i, kFp8EpiWarps);
    }
    mbar_init(drain, 2);
    s_dead = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
    for (int i = 0; i < 3; ++i) tma_prefetch_desc(&maps.a[i]);
    for (int i = 0; i < 2; ++i) tma_prefetch_desc(&maps.b[i]);
  }
  grid_dep_wait();
  int m_tiles = (p.M + 255) / 256;
  if (p.off && warp == 4) fp8_tables<256>(p, tabs, lane);
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers initialised before either signals one
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), S::kBufs * kW);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dep_launch();  // not before the tensor memory is held: the next kernel's CTAs may want it too
  const uint32_t tmem_base = *tmem_slot;
  if (p.off) m_tiles = tabs.first[p.G];
  const int U = m_tiles * n_tiles;
  auto mma_cols = [&](const Fp8Job& j) { return min(kW, (p.N - j.n0 + 31) & ~31); };  // a multiple of 32

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFp8RegsCopy));
    if (warp == 0) {
      // ---------------- copies (both CTAs) ----------------
      uint32_t issued = 0, s = 0, phase = 1;
      const uint64_t pol_a = l2_policy_evict_last(), pol_b = l2_policy_evict_first();
      const uint32_t lead_bar = mapa_shared(full, 0);
      const uint32_t dstA = smem_u32(sA), dstB = smem_u32(sB);
      auto a_box = [&](int rows) { return rows <= 0 ? -1 : (rows <= 16 ? 0 : (rows <= 64 ? 1 : 2)); };
      auto a_bytes = [&](int box) { return box < 0 ? 0u : (box == 0 ? 16u : (box == 1 ? 64u : 128u)) * 128u; };
      bool ok = true;
      for (int u = pair; u < U && ok; u += pairs) {
        const Fp8Job j = fp8_job<256>(p, tabs, u, m_tiles, n_tiles, kW);
        const int held = wt.hold == kHoldCopies && u == wt.unit && rank == 1 ? wt.block : -1;
        const int mine = a_box(j.row1 - (j.row0 + (int)rank * 128));
        uint32_t tx = a_bytes(a_box(j.row1 - j.row0)) + a_bytes(a_box(j.row1 - j.row0 - 128));
        const int n = mma_cols(j);
        const int box = n <= kW / 2 ? 0 : 1;  // kW / 4 or kW / 2 rows from each CTA
        const int yB = j.group * p.N + j.n0 + (int)rank * (n >> 1);
        tx += 2u * (uint32_t)(kW / (box ? 2 : 4)) * 128u;
        const int yA = j.row0 + (int)rank * 128;
#pragma unroll 1
        for (int kb = 0; kb < p.KB; ++kb) {
          if (!(ok = wait_or_die(acc_full + s * 8u, phase, dead, wt))) break;
          if (kb != held && elect_one()) {
            if (rank == 0) mbar_arrive_expect_tx(full + s * 8u, tx);
            if (mine >= 0) tma_load_2d_pair(dstA + s * S::kStageA, &maps.a[mine], lead_bar + s * 8u, kb * 128, yA, pol_a);
            tma_load_2d_pair(dstB + s * S::kStageB, &maps.b[box], lead_bar + s * 8u, kb * 128, yB, pol_b);
          }
          __syncwarp();
          ++issued;
          if (++s == S::kStages) {
            s = 0;
            phase ^= 1;
          }
        }
      }
      // the leader's full barriers count both CTAs' bytes: wait until all have landed
      if (rank == 0) {
        const uint32_t first = issued > (uint32_t)S::kStages ? issued - S::kStages : 0;
        for (uint32_t q = first; q < issued; ++q)
          wait_to_leave(full + (q % S::kStages) * 8u, (q / S::kStages) & 1, dead, wt);
      }
    } else if (warp == 1 || warp == 3) {
      if (rank == 0) {
        // ---------------- MMAs (leader) ----------------
        // Two warps take the blocks in turn: issuing a block's MMAs takes about as long
        // as they run, so one warp would leave the tensor cores idle while it waits
        // for the next block's barriers.
        const uint32_t m = warp >> 1;
        uint32_t s = m, phase = 0, b = m, b_phase = 1;
        int kb = (int)m;  // block of this warp within the unit
        const uint64_t descA = sdesc_k128(smem_u32(sA)), descB = sdesc_k128(smem_u32(sB));
        bool ok = true;  // of this lane's waits: the issuing lane stops at its own
        for (int u = pair; u < U && alive(dead); u += pairs) {
          const Fp8Job j = fp8_job<256>(p, tabs, u, m_tiles, n_tiles, kW);
          const uint32_t idesc = idesc_e4m3_f32(256, mma_cols(j));
#pragma unroll 1
          for (; kb < p.KB; kb += 2) {
            ok = ok && thread_wait(full + s * 8u, phase, dead, wt);
            ok = ok && thread_wait(acc_empty + b * 8u, b_phase, dead, wt);
            __syncwarp();
            tc_fence_after();
            if (elect_one() && ok) {
              const uint64_t da = descA + s * (S::kStageA / 16), db = descB + s * (S::kStageB / 16);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)  // 32 bytes on: 2 in the descriptor's 16-byte units
                umma_e4m3_pair(tmem_base + b * kW, da + 2 * kk, db + 2 * kk, idesc, kk > 0 ? 1u : 0u);
              umma_commit_pair_mc(acc_full + s * 8u, (uint16_t)3);
            }
            __syncwarp();
            b = (b + 2) % S::kBufs;
            if (b == m) b_phase ^= 1;
            s += 2;
            if (s >= S::kStages) {
              s -= S::kStages;
              phase ^= 1;
            }
          }
          kb -= p.KB;
        }
        if (elect_one()) umma_commit_pair(drain);
        wait_to_leave(drain, 0, dead, wt);
        // and the other CTA's last arrivals have come: none is on its way to a CTA that left
#pragma unroll
        for (int i = 0; i < S::kBufs / 2; ++i) {
          if (alive(dead)) wait_or_die(acc_empty + b * 8u, b_phase, dead, wt);
          b = (b + 2) % S::kBufs;
          if (b == m) b_phase ^= 1;
        }
      }
    } else if (warp == 2) {
      // ---------------- scales (both CTAs) ----------------
      // Asynchronous copies of four blocks' scales per slot, up to four slots ahead: a
      // load queues behind the copies of every stage, and waiting for one slot before
      // asking for the next set the pace of the whole kernel.
      uint32_t slot = 0, phase = 1;
      bool ok = true;
      for (int u = pair; u < U && ok; u += pairs) {
        const Fp8Job j = fp8_job<256>(p, tabs, u, m_tiles, n_tiles, kW);
        const int held = wt.hold == kHoldScales && u == wt.unit && rank == 0 ? wt.block & ~3 : -1;
        const float* src[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) src[i] = p.sa + min(j.row0 + (int)rank * 128 + 32 * i + lane, j.row1 - 1);
        const int blk = min((j.n0 + ((lane >> 2) & 1) * S::kCols) / kFp8Block, p.NB - 1);
        const float* const sb = p.sb + ((long long)j.group * p.NB + blk) * p.KB;
#pragma unroll 1
        for (int kb0 = 0; kb0 < p.KB; kb0 += 4) {
          if (!(ok = wait_or_die(sc_empty + slot * 8u, phase, dead, wt))) break;
          const uint32_t dst = smem_u32(s_scale + slot * S::kScaleSlot);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const long long at = (long long)min(kb0 + q, p.KB - 1) * p.lds;
#pragma unroll
            for (int i = 0; i < 4; ++i) cp_async4(dst + (uint32_t)((32 * i + lane) * 4 + q) * 4u, src[i] + at);
          }
          if (lane < 8) cp_async4(dst + (uint32_t)(4 * 128 + lane) * 4u, sb + min(kb0 + (lane & 3), p.KB - 1));
          if (kb0 != held) cp_async_arrive(sc_full + slot * 8u);
          if (++slot == S::kScaleSlots) {
            slot = 0;
            phase ^= 1;
          }
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  } else {
    // ---------------- epilogue (both CTAs; warps 4..11) ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kFp8RegsEpi));
    const int ew = warp - 4, quarter = warp & 3;  // tensor-memory lanes [32 quarter, +32)
    const int half = ew >> 2;                     // columns [half kCols, +kCols)
    const uint32_t lane_base = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(half * S::kCols);
    const uint32_t release_to = mapa_shared(acc_empty, 0);
    const float4* const my_sa = reinterpret_cast<const float4*>(s_scale) + quarter * 32 + lane;
    const float4* const my_sb = reinterpret_cast<const float4*>(s_scale) + 128 + half;
    uint32_t s = 0, s_phase = 0, b = 0, slot = 0, slot_phase = 0, turn_next = 0;
    bool releases = lane == 0;
    for (int u = pair; u < U; u += pairs) {
      const Fp8Job j = fp8_job<256>(p, tabs, u, m_tiles, n_tiles, kW);
      const int row_w0 = j.row0 + (int)rank * 128 + quarter * 32;
      const int col = j.n0 + half * S::kCols;
      const bool work = row_w0 < j.row1 && col < p.N;
      float acc[S::kCols];
#pragma unroll
      for (int i = 0; i < S::kCols; ++i) acc[i] = 0.f;
      float4 sc4;  // the scales of four blocks
      auto read_scales = [&]() {
        wait_or_keep(sc_full + slot * 8u, slot_phase, dead, wt, releases);
        const float4 a4 = my_sa[slot * (S::kScaleSlot / 4)], b4 = my_sb[slot * (S::kScaleSlot / 4)];
        sc4 = make_float4(a4.x * b4.x, a4.y * b4.y, a4.z * b4.z, a4.w * b4.w);
        __syncwarp();
        if (releases) mbar_arrive(sc_empty + slot * 8u);
        if (++slot == S::kScaleSlots) {
          slot = 0;
          slot_phase ^= 1;
        }
      };
      auto blocks = [&](auto works) {
#pragma unroll 1
        for (int kb = 0; kb < p.KB; ++kb) {
          const int q = kb & 3;
          const float sc = q < 2 ? (q == 0 ? sc4.x : sc4.y) : (q == 2 ? sc4.z : sc4.w);
          wait_or_keep(acc_full + s * 8u, s_phase, dead, wt, releases);
          tc_fence_after();
          // Two loads at a time, and the buffer is released before the last sums are
          // added: what lies between the barrier and the release is on the path
          // MMA - commit - epilogue - release - MMA that bounds the kernel.
          if constexpr (decltype(works)::value) {
            const uint32_t t0 = lane_base + b * kW;
            constexpr int kLd = S::kCols / 32, kTwo = kLd < 2 ? kLd : 2;
            uint32_t r[kTwo][32];
#pragma unroll
            for (int c0 = 0; c0 < kLd; c0 += kTwo) {
#pragma unroll
              for (int c = 0; c < kTwo; ++c) tmem_ld32_nowait(t0 + (c0 + c) * 32, r[c]);
#pragma unroll
              for (int c = 0; c < kTwo; ++c) tmem_wait32(r[c]);
              if (c0 + kTwo == kLd) {
                tc_fence_before();
                if (releases) mbar_arrive_peer(release_to + b * 8u);
              }
#pragma unroll
              for (int c = 0; c < kTwo; ++c)
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  acc[(c0 + c) * 32 + i] = fmaf(__uint_as_float(r[c][i]), sc, acc[(c0 + c) * 32 + i]);
            }
          } else {
            tc_fence_before();
            if (releases) mbar_arrive_peer(release_to + b * 8u);
          }
          b = (b + 1) % S::kBufs;
          if (++s == S::kStages) {
            s = 0;
            s_phase ^= 1;
          }
          if (q == 3 && kb + 1 < p.KB) read_scales();
        }
      };
      // two loops: a condition inside the loop cost a register move per loaded value
      if (alive(dead)) {
        read_scales();
        if (work) blocks(std::true_type{});
        else      blocks(std::false_type{});
      }
      const int row = row_w0 + lane;
      // a wait that ran out: what was added is not the product
      const float w = !alive(dead) ? __uint_as_float(0x7fffffffu) : (p.row_w && row < j.row1 ? __ldg(p.row_w + row) : 1.0f);
      // the copy engine clips at the matrix's edges only, not at a group's last row
      const int rows = min(32, j.row1 - row_w0);
      const bool whole = S::kCols * sizeof(TO) >= 128 && p.vec_out && (rows == 32 || !p.off);
      if (work)
        store_turned<TO, S::kCols>(s_turn + ew * 8192, whole ? &maps.out : nullptr, col, row_w0,
                                   static_cast<TO*>(p.out) + (long long)row_w0 * p.ldo + col, p.ldo, acc, w, lane, rows,
                                   p.N - col, p.vec_out != 0, turn_next);
    }
    if (lane == 0) bulk_wait_read<0>();
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // the pair's MMAs, copies and tensor-memory reads are all done
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem_base, S::kBufs * kW);
  __syncthreads();
  cluster_sync_all();
}

}  // namespace dg
