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
// A unit is 256 rows x kBN columns of one group.  Per block of 128 k (one
// stage: 128 bytes of each row, the width of the 128-byte swizzle) the
// leader issues four tcgen05.mma of M = 256, K = 32 into a fresh tensor-memory
// buffer; eight epilogue warps in each CTA take the block's sums out, multiply
// them by the scales and add them in registers, while the tensor cores work on
// the next block in another buffer.  fp32 throughout; one rounding at the
// store.  The fixed scale per 128 is why the sums leave tensor memory at every
// block: a 128 x 256 block takes the tensor cores 512 cycles, and its 256
// tcgen05.ld'ed columns per lane quarter are shared by two warps.
//
// Each CTA of a pair copies its own 128 rows of A and half of the columns of B
// (32 KB a stage at kBN = 256), so a pair reads (256 + kBN) rows per block.
// Copies of few rows use a smaller box (16 or 64 rows): the rest of the tile
// holds old bytes, and only rows that are not stored depend on them.
//
// Protocol of the barriers (rank 0 leads):
//   full[s]       rank 0's: both CTAs' copies of a stage have landed
//   empty[s]      both: the MMAs that read the stage are done
//   acc_full[b]   both: the block's sums are in tensor memory
//   acc_empty[b]  rank 0's: all 16 epilogue warps have read them
// All waits are bounded; after one runs out the CTA stops working and stores
// NaN for what it could not compute.
#pragma once

#include "fp8_small.cuh"
#include <type_traits>

#include "gemm_pair.cuh"

namespace dg {

constexpr int kFp8MaxGroups = 1024;
constexpr int kFp8EpiWarps = 8;
constexpr int kFp8Threads = 64 + 32 * kFp8EpiWarps;

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
// Arrive on a pair peer's (or this CTA's) mbarrier at the default scope.  What it
// orders are tensor-memory reads, by the tcgen05 fence before it; a release at
// cluster scope would add a memory barrier to every block of every warp, which
// measured 2900 cycles per block in place of about 600.
__device__ __forceinline__ void mbar_arrive_peer(uint32_t bar_cluster) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster) : "memory");
}
// acc (two fp32) += (lo, hi) * s (two equal fp32)
__device__ __forceinline__ void fma2(uint64_t& acc, uint32_t lo, uint32_t hi, uint64_t s) {
  asm("{\n\t.reg .b64 t;\n\tmov.b64 t, {%1, %2};\n\tfma.rn.f32x2 %0, t, %3, %0;\n\t}"
      : "+l"(acc)
      : "r"(lo), "r"(hi), "l"(s));
}
__device__ __forceinline__ uint64_t pack2(float v) {
  const uint32_t u = __float_as_uint(v);
  return ((uint64_t)u << 32) | u;
}

// tensor maps: A with boxes of 16, 64 and 128 rows, B with boxes of kBN / 4 and kBN / 2 rows
struct Fp8Maps {
  CUtensorMap a[3];
  CUtensorMap b[2];
};

struct Fp8Tables {
  int first[kFp8MaxGroups + 1];  // 256-row tiles of the groups before g
  int row0[kFp8MaxGroups];
  int row1[kFp8MaxGroups];
};

struct Fp8Job {
  int group, row0, row1, n0;  // the unit's rows [row0, row1) of at most 256, first column
};

__device__ __forceinline__ Fp8Job fp8_job(const Fp8GemmParams& p, const Fp8Tables* tb, int u, int m_tiles, int n_tiles,
                                          int bn) {
  Fp8Job j;
  if (!p.off) {
    const int nt = u / m_tiles, mt = u - nt * m_tiles;  // consecutive units share their columns of B
    j.group = 0;
    j.row0 = mt * 256;
    j.row1 = min(p.M, j.row0 + 256);
    j.n0 = nt * bn;
    return j;
  }
  int lo = 0, hi = p.G;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tb->first[mid] * n_tiles <= u) lo = mid;
    else hi = mid;
  }
  const int tiles = tb->first[lo + 1] - tb->first[lo];
  const int r = u - tb->first[lo] * n_tiles;
  const int nt = r / tiles, mt = r - nt * tiles;
  j.group = lo;
  j.row0 = tb->row0[lo] + mt * 256;
  j.row1 = min(tb->row1[lo], j.row0 + 256);
  j.n0 = nt * bn;
  return j;
}

template <int kBN>
struct Fp8Shape {
  static constexpr int kStageA = 128 * 128, kStageB = (kBN / 2) * 128, kStage = kStageA + kStageB;
  static constexpr int kBufs = kBN >= 256 ? 2 : 4;  // tensor-memory buffers of kBN columns
  static constexpr int kStages = kBN >= 256 ? 6 : 8;
  static constexpr int kSmem = 1024 + kStages * kStage + (2 * kStages + 2 * kBufs + 1) * 8 + 16;
};

// eight results of one row from column 0 of `o` on, `n` of them valid
template <class TO>
__device__ __forceinline__ void store8(TO* o, const float (&v)[8], int n, bool vec) {
  if (vec && n >= 8) {
    if constexpr (sizeof(TO) == 4) {
      reinterpret_cast<float4*>(o)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(o)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (std::is_same_v<TO, __half>) w[i] = pack_f16x2(v[2 * i], v[2 * i + 1]);
        else w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
      }
      *reinterpret_cast<uint4*>(o) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) store_out(o + i, v[i]);
  }
}

template <int kBN, class TO>
__global__ void __launch_bounds__(kFp8Threads, 1)
    fp8_pair_kernel(const __grid_constant__ Fp8Maps maps, const __grid_constant__ Fp8GemmParams p) {
  using S = Fp8Shape<kBN>;
  constexpr int kHalf = kBN / 2;             // columns of an epilogue warp
  constexpr int kAhead = kBN >= 256 ? 2 : 4;  // blocks of scales loaded ahead
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ Fp8Tables tabs;
  uint8_t* const smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* const sA = smem;
  uint8_t* const sB = smem + S::kStages * S::kStageA;
  uint64_t* const full = (uint64_t*)(sB + S::kStages * S::kStageB);
  uint64_t* const empty = full + S::kStages;
  uint64_t* const acc_full = empty + S::kStages;
  uint64_t* const acc_empty = acc_full + S::kBufs;
  uint64_t* const drain = acc_empty + S::kBufs;
  uint32_t* const tmem_slot = (uint32_t*)(drain + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = (int)(blockIdx.x >> 1), pairs = (int)(gridDim.x >> 1);
  const int n_tiles = (p.N + kBN - 1) / kBN;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int b = 0; b < S::kBufs; ++b) {
      mbar_init(smem_u32(&acc_full[b]), 1);
      mbar_init(smem_u32(&acc_empty[b]), 2 * kFp8EpiWarps);
    }
    mbar_init(smem_u32(drain), 1);
    fence_mbar_init();
    fence_proxy_async_smem();
    for (int i = 0; i < 3; ++i) tma_prefetch_desc(&maps.a[i]);
    for (int i = 0; i < 2; ++i) tma_prefetch_desc(&maps.b[i]);
  }
  grid_dep_wait();
  grid_dep_launch();
  int m_tiles = (p.M + 255) / 256;
  if (p.off) {
    if (warp == 2) {
      int sum = 0;
      for (int base = 0; base < p.G; base += 32) {
        const int g = base + lane;
        RowRange r{0, 0};
        if (g < p.G) r = group_rows(p.off, g, p.M);
        const int t = (r.row1 - r.row0 + 255) / 256;
        int inc = t;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += v;
        }
        if (g < p.G) {
          tabs.first[g] = sum + inc - t;
          tabs.row0[g] = r.row0;
          tabs.row1[g] = r.row1;
        }
        sum += __shfl_sync(0xffffffffu, inc, 31);
      }
      if (lane == 0) tabs.first[p.G] = sum;
    }
  }
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers initialised before either signals one
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), S::kBufs * kBN);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  if (p.off) m_tiles = tabs.first[p.G];
  const int U = m_tiles * n_tiles;

  if (warp == 0) {
    if (lane == 0) {
      // ---------------- copies (both CTAs) ----------------
      uint32_t it = 0;
      bool ok = true;
      const uint64_t pol_a = l2_policy_evict_last(), pol_b = l2_policy_evict_first();
      auto a_box = [&](int rows) { return rows <= 0 ? -1 : (rows <= 16 ? 0 : (rows <= 64 ? 1 : 2)); };
      auto a_bytes = [&](int box) { return box < 0 ? 0u : (box == 0 ? 16u : (box == 1 ? 64u : 128u)) * 128u; };
      for (int u = pair; u < U && ok; u += pairs) {
        const Fp8Job j = fp8_job(p, &tabs, u, m_tiles, n_tiles, kBN);
        const int mine = a_box(j.row1 - (j.row0 + (int)rank * 128));
        const int n_mma = min(kBN, (p.N - j.n0 + 31) & ~31);
        const int bb = n_mma <= kBN / 2 ? 0 : 1;
        const uint32_t tx = a_bytes(a_box(j.row1 - j.row0)) + a_bytes(a_box(j.row1 - j.row0 - 128)) +
                            2u * (uint32_t)(bb ? kBN / 2 : kBN / 4) * 128u;
        const int yA = j.row0 + (int)rank * 128;
        const int yB = j.group * p.N + j.n0 + (int)rank * (n_mma >> 1);
        for (int kb = 0; kb < p.KB; ++kb, ++it) {
          const int s = it % S::kStages;
          if (!mbar_wait(smem_u32(&empty[s]), ((it / S::kStages) & 1) ^ 1, nullptr)) { ok = false; break; }
          const uint32_t fb = mapa_shared(smem_u32(&full[s]), 0);
          if (rank == 0) mbar_arrive_expect_tx(smem_u32(&full[s]), tx);
          if (mine >= 0) tma_load_2d_pair(smem_u32(sA + s * S::kStageA), &maps.a[mine], fb, kb * 128, yA, pol_a);
          tma_load_2d_pair(smem_u32(sB + s * S::kStageB), &maps.b[bb], fb, kb * 128, yB, pol_b);
        }
      }
      // the leader's full barriers count both CTAs' bytes: wait until all have landed
      if (rank == 0) {
        const uint32_t first = it > (uint32_t)S::kStages ? it - S::kStages : 0;
        for (uint32_t q = first; q < it; ++q) mbar_wait(smem_u32(&full[q % S::kStages]), (q / S::kStages) & 1, nullptr);
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      // ---------------- MMAs (leader) ----------------
      uint32_t it = 0;
      bool ok = true;
      for (int u = pair; u < U && ok; u += pairs) {
        const Fp8Job j = fp8_job(p, &tabs, u, m_tiles, n_tiles, kBN);
        const uint32_t idesc = idesc_e4m3_f32(256, min(kBN, (p.N - j.n0 + 31) & ~31));
        for (int kb = 0; kb < p.KB; ++kb, ++it) {
          const int s = it % S::kStages, b = it % S::kBufs;
          if (!mbar_wait(smem_u32(&acc_empty[b]), ((it / S::kBufs) & 1) ^ 1, nullptr) ||
              !mbar_wait(smem_u32(&full[s]), (it / S::kStages) & 1, nullptr)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a0 = smem_u32(sA + s * S::kStageA), b0 = smem_u32(sB + s * S::kStageB);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_e4m3_pair(tmem_base + (uint32_t)(b * kBN), sdesc_k128(a0 + kk * 32), sdesc_k128(b0 + kk * 32), idesc,
                           kk > 0 ? 1u : 0u);
          umma_commit_pair_mc(smem_u32(&empty[s]), (uint16_t)3);
          umma_commit_pair_mc(smem_u32(&acc_full[b]), (uint16_t)3);
        }
      }
      umma_commit_pair(smem_u32(drain));
      mbar_wait(smem_u32(drain), 0, nullptr);
    }
  } else {
    // ---------------- epilogue (both CTAs; warps 2..9) ----------------
    const int quarter = warp & 3;              // tensor-memory lanes [32 quarter, +32)
    const int c_first = ((warp - 2) >> 2) * kHalf;  // columns [c_first, +kHalf)
    const uint32_t lane_base = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)c_first;
    const uint32_t release_to = mapa_shared(smem_u32(&acc_empty[0]), 0);
    uint32_t it = 0;
    bool ok = true;
    for (int u = pair; u < U; u += pairs) {
      const Fp8Job j = fp8_job(p, &tabs, u, m_tiles, n_tiles, kBN);
      const int row_w0 = j.row0 + (int)rank * 128 + quarter * 32;
      const int row = row_w0 + lane;
      const int n_left = p.N - (j.n0 + c_first);  // valid columns of this warp (may exceed kHalf)
      const bool work = row_w0 < j.row1 && n_left > 0;
      uint64_t acc[kHalf / 2];
#pragma unroll
      for (int i = 0; i < kHalf / 2; ++i) acc[i] = 0ull;
      // the scales of the next kAhead blocks are on their way
      const float* const sa = p.sa + min(row, j.row1 - 1);
      const float* const sb = p.sb + ((long long)j.group * p.NB + min((j.n0 + c_first) / kFp8Block, p.NB - 1)) * p.KB;
      float na[kAhead], nb[kAhead];
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {
        const int kb = min(q, p.KB - 1);
        na[q] = __ldg(sa + (long long)kb * p.lds);
        nb[q] = __ldg(sb + kb);
      }
#pragma unroll 1
      for (int kb = 0; kb < p.KB; ++kb) {
        const float sc = na[0] * nb[0];
#pragma unroll
        for (int q = 0; q + 1 < kAhead; ++q) {
          na[q] = na[q + 1];
          nb[q] = nb[q + 1];
        }
        {
          const int kn = min(kb + kAhead, p.KB - 1);
          na[kAhead - 1] = __ldg(sa + (long long)kn * p.lds);
          nb[kAhead - 1] = __ldg(sb + kn);
        }
        const int b = it % S::kBufs;
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&acc_full[b]), (it / S::kBufs) & 1, nullptr)) != 0;
        ++it;
        if (!ok) continue;
        tc_fence_after();
        if (work) {
          const uint32_t t0 = lane_base + (uint32_t)(b * kBN);
          const uint64_t s2 = pack2(sc);
          uint32_t ra[16], rb[16];
          tmem_ld16_nowait(t0, ra);
          tmem_wait_ld16(ra);
#pragma unroll
          for (int c = 0; c < kHalf / 16; c += 2) {
            tmem_ld16_nowait(t0 + (c + 1) * 16, rb);
#pragma unroll
            for (int i = 0; i < 8; ++i) fma2(acc[c * 8 + i], ra[2 * i], ra[2 * i + 1], s2);
            tmem_wait_ld16(rb);
            if (c + 2 < kHalf / 16) tmem_ld16_nowait(t0 + (c + 2) * 16, ra);
#pragma unroll
            for (int i = 0; i < 8; ++i) fma2(acc[(c + 1) * 8 + i], rb[2 * i], rb[2 * i + 1], s2);
            if (c + 2 < kHalf / 16) tmem_wait_ld16(ra);
          }
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_peer(release_to + (uint32_t)b * 8u);
      }
      if (work && row < j.row1) {
        const float w = !ok ? __uint_as_float(0x7fffffffu) : (p.row_w ? __ldg(p.row_w + row) : 1.0f);
        TO* const o = static_cast<TO*>(p.out) + (long long)row * p.ldo + j.n0 + c_first;
#pragma unroll
        for (int c = 0; c < kHalf / 8; ++c) {
          float v[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float((uint32_t)acc[c * 4 + i]) * w;
            v[2 * i + 1] = __uint_as_float((uint32_t)(acc[c * 4 + i] >> 32)) * w;
          }
          if (c * 8 < n_left) store8(o + c * 8, v, n_left - c * 8, p.vec_out != 0);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // the pair's MMAs, copies and tensor-memory reads are all done
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem_base, S::kBufs * kBN);
  __syncthreads();
  cluster_sync_all();
}

}  // namespace dg
