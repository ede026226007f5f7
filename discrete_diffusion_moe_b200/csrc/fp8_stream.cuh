// fp8_stream.cuh - the block-scaled e4m3 product for groups of up to a few dozen
// rows (experts of a canvas), where the time is the one read of the weights:
//
//   D[m, n] = w[m] * sum_kb sa[kb, m] * sb[n / 128, kb] * sum_{k in block kb} A[m, k] * B[n, k]
//
// Weights are the rows of the accumulator here: a unit is 128 features of one
// group times a chunk of at most kTok of its tokens, so an instruction is as wide
// as the tokens need (a multiple of 16 columns) and every copied byte of the
// large operand is used.  On the pair kernel a group of 24 rows fills a tenth of
// the 256 accumulator rows and its instructions take the time of 256: 64 rows of
// 262144 features take 212 us there and 127 here (weights at 0.89 of the copy
// bandwidth; 16 rows 110, all of it), 2048 rows on 84 of 128 experts of 1408
// features 62 us (0.84).
//
// Two CTAs per SM, each on its own, so that one's waits and stores are covered by
// the other.  Each stage holds one block of 128 k: 16 KB of weights and the
// chunk's token rows (boxes of 16, 32 or kTok rows); four stages in either CTA
// keep 128 KB of weights in flight per SM, about three times what the latency of
// HBM asks for.  Per block the MMA warp fills one of the tensor-memory buffers;
// four epilogue warps (32 features each) add it, scaled, to a thread's kTok sums:
// a column has its own token scale, read from shared memory, and the block's
// weight scale is one number for the CTA.  A warp's store is 32 consecutive
// features of one token.  Waits and their failure are as in fp8_gemm.cuh.
//
// Where there are fewer units than CTAs (single tokens) the blocks of a unit are
// split among the CTAs of a cluster: each leaves its sums in its shared memory
// (the stages, free by then), and the first adds them in the order of the ranks.
#pragma once

#include "fp8_gemm.cuh"

namespace dg {

constexpr int kStreamThreads = 256;  // warps: copies, MMAs, scales, idle, four of the epilogue

template <int kTok>
struct Fp8StreamShape {
  static constexpr int kStages = 4, kBufs = 4, kScaleSlots = 4;
  static constexpr int kStageA = 128 * 128, kStageB = kTok * 128;
  static constexpr int kScaleSlot = 4 * kTok + 4;  // [4][kTok] token scales, [4] weight scales
  static constexpr int kBars = 2 * kStages + 2 * kBufs + 2 * kScaleSlots + 1;
  static constexpr int kFixed = 1024 + kStages * (kStageA + kStageB) + kScaleSlots * kScaleSlot * 4 + kBars * 8 + 16;
  static constexpr int smem(int groups) { return kFixed + 4 * (3 * groups + 1); }  // with the groups' tables
};

// tensor maps: weights with a box of 128 rows, tokens with boxes of 16, 32 and kTok rows
struct Fp8StreamMaps {
  CUtensorMap w;
  CUtensorMap t[3];
};

__device__ __forceinline__ void umma_e4m3(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ float ld_dsmem_f1(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

template <int kTok, class TO>
__global__ void __launch_bounds__(kStreamThreads, 2)
    fp8_stream_kernel(const __grid_constant__ Fp8StreamMaps maps, const __grid_constant__ Fp8GemmParams p,
                      const int splits, const Fp8Waits wt) {
  using S = Fp8StreamShape<kTok>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ int s_dead;
  uint8_t* const smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* const sA = smem;
  uint8_t* const sB = sA + S::kStages * S::kStageA;
  float* const s_scale = (float*)(sB + S::kStages * S::kStageB);
  uint64_t* const bars = (uint64_t*)(s_scale + S::kScaleSlots * S::kScaleSlot);
  uint32_t* const tmem_slot = (uint32_t*)(bars + S::kBars);
  const Fp8Tables tabs((int*)(tmem_slot + 4), p.G);
  const uint32_t full = smem_u32(bars);                  // a stage's copies have landed
  const uint32_t empty = full + 8 * S::kStages;          // its MMAs are done
  const uint32_t acc_full = empty + 8 * S::kStages;      // a block's sums are in their buffer
  const uint32_t acc_empty = acc_full + 8 * S::kBufs;    // the four epilogue warps have read it
  const uint32_t sc_full = acc_empty + 8 * S::kBufs;
  const uint32_t sc_empty = sc_full + 8 * S::kScaleSlots;
  const uint32_t drain = sc_empty + 8 * S::kScaleSlots;
  const uint32_t dead = smem_u32(&s_dead);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // splits > 1: one unit per cluster, this CTA takes blocks [kb0, kb1)
  const int rank = splits > 1 ? (int)cluster_ctarank() : 0;
  const int first = (int)blockIdx.x / splits, stride = (int)gridDim.x / splits;
  const int kb_lo = p.KB * rank / splits, kb_hi = p.KB * (rank + 1) / splits;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(full + 8 * s, 1);
      mbar_init(empty + 8 * s, 1);
    }
    for (int b = 0; b < S::kBufs; ++b) {
      mbar_init(acc_full + 8 * b, 1);
      mbar_init(acc_empty + 8 * b, 4);
    }
    for (int i = 0; i < S::kScaleSlots; ++i) {
      mbar_init(sc_full + 8 * i, 32);
      mbar_init(sc_empty + 8 * i, 4);
    }
    mbar_init(drain, 1);
    s_dead = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
    tma_prefetch_desc(&maps.w);
    for (int i = 0; i < 3; ++i) tma_prefetch_desc(&maps.t[i]);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), S::kBufs * kTok);
    tmem_relinquish();
  }
  grid_dep_wait();
  if (p.off && warp == 4) fp8_tables<kTok>(p, tabs, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dep_launch();  // not before the tensor memory is held
  const uint32_t tmem_base = *tmem_slot;
  const int f_tiles = (p.N + 127) / 128;
  const int chunks = p.off ? tabs.first[p.G] : (p.M + kTok - 1) / kTok;
  // a cluster has one unit, whatever the offsets say
  const int U = splits > 1 ? min(f_tiles * chunks, stride) : f_tiles * chunks;
  // unit u: a group's feature tiles one after the other, the chunks of a tile side by side
  auto job = [&](int u) { return fp8_job<kTok>(p, tabs, u, chunks, f_tiles, 128); };

  if (warp == 0) {
    // ---------------- copies ----------------
    uint32_t it = 0;
    const uint64_t pol_w = l2_policy_evict_first(), pol_t = l2_policy_evict_last();
    const uint32_t dstA = smem_u32(sA), dstB = smem_u32(sB);
    bool ok = true;
    for (int u = first; u < U && ok; u += stride) {
      const Fp8Job j = job(u);
      const int held = wt.hold == kHoldCopies && u == wt.unit ? wt.block : -1;
      const int rows = j.row1 - j.row0;
      const int box = rows <= 16 ? 0 : (rows <= 32 ? 1 : 2);
      const uint32_t tx = (uint32_t)(128 + (box == 0 ? 16 : (box == 1 ? 32 : kTok))) * 128u;
#pragma unroll 1
      for (int kb = kb_lo; kb < kb_hi; ++kb, ++it) {
        const uint32_t s = it % S::kStages, bar = full + s * 8u;
        if (!(ok = wait_or_die(empty + s * 8u, ((it / S::kStages) & 1) ^ 1, dead, wt))) break;
        if (kb != held && elect_one()) {
          mbar_arrive_expect_tx(bar, tx);
          tma_load_2d_hint(dstA + s * S::kStageA, &maps.w, bar, kb * 128, j.group * p.N + j.n0, pol_w);
          tma_load_2d_hint(dstB + s * S::kStageB, &maps.t[box], bar, kb * 128, j.row0, pol_t);
        }
        __syncwarp();
      }
    }
    for (uint32_t q = it > (uint32_t)S::kStages ? it - S::kStages : 0; q < it; ++q)
      wait_to_leave(full + (q % S::kStages) * 8u, (q / S::kStages) & 1, dead, wt);
  } else if (warp == 1) {
    // ---------------- MMAs ----------------
    uint32_t it = 0;
    const uint64_t descA = sdesc_k128(smem_u32(sA)), descB = sdesc_k128(smem_u32(sB));
    bool ok = true;
    for (int u = first; u < U && ok; u += stride) {
      const Fp8Job j = job(u);
      const uint32_t idesc = idesc_e4m3_f32(128, (j.row1 - j.row0 + 15) & ~15);
#pragma unroll 1
      for (int kb = kb_lo; kb < kb_hi; ++kb, ++it) {
        const uint32_t s = it % S::kStages, b = it % S::kBufs;
        if (!(ok = wait_or_die(acc_empty + b * 8u, ((it / S::kBufs) & 1) ^ 1, dead, wt) &&
                   wait_or_die(full + s * 8u, (it / S::kStages) & 1, dead, wt)))
          break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t da = descA + s * (S::kStageA / 16), db = descB + s * (S::kStageB / 16);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_e4m3(tmem_base + b * kTok, da + 2 * kk, db + 2 * kk, idesc, kk > 0 ? 1u : 0u);
          umma_commit(empty + s * 8u);
          umma_commit(acc_full + b * 8u);
        }
        __syncwarp();
      }
    }
    if (elect_one()) umma_commit(drain);
    wait_to_leave(drain, 0, dead, wt);
  } else if (warp == 2) {
    // ---------------- scales: four blocks per slot ----------------
    uint32_t batch = 0;
    bool ok = true;
    for (int u = first; u < U && ok; u += stride) {
      const Fp8Job j = job(u);
      const int held = wt.hold == kHoldScales && u == wt.unit ? wt.block : -1;
      const float* const sb = p.sb + ((long long)j.group * p.NB + j.n0 / kFp8Block) * p.KB;
#pragma unroll 1
      for (int kb0 = kb_lo; kb0 < kb_hi; kb0 += 4, ++batch) {
        const uint32_t slot = batch % S::kScaleSlots;
        if (!(ok = wait_or_die(sc_empty + slot * 8u, ((batch / S::kScaleSlots) & 1) ^ 1, dead, wt))) break;
        const uint32_t dst = smem_u32(s_scale + slot * S::kScaleSlot);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float* const src = p.sa + (long long)min(kb0 + q, p.KB - 1) * p.lds;
#pragma unroll
          for (int i = 0; i < kTok / 32; ++i)
            cp_async4(dst + (uint32_t)(q * kTok + 32 * i + lane) * 4u, src + min(j.row0 + 32 * i + lane, j.row1 - 1));
        }
        if (lane < 4) cp_async4(dst + (uint32_t)(4 * kTok + lane) * 4u, sb + min(kb0 + lane, p.KB - 1));
        if (held < kb0 || held > kb0 + 3) cp_async_arrive(sc_full + slot * 8u);
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp >= 4) {
    // ---------------- epilogue: features [32 quarter, +32) ----------------
    const int quarter = warp & 3;
    const uint32_t lane_base = tmem_base + ((uint32_t)(quarter * 32) << 16);
    uint32_t it = 0, batch = 0;
    bool releases = lane == 0;
    for (int u = first; u < U; u += stride) {
      const Fp8Job j = job(u);
      const int n_ld = (j.row1 - j.row0 + 31) / 32;  // 32-token parts
      float acc[kTok], rw[kTok / 32];  // rw: the row weights of tokens lane, lane + 32, ..
#pragma unroll
      for (int i = 0; i < kTok; ++i) acc[i] = 0.f;
#pragma unroll
      for (int i = 0; i < kTok / 32; ++i) rw[i] = p.row_w ? __ldg(p.row_w + min(j.row0 + 32 * i + lane, j.row1 - 1)) : 1.f;
#pragma unroll 1
      for (int kb = alive(dead) ? kb_lo : kb_hi; kb < kb_hi; ++kb, ++it) {
        const uint32_t slot = batch % S::kScaleSlots, b = it % S::kBufs;
        const int q = (kb - kb_lo) & 3;
        if (q == 0) wait_or_keep(sc_full + slot * 8u, (batch / S::kScaleSlots) & 1, dead, wt, releases);
        const uint32_t at = smem_u32(s_scale + slot * S::kScaleSlot);
        const float sb = __int_as_float(ld_shared_flag(at + (uint32_t)(4 * kTok + q) * 4u));
        wait_or_keep(acc_full + b * 8u, (it / S::kBufs) & 1, dead, wt, releases);
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < kTok / 32; ++c) {
          if (c < n_ld) {
            uint32_t r[32];
            tmem_ld32_nowait(lane_base + b * kTok + c * 32, r);
            tmem_wait32(r);
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const float4 sa = ld_shared_f4(at + (uint32_t)(q * kTok + c * 32 + i) * 4u);
              acc[c * 32 + i] = fmaf(__uint_as_float(r[i]), sa.x * sb, acc[c * 32 + i]);
              acc[c * 32 + i + 1] = fmaf(__uint_as_float(r[i + 1]), sa.y * sb, acc[c * 32 + i + 1]);
              acc[c * 32 + i + 2] = fmaf(__uint_as_float(r[i + 2]), sa.z * sb, acc[c * 32 + i + 2]);
              acc[c * 32 + i + 3] = fmaf(__uint_as_float(r[i + 3]), sa.w * sb, acc[c * 32 + i + 3]);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (releases) mbar_arrive(acc_empty + b * 8u);
        if (q == 3 || kb + 1 == kb_hi) {
          if (releases) mbar_arrive(sc_empty + slot * 8u);
          ++batch;
        }
      }
      const int f = quarter * 32 + lane, n = j.n0 + f, rows = j.row1 - j.row0;
      if (splits > 1) {  // added and stored below, when the whole cluster has come there
        float* const sums = reinterpret_cast<float*>(smem);  // every copy into the stages has been used
#pragma unroll
        for (int i = 0; i < kTok; ++i)
          if (i < rows) sums[i * 128 + f] = acc[i];
        continue;
      }
      const bool bad = !alive(dead);  // a wait ran out: what was added is not the product
      TO* o = static_cast<TO*>(p.out) + (long long)j.row0 * p.ldo + n;
#pragma unroll
      for (int c = 0; c < kTok / 32; ++c) {
        if (c < n_ld) {
#pragma unroll
          for (int i = 0; i < 32; ++i, o += p.ldo) {
            const float w = __shfl_sync(0xffffffffu, rw[c], i);
            if (c * 32 + i < rows && n < p.N) store_out(o, bad ? __uint_as_float(0x7fffffffu) : acc[c * 32 + i] * w);
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, S::kBufs * kTok);
  if (splits > 1) {
    if (s_dead)  // a wait ran out: what was added is not the product
      for (int i = threadIdx.x; i < kTok * 128; i += kStreamThreads) reinterpret_cast<float*>(smem)[i] = __uint_as_float(0x7fffffffu);
    cluster_sync_all();  // every CTA's sums are written
    if (first < U) {
      // token i is added up (in the order of the ranks) and stored by CTA i % splits
      const Fp8Job j = job(first);
      const int f = threadIdx.x & 127, n = j.n0 + f, rows = j.row1 - j.row0;
      for (int i = rank + splits * (int)(threadIdx.x >> 7); i < rows; i += 2 * splits) {
        float v = 0.f;
        for (int r = 0; r < splits; ++r) v += ld_dsmem_f1(mapa_shared(smem_u32(smem) + (uint32_t)(i * 128 + f) * 4u, (uint32_t)r));
        if (p.row_w) v *= __ldg(p.row_w + j.row0 + i);
        if (n < p.N) store_out(static_cast<TO*>(p.out) + (long long)(j.row0 + i) * p.ldo + n, v);
      }
    }
    cluster_sync_all();  // no CTA leaves while another reads its shared memory
  }
}

}  // namespace dg
