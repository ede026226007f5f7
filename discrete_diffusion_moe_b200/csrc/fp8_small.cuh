// fp8_small.cuh - the block-scaled e4m3 product for at most eight rows and few
// features (a token's projections, its experts), where latency counts:
//
//   D[m, n] = w[m] * sum_kb sa[kb, m] * sb[n / 128, kb] * sum_{k in block kb} A[m, k] * B[n, k]
//
// A: activation codes [M, K], B: weight codes [N, K] (or [G, N, K] with the rows
// of A split among the groups).  The time is a launch and the one read of B.
//
// mma.sync m16n8k32 with 16 weight rows as its M side and the tokens as its N
// side: no tensor memory, tensor maps or barriers to set up (the streaming
// tcgen05 kernel starts about 3 us later), and the weights go from global memory
// to registers.  The order of k inside a block is free as long as A and B agree,
// so lane (g, t) of a warp takes bytes [16 t, 16 t + 16) of both halves of its
// rows' 128: two 16-byte loads per row, each of whole sectors, and four products
// per block.  The eight warps of a CTA share its 16 features and take every
// eighth block of K each.  One block per warp is in flight, so the 22 blocks of K = 2816
// are three trips to HBM one after another; 48 registers let five CTAs share an SM (at
// the price of 48 bytes of spill stores and 44 of loads).  With three blocks in flight
// and two CTAs 5632 features of one token took 7.7 us (two waves), so 6.3; 8 experts
// 14.0, so 10.3.  The
// warps' fp32 sums meet in shared memory in the order of the warps (the result
// does not depend on timing).
#pragma once

#include "common.cuh"
#include "fp8_quant.cuh"

namespace dg {

// Rows [row0, row1) of a group, held inside [0, M) whatever the offsets say.
struct RowRange {
  int row0, row1;
};
__device__ __forceinline__ RowRange held_inside(int off0, int off1, int M) {
  const int r0 = min(max(off0, 0), M);
  return {r0, min(max(off1, r0), M)};
}
__device__ __forceinline__ RowRange group_rows(const int32_t* off, int g, int M) {
  return held_inside(__ldg(off + g), __ldg(off + g + 1), M);
}

struct Fp8GemmParams {
  const uint8_t* a;
  long long lda;
  const float* sa;        // [KB][lds]
  long long lds;
  const uint8_t* b;       // [G][N] rows of ldb bytes
  long long ldb;
  const float* sb;        // [G][NB][KB]
  const float* row_w;     // optional [M]
  const int32_t* off;     // grouped: [G + 1]; null: one group of all rows
  void* out;
  long long ldo;
  int M, N, K, KB, NB, G;
  int vec_out;            // rows of the output start on 16-byte boundaries
};

__device__ __forceinline__ void store_out(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_out(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store_out(__half* p, float v) { *p = __float2half_rn(v); }

__device__ __forceinline__ void mma_e4m3(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 ld_stream(const uint8_t* p) {
  uint4 v;
  asm("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
      : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
      : "l"(p));
  return v;
}
// the first n bytes of a word
__device__ __forceinline__ uint32_t keep_bytes(uint32_t w, int n) {
  return n >= 4 ? w : (n <= 0 ? 0u : (w & ((1u << (8 * n)) - 1u)));
}
// A lane's 32 codes of one row's block: 16 from column k0 on and 16 from k0 + 64
// on; columns from K on read as 0.  A 16-byte word is read only where its first
// byte is inside the row, so the reads stay within the row's 16-byte pitch.
template <bool kStream>
__device__ __forceinline__ void load_codes32(uint32_t (&w)[8], const uint8_t* row, int k0, int K, bool on) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (on && k0 + 64 * h < K) {
      if constexpr (kStream) v = ld_stream(row + k0 + 64 * h);
      else v = __ldg(reinterpret_cast<const uint4*>(row + k0 + 64 * h));
    }
    w[4 * h] = v.x; w[4 * h + 1] = v.y; w[4 * h + 2] = v.z; w[4 * h + 3] = v.w;
  }
}

constexpr int kSmallWarps = 8, kSmallRows = 8, kSmallCtas = 5;  // CTAs per SM

template <class TO>
__global__ void __launch_bounds__(32 * kSmallWarps, kSmallCtas) fp8_small_kernel(const Fp8GemmParams p) {
  constexpr int kFeat = 16, kTok = kSmallRows;
  __shared__ float red[kSmallWarps][kTok][kFeat + 1];
  grid_dep_wait();
  grid_dep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * kFeat;

  // The blockIdx.y-th group that has rows: each lane looks at eight groups, their
  // offsets loaded together (one latency before the weights can be asked for).
  int grp = 0, row0 = 0, row1 = p.M;
  if (p.off) {
    int want = (int)blockIdx.y;
    grp = -1;
    for (int base = 0; base < p.G && grp < 0; base += 256) {
      const int g0 = base + 8 * lane;
      int o[9], has = 0;
#pragma unroll
      for (int i = 0; i < 9; ++i) o[i] = __ldg(p.off + min(g0 + i, p.G));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const RowRange r = held_inside(o[i], o[i + 1], p.M);
        has += g0 + i < p.G && r.row1 > r.row0;
      }
      int before = has;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, before, d);
        if (lane >= d) before += v;
      }
      const int total = __shfl_sync(0xffffffffu, before, 31);
      if (want < total) {
        before -= has;
        int fg = -1, f0 = 0, f1 = 0, at = before;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const RowRange r = held_inside(o[i], o[i + 1], p.M);
          if (g0 + i < p.G && r.row1 > r.row0) {
            if (at == want) {
              fg = g0 + i;
              f0 = r.row0;
              f1 = r.row1;
            }
            ++at;
          }
        }
        const int src = __ffs(__ballot_sync(0xffffffffu, fg >= 0)) - 1;
        grp = __shfl_sync(0xffffffffu, fg, src);
        row0 = __shfl_sync(0xffffffffu, f0, src);
        row1 = __shfl_sync(0xffffffffu, f1, src);
      }
      want -= total;
    }
    if (grp < 0) return;  // the same for every warp of the CTA
  }
  const uint8_t* const b = p.b + (long long)grp * p.N * p.ldb;
  const float* const sb = p.sb + ((long long)grp * p.NB + n0 / kFp8Block) * p.KB;

  for (int m0 = row0; m0 < row1; m0 += kTok) {
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int kb = warp; kb < p.KB; kb += kSmallWarps) {
      const int k0 = kb * kFp8Block + 16 * t;
      uint32_t wb[2][8], wa[8];
      float sc[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int n = n0 + 8 * h + g;
        load_codes32<true>(wb[h], b + (long long)n * p.ldb, k0, p.K, n < p.N);
      }
      load_codes32<false>(wa, p.a + (long long)(m0 + g) * p.lda, k0, p.K, m0 + g < row1);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int mc = m0 + 2 * t + e;
        sc[e] = mc < row1 ? __ldg(p.sa + (long long)kb * p.lds + mc) * __ldg(sb + kb) : 0.f;
      }
      if ((kb + 1) * kFp8Block > p.K) {
        // K ends inside this block: what lies behind it in the rows may be anything
#pragma unroll
        for (int w = 0; w < 8; ++w) {
          const int left = p.K - (k0 + 64 * (w >> 2) + 4 * (w & 3));
          wb[0][w] = keep_bytes(wb[0][w], left);
          wb[1][w] = keep_bytes(wb[1][w], left);
          wa[w] = keep_bytes(wa[w], left);
        }
      }
      float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < 4; ++s)
        mma_e4m3(c, wb[0][2 * s], wb[1][2 * s], wb[0][2 * s + 1], wb[1][2 * s + 1], wa[2 * s], wa[2 * s + 1]);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] = fmaf(c[e], sc[e & 1], acc[e]);
    }
    // features g (e 0, 1) and g + 8 (e 2, 3), tokens 2 t + (e & 1)
#pragma unroll
    for (int e = 0; e < 4; ++e) red[warp][2 * t + (e & 1)][g + 8 * (e >> 1)] = acc[e];
    __syncthreads();
    for (int o = threadIdx.x; o < kTok * kFeat; o += 32 * kSmallWarps) {
      const int tok = o / kFeat, f = o - tok * kFeat;
      const int m = m0 + tok, n = n0 + f;
      if (m < row1 && n < p.N) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kSmallWarps; ++w) s += red[w][tok][f];
        if (p.row_w) s *= __ldg(p.row_w + m);
        store_out(static_cast<TO*>(p.out) + (long long)m * p.ldo + n, s);
      }
    }
    __syncthreads();
  }
}

}  // namespace dg
