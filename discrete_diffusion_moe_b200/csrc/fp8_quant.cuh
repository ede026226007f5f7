// fp8_quant.cuh - quantisers to e4m3 with one fp32 scale for each block of 128:
// rows of activations (one scale per row and 128 columns) and weight matrices
// (one scale per 128 x 128 block).
//
// With a = max |x| of the block, raised to at least 2^-100 (so that 448 / a
// and a / 448 are normal numbers, and a block of zeros needs no case of its
// own):
//   scale = a / 448,   q = e4m3(x * (448 / a))
// the quotients and the product in fp32 (each rounded to nearest), the code
// rounded to nearest even and held to +-448.  The product with 448 / a instead
// of a quotient by the scale saves a division per element; it moves x / scale
// by at most 2^-23 of its value, 2^-19 of a code's rounding step.  A block that
// holds a NaN or an infinity gets the scale NaN and codes 0: every product it
// enters is NaN.
//
// One read of x, one write of the codes.  Bound by HBM: the weights (16 x 1408 x 2816
// bf16: 34 us, 0.86 of the copy bandwidth) and rows (32768 x 2816 bf16 47 us, 0.90).
// SwiGLU rows (32768 x 704 from interleaved bf16 columns: 28 us where the bytes alone
// would take 18) also by instruction issue, with an exponential, a quotient, a
// maximum and a conversion per element.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace dg {

constexpr int kFp8Block = 128;
constexpr float kE4m3Max = 448.0f;
constexpr float kFp8AmaxMin = 7.888609052210118e-31f;  // 2^-100

enum { kActNone = 0, kActSwiglu = 1, kActSwigluInterleaved = 2 };

// ---- loads -------------------------------------------------------------------
__device__ __forceinline__ float elem_f32(const __nv_bfloat16* p) { return __bfloat162float(__ldg(p)); }
__device__ __forceinline__ float elem_f32(const __half* p) { return __half2float(__ldg(p)); }
__device__ __forceinline__ float elem_f32(const float* p) { return __ldg(p); }

// eight consecutive elements (16-byte aligned) as raw words, and their values
template <class T>
struct Raw8 {
  static constexpr int kVecs = (int)sizeof(T) / 2;  // 16-byte vectors
  uint4 r[kVecs];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) r[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) r[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  }
  __device__ __forceinline__ float get(int i) const;
};
__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) {
  return i == 0 ? v.x : (i == 1 ? v.y : (i == 2 ? v.z : v.w));
}
template <>
__device__ __forceinline__ float Raw8<__nv_bfloat16>::get(int i) const {
  const uint32_t w = word_of(r[0], i >> 1);
  return __uint_as_float((i & 1) ? (w & 0xffff0000u) : (w << 16));
}
template <>
__device__ __forceinline__ float Raw8<__half>::get(int i) const {
  const uint32_t w = word_of(r[0], i >> 1);
  return __half2float(__ushort_as_half((unsigned short)((i & 1) ? (w >> 16) : (w & 0xffffu))));
}
template <>
__device__ __forceinline__ float Raw8<float>::get(int i) const {
  return __uint_as_float(word_of(r[i >> 2], i & 3));
}

// silu(g) * u with w = e^-|g|: silu(g) = g / (1 + e^-g) is g / (1 + w) for g >= 0 and
// g w / (1 + w) below, so that nothing overflows on the way and w keeps what a far
// negative gate leaves.  The quotient is the product with the approximate reciprocal
// (1 unit), corrected by its remainder.  e^x within 2 units, the quotient within 1 and
// three roundings: (2 + 1 + 3/2) 2^-23 of the value in all while w is a normal number
// (g above -87.3).  32768 x 704 interleaved bf16 columns 28 us; with e^x and the
// reciprocal straight from the approximate instructions 22, but off by |g| 2^-24 more.
__device__ __forceinline__ float swiglu(float g, float u) {
  const float w = expf(-fabsf(g)), den = 1.0f + w, num = g < 0.f ? g * w : g;
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(den));  // den in [1, 2]
  const float q = num * r;
  return fmaf(fmaf(-q, den, num), r, q) * u;
}

// ---- block scale and codes ------------------------------------------------------
struct BlockScale {
  float scale, inv;
};
// Bit patterns of magnitudes compare like the magnitudes, infinities and NaNs
// above all others.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }
// m: the block's largest magnitude (NaN where it holds one).  The quotient by the
// constant 448 is the product with its reciprocal corrected by the remainder
// (Markstein, 1990): rounded correctly, since every term is a normal number for m
// of 2^-100 and more.
__device__ __forceinline__ BlockScale block_scale(float m) {
  if (!(m <= 3.4028234663852886e38f)) return {__uint_as_float(0x7fffffffu), 0.f};
  const float a = fmaxf(m, kFp8AmaxMin), r = 1.0f / kE4m3Max, q = a * r;
  return {fmaf(fmaf(-q, kE4m3Max, a), r, q), __fdiv_rn(kE4m3Max, a)};
}
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// ---- rows ---------------------------------------------------------------------------
struct QuantRowsParams {
  const void* x;
  long long ldx;          // elements between rows of x
  const int32_t* index;   // optional [rows]: the row of x each output row takes
  long long x_rows;       // rows of x; an index outside [0, x_rows) reads as a row of zeros
  uint8_t* q;
  long long ldq;
  float* scale;           // [KB][lds]
  long long lds;
  int rows, K, KB;
};

// A few lanes take one (row, block of 128 columns), groups of eight elements each:
// group h of lane l starts at column (h * kLanes + l) * 8, so the lanes read
// consecutive 16-byte words of bf16, all of a thread's at once.  Instructions count as
// much as the bytes, so few lanes share what does not depend on the element (the task's
// place, the shuffles of the maximum, the scale), as far as registers allow for enough
// warps: 32768 x 2816 bf16 rows take 60 us with 16 lanes, 51 with 8, 47 with 4 and 71
// with 2; SwiGLU of 32768 x 704 (twice the inputs a result; with a cheaper exponential)
// 23.7 with 8, 26 with 4; fp32 rows, bound by HBM, 34.2 with 8 and 34.8 with 4.
// kVec: 16-byte loads and 8-byte stores (every row of x 16-byte aligned and K a
// multiple of 8); otherwise the elements are taken one by one, neighbours by
// neighbouring lanes, and more of them share a block, so that a step touches whole
// sectors: 32768 x 2815 bf16 rows take 208 us with 4 lanes, 110 with 8, 104 with 16;
// fp32 113 with 8, 102 with 16.
constexpr int kQuantThreads = 128;
template <class T, int ACT, bool kVec>
constexpr int kQuantLanes = !kVec ? 16 : (ACT == kActNone && sizeof(T) == 2 ? 4 : 8);

template <class T, int ACT, bool kVec>
__global__ void __launch_bounds__(kQuantThreads) quant_rows_kernel(const QuantRowsParams p) {
  grid_dep_wait();
  grid_dep_launch();
  constexpr int kLanes = kQuantLanes<T, ACT, kVec>, kElems = kFp8Block / kLanes, kGroups = kElems / 8;
  constexpr int kIn = ACT == kActNone ? 1 : 2;
  const int l = threadIdx.x % kLanes;
  // tasks below 2^31 (the host's check)
  const unsigned task = blockIdx.x * (kQuantThreads / kLanes) + threadIdx.x / kLanes;
  const int row = (int)(task / (unsigned)p.KB), k_lo = (int)(task - (unsigned)row * (unsigned)p.KB) * kFp8Block;
  const bool work = task < (unsigned)p.rows * (unsigned)p.KB;
  long long src = work ? row : -1;
  if (p.index && work) {
    src = __ldg(p.index + row);
    if (src >= p.x_rows) src = -1;
  }
  const T* const xr = static_cast<const T*>(p.x) + (src < 0 ? 0 : src) * p.ldx;

  float v[kElems];
  if constexpr (kVec) {
    Raw8<T> raw[kGroups][kIn];
#pragma unroll
    for (int h = 0; h < kGroups; ++h) {
      const int k = k_lo + (h * kLanes + l) * 8;
#pragma unroll
      for (int i = 0; i < kIn; ++i) raw[h][i].zero();
      if (src >= 0 && k < p.K) {  // K is a multiple of 8: all eight or none
        if constexpr (ACT == kActNone) {
          raw[h][0].load(xr + k);
        } else if constexpr (ACT == kActSwiglu) {
          raw[h][0].load(xr + k);
          raw[h][1].load(xr + p.K + k);
        } else {
          raw[h][0].load(xr + 2 * (long long)k);
          raw[h][1].load(xr + 2 * (long long)k + 8);
        }
      }
    }
#pragma unroll
    for (int h = 0; h < kGroups; ++h)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float& o = v[8 * h + i];
        if constexpr (ACT == kActNone) o = raw[h][0].get(i);
        else if constexpr (ACT == kActSwiglu) o = swiglu(raw[h][0].get(i), raw[h][1].get(i));
        else o = swiglu(raw[h][i >> 2].get((2 * i) & 7), raw[h][i >> 2].get(((2 * i) & 7) + 1));
      }
  } else {
#pragma unroll
    for (int i = 0; i < kElems; ++i) {
      const int k = k_lo + i * kLanes + l;
      const bool on = src >= 0 && k < p.K;
      if constexpr (ACT == kActNone) {
        v[i] = on ? elem_f32(xr + k) : 0.f;
      } else {
        const T* gp = ACT == kActSwiglu ? xr + k : xr + 2 * (long long)k;
        const T* up = ACT == kActSwiglu ? xr + p.K + k : gp + 1;
        v[i] = on ? swiglu(elem_f32(gp), elem_f32(up)) : 0.f;
      }
    }
  }
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < kElems; ++i) m = max(m, abs_bits(v[i]));
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (!work) return;
  const BlockScale s = block_scale(__uint_as_float(m));
  uint8_t* const qr = p.q + (long long)row * p.ldq;
#pragma unroll
  for (int h = 0; h < kGroups; ++h) {
    const float* const e = v + 8 * h;
    uint32_t lo = 0u, hi = 0u;
    if (s.inv != 0.f) {  // codes 0 where the scale is NaN
      lo = codes4(e[0] * s.inv, e[1] * s.inv, e[2] * s.inv, e[3] * s.inv);
      hi = codes4(e[4] * s.inv, e[5] * s.inv, e[6] * s.inv, e[7] * s.inv);
    }
    if constexpr (kVec) {
      const int k = k_lo + (h * kLanes + l) * 8;
      if (k < p.K) *reinterpret_cast<uint2*>(qr + k) = make_uint2(lo, hi);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int k = k_lo + (8 * h + i) * kLanes + l;
        if (k < p.K) qr[k] = (uint8_t)((i < 4 ? lo : hi) >> (8 * (i & 3)));
      }
    }
  }
  if (l == 0) p.scale[(long long)(k_lo / kFp8Block) * p.lds + row] = s.scale;
}

// ---- 128 x 128 blocks -------------------------------------------------------------------
struct QuantBlocksParams {
  const void* w;
  long long ldw;    // elements between rows; a group's rows follow the previous group's
  uint8_t* q;
  long long ldq;
  float* scale;     // [G][NB][KB]
  int N, K, NB, KB;
};

// One CTA per block: 256 threads hold its 16384 elements in registers (eight
// vectors of eight; all loads in flight together), take the maximum over the
// CTA and write the codes, so x is read once.
template <class T, bool kVec>
__global__ void __launch_bounds__(256) quant_blocks_kernel(const QuantBlocksParams p) {
  grid_dep_wait();
  grid_dep_launch();
  __shared__ uint32_t s_max[8];
  const int kb = (int)(blockIdx.x % (unsigned)p.KB);
  const unsigned rest = blockIdx.x / (unsigned)p.KB;
  const int nb = (int)(rest % (unsigned)p.NB);
  const long long g = rest / (unsigned)p.NB;
  const int c = threadIdx.x & 15, r0 = threadIdx.x >> 4;
  const long long row_base = g * p.N;
  const T* const w = static_cast<const T*>(p.w);

  Raw8<T> raw[kVec ? 8 : 1];
  float v[kVec ? 1 : 8][8];
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int n = nb * kFp8Block + u * 16 + r0;
    const T* wr = w + (row_base + n) * p.ldw;
    if constexpr (kVec) {
      raw[u].zero();
      const int k = kb * kFp8Block + c * 8;
      if (n < p.N && k < p.K) raw[u].load(wr + k);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int k = kb * kFp8Block + i * 16 + c;
        v[u][i] = (n < p.N && k < p.K) ? elem_f32(wr + k) : 0.f;
      }
    }
  }
  auto val = [&](int u, int i) -> float {
    if constexpr (kVec) return raw[u].get(i);
    else return v[u][i];
  };
  uint32_t m = 0u;
#pragma unroll
  for (int u = 0; u < 8; ++u)
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, abs_bits(val(u, i)));
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, s_max[i]);
  const BlockScale s = block_scale(__uint_as_float(m));
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int n = nb * kFp8Block + u * 16 + r0;
    if (n >= p.N) continue;
    uint8_t* const qr = p.q + (row_base + n) * p.ldq + kb * kFp8Block;
    uint32_t lo = 0u, hi = 0u;
    if (s.inv != 0.f) {
      lo = codes4(val(u, 0) * s.inv, val(u, 1) * s.inv, val(u, 2) * s.inv, val(u, 3) * s.inv);
      hi = codes4(val(u, 4) * s.inv, val(u, 5) * s.inv, val(u, 6) * s.inv, val(u, 7) * s.inv);
    }
    if constexpr (kVec) {
      if (kb * kFp8Block + c * 8 < p.K) *reinterpret_cast<uint2*>(qr + c * 8) = make_uint2(lo, hi);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (kb * kFp8Block + i * 16 + c < p.K) qr[i * 16 + c] = (uint8_t)((i < 4 ? lo : hi) >> (8 * (i & 3)));
    }
  }
  if (threadIdx.x == 0) p.scale[blockIdx.x] = s.scale;
}

}  // namespace dg
