// fp8_api.cu - host side of the 8-bit block-scaled operators of include/dg.h:
// argument checks, choice of kernel and launches.
#include <stdint.h>
#include <string.h>

#include <algorithm>

#include "../../include/dg.h"
#include "../../include/dg_testing.h"
#include "fp8_gemm.cuh"
#include "fp8_quant.cuh"
#include "fp8_small.cuh"
#include "fp8_stream.cuh"
#include "host.cuh"

using namespace dg;

namespace {

constexpr long long kMaxDim = 2147483647ll - 4096;  // tile coordinates stay within 32 bits

// The usual waits, or what dg_test_fp8_hold set for this thread's products.
constexpr Fp8Waits kUsualWaits{kWaitLimitNs, nullptr, kHoldNothing, 0, 0};
thread_local Fp8Waits g_waits = kUsualWaits;

size_t dtype_bytes(int dt) { return dt == DG_F32 ? 4 : 2; }
bool dtype_ok(int dt) { return dt == DG_BF16 || dt == DG_F16 || dt == DG_F32; }
bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

template <class T, int ACT, bool kVec>
dg_status launch_quant_rows(const QuantRowsParams& p, cudaStream_t st) {
  const long long tasks = (long long)p.rows * p.KB;
  const dim3 grid((unsigned)ceil_div(tasks, (long long)(kQuantThreads / kQuantLanes<T, ACT, kVec>)));
  DG_CUDA(Launch(grid, dim3(kQuantThreads), 0, st)(quant_rows_kernel<T, ACT, kVec>, p));
  return DG_OK;
}
template <class T, int ACT>
dg_status launch_quant_rows(const QuantRowsParams& p, bool vec, cudaStream_t st) {
  return vec ? launch_quant_rows<T, ACT, true>(p, st) : launch_quant_rows<T, ACT, false>(p, st);
}

template <class T>
dg_status launch_quant_rows(const QuantRowsParams& p, int act, bool vec, cudaStream_t st) {
  switch (act) {
    case DG_ACT_NONE: return launch_quant_rows<T, kActNone>(p, vec, st);
    case DG_ACT_SWIGLU: return launch_quant_rows<T, kActSwiglu>(p, vec, st);
    default: return launch_quant_rows<T, kActSwigluInterleaved>(p, vec, st);
  }
}

template <class T>
dg_status launch_quant_blocks(const QuantBlocksParams& p, long long blocks, bool vec, cudaStream_t st) {
  if (vec) DG_CUDA(Launch(dim3((unsigned)blocks), dim3(256), 0, st)(quant_blocks_kernel<T, true>, p));
  else     DG_CUDA(Launch(dim3((unsigned)blocks), dim3(256), 0, st)(quant_blocks_kernel<T, false>, p));
  return DG_OK;
}

template <class TO>
dg_status launch_small(const Fp8GemmParams& p, cudaStream_t st) {
  const dim3 grid((unsigned)ceil_div(p.N, 16), p.off ? (unsigned)std::min(p.G, p.M) : 1u);
  DG_CUDA(Launch(grid, dim3(32 * kSmallWarps), 0, st)(fp8_small_kernel<TO>, p));
  return DG_OK;
}

// Codes [rows, K] with `pitch` bytes between rows as a tensor of bytes; boxes of
// 128 columns (one block) x box_rows with the 128-byte swizzle.  Columns and
// rows outside read as zero codes.
dg_status make_tmap_codes(CUtensorMap* m, const uint8_t* base, long long K, long long rows, long long pitch,
                          int box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return fail(DG_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
  cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)pitch};
  cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
  cuuint32_t es[2] = {1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(base), dims, strides, box, es,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(DG_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  return DG_OK;
}

// The output [M, N] for stores of boxes of 128 bytes x 32 rows with the 128-byte
// swizzle, clipped at its edges.
template <class TO>
dg_status make_tmap_out(CUtensorMap* m, void* base, long long N, long long M, long long ldo) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return fail(DG_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
  const CUtensorMapDataType dt = std::is_same_v<TO, float> ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                 : std::is_same_v<TO, __half> ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                              : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  cuuint64_t dims[2] = {(cuuint64_t)N, (cuuint64_t)M};
  cuuint64_t strides[1] = {(cuuint64_t)ldo * sizeof(TO)};
  cuuint32_t box[2] = {128 / sizeof(TO), 32};
  cuuint32_t es[2] = {1, 1};
  const CUresult r = fn(m, dt, 2, base, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(DG_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  return DG_OK;
}

template <int kW, class TO>
dg_status launch_pair(const Fp8GemmParams& p, const Fp8Waits& wt, int pairs, cudaStream_t st) {
  using S = Fp8Shape<kW>;
  Fp8Maps maps;
  const int a_rows[3] = {16, 64, 128};
  for (int i = 0; i < 3; ++i) DG_TRY(make_tmap_codes(&maps.a[i], p.a, p.K, p.M, p.lda, a_rows[i]));
  for (int i = 0; i < 2; ++i) DG_TRY(make_tmap_codes(&maps.b[i], p.b, p.K, (long long)p.G * p.N, p.ldb, kW / (i ? 2 : 4)));
  memset(&maps.out, 0, sizeof maps.out);
  if (p.vec_out) DG_TRY(make_tmap_out<TO>(&maps.out, p.out, p.N, p.M, p.ldo));
  const void* fn = (const void*)fp8_pair_kernel<kW, TO>;
  DG_TRY(set_smem_attr(fn, S::kSmem, true));
  const long long tiles = p.off ? std::min(p.G, p.M) + (long long)p.M / 256 : ceil_div(p.M, 256);  // at most
  const unsigned grid = 2u * (unsigned)std::min<long long>(pairs, tiles * ceil_div(p.N, kW));
  DG_CUDA(Launch(dim3(grid), dim3(kFp8Threads), S::kSmem, st).cluster(2, 1, 1)(fp8_pair_kernel<kW, TO>, maps, p, wt));
  return DG_OK;
}

template <int kTok, class TO>
dg_status launch_stream(const Fp8GemmParams& p, const Fp8Waits& wt, int sms, cudaStream_t st) {
  using S = Fp8StreamShape<kTok>;
  Fp8StreamMaps maps;
  const int rows[3] = {16, 32, kTok};
  DG_TRY(make_tmap_codes(&maps.w, p.b, p.K, (long long)p.G * p.N, p.ldb, 128));
  for (int i = 0; i < 3; ++i) DG_TRY(make_tmap_codes(&maps.t[i], p.a, p.K, p.M, p.lda, rows[i]));
  DG_TRY(set_smem_attr((const void*)fp8_stream_kernel<kTok, TO>, S::smem(kFp8MaxGroups), true));
  const int smem = S::smem(p.G), ctas = smem <= 113 * 1024 ? 2 : 1;  // of an SM's 228 KB, 1 KB of each CTA reserved
  const long long chunks = p.off ? std::min(p.G, p.M) + (long long)p.M / kTok : ceil_div(p.M, kTok);  // at most
  const long long units = chunks * ceil_div(p.N, 128), slots = (long long)ctas * sms;
  // few units: split each one's blocks, two at least to a CTA, among a cluster
  const int splits = (int)std::max<long long>(1, std::min<long long>({slots / units, 8, p.KB / 2}));
  Launch l(dim3((unsigned)(splits > 1 ? splits * units : std::min(units, slots))), dim3(kStreamThreads), smem, st);
  if (splits > 1) l.cluster((unsigned)splits, 1, 1);
  DG_CUDA(l(fp8_stream_kernel<kTok, TO>, maps, p, splits, wt));
  return DG_OK;
}

// Which kernel, by rows and columns (us, K = 2816, bf16 out, where not said otherwise):
//   at most 8 rows and two waves of its CTAs: mma.sync, where the set-up counts
//     (one token, 5632 features: 6.6, streaming 9.7; 262144 features: 132, 108);
//   at most kStreamRows rows, or kStreamGroupRows a group on average: the streaming
//     kernel, which reads the weights once for 64 rows (262144 features: 64 rows
//     127, pairs 212, 80 rows 225, 216; 1408 features of 128 experts: 8192 rows
//     114, pairs 151, 12288 rows 159, 156);
//     but from 33 rows on pairs if one wave of them does it and keeps more than half
//     of them busy (5632 features, 64 rows: pairs 12.5, streaming 14.2; K = 704: 7.2,
//     11.7; 2816 features, a smaller part of a wave: 11.9, 10.9);
//   else CTA pairs, with tiles of 128 columns instead of 256 if that needs fewer than 5/3
//     as many waves, the ratio of what a wave takes (256 rows of 5632 features: 13.2, 17.5;
//     1024 rows: 27.6, 30.9; 8192 rows: 156, 138; 40000 rows of 128 features: 31.5, 40.1).
// For groups the row tiles are an estimate: the offsets are on the device.
constexpr int kStreamRows = 64, kStreamGroupRows = 80, kPairRows = 32;

template <class TO>
dg_status launch_product(const Fp8GemmParams& p, const Fp8Waits& wt, cudaStream_t st) {
  const int sms = device_sms(), pairs = sms / 2;
  const long long groups = p.off ? std::min(p.G, p.M) : 1;  // that may have rows
  if (p.M <= kSmallRows && groups * ceil_div(p.N, 16) <= 2ll * kSmallCtas * sms) return launch_small<TO>(p, st);
  const long long tiles = p.off ? std::max<long long>(groups, groups / 2 + p.M / 256) : ceil_div(p.M, 256);
  const long long units128 = tiles * ceil_div(p.N, 128), units256 = tiles * ceil_div(p.N, 256);
  const bool one_wave = units128 <= pairs && 2 * units128 > pairs;
  if (p.M <= (p.off ? kStreamGroupRows : kStreamRows) * groups && !(p.M > kPairRows * groups && one_wave))
    return launch_stream<64, TO>(p, wt, sms, st);
  if (3 * ceil_div(units128, pairs) < 5 * ceil_div(units256, pairs)) return launch_pair<128, TO>(p, wt, pairs, st);
  return launch_pair<256, TO>(p, wt, pairs, st);
}

dg_status product(const char* who, const Fp8GemmParams& p, int out_dtype, int* err, cudaStream_t st) {
  Fp8Waits wt = g_waits;
  wt.err = err;
  switch (out_dtype) {
    case DG_BF16: return launch_product<__nv_bfloat16>(p, wt, st);
    case DG_F16: return launch_product<__half>(p, wt, st);
    case DG_F32: return launch_product<float>(p, wt, st);
    default: return fail(DG_ERR_INVALID_ARG, "%s: output type %d", who, out_dtype);
  }
}

// Checks shared by the dense and the grouped product; fills `p`.
dg_status check_product(const char* who, const uint8_t* a, int64_t lda, const float* sa, int64_t lds,
                        const uint8_t* b, int64_t ldb, const float* sb, const int32_t* off, int64_t G, int64_t M,
                        int64_t N, int64_t K, const float* row_w, void* out, int32_t out_dtype, int64_t ldo,
                        Fp8GemmParams* p) {
  if (M < 0 || N < 1 || K < 1 || M > kMaxDim || N > kMaxDim || K > kMaxDim)
    return fail(DG_ERR_INVALID_ARG, "%s: sizes %lld x %lld x %lld", who, (long long)M, (long long)N, (long long)K);
  if (!dtype_ok(out_dtype)) return fail(DG_ERR_INVALID_ARG, "%s: output type %d", who, (int)out_dtype);
  if (G < 1 || G > kFp8MaxGroups) return fail(DG_ERR_INVALID_ARG, "%s: %lld groups (1..%d)", who, (long long)G, kFp8MaxGroups);
  if (G * N > kMaxDim) return fail(DG_ERR_INVALID_ARG, "%s: groups x N exceeds 2^31 - 4097", who);
  if (lda < K || lda % 16 || ldb < K || ldb % 16)
    return fail(DG_ERR_INVALID_ARG, "%s: row pitches %lld, %lld of the codes (multiples of 16, at least K = %lld)", who,
                (long long)lda, (long long)ldb, (long long)K);
  if (lds < M || ldo < N)
    return fail(DG_ERR_INVALID_ARG, "%s: pitch %lld of the row scales (at least M), %lld of the output (at least N)", who,
                (long long)lds, (long long)ldo);
  if (M == 0) { *p = Fp8GemmParams{}; return DG_OK; }
  if (!a || !sa || !b || !sb || !out) return fail(DG_ERR_INVALID_ARG, "%s: null pointer", who);
  if (!aligned(a, 16) || !aligned(b, 16)) return fail(DG_ERR_INVALID_ARG, "%s: codes must be 16-byte aligned", who);
  const size_t osz = dtype_bytes(out_dtype);
  if (!aligned(sa, 4) || !aligned(sb, 4) || !aligned(off, 4) || !aligned(row_w, 4) || !aligned(out, osz))
    return fail(DG_ERR_INVALID_ARG, "%s: misaligned pointer", who);
  Fp8GemmParams q{};
  q.a = a; q.lda = lda; q.sa = sa; q.lds = lds;
  q.b = b; q.ldb = ldb; q.sb = sb;
  q.row_w = row_w; q.off = off;
  q.out = out; q.ldo = ldo;
  q.M = (int)M; q.N = (int)N; q.K = (int)K;
  q.KB = (int)ceil_div(K, kFp8Block);
  q.NB = (int)ceil_div(N, kFp8Block);
  q.G = (int)G;
  q.vec_out = aligned(out, 16) && (ldo * (long long)osz) % 16 == 0;
  *p = q;
  return DG_OK;
}

}  // namespace

extern "C" dg_status dg_fp8_quantize(const void* d_x, int32_t dtype, int64_t ldx, int64_t x_rows,
                                     const int32_t* d_index, int32_t act, int64_t rows, int64_t cols, uint8_t* d_q,
                                     int64_t ldq, float* d_scale, int64_t lds, void* stream) {
  if (!dtype_ok(dtype)) return fail(DG_ERR_INVALID_ARG, "dg_fp8_quantize: input type %d", (int)dtype);
  if (act < DG_ACT_NONE || act > DG_ACT_SWIGLU_INTERLEAVED)
    return fail(DG_ERR_INVALID_ARG, "dg_fp8_quantize: activation %d", (int)act);
  if (rows < 0 || cols < 1 || x_rows < 0 || rows > kMaxDim || x_rows > kMaxDim || cols > kMaxDim / 2)
    return fail(DG_ERR_INVALID_ARG, "dg_fp8_quantize: sizes %lld (of %lld) x %lld", (long long)rows, (long long)x_rows,
                (long long)cols);
  const long long in_cols = act == DG_ACT_NONE ? cols : 2 * cols;
  if (ldx < in_cols || ldq < cols || ldq % 16 || lds < rows)
    return fail(DG_ERR_INVALID_ARG, "dg_fp8_quantize: pitches %lld of x, %lld of the codes (a multiple of 16), %lld of the scales",
                (long long)ldx, (long long)ldq, (long long)lds);
  if (!d_index && x_rows < rows)
    return fail(DG_ERR_INVALID_ARG, "dg_fp8_quantize: %lld rows of x for %lld output rows", (long long)x_rows, (long long)rows);
  if (rows == 0) return DG_OK;
  if ((!d_x && x_rows > 0) || !d_q || !d_scale) return fail(DG_ERR_INVALID_ARG, "dg_fp8_quantize: null pointer");
  const size_t sz = dtype_bytes(dtype);
  if (!aligned(d_x, sz) || !aligned(d_q, 16) || !aligned(d_scale, 4) || !aligned(d_index, 4))
    return fail(DG_ERR_INVALID_ARG, "dg_fp8_quantize: misaligned pointer (codes: 16 bytes)");
  QuantRowsParams p{};
  p.x = d_x; p.ldx = ldx; p.index = d_index; p.x_rows = x_rows;
  p.q = d_q; p.ldq = ldq; p.scale = d_scale; p.lds = lds;
  p.rows = (int)rows; p.K = (int)cols; p.KB = (int)ceil_div(cols, kFp8Block);
  if ((long long)p.rows * p.KB > kMaxDim)  // the kernel counts blocks in 32 bits
    return fail(DG_ERR_INVALID_ARG, "dg_fp8_quantize: too many blocks");
  const bool vec = cols % 8 == 0 && aligned(d_x, 16) && (ldx * (long long)sz) % 16 == 0;
  cudaStream_t st = (cudaStream_t)stream;
  switch (dtype) {
    case DG_BF16: return launch_quant_rows<__nv_bfloat16>(p, act, vec, st);
    case DG_F16: return launch_quant_rows<__half>(p, act, vec, st);
    default: return launch_quant_rows<float>(p, act, vec, st);
  }
}

extern "C" dg_status dg_fp8_quantize_blocks(const void* d_w, int32_t dtype, int64_t ldw, int64_t groups, int64_t rows,
                                            int64_t cols, uint8_t* d_q, int64_t ldq, float* d_scale, void* stream) {
  if (!dtype_ok(dtype)) return fail(DG_ERR_INVALID_ARG, "dg_fp8_quantize_blocks: input type %d", (int)dtype);
  if (groups < 0 || rows < 1 || cols < 1 || groups > kMaxDim || rows > kMaxDim || cols > kMaxDim)
    return fail(DG_ERR_INVALID_ARG, "dg_fp8_quantize_blocks: sizes %lld x %lld x %lld", (long long)groups, (long long)rows,
                (long long)cols);
  if (ldw < cols || ldq < cols || ldq % 16)
    return fail(DG_ERR_INVALID_ARG, "dg_fp8_quantize_blocks: pitches %lld of w, %lld of the codes (a multiple of 16)",
                (long long)ldw, (long long)ldq);
  if (groups == 0) return DG_OK;
  if (!d_w || !d_q || !d_scale) return fail(DG_ERR_INVALID_ARG, "dg_fp8_quantize_blocks: null pointer");
  const size_t sz = dtype_bytes(dtype);
  if (!aligned(d_w, sz) || !aligned(d_q, 16) || !aligned(d_scale, 4))
    return fail(DG_ERR_INVALID_ARG, "dg_fp8_quantize_blocks: misaligned pointer (codes: 16 bytes)");
  QuantBlocksParams p{};
  p.w = d_w; p.ldw = ldw; p.q = d_q; p.ldq = ldq; p.scale = d_scale;
  p.N = (int)rows; p.K = (int)cols;
  p.NB = (int)ceil_div(rows, kFp8Block); p.KB = (int)ceil_div(cols, kFp8Block);
  const double blocks_d = (double)groups * p.NB * p.KB;
  if (blocks_d > (double)kMaxDim) return fail(DG_ERR_INVALID_ARG, "dg_fp8_quantize_blocks: too many blocks");
  const long long blocks = (long long)groups * p.NB * p.KB;
  const bool vec = cols % 8 == 0 && aligned(d_w, 16) && (ldw * (long long)sz) % 16 == 0;
  cudaStream_t st = (cudaStream_t)stream;
  switch (dtype) {
    case DG_BF16: return launch_quant_blocks<__nv_bfloat16>(p, blocks, vec, st);
    case DG_F16: return launch_quant_blocks<__half>(p, blocks, vec, st);
    default: return launch_quant_blocks<float>(p, blocks, vec, st);
  }
}

extern "C" dg_status dg_fp8_gemm(const uint8_t* d_a, int64_t lda, const float* d_a_scale, int64_t lds,
                                 const uint8_t* d_b, int64_t ldb, const float* d_b_scale, int64_t M, int64_t N, int64_t K,
                                 const float* d_row_weight, void* d_out, int32_t out_dtype, int64_t ldo, void* stream) {
  Fp8GemmParams p;
  DG_TRY(check_product("dg_fp8_gemm", d_a, lda, d_a_scale, lds, d_b, ldb, d_b_scale, nullptr, 1, M, N, K, d_row_weight,
                       d_out, out_dtype, ldo, &p));
  if (M == 0) return DG_OK;
  return product("dg_fp8_gemm", p, out_dtype, nullptr, (cudaStream_t)stream);
}

dg_status dg::fp8_grouped_gemm(const uint8_t* d_a, int64_t lda, const float* d_a_scale, int64_t lds, const uint8_t* d_b,
                               int64_t ldb, const float* d_b_scale, const int32_t* d_off, int64_t groups, int64_t M,
                               int64_t N, int64_t K, const float* d_row_weight, void* d_out, int32_t out_dtype,
                               int64_t ldo, int* err, cudaStream_t st) {
  Fp8GemmParams p;
  if (!d_off) return fail(DG_ERR_INVALID_ARG, "dg_fp8_grouped_gemm: null offsets");
  DG_TRY(check_product("dg_fp8_grouped_gemm", d_a, lda, d_a_scale, lds, d_b, ldb, d_b_scale, d_off, groups, M, N, K,
                       d_row_weight, d_out, out_dtype, ldo, &p));
  if (M == 0) return DG_OK;
  return product("dg_fp8_grouped_gemm", p, out_dtype, err, st);
}

extern "C" dg_status dg_fp8_grouped_gemm(const uint8_t* d_a, int64_t lda, const float* d_a_scale, int64_t lds,
                                         const uint8_t* d_b, int64_t ldb, const float* d_b_scale, const int32_t* d_off,
                                         int64_t groups, int64_t M, int64_t N, int64_t K, const float* d_row_weight,
                                         void* d_out, int32_t out_dtype, int64_t ldo, void* stream) {
  return fp8_grouped_gemm(d_a, lda, d_a_scale, lds, d_b, ldb, d_b_scale, d_off, groups, M, N, K, d_row_weight, d_out,
                          out_dtype, ldo, nullptr, (cudaStream_t)stream);
}

extern "C" dg_status dg_test_fp8_hold(int32_t what, int32_t unit, int32_t block, int64_t limit_ns) {
  if (what < kHoldNothing || what > kHoldScales || unit < 0 || block < 0 || limit_ns < 0 || limit_ns > 5000000000ll)
    return fail(DG_ERR_INVALID_ARG, "dg_test_fp8_hold: bad arguments (a limit is at most 5 s)");
  g_waits = kUsualWaits;
  if (what != kHoldNothing)
    g_waits = Fp8Waits{limit_ns ? (unsigned long long)limit_ns : kWaitLimitNs, nullptr, what, unit, block};
  return DG_OK;
}
