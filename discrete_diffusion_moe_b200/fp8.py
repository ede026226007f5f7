"""Tensor-level calls of the 8-bit block-scaled operators (include/dg.h:
dg_fp8_quantize, dg_fp8_quantize_blocks, dg_fp8_gemm, dg_fp8_grouped_gemm).

Activations are a pair (codes [rows, K] float8_e4m3fn, scale
[ceil(K / 128), rows] float32), weights a pair (codes [N, K] or [G, N, K],
scale [(G,) ceil(N / 128), ceil(K / 128)]); a value is code * scale.  Rows of
codes start every multiple of 16 bytes, so for other K the codes are a view
of a wider buffer.  Tensors are on one CUDA device, which need not be the
current one; work goes to `stream` (the device's current stream by default).
That the inputs are ready on a given stream is the caller's part; that their
memory is not given away before the work has ended is seen to here.
Wrong shapes, types or strides raise ValueError, what the library itself
refuses raises DgError; nothing is launched then.  No gradients flow through
these calls."""

import torch

from . import DG_ACT_NONE, DG_ACT_SWIGLU, DG_ACT_SWIGLU_INTERLEAVED, DG_BF16, DG_F16, DG_F32, check, lib

_DTYPE = {torch.bfloat16: DG_BF16, torch.float16: DG_F16, torch.float32: DG_F32}
_ACT = {None: DG_ACT_NONE, "swiglu": DG_ACT_SWIGLU, "swiglu_interleaved": DG_ACT_SWIGLU_INTERLEAVED}
_E4M3 = torch.float8_e4m3fn


def _fail(what):
    raise ValueError(what)


def _blocks(n):
    return (n + 127) >> 7


def _launch(fn, device, stream, args, tensors):
    """One library call on `device` and `stream` (its current one for None),
    which the memory of `tensors` (None among them) outlives.  These calls take
    a few microseconds on the GPU, so the host side keeps to plain integers:
    the raw stream and the current device's number."""
    index = device.index
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(index)
    else:
        stream.device == device or _fail("the stream is on another device than the tensors")
        raw = stream.cuda_stream
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
    if torch._C._cuda_getDevice() == index:
        status = fn(*args, raw)
    else:
        with torch.cuda.device(device):
            status = fn(*args, raw)
    if status:
        check(status)


def _empty(shape, dtype, device, stream):
    """An output buffer owned by the stream that writes it (sizes one by one:
    torch takes 0.7 us longer over a tuple)."""
    if stream is None:
        return torch.empty(*shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(*shape, dtype=dtype, device=device)


def _new_codes(shape, device, stream):
    K = shape[-1]
    if K & 15 == 0:
        return _empty(shape, _E4M3, device, stream)
    return _empty((*shape[:-1], (K + 15) & ~15), _E4M3, device, stream)[..., :K]


def _check_codes(name, t, dim):
    if t.dtype is not _E4M3 or not t.is_cuda or t.dim() != dim:
        _fail(f"{name}: a {dim}-D float8_e4m3fn CUDA tensor is needed")
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        _fail(f"{name}: the columns must be contiguous")


def _row_scale_pitch(name, s, device, rows, blocks):
    """Elements between the blocks of a [blocks, rows] tensor of row scales."""
    if s.dtype is not torch.float32 or s.shape != (blocks, rows):
        _fail(f"{name}: float32 [{blocks}, {rows}] is needed, got {s.dtype} {list(s.shape)}")
    if s.device != device:
        _fail("tensors on different devices")
    pitch, inner = s.stride()
    if inner != 1 and rows > 1:
        _fail(f"{name}: each block's row scales must be contiguous")
    return pitch if blocks > 1 else rows


def _check_vector(name, t, device, dtype, n):
    if t.dtype is not dtype or t.shape != (n,) or not t.is_contiguous():
        _fail(f"{name}: contiguous {dtype} [{n}] is needed")
    if t.device != device:
        _fail("tensors on different devices")


def fp8_quantize(x, index=None, act=None, out=None, stream=None):
    """Quantise rows of x [x_rows, K] (bf16, fp16 or fp32; [x_rows, 2 K] with
    act = "swiglu", gate columns then up columns, or "swiglu_interleaved") to
    (codes [rows, K], scale [ceil(K / 128), rows]).  index (int32 [rows]):
    output row r takes row index[r] of x; indices outside x read as zeros.
    out: an earlier result to write into."""
    dtype = _DTYPE.get(x.dtype)
    if dtype is None or not x.is_cuda or x.dim() != 2:
        _fail("x: a 2-D bf16, fp16 or fp32 CUDA tensor is needed")
    if act not in _ACT:
        _fail(f"act: None, 'swiglu' or 'swiglu_interleaved', got {act!r}")
    device = x.device
    x_rows, cols = x.shape
    ldx, inner = x.stride()
    if inner != 1 and cols > 1:
        _fail("x: the columns must be contiguous")
    if cols < 1 or (act is not None and cols & 1):
        _fail("x: at least one column, and an even number of them for SwiGLU, is needed")
    K = cols if act is None else cols >> 1
    rows, index_ptr = x_rows, None
    if index is not None:
        if index.dim() != 1:
            _fail("index: a 1-D tensor is needed")
        rows = index.shape[0]
        _check_vector("index", index, device, torch.int32, rows)
        index_ptr = index.data_ptr()
    KB = (K + 127) >> 7
    if out is None:
        q, scale, lds = _new_codes((rows, K), device, stream), _empty((KB, rows), torch.float32, device, stream), rows
    else:
        q, scale = out
        _check_codes("out[0]", q, 2)
        if q.shape != (rows, K) or q.device != device:
            _fail(f"out[0]: [{rows}, {K}] on x's device is needed")
        lds = _row_scale_pitch("out[1]", scale, device, rows, KB)
    _launch(lib.dg_fp8_quantize, device, stream,
            (x.data_ptr(), dtype, ldx if x_rows > 1 else cols, x_rows, index_ptr, _ACT[act], rows, K, q.data_ptr(),
             q.stride(0) if rows > 1 else (K + 15) & ~15, scale.data_ptr(), lds), (x, index, q, scale))
    return q, scale


def _weight_pitch(name, t):
    """Elements between the rows of a [N, K] or [G, N, K] tensor (None: any)."""
    if t.dim() == 2:
        return t.stride(0) if t.shape[0] > 1 else None
    G, N = t.shape[:2]
    if N == 1:
        return t.stride(0) if G > 1 else None
    pitch = t.stride(1)
    if G > 1 and t.stride(0) != N * pitch:
        _fail(f"{name}: the matrices must follow one another")
    return pitch


def fp8_quantize_blocks(w, out=None, stream=None):
    """Quantise weights w [N, K] or [G, N, K] (bf16, fp16 or fp32) to (codes of
    the same shape, scale [(G,) ceil(N / 128), ceil(K / 128)])."""
    dtype = _DTYPE.get(w.dtype)
    if dtype is None or not w.is_cuda or w.dim() not in (2, 3):
        _fail("w: a 2-D or 3-D bf16, fp16 or fp32 CUDA tensor is needed")
    G, N, K = w.shape if w.dim() == 3 else (1, *w.shape)
    if N < 1 or K < 1:
        _fail("w: at least one row and one column are needed")
    if w.stride(-1) != 1 and K > 1:
        _fail("w: the columns must be contiguous")
    shape = (*w.shape[:-2], _blocks(N), _blocks(K))
    if out is None:
        q, scale = _new_codes(tuple(w.shape), w.device, stream), _empty(shape, torch.float32, w.device, stream)
    else:
        q, scale = out
        _check_codes("out[0]", q, w.dim())
        if q.shape != w.shape or q.device != w.device:
            _fail("out[0]: the shape and device of w are needed")
        if scale.dtype != torch.float32 or scale.shape != shape or not scale.is_contiguous() or scale.device != w.device:
            _fail(f"out[1]: contiguous float32 {list(shape)} on w's device is needed")
    ldw, ldq = _weight_pitch("w", w), _weight_pitch("out[0]", q)
    _launch(lib.dg_fp8_quantize_blocks, w.device, stream,
            (w.data_ptr(), dtype, K if ldw is None else ldw, G, N, K, q.data_ptr(),
             (K + 15) & ~15 if ldq is None else ldq, scale.data_ptr()), (w, q, scale))
    return q, scale


def _product(a, a_scale, b, b_scale, off, row_weight, out_dtype, out, stream):
    _check_codes("a", a, 2)
    _check_codes("b", b, 2 if off is None else 3)
    device = a.device
    M, K = a.shape
    KB, k16 = (K + 127) >> 7, (K + 15) & ~15
    N, k_b = b.shape[-2:]
    if k_b != K:
        _fail(f"a has {K} columns, b {k_b}")
    lds = _row_scale_pitch("a_scale", a_scale, device, M, KB)
    shape = ((N + 127) >> 7, KB) if off is None else (b.shape[0], (N + 127) >> 7, KB)
    if b_scale.dtype is not torch.float32 or b_scale.shape != shape or not b_scale.is_contiguous():
        _fail(f"b_scale: contiguous float32 {list(shape)} is needed")
    if b.device != device or b_scale.device != device:
        _fail("tensors on different devices")
    weight_ptr = None
    if row_weight is not None:
        _check_vector("row_weight", row_weight, device, torch.float32, M)
        weight_ptr = row_weight.data_ptr()
    if out is None:
        dtype = _DTYPE.get(out_dtype)
        if dtype is None:
            _fail(f"out_dtype: bf16, fp16 or fp32, got {out_dtype}")
        out, ldo = _empty((M, N), out_dtype, device, stream), N
    else:
        dtype = _DTYPE.get(out.dtype)
        if dtype is None or out.shape != (M, N) or out.device != device or (out.stride(1) != 1 and N > 1):
            _fail(f"out: bf16, fp16 or fp32 [{M}, {N}] with contiguous columns on a's device is needed")
        ldo = out.stride(0) if M > 1 else N
    ldb = _weight_pitch("b", b)
    lda = a.stride(0) if M > 1 else k16
    if ldb is None:
        ldb = k16
    if off is None:
        _launch(lib.dg_fp8_gemm, device, stream,
                (a.data_ptr(), lda, a_scale.data_ptr(), lds, b.data_ptr(), ldb, b_scale.data_ptr(), M, N, K, weight_ptr,
                 out.data_ptr(), dtype, ldo), (a, a_scale, b, b_scale, row_weight, out))
    else:
        G = shape[0]
        _check_vector("off", off, device, torch.int32, G + 1)
        _launch(lib.dg_fp8_grouped_gemm, device, stream,
                (a.data_ptr(), lda, a_scale.data_ptr(), lds, b.data_ptr(), ldb, b_scale.data_ptr(), off.data_ptr(), G, M, N,
                 K, weight_ptr, out.data_ptr(), dtype, ldo), (a, a_scale, b, b_scale, off, row_weight, out))
    return out


def fp8_gemm(a, a_scale, b, b_scale, row_weight=None, out_dtype=torch.bfloat16, out=None, stream=None):
    """out [M, N] = (a a_scale) (b b_scale)^T for activations (a, a_scale) [M, K]
    and weights (b, b_scale) [N, K]; fp32 sums, rounded once to out_dtype (the
    type of `out` when that is given).  row_weight (float32 [M]) multiplies
    the rows."""
    return _product(a, a_scale, b, b_scale, None, row_weight, out_dtype, out, stream)


def fp8_grouped_gemm(a, a_scale, b, b_scale, off, row_weight=None, out_dtype=torch.bfloat16, out=None, stream=None):
    """fp8_gemm with the rows split among the G matrices of b [G, N, K]: rows
    [off[g], off[g + 1]) take matrix g (off: int32 [G + 1], non-decreasing).
    Rows outside [off[0], off[G]) are not written: they keep what `out` holds,
    and are undefined when `out` is not given."""
    off is not None or _fail("off is needed")
    return _product(a, a_scale, b, b_scale, off, row_weight, out_dtype, out, stream)
