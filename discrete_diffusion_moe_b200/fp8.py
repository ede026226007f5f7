"""Tensor-level calls of the 8-bit block-scaled operators (include/dg.h:
dg_fp8_quantize, dg_fp8_quantize_blocks, dg_fp8_gemm, dg_fp8_grouped_gemm).

Activations are a pair (codes [rows, K] float8_e4m3fn, scale
[ceil(K / 128), rows] float32), weights a pair (codes [N, K] or [G, N, K],
scale [(G,) ceil(N / 128), ceil(K / 128)]); a value is code * scale.  Rows of
codes start every multiple of 16 bytes, so for other K the codes are a view
of a wider buffer.  Tensors are on one CUDA device, which need not be the
current one; work goes to `stream` (the device's current stream by default).
Wrong shapes, types or strides raise ValueError, what the library itself
refuses raises DgError; nothing is launched then."""

import ctypes

import torch

from . import DG_ACT_NONE, DG_ACT_SWIGLU, DG_ACT_SWIGLU_INTERLEAVED, DG_BF16, DG_F16, DG_F32, check, lib

_DTYPE = {torch.bfloat16: DG_BF16, torch.float16: DG_F16, torch.float32: DG_F32}
_ACT = {None: DG_ACT_NONE, "swiglu": DG_ACT_SWIGLU, "swiglu_interleaved": DG_ACT_SWIGLU_INTERLEAVED}
_E4M3 = torch.float8_e4m3fn


def _require(ok, what):
    if not ok:
        raise ValueError(what)


def _blocks(n):
    return (n + 127) // 128


def _pitch(t, least):
    """Elements between rows of a 2-D tensor (any value will do for one row)."""
    return t.stride(0) if t.shape[0] > 1 else least


def _on(device, *tensors):
    for t in tensors:
        _require(t is None or t.device == device, "tensors on different devices")


def _launch(fn, device, stream, *args):
    """One library call on `device` and `stream`."""
    s = stream if stream is not None else torch.cuda.current_stream(device)
    _require(s.device == device, "the stream is on another device than the tensors")
    if torch.cuda.current_device() == device.index:
        check(fn(*args, s.cuda_stream))
    else:
        with torch.cuda.device(device):
            check(fn(*args, s.cuda_stream))


def _empty(shape, dtype, device, stream):
    """An output buffer owned by the stream that writes it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _new_codes(shape, device, stream):
    K = shape[-1]
    pitch = (K + 15) // 16 * 16
    q = _empty((*shape[:-1], pitch), _E4M3, device, stream)
    return q if pitch == K else q[..., :K]


def _check_codes(name, t, dim):
    _require(t.dtype == _E4M3 and t.is_cuda and t.dim() == dim, f"{name}: a {dim}-D float8_e4m3fn CUDA tensor is needed")
    _require(t.shape[-1] <= 1 or t.stride(-1) == 1, f"{name}: the columns must be contiguous")


def _check_row_scale(name, s, rows, K):
    _require(s.dtype == torch.float32 and s.dim() == 2 and tuple(s.shape) == (_blocks(K), rows),
             f"{name}: float32 [{_blocks(K)}, {rows}] is needed, got {s.dtype} {list(s.shape)}")
    _require(rows <= 1 or s.stride(1) == 1, f"{name}: each block's row scales must be contiguous")


def fp8_quantize(x, index=None, act=None, out=None, stream=None):
    """Quantise rows of x [x_rows, K] (bf16, fp16 or fp32; [x_rows, 2 K] with
    act = "swiglu", gate columns then up columns, or "swiglu_interleaved") to
    (codes [rows, K], scale [ceil(K / 128), rows]).  index (int32 [rows]):
    output row r takes row index[r] of x; indices outside x read as zeros.
    out: an earlier result to write into."""
    _require(x.is_cuda and x.dim() == 2 and x.dtype in _DTYPE, "x: a 2-D bf16, fp16 or fp32 CUDA tensor is needed")
    _require(act in _ACT, f"act: None, 'swiglu' or 'swiglu_interleaved', got {act!r}")
    _require(x.shape[1] <= 1 or x.stride(1) == 1, "x: the columns must be contiguous")
    K = x.shape[1]
    if act is not None:
        _require(K % 2 == 0, "x: an even number of columns is needed for SwiGLU")
        K //= 2
    _require(K >= 1, "x: at least one column is needed")
    rows = x.shape[0]
    if index is not None:
        _require(index.dtype == torch.int32 and index.dim() == 1 and index.is_contiguous(),
                 "index: a contiguous 1-D int32 tensor is needed")
        rows = index.shape[0]
    if out is None:
        q, scale = _new_codes((rows, K), x.device, stream), _empty((_blocks(K), rows), torch.float32, x.device, stream)
    else:
        q, scale = out
        _check_codes("out[0]", q, 2)
        _require(tuple(q.shape) == (rows, K), f"out[0]: [{rows}, {K}] is needed")
        _check_row_scale("out[1]", scale, rows, K)
    _on(x.device, index, q, scale)
    _launch(lib.dg_fp8_quantize, x.device, stream, x.data_ptr(), _DTYPE[x.dtype], _pitch(x, x.shape[1]), x.shape[0],
            index.data_ptr() if index is not None else None, _ACT[act], rows, K, q.data_ptr(),
            _pitch(q, (K + 15) // 16 * 16), scale.data_ptr(), max(scale.stride(0), rows))
    return q, scale


def _weight_pitch(name, t):
    """Elements between the rows of a [N, K] or [G, N, K] tensor."""
    G, N, K = t.shape if t.dim() == 3 else (1, *t.shape)
    _require(K <= 1 or t.stride(-1) == 1, f"{name}: the columns must be contiguous")
    if N > 1:
        pitch = t.stride(-2)
        _require(G <= 1 or t.stride(0) == N * pitch, f"{name}: the matrices must follow one another")
        return pitch
    return t.stride(0) if G > 1 else None


def fp8_quantize_blocks(w, out=None, stream=None):
    """Quantise weights w [N, K] or [G, N, K] (bf16, fp16 or fp32) to (codes of
    the same shape, scale [(G,) ceil(N / 128), ceil(K / 128)])."""
    _require(w.is_cuda and w.dim() in (2, 3) and w.dtype in _DTYPE,
             "w: a 2-D or 3-D bf16, fp16 or fp32 CUDA tensor is needed")
    G, N, K = w.shape if w.dim() == 3 else (1, *w.shape)
    _require(N >= 1 and K >= 1, "w: at least one row and one column are needed")
    shape = (*w.shape[:-2], _blocks(N), _blocks(K))
    if out is None:
        q, scale = _new_codes(tuple(w.shape), w.device, stream), _empty(shape, torch.float32, w.device, stream)
    else:
        q, scale = out
        _check_codes("out[0]", q, w.dim())
        _require(q.shape == w.shape, "out[0]: the shape of w is needed")
        _require(scale.dtype == torch.float32 and tuple(scale.shape) == shape and scale.is_contiguous(),
                 f"out[1]: contiguous float32 {list(shape)} is needed")
    _on(w.device, q, scale)
    ldw, ldq = _weight_pitch("w", w), _weight_pitch("out[0]", q)
    _launch(lib.dg_fp8_quantize_blocks, w.device, stream, w.data_ptr(), _DTYPE[w.dtype], K if ldw is None else ldw, G, N,
            K, q.data_ptr(), (K + 15) // 16 * 16 if ldq is None else ldq, scale.data_ptr())
    return q, scale


def _product(a, a_scale, b, b_scale, off, row_weight, out_dtype, out, stream):
    grouped = off is not None
    _check_codes("a", a, 2)
    _check_codes("b", b, 3 if grouped else 2)
    M, K = a.shape
    N = b.shape[-2]
    G = b.shape[0] if grouped else 1
    _require(b.shape[-1] == K, f"a has {K} columns, b {b.shape[-1]}")
    _check_row_scale("a_scale", a_scale, M, K)
    shape = (G, _blocks(N), _blocks(K)) if grouped else (_blocks(N), _blocks(K))
    _require(b_scale.dtype == torch.float32 and tuple(b_scale.shape) == shape and b_scale.is_contiguous(),
             f"b_scale: contiguous float32 {list(shape)} is needed")
    if grouped:
        _require(off.dtype == torch.int32 and off.dim() == 1 and off.shape[0] == G + 1 and off.is_contiguous(),
                 f"off: contiguous int32 [{G + 1}] is needed")
    if row_weight is not None:
        _require(row_weight.dtype == torch.float32 and tuple(row_weight.shape) == (M,) and row_weight.is_contiguous(),
                 f"row_weight: contiguous float32 [{M}] is needed")
    if out is None:
        _require(out_dtype in _DTYPE, f"out_dtype: bf16, fp16 or fp32, got {out_dtype}")
        out = _empty((M, N), out_dtype, a.device, stream)
    else:
        _require(out.dtype in _DTYPE and tuple(out.shape) == (M, N) and (N <= 1 or out.stride(1) == 1),
                 f"out: bf16, fp16 or fp32 [{M}, {N}] with contiguous columns is needed")
    _on(a.device, a_scale, b, b_scale, off, row_weight, out)
    k16 = (K + 15) // 16 * 16
    ldb = _weight_pitch("b", b)
    head = (a.data_ptr(), _pitch(a, k16), a_scale.data_ptr(), max(a_scale.stride(0), M), b.data_ptr(),
            k16 if ldb is None else ldb, b_scale.data_ptr())
    tail = (M, N, K, row_weight.data_ptr() if row_weight is not None else None, out.data_ptr(), _DTYPE[out.dtype],
            _pitch(out, N))
    if grouped:
        _launch(lib.dg_fp8_grouped_gemm, a.device, stream, *head, off.data_ptr(), G, *tail)
    else:
        _launch(lib.dg_fp8_gemm, a.device, stream, *head, *tail)
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
    _require(off is not None, "off is needed")
    return _product(a, a_scale, b, b_scale, off, row_weight, out_dtype, out, stream)
