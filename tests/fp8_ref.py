"""Plain 64-bit forms of the 8-bit block-scaled operators, their inputs and
error bounds (numpy and torch on the CPU; no code shared with the library)."""

import numpy as np
import torch

BLOCK = 128
E4M3_MAX = 448.0
AMAX_MIN = 2.0 ** -100

# every e4m3 code's value (0x7f and 0xff are NaN)
_CODES = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
_POS = _CODES[:127]  # 0 .. 448, ascending


def blocks(n):
    return (n + BLOCK - 1) // BLOCK


def e4m3(v):
    """Values of v (float64, |v| <= 448) rounded to e4m3, ties to the even code."""
    a = np.abs(v)
    hi = np.clip(np.searchsorted(_POS, a, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = _POS[hi] - a, a - _POS[lo]
    pick = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return np.copysign(_POS[pick], v)


def quantize_block(x, amax):
    """Codes' values and scale of one block: 448 / a and the product are held
    in 32 bits (a quotient of two fp32 values computed in 64 bits and rounded
    to 32 is the correctly rounded one)."""
    if not np.isfinite(amax):
        return np.zeros_like(x), np.float32(np.nan)
    a = np.float64(max(amax, AMAX_MIN))
    inv = np.float64(np.float32(E4M3_MAX / a))
    v = (x * inv).astype(np.float32).astype(np.float64)
    return e4m3(np.clip(v, -E4M3_MAX, E4M3_MAX)), np.float32(a / E4M3_MAX)


def quantize_rows(x):
    rows, K = x.shape
    q, s = np.zeros((rows, K)), np.zeros((blocks(K), rows), dtype=np.float32)
    for r in range(rows):
        for kb in range(blocks(K)):
            part = x[r, kb * BLOCK:(kb + 1) * BLOCK]
            amax = np.abs(part).max() if np.isfinite(part).all() else np.inf
            q[r, kb * BLOCK:(kb + 1) * BLOCK], s[kb, r] = quantize_block(part, amax)
    return q, s


def quantize_blocks(w):
    N, K = w.shape
    q, s = np.zeros((N, K)), np.zeros((blocks(N), blocks(K)), dtype=np.float32)
    for nb in range(blocks(N)):
        for kb in range(blocks(K)):
            sl = (slice(nb * BLOCK, (nb + 1) * BLOCK), slice(kb * BLOCK, (kb + 1) * BLOCK))
            part = w[sl]
            amax = np.abs(part).max() if np.isfinite(part).all() else np.inf
            q[sl], s[nb, kb] = quantize_block(part, amax)
    return q, s


def swiglu(g, u):
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u


# ---- products ------------------------------------------------------------------

def dequantize_rows(q, s):
    """[rows, K] float64 from codes and scales [KB, rows] (tensors)."""
    return q.double().cpu().numpy() * np.repeat(s.double().cpu().numpy().T, BLOCK, axis=1)[:, :q.shape[1]]


def dequantize_blocks(q, s):
    v = s.double().cpu().numpy()
    v = np.repeat(np.repeat(v, BLOCK, axis=-2), BLOCK, axis=-1)
    return q.double().cpu().numpy() * v[..., :q.shape[-2], :q.shape[-1]]


def product(a, b):
    """(a b^T, |a| |b|^T) in 64 bits."""
    return a @ b.T, np.abs(a) @ np.abs(b).T


def product_bound(want, want_abs, K, out_dtype, weighted=False):
    """Per-element bound of the kernels' error.
      - The products of two e4m3 codes (8 significant bits) are exact in fp32.
        A block's 128 of them are added in fp32 in the tensor cores' own order,
        each addition off by at most one unit in the last place (2^-23, which
        covers truncation) of a partial sum no larger than the sum of |a b|:
        127 * 2^-23 of it.
      - The block sum is multiplied by sa * sb (rounded: 2^-24) and added to the
        running fp32 sum over the blocks (2^-24 each for the fused product or
        the addition, then at most 8 partial sums of a split K): (KB + 9) 2^-24.
      - The row weight: 2^-24 more.
      - The output's rounding: half a step, eps / 2 of the value (fp16
        subnormals: 2^-25 absolute)."""
    kb = blocks(K)
    f32 = (127 * 2.0 ** -23 + (kb + 10 + int(weighted)) * 2.0 ** -24) * want_abs
    half = torch.finfo(out_dtype).eps / 2 if out_dtype != torch.float32 else 0.0
    tiny = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -149}[out_dtype]
    return f32 + half * (np.abs(want) + f32) + tiny


# ---- inputs ---------------------------------------------------------------------

def padded_codes(values, pitch=None, fill=0x7F):
    """e4m3 tensor (device) of `values` [..., K] whose rows are `pitch` bytes
    apart; the bytes behind column K hold `fill` (a NaN code)."""
    K = values.shape[-1]
    pitch = pitch or (K + 15) // 16 * 16
    buf = torch.full((*values.shape[:-1], pitch), fill, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    buf[..., :K] = torch.as_tensor(values, dtype=torch.float32).to(torch.float8_e4m3fn).cuda()
    return buf[..., :K]


def random_operand(rng, rows, K, pitch=None):
    """Random codes over the whole e4m3 range and uneven row scales."""
    v = _CODES[rng.integers(0, 127, (rows, K)) + 128 * rng.integers(0, 2, (rows, K))]
    s = torch.from_numpy(np.exp(rng.uniform(-6, 2, (blocks(K), rows))).astype(np.float32)).cuda()
    return padded_codes(v, pitch), s


def random_weights(rng, N, K, G=None, pitch=None):
    shape = (N, K) if G is None else (G, N, K)
    v = _CODES[rng.integers(0, 127, shape) + 128 * rng.integers(0, 2, shape)]
    sshape = (blocks(N), blocks(K)) if G is None else (G, blocks(N), blocks(K))
    return padded_codes(v, pitch), torch.from_numpy(np.exp(rng.uniform(-6, 2, sshape)).astype(np.float32)).cuda()
