"""The 8-bit block-scaled operators on the GPU against plain 64-bit forms:
quantisers bit for bit, products within bounds derived from their roundings
(fp8_ref.product_bound), masks, strides, streams and graphs."""

import numpy as np
import pytest
import torch

import fp8_ref as ref

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16, torch.float32]


def _dg():
    import discrete_diffusion_moe_b200 as dg
    return dg


def _hidden(rng, rows, K, dtype):
    x = rng.standard_normal((rows, K)) * np.exp(rng.uniform(-3, 3, (rows, 1)))
    return torch.from_numpy(x.astype(np.float32)).to(dtype)


def _same_codes(q, want):
    got = q.double().cpu().numpy()
    assert got.shape == want.shape
    bad = np.flatnonzero((got != want).ravel())
    assert bad.size == 0, (bad[:5], got.ravel()[bad[:5]], want.ravel()[bad[:5]])


def _same_scales(s, want):
    got = s.cpu().numpy()
    assert np.array_equal(got, want, equal_nan=True), np.flatnonzero((got != want).ravel())[:5]


# ---- quantisers -------------------------------------------------------------------

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,K", [(1, 1), (1, 16), (3, 127), (2, 128), (5, 129), (1, 2816), (7, 2816), (33, 704),
                                    (64, 1000), (129, 257)])
def test_quantize_rows(rows, K, dtype):
    dg = _dg()
    x = _hidden(np.random.default_rng(rows * 7 + K), rows, K, dtype)
    q, s = dg.fp8_quantize(x.cuda())
    want_q, want_s = ref.quantize_rows(x.double().numpy())
    _same_codes(q, want_q)
    _same_scales(s, want_s)


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_rows_special_values(dtype):
    """Zero blocks, the smallest and largest values, a NaN and infinities."""
    dg = _dg()
    x = _hidden(np.random.default_rng(3), 9, 300, dtype)
    fi = torch.finfo(dtype)
    x[0] = 0.0
    x[1, :128] = 0.0
    x[2] = fi.smallest_normal
    x[3] = fi.max
    x[4, 5] = float("nan")
    x[5, 130] = float("inf")
    x[6, 299] = -float("inf")
    x[7] = -0.0
    x[8, 1:] = fi.tiny * fi.eps   # the smallest subnormal
    q, s = dg.fp8_quantize(x.cuda())
    want_q, want_s = ref.quantize_rows(x.double().numpy())
    _same_codes(q, want_q)
    _same_scales(s, want_s)
    assert np.isnan(want_s).sum() == 3


@pytest.mark.parametrize("K", [704, 130, 99])
def test_quantize_gathered_rows(K):
    """Rows taken by index, the same index twice; indices outside x give zeros."""
    dg = _dg()
    rng = np.random.default_rng(K)
    x = _hidden(rng, 40, K, torch.bfloat16)
    index = torch.from_numpy(rng.integers(0, 40, 77).astype(np.int32))
    index[3], index[9], index[20] = -1, 40, 2 ** 31 - 1
    q, s = dg.fp8_quantize(x.cuda(), index=index.cuda())
    src = torch.zeros(77, K, dtype=torch.bfloat16)
    inside = (index >= 0) & (index < 40)
    src[inside] = x[index[inside].long()]
    want_q, want_s = ref.quantize_rows(src.double().numpy())
    _same_codes(q, want_q)
    _same_scales(s, want_s)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ["swiglu", "swiglu_interleaved"])
@pytest.mark.parametrize("rows,K", [(1, 704), (9, 704), (33, 129), (4, 1), (17, 1000)])
def test_quantize_swiglu(rows, K, act, dtype):
    dg = _dg()
    rng = np.random.default_rng(rows + K)
    y = torch.from_numpy((4 * rng.standard_normal((rows, 2 * K))).astype(np.float32)).to(dtype)
    y[0, :] *= 10.0   # gates far into silu's limits
    q, s = dg.fp8_quantize(y.cuda(), act=act)
    d = y.double().numpy()
    g, u = (d[:, :K], d[:, K:]) if act == "swiglu" else (d[:, 0::2], d[:, 1::2])
    v = ref.swiglu(g, u)
    # e^-g: 2 units plus the rounding of g log2(e) (|g| 2^-24 of e^-g each way),
    # the sum, the quotient (2 units) and the product with u: (7 + 2 |g|) 2^-24
    # for positive g; for negative g the denominator is e^-g itself: the same
    rel = (8 + 2 * np.abs(g)) * 2.0 ** -23
    got_s = s.double().cpu().numpy()
    for kb in range(ref.blocks(K)):
        sl = slice(kb * 128, min(K, kb * 128 + 128))
        amax = np.maximum(np.abs(v[:, sl]).max(1), ref.AMAX_MIN)
        assert np.all(np.abs(got_s[kb] - amax / 448) <= (rel[:, sl].max(1) + 2.0 ** -23) * amax / 448)
    got = ref.dequantize_rows(q, s)
    step = np.repeat(got_s.T, 128, axis=1)[:, :K]
    # half a step of a normal code is 2^-4 of the value, of a subnormal one 2^-10;
    # the largest values may be held to 448: off by the scale's own error
    bound = (2.0 ** -4 + 2 * rel + 2.0 ** -20) * np.abs(v) + 2.0 ** -10 * step
    assert np.all(np.abs(got - v) <= bound), float((np.abs(got - v) / bound).max())


@pytest.mark.parametrize("act", ["swiglu", "swiglu_interleaved"])
def test_quantize_swiglu_is_as_exact_as_fp32_allows(act):
    """One element per block, so that its scale is the element's own magnitude
    over 448: gates over silu's whole range, the far negative ones (e^-g above
    2^126) too.  Relative error of fp32 steps: e^-|g| 2 units of 2^-23, the
    product with it, the sum and the product with u half a unit each, the
    quotient one, the scale's own quotient half a unit: 5 units.  Below g = -87.3
    e^-|g| is subnormal, off by up to 2 of its steps of 2^-149."""
    dg = _dg()
    rng = np.random.default_rng(21)
    g = np.concatenate([np.linspace(-88.6, -87.0, 33), rng.uniform(-90, 90, 4000), rng.uniform(-1, 1, 500)])
    u = np.exp(rng.uniform(5, 20, g.size)) * np.where(g < -30, 2.0 ** 60, 1.0)
    x = torch.from_numpy(np.stack((g, u), 1).astype(np.float32))
    q, s = dg.fp8_quantize(x.cuda(), act=act)   # K = 1: both orders are (gate, up)
    gd, ud = x.double().numpy().T
    v = np.abs(ref.swiglu(gd, ud))
    assert v.min() > ref.AMAX_MIN
    rel = 5 * 2.0 ** -23 + np.where(gd < -87.3, 2 * 2.0 ** -149 * np.exp(np.abs(gd)), 0.0)
    err = np.abs(s[0].double().cpu().numpy() * 448 / v - 1)
    assert np.all(err <= rel), float((err / rel).max())
    assert np.array_equal(q.double().cpu().numpy()[:, 0], 448 * np.sign(gd))


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_swiglu_of_the_largest_gates(dtype):
    """Gates of the type's largest magnitude with small factors: silu is the gate itself, or
    0 for negative ones (a block of zeros has the smallest scale).  The scale is within 5
    units of 2^-23."""
    dg = _dg()
    big = torch.finfo(dtype).max
    x = torch.tensor([[big, 2.0 ** -20], [-big, 2.0 ** -20], [big / 2, -2.0 ** -14]], dtype=dtype)
    q, s = dg.fp8_quantize(x.cuda(), act="swiglu")
    d = x.double().numpy()
    want = np.maximum(np.abs(np.where(d[:, 0] > 0, d[:, 0], 0.0) * d[:, 1]), ref.AMAX_MIN) / 448
    assert np.all(np.abs(s[0].double().cpu().numpy() / want - 1) <= 5 * 2.0 ** -23)
    assert q.double().cpu().numpy()[:, 0].tolist() == [448.0, 0.0, -448.0]


@pytest.mark.parametrize("act", ["swiglu", "swiglu_interleaved"])
def test_quantize_swiglu_special_values(act):
    """Gates of either infinity and far from zero, NaN gates and values: the
    blocks that hold no finite result are NaN, the others as the formula says."""
    dg = _dg()
    K = 130
    g, u = torch.ones(8, K), torch.full((8, K), 2.0)
    g[0, 3], g[1, 129], g[2, 0] = float("nan"), float("inf"), -float("inf")
    u[3, 5], u[4, 128] = float("nan"), -float("inf")
    g[5], g[6], g[7] = -200.0, 200.0, 0.0
    x = torch.stack((g, u), -1).view(8, 2 * K) if act != "swiglu" else torch.cat((g, u), 1)
    q, s = dg.fp8_quantize(x.cuda(), act=act)
    bad = torch.zeros(2, 8, dtype=torch.bool)
    bad[0, 0] = bad[1, 1] = bad[0, 2] = bad[0, 3] = bad[1, 4] = True
    assert torch.equal(torch.isnan(s).cpu(), bad)
    v = ref.dequantize_rows(q, s)
    assert np.all(v[5] == 0.0) and np.all(v[7] == 0.0)
    assert np.all(np.abs(v[6] - 400.0) <= 400.0 * 2.0 ** -20)   # the block's largest value takes the largest code


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("G,N,K", [(None, 1, 1), (None, 128, 128), (None, 130, 257), (2, 64, 704), (3, 129, 99), (1, 300, 1024)])
def test_quantize_blocks(G, N, K, dtype):
    dg = _dg()
    rng = np.random.default_rng(N + K)
    shape = (N, K) if G is None else (G, N, K)
    w = torch.from_numpy((rng.standard_normal(shape) * 0.02).astype(np.float32)).to(dtype)
    if N > 128:
        w[..., 0, 0] = float("nan")
        w[..., 128:, :128] = 0.0
    q, s = dg.fp8_quantize_blocks(w.cuda())
    d = w.double().numpy().reshape(-1, N, K)
    for g in range(d.shape[0]):
        want_q, want_s = ref.quantize_blocks(d[g])
        _same_codes(q.reshape(-1, N, K)[g] if G is None else q[g], want_q)
        _same_scales(s if G is None else s[g], want_s)


def test_quantize_strides_and_given_outputs():
    """Views of wider tensors in and out: what lies between the rows stays."""
    dg = _dg()
    rng = np.random.default_rng(11)
    wide = _hidden(rng, 20, 400, torch.bfloat16).cuda()
    for x in (wide[:, :256], wide[:, 3:260], wide[::2, 8:264]):
        rows, K = x.shape
        buf = torch.full((rows, 400), 0x55, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        sbuf = torch.full((ref.blocks(K) + 1, rows + 5), -1.0, device="cuda")
        out = (buf[:, :K], sbuf[:ref.blocks(K), :rows])
        q, s = dg.fp8_quantize(x, out=out)
        assert q.data_ptr() == buf.data_ptr()
        want_q, want_s = ref.quantize_rows(x.double().cpu().numpy())
        _same_codes(q, want_q)
        _same_scales(s, want_s)
        assert torch.all(buf.view(torch.uint8)[:, K:] == 0x55)
        assert torch.all(sbuf[:, rows:] == -1.0) and torch.all(sbuf[-1] == -1.0)


# ---- products ----------------------------------------------------------------------

def _check(got, want, want_abs, K, weighted=False):
    out = got.double().cpu().numpy()
    bound = ref.product_bound(want, want_abs, K, got.dtype, weighted)
    err = np.abs(out - want)
    assert np.all(err <= bound), float((err / bound).max())


@pytest.mark.parametrize("out_dtype", TYPES)
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 1), (1, 16, 16), (3, 5, 7), (1, 5632, 2816), (8, 704, 2816), (9, 130, 385), (16, 1408, 128), (17, 256, 2816),
    (64, 33, 1000), (127, 257, 129), (128, 128, 128), (129, 640, 704), (256, 2816, 2816), (255, 1001, 1111),
    (300, 384, 8192), (1000, 513, 256), (2, 20000, 64), (513, 96, 90)])
def test_gemm(M, N, K, out_dtype):
    dg = _dg()
    rng = np.random.default_rng(M + N + K)
    a, sa = ref.random_operand(rng, M, K)
    b, sb = ref.random_weights(rng, N, K)
    got = dg.fp8_gemm(a, sa, b, sb, out_dtype=out_dtype)
    if out_dtype == torch.float16:   # the whole e4m3 range overflows fp16: smaller scales
        sa = sa * 2.0 ** -14
        got = dg.fp8_gemm(a, sa, b, sb, out_dtype=out_dtype)
    want, want_abs = ref.product(ref.dequantize_rows(a, sa), ref.dequantize_blocks(b, sb))
    _check(got, want, want_abs, K)


@pytest.mark.parametrize("M,N,K", [(1, 100, 300), (5, 100, 300), (40, 100, 300), (300, 300, 300)])
def test_gemm_strides_weights_and_given_output(M, N, K):
    """Wider pitches (with NaN codes between the rows), row weights, and an
    output whose rows are views: nothing beside them is written."""
    dg = _dg()
    rng = np.random.default_rng(M)
    a, sa = ref.random_operand(rng, M, K, pitch=368)
    b, sb = ref.random_weights(rng, N, K, pitch=512)
    sa_wide = torch.full((sa.shape[0], M + 3), float("nan"), device="cuda")
    sa_wide[:, 1:M + 1] = sa
    sa = sa_wide[:, 1:M + 1]
    w = torch.from_numpy(rng.standard_normal(M).astype(np.float32)).cuda()
    for dtype, ld, first in ((torch.bfloat16, N + 12, 0), (torch.bfloat16, N + 7, 3), (torch.float32, N + 5, 1)):
        buf = torch.full((M + 1, ld), -7.0, dtype=dtype, device="cuda")
        out = buf[:M, first:first + N]
        got = dg.fp8_gemm(a, sa, b, sb, row_weight=w, out=out)
        assert got.data_ptr() == out.data_ptr()
        want, want_abs = ref.product(ref.dequantize_rows(a, sa), ref.dequantize_blocks(b, sb))
        wd = w.double().cpu().numpy()[:, None]
        _check(got, want * wd, want_abs * np.abs(wd), K, weighted=True)
        rest = torch.ones_like(buf, dtype=torch.bool)
        rest[:M, first:first + N] = False
        assert torch.all(buf[rest] == -7.0)


@pytest.mark.parametrize("M,N", [(200, 1003), (600, 700), (300, 20013)])
@pytest.mark.parametrize("out_dtype", TYPES)
def test_gemm_columns_end_inside_a_unit_of_the_output_rows(M, N, out_dtype):
    """Aligned output rows whose last column is not at a 16-byte boundary, with
    every width of tile: the rest of the row stays."""
    dg = _dg()
    K = 130
    rng = np.random.default_rng(N)
    a, sa = ref.random_operand(rng, M, K)
    b, sb = ref.random_weights(rng, N, K)
    sa = sa * 2.0 ** -14
    buf = torch.full((M, (N + 15) // 16 * 16), -7.0, dtype=out_dtype, device="cuda")
    got = dg.fp8_gemm(a, sa, b, sb, out=buf[:, :N])
    want, want_abs = ref.product(ref.dequantize_rows(a, sa), ref.dequantize_blocks(b, sb))
    _check(got, want, want_abs, K)
    assert torch.all(buf[:, N:] == -7.0)


@pytest.mark.parametrize("M", [1, 12, 200])
def test_gemm_nan_stays_in_its_row_and_column(M):
    """A NaN scale makes exactly its row's (its 128 columns') results NaN; so
    does a NaN code for its row."""
    dg = _dg()
    N, K = 300, 400
    rng = np.random.default_rng(M)
    a, sa = ref.random_operand(rng, M, K)
    b, sb = ref.random_weights(rng, N, K)
    sa[1, M // 2] = float("nan")
    sb[1, 3] = float("nan")
    a.view(torch.uint8)[M - 1, 17] = 0x7F
    got = torch.isnan(dg.fp8_gemm(a, sa, b, sb))
    want = torch.zeros(M, N, dtype=torch.bool)
    want[M // 2] = want[M - 1] = True
    want[:, 128:256] = True
    assert torch.equal(got.cpu(), want)


def _sizes(rng, G, rows, empty):
    w = rng.random(G) ** 3
    w[rng.permutation(G)[:empty]] = 0
    return rng.multinomial(rows, w / w.sum())


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("sizes,N,K", [
    ([1], 16, 16), ([0, 1, 0], 40, 100), ([1] * 8, 704, 256), ([3, 0, 0, 17, 1], 130, 704), ([0, 0, 300], 257, 129),
    ([128, 256, 129, 0, 255], 384, 384), ([5] * 40, 96, 128), ([1000, 1], 200, 64), ([0, 64, 0, 0, 700, 2], 1408, 300)])
def test_grouped_gemm(sizes, N, K, out_dtype):
    """Ragged groups, empty ones, rows before the first and behind the last."""
    dg = _dg()
    G, lead, tail = len(sizes), 2, 3
    rng = np.random.default_rng(sum(sizes) + N + K)
    M = lead + sum(sizes) + tail
    off = np.concatenate([[0], np.cumsum(sizes)]) + lead
    a, sa = ref.random_operand(rng, M, K)
    b, sb = ref.random_weights(rng, N, K, G=G)
    w = torch.from_numpy(rng.random(M).astype(np.float32)).cuda()
    out = torch.full((M, N), -3.0, dtype=out_dtype, device="cuda")
    got = dg.fp8_grouped_gemm(a, sa, b, sb, torch.from_numpy(off.astype(np.int32)).cuda(), row_weight=w, out=out)
    av, bv, wd = ref.dequantize_rows(a, sa), ref.dequantize_blocks(b, sb), w.double().cpu().numpy()[:, None]
    for g in range(G):
        r = slice(off[g], off[g + 1])
        want, want_abs = ref.product(av[r], bv[g])
        _check(got[r], want * wd[r], want_abs * wd[r], K, weighted=True)
    assert torch.all(out[:lead] == -3.0) and torch.all(out[M - tail:] == -3.0)


@pytest.mark.parametrize("G,rows,empty", [(16, 512, 4), (128, 2048, 44), (128, 200, 60), (1000, 1500, 500)])
def test_grouped_gemm_like_an_expert_layer(G, rows, empty):
    dg = _dg()
    N, K = 160, 192
    rng = np.random.default_rng(G + rows)
    sizes = _sizes(rng, G, rows, empty)
    off = np.concatenate([[0], np.cumsum(sizes)])
    a, sa = ref.random_operand(rng, rows, K)
    b, sb = ref.random_weights(rng, N, K, G=G)
    got = dg.fp8_grouped_gemm(a, sa, b, sb, torch.from_numpy(off.astype(np.int32)).cuda())
    av, bv = ref.dequantize_rows(a, sa), ref.dequantize_blocks(b, sb)
    for g in range(G):
        r = slice(off[g], off[g + 1])
        _check(got[r], *ref.product(av[r], bv[g]), K)


def test_grouped_gemm_offsets_outside_are_held_inside():
    dg = _dg()
    N, K, M = 48, 80, 30
    rng = np.random.default_rng(5)
    a, sa = ref.random_operand(rng, M, K)
    b, sb = ref.random_weights(rng, N, K, G=3)
    out = torch.full((M, N), -3.0, device="cuda")
    dg.fp8_grouped_gemm(a, sa, b, sb, torch.tensor([-9, 4, 20, 1000], dtype=torch.int32, device="cuda"), out=out)
    av, bv = ref.dequantize_rows(a, sa), ref.dequantize_blocks(b, sb)
    for g, (lo, hi) in enumerate([(0, 4), (4, 20), (20, 30)]):
        _check(out[lo:hi], *ref.product(av[lo:hi], bv[g]), K)


def test_grouped_gemm_decreasing_offsets_stay_inside():
    """Offsets that decrease are the caller's mistake: whatever is computed, rows
    of no group and the memory around the output stay."""
    dg = _dg()
    rng = np.random.default_rng(6)
    N, K, M = 160, 256, 200
    a, sa = ref.random_operand(rng, M, K)
    b, sb = ref.random_weights(rng, N, K, G=4)
    buf = torch.full((M + 8, N), -3.0, device="cuda")
    for off in ([0, 100, 50, 120, 90], [180, 20, 5, 0, 0], [7, 7, 3, 9, 2]):
        buf.fill_(-3.0)
        dg.fp8_grouped_gemm(a, sa, b, sb, torch.tensor(off, dtype=torch.int32, device="cuda"), out=buf[4:4 + M])
        inside = torch.zeros(M + 8, dtype=torch.bool)
        for lo, hi in zip(off, off[1:]):
            inside[4 + lo:4 + max(lo, hi)] = True
        assert torch.all(buf.cpu()[~inside] == -3.0)


def test_no_rows():
    dg = _dg()
    rng = np.random.default_rng(1)
    b, sb = ref.random_weights(rng, 32, 64, G=2)
    a = torch.empty(0, 64, dtype=torch.float8_e4m3fn, device="cuda")
    sa = torch.empty(1, 0, device="cuda")
    assert dg.fp8_gemm(a, sa, b[0], sb[0]).shape == (0, 32)
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert dg.fp8_grouped_gemm(a, sa, b, sb, off).shape == (0, 32)
    q, s = dg.fp8_quantize(torch.empty(0, 64, device="cuda"))
    assert q.shape == (0, 64) and s.shape == (1, 0)
    # groups that are all empty: nothing is written
    a, sa = ref.random_operand(rng, 5, 64)
    out = torch.full((5, 32), 2.0, device="cuda")
    dg.fp8_grouped_gemm(a, sa, b, sb, off, out=out)
    assert torch.all(out == 2.0)


def test_offsets_beyond_32_bits():
    """An output and a set of weights of more than 2^32 bytes: their last rows."""
    dg = _dg()
    rng = np.random.default_rng(12)
    M, N, K = 8200, 262144, 48
    a, sa = ref.random_operand(rng, M, K)
    b, sb = ref.random_weights(rng, N, K)
    got = dg.fp8_gemm(a, sa, b, sb)
    assert got.numel() * 2 > 2 ** 32
    want, want_abs = ref.product(ref.dequantize_rows(a, sa)[-9:], ref.dequantize_blocks(b, sb))
    _check(got[-9:], want, want_abs, K)
    del got, b

    G, N, K = 512, 4096, 2064   # 4.3 GB of codes; the rows all belong to the last matrices
    codes = torch.randint(0, 112, (G, N, K), device="cuda", dtype=torch.uint8)
    sb = torch.rand(G, ref.blocks(N), ref.blocks(K), device="cuda")
    assert codes.numel() > 2 ** 32
    for sizes in ((1, 2), (40, 30), (300, 700), (500, 40600)):
        M = sum(sizes)
        a, sa = ref.random_operand(rng, M, K)
        off = torch.full((G + 1,), M, dtype=torch.int32, device="cuda")
        off[:G - 1], off[G - 1] = 0, sizes[0]
        out = dg.fp8_grouped_gemm(a, sa, codes.view(torch.float8_e4m3fn), sb, off)
        av, row = ref.dequantize_rows(a, sa), 0
        for g, n in zip((G - 2, G - 1), sizes):
            some = np.unique(np.r_[row:row + min(n, 20), row + n - min(n, 20):row + n])   # its first and last rows
            want = ref.product(av[some], ref.dequantize_blocks(codes[g].view(torch.float8_e4m3fn), sb[g]))
            _check(out[torch.from_numpy(some).cuda()], *want, K)
            row += n


def test_quantised_offsets_beyond_32_bits():
    """Inputs and codes of more than 2^32 bytes: the last rows and blocks."""
    dg = _dg()
    rows, K = 70003, 65544   # K ends inside a block
    x = torch.empty(rows, K, dtype=torch.bfloat16, device="cuda").normal_()
    q, s = dg.fp8_quantize(x)
    assert q.numel() > 2 ** 32
    last = x[-2:].double().cpu().numpy()
    want_q, want_s = ref.quantize_rows(last)
    _same_codes(q[-2:], want_q)
    _same_scales(s[:, -2:], want_s)
    del q, s
    q, s = dg.fp8_quantize(x, index=torch.tensor([rows - 1, rows, rows - 2, rows - 1], dtype=torch.int32, device="cuda"))
    for r, w in ((0, 1), (2, 0), (3, 1)):
        _same_codes(q[r:r + 1], want_q[w:w + 1])
        _same_scales(s[:, r:r + 1], want_s[:, w:w + 1])
    assert not q[1].float().any()
    y, sy = dg.fp8_quantize(x, act="swiglu")
    halves = ref.swiglu(last[:, :K // 2], last[:, K // 2:])
    got = ref.dequantize_rows(y[-2:], sy[:, -2:])
    step = np.repeat(sy[:, -2:].double().cpu().numpy().T, 128, axis=1)[:, :K // 2]
    assert np.all(np.abs(got - halves) <= (2.0 ** -4 + 2.0 ** -19) * np.abs(halves) + 2.0 ** -10 * step)
    del y, sy
    w = x[:70000].view(2, 35000, K)
    q, s = dg.fp8_quantize_blocks(w)
    assert q.numel() > 2 ** 32
    r0 = 35000 // 128 * 128
    want_q, want_s = ref.quantize_blocks(w[1, r0:, -264:].double().cpu().numpy())   # from a block's first row and column
    _same_codes(q[1, r0:, -264:], want_q)
    _same_scales(s[1, -1:, -3:], want_s)


def _in_range(got, want, want_abs, K):
    """The results without those outside got's type.  A value is rounded to an infinity from
    half a step above the largest finite one on (fp16: 65504 + 16); within the bound's
    distance of that point both are right."""
    if got.dtype != torch.float16:
        return got, want, want_abs
    edge, bound = 65520.0, ref.product_bound(want, want_abs, K, torch.float32)
    out = got.double().cpu().numpy()
    over = np.abs(want) - bound >= edge
    assert np.all(np.isinf(out[over]) & (np.sign(out[over]) == np.sign(want[over])))
    assert np.all(np.isfinite(out[np.abs(want) + bound < edge]))
    keep = np.isfinite(out)
    return got[torch.from_numpy(keep).cuda()], want[keep], want_abs[keep]


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("sizes,N,K", [([255, 256, 257, 0, 1, 300, 31, 420], 2000, 333), ([1790], 2299, 128),
                                       ([600, 2, 0, 900], 4100, 1000)])
def test_grouped_gemm_many_columns(sizes, N, K, out_dtype):
    """Enough tiles that the widest ones are taken; groups that end inside a tile and a quarter of one."""
    dg = _dg()
    rng = np.random.default_rng(N + K)
    off = np.concatenate([[0], np.cumsum(sizes)])
    M, G = int(off[-1]), len(sizes)
    a, sa = ref.random_operand(rng, M, K)
    b, sb = ref.random_weights(rng, N, K, G=G)
    w = torch.from_numpy(rng.standard_normal(M).astype(np.float32)).cuda()
    got = dg.fp8_grouped_gemm(a, sa, b, sb, torch.from_numpy(off.astype(np.int32)).cuda(), row_weight=w, out_dtype=out_dtype)
    av, wd = ref.dequantize_rows(a, sa), w.double().cpu().numpy()[:, None]
    for g in range(G):
        r = slice(off[g], off[g + 1])
        want, want_abs = ref.product(av[r], ref.dequantize_blocks(b[g], sb[g]))
        _check(got[r], want * wd[r], want_abs * np.abs(wd[r]), K, weighted=True)


@pytest.mark.parametrize("N,K,out", [(40, 3054, torch.bfloat16), (24, 4096, torch.float32), (128, 2816, torch.bfloat16),
                                     (120, 1000, torch.float16)])
def test_few_columns_many_groups(N, K, out):
    """One tile of columns per group and many ragged tiles of rows: units follow one
    another quickly, and copies of far weights land out of order.  The same call again and
    again gives the same bits."""
    dg = _dg()
    rng = np.random.default_rng(N)
    sizes = [0 if g == 17 else int(rng.integers(130, 520)) for g in range(57)]
    M = sum(sizes)
    off = torch.from_numpy(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)).cuda()
    a, sa = ref.random_operand(rng, M, K)
    b, sb = ref.random_weights(rng, N, K, G=len(sizes))
    first = dg.fp8_grouped_gemm(a, sa, b, sb, off, out_dtype=out)
    av, row = ref.dequantize_rows(a, sa), 0
    for g, n in enumerate(sizes):
        if n:
            want, want_abs = ref.product(av[row:row + n], ref.dequantize_blocks(b[g], sb[g]))
            _check(*_in_range(first[row:row + n], want, want_abs, K), K)
        row += n
    for _ in range(50):
        again = [dg.fp8_grouped_gemm(a, sa, b, sb, off, out_dtype=out) for _ in range(8)]
        assert all(torch.equal(first, x) for x in again)


# ---- as they are used together ----------------------------------------------------------

def _expert_block(dg, x, index, off, w1, w2, row_weight):
    """Gather + quantise, gate/up, SwiGLU + quantise, down with routing weights."""
    q, s = dg.fp8_quantize(x, index=index)
    y = dg.fp8_grouped_gemm(q, s, *w1, off)
    h, hs = dg.fp8_quantize(y, act="swiglu_interleaved")
    return (q, s), y, (h, hs), dg.fp8_grouped_gemm(h, hs, *w2, off, row_weight=row_weight, out_dtype=torch.float32)


def _expert_inputs(T, k, G, d, f, seed=0):
    dg = _dg()
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.standard_normal((T, d)).astype(np.float32)).to(torch.bfloat16).cuda()
    expert = np.stack([rng.permutation(G)[:k] for _ in range(T)]).ravel()
    order = np.argsort(expert, kind="stable")
    off = np.concatenate([[0], np.cumsum(np.bincount(expert, minlength=G))]).astype(np.int32)
    w1 = dg.fp8_quantize_blocks(torch.from_numpy((rng.standard_normal((G, 2 * f, d)) * 0.05).astype(np.float32)).cuda())
    w2 = dg.fp8_quantize_blocks(torch.from_numpy((rng.standard_normal((G, d, f)) * 0.05).astype(np.float32)).cuda())
    index = torch.from_numpy((order // k).astype(np.int32)).cuda()
    rw = torch.from_numpy(rng.random(T * k).astype(np.float32)).cuda()
    return x, index, torch.from_numpy(off).cuda(), w1, w2, rw


@pytest.mark.parametrize("T,k,G,d,f", [(1, 2, 16, 256, 512), (1, 8, 32, 320, 192), (64, 2, 16, 256, 512), (256, 4, 8, 256, 96)])
def test_expert_block_stage_by_stage(T, k, G, d, f):
    """Each stage against the 64-bit form on the stage's own input."""
    dg = _dg()
    x, index, off, w1, w2, rw = _expert_inputs(T, k, G, d, f)
    (q, s), y, (h, hs), out = _expert_block(dg, x, index, off, w1, w2, rw)
    want_q, want_s = ref.quantize_rows(x.double().cpu().numpy()[index.cpu().numpy()])
    _same_codes(q, want_q)
    _same_scales(s, want_s)
    o = off.cpu().numpy()
    qv, hv = ref.dequantize_rows(q, s), ref.dequantize_rows(h, hs)
    w1v, w2v = ref.dequantize_blocks(*w1), ref.dequantize_blocks(*w2)
    wd = rw.double().cpu().numpy()[:, None]
    for g in range(G):
        r = slice(o[g], o[g + 1])
        _check(y[r], *ref.product(qv[r], w1v[g]), d)
        want, want_abs = ref.product(hv[r], w2v[g])
        _check(out[r], want * wd[r], want_abs * wd[r], f, weighted=True)
    yd = y.double().cpu().numpy()
    v = ref.swiglu(yd[:, 0::2], yd[:, 1::2])
    step = np.repeat(hs.double().cpu().numpy().T, 128, axis=1)[:, :f]
    assert np.all(np.abs(hv - v) <= (2.0 ** -4 + 2.0 ** -15) * np.abs(v) + 2.0 ** -10 * step)


def test_streams_and_captured_graphs_give_the_same_bits():
    """The block on the current stream, on two streams at once, and replayed
    from two graphs that run at the same time on new inputs."""
    dg = _dg()
    a_in, b_in = _expert_inputs(96, 4, 16, 256, 192, seed=1), _expert_inputs(40, 4, 16, 256, 192, seed=2)
    want = [_expert_block(dg, *i)[-1].clone() for i in (a_in, b_in)]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = [None, None]
    for _ in range(3):
        for n, (st, i) in enumerate(((s1, a_in), (s2, b_in))):
            with torch.cuda.stream(st):
                got[n] = _expert_block(dg, *i)[-1]
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])

    graphs, outs = [], []
    xs = [a_in[0].clone(), b_in[0].clone()]
    for st, i, x in ((s1, a_in, xs[0]), (s2, b_in, xs[1])):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            outs.append(_expert_block(dg, x, *i[1:])[-1])
        graphs.append(g)
    for x in xs:
        x.mul_(-1.5)
    torch.cuda.synchronize()
    for _ in range(3):
        for st, g in zip((s1, s2), graphs):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for n, (i, x) in enumerate(((a_in, xs[0]), (b_in, xs[1]))):
        assert torch.equal(outs[n], _expert_block(dg, x, *i[1:])[-1])


def test_given_stream():
    dg = _dg()
    rng = np.random.default_rng(8)
    a, sa = ref.random_operand(rng, 33, 256)
    b, sb = ref.random_weights(rng, 70, 256)
    want = dg.fp8_gemm(a, sa, b, sb)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = dg.fp8_gemm(a, sa, b, sb, stream=st)
    q, s = dg.fp8_quantize(want, stream=st)
    st.synchronize()
    assert torch.equal(got, want)
    assert torch.equal(q.view(torch.uint8), dg.fp8_quantize(want)[0].view(torch.uint8))


def test_given_stream_keeps_its_inputs():
    """Inputs (and outputs) that the caller lets go while a busy stream has yet to
    read them are not given to other tensors."""
    dg = _dg()
    rng = np.random.default_rng(10)
    M, N, K, G = 300, 256, 512, 2
    a, sa = ref.random_operand(rng, M, K)
    b, sb = ref.random_weights(rng, N, K, G=G)
    inputs = dict(x=torch.randn(M, K, device="cuda").to(torch.bfloat16),
                  index=torch.from_numpy(rng.permutation(M).astype(np.int32)).cuda(),
                  w=torch.randn(G, N, K, device="cuda"), a=a, sa=sa, b=b, sb=sb, rw=torch.rand(M, device="cuda"),
                  off=torch.tensor([0, 100, M], dtype=torch.int32, device="cuda"))

    def calls(i, stream):
        return (*dg.fp8_quantize(i["x"], index=i["index"], stream=stream), *dg.fp8_quantize_blocks(i["w"], stream=stream),
                dg.fp8_gemm(i["a"], i["sa"], i["b"][1], i["sb"][1], row_weight=i["rw"], stream=stream),
                dg.fp8_grouped_gemm(i["a"], i["sa"], i["b"], i["sb"], i["off"], row_weight=i["rw"], stream=stream))
    want = calls(inputs, None)
    side = torch.cuda.Stream()
    mine = {k: t.view(torch.uint8).clone().view(t.dtype) if t.dtype == torch.float8_e4m3fn else t.clone()
            for k, t in inputs.items()}
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    at = {t.untyped_storage().data_ptr() for t in mine.values()}
    sizes = [t.untyped_storage().nbytes() for t in mine.values()]
    got = calls(mine, side)
    del mine
    new = [torch.full((n,), 0x55, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
    assert not at & {t.untyped_storage().data_ptr() for t in new}
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_captured_on_a_given_stream():
    """A graph of calls that name the stream they are captured on, replayed on new inputs."""
    dg = _dg()
    rng = np.random.default_rng(11)
    b, sb = ref.random_weights(rng, 192, 256)
    x = torch.randn(70, 256, device="cuda").to(torch.bfloat16)

    def block(stream):
        return dg.fp8_gemm(*dg.fp8_quantize(x, stream=stream), b, sb, stream=stream)
    want = block(None).clone()
    torch.cuda.synchronize()
    st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        out = block(st)
    for factor in (1.0, -2.0):
        x.mul_(factor)
        g.replay()
        assert torch.equal(out, block(None))
    assert torch.equal(out, -2.0 * want)   # a power of two scales every step exactly


def _held(dg, what, unit, block, call):
    """`call` with something left out of one unit of its kernel, so that waits run out."""
    dg.check(dg.lib.dg_test_fp8_hold(what, unit, block, 20_000_000))
    try:
        out = call()
    finally:
        dg.check(dg.lib.dg_test_fp8_hold(0, 0, 0, 0))
    torch.cuda.synchronize()
    return out


# rows and columns of a unit and the units a CTA (pair) takes in turn, as the host chooses them on 148 SMs
@pytest.mark.parametrize("what", [1, 2], ids=["copies", "scales"])
@pytest.mark.parametrize("M,N,K,rows,cols,step", [
    (600, 400, 1408, 256, 128, 74),      # pairs, 128 columns
    (4096, 2048, 1408, 256, 256, 74),    # pairs, 256 columns, two units each
    (64, 37888, 1408, 64, 128, 296),     # streaming, one unit each
    (64, 75776, 1000, 64, 128, 296),     # streaming, two units each
    (40, 512, 1408, 64, 128, 0)],        # streaming, a unit's blocks split among a cluster
    ids=["pair128", "pair256", "stream", "stream2", "split"])
def test_a_wait_that_runs_out_leaves_no_wrong_number(what, M, N, K, rows, cols, step):
    """A unit whose copies or scales never come: the kernel returns, the unit and those
    its CTAs would have taken after it hold NaN wherever they do not hold the product,
    and all others are right.  Afterwards everything is as usual."""
    dg = _dg()
    rng = np.random.default_rng(M + N)
    a, sa = ref.random_operand(rng, M, K)
    b, sb = ref.random_weights(rng, N, K)
    good = dg.fp8_gemm(a, sa, b, sb, out_dtype=torch.float32)
    m_tiles, unit = (M + rows - 1) // rows, 2
    out = torch.full_like(good, -3.0)
    _held(dg, what, unit, 6, lambda: dg.fp8_gemm(a, sa, b, sb, out=out))

    def tile(u):
        return (slice(u % m_tiles * rows, (u % m_tiles + 1) * rows), slice(u // m_tiles * cols, (u // m_tiles + 1) * cols))
    affected = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    for u in range(unit, m_tiles * ((N + cols - 1) // cols), step or 10 ** 6):
        affected[tile(u)] = True
    assert torch.equal(out[~affected], good[~affected])
    nan = torch.isnan(out)
    assert torch.all(nan | (out == good))
    held = nan[tile(unit)]
    if rows == 256 and what == 2:
        held = held[:128]   # the CTA whose scales do not come; the other one may have had all it needs
    assert torch.all(held)
    assert torch.equal(dg.fp8_gemm(a, sa, b, sb, out_dtype=torch.float32), good)


def test_grouped_wait_that_runs_out_leaves_no_wrong_number():
    """The same with groups: rows of no group stay as they were."""
    dg = _dg()
    rng = np.random.default_rng(4)
    off = torch.tensor([3, 300, 300, 900, 1000], dtype=torch.int32, device="cuda")
    a, sa = ref.random_operand(rng, 1010, 1000)
    b, sb = ref.random_weights(rng, 384, 1000, G=4)
    outs = [torch.full((1010, 384), -3.0, device="cuda") for _ in range(2)]
    dg.fp8_grouped_gemm(a, sa, b, sb, off, out=outs[0])
    _held(dg, 1, 1, 3, lambda: dg.fp8_grouped_gemm(a, sa, b, sb, off, out=outs[1]))
    nan = torch.isnan(outs[1])
    assert nan.any() and torch.all(nan | (outs[0] == outs[1]))
    assert torch.all(outs[1][:3] == -3.0) and torch.all(outs[1][1000:] == -3.0)


def test_python_refusals():
    """Wrong shapes, types and strides are refused before any launch."""
    dg = _dg()
    rng = np.random.default_rng(9)
    a, sa = ref.random_operand(rng, 8, 64)
    b, sb = ref.random_weights(rng, 32, 64)
    off = torch.zeros(2, dtype=torch.int32, device="cuda")
    x = torch.zeros(4, 64, device="cuda")
    for call in (
            lambda: dg.fp8_gemm(a.float(), sa, b, sb), lambda: dg.fp8_gemm(a, sa[:, :7], b, sb),
            lambda: dg.fp8_gemm(a, sa.double(), b, sb), lambda: dg.fp8_gemm(a[:, :32], sa, b, sb),
            lambda: dg.fp8_gemm(a, sa, b, sb.expand(2, 1)), lambda: dg.fp8_gemm(a, sa, b, sb, out_dtype=torch.float64),
            lambda: dg.fp8_gemm(a, sa, b, sb, out=torch.empty(8, 31, device="cuda")),
            lambda: dg.fp8_gemm(a, sa, b, sb, out=torch.empty(32, 8, device="cuda").t()),
            lambda: dg.fp8_gemm(a, sa, b, sb, row_weight=torch.ones(7, device="cuda")),
            lambda: dg.fp8_gemm(a, sa.cpu(), b, sb), lambda: dg.fp8_gemm(a[:, ::2], sa, b[:, ::2], sb),
            lambda: dg.fp8_grouped_gemm(a, sa, b, sb, off), lambda: dg.fp8_grouped_gemm(a, sa, b[None], sb[None], None),
            lambda: dg.fp8_grouped_gemm(a, sa, b[None], sb[None], off.long()),
            lambda: dg.fp8_grouped_gemm(a, sa, b[None], sb[None], off[:1]),
            lambda: dg.fp8_quantize(x.double()), lambda: dg.fp8_quantize(x, act="relu"), lambda: dg.fp8_quantize(x.t()),
            lambda: dg.fp8_quantize(x[:, :63], act="swiglu"), lambda: dg.fp8_quantize(x, index=off.long()),
            lambda: dg.fp8_quantize(x, out=(a, sa)), lambda: dg.fp8_quantize_blocks(x[0]),
            lambda: dg.fp8_quantize_blocks(x.t()), lambda: dg.fp8_quantize_blocks(x.view(2, 2, 64).transpose(0, 1))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(dg.DgError):   # rows of 40 bytes cannot start on 16-byte boundaries
        odd = torch.zeros(8, 40, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        dg.fp8_gemm(odd, sa, torch.zeros(32, 48, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)[:, :40], sb)
