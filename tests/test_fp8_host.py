"""Argument checks of the 8-bit operators' C entry points (no GPU: every call
here is refused, or has nothing to do, before any device work; the addresses
are never dereferenced)."""

import pytest

A, S, B, T, O, D = (1 << 20) * 1, (1 << 20) * 2, (1 << 20) * 3, (1 << 20) * 4, (1 << 20) * 5, (1 << 20) * 6


def _gemm(dg, M=8, N=32, K=64, lda=64, lds=8, ldb=64, ldo=32, a=A, sa=S, b=B, sb=T, out=D, w=None, dt=0):
    return dg.lib.dg_fp8_gemm(a, lda, sa, lds, b, ldb, sb, M, N, K, w, out, dt, ldo, None)


def _grouped(dg, G=4, M=8, N=32, K=64, lda=64, lds=8, ldb=64, ldo=32, a=A, sa=S, b=B, sb=T, off=O, out=D, w=None, dt=0):
    return dg.lib.dg_fp8_grouped_gemm(a, lda, sa, lds, b, ldb, sb, off, G, M, N, K, w, out, dt, ldo, None)


BAD = [dict(M=-1), dict(N=0), dict(K=0), dict(M=1 << 31, lds=1 << 31), dict(N=1 << 31, ldo=1 << 31),
       dict(K=1 << 31, lda=1 << 31, ldb=1 << 31), dict(lda=63), dict(lda=48), dict(lda=72), dict(ldb=72), dict(ldb=48),
       dict(lds=7), dict(ldo=31), dict(a=A + 8), dict(b=B + 1), dict(sa=S + 2), dict(sb=T + 1), dict(out=D + 1),
       dict(out=D + 2, dt=2), dict(w=A + 3), dict(a=None), dict(sa=None), dict(b=None), dict(sb=None), dict(out=None),
       dict(dt=3), dict(dt=-1)]


@pytest.mark.parametrize("bad", BAD, ids=str)
def test_products_refuse(bad):
    import discrete_diffusion_moe_b200 as dg
    for call, name in ((_gemm, "dg_fp8_gemm"), (_grouped, "dg_fp8_grouped_gemm")):
        assert call(dg, **bad) == dg.DG_ERR_INVALID_ARG
        assert name in dg.last_error()


@pytest.mark.parametrize("bad", [dict(G=0), dict(G=-1), dict(G=1025), dict(off=None), dict(off=O + 2),
                                 dict(G=1024, N=1 << 22, ldo=1 << 22)], ids=str)
def test_grouped_product_refuses(bad):
    import discrete_diffusion_moe_b200 as dg
    assert _grouped(dg, **bad) == dg.DG_ERR_INVALID_ARG
    assert "dg_fp8_grouped_gemm" in dg.last_error()


def test_no_rows_is_a_call_that_does_nothing():
    import discrete_diffusion_moe_b200 as dg
    assert _gemm(dg, M=0, a=None, sa=None, out=None) == dg.DG_OK
    assert _grouped(dg, M=0, a=None, sa=None, out=None) == dg.DG_OK
    assert dg.lib.dg_fp8_quantize(None, 0, 64, 0, None, 0, 0, 64, None, 64, None, 0, None) == dg.DG_OK
    assert dg.lib.dg_fp8_quantize_blocks(None, 0, 64, 0, 8, 64, None, 64, None, None) == dg.DG_OK


def _quant(dg, x=A, dt=0, ldx=64, x_rows=8, index=None, act=0, rows=8, cols=64, q=B, ldq=64, s=S, lds=8):
    return dg.lib.dg_fp8_quantize(x, dt, ldx, x_rows, index, act, rows, cols, q, ldq, s, lds, None)


@pytest.mark.parametrize("bad", [
    dict(dt=3), dict(act=3), dict(act=-1), dict(rows=-1), dict(cols=0), dict(x_rows=-1), dict(ldx=63), dict(act=1),
    dict(act=2, ldx=127), dict(ldq=63), dict(ldq=72), dict(ldq=48), dict(lds=7), dict(x_rows=7), dict(x=None),
    dict(q=None), dict(s=None), dict(x=A + 1), dict(x=A + 2, dt=2), dict(q=B + 8), dict(s=S + 1), dict(index=O + 1),
    dict(rows=1 << 31, lds=1 << 31, x_rows=1 << 31), dict(cols=1 << 30, ldx=1 << 31, ldq=1 << 30)], ids=str)
def test_quantize_refuses(bad):
    import discrete_diffusion_moe_b200 as dg
    assert _quant(dg, **bad) == dg.DG_ERR_INVALID_ARG
    assert "dg_fp8_quantize:" in dg.last_error()


@pytest.mark.parametrize("bad", [
    dict(dt=9), dict(ldw=63), dict(G=-1), dict(rows=0), dict(cols=0), dict(ldq=40), dict(ldq=72), dict(w=None),
    dict(q=None), dict(s=None), dict(w=A + 1), dict(q=B + 4), dict(s=S + 2),
    dict(G=1 << 30, rows=1 << 30)], ids=str)
def test_quantize_blocks_refuses(bad):
    import discrete_diffusion_moe_b200 as dg
    v = dict(w=A, dt=0, ldw=64, G=2, rows=8, cols=64, q=B, ldq=64, s=S)
    v.update(bad)
    assert dg.lib.dg_fp8_quantize_blocks(v["w"], v["dt"], v["ldw"], v["G"], v["rows"], v["cols"], v["q"], v["ldq"], v["s"],
                                         None) == dg.DG_ERR_INVALID_ARG
    assert "dg_fp8_quantize_blocks" in dg.last_error()


def test_tensors_on_the_cpu_are_refused():
    import torch
    import discrete_diffusion_moe_b200 as dg
    x = torch.zeros(4, 64)
    e = torch.zeros(4, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    for call in (lambda: dg.fp8_quantize(x), lambda: dg.fp8_quantize_blocks(x),
                 lambda: dg.fp8_gemm(e, torch.ones(1, 4), e, torch.ones(1, 1)),
                 lambda: dg.fp8_grouped_gemm(e, torch.ones(1, 4), e[None], torch.ones(1, 1, 1), torch.zeros(2).int())):
        with pytest.raises(ValueError):
            call()


def test_expert_buffer_sizes_and_null_contexts():
    import ctypes
    import discrete_diffusion_moe_b200 as dg
    cfg = dg.model_config(30, 2816, 16, 8, 176, 128, 8, 704, 262144)
    codes, scales = 128 * 3 * 704 * 2816, 128 * 4 * (11 * 22 + 22 * 6)
    assert dg.lib.dg_fp8_experts_bytes(ctypes.byref(cfg)) == 30 * (codes + scales)   # parts are multiples of 256 here
    bad = dg.model_config(1, 100, 1, 1, 32, 4, 2, 64, 4096)
    assert dg.lib.dg_fp8_experts_bytes(ctypes.byref(bad)) == 0
    assert dg.lib.dg_fp8_experts_scratch_bytes(None) == 0
    assert dg.lib.dg_fp8_experts_quantize(None, A, 1 << 30, None) == dg.DG_ERR_INVALID_ARG
    assert dg.lib.dg_fp8_experts_use(None, None, None, 0) == dg.DG_ERR_INVALID_ARG
