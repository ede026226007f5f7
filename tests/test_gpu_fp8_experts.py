"""A context on 8-bit experts (Model.use_fp8_experts): the matrices against the
plain 64-bit quantiser, the expert block bit for bit against the public
operators on the round's own inputs, every call that runs the layers, and back
to bf16 experts without a trace."""

import ctypes

import numpy as np
import pytest
import torch

import fp8_ref as ref
import oracle
import synth
from oracle.numerics import bf16_bits_to_f64
from parity import TINY

pytestmark = pytest.mark.gpu

CONFIGS = [TINY, dict(TINY, n_layers=1, d_model=320, n_experts=32, top_k=8, d_ff=192),
           dict(TINY, n_layers=1, d_model=256, n_experts=5, top_k=3, d_ff=64)]


def _align(n):
    return (n + 255) // 256 * 256


def _layer_views(cfg, experts, layer):
    """(gate/up codes, scales, down codes, scales) of one layer in the documented layout."""
    E, f, d = cfg.n_experts, cfg.d_ff, cfg.d_model
    bf, b2f, bd = ref.blocks(f), ref.blocks(2 * f), ref.blocks(d)
    sizes = [E * 2 * f * d, E * d * f, 4 * E * b2f * bd, 4 * E * bd * bf]
    at = layer * sum(_align(n) for n in sizes)
    parts = []
    for n in sizes:
        parts.append(experts[at:at + n])
        at += _align(n)
    gu, dn, sgu, sdn = parts
    return (gu.view(torch.float8_e4m3fn).view(E, 2 * f, d), sgu.view(torch.float32).view(E, b2f, bd),
            dn.view(torch.float8_e4m3fn).view(E, d, f), sdn.view(torch.float32).view(E, bd, bf))


def _buffer(dg, model, name, dtype, shape):
    ptr, size = ctypes.c_void_p(), ctypes.c_size_t()
    dg.check(dg.lib.dg_test_workspace_buffer(model.ctx, name.encode(), ctypes.byref(ptr), ctypes.byref(size)))
    off = ptr.value - model.workspace.data_ptr()
    n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
    assert n <= size.value
    return model.workspace[off:off + n].view(dtype).view(*shape)


def _round(dg, model, cfg, batch, graph=False, ctx_len=20):
    kv = dg.KVCache(cfg, batch, ctx_len + 256 * 3)
    tok = synth.context_tokens(batch, ctx_len, 5, cfg.vocab).astype(np.int32)
    model.encode(kv, torch.from_numpy(tok).cuda())
    cv = dg.Canvas(cfg, batch)
    model.canvas_init(cv, 0, 1234)
    out = dg.StepOutputs(cfg, batch, logits=True)
    for s in range(2):
        model.step(kv, cv, 0, s, dg.sampler_config(seed=1234, max_steps=4), out, graph=graph)
    model.check_device()
    return out.logits.clone(), cv.tokens.clone(), kv


@pytest.mark.parametrize("cfg_d", CONFIGS, ids=["tiny", "wide", "odd"])
@pytest.mark.parametrize("batch", [1, 2])
def test_expert_block_is_the_public_operators(cfg_d, batch):
    import discrete_diffusion_moe_b200 as dg
    cfg = dg.model_config(**cfg_d)
    model = dg.Model(cfg, batch, seed=0)
    before = _round(dg, model, cfg, batch)
    experts = model.quantize_experts()
    model.use_fp8_experts(experts)
    logits, tokens, _ = _round(dg, model, cfg, batch)
    assert torch.isfinite(logits).all() and not torch.equal(logits, before[0])

    # the matrices: every scale and code of two experts of the last layer
    W = oracle.Weights(oracle.ModelConfig(**cfg_d), seed=0).layer(cfg.n_layers - 1)
    w1, s1, w2, s2 = _layer_views(cfg, experts, cfg.n_layers - 1)
    for e in (0, cfg.n_experts - 1):
        gu = np.empty((2 * cfg.d_ff, cfg.d_model))
        gu[0::2], gu[1::2] = bf16_bits_to_f64(W["wg"][e]), bf16_bits_to_f64(W["wu"][e])
        for codes, scale, want in ((w1[e], s1[e], gu), (w2[e], s2[e], bf16_bits_to_f64(W["wd"][e]))):
            q, s = ref.quantize_blocks(want)
            assert np.array_equal(codes.double().cpu().numpy(), q)
            assert np.array_equal(scale.cpu().numpy(), s)

    # the last layer's expert block on its own inputs
    P = batch * 256 * cfg.top_k
    x = _buffer(dg, model, "xperm", torch.bfloat16, (P, cfg.d_model))
    off = _buffer(dg, model, "off", torch.int32, (cfg.n_experts + 1,))
    rw = _buffer(dg, model, "wperm", torch.float32, (P,))
    got = _buffer(dg, model, "yperm", torch.float32, (P, cfg.d_model))
    assert int(off[-1]) == P
    q, s = dg.fp8_quantize(x)
    y = dg.fp8_grouped_gemm(q, s, w1, s1, off)
    h, hs = dg.fp8_quantize(y, act="swiglu_interleaved")
    want = dg.fp8_grouped_gemm(h, hs, w2, s2, off, row_weight=rw, out_dtype=torch.float32)
    assert torch.equal(got, want)

    # the captured round gives the same bits; back on bf16 experts everything is as before
    g_logits, g_tokens, _ = _round(dg, model, cfg, batch, graph=True)
    assert torch.equal(g_logits, logits) and torch.equal(g_tokens, tokens)
    model.use_fp8_experts(None)
    for graph in (False, True):
        again = _round(dg, model, cfg, batch, graph=graph)
        assert torch.equal(again[0], before[0]) and torch.equal(again[1], before[1])
    model.close()


def test_switching_drops_the_captured_round():
    """A round captured on bf16 experts is not replayed after the switch."""
    import discrete_diffusion_moe_b200 as dg
    cfg = dg.model_config(**TINY)
    model = dg.Model(cfg, 1, seed=0)
    experts = model.quantize_experts()
    kv, cv, out = dg.KVCache(cfg, 1, 512), dg.Canvas(cfg, 1), dg.StepOutputs(cfg, 1, logits=True)
    got = []
    for e in (None, experts, None, experts):
        model.use_fp8_experts(e)
        model.canvas_init(cv, 0, 7)
        model.step(kv, cv, 0, 0, dg.sampler_config(seed=7, max_steps=2), out, graph=True)
        got.append(out.logits.clone())
    assert torch.equal(got[0], got[2]) and torch.equal(got[1], got[3]) and not torch.equal(got[0], got[1])
    model.close()


def test_blocks_and_autoregressive_steps_on_shared_experts():
    """Two contexts on one set of 8-bit experts: the same blocks and tokens."""
    import discrete_diffusion_moe_b200 as dg
    cfg = dg.model_config(**TINY)
    first = dg.Model(cfg, 1, seed=0)
    experts = first.quantize_experts()
    second = dg.Model(cfg, 1, weights_of=first)
    results = []
    for model in (first, second):
        model.use_fp8_experts(experts)
        kv, cv = dg.KVCache(cfg, 1, 1024), dg.Canvas(cfg, 1)
        model.encode(kv, torch.from_numpy(synth.context_tokens(1, 33, 3, cfg.vocab).astype(np.int32)).cuda())
        block = torch.zeros(1, 256, dtype=torch.int32, device="cuda")
        steps, rounds = model.decode_block(kv, cv, 0, dg.sampler_config(seed=3, max_steps=3), block)
        amax, samp = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        logits = torch.zeros(1, cfg.vocab, device="cuda")
        model.ar_step(kv, block[:, -1].contiguous(), 0.8, 3, amax, samp, logits)
        model.check_device()
        assert torch.isfinite(logits).all() and kv.length == 33 + 256 + 1
        results.append((block, logits, samp))
    for a, b in zip(*results):
        assert torch.equal(a, b)
    first.close()
    second.close()


@pytest.mark.parametrize("n_experts,tokens", [(4, 256), (16, 40)], ids=["pairs", "streaming"])
def test_an_expert_product_whose_wait_runs_out_is_reported(n_experts, tokens):
    """Copies that never come in an expert product of an encode pass (of one layer,
    after whose expert block nothing reads the result): the error word says so, and
    after it the context gives what it gave before."""
    import discrete_diffusion_moe_b200 as dg
    cfg = dg.model_config(**dict(TINY, n_layers=1, n_experts=n_experts, top_k=2))
    model = dg.Model(cfg, 1, seed=0)
    model.use_fp8_experts(model.quantize_experts())
    kv = dg.KVCache(cfg, 1, tokens + 256)
    toks = torch.from_numpy(synth.context_tokens(1, tokens, 3, cfg.vocab).astype(np.int32)).cuda()
    y = _buffer(dg, model, "yperm", torch.float32, (tokens * 2, cfg.d_model))
    inv = _buffer(dg, model, "inv", torch.int32, (tokens * 2,))

    def encode():
        """The expert block's rows by token (their order within an expert may differ between passes)."""
        kv.s.length = 0
        model.encode(kv, toks)
        return y[inv.long()]
    want = encode()
    model.check_device()
    dg.check(dg.lib.dg_test_fp8_hold(1, 0, 0, 20_000_000))
    try:
        got = encode()
    finally:
        dg.check(dg.lib.dg_test_fp8_hold(0, 0, 0, 0))
    with pytest.raises(dg.DgError) as e:
        model.check_device()
    assert e.value.status == dg.DG_ERR_TIMEOUT
    nan = torch.isnan(got)
    assert nan.any() and torch.all(nan | (got == want))
    assert torch.equal(encode(), want)
    model.check_device()
    model.close()


def _busy(stream, ms=60):
    """Keeps `stream` busy for about `ms` milliseconds."""
    with torch.cuda.stream(stream):
        torch.cuda._sleep(int(ms * 2e6))


def test_experts_quantised_on_another_stream_are_its_memory():
    """The buffer is not one that work on the current stream still writes to."""
    import discrete_diffusion_moe_b200 as dg
    cfg = dg.model_config(**TINY)
    model = dg.Model(cfg, 1, seed=0)
    want = model.quantize_experts()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(2):   # the second time the allocator has blocks of this size to give
        _busy(torch.cuda.current_stream())
        old = torch.empty(want.numel(), dtype=torch.uint8, device="cuda")
        old.fill_(7)
        del old          # free for the current stream, whose fill is still to come
        got = model.quantize_experts(stream=side)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    model.close()


@pytest.mark.parametrize("to_bf16", [True, False], ids=["back to bf16", "to other matrices"])
def test_a_switch_does_not_touch_the_work_before_it(to_bf16):
    """A round enqueued on a side stream keeps its matrices and scratch, whatever is
    allocated after the switch; so do the rounds after it."""
    import discrete_diffusion_moe_b200 as dg
    cfg = dg.model_config(**TINY)
    model = dg.Model(cfg, 1, seed=0)
    n = dg.lib.dg_fp8_experts_scratch_bytes(model.ctx)
    kv, cv, out = dg.KVCache(cfg, 1, 512), dg.Canvas(cfg, 1), dg.StepOutputs(cfg, 1, logits=True)

    def step(stream):
        model.canvas_init(cv, 0, 7, stream=stream)
        model.step(kv, cv, 0, 0, dg.sampler_config(seed=7, max_steps=2), out, stream=stream)
    model.use_fp8_experts(model.quantize_experts())
    step(torch.cuda.current_stream())
    torch.cuda.synchronize()
    want = out.logits.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    _busy(side)
    step(side)
    other = None if to_bf16 else model.quantize_experts()
    model.use_fp8_experts(other)
    size = dg.lib.dg_fp8_experts_bytes(ctypes.byref(cfg))
    new = [torch.full((k,), 0x7F, dtype=torch.uint8, device="cuda") for k in (n, size, n, size)]
    torch.cuda.synchronize()
    assert torch.equal(out.logits, want)
    if not to_bf16:
        out.logits.zero_()
        step(torch.cuda.current_stream())
        assert torch.equal(out.logits, want)
    assert all(bool((t == 0x7F).all()) for t in new)
    model.check_device()
    model.close()


def test_refusals():
    import discrete_diffusion_moe_b200 as dg
    cfg = dg.model_config(**TINY)
    model = dg.Model(cfg, 1, seed=0)
    lib, n = dg.lib, dg.lib.dg_fp8_experts_bytes(ctypes.byref(cfg))
    s = lib.dg_fp8_experts_scratch_bytes(model.ctx)
    buf, scratch = torch.zeros(n + 256, dtype=torch.uint8, device="cuda"), torch.zeros(s + 256, dtype=torch.uint8, device="cuda")
    e, w = buf.data_ptr(), scratch.data_ptr()
    bad = dg.DG_ERR_INVALID_ARG
    assert lib.dg_fp8_experts_quantize(model.ctx, e, n - 1, None) == bad
    assert lib.dg_fp8_experts_quantize(model.ctx, e + 16, n, None) == bad
    assert lib.dg_fp8_experts_quantize(model.ctx, None, n, None) == bad
    assert lib.dg_fp8_experts_use(model.ctx, e, None, s) == bad
    assert lib.dg_fp8_experts_use(model.ctx, e + 16, w, s) == bad
    assert lib.dg_fp8_experts_use(model.ctx, e, w + 8, s) == bad
    assert lib.dg_fp8_experts_use(model.ctx, e, w, s - 1) == dg.DG_ERR_WORKSPACE
    with pytest.raises(ValueError):
        model.use_fp8_experts(buf[:n - 1])
    with pytest.raises(ValueError):
        model.use_fp8_experts(buf.view(torch.int8))
    model.close()


def test_experts_elsewhere_are_refused():
    import discrete_diffusion_moe_b200 as dg
    cfg = dg.model_config(**TINY)
    model = dg.Model(cfg, 1, seed=0)
    n = dg.lib.dg_fp8_experts_bytes(ctypes.byref(cfg))
    with pytest.raises(ValueError):
        model.use_fp8_experts(torch.zeros(n, dtype=torch.uint8))                         # host memory
    with pytest.raises(ValueError):
        model.use_fp8_experts(torch.zeros(2 * n, dtype=torch.uint8, device="cuda")[::2])  # every second byte
    model.close()
