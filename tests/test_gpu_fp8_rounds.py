"""Whole passes of a context on 8-bit experts.

Denoising rounds stage by stage, each stage on the GPU's own input to it
(tests/parity.py), with an oracle whose experts are the 8-bit operators'
definition in 64 bits: the context's bf16 matrices and each expert's input rows
quantised, the gate/up products rounded to bf16, SwiGLU and its rows quantised.
Every decision bit for bit except near ties, streams and logits within 2e-2.
(Not end to end: a value that is off by a relative d gets another code, up to 2^-3 of
itself away, with a probability of about 8 d, so two chains that differ by 5e-4, as those
of bf16 experts do, differ by about sqrt(8 d) 2^-3 = 0.8 % behind the first
quantiser and 3 % behind the second, rightly.)

Every other pass (encode, prefill, a round that appends a block, decoded
blocks, autoregressive steps): the last layer's expert block bit for bit the
public operators' on the pass's own rows."""

import numpy as np
import pytest
import torch

import fp8_ref as ref
import oracle
import synth
from oracle import model as OM
from oracle.numerics import bf16_round, f32_round
from parity import (TINY, Case, Report, gpu_layer_kv, gpu_sampler, tf_embedding, tf_expected_embedding, tf_layer_halves,
                    tf_lm_head, tf_router, tf_update, _sampler)
from test_gpu_fp8_experts import _buffer, _layer_views

pytestmark = pytest.mark.gpu


def _quantized_rows(x):
    q, s = ref.quantize_rows(x)
    return q * np.repeat(s.astype(np.float64).T, ref.BLOCK, axis=1)[:, :x.shape[1]]


def _quantized_blocks(w):
    q, s = ref.quantize_blocks(w)
    s = np.repeat(np.repeat(s.astype(np.float64), ref.BLOCK, axis=0), ref.BLOCK, axis=1)
    return q * s[:w.shape[0], :w.shape[1]]


@pytest.fixture
def oracle8(monkeypatch):
    """The oracle's experts by the 8-bit operators' definition."""
    matrices = {}

    def expert_ffn(x, wg, wu, wd):
        key = (wg.shape, wg[0, :4].tobytes(), wd[-1, -4:].tobytes())
        if key not in matrices:
            gu = np.empty((2 * wg.shape[0], wg.shape[1]))
            gu[0::2], gu[1::2] = wg, wu   # the layers' order: blocks of 128 rows hold both
            matrices[key] = _quantized_blocks(gu), _quantized_blocks(wd)
        w1, w2 = matrices[key]
        y = bf16_round(_quantized_rows(x) @ w1.T)
        return f32_round(_quantized_rows(OM.silu(y[:, 0::2]) * y[:, 1::2]) @ w2.T)
    monkeypatch.setattr(OM, "expert_ffn", expert_ffn)
    yield
    assert matrices


@pytest.mark.parametrize("case", [
    Case(cfg=TINY, ctx_len=64, steps=3),
    Case(cfg=TINY, self_cond=True, ctx_len=77, batch=2, steps=2),
    Case(cfg=dict(TINY, n_experts=4, d_ff=192), ctx_len=20, batch=8, steps=1),
    Case(cfg=dict(TINY, n_layers=1, d_model=320, n_experts=5, top_k=3, d_ff=64), ctx_len=30, steps=2),
    Case(cfg=TINY, ctx_len=300, steps=1, prefill=512)],
    ids=["steps", "selfcond", "many rows", "odd", "prefill"])
def test_rounds_stage_by_stage(oracle8, case):
    import discrete_diffusion_moe_b200 as dg
    rep = Report()
    c, B, V = case.cfg, case.batch, case.cfg["vocab"]
    L, d, T = c["n_layers"], c["d_model"], case.batch * 256
    ocfg = oracle.ModelConfig(**c, self_cond=case.self_cond)
    W = oracle.Weights(ocfg, seed=0)
    sc = _sampler(case)
    gcfg = dg.model_config(**c, self_cond=case.self_cond)
    model = dg.Model(gcfg, B, seed=0, prefill_tokens=case.prefill)
    model.use_fp8_experts(model.quantize_experts())
    gkv = dg.KVCache(gcfg, B, case.ctx_len + 256)
    model.encode(gkv, torch.from_numpy(synth.context_tokens(B, case.ctx_len, case.ctx_seed, V).astype(np.int32)).cuda())
    gcv = dg.Canvas(gcfg, B)
    model.canvas_init(gcv, case.block, sc.seed)
    kv = [gpu_layer_kv(gkv, l, case.ctx_len) for l in range(L)]
    for s in range(case.steps):
        tokens_in, prev_in = gcv.tokens.cpu().numpy(), gcv.prev_argmax.cpu().numpy()
        done_in, locked_in = gcv.done.cpu().numpy().astype(bool), gcv.locked.cpu().numpy().astype(bool)
        sc_in = gcv.sc_state.float().cpu().numpy().astype(np.float64)
        out = dg.StepOutputs(gcfg, B, logits=True, routing=True, hidden=True)
        model.step(gkv, gcv, case.block, s, gpu_sampler(dg, sc), out)
        model.check_device()
        gh, ga = out.hidden.cpu().numpy().astype(np.float64), out.hidden_attn.cpu().numpy().astype(np.float64)
        gi, gr = out.route_idx.cpu().numpy(), out.route_logits.cpu().numpy().astype(np.float64)
        gl = out.logits.cpu().numpy().reshape(T, V)
        tf_embedding(rep, ocfg, W, tokens_in, sc_in, gh[0])
        for l in range(L):
            tf_router(rep, ocfg, W.layer(l), l, ga[l], gi[l], gr[l])
            tf_layer_halves(rep, ocfg, W.layer(l), l, gh[l], ga[l], gh[l + 1], gi[l], *kv[l], case.ctx_len, B)
        flat = [t.cpu().numpy().reshape(T) for t in (out.argmax, out.sample)]
        stats = [t.cpu().numpy().astype(np.float64).reshape(T) for t in (out.entropy, out.pmax)]
        tf_lm_head(rep, ocfg, W, sc, gh[L], gl, *flat, *stats, case.block, s, np.arange(T), B)
        tf_update(rep, ocfg, sc, out, tokens_in, prev_in, done_in, gcv.tokens.cpu().numpy(), case.block, s, locked_in,
                  gcv.locked.cpu().numpy())
        live = np.nonzero(np.repeat(~done_in, 256))[0]
        if case.self_cond and live.size:
            ge = gcv.sc_state.float().cpu().numpy().astype(np.float64).reshape(T, d)
            tf_expected_embedding(rep, W, gl[live], ge[live], live)
    assert rep.tf_decisions > 0 and rep.tf_moe_rel > 0.0
    print(rep)
    model.close()


def _check_last_expert_block(dg, model, cfg, experts, rows):
    """The last pass's last expert block, of `rows` (token, expert) rows."""
    w1, s1, w2, s2 = _layer_views(cfg, experts, cfg.n_layers - 1)
    x = _buffer(dg, model, "xperm", torch.bfloat16, (rows, cfg.d_model))
    off = _buffer(dg, model, "off", torch.int32, (cfg.n_experts + 1,))
    rw = _buffer(dg, model, "wperm", torch.float32, (rows,))
    got = _buffer(dg, model, "yperm", torch.float32, (rows, cfg.d_model))
    assert int(off[-1]) == rows
    q, s = dg.fp8_quantize(x)
    h, hs = dg.fp8_quantize(dg.fp8_grouped_gemm(q, s, w1, s1, off), act="swiglu_interleaved")
    assert torch.equal(got, dg.fp8_grouped_gemm(h, hs, w2, s2, off, row_weight=rw, out_dtype=torch.float32))
    assert torch.isfinite(got).all() and got.abs().max() > 0


@pytest.mark.parametrize("prefill", [0, 2048])
@pytest.mark.parametrize("B", [1, 2])
def test_every_pass_runs_the_operators(B, prefill):
    import discrete_diffusion_moe_b200 as dg
    cfg = dg.model_config(**TINY)
    k = cfg.top_k
    model = dg.Model(cfg, B, seed=0, prefill_tokens=prefill or 512 * B)
    experts = model.quantize_experts()
    model.use_fp8_experts(experts)
    sampler = dg.sampler_config(seed=3, max_steps=3)
    kv, cv = dg.KVCache(cfg, B, 4096), dg.Canvas(cfg, B)
    chunk = max(256, max(prefill, 512 * B) // B)
    for n in (1, 37, chunk):   # one token a canvas, an odd count, a whole pass
        model.encode(kv, torch.from_numpy(synth.context_tokens(B, n, n, cfg.vocab).astype(np.int32)).cuda())
        model.check_device()
        _check_last_expert_block(dg, model, cfg, experts, B * n * k)
    kv = dg.KVCache(cfg, B, 2048)
    model.encode(kv, torch.from_numpy(synth.context_tokens(B, 37, 37, cfg.vocab).astype(np.int32)).cuda())
    block = torch.zeros(B, 256, dtype=torch.int32, device="cuda")
    model.decode_block(kv, cv, 0, sampler, block, defer_append=True)
    _check_last_expert_block(dg, model, cfg, experts, B * 256 * k)
    model.canvas_init(cv, 1, 3)
    model.step_append(kv, cv, 1, 0, sampler, block)
    model.check_device()
    assert kv.length == 37 + 256
    _check_last_expert_block(dg, model, cfg, experts, B * 512 * k)
    token = block[:, -1].contiguous()
    amax, samp = torch.zeros_like(token), torch.zeros_like(token)
    for _ in range(2):
        model.ar_step(kv, token, 0.8, 3, amax, samp)
        model.check_device()
        _check_last_expert_block(dg, model, cfg, experts, B * k)
    model.close()
