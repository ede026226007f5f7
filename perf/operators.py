"""Cases, inputs and plain forms of the 8-bit operators: the block-scaled
product (dense and grouped by expert) and the quantiser of its operands.

Formats.  Activations: e4m3 codes [rows, K], one fp32 scale for each row and
block of 128 columns, stored [ceil(K / 128), rows].  Weights: e4m3 codes
[N, K] (or [G, N, K]), one fp32 scale for each 128 x 128 block, stored
[ceil(N / 128), ceil(K / 128)] (or with G in front).  Rows of codes start
every multiple of 16 bytes.
"""

import math
import random

import numpy as np
import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
AMAX_MIN = 2.0 ** -100
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp16": 2, "fp32": 4}


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


# ---- the cases ---------------------------------------------------------------

def listed():
    return [
        # one token's normed hidden state before its projections (autoregressive mode)
        dict(name="quantize 1 token", op="quantize", form="rows", rows=1, K=2816, dtype="bf16"),
        # a canvas's 256 tokens gathered into expert order, 8 experts each
        dict(name="quantize gathered canvas", op="quantize", form="gather", rows=2048, src=256, K=2816, dtype="bf16"),
        # 16 canvases after the gate/up product: SwiGLU and the down product's operand
        dict(name="quantize swiglu 16 canvases", op="quantize", form="swiglu_interleaved", rows=32768, K=704, dtype="bf16"),
        # loading a model: the gate/up matrices of 16 experts (of 128), one after the other in one call
        dict(name="quantize weights", op="quantize", form="blocks", G=16, rows=1408, K=2816, dtype="bf16"),
        # one token through the QKV projection
        dict(name="gemm 1 token", op="gemm", M=1, N=5632, K=2816, out="bf16"),
        # a canvas through the QKV projection
        dict(name="gemm canvas", op="gemm", M=256, N=5632, K=2816, out="bf16"),
        # a long prompt (odd length) through the QKV projection
        dict(name="gemm prompt", op="gemm", M=8191, N=5632, K=2816, out="bf16"),
        # a canvas through the LM head, logits in fp32
        dict(name="gemm lm head", op="gemm", M=256, N=262144, K=2816, out="fp32"),
        # one token's 8 experts, gate/up
        dict(name="grouped 1 token", op="grouped", rows=8, G=128, active=8, N=1408, K=2816, out="bf16", weighted=False),
        # a canvas, 256 tokens on 84 distinct experts, gate/up
        dict(name="grouped canvas", op="grouped", rows=2048, G=128, active=84, N=1408, K=2816, out="bf16", weighted=False),
        # the same canvas's down product with the routing weights, fp32 for the combine; K ends inside a block
        dict(name="grouped canvas down", op="grouped", rows=2048, G=128, active=84, N=2816, K=704, out="fp32", weighted=True),
        # 16 canvases, gate/up
        dict(name="grouped 16 canvases", op="grouped", rows=32768, G=128, active=128, N=1408, K=2816, out="bf16", weighted=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "gemm", "gemm", "grouped", "grouped"])
    dtype = rng.choice(["bf16", "fp16", "fp32"])
    out = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "quantize":
        form = rng.choice(["rows", "gather", "swiglu", "swiglu_interleaved", "blocks"])
        K = _log_int(rng, 64, 8192)
        rows = _log_int(rng, 1, max(1, min(32768, (1 << 26) // K)))
        case = dict(op=op, form=form, rows=rows, K=K, dtype=dtype)
        if form == "gather":
            case["src"] = _log_int(rng, 1, 4096)
        if form == "blocks":
            case["G"] = rng.randint(1, max(1, min(16, (1 << 26) // (rows * K))))
        return case
    K = _log_int(rng, 64, 8192)
    if op == "gemm":
        N = _log_int(rng, 16, 16384)
        M = _log_int(rng, 1, max(1, min(8192, 130_000_000_000 // (N * K))))
        return dict(op=op, M=M, N=N, K=K, out=out)
    G = _log_int(rng, 1, 128)
    N = _log_int(rng, 16, max(16, min(8192, 400_000_000 // (G * K))))
    rows = _log_int(rng, 1, max(1, min(32768, 130_000_000_000 // (N * K))))
    return dict(op=op, rows=rows, G=G, active=rng.randint(1, min(G, rows)), N=N, K=K, out=out, weighted=rng.random() < 0.5)


# ---- inputs --------------------------------------------------------------------

def _padded(rows, K):
    """Codes with rows on 16-byte boundaries: a [*rows, K] view of a wider buffer."""
    return torch.zeros(*rows, (K + 15) // 16 * 16, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)[..., :K]


def _hidden(gen, rows, K, dtype):
    """Normed hidden states: about N(0, 1), a few columns ten times larger."""
    x = torch.randn(rows, K, generator=gen, device="cuda")
    x[:, torch.randint(0, K, (max(1, K // 256),), generator=gen, device="cuda")] *= 10.0
    return x.to(TYPES[dtype])


def _codes(x, scale):
    return (x / scale).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _activations(gen, rows, K):
    """An operand as a program holds it after quantising: codes and scales."""
    KB = _blocks(K)
    x = torch.zeros(rows, KB * BLOCK, device="cuda")
    x[:, :K] = _hidden(gen, rows, K, "fp32")
    x = x.view(rows, KB, BLOCK)
    scale = x.abs().amax(-1, keepdim=True).clamp_(min=AMAX_MIN) / E4M3_MAX
    q = _padded((rows,), K)
    q.copy_(_codes(x, scale).view(rows, KB * BLOCK)[:, :K])
    return q, scale[:, :, 0].t().contiguous()


def _weights(gen, G, N, K):
    """Weights N(0, 0.02) in 8 bits with their block scales."""
    NB, KB = _blocks(N), _blocks(K)
    q = _padded((G, N), K)
    scale = torch.empty(G, NB, KB, device="cuda")
    step = max(1, (1 << 28) // (NB * KB * BLOCK * BLOCK))
    for g in range(0, G, step):
        n = min(step, G - g)
        w = torch.zeros(n, NB * BLOCK, KB * BLOCK, device="cuda")
        w[:, :N, :K] = torch.randn(n, N, K, generator=gen, device="cuda").mul_(0.02)
        w = w.view(n, NB, BLOCK, KB, BLOCK)
        s = w.abs().amax((2, 4), keepdim=True).clamp_(min=AMAX_MIN) / E4M3_MAX
        q[g:g + n] = _codes(w, s).view(n, NB * BLOCK, KB * BLOCK)[:, :N, :K]
        scale[g:g + n] = s[:, :, 0, :, 0]
    return q, scale


def _group_sizes(case, seed):
    """Rows of each group: `active` groups of uneven popularity, the others empty."""
    rng = random.Random(seed * 7919 + 17)
    G, active, rows = case["G"], case["active"], case["rows"]
    chosen = sorted(rng.sample(range(G), active))
    share = np.array([rng.lognormvariate(0.0, 0.5) for _ in chosen])
    sizes = np.zeros(G, dtype=np.int64)
    sizes[chosen] = 1 + np.random.RandomState(rng.randrange(1 << 31)).multinomial(rows - active, share / share.sum())
    return sizes


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    state = dict(case=dict(case))
    if op == "quantize":
        form, rows, K, dtype = case["form"], case["rows"], case["K"], case["dtype"]
        if form == "blocks":
            state["x"] = (torch.randn(case["G"], rows, K, generator=gen, device="cuda") * 0.02).to(TYPES[dtype])
        elif form == "gather":
            state["x"] = _hidden(gen, case["src"], K, dtype)
            state["index"] = torch.randint(0, case["src"], (rows,), generator=gen, device="cuda", dtype=torch.int32)
        else:
            state["x"] = _hidden(gen, rows, K if form == "rows" else 2 * K, dtype)
    elif op == "gemm":
        state["a"], state["sa"] = _activations(gen, case["M"], case["K"])
        b, sb = _weights(gen, 1, case["N"], case["K"])
        state["b"], state["sb"] = b[0], sb[0]
    else:
        sizes = _group_sizes(case, seed)
        state["a"], state["sa"] = _activations(gen, case["rows"], case["K"])
        state["b"], state["sb"] = _weights(gen, case["G"], case["N"], case["K"])
        state["off"] = torch.from_numpy(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)).cuda()
        # the plain form's groups (those that have rows) and its padding
        state["groups"], state["most"] = torch.from_numpy(np.flatnonzero(sizes)).cuda(), int(sizes.max())
        state["row_weight"] = torch.rand(case["rows"], generator=gen, device="cuda") if case["weighted"] else None
    return state


# ---- the plain forms -------------------------------------------------------------

def _act(x, form, K):
    if form == "swiglu":
        g, u = x[:, :K].float(), x[:, K:].float()
    elif form == "swiglu_interleaved":
        g, u = x[:, 0::2].float(), x[:, 1::2].float()
    else:
        return x.float()
    return g / (1.0 + torch.exp(-g)) * u


def _plain_rows(x, K):
    rows, KB = x.shape[0], _blocks(K)
    x = torch.nn.functional.pad(x, (0, KB * BLOCK - K)).view(rows, KB, BLOCK)
    amax = x.abs().amax(-1, keepdim=True).clamp(min=AMAX_MIN)
    q = (x * (E4M3_MAX / amax)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.view(rows, KB * BLOCK)[:, :K], (amax[:, :, 0] / E4M3_MAX).t()


def _plain_blocks(w, K):
    G, N = w.shape[:2]
    NB, KB = _blocks(N), _blocks(K)
    w = torch.nn.functional.pad(w.float(), (0, KB * BLOCK - K, 0, NB * BLOCK - N)).view(G, NB, BLOCK, KB, BLOCK)
    amax = w.abs().amax((2, 4), keepdim=True).clamp(min=AMAX_MIN)
    q = (w * (E4M3_MAX / amax)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.view(G, NB * BLOCK, KB * BLOCK)[:, :N, :K], amax[:, :, 0, :, 0] / E4M3_MAX


def _a_values(a, sa):
    return a.float() * sa.t().repeat_interleave(BLOCK, 1)[:, :a.shape[1]]


def _b_values(b, sb):
    N, K = b.shape[-2:]
    return b.float() * sb.repeat_interleave(BLOCK, -2)[..., :N, :].repeat_interleave(BLOCK, -1)[..., :K]


def _plain_grouped(s):
    case, a, off = s["case"], _a_values(s["a"], s["sa"]), s["off"].long()
    row = torch.arange(case["rows"], device=a.device)
    groups = s["groups"]
    group = torch.searchsorted(off[groups + 1], row, right=True)
    at = row - off[groups[group]]
    padded = torch.zeros(len(groups), s["most"], case["K"], device=a.device)
    padded[group, at] = a
    b = s["b"].view(torch.uint8)[groups].view(torch.float8_e4m3fn)
    out = torch.bmm(padded, _b_values(b, s["sb"][groups]).transpose(1, 2))[group, at]
    if s["row_weight"] is not None:
        out = out * s["row_weight"][:, None]
    return out.to(TYPES[case["out"]])


def run(state):
    case, op = state["case"], state["case"]["op"]
    if own:
        import discrete_diffusion_moe_b200 as dg
        if op == "quantize":
            form = case["form"]
            if form == "blocks":
                return dg.fp8_quantize_blocks(state["x"])
            if form == "gather":
                return dg.fp8_quantize(state["x"], index=state["index"])
            return dg.fp8_quantize(state["x"], act=None if form == "rows" else form)
        if op == "gemm":
            return dg.fp8_gemm(state["a"], state["sa"], state["b"], state["sb"], out_dtype=TYPES[case["out"]])
        return dg.fp8_grouped_gemm(state["a"], state["sa"], state["b"], state["sb"], state["off"],
                                   row_weight=state["row_weight"], out_dtype=TYPES[case["out"]])
    if op == "quantize":
        form, K = case["form"], case["K"]
        if form == "blocks":
            return _plain_blocks(state["x"], K)
        if form == "gather":
            return _plain_rows(state["x"][state["index"].long()].float(), K)
        return _plain_rows(_act(state["x"], form, K), K)
    if op == "gemm":
        return (_a_values(state["a"], state["sa"]) @ _b_values(state["b"], state["sb"]).t()).to(TYPES[case["out"]])
    return _plain_grouped(state)


# ---- what a pass cannot do without ------------------------------------------------

def work(case):
    K = case["K"]
    if case["op"] == "quantize":
        form, rows, size = case["form"], case["rows"], SIZES[case["dtype"]]
        if form == "blocks":
            n = case["G"] * rows * K
            return dict(bytes=n * (size + 1) + 4 * case["G"] * _blocks(rows) * _blocks(K), flops=2 * n)
        written = rows * K + 4 * rows * _blocks(K)
        if form == "gather":
            return dict(bytes=min(rows, case["src"]) * K * size + 4 * rows + written, flops=2 * rows * K)
        if form == "rows":
            return dict(bytes=rows * K * size + written, flops=2 * rows * K)
        return dict(bytes=2 * rows * K * size + written, flops=7 * rows * K)
    M, G = (case["M"], 1) if case["op"] == "gemm" else (case["rows"], case["active"])
    N = case["N"]
    scales = 4 * (M * _blocks(K) + G * _blocks(N) * _blocks(K))
    return dict(bytes=M * K + G * N * K + scales + M * N * SIZES[case["out"]], flops=2 * M * N * K)


# ---- the definitions in 64 bits -----------------------------------------------------

def _exact_codes(x, amax):
    """Codes and scales of blocks x [..., n] in 64 bits.  The definition holds
    448 / amax and the product in 32 bits."""
    inv = (E4M3_MAX / amax).float().double()
    v = (x * inv).float().double().clamp(-E4M3_MAX, E4M3_MAX)
    # e4m3: 4 significant bits down to 2^-6, steps of 2^-9 below; ties to even
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(v / step) * step, amax / E4M3_MAX


def exact(case, seed):
    s = prepare(case, seed)
    K, KB = case["K"], _blocks(case["K"])
    edges = [(k * BLOCK, min(K, k * BLOCK + BLOCK)) for k in range(KB)]
    if case["op"] == "quantize":
        form, x = case["form"], s["x"].double()
        if form == "blocks":
            G, N = x.shape[:2]
            q, scale = torch.empty_like(x), torch.empty(G, _blocks(N), KB, dtype=torch.float64, device=x.device)
            for r in range(_blocks(N)):
                rows = slice(r * BLOCK, min(N, r * BLOCK + BLOCK))
                for k, (lo, hi) in enumerate(edges):
                    part = x[:, rows, lo:hi]
                    v, sc = _exact_codes(part, part.abs().amax((1, 2), keepdim=True).clamp(min=AMAX_MIN))
                    q[:, rows, lo:hi], scale[:, r, k] = v, sc[:, 0, 0]
            return q, scale
        if form == "gather":
            x = torch.index_select(x, 0, s["index"].long())
        elif form == "swiglu":
            x = torch.sigmoid(x[:, :K]) * x[:, :K] * x[:, K:]
        elif form == "swiglu_interleaved":
            x = x.view(-1, K, 2)
            x = torch.sigmoid(x[..., 0]) * x[..., 0] * x[..., 1]
        q, scale = torch.empty_like(x), torch.empty(KB, x.shape[0], dtype=torch.float64, device=x.device)
        for k, (lo, hi) in enumerate(edges):
            v, sc = _exact_codes(x[:, lo:hi], x[:, lo:hi].abs().amax(1, keepdim=True).clamp(min=AMAX_MIN))
            q[:, lo:hi], scale[k] = v, sc[:, 0]
        return q, scale

    def product(a, sa, b, sb):
        """sum over blocks of sa sb (A B^T), block by block."""
        out = torch.zeros(a.shape[0], b.shape[0], dtype=torch.float64, device=a.device)
        block = torch.arange(b.shape[0], device=a.device) // BLOCK
        for k, (lo, hi) in enumerate(edges):
            out += (a[:, lo:hi].double() @ b[:, lo:hi].double().t()) * sa[k].double()[:, None] * sb[block, k].double()
        return out

    if case["op"] == "gemm":
        return product(s["a"], s["sa"], s["b"], s["sb"])
    off = s["off"].tolist()
    out = torch.zeros(case["rows"], case["N"], dtype=torch.float64, device="cuda")
    for g in range(case["G"]):
        if off[g + 1] > off[g]:
            rows = slice(off[g], off[g + 1])
            out[rows] = product(s["a"][rows], s["sa"][:, rows], s["b"][g], s["sb"][g])
    return out if s["row_weight"] is None else out * s["row_weight"].double()[:, None]
