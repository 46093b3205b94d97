"""Measured cases of the 8-bit projections: RMSNorm with the residual's addition and
quantisation of rows to e4m3 with one power-of-two scale per 128 columns, the product
of such rows with e4m3 weights that have one scale per block of 128 x 128, and the
gated half of the MLP, SiLU(x·W1) * (x·W3), from and to e4m3 rows.

With ``own`` false, ``run`` computes each operator in elementary torch operations in
fp32; with ``own`` true it calls the framework."""
import math

import torch

own = False

BLOCK = 128
E_MIN, E_MAX = -100, 120        # exponents of a block's power-of-two scale
EPS = 1e-5
BF16, F32, CODE, SCALE = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.float8_e8m0fnu


def listed():
    return [
        # -- RMSNorm, the residual's addition on the way, to e4m3
        # one token's row between two projections of the 4096-wide block: all latency
        _norm("norm_one", M=1, d=4096, x="bf16", r="bf16"),
        # an odd batch of prompts of the 768-wide block, the residual stream in fp32
        _norm("norm_odd", M=3777, d=768, x="f32", r="bf16"),
        # the benchmark's prefill, 4 x 8192 tokens: memory rate
        _norm("norm_chunk", M=32768, d=4096, x="bf16", r="bf16"),
        # -- quantisation alone: the attention's output before its projection
        # a decode step of 32 sequences
        _quant("quant_step", M=32, d=4096, x="bf16"),
        # a prompt of 8192 tokens of the 11008-wide gated branch, held in fp32
        _quant("quant_chunk", M=8192, d=11008, x="f32"),
        # -- the product
        # one token through the fused q, k, v projection of 32 + 2·8 heads of 128: the weights' stream
        _gemm("gemm_one", M=1, N=6144, K=4096),
        # a decode step of 32 tokens through the MLP's second projection, added to the residual stream
        _gemm("gemm_step", M=32, N=4096, K=14336, res=True),
        # an odd chunk through the q, k, v projection of the 12-head block
        _gemm("gemm_odd", M=1371, N=2304, K=768, y="f32"),
        # a prompt's 16384 tokens through the second projection, added to the stream: matrix instructions
        _gemm("gemm_chunk", M=16384, N=4096, K=14336, res=True),
        # -- both first projections of the MLP, the activation and the product
        # a decode step of 32 tokens
        _gated("gated_step", M=32, N=14336, K=4096),
        # a few hundred tokens of the 768-wide block, the result kept in bf16
        _gated("gated_odd", M=333, N=2048, K=768, y="bf16"),
        # a prompt of 8192 tokens
        _gated("gated_chunk", M=8192, N=14336, K=4096),
    ]


def _norm(name, M, d, x, r):
    return dict(name=name, op="norm", M=M, N=d, K=d, x=x, r=r, res=False, y="e4m3")


def _quant(name, M, d, x):
    return dict(name=name, op="quant", M=M, N=d, K=d, x=x, r="", res=False, y="e4m3")


def _gemm(name, M, N, K, res=False, y="bf16"):
    return dict(name=name, op="gemm", M=M, N=N, K=K, x="e4m3", r="", res=res, y=y)


def _gated(name, M, N, K, y="e4m3"):
    return dict(name=name, op="gated", M=M, N=N, K=K, x="e4m3", r="", res=False, y=y)


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "quant", "gemm", "gemm", "gated", "gated"])
    step = rng.choice([16, 16, 64, 128])

    def width(lo, hi):
        return max(step, _log(rng, lo, hi) // step * step)

    if op in ("norm", "quant"):
        d = width(64, 16384)
        M = max(1, min(_log(rng, 1, 32768), 120_000_000 // d))
        x = rng.choice(["bf16", "bf16", "f32"])
        c = _quant("drawn", M, d, x) if op == "quant" else _norm("drawn", M, d, x, rng.choice(["", "bf16", "bf16", "f32"]))
    else:
        N, K = width(64, 14336), width(64, 14336)
        M = _log(rng, 1, 16384)
        if rng.random() < 0.3:
            M = rng.randint(1, 300)
        M = max(1, min(M, 400_000_000_000 // (N * K)))
        c = _gemm("drawn", M, N, K, rng.random() < 0.5, rng.choice(["bf16", "bf16", "f32"])) if op == "gemm" else \
            _gated("drawn", M, N, K, rng.choice(["e4m3", "e4m3", "bf16"]))
    del c["name"]
    return c


# ---- sizes of a case -------------------------------------------------------

def _blocks(n):
    return -(-n // BLOCK)


def _bytes(kind):
    return {"": 0, "e4m3": 1, "bf16": 2, "f32": 4}[kind]


def work(case):
    c = case
    M, N, K = c["M"], c["N"], c["K"]
    if c["op"] in ("norm", "quant"):
        through = _bytes(c["x"]) * (2 if c["r"] else 1) + _bytes(c["r"])       # x, the sum, r
        return {"bytes": M * K * (through + 1) + M * _blocks(K) + (K * _bytes(c["x"]) if c["op"] == "norm" else 0),
                "flops": (6 if c["op"] == "norm" else 2) * M * K}
    mats = 2 if c["op"] == "gated" else 1
    out = _bytes(c["y"]) * (2 if c["res"] else 1)
    return {"bytes": M * (K + _blocks(K)) + mats * (N * K + _blocks(N) * _blocks(K)) + M * N * out
            + (M * _blocks(N) if c["y"] == "e4m3" else 0), "flops": 2 * mats * M * N * K}


# ---- inputs ----------------------------------------------------------------

def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    M, N, K = c["M"], c["N"], c["K"]
    kinds = {"bf16": BF16, "f32": F32}

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    s = {"case": c}
    if c["op"] in ("norm", "quant"):
        x = randn(M, K)
        x[:, torch.randint(0, K, (1 + K // 512,), generator=g, device=dev)] *= 20        # a few large channels, as streams have
        s["x"] = x.to(kinds[c["x"]])
        s["codes"], s["scale"] = _empty(M, K, dev)
        if c["op"] == "norm":
            s["g"] = (1 + 0.1 * randn(K)).to(kinds[c["x"]])
            s["r"] = (0.5 * randn(M, K)).to(kinds[c["r"]]) if c["r"] else None
            s["h"] = torch.zeros(M, K, dtype=kinds[c["x"]], device=dev) if c["r"] else None
    else:
        s["x"], s["x_scale"] = _rows_of(randn(M, K))
        for name in ("w", "w3")[:2 if c["op"] == "gated" else 1]:
            s[name], s[name + "_scale"] = _weights_of(randn(N, K).mul_(0.02))
        s["res"] = randn(M, N).to(kinds[c["y"]]) if c["res"] else None
        if c["y"] == "e4m3":
            s["codes"], s["scale"] = _empty(M, N, dev)
        else:
            s["y"] = torch.zeros(M, N, dtype=kinds[c["y"]], device=dev)
    if own:
        import causal_gqa_attention_rmsnorm_gb300 as tb
        if c["op"] in ("gemm", "gated"):
            s["x8"] = tb.E4M3Rows(s["x"], s["x_scale"])
            for name in ("w", "w3")[:2 if c["op"] == "gated" else 1]:
                s[name + "8"] = tb.E4M3Weight(s[name], s[name + "_scale"])
        if c["y"] == "e4m3":
            s["out"] = tb.E4M3Rows(s["codes"], s["scale"])
    return s


def _empty(M, n, dev):
    return (torch.zeros(M, n, dtype=torch.uint8, device=dev).view(CODE),
            torch.zeros(M, _blocks(n), dtype=torch.uint8, device=dev).view(SCALE))


# ---- the operators ---------------------------------------------------------

def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        import causal_gqa_attention_rmsnorm_gb300 as tb
        if op == "norm":
            tb.tb_rmsnorm_e4m3(s["x"], s["g"], EPS, r=s["r"], h=s["h"], out=s["out"])
        elif op == "quant":
            tb.tb_quant_e4m3(s["x"], out=s["out"])
        elif op == "gemm":
            tb.tb_gemm_e4m3(s["x8"], s["w8"], res=s["res"], y=s["y"])
        else:
            tb.tb_gated_e4m3(s["x8"], s["w8"], s["w38"], out=s["out"] if s["case"]["y"] == "e4m3" else s["y"])
    else:
        _plain(s, op)
    if op == "norm" and s["h"] is not None:
        return {"codes": s["codes"], "scale": s["scale"], "h": s["h"]}
    return {"codes": s["codes"], "scale": s["scale"]} if s["case"]["y"] == "e4m3" else s["y"]


def _plain(s, op):
    if op in ("norm", "quant"):
        v = s["x"].float()
        if op == "norm":
            if s["r"] is not None:
                v = v + s["r"].float()
                s["h"].copy_(v)
            v = v / torch.sqrt(v.square().mean(-1, keepdim=True) + EPS) * s["g"].float()
    else:
        x = _values(s["x"], s["x_scale"], 1)
        v = x @ _values(s["w"], s["w_scale"], BLOCK).T
        if op == "gated":
            v = v / (1 + torch.exp(-v)) * (x @ _values(s["w3"], s["w3_scale"], BLOCK).T)
        elif s["res"] is not None:
            v = v + s["res"].float()
    if s["case"]["y"] == "e4m3":
        codes, scale = _rows_of(v)
        s["codes"].copy_(codes)
        s["scale"].copy_(scale)
    else:
        s["y"].copy_(v)


def _values(codes, scale, rows):
    """The fp32 values of codes [n, K] with a scale for each block of `rows` x BLOCK."""
    n, K = codes.shape
    f = scale.float().repeat_interleave(rows, 0)[:n] if rows > 1 else scale.float()
    return codes.float() * f.repeat_interleave(BLOCK, 1)[:, :K]


def _exponent(top):
    m, e = torch.frexp(top)                                                    # top = m 2^e, m in [1/2, 1)
    return torch.where(top > 0, e - 9 + (m > 0.875), E_MIN).clamp(E_MIN, E_MAX)  # 448 = 0.875 * 2^9


def _coded(blocks, e):
    return (blocks * torch.exp2(-e.float())).clamp(-448, 448).to(CODE)


def _scales(e):
    return (e + 127).to(torch.uint8).view(SCALE)


def _rows_of(v):
    """Codes [M, n] and scales [M, blocks] of fp32 rows, a scale for BLOCK columns of a row."""
    M, n = v.shape
    blocks = torch.nn.functional.pad(v, (0, -n % BLOCK)).view(M, -1, BLOCK)
    e = _exponent(blocks.abs().amax(-1))
    codes = _coded(blocks, e[..., None]).view(torch.uint8).view(M, -1)[:, :n].contiguous()
    return codes.view(CODE), _scales(e)


def _weights_of(w):
    """Codes [N, K] and scales [N blocks, K blocks] of fp32 weights."""
    N, K = w.shape
    blocks = torch.nn.functional.pad(w, (0, -K % BLOCK, 0, -N % BLOCK)).unflatten(0, (-1, BLOCK)).unflatten(2, (-1, BLOCK))
    e = _exponent(blocks.abs().amax((1, 3)))
    codes = _coded(blocks, e[:, None, :, None]).view(torch.uint8).flatten(2, 3).flatten(0, 1)[:N, :K].contiguous()
    return codes.view(CODE), _scales(e)


# ---- the same in 64 bits ---------------------------------------------------

def exact(case, seed):
    """Outputs in 64 bits; codes as the quotients that are rounded to 8 bits."""
    s = prepare(case, seed)
    f64, op = torch.float64, case["op"]
    h = None
    if op in ("norm", "quant"):
        z = s["x"].to(f64)
        if op == "norm":
            if s["r"] is not None:
                z = h = z + s["r"].to(f64)
            z = s["g"].to(f64) * z * torch.rsqrt((z * z).sum(1, keepdim=True) / z.shape[1] + EPS)
    else:
        def product(w, ws):
            total = torch.zeros(case["M"], case["N"], dtype=f64, device=s["x"].device)
            for b in range(_blocks(case["K"])):            # one block of the reduction at a time
                at = slice(b * BLOCK, (b + 1) * BLOCK)
                part = s["x"][:, at].float().to(f64) @ w[:, at].float().to(f64).T
                cols = torch.arange(case["N"], device=part.device) // BLOCK
                total += part * s["x_scale"][:, b].double()[:, None] * ws[:, b].double()[cols][None]
            return total

        z = product(s["w"], s["w_scale"])
        if op == "gated":
            z = torch.sigmoid(z) * z * product(s["w3"], s["w3_scale"])
        elif s["res"] is not None:
            z = z + s["res"].to(f64)
    if case["y"] != "e4m3":
        return z
    width = z.shape[1]
    top = torch.stack([z[:, i:i + BLOCK].abs().amax(1) for i in range(0, width, BLOCK)], 1)
    steps = torch.tensor([2.0 ** e for e in range(E_MIN, E_MAX + 1)], dtype=f64, device=z.device)
    step = steps[torch.searchsorted(448 * steps, top).clamp_(max=len(steps) - 1)]    # the least that holds the largest
    out = {"codes": z / step.repeat_interleave(BLOCK, 1)[:, :width], "scale": step}
    return {**out, "h": h} if op == "norm" and case["r"] else out
