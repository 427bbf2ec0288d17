"""The cases on which the block operators are measured: the linear layer with
4-bit weights and group scales (``w4_linear``), the norms around a block with
its gate and residual scale (``block_norm``) and the gated activation between
the two halves of an MLP (``glu_act``).

``own`` false: ``run`` is the plain form, elementary torch operations in fp32
(statistics and the gated activation in fp64: their results are rounded to
INT8 codes, and an fp32 sum moves values across the rounding borders).
``own`` true: ``run`` calls the library.
"""
from __future__ import annotations

import math

import torch

own = False

# Sizes are those of the repository's workloads (4096 -> 14336 MLP, 1024-wide
# key/value projection, 128256-entry vocabulary, 1280-wide vision encoder at
# 1601 tokens, prefill of 2048) and ragged ones.


def _w4(name, M, K, N, group, zeros, out):
    return dict(name=name, op="w4", M=M, K=K, N=N, group=group, zeros=zeros, out=out)


def _norm(name, M, K, h, branch, kind, post, gate, scale, out):
    return dict(name=name, op="norm", M=M, K=K, h=h, branch=branch, kind=kind, post=post, gate=gate,
                residual_scale=scale, out=out)


def _glu(name, M, K, dtype, fused, out):
    return dict(name=name, op="glu", M=M, K=K, dtype=dtype, fused=fused, out=out)


def listed():
    return [
        # key / value projection of one decoded token: the smallest matrix, latency counts
        _w4("w4-kv-1", 1, 4096, 1024, 128, False, "f32"),
        # gate or up projection of one decoded token: one read of the weights
        _w4("w4-up-1", 1, 4096, 14336, 64, False, "f32"),
        # the vocabulary projection for the 8 positions of a drafted continuation
        _w4("w4-vocab-8", 8, 4096, 128256, 128, False, "f32"),
        # a short ragged prompt, columns that end inside a group, zero points, small groups
        _w4("w4-ragged-21", 21, 1296, 1003, 32, True, "f32"),
        # vision encoder, MLP down-projection: few outputs, long rows
        _w4("w4-vision-1601", 1601, 5120, 1280, 128, True, "bf16"),
        # prefill of 2048 tokens: the largest product
        _w4("w4-prefill-2048", 2048, 4096, 14336, 64, False, "bf16"),
        # one decoded token between attention and MLP: residual add, norm, codes
        _norm("norm-decode-1", 1, 4096, "f32", "f32", "rms", False, "none", 1.0, "codes"),
        # prefill with a norm after the block as well and a scaled residual
        _norm("norm-prefill-2048", 2048, 4096, "bf16", "bf16", "rms", True, "none", 0.5, "codes"),
        # vision encoder layer: LayerNorm, the block's output through a tanh gate
        _norm("norm-vision-1601", 1601, 1280, "f32", "bf16", "layer", False, "tanh", 1.0, "bf16"),
        # gated activation of one decoded token
        _glu("glu-decode-1", 1, 14336, "f32", False, "codes"),
        # a few drafted tokens, gate and up as the halves of one matrix, ragged width
        _glu("glu-ragged-5", 5, 1744, "bf16", True, "f32"),
        # prefill: gate and up of 2048 tokens
        _glu("glu-prefill-2048", 2048, 14336, "bf16", True, "codes"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["w4", "w4", "norm", "glu"])
    if op == "w4":
        while True:
            M, K, N = _log(rng, 1, 2048), 16 * _log(rng, 4, 896), _log(rng, 16, 128256)
            # no dearer than the prefill product or the vocabulary matrix
            if M * K * N <= 2048 * 4096 * 14336 and K * N <= 4096 * 14336:
                break
        return _w4("", M, K, N, rng.choice([32, 64, 96, 128, 256]), rng.random() < 0.5, rng.choice(["f32", "bf16"]))
    if op == "norm":
        while True:
            M, K = _log(rng, 1, 8192), 16 * _log(rng, 4, 896)
            if M * K <= 2048 * 4096:
                break
        return _norm("", M, K, rng.choice(["f32", "bf16"]), rng.choice(["f32", "bf16"]), rng.choice(["rms", "layer"]),
                     rng.random() < 0.5, rng.choice(["none", "scalar", "tanh", "channel"]), rng.choice([1.0, 0.5]),
                     rng.choice(["codes", "codes", "f32", "bf16"]))
    while True:
        M, K = _log(rng, 1, 8192), 16 * _log(rng, 4, 1024)
        if M * K <= 2048 * 14336:
            break
    return _glu("", M, K, rng.choice(["f32", "bf16"]), rng.random() < 0.5, rng.choice(["codes", "codes", "f32", "bf16"]))


_DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}


def _inputs(case, seed):
    """The tensors of a case: activations ~ N(0, 1) with 1% outliers of 20 times, weights as a 4-bit encoder leaves them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    M, K = case["M"], case["K"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def outlying(*shape):
        x = normal(*shape)
        return torch.where(torch.rand(shape, generator=g, device="cuda") < 0.01, x * 20, x)

    if case["op"] == "w4":
        N, groups = case["N"], -(-K // case["group"])
        x = outlying(M, K)
        xs = x.abs().amax(1) / 127
        xq = torch.round(x / xs[:, None]).clamp_(-127, 127).to(torch.int8)
        q = torch.empty((N, K), dtype=torch.uint8, device="cuda")
        rows = max(1, (1 << 26) // K)
        for r in range(0, N, rows):  # in slices: the vocabulary matrix is 2 GB in fp32
            q[r:r + rows] = (normal(min(rows, N - r), K) * 2.5 + 8).round_().clamp_(0, 15).to(torch.uint8)
        packed = q[:, 0::2] | (q[:, 1::2] << 4)
        scales = torch.exp(normal(N, groups) * 0.3 - 5.5).to(torch.bfloat16)
        zeros = torch.randint(5, 12, (N, groups), generator=g, device="cuda").to(torch.uint8) if case["zeros"] else None
        return dict(xq=xq, xs=xs, packed=packed, scales=scales, zeros=zeros)
    if case["op"] == "norm":
        layer, post, gate = case["kind"] == "layer", case["post"], case["gate"]
        return dict(
            h=outlying(M, K).to(_DTYPE[case["h"]]), branch=(normal(M, K) * 0.5).to(_DTYPE[case["branch"]]),
            weight=1 + 0.1 * normal(K), bias=0.1 * normal(K) if layer else None,
            post_weight=1 + 0.1 * normal(K) if post else None, post_bias=0.1 * normal(K) if post and layer else None,
            gate=None if gate == "none" else normal(K if gate == "channel" else 1) * 0.7)
    if case["fused"]:  # one matrix [M][2K], as one product with both weights leaves it
        both = normal(M, 2 * K).to(_DTYPE[case["dtype"]])
        return dict(gate=both[:, :K], up=both[:, K:])
    return dict(gate=normal(M, K).to(_DTYPE[case["dtype"]]), up=normal(M, K).to(_DTYPE[case["dtype"]]))


def prepare(case, seed):
    state = dict(case=case, **_inputs(case, seed))
    if own and case["op"] == "w4":
        import w2_a8_matmul_amd as s3d8

        # what a program keeps for a matrix: its weights in the kernels' layout, laid out once
        state["linear"] = s3d8.W4Linear(state.pop("packed"), state.pop("scales"), case["group"], state.pop("zeros"))
    return state


def run(state):
    if own:
        return _library(state)
    return {"w4": _plain_w4, "norm": _plain_norm, "glu": _plain_glu}[state["case"]["op"]](state)


# ------------------------------------------------------------------ the library


def _library(state):
    import w2_a8_matmul_amd as s3d8

    c = state["case"]
    if c["op"] == "w4":
        return state["linear"].linear(state["xq"], state["xs"], out=c["out"])
    if c["op"] == "norm":
        return s3d8.block_norm(state["h"], state["weight"], state["bias"], branch=state["branch"],
                               post_weight=state["post_weight"], post_bias=state["post_bias"], gate=state["gate"],
                               tanh_gate=c["gate"] == "tanh", residual_scale=c["residual_scale"], eps=1e-5,
                               kind=c["kind"], out=c["out"])
    return s3d8.glu_act(state["gate"], state["up"], out=c["out"])


# ------------------------------------------------------------------ plain forms


def _finish(u, out):
    """fp32 rows as they are, rounded to bf16, or as INT8 codes with one scale a row."""
    if out != "codes":
        return (u.to(_DTYPE[out]),)
    amax = u.abs().amax(1)
    xs = amax / torch.full_like(amax, 127)  # a division: by a plain number torch multiplies with its reciprocal
    codes = torch.round(u / torch.where(amax == 0, 1, xs)[:, None]).clamp(-127, 127).to(torch.int8)
    return codes, xs


def _plain_w4(s):
    c = s["case"]
    N, K = c["N"], c["K"]
    q = torch.stack((s["packed"] & 15, s["packed"] >> 4), 2).view(N, K).float()
    zeros = 8.0 if s["zeros"] is None else s["zeros"].float().repeat_interleave(c["group"], 1)[:, :K]
    w = (q - zeros) * s["scales"].float().repeat_interleave(c["group"], 1)[:, :K]
    return ((s["xq"].float() @ w.t()) * s["xs"][:, None]).to(_DTYPE[c["out"]])


def _plain_normalised(v, kind, weight, bias):
    # statistics in fp64, each elementwise step in fp32
    d = v.double()
    if kind == "rms":
        r = (d.square().mean(1, keepdim=True) + 1e-5).rsqrt().float()
        return v * r * weight
    mean = d.mean(1, keepdim=True)
    r = ((d - mean).square().mean(1, keepdim=True) + 1e-5).rsqrt().float()
    return (v - mean.float()) * r * weight + bias


def _plain_norm(s):
    c = s["case"]
    b = s["branch"].float()
    if c["post"]:
        b = _plain_normalised(b, c["kind"], s["post_weight"], s["post_bias"])
    if s["gate"] is not None:
        b = (s["gate"].double().tanh().float() if c["gate"] == "tanh" else s["gate"]) * b
    h = (c["residual_scale"] * s["h"].float() + b).to(s["h"].dtype)
    return h, *_finish(_plain_normalised(h.float(), c["kind"], s["weight"], s["bias"]), c["out"])


def _plain_glu(s):
    g = s["gate"].double()
    rows = _finish((g / (1 + torch.exp(-g)) * s["up"].double()).float(), s["case"]["out"])
    return rows if len(rows) > 1 else rows[0]


# ------------------------------------------------------------------ work


def work(case):
    M, K = case["M"], case["K"]
    size = {"f32": 4, "bf16": 2}
    out = M * (K + 4) if case["out"] == "codes" else M * K * size[case["out"]]
    if case["op"] == "w4":
        N, groups = case["N"], -(-K // case["group"])
        weights = N * K // 2 + N * groups * (3 if case["zeros"] else 2)
        return {"bytes": weights + M * K + 4 * M + M * N * size[case["out"]], "flops": 2 * M * N * K}
    if case["op"] == "norm":
        vectors = 1 + (case["kind"] == "layer") * (1 + case["post"]) + case["post"] + (case["gate"] == "channel")
        rows = M * K * (2 * size[case["h"]] + size[case["branch"]])
        return {"bytes": rows + out + 4 * K * vectors, "flops": M * K * (16 if case["post"] else 10)}
    return {"bytes": 2 * M * K * size[case["dtype"]] + out, "flops": M * K * 30}


# ------------------------------------------------------------------ 64 bits


def _exact_rows(u, out):
    # u: the rows, rounded to fp32 where the codes' definition rounds them
    if out != "codes":
        return [u]
    amax = u.abs().max(dim=1).values
    step = (amax / 127).to(torch.float32).double()  # the scale is an fp32 number
    ratio = u / step.clamp(min=2.0 ** -149).unsqueeze(1)
    codes = ratio.to(torch.float32).double().round()  # the quotient too, then to nearest even
    return [codes.clamp(-127, 127).to(torch.int8), amax / 127]


def _exact_norm_of(v, weight, bias, kind):
    width = v.shape[1]
    centre = v.sum(1, keepdim=True) / width if kind == "layer" else torch.zeros_like(v[:, :1])
    var = ((v - centre) ** 2).sum(1, keepdim=True) / width
    u = (v - centre) / torch.sqrt(var + 1e-5) * weight.double()
    return u if bias is None else u + bias.double()


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "w4":
        M, K, N, G = case["M"], case["K"], case["N"], case["group"]
        x = s["xq"].double() * s["xs"].double().unsqueeze(1)
        y = torch.empty((M, N), dtype=torch.float64, device="cuda")
        column = torch.arange(K, device="cuda")
        for r in range(0, N, 8192):  # rows of the matrix in slices
            byte = s["packed"][r:r + 8192][:, column // 2].to(torch.int32)
            q = torch.where(column % 2 == 1, byte // 16, byte % 16).double()
            z = s["zeros"][r:r + 8192][:, column // G].double() if case["zeros"] else 8
            y[:, r:r + 8192] = x @ ((q - z) * s["scales"][r:r + 8192][:, column // G].double()).t().contiguous()
        return y
    if case["op"] == "glu":
        g, u = s["gate"].double(), s["up"].double()
        a = g * torch.sigmoid(g) * u
        rows = _exact_rows(a.float().double() if case["out"] == "codes" else a, case["out"])
        return rows if len(rows) > 1 else rows[0]
    b = s["branch"].double()
    if case["post"]:
        b = _exact_norm_of(b, s["post_weight"], s["post_bias"], case["kind"])
    if s["gate"] is not None:
        gate = s["gate"].double()
        b = b * (torch.tanh(gate) if case["gate"] == "tanh" else gate)
    h = case["residual_scale"] * s["h"].double() + b
    # the norm reads the residual as it is stored
    u = _exact_norm_of(h.to(s["h"].dtype).double(), s["weight"], s["bias"], case["kind"])
    rows = _exact_rows(u, case["out"])
    if case["out"] == "codes":
        rows[0] = None  # codes next to a rounding border follow the definition's fp32 steps, not the real numbers
    return [h, *rows]
