"""Plain numpy forms of the 4-bit linear layer, the block norm and the gated
activation: integers exactly, statistics in 64 bits, and each fp32 rounding
that the definitions in include/s3d8.h name as one numpy float32 operation."""
from __future__ import annotations

import numpy as np

F = np.float32


def bf16_bits(x) -> np.ndarray:
    """Round to nearest even of finite fp32 values to bfloat16 bit patterns."""
    u = np.asarray(x, F).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def bf16_value(bits) -> np.ndarray:
    return (np.asarray(bits).astype(np.uint32) << 16).view(F)


def round_bf16(x) -> np.ndarray:
    return bf16_value(bf16_bits(x))


# ------------------------------------------------------------------ 4-bit weights
def w4_encode(W, group: int, affine: bool):
    """Per group, one after the other: (codes [N][K], scale bits, zeros)."""
    N, K = W.shape
    G = -(-K // group)
    q, scales, zeros = np.zeros((N, K), np.uint8), np.zeros((N, G), np.uint16), np.zeros((N, G), np.uint8)
    for n in range(N):
        for g in range(G):
            w = W[n, g * group:(g + 1) * group].astype(F)
            lo, hi = min(F(0), w.min()), max(F(0), w.max())
            bits = bf16_bits((hi - lo) / F(15) if affine else max(hi, -lo) / F(7))
            s = bf16_value(bits)
            z = F(8)
            if s == 0:
                code = np.full(w.shape, F(8))
            else:
                if affine:
                    z = np.clip(np.rint(-lo / s), F(0), F(15))
                code = np.clip(np.rint(w / s) + z, F(0), F(15))
            q[n, g * group:(g + 1) * group], scales[n, g], zeros[n, g] = code, bits, z
    return q, scales, zeros


def pack(q) -> np.ndarray:
    return (q[:, 0::2] | (q[:, 1::2] << 4)).astype(np.uint8)


def w4_linear(xq, xs, q, scales, zeros, group: int):
    """(y, sum of the absolute group terms) in 64 bits: y[m][n] = xs[m] sum_g s[n][g] sum_k xq (q - z)."""
    K = q.shape[1]
    y = np.zeros((xq.shape[0], q.shape[0]))
    size = np.zeros_like(y)
    for g in range(scales.shape[1]):
        k = slice(g * group, min((g + 1) * group, K))
        z = 8 if zeros is None else zeros[:, g:g + 1].astype(np.int64)
        # float64 products of small integers are exact
        acc = xq[:, k].astype(np.float64) @ (q[:, k].astype(np.int64) - z).astype(np.float64).T
        term = acc * bf16_value(scales[:, g]).astype(np.float64)
        y += term
        size += np.abs(term)
    s = xs.astype(np.float64)[:, None]
    return y * s, size * np.abs(s)


def w4_tolerance(y, size, K: int, bf16: bool):
    """fp32 accumulation of n terms t_i, in any order, is off by at most
    n 2^-24 sum |t_i| (to first order); here at most one term per 32 columns,
    16 partial sums, and 3 more roundings.  bf16 adds half a step, 2^-8 of the
    value (2^-133 where that is subnormal)."""
    n = -(-K // 32) + 16 + 3
    tol = n * 2.0 ** -24 * size * 1.01 + 2.0 ** -149
    return tol + (2.0 ** -8 * (np.abs(y) + tol) + 2.0 ** -133 if bf16 else 0)


# ------------------------------------------------------------------ rows
def quantise(u):
    """Codes and scales of fp32 rows as s3d8_quant_act defines them."""
    a = np.abs(u).max(1)
    xs = (a / F(127)).astype(F)
    with np.errstate(divide="ignore", invalid="ignore"):
        codes = np.clip(np.rint(u / xs[:, None]), F(-127), F(127))
    codes[a == 0] = 0
    return codes.astype(np.int8), xs


def normalise(v, kind: str, eps: float, w, b):
    d = v.astype(np.float64)
    mu = d.mean(1, keepdims=True) if kind == "layer" else 0.0
    var = ((d - mu) ** 2).mean(1, keepdims=True)
    r = (1.0 / np.sqrt(var + eps)).astype(F)
    u = (v - mu.astype(F)) * r if kind == "layer" else v * r
    u = u * w
    return u + b if b is not None else u


def block_norm(h, w, b=None, branch=None, post_w=None, post_b=None, gate=None, tanh_gate=False, residual_scale=1.0,
               eps=1e-5, kind="rms", h_bf16=False):
    """(h', u): h and branch fp32 values (of whatever type they are stored in)."""
    if branch is not None:
        t = branch if post_w is None else normalise(branch, kind, eps, post_w, post_b)
        if gate is not None:
            g = np.tanh(gate.astype(np.float64)).astype(F) if tanh_gate else gate
            t = g * t
        h = F(residual_scale) * h + t
        if h_bf16:
            h = round_bf16(h)
    return h, normalise(h, kind, eps, w, b)


def glu(g, u):
    g, u = g.astype(np.float64), u.astype(np.float64)
    with np.errstate(over="ignore"):
        return (g / (1 + np.exp(-g)) * u).astype(F)
