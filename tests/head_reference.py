"""Plain forms in 64 bits of the operators of heads and tokens: rotary
frequencies, the norm and rotary position of heads, attention and sampling, each
with a bound of what fp32 arithmetic may be off by."""
from __future__ import annotations

import math

import numpy as np

HALF_BF16 = 2.0 ** -8  # half a step of bfloat16, relative to the value
HALF_F32 = 2.0 ** -24


def frequencies(rot, base, scaling="none", factor=1.0, original_length=8192, low=1.0, high=4.0):
    """(radians per position of each pair, factor on cosine and sine), one pair after the other."""
    f = []
    for j in range(rot // 2):
        x = math.exp(-2 * j / rot * math.log(base))
        if scaling == "linear":
            x /= factor
        elif scaling == "llama3":
            wave = 2 * math.pi / x
            if wave > original_length / low:
                x /= factor
            elif wave > original_length / high:
                smooth = (original_length / wave - low) / (high - low)
                x = (1 - smooth) * x / factor + smooth * x
        elif scaling == "yarn":
            def pair(turns):
                return rot * math.log(original_length / (turns * 2 * math.pi)) / (2 * math.log(base))
            a, b = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), rot - 1)
            share = min(max((j - a) / max(b - a, 0.001), 0), 1)
            x = x / factor * share + x * (1 - share)
        f.append(x)
    return np.array(f), 0.1 * math.log(factor) + 1 if scaling == "yarn" else 1.0


def head_rope(x, positions, f, factor, interleaved, weight, eps):
    """(result, bound of an fp32 result's error) of heads [M][H][D].

    r = 1 / sqrt(mean square): D - 1 additions and D products of positive terms, a division and
    an addition, halved by the root, and the root's own step: (D / 2 + 4) steps, then
    two products.  Cosine and sine: their argument, a polynomial of rising terms and the
    factor: 6 steps of 1; the angle itself 2^-52.  A turned value: two products and a
    sum more."""
    x = x.astype(np.float64)
    D = x.shape[2]
    steps = 0.0
    if weight is not None:
        x = x / np.sqrt((x * x).mean(2, keepdims=True) + eps) * weight.astype(np.float64)
        steps = D / 2 + 6
    rot = 2 * len(f)
    y, size = x.copy(), np.abs(x)
    turned = np.zeros(D)
    if rot:
        angle = positions.astype(np.float64)[:, None] * f
        c, s = factor * np.cos(angle)[:, None], factor * np.sin(angle)[:, None]
        a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
        size[..., a] = size[..., b] = abs(factor) * (np.abs(x[..., a]) + np.abs(x[..., b]))
        turned[a] = turned[b] = 9 + 2.0 ** -28 * np.abs(angle).max(0)
    return y, (steps + turned) * HALF_F32 * size * 1.01 + 2.0 ** -149


def attention(q, k, v, scale, lens=None, mask=None):
    """(result, bound of the error of a bf16 result) of q [B][Lq][H][D], k and v [B or 1][Lk][Hk][D].

    A score is off by (D + 1) fp32 steps of the sum of its absolute products and 4 steps of its own
    and the maximum's size (scaling, its constant, the difference), all in powers of e;
    p by that, 4 steps of the exponential and its rounding to bf16; the two sums of n
    terms by n steps (with as many again for joining parts); the result by the
    quotient's 2 steps and its rounding to bf16."""
    q, k, v = (t.astype(np.float64) for t in (q, k, v))
    B, Lq, H, D = q.shape
    Lk, Hk = k.shape[1:3]
    o, bound = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(B):
        kb = min(b, k.shape[0] - 1)
        n = Lk if lens is None else max(0, min(int(lens[min(b, len(lens) - 1)]), Lk))
        sees = np.ones((Lq, n), bool)
        if mask is not None:
            sees &= np.broadcast_to(mask[min(b, mask.shape[0] - 1)], (Lq, Lk))[:, :n]
        if n == 0:
            continue
        for h in range(H):
            g = h // (H // Hk)
            kh, vh = np.nan_to_num(k[kb, :n, g], posinf=0, neginf=0), np.nan_to_num(v[kb, :n, g], posinf=0, neginf=0)
            x = scale * (q[b, :, h] @ kh.T)
            off = scale * (D + 1) * HALF_F32 * (np.abs(q[b, :, h]) @ np.abs(kh).T)
            x = np.where(sees, x, -np.inf)
            top = x.max(1, keepdims=True)
            top = np.where(np.isneginf(top), 0, top)
            p = np.exp(x - top)
            with np.errstate(invalid="ignore"):
                off = np.where(sees, off + 4 * HALF_F32 * (np.abs(np.where(sees, x, 0)) + np.abs(top)), 0).max(1, keepdims=True)
            total = p.sum(1, keepdims=True)
            total[total == 0] = 1
            o[b, :, h] = p @ vh / total
            mean = p @ np.abs(vh) / total
            off = 2 * off + (4 + 2 * n + 2) * 2 * HALF_F32
            bound[b, :, h] = (mean * (HALF_BF16 + off) + np.abs(o[b, :, h]) * HALF_BF16) * 1.02 + 2.0 ** -133
    return o, bound


def sample(logits, u, temperature, top_k, top_p, min_p):
    """(token, probability) of one row, in whole numbers of unlimited size."""
    l = [-math.inf if math.isnan(x) else float(x) for x in np.asarray(logits, np.float32)]
    m = max(l)
    if m == -math.inf:
        return -1, 0.0
    order = sorted(range(len(l)), key=lambda i: (-l[i], i))
    T = float(np.float32(temperature))
    if not T > 0:
        return order[0], 1.0
    w = {}
    for i in order:
        w[i] = 2 ** 44 if l[i] == m else 0 if l[i] == -math.inf or m == math.inf else round(2.0 ** 44 * math.exp((l[i] - m) / T))
    kept = order if top_k <= 0 else order[:top_k]
    p = float(np.float32(top_p))
    if p < 1:
        limit, before, some = max(1, math.ceil(max(p, 0.0) * float(sum(w[i] for i in kept)))), 0, []
        for i in kept:
            if before >= limit:
                break
            some.append(i)
            before += w[i]
        kept = some
    least = math.ceil(min(max(float(np.float32(min_p)), 0.0), 1.0) * 2 ** 44)
    kept = sorted(i for i in kept if w[i] >= least)
    total = sum(w[i] for i in kept)
    target, upto = min(math.floor(max(float(np.float32(u)), 0.0) * float(total)), total - 1), 0
    for i in kept:
        upto += w[i]
        if upto > target:
            return i, w[i] / total
    raise AssertionError
