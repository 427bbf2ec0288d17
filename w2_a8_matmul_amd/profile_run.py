"""Fixed launch sequences for hardware-counter profiling (rocprofv3 --pmc).

Runs, in one process and in this order:
  1. ``copy``: a plain device-to-device copy of 256 MiB (torch ``copy_``),
     repeated 4 times; its FETCH_SIZE / WRITE_SIZE per dispatch against the
     known 256 MiB gives the counter scale factor;
  2. ``gemv_c1_m1``: s3d8_forward on the decode GEMV shape M=1, K=4096,
     N=14336, 28 distinct weight copies (so that every launch reads its
     weights from HBM, not from the Infinity Cache), 2 passes over them;
  3. ``gemm_c3``: s3d8_linear on the prefill shape M=2048, K=4096, N=14336,
     150 warm-up launches (the clocks settle under sustained load), then 4
     launches: the summaries use the last 4 dispatches;
  4. the same problem through s3d8_linear_unfused (dequant_tiled_kernel +
     gemm_i8_kernel), 4 calls;
  5. ``gemv_codes_c1_m8``: s3d8_linear at M=8 on the decode GEMV shape (the
     GEMV on INT8 codes), 28 weight copies, 2 passes;
  6. ``splitk_vision_down``: s3d8_linear_splitk on M=1601, K=5120, N=1280 at
     the library's split count, 50 warm-up launches, then 4.
Weights are random S3D8 formats (uniform bytes, random table and scales):
the bytes moved do not depend on the values.

With ``block``, the operators around the linear layers instead: each call of
``block_calls()`` CALLS times, over enough copies of its operands that none is
still in a cache, one after the other in that order; with a part of a label
after it, only the calls whose label holds it.  With ``heads``, those on heads and
logits, ``head_calls()``.

Usage: python -m w2_a8_matmul_amd.profile_run [block|heads [PART]]   (from the repository root)
"""
from __future__ import annotations

import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


CALLS = 60
_CACHES = 320 * 2 ** 20  # bytes that the caches do not hold


def block_calls():
    """(label, operand bytes, maker): ``maker()`` makes random operands and returns one call on them."""
    import torch

    import w2_a8_matmul_amd as s3d8

    dev = torch.device("cuda:0")
    bf, f32 = torch.bfloat16, torch.float32

    def w4(M, K, N, group, zeros=False, out="f32", fp32_x=False):
        def make():
            packed = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device=dev)
            scales = torch.exp(torch.randn(N, -(-K // group), device=dev) * 0.3 - 5.5).to(bf)
            z = torch.randint(5, 12, scales.shape, dtype=torch.uint8, device=dev) if zeros else None
            lin = s3d8.W4Linear(packed, scales, group, z)
            x = torch.randn(M, K, device=dev)
            xq, xs = s3d8.quant_act(x)
            y = torch.empty(M, N, dtype=f32 if out == "f32" else bf, device=dev)
            if fp32_x:
                return lambda: s3d8.w4_forward(x, lin.tiled, N, group, zeros, y=y, xq=xq, xs=xs)
            return lambda: lin.linear(xq, xs, y=y, out=out)
        name = "w4_forward" if fp32_x else "w4_linear"
        label = f"{name} {M} x {K} -> {N}, groups of {group}{', zero points' if zeros else ''}"
        return label, N * K // 2 + M * K + M * N * (4 if out == "f32" else 2), make

    def norm(M, K, h, branch, kind="rms", post=False, tanh=False, out="codes"):
        def make():
            a, b = torch.randn(M, K, device=dev).to(h), torch.randn(M, K, device=dev).to(branch)
            w = 1 + 0.1 * torch.randn(K, device=dev)
            bias = 0.1 * torch.randn(K, device=dev) if kind == "layer" else None
            gate = torch.randn(1, device=dev) if tanh else None
            return lambda: s3d8.block_norm(a, w, bias, branch=b, post_weight=w if post else None, gate=gate,
                                           tanh_gate=tanh, kind=kind, out=out)
        label = (f"block_norm {M} x {K}, {h}, {branch} branch, {kind}{', post norm' if post else ''}"
                 f"{', tanh gate' if tanh else ''}, {out}".replace("torch.", ""))
        return label, 3 * M * K * h.itemsize, make

    def glu(M, K, dtype, out="codes", far=False):
        def make():
            g, u = torch.randn(M, K, device=dev).to(dtype), torch.randn(M, K, device=dev).to(dtype)
            if far:
                g[:, 0] = -80
            return lambda: s3d8.glu_act(g, u, out=out)
        label = f"glu_act {M} x {K}, {dtype}, {out}{', a gate below -64 in each row' if far else ''}".replace("torch.", "")
        return label, 3 * M * K * dtype.itemsize, make

    return [
        w4(1, 4096, 1024, 128), w4(1, 4096, 14336, 64), w4(1, 14336, 4096, 128), w4(8, 4096, 128256, 128),
        w4(16, 4096, 14336, 128), w4(16, 4096, 14336, 32, True), w4(21, 1296, 1003, 32, True),
        w4(1601, 5120, 1280, 128, True, "bf16"), w4(2048, 4096, 14336, 64, False, "bf16"),
        w4(2048, 4096, 14336, 64, True, "bf16"), w4(2048, 4096, 14336, 128, False, "bf16"),
        w4(1, 4096, 14336, 64, fp32_x=True),
        norm(1, 4096, f32, f32), norm(2048, 4096, bf, bf, post=True), norm(1601, 1280, f32, bf, "layer", tanh=True, out="bf16"),
        norm(64, 53248, bf, bf), glu(1, 14336, f32), glu(5, 1744, bf, "f32"), glu(2048, 14336, bf),
        glu(2048, 14336, bf, "bf16"), glu(2048, 14336, bf, far=True), glu(64, 53248, bf),
    ]


def head_calls():
    """The same of head_rope, cross_attention and sample."""
    import torch

    import w2_a8_matmul_amd as s3d8

    dev = torch.device("cuda:0")
    bf, f32 = torch.bfloat16, torch.float32

    def rope(M, H, Hk, D, dtype, norm=True, out="bf16", position=True):
        def make():
            x = torch.randn(M, (H + 2 * Hk) * D, device=dev).to(dtype)
            handle = s3d8.Rope(D, 500000.0, scaling="llama3", factor=8.0, original_length=8192)
            w = 1 + 0.1 * torch.randn(D, device=dev) if norm else None
            q, k = x[:, :H * D].view(M, H, D), x[:, H * D:(H + Hk) * D].view(M, Hk, D)
            pos = torch.arange(M, device=dev) if position else None
            return lambda: s3d8.head_rope(q, k, pos, handle if position else None, q_weight=w, k_weight=w, out=out)
        label = f"head_rope {M} x ({H} + {Hk}) x {D}, {dtype}{', norm' if norm else ''}{'' if position else ' alone'}, {out}"
        label = label.replace("torch.", "")
        return label, M * (H + Hk) * D * (dtype.itemsize + (2 if out == "bf16" else 4)), make

    def attention(B, Lq, Lk, H, Hk, D, lens=False, shared=False, mask=False, out="bf16", lost=False):
        def make():
            n = 1 if shared else B
            q, k, v = (torch.randn(b, L, h, D, device=dev).to(bf) for b, L, h in ((B, Lq, H), (n, Lk, Hk), (n, Lk, Hk)))
            ls = torch.linspace(Lk // 2, Lk, B, device=dev).to(torch.int32) if lens else None
            m = None
            if mask:  # four images, each seen by the tokens after it
                starts = torch.tensor([0.05, 0.15, 0.3, 0.45], device=dev) * Lq
                m = (torch.arange(Lq, device=dev)[:, None] >= starts).repeat_interleave(-(-Lk // 4), 1)[None, :, :Lk].contiguous()
            if lost:  # a value of the first image, which most tokens see
                v[:, 0, :, 0] = float("inf")
            return lambda: s3d8.cross_attention(q, k, v, kv_lens=ls, mask=m, out=out)
        label = (f"cross_attention {B} x {Lq} on {Lk}, {H} on {Hk} x {D}{', lengths from a half' if lens else ''}"
                 f"{', shared states' if shared else ''}{', mask of four images' if mask else ''}"
                 f"{', an infinite value' if lost else ''}{', codes' if out == 'codes' else ''}")
        return label, 4 * (1 if shared else B) * Lk * Hk * D + 4 * B * Lq * H * D + mask * Lq * Lk, make

    def sample(M, V, dtype, temperature=0.9, **limits):
        def make():
            l = torch.randn(M, V, device=dev) * 2
            at = torch.rand(M, V, device=dev) < 40 / V
            l = torch.where(at, l + 8 * torch.rand(M, V, device=dev), l).to(dtype)
            u = torch.rand(M, device=dev)
            return lambda: s3d8.sample(l, u, temperature=temperature, **limits)
        label = ", ".join([f"sample {M} x {V}", str(dtype), f"temperature {temperature}", *(f"{k} {v}" for k, v in limits.items())])
        label = label.replace("torch.", "")
        return label, M * V * dtype.itemsize, make

    return [
        rope(1, 32, 8, 128, f32, norm=False), rope(77, 16, 4, 80, bf, out="f32"), rope(2048, 32, 8, 128, bf), rope(8192, 32, 8, 128, bf),
        attention(1, 1, 1601, 32, 8, 128), attention(8, 1, 6404, 32, 8, 128, lens=True),
        attention(16, 1, 6404, 32, 8, 128, shared=True), attention(1, 1601, 1601, 16, 16, 80),
        attention(1, 2048, 6404, 32, 8, 128), attention(1, 2048, 6404, 32, 8, 128, mask=True),
        sample(1, 128256, f32, top_k=50, top_p=0.9), sample(8, 128256, bf, top_p=0.95),
        sample(33, 5003, f32, top_k=200, top_p=0.8, min_p=0.05), sample(512, 128256, f32, top_k=50, top_p=0.95, min_p=0.01),
        sample(512, 128256, f32, top_p=0.95), sample(1, 128256, f32, top_k=1000, top_p=0.9), sample(1, 1000, f32, top_k=50, top_p=0.9),
        sample(512, 128256, f32), sample(512, 128256, f32, temperature=0.0), sample(1, 128256, f32, temperature=0.0),
        rope(2048, 32, 8, 128, bf, position=False), attention(1, 1, 1601, 32, 8, 128, out="codes"),
        attention(1, 2048, 6404, 32, 8, 128, out="codes"), attention(1, 2048, 6404, 32, 8, 128, mask=True, lost=True),
        attention(33, 1, 1601, 32, 8, 128),
    ]


def block(part: str = "", calls=block_calls) -> None:
    import torch

    torch.manual_seed(1)
    for label, nbytes, make in calls():
        if part not in label:
            continue
        copies = [make() for _ in range(max(1, min(CALLS, -(-_CACHES // nbytes))))]
        torch.cuda.synchronize()
        for i in range(CALLS):
            copies[i % len(copies)]()
        torch.cuda.synchronize()
        print(f"[profile_run] {CALLS} x {label} ({len(copies)} copies)", flush=True)


def main() -> None:
    import numpy as np
    import torch

    import w2_a8_matmul_amd as s3d8
    import workloads

    dev = torch.device("cuda:0")
    torch.cuda.set_device(dev)

    def say(msg):
        print(f"[profile_run] {msg}", flush=True)

    # 1. copy kernel of known size
    nbytes = 256 * 2 ** 20
    src = torch.empty(nbytes, dtype=torch.uint8, device=dev).random_(0, 255)
    dst = torch.empty_like(src)
    for _ in range(4):
        dst.copy_(src)
    torch.cuda.synchronize()
    say(f"copy: 4 x {nbytes} bytes")
    del src, dst

    def fmt(seed, N, K):
        T = s3d8.num_triples(N)
        C = torch.from_numpy(workloads.random_centroids(seed)).to(dev)
        S = torch.from_numpy(workloads.random_scales_bf16(seed, 3 * T).view(np.int16)).to(dev)
        P = torch.from_numpy(workloads.random_packed(seed, T, K)).to(dev)
        return C, S, s3d8.tile(P, N)

    # 2. decode GEMV, fused forward
    M, K, N = 1, 4096, 14336
    C, S, tiled = fmt(11, N, K)
    copies = [tiled.clone() for _ in range(28)]
    x = torch.randn((M, K), dtype=torch.float32, device=dev)
    y = torch.empty((M, N), dtype=torch.float32, device=dev)
    xq = torch.empty((M, K), dtype=torch.int8, device=dev)
    xs = torch.empty((M,), dtype=torch.float32, device=dev)
    for _ in range(2):
        for t in copies:
            s3d8.forward(x, t, C, S, N, y=y, xq=xq, xs=xs)
    torch.cuda.synchronize()
    say(f"gemv_c1_m1: {2 * len(copies)} launches of s3d8_forward M={M} K={K} N={N}")
    del copies, tiled

    # 3. prefill GEMM
    M = 2048
    C, S, tiled = fmt(12, N, K)
    x = torch.randn((M, K), dtype=torch.float32, device=dev)
    xq, xs = s3d8.quant_act(x)
    y = torch.empty((M, N), dtype=torch.float32, device=dev)
    for _ in range(150 + 4):
        s3d8.linear(xq, xs, tiled, C, S, N, y=y)
    torch.cuda.synchronize()
    say(f"gemm_c3: 150 + 4 launches of s3d8_linear M={M} K={K} N={N}")

    # 4. the unfused prefill path on the same problem
    ws = torch.empty((s3d8.unfused_workspace_bytes(N, K),), dtype=torch.int8, device=dev)
    for _ in range(4):
        s3d8.linear_unfused(xq, xs, tiled, C, S, N, workspace=ws, y=y)
    torch.cuda.synchronize()
    say(f"gemm_c3 unfused: 4 calls of s3d8_linear_unfused M={M} K={K} N={N}")
    del ws, tiled, y

    # 5. the GEMV on INT8 codes, eight tokens
    M = 8
    C, S, tiled = fmt(13, N, K)
    copies = [tiled.clone() for _ in range(28)]
    xq, xs = s3d8.quant_act(torch.randn((M, K), dtype=torch.float32, device=dev))
    y = torch.empty((M, N), dtype=torch.float32, device=dev)
    for _ in range(2):
        for t in copies:
            s3d8.linear(xq, xs, t, C, S, N, y=y)
    torch.cuda.synchronize()
    say(f"gemv_codes_c1_m8: {2 * len(copies)} launches of s3d8_linear M={M} K={K} N={N}")
    del copies, tiled

    # 6. split-K on the vision down-projection
    M, K, N = 1601, 5120, 1280
    C, S, tiled = fmt(14, N, K)
    xq, xs = s3d8.quant_act(torch.randn((M, K), dtype=torch.float32, device=dev))
    y = torch.empty((M, N), dtype=torch.float32, device=dev)
    splits = s3d8.splitk_auto(M, K, N, torch.cuda.get_device_properties(dev).multi_processor_count)
    wsk = torch.zeros((max(1, s3d8.splitk_workspace_bytes(M, K, N, splits)),), dtype=torch.uint8, device=dev)
    for _ in range(50 + 4):
        s3d8.linear_splitk(xq, xs, tiled, C, S, N, splits=splits, workspace=wsk, y=y)
    torch.cuda.synchronize()
    say(f"splitk_vision_down: 50 + 4 launches of s3d8_linear_splitk M={M} K={K} N={N} splits={splits}")


if __name__ == "__main__":
    if sys.argv[1:2] in (["block"], ["heads"]):
        block("".join(sys.argv[2:3]), block_calls if sys.argv[1] == "block" else head_calls)
    else:
        main()
