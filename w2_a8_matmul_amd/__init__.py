"""S3D8 weight-decode-fused linear layer for AMD Instinct MI355X (gfx950).

Thin Python binding over the C ABI of ``libs3d8.so`` (``include/s3d8.h``):
argument marshalling only.  Host functions take numpy arrays; device
functions take torch tensors (device memory and the current HIP stream) and
run the library's HIP kernels.  There is no fallback path: if the library
is missing, importing ``w2_a8_matmul_amd._lib`` raises.

Format: the S3D8 storage format of "Llama-Mobile: Efficient 2.7-Bit
Quantization of VLMs" (Sec. 3.4, Eq. 1) with the byte layout of the blog
"11 billion parameters on a phone" ("Bit layout").  The device functions also
take 3D8 weights (``fmt="3d8"``: the table is int8 [256][3] signed
centroids indexed by the whole byte, the format the blog sets beside S3D8)
and write bf16 outputs (``out="bf16"``, as the blog's fused kernel does).

Beside it: the same linear layer on plain 4-bit weights with group scales
(``w4_linear``, ``W4Linear``), and what stands between the linears of a block,
ending in the INT8 codes they read: ``block_norm`` (norms around a block, gate,
residual sum) and ``glu_act`` (SiLU-gated activation).

Between the projections of heads, and after the vocabulary projection:
``head_rope`` (norm of query and key heads, rotary position; ``Rope`` holds its
frequencies), ``cross_attention`` (attention to an encoder's states) and
``sample`` (the next token from its logits and a random number).
"""
from __future__ import annotations

import ctypes
import math

import numpy as np

from ._lib import S3D8Error, call, lib  # noqa: F401

__all__ = [
    "S3D8Error", "num_triples", "packed_bytes", "format_bytes", "tiled_bytes", "pack", "encode",
    "tile", "quant_act", "linear", "linear_unfused", "unfused_workspace_bytes", "forward", "dequant",
    "PackedLinear", "hbm_read_probe", "mfma_rate_probe", "encode_device", "forward_batch",
    "linear_splitk", "splitk_auto", "splitk_workspace_bytes",
    "w4_encode", "w4_tiled_bytes", "w4_tile", "w4_linear", "w4_forward", "W4Linear", "block_norm", "glu_act",
    "Rope", "head_rope", "cross_attention", "sample",
]


def _np_ptr(a: np.ndarray):
    assert a.flags["C_CONTIGUOUS"]
    return a.ctypes.data_as(ctypes.c_void_p)


def num_triples(N: int) -> int:
    return int(lib().s3d8_num_triples(N))


def packed_bytes(N: int, K: int) -> int:
    return int(lib().s3d8_packed_bytes(N, K))


def format_bytes(N: int, K: int) -> int:
    return int(lib().s3d8_format_bytes(N, K))


def tiled_bytes(N: int, K: int) -> int:
    return int(lib().s3d8_tiled_bytes(N, K))


# ------------------------------------------------------------------ host
def pack(W, seed: int = 1, max_iters: int = 50, num_threads: int = 0, return_stats: bool = False):
    """Fit centroids (k-means++ / Lloyd-Max) and encode W (fp32 [N][K]).

    Returns (centroids uint8 [32][3], scales_bf16 uint16 [3T], packed uint8
    [T][K]) and, with ``return_stats``, also (distortion per iteration,
    iterations)."""
    W = np.ascontiguousarray(W, dtype=np.float32)
    N, K = W.shape
    T = num_triples(N)
    C = np.empty((32, 3), np.uint8)
    scales = np.empty((3 * T,), np.uint16)
    packed = np.empty((T, K), np.uint8)
    dist = np.zeros((max(max_iters, 0) + 1,), np.float64)
    iters = ctypes.c_int32(0)
    call("s3d8_pack", _np_ptr(W), N, K, seed, max_iters, num_threads, _np_ptr(C), _np_ptr(scales),
         _np_ptr(packed), _np_ptr(dist), ctypes.byref(iters))
    if return_stats:
        return C, scales, packed, dist[: iters.value + 1].copy(), iters.value
    return C, scales, packed


def encode(W, centroids, num_threads: int = 0):
    """Frozen-centroid encode: returns (scales_bf16 [3T], packed [T][K])."""
    W = np.ascontiguousarray(W, dtype=np.float32)
    C = np.ascontiguousarray(centroids, dtype=np.uint8)
    N, K = W.shape
    T = num_triples(N)
    scales = np.empty((3 * T,), np.uint16)
    packed = np.empty((T, K), np.uint8)
    call("s3d8_encode", _np_ptr(W), N, K, _np_ptr(C), num_threads, _np_ptr(scales), _np_ptr(packed))
    return scales, packed


# ------------------------------------------------------------------ device
_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:  # (the host functions do without torch)
        import torch
        _torch_module = torch
    return _torch_module


def _stream(t) -> int:
    torch = _torch()
    return torch.cuda.current_stream(t.device).cuda_stream


def _enqueue(name, dev, *args):
    """Call a device entry point on ``dev`` and its current stream (the last
    argument).  The stream's handle comes from torch's raw accessor (0.06 us
    against 1.7 us for a Stream object) and the device is only changed when it
    is not the current one: the call of a small kernel is bound by the host."""
    torch = _torch()
    i = dev.index
    if i == torch.cuda.current_device():
        rc = getattr(lib(), name)(*args, torch._C._cuda_getCurrentRawStream(i))
    else:
        with torch.cuda.device(dev):
            rc = getattr(lib(), name)(*args, torch._C._cuda_getCurrentRawStream(i))
    if rc:
        _lib.check(rc, name)


def _dev_check(t, dtype, name, device=None, numel=None, min_numel=None):
    """A device tensor argument: torch tensor on the GPU (on `device` when
    given), of `dtype`, contiguous, and with exactly `numel` (or at least
    `min_numel`) elements when given.  Outputs are checked with numel, so the
    kernels never write past a caller-supplied buffer."""
    if not isinstance(t, _torch().Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA/HIP torch tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the other arguments on {device}")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} must have {numel} elements, got {t.numel()}")
    if min_numel is not None and t.numel() < min_numel:
        raise ValueError(f"{name} must have at least {min_numel} elements, got {t.numel()}")


def quant_act(x, xq=None, xs=None):
    """Per-token INT8 quantisation of fp32 x [M][K] on the GPU: (xq, xs)."""
    torch = _torch()
    _dev_check(x, torch.float32, "x")
    M, K = x.shape
    xq, xs = _codes_out(xq, xs, M, K, x.device)
    with torch.cuda.device(x.device):
        call("s3d8_quant_act", x.data_ptr(), M, K, xq.data_ptr(), xs.data_ptr(), _stream(x))
    return xq, xs


def tile(packed, N: int, tiled=None):
    """Re-lay a device packed matrix [T][K] into the tiled layout read by
    linear/forward (done once per matrix)."""
    torch = _torch()
    _dev_check(packed, torch.uint8, "packed")
    T, K = packed.shape
    if T != num_triples(N):
        raise ValueError("packed rows do not match N")
    if tiled is None:
        tiled = torch.empty((tiled_bytes(N, K),), dtype=torch.uint8, device=packed.device)
    _dev_check(tiled, torch.uint8, "tiled", packed.device, min_numel=tiled_bytes(N, K))
    with torch.cuda.device(packed.device):
        call("s3d8_tile", packed.data_ptr(), N, K, tiled.data_ptr(), _stream(packed))
    return tiled


def _scales_view(scales):
    torch = _torch()
    if scales.dtype in (torch.bfloat16, torch.uint16):
        scales = scales.view(torch.int16)
    _dev_check(scales, torch.int16, "scales")
    return scales


_FORMATS = {"s3d8": 0, "3d8": 1}
_OUTS = {"f32": 0, "bf16": 1}


def _other_matrix(t, rows) -> bool:
    """A matrix of other rows than it should have (a vector, also as a matrix of
    one row or column, or more dimensions are taken as the rows in a row)."""
    return t.dim() == 2 and t.shape[0] != rows and 1 not in t.shape


def _variant(fmt: str, out: str = "f32"):
    if fmt not in _FORMATS or out not in _OUTS:
        raise ValueError(f"fmt must be one of {list(_FORMATS)}, out one of {list(_OUTS)}")
    return _FORMATS[fmt], _OUTS[out]


def _out_type(out: str) -> int:
    if out not in _OUTS:
        raise ValueError(f"out must be one of {list(_OUTS)}")
    return _OUTS[out]


def _table_view(table, fmt: str):
    """S3D8: uint8 [32][3] centroids; 3D8: int8 [256][3] signed table (uint8 views accepted)."""
    torch = _torch()
    if fmt == "3d8" and table.dtype == torch.int8:
        table = table.view(torch.uint8)
    _dev_check(table, torch.uint8, "centroids" if fmt == "s3d8" else "table")
    if table.numel() != (96 if fmt == "s3d8" else 768):
        raise ValueError("table size does not match the format")
    return table


def _check_weights(tiled, centroids, scales, N, K, fmt: str = "s3d8", device=None):
    torch = _torch()
    _dev_check(tiled, torch.uint8, "tiled", device)
    table = _table_view(centroids, fmt)
    _dev_check(table, torch.uint8, "centroids", device)
    _dev_check(scales, torch.int16, "scales", device)
    T = num_triples(N)
    if tiled.numel() < tiled_bytes(N, K) or scales.numel() < 3 * T:
        raise ValueError("tiled / centroids / scales do not match (N, K)")


def _y_out(y, M, N, out, device):
    """The output buffer: a new one, or a caller's of the right type and size."""
    torch = _torch()
    dtype = torch.float32 if out == "f32" else torch.bfloat16
    if y is None:
        return torch.empty(M, N, dtype=dtype, device=device)
    _dev_check(y, dtype, "y", device, numel=M * N)
    return y


def _acc_out(acc, want, M, N, device):
    torch = _torch()
    if acc is None:
        return torch.empty((M, N), dtype=torch.int32, device=device) if want else None
    _dev_check(acc, torch.int32, "acc", device, numel=M * N)
    return acc


def _codes_out(xq, xs, M, K, device):
    """Activation codes and scales written by quant_act / forward."""
    torch = _torch()
    if xq is None:
        xq = torch.empty(M, K, dtype=torch.int8, device=device)
    else:
        _dev_check(xq, torch.int8, "xq", device, numel=M * K)
    if xs is None:
        xs = torch.empty(M, dtype=torch.float32, device=device)
    else:
        _dev_check(xs, torch.float32, "xs", device, numel=M)
    return xq, xs


def linear(xq, xs, tiled, centroids, scales, N: int, y=None, acc=None, return_acc: bool = False,
           fmt: str = "s3d8", out: str = "f32"):
    """Fused S3D8 (or 3D8) linear on pre-quantised activations: y [M][N],
    fp32 or bf16 (and the INT32 accumulators)."""
    torch = _torch()
    f, o = _variant(fmt, out)
    _dev_check(xq, torch.int8, "xq")
    M, K = xq.shape
    _dev_check(xs, torch.float32, "xs", xq.device, min_numel=M)
    scales = _scales_view(scales)
    _check_weights(tiled, centroids, scales, N, K, fmt, xq.device)
    y = _y_out(y, M, N, out, xq.device)
    acc = _acc_out(acc, return_acc, M, N, xq.device)
    with torch.cuda.device(xq.device):
        args = (xq.data_ptr(), xs.data_ptr(), M, K, N, tiled.data_ptr(), tiled.numel(), centroids.data_ptr())
        tail = (acc.data_ptr() if acc is not None else None, _stream(xq))
        if f == 0 and o == 0:
            call("s3d8_linear", *args, scales.data_ptr(), y.data_ptr(), *tail)
        else:
            call("s3d8_linear_ex", *args, f, scales.data_ptr(), y.data_ptr(), o, *tail)
    if return_acc:
        return y, acc
    return y


def unfused_workspace_bytes(N: int, K: int) -> int:
    return int(lib().s3d8_unfused_workspace_bytes(N, K))


def linear_unfused(xq, xs, tiled, centroids, scales, N: int, workspace=None, y=None, acc=None,
                   return_acc: bool = False, fmt: str = "s3d8", out: str = "f32"):
    """Same result as ``linear``: the matrix is decoded once into an INT8
    workspace (allocated here unless given), then an INT8 GEMM runs on it."""
    torch = _torch()
    f, o = _variant(fmt, out)
    _dev_check(xq, torch.int8, "xq")
    M, K = xq.shape
    _dev_check(xs, torch.float32, "xs", xq.device, min_numel=M)
    scales = _scales_view(scales)
    _check_weights(tiled, centroids, scales, N, K, fmt, xq.device)
    wbytes = unfused_workspace_bytes(N, K)
    if workspace is None:
        workspace = torch.empty((wbytes,), dtype=torch.int8, device=xq.device)
    _dev_check(workspace, torch.int8, "workspace", xq.device, min_numel=wbytes)
    y = _y_out(y, M, N, out, xq.device)
    acc = _acc_out(acc, return_acc, M, N, xq.device)
    with torch.cuda.device(xq.device):
        args = (xq.data_ptr(), xs.data_ptr(), M, K, N, tiled.data_ptr(), tiled.numel(), centroids.data_ptr())
        tail = (acc.data_ptr() if acc is not None else None, workspace.data_ptr(), workspace.numel(),
                _stream(xq))
        if f == 0 and o == 0:
            call("s3d8_linear_unfused", *args, scales.data_ptr(), y.data_ptr(), *tail)
        else:
            call("s3d8_linear_unfused_ex", *args, f, scales.data_ptr(), y.data_ptr(), o, *tail)
    if return_acc:
        return y, acc
    return y


def splitk_auto(M: int, K: int, N: int, num_cus: int) -> int:
    return int(lib().s3d8_splitk_auto(M, K, N, num_cus))


def splitk_workspace_bytes(M: int, K: int, N: int, splits: int) -> int:
    return int(lib().s3d8_splitk_workspace_bytes(M, K, N, splits))


def linear_splitk(xq, xs, tiled, centroids, scales, N: int, splits: int = 0, workspace=None, y=None, acc=None,
                  return_acc: bool = False, fmt: str = "s3d8", out: str = "f32"):
    """Same result as ``linear``, with the fused GEMM's input columns split
    into ``splits`` ranges whose INT32 partial sums are added before the
    epilogue (0: the library's choice for this GPU).  The workspace holds the
    partial sums and per-tile counters; it is allocated here, zero-filled,
    unless given (a given one must have been zero-filled before its first
    use; each call leaves it ready for the next)."""
    torch = _torch()
    f, o = _variant(fmt, out)
    _dev_check(xq, torch.int8, "xq")
    M, K = xq.shape
    _dev_check(xs, torch.float32, "xs", xq.device, min_numel=M)
    scales = _scales_view(scales)
    _check_weights(tiled, centroids, scales, N, K, fmt, xq.device)
    if splits == 0:
        splits = splitk_auto(M, K, N, torch.cuda.get_device_properties(xq.device).multi_processor_count)
    if splits < 1:
        raise ValueError("splits must be 0 (automatic) or positive")
    wbytes = splitk_workspace_bytes(M, K, N, splits)
    if workspace is None:
        workspace = torch.zeros((max(wbytes, 1),), dtype=torch.uint8, device=xq.device)
    _dev_check(workspace, torch.uint8, "workspace", xq.device, min_numel=wbytes)
    y = _y_out(y, M, N, out, xq.device)
    acc = _acc_out(acc, return_acc, M, N, xq.device)
    with torch.cuda.device(xq.device):
        call("s3d8_linear_splitk", xq.data_ptr(), xs.data_ptr(), M, K, N, tiled.data_ptr(), tiled.numel(),
             centroids.data_ptr(), f, scales.data_ptr(), y.data_ptr(), o,
             acc.data_ptr() if acc is not None else None, splits, workspace.data_ptr(), workspace.numel(),
             _stream(xq))
    if return_acc:
        return y, acc
    return y


def forward(x, tiled, centroids, scales, N: int, y=None, xq=None, xs=None, acc=None,
            return_all: bool = False, fmt: str = "s3d8", out: str = "f32"):
    """The whole path from fp32 x [M][K]: quantise and apply the S3D8 (or
    3D8) linear (one kernel launch for M <= 4).  Returns y, or (y, xq, xs,
    acc) with ``return_all``."""
    torch = _torch()
    f, o = _variant(fmt, out)
    _dev_check(x, torch.float32, "x")
    scales = _scales_view(scales)
    M, K = x.shape
    _check_weights(tiled, centroids, scales, N, K, fmt, x.device)
    y = _y_out(y, M, N, out, x.device)
    xq, xs = _codes_out(xq, xs, M, K, x.device)
    acc = _acc_out(acc, return_all, M, N, x.device)
    with torch.cuda.device(x.device):
        tail = (xq.data_ptr(), xs.data_ptr(), acc.data_ptr() if acc is not None else None, _stream(x))
        if f == 0 and o == 0:
            call("s3d8_forward", x.data_ptr(), M, K, N, tiled.data_ptr(), tiled.numel(), centroids.data_ptr(),
                 scales.data_ptr(), y.data_ptr(), *tail)
        else:
            call("s3d8_forward_ex", x.data_ptr(), M, K, N, tiled.data_ptr(), tiled.numel(), centroids.data_ptr(),
                 f, scales.data_ptr(), y.data_ptr(), o, *tail)
    if return_all:
        return y, xq, xs, acc
    return y


def forward_batch(items, return_all: bool = False):
    """Several ``forward`` calls in one go (one kernel launch when they fit
    the streaming GEMV together, see s3d8_forward_batch).  ``items`` is a
    list of dicts with keys x, tiled, centroids, scales, N and optionally y,
    xq, xs, acc.  Returns the list of y (or of (y, xq, xs, acc) tuples with
    ``return_all``)."""
    torch = _torch()
    arr = (_lib.ForwardItem * max(1, len(items)))()
    outs = []
    dev = None
    for i, it in enumerate(items):
        x = it["x"]
        _dev_check(x, torch.float32, "x")
        scales = _scales_view(it["scales"])
        M, K = x.shape
        N = int(it["N"])
        if dev is None:
            dev = x.device
        elif x.device != dev:
            raise ValueError("all items must be on one device")
        _check_weights(it["tiled"], it["centroids"], scales, N, K, device=dev)
        y = _y_out(it.get("y"), M, N, "f32", dev)
        xq, xs = _codes_out(it.get("xq"), it.get("xs"), M, K, dev)
        acc = _acc_out(it.get("acc"), return_all, M, N, dev)
        arr[i] = _lib.ForwardItem(x.data_ptr(), M, K, N, it["tiled"].data_ptr(), it["tiled"].numel(),
                                  it["centroids"].data_ptr(), scales.data_ptr(), y.data_ptr(), xq.data_ptr(),
                                  xs.data_ptr(), acc.data_ptr() if acc is not None else None)
        outs.append((y, xq, xs, acc, x, scales))
    if items:
        with torch.cuda.device(dev):
            call("s3d8_forward_batch", len(items), ctypes.addressof(arr), _stream(items[0]["x"]))
    if return_all:
        return [o[:4] for o in outs]
    return [o[0] for o in outs]


def encode_device(W, centroids):
    """Frozen-centroid encode on the GPU (same results as ``encode``):
    returns (scales bf16 bits as int16 [3T], packed uint8 [T][K])."""
    torch = _torch()
    _dev_check(W, torch.float32, "W")
    _dev_check(centroids, torch.uint8, "centroids")
    N, K = W.shape
    T = num_triples(N)
    scales = torch.empty((3 * T,), dtype=torch.int16, device=W.device)
    packed = torch.empty((T, K), dtype=torch.uint8, device=W.device)
    with torch.cuda.device(W.device):
        call("s3d8_encode_device", W.data_ptr(), N, K, centroids.data_ptr(), scales.data_ptr(), packed.data_ptr(),
             _stream(W))
    return scales, packed


def dequant(packed, centroids, N: int, w=None, fmt: str = "s3d8"):
    """Standalone decode to channel-INT8: w int8 [N][K]."""
    torch = _torch()
    f, _ = _variant(fmt)
    _dev_check(packed, torch.uint8, "packed")
    centroids = _table_view(centroids, fmt)
    T, K = packed.shape
    if T != num_triples(N):
        raise ValueError("packed rows do not match N")
    if w is None:
        w = torch.empty((N, K), dtype=torch.int8, device=packed.device)
    _dev_check(centroids, torch.uint8, "centroids", packed.device)
    _dev_check(w, torch.int8, "w", packed.device, numel=N * K)
    with torch.cuda.device(packed.device):
        if f == 0:
            call("s3d8_dequant", packed.data_ptr(), centroids.data_ptr(), N, K, w.data_ptr(), _stream(packed))
        else:
            call("s3d8_dequant_ex", packed.data_ptr(), centroids.data_ptr(), f, N, K, w.data_ptr(),
                 _stream(packed))
    return w


def mfma_rate_probe(iters: int, workgroups: int, v: int = 1, out=None, device="cuda"):
    """Matrix-core rate probe (a measurement utility): `workgroups` x 4
    waves each run `iters` rounds of four independent 32x32x32 INT8 MFMAs;
    every word of out (int32 [256 * workgroups]) becomes 2048 v^2 iters
    (mod 2^32).  Returns (out, integer operations performed)."""
    torch = _torch()
    if out is None:
        out = torch.empty((256 * workgroups,), dtype=torch.int32, device=device)
    _dev_check(out, torch.int32, "out")
    if out.numel() < 256 * workgroups:
        raise ValueError("out must hold 256 * workgroups int32")
    with torch.cuda.device(out.device):
        call("s3d8_mfma_rate_probe", iters, workgroups, v, out.data_ptr(), _stream(out))
    return out, workgroups * 4 * 4 * iters * 65536


def hbm_read_probe(buf, workgroups: int, out=None):
    """Memory read probe (a measurement utility): `workgroups` workgroups of
    256 threads stream the bytes of the device tensor `buf` (a multiple of 16
    bytes) and workgroup w stores the XOR of the 32-bit words it read into
    out[w] (uint32 as int32 [workgroups]).  Returns out."""
    torch = _torch()
    if not isinstance(buf, torch.Tensor) or buf.device.type != "cuda" or not buf.is_contiguous():
        raise TypeError("buf must be a contiguous CUDA/HIP torch tensor")
    if out is None:
        out = torch.empty((workgroups,), dtype=torch.int32, device=buf.device)
    _dev_check(out, torch.int32, "out", buf.device, min_numel=workgroups)
    nbytes = buf.numel() * buf.element_size()
    with torch.cuda.device(buf.device):
        call("s3d8_hbm_read_probe", buf.data_ptr(), nbytes, workgroups, out.data_ptr(), _stream(buf))
    return out


class PackedLinear:
    """An S3D8 weight matrix resident in device memory, in the tiled layout."""

    def __init__(self, centroids, scales, packed, N: int, device="cuda"):
        torch = _torch()
        self.N = int(N)
        self.K = int(packed.shape[1])
        self.centroids = torch.as_tensor(np.ascontiguousarray(centroids, np.uint8)).to(device)
        self.scales = torch.as_tensor(np.ascontiguousarray(scales, np.uint16).view(np.int16)).to(device)
        packed_dev = torch.as_tensor(np.ascontiguousarray(packed, np.uint8)).to(device)
        self.tiled = tile(packed_dev, self.N)

    @classmethod
    def from_weights(cls, W, seed: int = 1, max_iters: int = 50, device="cuda"):
        C, s, p = pack(W, seed=seed, max_iters=max_iters)
        return cls(C, s, p, W.shape[0], device)

    def __call__(self, x):
        return forward(x, self.tiled, self.centroids, self.scales, self.N)


# ------------------------------------------------------------------ 4-bit weights, group scales
def w4_tiled_bytes(N: int, K: int, group: int, zeros: bool = False) -> int:
    return int(lib().s3d8_w4_tiled_bytes(N, K, group, int(zeros)))


def w4_encode(W, group: int = 64, zeros: bool = False, num_threads: int = 0):
    """Encode W (fp32 [N][K], host) to 4-bit codes with a bf16 scale per
    ``group`` columns, with zero points if ``zeros``: (packed uint8 [N][K/2],
    scales_bf16 uint16 [N][ceil(K/group)], zeros uint8 of that shape or None)."""
    W = np.ascontiguousarray(W, dtype=np.float32)
    N, K = W.shape
    shape = (N, -(-K // max(group, 1)))
    packed = np.empty((N, K // 2), np.uint8)
    scales = np.empty(shape, np.uint16)
    z = np.empty(shape, np.uint8) if zeros else None
    call("s3d8_w4_encode", _np_ptr(W), N, K, group, num_threads, _np_ptr(packed), _np_ptr(scales),
         _np_ptr(z) if zeros else None)
    return packed, scales, z


def w4_tile(packed, scales, group: int, zeros=None, tiled=None):
    """Re-lay a device W4 matrix (packed [N][K/2], scales and optionally zeros
    [N][ceil(K/group)]) into the layout read by w4_linear (done once per
    matrix)."""
    torch = _torch()
    _dev_check(packed, torch.uint8, "packed")
    if packed.dim() != 2:
        raise ValueError(f"packed must be [N][K/2], got {tuple(packed.shape)}")
    N, K = packed.shape[0], 2 * packed.shape[1]
    scales = _scales_view(scales)
    groups = N * -(-K // max(group, 1))
    _dev_check(scales, torch.int16, "scales", packed.device, numel=groups)
    if zeros is not None:
        _dev_check(zeros, torch.uint8, "zeros", packed.device, numel=groups)
    for name, t in (("scales", scales), ("zeros", zeros)):
        if t is not None and _other_matrix(t, N):
            raise ValueError(f"{name} must be [N][ceil(K/group)], got {tuple(t.shape)}")
    nbytes = max(w4_tiled_bytes(N, K, group, zeros is not None), 0)
    if tiled is None:
        tiled = torch.empty((nbytes,), dtype=torch.uint8, device=packed.device)
    _dev_check(tiled, torch.uint8, "tiled", packed.device, numel=nbytes)
    with torch.cuda.device(packed.device):
        call("s3d8_w4_tile", packed.data_ptr(), scales.data_ptr(), zeros.data_ptr() if zeros is not None else None,
             N, K, group, tiled.data_ptr(), _stream(packed))
    return tiled


def w4_linear(xq, xs, tiled, N: int, group: int, zeros: bool = False, y=None, out: str = "f32"):
    """Linear layer on a tiled W4 matrix and pre-quantised activations: y [M][N],
    fp32 or bf16.  ``N``, ``group``, ``zeros`` (whether the matrix has zero points)
    and the width of ``xq`` as it was laid out: the size of ``tiled`` shows a
    mismatch only where it changes the number of 16-channel tiles, of 128-column
    blocks or of scales per block (a W4Linear knows its width)."""
    _dev_check(tiled, _torch().uint8, "tiled")
    return _w4_linear(xq, xs, tiled, N, group, zeros, y, out)


def _w4_linear(xq, xs, tiled, N, group, zeros, y, out):
    torch = _torch()
    o = _out_type(out)
    _dev_check(xq, torch.int8, "xq", tiled.device)
    dev = xq.device
    M, K = xq.shape
    _dev_check(xs, torch.float32, "xs", dev, min_numel=M)
    y = _y_out(y, M, N, out, dev)
    _enqueue("s3d8_w4_linear", dev, xq.data_ptr(), xs.data_ptr(), M, K, N, tiled.data_ptr(), tiled.numel(), group,
             zeros, y.data_ptr(), o)
    return y


def w4_forward(x, tiled, N: int, group: int, zeros: bool = False, y=None, xq=None, xs=None, return_all: bool = False,
               out: str = "f32"):
    """The whole path from fp32 x [M][K]: quantise, then w4_linear.  Returns y,
    or (y, xq, xs) with ``return_all``."""
    torch = _torch()
    o = _out_type(out)
    _dev_check(x, torch.float32, "x")
    dev = x.device
    M, K = x.shape
    _dev_check(tiled, torch.uint8, "tiled", dev)
    y = _y_out(y, M, N, out, dev)
    xq, xs = _codes_out(xq, xs, M, K, dev)
    _enqueue("s3d8_w4_forward", dev, x.data_ptr(), M, K, N, tiled.data_ptr(), tiled.numel(), group, zeros,
             y.data_ptr(), o, xq.data_ptr(), xs.data_ptr())
    return (y, xq, xs) if return_all else y


class W4Linear:
    """A W4 weight matrix resident in device memory, in the tiled layout
    (``packed``, ``scales``, ``zeros``: numpy arrays or device tensors; on the
    device of ``packed`` unless ``device`` says another)."""

    def __init__(self, packed, scales, group: int, zeros=None, device=None):
        torch = _torch()
        if device is None:
            device = packed.device if isinstance(packed, torch.Tensor) else "cuda"

        def resident(a, kind):
            if isinstance(a, torch.Tensor):
                return a.to(device).contiguous()
            a = np.ascontiguousarray(a)
            if a.dtype != kind:  # (float scales would become zeros)
                raise TypeError(f"packed and zeros must be uint8, scales uint16 bf16 bits, got {a.dtype}")
            return torch.as_tensor(a.view(np.int16 if kind is np.uint16 else kind)).to(device)

        packed = resident(packed, np.uint8)
        self.N, self.K, self.group, self.zeros = packed.shape[0], 2 * packed.shape[1], int(group), zeros is not None
        self.tiled = w4_tile(packed, resident(scales, np.uint16), self.group,
                             resident(zeros, np.uint8) if self.zeros else None)

    @classmethod
    def from_weights(cls, W, group: int = 64, zeros: bool = False, device="cuda"):
        packed, scales, z = w4_encode(W, group, zeros)
        return cls(packed, scales, group, z, device)

    def _check_width(self, x, func):
        # the size of the tiled matrix tells widths apart only by their number of 128-column blocks
        if isinstance(x, _torch().Tensor) and x.dim() == 2 and x.shape[1] != self.K:
            raise S3D8Error(_lib.S3D8_ERR_INVALID_ARG, func, f"activations of {x.shape[1]} columns, weights of {self.K}")

    def linear(self, xq, xs, y=None, out: str = "f32"):
        self._check_width(xq, "s3d8_w4_linear")
        return _w4_linear(xq, xs, self.tiled, self.N, self.group, self.zeros, y, out)

    def __call__(self, x, out: str = "f32"):
        self._check_width(x, "s3d8_w4_forward")
        return w4_forward(x, self.tiled, self.N, self.group, self.zeros, out=out)


# ------------------------------------------------------------------ between the linears of a block
_ROWS = {"f32": 0, "bf16": 1, "codes": 2}
_KINDS = {"rms": 0, "layer": 1}


def _row_type(t, name):
    torch = _torch()
    if isinstance(t, torch.Tensor):
        if t.dtype is torch.float32:
            return 0
        if t.dtype is torch.bfloat16:
            return 1
    raise TypeError(f"{name} must be float32 or bfloat16, got {getattr(t, 'dtype', type(t))}")


def _rows_out(out, rows, xq, xs, M, K, device):
    """The outputs of block_norm / glu_act: (rows, None, None) or (None, xq, xs)."""
    torch = _torch()
    if out not in _ROWS:
        raise ValueError(f"out must be one of {list(_ROWS)}")
    if out == "codes":
        if rows is not None:
            raise ValueError("rows goes with out='f32' or 'bf16'")
        return (None, *_codes_out(xq, xs, M, K, device))
    if xq is not None or xs is not None:
        raise ValueError("xq and xs go with out='codes'")
    dtype = torch.float32 if out == "f32" else torch.bfloat16
    if rows is None:
        rows = torch.empty(M, K, dtype=dtype, device=device)
    else:
        _dev_check(rows, dtype, "rows", device, numel=M * K)
    return rows, None, None


def _ptr(t):
    return t.data_ptr() if t is not None else 0


def block_norm(h, weight, bias=None, *, branch=None, post_weight=None, post_bias=None, gate=None,
               tanh_gate: bool = False, residual_scale: float = 1.0, eps: float = 1e-5, kind: str = "rms",
               out: str = "codes", h_out=None, rows=None, xq=None, xs=None):
    """Norm after a block, gate, residual sum, norm before the next block and its
    activation quantisation, in one launch (see s3d8_block_norm):

      h' = residual_scale * h + gate * N(branch; post_weight, post_bias),  u = N(h'; weight, bias)

    ``h``, ``branch``: fp32 or bf16 [M][K]; ``weight``, ``bias``, ``post_weight``,
    ``post_bias``: fp32 [K] (no post norm without ``post_weight``); ``gate``: fp32
    [1] or [K], used as tanh(gate) with ``tanh_gate``; ``kind``: "rms" or "layer".
    ``h_out`` may be ``h``.  Without ``branch``, u is the norm of h.

    Returns (h', xq, xs) for ``out="codes"`` and (h', u) for "f32" / "bf16";
    without ``branch``, (xq, xs) or u."""
    torch = _torch()
    if kind not in _KINDS:
        raise ValueError(f"kind must be one of {list(_KINDS)}")
    ht = _row_type(h, "h")
    _dev_check(h, h.dtype, "h")
    M, K = h.shape
    dev = h.device
    bt = 0
    if branch is not None:
        bt = _row_type(branch, "branch")
        _dev_check(branch, branch.dtype, "branch", dev, numel=M * K)
        if branch.shape != h.shape and _other_matrix(branch, M):
            raise ValueError(f"branch must be [{M}][{K}], got {tuple(branch.shape)}")
        if h_out is None:
            h_out = torch.empty_like(h)
        else:
            _dev_check(h_out, h.dtype, "h_out", dev, numel=M * K)
    elif h_out is not None:
        raise ValueError("h_out goes with branch")
    _dev_check(weight, torch.float32, "weight", dev, numel=K)
    if bias is not None:
        _dev_check(bias, torch.float32, "bias", dev, numel=K)
    if post_weight is not None:
        _dev_check(post_weight, torch.float32, "post_weight", dev, numel=K)
    if post_bias is not None:
        _dev_check(post_bias, torch.float32, "post_bias", dev, numel=K)
    channels = 0
    if gate is not None:
        channels = int(not isinstance(gate, torch.Tensor) or gate.numel() != 1)
        _dev_check(gate, torch.float32, "gate", dev, numel=K if channels else 1)
    rows, xq, xs = _rows_out(out, rows, xq, xs, M, K, dev)
    args = _lib.BLOCK_NORM_ARGS(h.data_ptr(), _ptr(branch), _ptr(post_weight), _ptr(post_bias), _ptr(gate),
                                weight.data_ptr(), _ptr(bias), _ptr(h_out), _ptr(rows), _ptr(xq), _ptr(xs), M, K,
                                eps, residual_scale, _KINDS[kind], ht, bt, _ROWS[out], channels, bool(tanh_gate))
    _enqueue("s3d8_block_norm", dev, args)
    u = (xq, xs) if rows is None else (rows,)
    if branch is not None:
        return (h_out, *u)
    return u if rows is None else rows


def glu_act(gate, up, out: str = "codes", rows=None, xq=None, xs=None):
    """SiLU(gate) * up, and its activation quantisation, in one launch (see
    s3d8_glu_act).  ``gate``, ``up``: fp32 or bf16 [M][K], rows contiguous (any row
    stride that is a multiple of 4, e.g. the halves of one [M][2K] matrix).

    Returns (xq, xs) for ``out="codes"``, the rows for "f32" / "bf16"."""
    torch = _torch()
    t = _row_type(gate, "gate")
    for name, v in (("gate", gate), ("up", up)):
        if not isinstance(v, torch.Tensor) or not v.is_cuda:
            raise TypeError(f"{name} must be a CUDA/HIP torch tensor")
        if v.dim() != 2 or v.stride(1) != 1:
            raise ValueError(f"{name} must be [M][K] with contiguous rows")
    if up.dtype != gate.dtype or up.shape != gate.shape or up.device != gate.device:
        raise ValueError("gate and up must have one type, shape and device")
    M, K = gate.shape
    dev = gate.device
    rows, xq, xs = _rows_out(out, rows, xq, xs, M, K, dev)
    _enqueue("s3d8_glu_act", dev, gate.data_ptr(), gate.stride(0) if M > 1 else K, up.data_ptr(),
             up.stride(0) if M > 1 else K, M, K, t, _ROWS[out], _ptr(rows), _ptr(xq), _ptr(xs))
    return (xq, xs) if rows is None else rows


# ------------------------------------------------------------------ heads and tokens
_SCALINGS = {"none": 0, "linear": 1, "llama3": 2, "yarn": 3}
_LAYOUTS = {"half": 0, "interleaved": 1}


class Rope:
    """The frequencies of a rotary position, kept on a device for head_rope.

    ``rotary_dim``: the entries of a head that are turned, in pairs (j, j + rotary_dim / 2)
    ("half") or (2 j, 2 j + 1) ("interleaved").  ``scaling`` stretches them for long
    contexts (see s3d8_rope_frequencies): "linear" by ``factor``; "llama3" by ``factor``
    below ``low`` turns over ``original_length`` positions, not above ``high``; "yarn"
    between the pairs of ``beta_slow`` and ``beta_fast`` turns, with cosine and sine times
    ``attention_factor`` (0.1 ln(factor) + 1 unless given).  ``frequencies``: float64
    [rotary_dim / 2] on ``device``."""

    def __init__(self, rotary_dim: int, base: float = 10000.0, *, layout: str = "half", scaling: str = "none",
                 factor: float = 1.0, original_length: float = 8192, low: float = 1.0, high: float = 4.0,
                 beta_fast: float = 32.0, beta_slow: float = 1.0, attention_factor=None, device="cuda"):
        torch = _torch()
        if layout not in _LAYOUTS:
            raise ValueError(f"layout must be one of {list(_LAYOUTS)}")
        if scaling not in _SCALINGS:
            raise ValueError(f"scaling must be one of {list(_SCALINGS)}")
        if scaling == "yarn":
            low, high = beta_slow, beta_fast
        self.rotary_dim, self.layout = int(rotary_dim), layout
        f = np.empty(max(self.rotary_dim // 2, 1), np.float64)
        own = ctypes.c_double()
        call("s3d8_rope_frequencies", self.rotary_dim, base, _SCALINGS[scaling], factor, original_length, low, high,
             _np_ptr(f), ctypes.byref(own))
        self.factor = own.value if attention_factor is None else float(attention_factor)
        self.frequencies = torch.as_tensor(f).to(device)


def _heads(t, name, dtype=None, shape=None, device=None):
    """A device tensor [M][heads][D] with the entries of a head in a row: its row
    and head strides."""
    if not isinstance(t, _torch().Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA/HIP torch tensor")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if t.dim() != 3 or (shape is not None and t.shape != shape):
        raise ValueError(f"{name} must be {list(shape) if shape is not None else '[M][heads][D]'}, got {tuple(t.shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the other arguments on {device}")
    M, H, D = t.shape
    row, head, one = t.stride()
    if one != 1 and D > 1:
        raise ValueError(f"the entries of a head of {name} must be contiguous")
    return (row if M > 1 else 0), (head if H > 1 else 0)


def head_rope(q, k=None, positions=None, rope=None, *, q_weight=None, k_weight=None, eps: float = 1e-5,
              out: str = "bf16", q_out=None, k_out=None):
    """The RMS norm of each query and key head and its rotary position, in one
    launch (see s3d8_head_rope).  ``q``, ``k``: fp32 or bf16 [M][heads][D] with any
    row and head strides, e.g. parts of one [M][(heads + 2 kv_heads) D] matrix;
    ``positions``: int32 or int64 [M], with ``rope`` (a Rope); ``q_weight``,
    ``k_weight``: fp32 [D], the norms' (none without).  ``out``: "bf16" or "f32";
    ``q_out``, ``k_out`` (rows of a cache, or q and k themselves) take the results.

    Returns (q', k'), or q' without ``k``."""
    torch = _torch()
    o = _out_type(out)
    t = _row_type(q, "q")
    strides = [*_heads(q, "q")]
    M, H, D = q.shape
    dev = q.device
    dtype = torch.bfloat16 if o else torch.float32
    Hk = 0
    if k is not None:
        if not isinstance(k, torch.Tensor) or k.dim() != 3:
            raise TypeError("k must be a CUDA/HIP torch tensor [M][heads][D]")
        Hk = k.shape[1]
        strides += _heads(k, "k", q.dtype, (M, Hk, D), dev)
    elif k_out is not None or k_weight is not None:
        raise ValueError("k_out and k_weight go with k")
    else:
        strides += (0, 0)
    if q_out is None:
        q_out = torch.empty(M, H, D, dtype=dtype, device=dev)
        strides += (H * D, D)
    else:
        strides += _heads(q_out, "q_out", dtype, (M, H, D), dev)
    if k is None:
        strides += (0, 0)
    elif k_out is None:
        k_out = torch.empty(M, Hk, D, dtype=dtype, device=dev)
        strides += (Hk * D, D)
    else:
        strides += _heads(k_out, "k_out", dtype, (M, Hk, D), dev)
    if q_weight is not None:
        _dev_check(q_weight, torch.float32, "q_weight", dev, numel=D)
    if k_weight is not None:
        _dev_check(k_weight, torch.float32, "k_weight", dev, numel=D)
    if (positions is None) != (rope is None):
        raise ValueError("positions and rope go together")
    wide, frequencies, rotary_dim, factor, side_by_side = False, None, 0, 1.0, False
    if rope is not None:
        wide = isinstance(positions, torch.Tensor) and positions.dtype is torch.int64
        _dev_check(positions, torch.int64 if wide else torch.int32, "positions", dev, numel=M)
        frequencies, rotary_dim, factor = rope.frequencies, rope.rotary_dim, rope.factor
        side_by_side = rope.layout == "interleaved"
        _dev_check(frequencies, torch.float64, "rope.frequencies", dev, numel=rotary_dim // 2)
    _enqueue("s3d8_head_rope", dev,
             _lib.HEAD_ROPE_ARGS(q.data_ptr(), _ptr(k), q_out.data_ptr(), _ptr(k_out), _ptr(q_weight), _ptr(k_weight),
                                 _ptr(positions), _ptr(frequencies), M, H, Hk, D, rotary_dim, *strides, eps, factor, t, o,
                                 wide, side_by_side))
    return q_out if k is None else (q_out, k_out)


_workspace_bytes = {}


def _workspace(name, dev, key, args) -> int:
    """Workspace bytes of an entry point on a device, remembered by what they depend on."""
    key = (name, dev.index, key)
    nbytes = _workspace_bytes.get(key)
    if nbytes is None:
        nbytes = getattr(lib(), name)(args(), _torch().cuda.get_device_properties(dev).multi_processor_count)
        if len(_workspace_bytes) >= 4096:
            _workspace_bytes.clear()
        _workspace_bytes[key] = nbytes
    return nbytes


def _result(t, dtype, name, dev, shape):
    """A caller's buffer for a result of ``shape``, or of that shape with neighbouring dimensions joined: another
    order of the dimensions has as many elements, but not in these places."""
    _dev_check(t, dtype, name, dev, numel=math.prod(shape))
    left = [n for n in shape if n != 1]
    for n in t.shape:
        size = 1
        while size < n and left:
            size *= left.pop(0)
        if size != n:
            raise ValueError(f"{name} must be {list(shape)}, or that with neighbouring dimensions joined, got {tuple(t.shape)}")


def cross_attention(q, k, v, *, kv_lens=None, mask=None, scale=None, out: str = "bf16", o=None, xq=None, xs=None):
    """Attention of query tokens to an encoder's states (see s3d8_cross_attention).

    ``q``: bf16 [B][Lq][heads][D]; ``k``, ``v``: bf16 [B][Lk][kv_heads][D], or [1]... for
    states that all sequences share; any strides that are multiples of 8, the entries of
    a head in a row.  ``kv_lens``: int32 [B] ([1] if shared), the states of each sequence
    (all Lk without).  ``mask``: bool [B or 1][Lq or 1][Lk], true where a token sees a
    state.  A token that sees none has 0.  ``scale``: 1 / sqrt(D) unless given.  ``o`` takes the
    result (also as [B][Lq][heads D] or [B Lq][heads D]; not over q, k or v).

    Returns o bf16 [B][Lq][heads][D], or its INT8 codes and scales for the output
    projection (xq [B Lq][heads D], xs [B Lq]) with ``out="codes"``."""
    torch = _torch()
    if out not in ("bf16", "codes"):
        raise ValueError("out must be one of ['bf16', 'codes']")
    bf16 = torch.bfloat16
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA/HIP torch tensor")
        if t.dtype is not bf16:
            raise TypeError(f"{name} must have dtype {bf16}, got {t.dtype}")
        if t.dim() != 4 or (t.stride(3) != 1 and t.shape[3] > 1):
            raise ValueError(f"{name} must be [B][L][heads][D], the entries of a head contiguous")
    dev = q.device
    if k.device != dev or v.device != dev:
        raise ValueError("q, k and v must be on one device")
    B, Lq, H, D = q.shape
    Bk, Lk, Hk, Dk = k.shape
    if v.shape != k.shape or Dk != D or (Bk != B and Bk != 1):
        raise ValueError(f"k and v must be [{B} or 1][Lk][kv_heads][{D}], got {tuple(k.shape)} and {tuple(v.shape)}")
    shared = Bk == 1 and B > 1
    strides = []
    for (seq, row, head, _), n in ((q.stride(), q.shape), (k.stride(), k.shape), (v.stride(), v.shape)):
        strides += (seq if n[0] > 1 else 0, row if n[1] > 1 else 0, head if n[2] > 1 else 0)
    if kv_lens is not None:
        _dev_check(kv_lens, torch.int32, "kv_lens", dev, numel=Bk)
    mask_seq = mask_row = 0
    if mask is not None:
        if not isinstance(mask, torch.Tensor) or not mask.is_cuda:
            raise TypeError("mask must be a CUDA/HIP torch tensor")
        if mask.dtype is not torch.bool:
            raise TypeError(f"mask must have dtype torch.bool, got {mask.dtype}")
        if mask.device != dev:
            raise ValueError(f"mask is on {mask.device}, the other arguments on {dev}")
        if mask.dim() != 3 or mask.shape[0] not in (1, B) or mask.shape[1] not in (1, Lq) or mask.shape[2] != Lk or (
                mask.stride(2) != 1 and Lk > 1):
            raise ValueError(f"mask must be [{B} or 1][{Lq} or 1][{Lk}], its rows contiguous, got {tuple(mask.shape)}")
        mask_seq = mask.stride(0) if mask.shape[0] > 1 else 0
        mask_row = mask.stride(1) if mask.shape[1] > 1 else 0
    if o is None:
        o = torch.empty(B, Lq, H, D, dtype=bf16, device=dev)
    else:
        _result(o, bf16, "o", dev, (B, Lq, H, D))
    if out == "codes":
        xq, xs = _codes_out(xq, xs, B * Lq, H * D, dev)
    elif xq is not None or xs is not None:
        raise ValueError("xq and xs go with out='codes'")
    if scale is None:
        scale = D ** -0.5 if D else 1.0
    sizes = (B, Lq, Lk, H, Hk, D, *strides, mask_seq, mask_row, scale, shared)
    nbytes = _workspace("s3d8_cross_attention_workspace_bytes", dev,
                        (B, Lq, Lk, H, Hk, D, shared, mask is not None, mask_seq != 0, mask_row != 0),
                        lambda: _lib.CROSS_ATTENTION_ARGS(0, 0, 0, 0, _ptr(mask), 0, 0, 0, 0, 0, *sizes))
    workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes > 0 else None
    _enqueue("s3d8_cross_attention", dev,
             _lib.CROSS_ATTENTION_ARGS(q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(kv_lens), _ptr(mask), o.data_ptr(),
                                       _ptr(xq), _ptr(xs), _ptr(workspace), max(nbytes, 0), *sizes))
    return o if out == "bf16" else (xq, xs)


def sample(logits, u, *, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, token=None, prob=None):
    """The next token of each row of logits, from a random number (see s3d8_sample).

    ``logits``: fp32 or bf16 [M][V], rows contiguous, any distance apart; ``u``: fp32 [M],
    uniform from [0, 1); ``temperature`` (0: the largest logit), ``top_k`` (0: all), ``top_p``
    (1: all), ``min_p`` (0: all): a number, or a device tensor [M] (fp32, ``top_k`` int32).
    ``token``, ``prob``: buffers [M] for the results.

    Returns (token int32 [M], prob fp32 [M]), the probability among the tokens kept;
    -1 and 0 for a row of -infinity."""
    torch = _torch()
    t = _row_type(logits, "logits")
    if not logits.is_cuda:
        raise TypeError("logits must be a CUDA/HIP torch tensor")
    if logits.dim() != 2 or (logits.stride(1) != 1 and logits.shape[1] > 1):
        raise ValueError("logits must be [M][V] with contiguous rows")
    M, V = logits.shape
    dev = logits.device
    _dev_check(u, torch.float32, "u", dev, numel=M)
    pointers, numbers = [], []
    for name, x, dtype in (("temperature", temperature, torch.float32), ("top_k", top_k, torch.int32),
                           ("top_p", top_p, torch.float32), ("min_p", min_p, torch.float32)):
        if isinstance(x, torch.Tensor):
            _dev_check(x, dtype, name, dev, numel=M)
            pointers.append(x.data_ptr())
            numbers.append(0)
        else:
            pointers.append(0)
            numbers.append(x)
    numbers[1] = max(-1, min(int(numbers[1]), 0x7FFFFFFF))
    if token is None:
        token = torch.empty(M, dtype=torch.int32, device=dev)
    else:
        _result(token, torch.int32, "token", dev, (M,))
    if prob is None:
        prob = torch.empty(M, dtype=torch.float32, device=dev)
    else:
        _result(prob, torch.float32, "prob", dev, (M,))
    tail = (M, V, logits.stride(0) if M > 1 else V, *numbers, t)
    # what the workspace's size depends on
    nbytes = _workspace("s3d8_sample_workspace_bytes", dev, (M, V, t, numbers[1], pointers[1] != 0, pointers[2] != 0),
                        lambda: _lib.SAMPLE_ARGS(0, 0, *pointers, 0, 0, 0, 0, *tail))
    workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes > 0 else None
    _enqueue("s3d8_sample", dev,
             _lib.SAMPLE_ARGS(logits.data_ptr(), u.data_ptr(), *pointers, token.data_ptr(), prob.data_ptr(),
                              _ptr(workspace), max(nbytes, 0), *tail))
    return token, prob
