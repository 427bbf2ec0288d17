"""Host side of the 4-bit linear layer, the block norm and the gated
activation: the encoder against a plain one, size helpers, and every refusal
of the C entry points (which come before any GPU call)."""
import ctypes

import numpy as np
import pytest

import block_reference as ref
import workloads
from w2_a8_matmul_amd import _lib, w4_encode, w4_tiled_bytes

A = 0x10000  # device-looking addresses, never touched: validation fails first
OK, INVALID, SHAPE, ALIGN = _lib.S3D8_OK, _lib.S3D8_ERR_INVALID_ARG, _lib.S3D8_ERR_SHAPE, _lib.S3D8_ERR_ALIGN


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("N,K,group", [(1, 16, 32), (3, 32, 32), (5, 80, 32), (17, 208, 64), (4, 400, 128),
                                       (2, 272, 96), (2, 64, 4096)])
def test_encode_matches_the_plain_encoder(N, K, group, zeros):
    W = workloads.gaussian_matrix([7100, N, K, group], N, K, 0.02)
    W[0, :group] = 0.0          # a group without a scale
    W[-1] = np.abs(W[-1])       # one-sided groups
    W[N // 2, 0] = -0.0
    packed, scales, z = w4_encode(W, group, zeros)
    q_r, s_r, z_r = ref.w4_encode(W, group, zeros)
    assert np.array_equal(scales, s_r)
    assert np.array_equal(packed, ref.pack(q_r))
    assert (z is None) if not zeros else np.array_equal(z, z_r)


def test_encode_extremes():
    W = np.zeros((4, 32), np.float32)
    W[0, ::2], W[0, 1::2] = 7.0, -7.0
    W[1, 0] = 1e-40                       # subnormal: the bf16 scale is subnormal too, or 0
    W[2] = 3.0e38
    W[3] = np.arange(32, dtype=np.float32) - 15.5
    for zeros in (False, True):
        packed, scales, z = w4_encode(W, 32, zeros)
        q_r, s_r, z_r = ref.w4_encode(W, 32, zeros)
        assert np.array_equal(scales, s_r) and np.array_equal(packed, ref.pack(q_r))
    packed, scales, _ = w4_encode(W, 32)
    assert ref.bf16_value(scales)[0, 0] == 1.0 and packed[0, 0] == 15 | (1 << 4)


@pytest.mark.parametrize("threads", [1, 2, 7, 1000])
def test_encode_does_not_depend_on_the_threads(threads):
    W = workloads.gaussian_matrix([7101], 40, 96)
    base = w4_encode(W, 32, True)
    for a, b in zip(base, w4_encode(W, 32, True, num_threads=threads)):
        assert np.array_equal(a, b)


def test_tiled_bytes():
    assert w4_tiled_bytes(14336, 4096, 64) == 896 * 32 * (1024 + 64)
    assert w4_tiled_bytes(14336, 4096, 128, True) == 896 * 32 * (1024 + 48)
    assert w4_tiled_bytes(1, 16, 32) == 1024 + 32        # one group, whatever its size
    assert w4_tiled_bytes(17, 144, 32, True) == 2 * 2 * (1024 + 4 * 48)
    assert w4_tiled_bytes(16, 256, 96) == 2 * (1024 + 128)   # 96 is three groups of 32
    for bad in ((0, 16, 32), (16, 0, 32), (16, 16, 0), (16, 16, 48), (-1, 16, 32), (1 << 62, 16, 32)):
        assert w4_tiled_bytes(*bad) == -1


def _rc(name, *args):
    rc = getattr(_lib.lib(), name)(*args)
    assert rc == OK or _lib.lib().s3d8_last_error()
    return rc


def test_encode_refusals():
    W = np.zeros((2, 32), np.float32)
    p, s = np.empty(64, np.uint8), np.empty(8, np.uint16)
    a = [W.ctypes.data, 2, 32, 32, 1, p.ctypes.data, s.ctypes.data, None]

    def call(i, v):
        return _rc("s3d8_w4_encode", *(a[:i] + [v] + a[i + 1:]))

    assert call(4, 1) == OK
    assert call(0, None) == INVALID and call(5, None) == INVALID and call(6, None) == INVALID
    assert call(1, 0) == INVALID and call(2, -16) == INVALID and call(3, 0) == INVALID
    assert call(2, 24) == SHAPE and call(3, 48) == SHAPE


def test_tile_refusals():
    good = dict(p=A, s=A, z=None, N=16, K=128, g=32, t=A)

    def call(**kw):
        a = {**good, **kw}
        return _rc("s3d8_w4_tile", a["p"], a["s"], a["z"], a["N"], a["K"], a["g"], a["t"], None)

    assert call(p=None) == INVALID and call(s=None) == INVALID and call(t=None) == INVALID
    assert call(N=0) == INVALID and call(K=-16) == INVALID and call(g=0) == INVALID
    assert call(K=24) == SHAPE and call(g=33) == SHAPE
    assert call(N=1 << 20, K=1 << 13) == SHAPE and call(N=1 << 62) == SHAPE and call(K=1 << 62) == SHAPE
    assert call(t=A + 8) == ALIGN and call(s=A + 1) == ALIGN


@pytest.mark.parametrize("entry", ["linear", "forward"])
def test_linear_refusals(entry):
    good = dict(x=A, xs=A, M=2, K=128, N=16, t=A, tb=None, g=32, z=0, y=A, o=0, xq=A)

    def call(**kw):
        a = {**good, **kw}
        if a["tb"] is None:
            a["tb"] = w4_tiled_bytes(a["N"], a["K"], a["g"], bool(a["z"]))
        head = (a["M"], a["K"], a["N"], a["t"], a["tb"], a["g"], a["z"], a["y"], a["o"])
        if entry == "linear":
            return _rc("s3d8_w4_linear", a["xq"], a["xs"], *head, None)
        return _rc("s3d8_w4_forward", a["x"], *head, a["xq"], a["xs"], None)

    for k in ("xq", "xs", "t", "y") + (("x",) if entry == "forward" else ()):
        assert call(**{k: None}) == INVALID, k
    assert call(M=0) == INVALID and call(N=0) == INVALID and call(K=0) == INVALID and call(g=-32) == INVALID
    assert call(o=2) == INVALID and call(z=2, tb=1) == INVALID
    assert call(K=120) == SHAPE and call(g=48) == SHAPE
    assert call(M=(1 << 19) + 1) == SHAPE and call(M=1 << 40) == SHAPE and call(N=1 << 40) == SHAPE
    assert call(M=17, K=16, N=1 << 22) == SHAPE
    assert call(M=1 << 19, K=1 << 13) == SHAPE and call(M=1 << 18, N=1 << 13) == SHAPE
    # laid out for other arguments
    assert call(tb=16 * 64) == INVALID
    assert call(tb=w4_tiled_bytes(16, 128, 64)) == INVALID
    assert call(tb=w4_tiled_bytes(16, 128, 32, True)) == INVALID
    for k, v in (("xq", A + 8), ("t", A + 4), ("xs", A + 2), ("y", A + 2)):
        assert call(**{k: v}) == ALIGN, k
    if entry == "forward":
        assert call(x=A + 4) == ALIGN


def test_block_norm_refusals():
    good = dict(h=A, branch=A, post_weight=A, post_bias=None, gate=A, weight=A, bias=None, h_out=A, rows=None, xq=A,
                xs=A, M=2, K=64, residual_scale=1.0, eps=1e-5, kind=0, h_type=0, branch_type=1, out_type=2,
                gate_channels=0, gate_tanh=0)

    def call(**kw):
        args = _lib.BlockNormArgs(**{**good, **kw})
        return _rc("s3d8_block_norm", ctypes.addressof(args), None)

    assert _rc("s3d8_block_norm", None, None) == INVALID
    assert call(h=None) == INVALID and call(weight=None) == INVALID
    assert call(h_out=None) == INVALID and call(branch=None) == INVALID
    assert call(branch=None, h_out=None) == INVALID                      # a post norm without a branch
    assert call(branch=None, h_out=None, post_weight=None) == INVALID    # a gate without one
    assert call(kind=2) == INVALID and call(bias=A) == INVALID and call(post_bias=A) == INVALID
    assert call(kind=1, post_weight=None, post_bias=A) == INVALID
    assert call(h_type=2) == INVALID and call(branch_type=-1) == INVALID and call(out_type=3) == INVALID
    assert call(rows=A) == INVALID and call(xq=None) == INVALID and call(xs=None) == INVALID
    assert call(out_type=0) == INVALID and call(out_type=1, rows=A, xs=None) == INVALID
    assert call(eps=0.0) == INVALID and call(eps=-1.0) == INVALID and call(eps=float("nan")) == INVALID
    assert call(M=0) == INVALID and call(K=0) == INVALID
    assert call(K=40) == SHAPE and call(K=65552) == SHAPE and call(M=(1 << 19) + 1) == SHAPE
    for k in ("h", "branch", "post_weight", "weight", "h_out", "xq"):
        assert call(**{k: A + 8}) == ALIGN, k
    assert call(gate=A + 2) == ALIGN and call(gate=A + 4, gate_channels=1) == ALIGN and call(xs=A + 2) == ALIGN
    assert call(kind=1, bias=A + 4) == ALIGN and call(out_type=0, rows=A + 8, xq=None, xs=None) == ALIGN


def test_glu_refusals():
    good = dict(g=A, lg=64, u=A, lu=64, M=2, K=64, t=0, o=2, rows=None, xq=A, xs=A)

    def call(**kw):
        a = {**good, **kw}
        return _rc("s3d8_glu_act", *a.values(), None)

    assert call(g=None) == INVALID and call(u=None) == INVALID
    assert call(t=2) == INVALID and call(o=5) == INVALID
    assert call(M=0) == INVALID and call(K=0) == INVALID
    assert call(K=72, lg=72, lu=72) == SHAPE and call(K=1 << 17, lg=1 << 17, lu=1 << 17) == SHAPE
    assert call(M=1 << 20) == SHAPE
    assert call(lg=60) == INVALID and call(lu=32) == INVALID and call(lu=1 << 60) == INVALID
    assert call(lg=66) == ALIGN and call(lu=70) == ALIGN
    assert call(g=A + 8) == ALIGN and call(u=A + 8) == ALIGN and call(t=1, u=A + 4) == ALIGN
    assert call(xq=A + 8) == ALIGN and call(xs=A + 1) == ALIGN
    assert call(rows=A) == INVALID and call(xq=None) == INVALID and call(o=1) == INVALID
    assert call(o=0, rows=A + 8, xq=None, xs=None) == ALIGN


def test_encode_ranges_past_the_largest_fp32():
    """Finite groups whose hi - lo is over the largest fp32: a finite scale, the codes of the definition with it."""
    ends = [(3.0e38, -3.0e38), (2.5e38, -1.5e38), (1.0e38, -3.25e38), (3.4028235e38, -3.4028235e38)]
    W = np.zeros((len(ends), 32), np.float32)
    for r, (hi, lo) in enumerate(ends):
        W[r] = np.linspace(lo, hi, 32, dtype=np.float64).astype(np.float32)
    packed, scales, z = w4_encode(W, 32, True)
    wide = W.astype(np.float64)
    # the range in 64 bits; rounded to fp32, then to bf16 (none of these lies near a border of the latter)
    s = ref.bf16_bits(((wide.max(1) - wide.min(1)) / 15).astype(np.float32))
    assert np.array_equal(scales[:, 0], s)
    step = ref.bf16_value(s).astype(np.float64)[:, None]
    z_r = np.clip(np.rint(-wide.min(1, keepdims=True) / step), 0, 15)
    q_r = np.clip(np.rint(wide / step) + z_r, 0, 15).astype(np.uint8)
    assert np.array_equal(z, z_r) and np.array_equal(packed, ref.pack(q_r))
    # without zero points the largest magnitude decides, which cannot overflow
    packed, scales, _ = w4_encode(W, 32)
    q_r, s_r, _ = ref.w4_encode(W, 32, False)
    assert np.isfinite(ref.bf16_value(scales)).all()
    assert np.array_equal(scales, s_r) and np.array_equal(packed, ref.pack(q_r))


def test_block_norm_eps_range():
    """1 / sqrt(eps), what a zero row is multiplied by, has to be a finite fp32 number, and not 0."""
    good = dict(h=A, weight=A, xq=A + 8, xs=A, M=2, K=64, residual_scale=1.0, kind=0, h_type=0, branch_type=0,
                out_type=2)  # (xq is misaligned, which is refused after eps)

    def call(eps):
        args = _lib.BlockNormArgs(**good, eps=eps)
        return _rc("s3d8_block_norm", ctypes.addressof(args), None)

    for eps in (float("inf"), 1e-80, 5e-324, 2.0 ** -252 * (1 - 2.0 ** -52), 2.0 ** 252 * (1 + 2.0 ** -52)):
        assert call(eps) == INVALID, eps
    for eps in (2.0 ** -252, 1e-12, 1e-5, 1.0, 2.0 ** 252):
        assert call(eps) == ALIGN, eps
