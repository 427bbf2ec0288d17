"""The operators of heads and tokens on the host (no GPU): rotary frequencies
against a form of their own, workspace sizes, and what the entry points refuse
before anything is queued."""
import ctypes

import numpy as np
import pytest

import head_reference as ref
import w2_a8_matmul_amd as s3d8
from w2_a8_matmul_amd import _lib

A16 = 0x10000  # never touched


def rc(name, args):
    return getattr(_lib.lib(), name)(ctypes.byref(args) if args is not None else None, None)


def frequencies(rot, base=10000.0, scaling=0, factor=1.0, length=8192.0, low=1.0, high=4.0):
    f, a = np.full(128, -1.0), ctypes.c_double(-1)
    status = _lib.lib().s3d8_rope_frequencies(rot, base, scaling, factor, length, low, high, f.ctypes.data, ctypes.byref(a))
    return status, f, a.value


@pytest.mark.parametrize("rot", [2, 10, 64, 128, 256])
@pytest.mark.parametrize("scaling", ["none", "linear", "llama3", "yarn"])
@pytest.mark.parametrize("base,factor,length,low,high", [(10000.0, 4.0, 4096, 1.0, 32.0), (500000.0, 8.0, 8192, 1.0, 4.0),
                                                         (1e6, 1.0, 32768, 1.0, 32.0), (10.0, 40.0, 16, 0.5, 2.0)])
def test_rope_frequencies(rot, scaling, base, factor, length, low, high):
    status, f, a = frequencies(rot, base, ["none", "linear", "llama3", "yarn"].index(scaling), factor, length, low, high)
    want, factor_a = ref.frequencies(rot, base, scaling, factor, length, low, high)
    assert status == 0 and (f[rot // 2:] == -1).all()
    np.testing.assert_allclose(f[:rot // 2], want, rtol=1e-13)
    assert a == pytest.approx(factor_a, rel=1e-15)


def test_rope_frequencies_refusals():
    nan = float("nan")
    assert _lib.lib().s3d8_rope_frequencies(8, 1e4, 0, 1.0, 1.0, 1.0, 2.0, None, None) == _lib.S3D8_ERR_INVALID_ARG
    for rot in (0, -2, 3, 258):
        assert frequencies(rot)[0] == _lib.S3D8_ERR_SHAPE
    for kw in (dict(base=1.0), dict(base=nan), dict(base=float("inf")), dict(scaling=4), dict(scaling=-1),
               dict(scaling=1, factor=0.5), dict(scaling=1, factor=nan), dict(scaling=2, length=0.0),
               dict(scaling=2, low=4.0), dict(scaling=3, low=0.0), dict(scaling=3, high=nan)):
        assert frequencies(8, **kw)[0] == _lib.S3D8_ERR_INVALID_ARG
    for kw in (dict(layout="other"), dict(scaling="other")):
        with pytest.raises(ValueError):
            s3d8.Rope(8, device="cpu", **kw)
    with pytest.raises(s3d8.S3D8Error):
        s3d8.Rope(7, device="cpu")


def test_rope_handle():
    r = s3d8.Rope(8, 100.0, layout="interleaved", scaling="yarn", factor=2.0, original_length=64, device="cpu")
    f, a = ref.frequencies(8, 100.0, "yarn", 2.0, 64, 1.0, 32.0)
    np.testing.assert_allclose(r.frequencies.numpy(), f, rtol=1e-13)
    assert r.factor == pytest.approx(a)
    assert s3d8.Rope(8, scaling="yarn", factor=2.0, attention_factor=1.0, device="cpu").factor == 1.0


def rope_args(**kw):
    a = dict(q=A16, k=A16, q_out=A16, k_out=A16, positions=A16, frequencies=A16, M=4, q_heads=4, k_heads=2, D=64,
             rotary_dim=64, q_row=256, q_head=64, k_row=128, k_head=64, q_out_row=256, q_out_head=64, k_out_row=128,
             k_out_head=64, eps=1e-5, factor=1.0, in_type=1, out_type=1, positions_64=1, interleaved=0)
    a.update(kw)
    return _lib.HeadRopeArgs(**a)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(q_out=None), 1), (dict(k=None), 1), (dict(k_out=None), 1), (dict(k_heads=0), 1),
    (dict(k=None, k_out=None, k_heads=0, k_weight=A16), 1), (dict(M=0), 1), (dict(D=0), 1), (dict(q_heads=-1), 1),
    (dict(rotary_dim=-2), 1), (dict(D=63), 2), (dict(D=258, rotary_dim=64), 2), (dict(rotary_dim=66), 2), (dict(rotary_dim=31), 2),
    (dict(M=(1 << 19) + 1), 2), (dict(q_heads=4097), 2), (dict(M=1 << 19, q_heads=127), 2), (dict(positions=None), 1), (dict(frequencies=None), 1),
    (dict(rotary_dim=0), 1), (dict(in_type=2), 1), (dict(out_type=3), 1), (dict(eps=0.0), 1), (dict(eps=float("nan")), 1),
    (dict(factor=float("inf")), 1), (dict(factor=float("nan")), 1), (dict(q_row=63), 1), (dict(k_out_head=32), 1),
    (dict(k_row=-128), 1), (dict(q_row=1 << 41), 1), (dict(q=A16 + 1), 3), (dict(q_out=A16 + 2, out_type=0), 3),
    (dict(positions=A16 + 4), 3), (dict(frequencies=A16 + 4), 3), (dict(q_weight=A16 + 2), 3)])
def test_head_rope_refusals(kw, status):
    assert rc("s3d8_head_rope", rope_args(**kw)) == status
    assert _lib.lib().s3d8_last_error()


def attention_args(**kw):
    a = dict(q=A16, k=A16, v=A16, o=A16, B=2, Lq=3, Lk=100, heads=4, kv_heads=2, D=64, q_seq=768, q_row=256, q_head=64,
             k_seq=12800, k_row=128, k_head=64, v_seq=12800, v_row=128, v_head=64, scale=0.125)
    a.update(kw)
    return _lib.CrossAttentionArgs(**a)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(o=None), 1), (dict(B=0), 1), (dict(Lq=0), 1), (dict(Lk=0), 1),
    (dict(heads=0), 1), (dict(kv_heads=0), 1), (dict(D=0), 1), (dict(D=72), 2), (dict(D=144), 2), (dict(heads=5), 2),
    (dict(heads=8192), 2), (dict(B=65536), 2), (dict(Lq=(1 << 24) + 1), 2), (dict(Lk=(1 << 24) + 1), 2),
    (dict(B=1024, Lq=1 << 19), 2), (dict(xq=A16), 1), (dict(xs=A16), 1), (dict(scale=0.0), 1), (dict(scale=-1.0), 1),
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(q_row=252), 3), (dict(k_head=4), 3),
    (dict(v_seq=-8), 1), (dict(q_seq=1 << 41), 1), (dict(k_row=56), 1), (dict(v_row=0), 1), (dict(k_row=1 << 23), 1),
    (dict(mask=A16, mask_row=-1), 1), (dict(q=A16 + 8), 3), (dict(v=A16 + 2), 3), (dict(o=A16 + 8), 3),
    (dict(workspace=A16 + 8), 3), (dict(kv_lens=A16 + 2), 3), (dict(xq=A16, xs=A16 + 2), 3),
    (dict(xq=A16, xs=A16, heads=2048, kv_heads=1), 2), (dict(xq=A16, xs=A16, Lq=1 << 19), 2)])
def test_cross_attention_refusals(kw, status):
    assert rc("s3d8_cross_attention", attention_args(**kw)) == status
    assert _lib.lib().s3d8_last_error()


def test_cross_attention_workspace():
    def size(cus=256, **kw):
        a = attention_args(**kw)
        return _lib.lib().s3d8_cross_attention_workspace_bytes(ctypes.byref(a), cus)

    assert size(D=72) == -1 and size(cus=0) == -1 and size(Lk=0) == -1
    assert _lib.lib().s3d8_cross_attention_workspace_bytes(None, 256) == -1
    assert size(Lk=64) == 0                                  # one block of keys: nothing to split
    assert size(Lk=64, mask=A16, mask_seq=300, mask_row=100) == 2 * 3 * 8
    assert size(Lk=64, mask=A16, mask_row=100) == 32         # one mask for both sequences, in 16 bytes
    assert size(Lk=64, mask=A16) == 16
    assert size(Lk=4096) > 0
    assert size(Lk=4096, B=4096) == 0                        # as many workgroups as the device takes


def sample_args(**kw):
    a = dict(logits=A16, u=A16, token=A16, M=2, V=100, row=100, temperature_all=1.0, top_k_all=0, top_p_all=1.0, min_p_all=0.0,
             type=0)
    a.update(kw)
    return _lib.SampleArgs(**a)


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), 1), (dict(u=None), 1), (dict(token=None), 1), (dict(M=0), 1), (dict(V=0), 1), (dict(V=262145), 2),
    (dict(M=(1 << 19) + 1), 2), (dict(type=2), 1), (dict(row=99), 1), (dict(row=-1, M=1), 1), (dict(row=1 << 41), 1),
    (dict(temperature_all=-0.5), 1), (dict(temperature_all=float("nan")), 1), (dict(temperature_all=float("inf")), 1),
    (dict(top_k_all=-1), 1), (dict(top_p_all=1.5), 1), (dict(top_p_all=-0.1), 1), (dict(top_p_all=float("nan")), 1),
    (dict(min_p_all=1.5), 1), (dict(min_p_all=float("nan")), 1), (dict(logits=A16 + 2), 3), (dict(logits=A16 + 1, type=1), 3),
    (dict(u=A16 + 1), 3), (dict(top_k=A16 + 2), 3), (dict(prob=A16 + 2), 3), (dict(workspace=A16 + 8), 3)])
def test_sample_refusals(kw, status):
    assert rc("s3d8_sample", sample_args(**kw)) == status
    assert _lib.lib().s3d8_last_error()


def test_sample_workspace():
    def size(cus=256, **kw):
        a = sample_args(**kw)
        return _lib.lib().s3d8_sample_workspace_bytes(ctypes.byref(a), cus)

    assert size(V=0) == -1 and size(V=262145) == -1 and size(type=2) == -1 and size(cus=0) == -1
    assert _lib.lib().s3d8_sample_workspace_bytes(None, 256) == -1
    assert size() == size(top_k=A16) == size(V=3584) == 0        # a row's tokens are all listed
    V = 128256
    assert 0 < size(V=V) < size(V=V, top_k=A16)                  # rows with and without a top-k
    assert size(V=V, top_k_all=50) != size(V=V) and size(V=V, top_k_all=V) == size(V=V)
    assert size(M=1024, V=128256) == size(M=100000, V=128256)    # sets of 1024 rows share it
    assert size(V=128256, top_k_all=2000) < 1024                 # done by rows alone


@pytest.mark.parametrize("name", ["s3d8_head_rope", "s3d8_cross_attention", "s3d8_sample"])
def test_null_arguments(name):
    assert rc(name, None) == _lib.S3D8_ERR_INVALID_ARG


def test_binding_refuses_host_tensors():
    import torch

    q, x = torch.zeros(1, 2, 64), torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        s3d8.head_rope(q, q_weight=torch.ones(64))
    with pytest.raises(TypeError):
        s3d8.cross_attention(x, x, x)
    with pytest.raises(TypeError):
        s3d8.sample(torch.zeros(1, 10), torch.zeros(1))
    with pytest.raises(ValueError):
        s3d8.cross_attention(x, x, x, out="f32")
