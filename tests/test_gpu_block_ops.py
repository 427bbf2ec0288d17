"""The block norm and the gated activation on the GPU, bit for bit against
their definitions in numpy, and a run of a whole MLP block."""
import numpy as np
import pytest

import block_reference as ref
import oracle
import workloads
from parity_inputs import random_format

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
s3d8 = pytest.importorskip("w2_a8_matmul_amd")

F = np.float32


def rng(*words):
    return np.random.Generator(np.random.PCG64(np.random.SeedSequence(list(words))))


def rows(g, M, K, bf16, scale=1.0):
    x = (g.standard_normal((M, K)) * scale * np.where(g.random((M, K)) < 0.01, 20, 1)).astype(F)
    return ref.round_bf16(x) if bf16 else x


def dev(x, gpu, bf16=False):
    t = torch.from_numpy(np.ascontiguousarray(x)).to(gpu)
    return t.to(torch.bfloat16) if bf16 else t


def same(t, x):
    """Bit for bit (bf16 tensors as the fp32 values they hold); -0 and 0 differ."""
    got = t.float().cpu().numpy() if t.dtype == torch.bfloat16 else t.cpu().numpy()
    if got.dtype == F:
        assert np.array_equal(got.view(np.uint32), np.asarray(x, F).view(np.uint32)), np.abs(got - x).max()
    else:
        assert np.array_equal(got, x)


def check_rows(out, got, u):
    if out == "codes":
        codes, xs = ref.quantise(u)
        same(got[0], codes)
        same(got[1], xs)
    else:
        same(got, ref.round_bf16(u) if out == "bf16" else u)


def norm_case(gpu, M, K, kind="rms", h_bf=False, b_bf=False, branch=True, post=False, post_bias=False, bias=False,
              gate=None, rs=1.0, out="codes", eps=1e-5, in_place=False, seed=0):
    g = rng(7300, M, K, seed)
    h = rows(g, M, K, h_bf)
    w = (1 + 0.1 * g.standard_normal(K)).astype(F)
    vec = lambda: (0.1 * g.standard_normal(K)).astype(F)  # noqa: E731
    b = vec() if bias else None
    br = rows(g, M, K, b_bf, 0.5) if branch else None
    pw = vec() + F(1) if post else None
    pb = vec() if post_bias else None
    gt = None if gate is None else g.standard_normal(K if "channel" in gate else 1).astype(F)
    tanh = gate is not None and "tanh" in gate
    h_r, u_r = ref.block_norm(h, w, b, br, pw, pb, gt, tanh, rs, eps, kind, h_bf)
    to = lambda x: None if x is None else dev(x, gpu)  # noqa: E731
    dh = dev(h, gpu, h_bf)
    got = s3d8.block_norm(dh, to(w), to(b), branch=None if br is None else dev(br, gpu, b_bf), post_weight=to(pw),
                          post_bias=to(pb), gate=to(gt), tanh_gate=tanh, residual_scale=rs, eps=eps, kind=kind, out=out,
                          h_out=dh if in_place else None)
    if branch:
        assert (got[0] is dh) == in_place
        same(got[0], h_r)
        got = got[1:] if out == "codes" else got[1]
        if not in_place:
            same(dh, h)
    check_rows(out, got, u_r)


@pytest.mark.parametrize("out", ["codes", "f32", "bf16"])
@pytest.mark.parametrize("h_bf,b_bf", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norm_types(gpu, kind, h_bf, b_bf, out):
    for post in (False, True):
        norm_case(gpu, 5, 656, kind, h_bf, b_bf, post=post, post_bias=post and kind == "layer", bias=kind == "layer",
                  out=out, rs=0.5)


@pytest.mark.parametrize("gate", [None, "scalar", "tanh", "channel", "channel tanh"])
@pytest.mark.parametrize("kind,post", [("rms", False), ("rms", True), ("layer", False), ("layer", True)])
def test_norm_gates(gpu, kind, post, gate):
    norm_case(gpu, 3, 1280, kind, b_bf=True, post=post, post_bias=kind == "layer" and post, gate=gate, rs=1.25)
    norm_case(gpu, 2, 48, kind, h_bf=True, post=post, gate=gate, in_place=True, bias=kind == "layer")


# widths at and around every thread-count and register step
@pytest.mark.parametrize("K", [16, 32, 240, 1024, 1040, 2048, 2064, 4080, 4096, 4112, 8192, 8208, 14336, 16384, 16400,
                               32768, 65536])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norm_widths(gpu, kind, K):
    norm_case(gpu, 2, K, kind, post=True, gate="tanh", bias=kind == "layer")
    norm_case(gpu, 1, K, kind, h_bf=True, b_bf=True, out="f32")
    norm_case(gpu, 3, K, kind, branch=False)


@pytest.mark.parametrize("M", [1, 2, 7, 64, 511, 2048, 5000])
def test_norm_rows(gpu, M):
    norm_case(gpu, M, 512, h_bf=True, b_bf=True, post=True, seed=1)
    norm_case(gpu, M, 1280, "layer", gate="tanh", out="bf16", seed=2)


def test_norm_small_rows_see_eps(gpu):
    """Rows whose mean square is near eps, and another eps."""
    g = rng(7307)
    K = 1280
    h = (g.standard_normal((6, K)) * np.geomspace(1e-5, 1e-1, 6)[:, None]).astype(F)
    w = np.ones(K, F)
    for kind in ("rms", "layer"):
        for eps in (1e-5, 1e-6, 1e-12):
            _, u_r = ref.block_norm(h, w, eps=eps, kind=kind)
            check_rows("codes", s3d8.block_norm(dev(h, gpu), dev(w, gpu), eps=eps, kind=kind), u_r)


def test_norm_edge_rows(gpu):
    """Zero rows (codes and scale 0), a single value, a constant row under LAYER, tiny and large values."""
    K = 256
    h = np.zeros((7, K), F)
    h[1, 17] = -3.5
    h[2] = 4.25
    h[3] = 1e-30 * np.arange(1, K + 1, dtype=F)
    h[4] = 1e15
    h[4, 3] = -3e15
    h[5] = 1e-42
    h[6, ::2], h[6, 1::2] = 1.0, -1.0
    w = np.ones(K, F)
    w[5] = -2.0
    w[7] = 0.0
    for kind in ("rms", "layer"):
        for br in (None, np.zeros_like(h), h * F(0.5)):
            for out in ("codes", "f32"):
                h_r, u_r = ref.block_norm(h, w, None, br, kind=kind)
                got = s3d8.block_norm(dev(h, gpu), dev(w, gpu), branch=None if br is None else dev(br, gpu), kind=kind,
                                      out=out)
                if br is not None:
                    same(got[0], h_r)
                    got = got[1:] if out == "codes" else got[1]
                check_rows(out, got, u_r)


def test_norm_leaves_its_neighbours(gpu):
    M, K = 3, 272
    g = rng(7301)
    h, br, w = rows(g, M, K, True), rows(g, M, K, True), np.ones(K, F)
    pad = 1024
    hb = torch.full((M * K + 2 * pad,), 5.0, dtype=torch.bfloat16, device=gpu)
    qb = torch.full((M * K + 2 * pad,), 9, dtype=torch.int8, device=gpu)
    sb = torch.full((M + 16,), 3.0, device=gpu)
    s3d8.block_norm(dev(h, gpu, True), dev(w, gpu), branch=dev(br, gpu, True), h_out=hb[pad:pad + M * K].view(M, K),
                    xq=qb[pad:pad + M * K].view(M, K), xs=sb[8:8 + M])
    h_r, u_r = ref.block_norm(h, w, None, br, h_bf16=True)
    same(hb[pad:pad + M * K].view(M, K), h_r)
    check_rows("codes", (qb[pad:pad + M * K].view(M, K), sb[8:8 + M]), u_r)
    for t, v in ((hb, 5), (qb, 9)):
        assert (t[:pad] == v).all() and (t[pad + M * K:] == v).all()
    assert (sb[:8] == 3).all() and (sb[8 + M:] == 3).all()


# ------------------------------------------------------------------ gated activation
@pytest.mark.parametrize("out", ["codes", "f32", "bf16"])
@pytest.mark.parametrize("bf", [False, True])
@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("M,K", [(1, 16), (1, 4096), (1, 14336), (5, 1744), (33, 4112), (130, 8192), (700, 1040),
                                 (2, 16400), (2, 65536), (1, 32768)])
def test_glu(gpu, M, K, fused, bf, out):
    g = rng(7302, M, K)
    both = rows(g, M, 2 * K, bf, 2.0)
    gate, up = both[:, :K], both[:, K:]
    d = dev(both, gpu, bf)
    dg, du = (d[:, :K], d[:, K:]) if fused else (d[:, :K].contiguous(), d[:, K:].contiguous())
    check_rows(out, s3d8.glu_act(dg, du, out=out), ref.glu(gate, up))


def test_glu_values(gpu):
    """Every magnitude: far negative gates (the result underflows to -0), far positive ones, zeros, subnormals."""
    K = 4096
    mag = np.concatenate([np.geomspace(1e-44, 3e38, K // 2 - 2), [0.0, 1.0]]).astype(F)
    gate = np.stack([np.concatenate([mag, -mag]), np.linspace(-110, 110, K).astype(F),
                     np.linspace(-800, -80, K).astype(F), np.linspace(-1e-3, 1e-3, K).astype(F),
                     np.zeros(K, F), np.full(K, -2000, F)])
    up = np.stack([np.ones(K, F), np.full(K, -1.5, F), np.full(K, 1e30, F), np.linspace(-2, 2, K).astype(F),
                   np.ones(K, F), np.full(K, 3e38, F)])
    a = ref.glu(gate, up)
    assert np.isfinite(a).all()
    for out in ("f32", "codes"):
        check_rows(out, s3d8.glu_act(dev(gate, gpu), dev(up, gpu), out=out), a)


def test_glu_equal_values(gpu):
    """Rows of few distinct values: everything is the row's maximum, or on a border with it."""
    for K in (48, 1040, 4096, 14336):
        gate = np.stack([np.full(K, 1.25), np.where(np.arange(K) % 2, -2.0, 2.0), np.full(K, 30.0),
                         np.where(np.arange(K) == K - 1, 3.0, 1e-3)]).astype(F)
        up = np.stack([np.full(K, -0.75), np.full(K, 1.0), np.where(np.arange(K) % 3, 127.0, 63.5),
                       np.full(K, 1.0)]).astype(F)
        for bf in (False, True):
            g, u = (ref.round_bf16(gate), ref.round_bf16(up)) if bf else (gate, up)
            check_rows("codes", s3d8.glu_act(dev(g, gpu, bf), dev(u, gpu, bf)), ref.glu(g, u))


def test_glu_rounding_borders(gpu):
    """Rows whose quotients x / s lie on and one fp32 step around k + 1/2."""
    K = 2048
    g = rng(7303)
    gate = np.full((8, K), 60.0, F)  # SiLU(60) = 60 to the last bit
    up = np.zeros((8, K), F)
    for r in range(8):
        top = F(127) * F(2.0 ** (r - 4))
        v = ((g.integers(-126, 126, K) + 0.5) * 2.0 ** (r - 4)).astype(F)
        v = np.where(np.arange(K) % 3 == 0, np.nextafter(v, F(np.inf)), np.where(np.arange(K) % 3 == 1, v, np.nextafter(v, F(-np.inf))))
        up[r] = v / F(60)
        up[r, 0] = top / F(60)
    check_rows("codes", s3d8.glu_act(dev(gate, gpu), dev(up, gpu)), ref.glu(gate, up))


def test_refusals(gpu):
    h, w = torch.zeros((2, 64), device=gpu), torch.ones(64, device=gpu)
    with pytest.raises(TypeError):
        s3d8.block_norm(h.half(), w)
    with pytest.raises(TypeError):
        s3d8.block_norm(h, w.bfloat16())
    with pytest.raises(ValueError):
        s3d8.block_norm(h, w[:32])
    with pytest.raises(ValueError):
        s3d8.block_norm(h.t(), w[:2])
    with pytest.raises(ValueError):
        s3d8.block_norm(h, w, branch=h[:1])
    with pytest.raises(ValueError):
        s3d8.block_norm(h, w, branch=h, gate=torch.ones(3, device=gpu))
    with pytest.raises(ValueError):
        s3d8.block_norm(h, w, h_out=h)
    with pytest.raises(ValueError):
        s3d8.block_norm(h, w, kind="batch")
    with pytest.raises(ValueError):
        s3d8.block_norm(h, w, out="int8")
    with pytest.raises(ValueError):
        s3d8.block_norm(h, w, rows=torch.empty_like(h))
    with pytest.raises(ValueError):
        s3d8.block_norm(h, w, out="f32", xs=torch.empty(2, device=gpu))
    with pytest.raises(TypeError):
        s3d8.block_norm(h, w, out="bf16", rows=torch.empty_like(h))
    with pytest.raises(s3d8.S3D8Error):
        s3d8.block_norm(h, w, gate=torch.ones(1, device=gpu))  # no branch
    with pytest.raises(s3d8.S3D8Error):
        s3d8.block_norm(h, w, w)  # RMS takes no bias
    with pytest.raises(s3d8.S3D8Error):
        s3d8.block_norm(h[:, :40].contiguous(), w[:40].contiguous())
    with pytest.raises(ValueError):
        s3d8.glu_act(h, h[:1])
    with pytest.raises(ValueError):
        s3d8.glu_act(h.t(), h.t())
    with pytest.raises(TypeError):
        s3d8.glu_act(h.half(), h.half())
    with pytest.raises(ValueError):
        s3d8.glu_act(h, h.bfloat16())
    with pytest.raises(s3d8.S3D8Error):
        s3d8.glu_act(torch.zeros((2, 66), device=gpu)[:, 1:65], h)  # rows not aligned to 4 elements
    torch.cuda.synchronize()


# ------------------------------------------------------------------ together
class Block:
    """An MLP block: norm -> gate and up (one W4 matrix) -> gated activation -> down (S3D8) -> residual and next norm."""

    def __init__(self, gpu, M, K, I, seed):
        g = rng(7304, M, K, I, seed)
        self.M, self.K, self.I = M, K, I
        self.h, self.attn = rows(g, M, K, True), rows(g, M, K, False, 0.3)
        self.w1, self.w2 = ((1 + 0.1 * g.standard_normal(K)).astype(F) for _ in range(2))
        self.q = g.integers(0, 16, (2 * I, K), dtype=np.uint8)
        self.scales = ref.bf16_bits(g.lognormal(-5, 0.3, (2 * I, -(-K // 64))).astype(F))
        self.C, self.alpha, self.packed = random_format([7305, K, I], K, I)
        self.lin = s3d8.W4Linear(ref.pack(self.q), self.scales, 64, device=gpu)
        self.tiled = s3d8.tile(dev(self.packed, gpu), K)
        self.dC, self.dalpha = dev(self.C, gpu), dev(self.alpha.view(np.int16), gpu)
        self.dh, self.dattn, self.dw1, self.dw2 = dev(self.h, gpu, True), dev(self.attn, gpu), dev(self.w1, gpu), dev(self.w2, gpu)

    def run(self):
        h1, xq, xs = s3d8.block_norm(self.dh, self.dw1, branch=self.dattn)
        both = self.lin.linear(xq, xs)
        aq, as_ = s3d8.glu_act(both[:, :self.I], both[:, self.I:])
        down = s3d8.linear(aq, as_, self.tiled, self.dC, self.dalpha, self.K)
        h2, nq, ns = s3d8.block_norm(h1, self.dw2, branch=down, residual_scale=0.5)
        return h1, xq, xs, both, aq, as_, down, h2, nq, ns

    def check(self, out):
        """Every stage against its definition on the inputs that the stage had."""
        h1, xq, xs, both, aq, as_, down, h2, nq, ns = (t.float().cpu().numpy() if t.dtype == torch.bfloat16
                                                       else t.cpu().numpy() for t in out)
        h_r, u = ref.block_norm(self.h, self.w1, None, self.attn, h_bf16=True)
        codes, s = ref.quantise(u)
        assert np.array_equal(h1, h_r) and np.array_equal(xq, codes) and np.array_equal(xs, s)
        y, size = ref.w4_linear(xq, xs, self.q, self.scales, None, 64)
        assert (np.abs(both - y) <= ref.w4_tolerance(y, size, self.K, False)).all()
        codes, s = ref.quantise(ref.glu(both[:, :self.I], both[:, self.I:]))
        assert np.array_equal(aq, codes) and np.array_equal(as_, s)
        w = oracle.decode(self.packed, self.C, self.K, self.I)
        acc = aq.astype(np.int64) @ w.astype(np.int64).T
        y = (as_[:, None] * acc.astype(F)) * ref.bf16_value(self.alpha[:self.K])[None, :]
        assert np.array_equal(down, y)
        h_r, u = ref.block_norm(h1, self.w2, None, down, residual_scale=0.5, h_bf16=True)
        codes, s = ref.quantise(u)
        assert np.array_equal(h2, h_r) and np.array_equal(nq, codes) and np.array_equal(ns, s)


@pytest.mark.parametrize("M,K,I", [(1, 256, 768), (6, 1040, 656), (40, 512, 1296)])
def test_mlp_block(gpu, M, K, I):
    b = Block(gpu, M, K, I, 0)
    b.check(b.run())


@pytest.mark.parametrize("M", [1, 24])
def test_mlp_block_in_a_graph(gpu, M):
    """Captured once and replayed, with eager work and new inputs between the replays."""
    b, other = Block(gpu, M, 512, 768, 1), Block(gpu, M, 512, 768, 2)
    b.run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream(gpu)
    side.wait_stream(torch.cuda.current_stream(gpu))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = b.run()
    for seed in (3, 4, 5):
        g = rng(7306, seed)
        b.h, b.attn = rows(g, M, 512, True), rows(g, M, 512, False, 0.3)
        b.dh.copy_(dev(b.h, gpu, True))
        b.dattn.copy_(dev(b.attn, gpu))
        graph.replay()
        other.check(other.run())
        torch.cuda.synchronize()
        b.check(out)
        for e, r in zip(b.run(), out):
            assert torch.equal(e, r)


def test_side_streams_at_once(gpu):
    """The norm on one stream and the gated activation on another, both at once, several calls each."""
    g = rng(7307)
    M, K = 300, 2064
    h, br, w = rows(g, M, K, True), rows(g, M, K, True, 0.5), (1 + 0.1 * g.standard_normal(K)).astype(F)
    gate, up = rows(g, M, K, False, 2.0), rows(g, M, K, False)
    dh, dbr, dw, dg, du = dev(h, gpu, True), dev(br, gpu, True), dev(w, gpu), dev(gate, gpu), dev(up, gpu)
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(gpu), torch.cuda.Stream(gpu)
    with torch.cuda.stream(one):
        norms = [s3d8.block_norm(dh, dw, branch=dbr) for _ in range(4)]
    with torch.cuda.stream(two):
        glus = [s3d8.glu_act(dg, du) for _ in range(4)]
    torch.cuda.synchronize()
    h_r, u_r = ref.block_norm(h, w, None, br, h_bf16=True)
    a_r = ref.glu(gate, up)
    for n in norms:
        same(n[0], h_r)
        check_rows("codes", n[1:], u_r)
    for a in glus:
        check_rows("codes", a, a_r)


def test_most_rows(gpu):
    """2^19 rows of 16."""
    M, K = 1 << 19, 16
    norm_case(gpu, M, K, post=True)
    norm_case(gpu, M, K, "layer", h_bf=True, b_bf=True, out="bf16")
    g = rng(7308)
    gate, up = rows(g, M, K, True, 2.0), rows(g, M, K, True)
    check_rows("codes", s3d8.glu_act(dev(gate, gpu, True), dev(up, gpu, True)), ref.glu(gate, up))


def test_offsets_past_32_bits(gpu):
    """Row matrices of more than 2^31 elements (and 2^32 bytes): the rows at the ends."""
    K, few = 65536, 3
    g = rng(7309)
    h, br, w = rows(g, few, K, True), rows(g, few, K, True, 0.5), (1 + 0.1 * g.standard_normal(K)).astype(F)
    h_r, u_r = ref.block_norm(h, w, None, br, h_bf16=True)
    M = 33000  # 2.16e9 elements
    dh = torch.zeros((M, K), dtype=torch.bfloat16, device=gpu)
    dbr = torch.zeros_like(dh)
    for d, x in ((dh, h), (dbr, br)):
        d[:few] = dev(x, gpu, True)
        d[M - few:] = dev(x, gpu, True)
    h1, xq, xs = s3d8.block_norm(dh, dev(w, gpu), branch=dbr)
    for at in (slice(0, few), slice(M - few, M)):
        same(h1[at], h_r)
        check_rows("codes", (xq[at], xs[at]), u_r)
    assert not h1[few:M - few:97].any() and not xq[few:M - few:97].any() and not xs[few:M - few].any()
    del h1, xq, xs, dbr
    # the halves of one matrix, twice the row stride
    M = 17000
    both = torch.zeros((M, 2 * K), dtype=torch.bfloat16, device=gpu)
    for at in (slice(0, few), slice(M - few, M)):
        both[at, :K] = dev(h, gpu, True)
        both[at, K:] = dev(br, gpu, True)
    out = s3d8.glu_act(both[:, :K], both[:, K:], out="bf16")
    for at in (slice(0, few), slice(M - few, M)):
        check_rows("bf16", out[at], ref.glu(h, br))
    assert not out[few:M - few:97].any()


def test_gate_must_be_a_tensor(gpu):
    h = torch.zeros((2, 64), device=gpu)
    w = torch.ones(64, device=gpu)
    with pytest.raises(TypeError):
        s3d8.block_norm(h, w, branch=h.clone(), gate=0.5)


def test_norm_gate_of_nan(gpu):
    """tanh(NaN) is NaN: a scalar gate spoils every row, a channel's its channel of h'."""
    M, K = 3, 64
    g = rng(7310)
    h, br, w = rows(g, M, K, False), rows(g, M, K, False, 0.5), np.ones(K, F)
    args = dict(branch=dev(br, gpu), tanh_gate=True, out="f32")
    for kind in ("rms", "layer"):
        for bad in (np.nan, -np.nan):
            h1, u = s3d8.block_norm(dev(h, gpu), dev(w, gpu), gate=dev(np.full(1, bad, F), gpu), kind=kind, **args)
            assert h1.isnan().all() and u.isnan().all()
            gate = g.standard_normal(K).astype(F)
            gate[[0, 37]] = bad
            h1, u = s3d8.block_norm(dev(h, gpu), dev(w, gpu), gate=dev(gate, gpu), kind=kind, **args)
            at = np.isnan(gate)
            assert np.array_equal(h1.isnan().cpu().numpy(), np.broadcast_to(at, (M, K))) and u.isnan().all()
            h_r, _ = ref.block_norm(h, w, None, br, None, None, np.where(at, F(0), gate), True)
            same(h1[:, torch.from_numpy(~at).to(gpu)], h_r[:, ~at])


@pytest.mark.parametrize("K", [64, 1040, 4096, 14336])
def test_codes_of_rows_past_the_largest_fp32(gpu, K):
    """Finite operands whose product overflows: the codes and scale that quant_act makes of the infinite values."""
    g = rng(7311, K)
    up, gate = rows(g, 4, K, False), np.full((4, K), 50.0, F)
    gate[0, 3], up[0, 3] = 1e30, 1e30
    gate[1, [0, K - 1]], up[1, [0, K - 1]] = 3e38, (-3e38, 3e38)
    gate[2], up[2] = 1e25, 1e25
    a = s3d8.glu_act(dev(gate, gpu), dev(up, gpu), out="f32")
    same(a, np.where(np.isinf(a.cpu().numpy()), np.copysign(F(np.inf), up), ref.glu(gate, np.where(gate > 60, F(0), up))))
    assert a.isinf().sum(1).tolist() == [1, 2, K, 0]
    for got, want in zip(s3d8.glu_act(dev(gate, gpu), dev(up, gpu)), s3d8.quant_act(a)):
        same(got, want.cpu().numpy())
    h, w, b = rows(g, 3, K, False), np.full(K, 3e38, F), np.full(K, 3e38, F)
    for kind in ("rms", "layer"):
        bias = dev(b, gpu) if kind == "layer" else None
        u = s3d8.block_norm(dev(h, gpu), dev(w, gpu), bias, kind=kind, out="f32")
        assert u.isinf().any(1).all() and not u.isnan().any()
        for got, want in zip(s3d8.block_norm(dev(h, gpu), dev(w, gpu), bias, kind=kind), s3d8.quant_act(u)):
            same(got, want.cpu().numpy())


def test_norm_refuses_a_branch_of_another_shape(gpu):
    """As many elements in other rows."""
    h, w = torch.zeros((32, 64), device=gpu), torch.ones(64, device=gpu)
    for shape in ((64, 32), (16, 128), (1024, 2)):
        with pytest.raises(ValueError):
            s3d8.block_norm(h, w, branch=torch.ones(shape, device=gpu))
    for shape in ((32, 64), (2048,), (1, 2048), (4, 8, 64)):  # the rows in a row
        h1, xq, xs = s3d8.block_norm(h, w, branch=torch.ones(shape, device=gpu))
        assert (h1 == 1).all() and (xq == 127).all()


# Rows for every CU (512 on 256 CUs): the fewest threads that hold a row in 7 float4 each.  Every build of that rule:
# 64 threads with 1, 2, 4, 5, 7 float4, 256 with 2, 4, 5, 7, 512 with 4, 5, 7, 1024 with 4, 5, 7, 16.
MANY = 520
MANY_WIDTHS = [256, 272, 1024, 1040, 1792, 2048, 2064, 4096, 4112, 7168, 8192, 8208, 14336, 14352, 16400, 28672, 28688]
SOME = [0, 1, 2, 100, 255, 256, 257, 400, 511, 512, 518, 519]


@pytest.mark.parametrize("K", MANY_WIDTHS)
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norm_of_many_rows(gpu, kind, K):
    """Every row like another one that the definition is computed for."""
    g = rng(7312, K)
    n = len(SOME)
    h, br = rows(g, n, K, True), rows(g, n, K, True, 0.5)
    w, pw = ((1 + 0.1 * g.standard_normal(K)).astype(F) for _ in range(2))
    b = (0.1 * g.standard_normal(K)).astype(F) if kind == "layer" else None
    which = np.arange(MANY) % n
    which[SOME] = np.arange(n)
    for post, gate, bf in ((True, None, True), (False, F([0.3]), False)):
        h_r, u_r = ref.block_norm(h, w, b, br, pw if post else None, b if post else None, gate, gate is not None, 0.5,
                                  kind=kind, h_bf16=bf)
        for out in ("codes", "bf16", "f32"):
            to = lambda x: None if x is None else dev(x, gpu)  # noqa: E731
            got = s3d8.block_norm(dev(h[which], gpu, bf), to(w), to(b), branch=dev(br[which], gpu, True),
                                  post_weight=to(pw) if post else None, post_bias=to(b) if post else None, gate=to(gate),
                                  tanh_gate=gate is not None, residual_scale=0.5, kind=kind, out=out)
            same(got[0], h_r[which])
            check_rows(out, got[1:] if out == "codes" else got[1], u_r[which])


@pytest.mark.parametrize("K", MANY_WIDTHS)
@pytest.mark.parametrize("bf", [False, True])
def test_glu_of_many_rows(gpu, bf, K):
    g = rng(7313, K)
    n = len(SOME)
    both = rows(g, n, 2 * K, bf, 2.0)
    both[1, 5] = -80                            # a row for the 64-bit form
    both[2, :K], both[2, K:] = 1.25, -0.75      # every value the maximum
    both[3, :K:2], both[3, K:] = 60.0, 1.0 / 64  # most on a border or at the maximum
    a = ref.glu(both[:, :K], both[:, K:])
    which = np.arange(MANY) % n
    which[SOME] = np.arange(n)
    d = dev(both[which], gpu, bf)
    for out in ("codes", "bf16", "f32"):
        check_rows(out, s3d8.glu_act(d[:, :K], d[:, K:], out=out), a[which])
