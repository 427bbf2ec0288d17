"""head_rope, cross_attention and sample on the GPU against plain forms in 64
bits (head_reference): types, layouts, odd sizes, strides, lengths of zero and
one, masks that leave nothing, values that are not finite in places that do not
count, streams, graphs, and a run of them with the linear layers around them."""
import numpy as np
import pytest

import head_reference as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
s3d8 = pytest.importorskip("w2_a8_matmul_amd")

BF16, F32 = torch.bfloat16, torch.float32


def gen(*seed):
    return np.random.Generator(np.random.PCG64(np.random.SeedSequence(list(seed))))


def dev(a, gpu, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(gpu)
    return t if dtype is None else t.to(dtype)


def host(t):
    return t.detach().double().cpu().numpy()


def close(got, want, bound):
    got = host(got)
    off = np.abs(got - want)
    assert (off <= bound).all(), f"off by {off[~(off <= bound)].max()} where {bound[~(off <= bound)].min()} is allowed"


# ------------------------------------------------------------------ head_rope
ROPE_CASES = [
    # M, heads, kv_heads, D, rot, layout, norm, in, out
    (1, 32, 8, 128, 128, "half", False, F32, "bf16"),
    (1, 1, 1, 2, 2, "half", True, F32, "f32"),
    (5, 3, 1, 80, 20, "half", True, BF16, "f32"),        # half of 10: no fours
    (5, 3, 1, 80, 20, "interleaved", False, BF16, "f32"),
    (7, 4, 2, 64, 64, "interleaved", True, F32, "bf16"),
    (33, 5, 5, 96, 24, "half", True, F32, "f32"),
    (33, 5, 5, 96, 48, "interleaved", False, BF16, "bf16"),
    (3, 2, 2, 256, 256, "half", True, BF16, "f32"),
    (3, 2, 2, 250, 130, "half", True, F32, "f32"),       # two pairs a lane
    (3, 2, 2, 254, 250, "interleaved", True, F32, "f32"),
    (1025, 20, 4, 128, 64, "half", True, BF16, "bf16"),  # four tokens a workgroup, one left over
    (1027, 16, 16, 64, 64, "interleaved", True, F32, "f32"),
    (2050, 32, 8, 80, 80, "half", False, F32, "f32"),
]


@pytest.mark.parametrize("M,H,Hk,D,rot,layout,norm,dtype,out", ROPE_CASES)
def test_head_rope(gpu, M, H, Hk, D, rot, layout, norm, dtype, out):
    g = gen(7000, M, H, D, rot)
    q, k = (dev(g.standard_normal((M, n, D)).astype(np.float32), gpu, dtype) for n in (H, Hk))
    w = [dev((1 + 0.1 * g.standard_normal(D)).astype(np.float32), gpu) if norm else None for _ in range(2)]
    positions = g.integers(0, 130000, M)
    rope = s3d8.Rope(rot, 500000.0, layout=layout, scaling="llama3", factor=8.0, device=gpu)
    f, factor = ref.frequencies(rot, 500000.0, "llama3", 8.0)
    for pos in (positions, positions.astype(np.int32)):
        both = s3d8.head_rope(q, k, dev(pos, gpu), rope, q_weight=w[0], k_weight=w[1], out=out)
        for x, y, weight in zip((q, k), both, w):
            assert y.shape == x.shape and y.dtype is (BF16 if out == "bf16" else F32)
            want, bound = ref.head_rope(host(x), pos, f, factor, layout == "interleaved",
                                        None if weight is None else host(weight), 1e-5)
            if out == "bf16":
                bound = bound + ref.HALF_BF16 * (np.abs(want) + bound)
            close(y, want, bound)


def test_head_rope_yarn_factor_and_far_positions(gpu):
    g = gen(7100)
    M, D = 9, 64
    q = dev(g.standard_normal((M, 2, D)).astype(np.float32), gpu)
    pos = np.array([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 40, 123456789, 2, -77777])
    rope = s3d8.Rope(D, 10000.0, scaling="yarn", factor=4.0, original_length=4096, device=gpu)
    f, factor = ref.frequencies(D, 10000.0, "yarn", 4.0, 4096, 1.0, 32.0)
    assert rope.factor == pytest.approx(factor, rel=1e-15)
    y = s3d8.head_rope(q, positions=dev(pos, gpu), rope=rope, out="f32")
    # the frequency's own rounding, 2^-52 of the angle, is in the bound: the library's are compared too
    want, bound = ref.head_rope(host(q), pos, host(rope.frequencies), factor, False, None, 1e-5)
    close(y, want, bound + ref.HALF_F32 * np.abs(want))
    np.testing.assert_allclose(host(rope.frequencies), f, rtol=1e-14)


def test_head_rope_norm_alone_and_zero_heads(gpu):
    g = gen(7200)
    q = g.standard_normal((4, 3, 80)).astype(np.float32)
    q[1] = 0
    w = (1 + 0.1 * g.standard_normal(80)).astype(np.float32)
    y = s3d8.head_rope(dev(q, gpu), q_weight=dev(w, gpu), out="f32", eps=1e-6)
    want, bound = ref.head_rope(q, np.zeros(4), np.zeros(0), 1.0, False, w, 1e-6)
    close(y, want, bound)
    assert (y[1] == 0).all()


@pytest.mark.parametrize("D,rot,layout", [(64, 64, "half"), (64, 32, "interleaved"), (20, 10, "half")])
def test_head_rope_strides_in_place_and_cache_rows(gpu, D, rot, layout):
    """Heads as parts of one matrix, results into rows of a larger cache or over the input: the bits of the plain
    call, and nothing beside them is written."""
    g = gen(7300, D)
    M, H, Hk = 6, 3, 2
    qkv = dev(g.standard_normal((M, (H + 2 * Hk) * D)).astype(np.float32), gpu, BF16)
    q, k = qkv[:, :H * D].view(M, H, D), qkv[:, H * D:(H + Hk) * D].view(M, Hk, D)
    rope = s3d8.Rope(rot, layout=layout, device=gpu)
    pos = torch.arange(3, 3 + M, device=gpu)
    w = dev((1 + 0.1 * g.standard_normal(D)).astype(np.float32), gpu)
    kw = dict(q_weight=w, k_weight=w)
    a, b = s3d8.head_rope(q.contiguous(), k.contiguous(), pos, rope, **kw)
    a2, b2 = s3d8.head_rope(q, k, pos, rope, **kw)
    assert torch.equal(a, a2) and torch.equal(b, b2)
    cache = torch.full((Hk, 20, D), 7.0, dtype=BF16, device=gpu)  # heads outermost
    s3d8.head_rope(q, k, pos, rope, **kw, k_out=cache[:, 5:5 + M].transpose(0, 1))
    assert torch.equal(cache[:, 5:5 + M].transpose(0, 1), b)
    assert (cache[:, :5] == 7).all() and (cache[:, 5 + M:] == 7).all()
    before = qkv[:, (H + Hk) * D:].clone()
    s3d8.head_rope(q, k, pos, rope, **kw, q_out=q, k_out=k)
    assert torch.equal(q, a) and torch.equal(k, b) and torch.equal(qkv[:, (H + Hk) * D:], before)
    odd = torch.empty(M * H * D + 1, dtype=BF16, device=gpu)[1:].view(M, H, D)  # an element off every alignment
    odd.copy_(a)
    assert torch.equal(s3d8.head_rope(odd, positions=pos, rope=rope), s3d8.head_rope(a, positions=pos, rope=rope))


# ------------------------------------------------------------------ cross_attention
def states(g, gpu, B, Lq, Lk, H, Hk, D, Bk=None, sharp=1.0):
    q = dev((sharp * g.standard_normal((B, Lq, H, D))).astype(np.float32), gpu, BF16)
    k, v = (dev(g.standard_normal((B if Bk is None else Bk, Lk, Hk, D)).astype(np.float32), gpu, BF16) for _ in range(2))
    return q, k, v + 0.5


ATTENTION_CASES = [
    # B, Lq, Lk, H, Hk, D
    (1, 1, 1, 1, 1, 16),
    (1, 1, 1, 4, 1, 128),
    (2, 1, 63, 4, 2, 64),
    (2, 1, 64, 8, 2, 80),
    (2, 1, 65, 8, 8, 96),
    (1, 1, 1601, 32, 8, 128),      # split over workgroups
    (3, 1, 700, 15, 3, 112),
    (1, 7, 130, 6, 2, 48),
    (2, 33, 257, 4, 4, 32),
    (1, 31, 1, 3, 1, 80),
    (1, 96, 300, 1, 1, 128),       # the most rows of one wave's tiles
    (1, 97, 300, 1, 1, 128),       # four waves
    (2, 129, 513, 4, 1, 64),
    (1, 200, 1000, 10, 2, 80),
    (1, 300, 190, 16, 16, 96),
    (2, 260, 320, 8, 2, 128),
]


@pytest.mark.parametrize("B,Lq,Lk,H,Hk,D", ATTENTION_CASES)
@pytest.mark.parametrize("kind", ["all", "lens", "mask", "both"])
def test_cross_attention(gpu, B, Lq, Lk, H, Hk, D, kind):
    g = gen(7400, B, Lq, Lk, H, D)
    q, k, v = states(g, gpu, B, Lq, Lk, H, Hk, D, sharp=2.0)
    lens = mask = None
    if kind in ("lens", "both"):
        lens = g.integers(0, Lk + 1, B).astype(np.int32)
        lens[0] = min(Lk, 1)
    if kind in ("mask", "both"):
        mask = g.random((B, Lq, Lk)) < 0.6
        mask[:, 0] = False                       # sees nothing
        mask[:, Lq // 2:, : Lk // 2] = False     # blocks that are hidden throughout
        mask[:, -1, :] = True
    o = s3d8.cross_attention(q, k, v, kv_lens=None if lens is None else dev(lens, gpu),
                             mask=None if mask is None else dev(mask, gpu))
    assert o.shape == q.shape and o.dtype is BF16 and o.is_contiguous()
    want, bound = ref.attention(host(q), host(k), host(v), D ** -0.5, lens, mask)
    close(o, want, bound)
    if mask is not None and Lq > 1:
        assert (o[:, 0] == 0).all()


def test_cross_attention_lengths_of_zero_and_outside(gpu):
    g = gen(7500)
    q, k, v = states(g, gpu, 4, 3, 70, 4, 2, 64)
    o = s3d8.cross_attention(q, k, v, kv_lens=torch.tensor([0, -5, 70, 1000], dtype=torch.int32, device=gpu))
    assert (o[:2] == 0).all()
    assert torch.equal(o[2:], s3d8.cross_attention(q[2:], k[2:], v[2:]))


@pytest.mark.parametrize("Lq", [1, 5, 140])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_cross_attention_ignores_what_is_hidden(gpu, Lq, bad):
    """Infinities and NaN past a sequence's length, and in keys and values that the mask hides, change nothing; what a
    row sees of them counts."""
    g = gen(7600, Lq)
    B, Lk, H, Hk, D = 2, 300, 4, 2, 80
    q, k, v = states(g, gpu, B, Lq, Lk, H, Hk, D)
    lens = np.array([300, 210], np.int32)
    mask = g.random((B, Lq, Lk)) < 0.7
    mask[:, :, 17] = mask[:, :, 130:133] = False
    mask[:, 0, 40] = False
    mask[:, 1:, 40] = True
    want, bound = ref.attention(host(q), host(k), host(v), D ** -0.5, lens, mask)
    kb, vb = k.clone(), v.clone()
    kb[1, 210:], vb[1, 210:] = bad, bad
    for t in (kb, vb):
        t[:, 17] = t[:, 130:133] = bad
    vb[0, 40, 0] = bad  # seen by rows 1.., not by row 0
    o = s3d8.cross_attention(q, kb, vb, kv_lens=dev(lens, gpu), mask=dev(mask, gpu))
    seen = np.zeros(o.shape, bool)
    seen[0, 1:, :H // Hk] = True
    fine = host(o)[~seen]
    off = np.abs(fine - want[~seen])
    assert (off <= bound[~seen]).all()
    if Lq > 1:
        assert not torch.isfinite(o[0, 1:, :H // Hk]).any()


@pytest.mark.parametrize("Lq", [1, 3, 20])
def test_cross_attention_shared_states(gpu, Lq):
    g = gen(7700, Lq)
    B, Lk, H, Hk, D = 5, 333, 8, 2, 128
    q, k, v = states(g, gpu, B, Lq, Lk, H, Hk, D, Bk=1)
    mask = g.random((B, Lq, Lk)) < 0.5
    lens = np.array([301], np.int32)
    o = s3d8.cross_attention(q, k, v, kv_lens=dev(lens, gpu), mask=dev(mask, gpu))
    want, bound = ref.attention(host(q), host(k), host(v), D ** -0.5, lens, mask)
    close(o, want, bound)


@pytest.mark.parametrize("shape", [(1, 1), (1, 9), (3, 1), (3, 9)])
def test_cross_attention_mask_of_one_row_for_all(gpu, shape):
    g = gen(7800, *shape)
    q, k, v = states(g, gpu, 3, 9, 150, 4, 2, 64)
    mask = dev(g.random((*shape, 150)) < 0.5, gpu)
    full = s3d8.cross_attention(q, k, v, mask=mask.expand(3, 9, 150).contiguous())
    assert torch.equal(s3d8.cross_attention(q, k, v, mask=mask), full)
    assert torch.equal(s3d8.cross_attention(q, k, v, mask=mask.expand(3, 9, 150)), full)
    wide = torch.zeros(3, 9, 163, dtype=torch.bool, device=gpu)
    wide[..., 13:] = mask
    assert torch.equal(s3d8.cross_attention(q, k, v, mask=wide[..., 13:]), full)


@pytest.mark.parametrize("Lk", [1, 1025, 1153])
def test_cross_attention_mask_rows_at_every_alignment(gpu, Lk):
    g = gen(7850, Lk)
    B, Lq = 2, 5
    q, k, v = states(g, gpu, B, Lq, Lk, 2, 2, 32)
    mask = dev(g.random((B, Lq, Lk)) < 0.6, gpu)
    want = None
    for at in range(4):
        for width in (Lk + at, (Lk + 11) // 4 * 4):
            wide = torch.ones(B, Lq, width, dtype=torch.bool, device=gpu)
            wide[..., at:at + Lk] = mask
            o = s3d8.cross_attention(q, k, v, mask=wide[..., at:at + Lk])
            want = o if want is None else want
            assert torch.equal(o, want)
    o, bound = ref.attention(host(q), host(k), host(v), 32 ** -0.5, mask=host(mask) > 0)
    close(want, o, bound)


def test_cross_attention_strides(gpu):
    """Queries as part of a matrix, states with heads outermost or beside each other: the bits of the plain call."""
    g = gen(7900)
    B, Lq, Lk, H, Hk, D = 2, 11, 203, 6, 2, 80
    q, k, v = states(g, gpu, B, Lq, Lk, H, Hk, D)
    want = s3d8.cross_attention(q, k, v)
    wide = torch.empty(B, Lq, 2 * H * D, dtype=BF16, device=gpu)
    qs = wide[..., H * D:].view(B, Lq, H, D)
    qs.copy_(q)
    ks = k.transpose(1, 2).contiguous().transpose(1, 2)
    kv = torch.cat((k, v), 2)
    assert torch.equal(s3d8.cross_attention(qs, ks, v.transpose(1, 2).contiguous().transpose(1, 2)), want)
    assert torch.equal(s3d8.cross_attention(q, kv[:, :, :Hk], kv[:, :, Hk:]), want)
    o = torch.full((B + 1, Lq, H, D), 3.0, dtype=BF16, device=gpu)
    assert s3d8.cross_attention(q, k, v, o=o[:B]).data_ptr() == o.data_ptr()
    assert torch.equal(o[:B], want) and (o[B] == 3).all()


def test_cross_attention_scores_far_apart(gpu):
    """Scores of some thousands, with the largest in the first, a middle and the last block, and rows of equal scores."""
    g = gen(8000)
    q, k, v = states(g, gpu, 1, 40, 400, 2, 1, 64)
    q, k = q * 30, k * 8
    k[0, 5] *= 3
    k[0, 390] *= -4
    q[0, 7] = 0
    o = s3d8.cross_attention(q, k, v)
    want, bound = ref.attention(host(q), host(k), host(v), 0.125)
    close(o, want, bound)


def test_cross_attention_offsets_past_32_bits(gpu):
    """A row of states every 8 million entries: the last lie 6 GB from the first."""
    row, Lk, D = (1 << 23) - 8, 400, 16
    big = torch.zeros((Lk - 1) * row + 2 * D, dtype=BF16, device=gpu)
    g = gen(8100)
    q, k, v = states(g, gpu, 1, 2, Lk, 1, 1, D)
    ks, vs = (torch.as_strided(big, (1, Lk, 1, D), (0, row, 0, 1), at) for at in (0, D))
    ks.copy_(k)
    vs.copy_(v)
    assert torch.equal(s3d8.cross_attention(q, ks, vs), s3d8.cross_attention(q, k, v))


@pytest.mark.parametrize("B,Lq,H,D", [(1, 1, 32, 128), (3, 50, 5, 80)])
def test_cross_attention_codes(gpu, B, Lq, H, D):
    g = gen(8200, B)
    q, k, v = states(g, gpu, B, Lq, 77, H, 1, D)
    o = torch.empty_like(q)
    xq, xs = s3d8.cross_attention(q, k, v, out="codes", o=o)
    want = s3d8.quant_act(o.float().view(B * Lq, H * D))
    assert torch.equal(o, s3d8.cross_attention(q, k, v))
    assert torch.equal(xq, want[0]) and torch.equal(xs, want[1])


# ------------------------------------------------------------------ sample
def check_sample(gpu, logits, u, T, k, p, mp, dtype=F32):
    l = dev(logits, gpu, dtype)
    token, prob = s3d8.sample(l, dev(u, gpu), temperature=T if np.isscalar(T) else dev(T, gpu),
                              top_k=k if np.isscalar(k) else dev(k, gpu), top_p=p if np.isscalar(p) else dev(p, gpu),
                              min_p=mp if np.isscalar(mp) else dev(mp, gpu))
    rows = l.float().cpu().numpy()
    for m in range(len(rows)):
        at = [x if np.isscalar(x) else x[m] for x in (T, k, p, mp)]
        want, share = ref.sample(rows[m], u[m], *at)
        assert int(token[m]) == want, (m, at)
        # the quotient's rounding, and weights that a last bit of the exponential may move by one
        assert abs(float(prob[m]) - share) <= 2.0 ** -24 * share * 1.01 + 2.0 ** -43


@pytest.mark.parametrize("V", [1, 2, 7, 64, 128, 129, 300, 512, 513, 1000, 1024, 1025, 3584, 3585, 5003, 40001])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_sample(gpu, V, dtype):
    g = gen(8300, V)
    M = 12
    logits = (3 * g.standard_normal((M, V))).astype(np.float32)
    u = g.random(M, dtype=np.float32)
    u[0], u[1] = 0, np.float32(1 - 2.0 ** -24)
    T = (0.3 + g.random(M)).astype(np.float32)
    T[2] = 0
    k = g.integers(0, 60, M).astype(np.int32)
    p = g.random(M, dtype=np.float32)
    p[3:5] = 1
    mp = (0.2 * g.random(M)).astype(np.float32)
    mp[::3] = 0
    check_sample(gpu, logits, u, T, k, p, mp, dtype)
    check_sample(gpu, logits, u, T, 0, p, 0.0, dtype)
    check_sample(gpu, logits, u, 1.0, 0, 1.0, 0.0, dtype)
    check_sample(gpu, logits, u, 0.7, 5000, 0.9, 0.01, dtype)   # more than are listed in LDS
    check_sample(gpu, logits, u, 5.0, 0, 0.999, 0.0, dtype)
    check_sample(gpu, logits, u, 0.0, 0, 0.5, 0.0, dtype)


def test_sample_equal_logits(gpu):
    """Ties go to the lowest index, at every limit."""
    V = 9000
    g = gen(8400)
    logits = np.zeros((10, V), np.float32)
    logits[4:] = np.float32(1.5) * g.integers(0, 3, (6, V))
    logits[5] = np.where(g.random(V) < 0.5, np.float32(0), np.float32(-0.0))
    u = g.random(10, dtype=np.float32)
    for k, p, mp in [(0, 1.0, 0.0), (1, 1.0, 0.0), (100, 1.0, 0.0), (0, 0.25, 0.0), (5000, 0.5, 0.0), (3000, 0.3, 1.0),
                     (0, 0.0, 0.0), (8999, 1.0, 0.0), (9000, 1.0, 0.0), (10 ** 9, 1.0, 0.0)]:
        check_sample(gpu, logits, u, 1.0, k, p, mp)


def test_sample_values_that_are_not_finite(gpu):
    inf, nan = np.inf, np.nan
    rows = np.array([
        [-inf] * 8,
        [nan] * 8,
        [-inf, nan, -inf, 2.0, nan, -inf, -inf, 1.0],
        [1, inf, 0, inf, -inf, nan, 3e38, 2],
        [-3.4e38, 3.4e38, 0, 0, 0, 0, 0, 0],
        [-3.4e38, -3.4e38, -inf, nan, -3.4e38, -inf, -inf, -inf],
        [1e-45, 0, -1e-45, -0.0, 0, 0, 0, 0],
    ], np.float32)
    for u0 in (0.0, 0.4, 0.999):
        u = np.full(len(rows), u0, np.float32)
        for args in [(1.0, 0, 1.0, 0.0), (1.0, 2, 1.0, 0.0), (1.0, 0, 0.6, 0.0), (0.0, 0, 1.0, 0.0), (1e-30, 0, 0.9, 0.1),
                     (1e30, 3, 0.9, 0.0)]:
            check_sample(gpu, rows, u, *args)


def test_sample_limits_outside_their_range(gpu):
    """Values of rows outside their ranges count as the ends; u of 1 or more takes the last token."""
    g = gen(8500)
    logits = g.standard_normal((6, 50)).astype(np.float32)
    u = np.array([0.3, 1.0, 2.0, -1.0, np.nan, 0.5], np.float32)
    T = np.array([-1.0, 1.0, 1.0, np.nan, 1.0, 1.0], np.float32)
    p = np.array([1.0, 1.5, 0.9, 0.9, -0.5, 0.7], np.float32)
    mp = np.array([0, -1, 0, 0, 0, 3.0], np.float32)
    k = np.array([-3, 0, 10, 0, 0, 2 ** 31 - 1], np.int32)
    token, prob = s3d8.sample(dev(logits, gpu), dev(u, gpu), temperature=dev(T, gpu), top_k=dev(k, gpu), top_p=dev(p, gpu),
                              min_p=dev(mp, gpu))
    fine_u, fine_T = np.where(np.isnan(u), 0, u), np.where(np.isnan(T), 0, T)
    for m in range(6):
        want, share = ref.sample(logits[m], fine_u[m], fine_T[m], k[m], p[m], mp[m])
        assert int(token[m]) == want
        assert abs(float(prob[m]) - share) <= 2.0 ** -24 * share * 1.01 + 2.0 ** -43


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_sample_rows_at_every_alignment(gpu, dtype):
    g = gen(8600)
    M, V = 17, 1003  # rows begin at every multiple of an element within 16 bytes
    wide = dev((3 * g.standard_normal((M, V + 4))).astype(np.float32), gpu, dtype)
    u = dev(g.random(M, dtype=np.float32), gpu)
    want = s3d8.sample(wide[:, 3:3 + V].contiguous(), u, top_k=40, top_p=0.9)
    got = s3d8.sample(wide[:, 3:3 + V], u, top_k=40, top_p=0.9)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for m in range(0, M, 5):
        t, p = ref.sample(wide[m, 3:3 + V].float().cpu().numpy(), float(u[m]), 1.0, 40, 0.9, 0.0)
        assert int(got[0][m]) == t


def test_sample_large_vocabulary(gpu):
    g = gen(8700)
    logits = (2 * g.standard_normal((3, 262144))).astype(np.float32)
    logits[2] = 0  # the largest sum
    u = g.random(3, dtype=np.float32)
    check_sample(gpu, logits, u, 1.0, 0, 1.0, 0.0)
    check_sample(gpu, logits, u, 1.0, 0, 0.9, 0.0)
    check_sample(gpu, logits, u, 1.0, 200000, 0.9, 0.0)


@pytest.mark.parametrize("M,V,dtype", [(3, 128256, F32), (3, 128256, BF16), (40, 20011, F32), (300, 9001, F32)])
@pytest.mark.parametrize("order", ["none", "rising", "falling", "ends"])
def test_sample_orders_of_logits(gpu, M, V, dtype, order):
    """Rows cut into parts or whole, with the largest logits spread, at one end, or one in each segment's last places;
    limits from one token to more than are listed; a sample of the rows against the plain form, and every row's
    token with a list of limits against the same limits one by one."""
    g = gen(8750, M, V)
    logits = (2 * g.standard_normal((M, V))).astype(np.float32)
    if order in ("rising", "falling"):
        logits.sort(1)
        logits = np.ascontiguousarray(logits[:, ::-1]) if order == "falling" else logits
    elif order == "ends":
        logits[:, 2047::2048] += 12
    u = g.random(M, dtype=np.float32)
    l, du = dev(logits, gpu, dtype), dev(u, gpu)
    ks = np.array([1, 7, 50, 200, 1000, 1024, 1025, 4000, 0], np.int32)[np.arange(M) % 9]
    listed, prob = s3d8.sample(l, du, top_k=dev(ks, gpu), top_p=0.9, min_p=0.001, temperature=0.8)
    rows = l.float().cpu().numpy()
    for k in np.unique(ks):
        at = np.flatnonzero(ks == k)
        token, share = s3d8.sample(l, du, top_k=int(k), top_p=0.9, min_p=0.001, temperature=0.8)
        assert torch.equal(token[at], listed[at]) and torch.equal(share[at], prob[at])
        assert int(token[at[0]]) == ref.sample(rows[at[0]], u[at[0]], 0.8, int(k), 0.9, 0.001)[0]


def test_sample_many_equal_logits(gpu):
    """More equal logits than a list holds, in a part and in the step where top-p ends."""
    g = gen(8760)
    V = 60000
    logits = np.zeros((4, V), np.float32)
    logits[1, ::7] = 3
    logits[2, 30000:] = -np.inf
    logits[3] = np.where(g.random(V) < 0.5, np.float32(1), np.float32(0.999))
    u = g.random(4, dtype=np.float32)
    for k, p, mp in [(50, 1.0, 0.0), (0, 0.9, 0.0), (1000, 0.5, 0.0), (0, 0.3, 0.9995), (0, 1.0, 1.0)]:
        check_sample(gpu, logits, u, 1.0, k, p, mp)


def test_sample_more_rows_than_a_set(gpu):
    g = gen(8770)
    M, V = 2500, 130
    logits = (3 * g.standard_normal((M, V))).astype(np.float32)
    u, T = g.random(M, dtype=np.float32), (0.5 + g.random(M)).astype(np.float32)
    k, p = g.integers(0, 20, M).astype(np.int32), (0.5 + 0.6 * g.random(M)).astype(np.float32)
    check_sample(gpu, logits, u, T, k, p, 0.0)
    check_sample(gpu, logits, u, T, 0, p, 0.0, BF16)


def test_sample_follows_the_distribution(gpu):
    """Over evenly spaced random numbers, tokens come up as often as their probability says, to one number each."""
    p = np.array([0.4, 0.3, 0.2, 0.1])
    n = 1000
    logits = np.tile(np.log(p), (n, 1)).astype(np.float32)
    token, _ = s3d8.sample(dev(logits, gpu), dev(((np.arange(n) + 0.5) / n).astype(np.float32), gpu))
    counts = np.bincount(token.cpu().numpy(), minlength=4)
    assert np.abs(counts - n * p).max() <= 1


# ------------------------------------------------------------------ together
def test_heads_run_together_on_a_stream_and_in_a_graph(gpu):
    """A decoder layer's way from the hidden rows to the next token: linear layer, heads, attention to the encoder's
    states, output projection, norm, vocabulary, token; each step against its own plain form, the whole run
    on another stream and as a replayed graph with the same bits."""
    g = gen(8800)
    M, K, H, Hk, D, Lk, V = 3, 256, 8, 2, 64, 200, 1000

    def linear(N, width, n):
        return s3d8.W4Linear.from_weights((0.1 * gen(8801, n).standard_normal((N, width))).astype(np.float32), 64, device=gpu)

    wq, wk, wv, wo, wvoc = (linear(N, width, n) for n, (N, width) in
                            enumerate([(H * D, K), (Hk * D, K), (Hk * D, K), (K, H * D), (V, K)]))
    x = dev(g.standard_normal((M, K)).astype(np.float32), gpu)
    enc = dev(g.standard_normal((M * Lk, K)).astype(np.float32), gpu)
    qn, kn = (dev((1 + 0.1 * g.standard_normal(D)).astype(np.float32), gpu) for _ in range(2))
    norm = dev((1 + 0.1 * g.standard_normal(K)).astype(np.float32), gpu)
    rope = s3d8.Rope(D, 500000.0, scaling="llama3", factor=8.0, device=gpu)
    pos, kpos = torch.tensor([70000, 3, 12], device=gpu), torch.arange(M * Lk, device=gpu) % Lk
    lens = torch.tensor([200, 64, 1], dtype=torch.int32, device=gpu)
    u = dev(g.random(M, dtype=np.float32), gpu)

    def step():
        k = s3d8.head_rope(wk(enc).view(M * Lk, Hk, D), positions=kpos, rope=rope, q_weight=kn)
        v = wv(enc, out="bf16")
        q0 = wq(x)
        q = s3d8.head_rope(q0.view(M, H, D), positions=pos, rope=rope, q_weight=qn)
        o = torch.empty(M, 1, H, D, dtype=BF16, device=gpu)
        codes = s3d8.cross_attention(q.view(M, 1, H, D), k.view(M, Lk, Hk, D), v.view(M, Lk, Hk, D), kv_lens=lens,
                                     out="codes", o=o)
        h, xq, xs = s3d8.block_norm(x, norm, branch=wo.linear(*codes))
        logits = wvoc.linear(xq, xs)
        token, prob = s3d8.sample(logits, u, temperature=0.8, top_k=50, top_p=0.9)
        return dict(q0=q0, q=q, k=k, v=v, o=o, h=h, logits=logits, token=token, prob=prob)

    r = step()
    f, factor = ref.frequencies(D, 500000.0, "llama3", 8.0)
    want, bound = ref.head_rope(host(r["q0"]).reshape(M, H, D), host(pos), f, factor, False, host(qn), 1e-5)
    close(r["q"], want, bound + ref.HALF_BF16 * (np.abs(want) + bound))
    want, bound = ref.attention(host(r["q"]).reshape(M, 1, H, D), host(r["k"]).reshape(M, Lk, Hk, D),
                                host(r["v"]).reshape(M, Lk, Hk, D), D ** -0.5, host(lens))
    close(r["o"], want, bound)
    for m in range(M):
        token, prob = ref.sample(r["logits"][m].cpu().numpy(), float(u[m]), 0.8, 50, 0.9, 0.0)
        assert int(r["token"][m]) == token and float(r["prob"][m]) == pytest.approx(prob, rel=1e-6)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(again[n], r[n]) for n in r)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    saved = x.clone()
    for n in range(3):
        x.copy_(saved * (1 + n))
        eager = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(held[name], eager[name]) for name in r)
    x.copy_(saved)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(held[name], r[name]) for name in r)


def test_heads_calls_at_once_and_two_graphs(gpu):
    """Calls whose keys are split and rows cut, so that they have workspaces: on two streams at once and as two graphs
    replayed at once, the bits of each by itself."""
    g = gen(8900)
    B, Lk, V = 3, 1000, 20011
    sets = []
    for _ in range(2):
        q, k, v = states(g, gpu, B, 1, Lk, 8, 2, 64)
        mask = dev(g.random((B, 1, Lk)) < 0.5, gpu)
        logits, u = dev(g.standard_normal((B, V)).astype(np.float32) * 3, gpu), dev(g.random(B, dtype=np.float32), gpu)
        sets.append((q, k, v, mask, logits, u))

    def run(q, k, v, mask, logits, u):
        return (s3d8.cross_attention(q, k, v), s3d8.cross_attention(q, k, v, mask=mask), *s3d8.sample(logits, u, top_p=0.9),
                *s3d8.sample(logits, u, top_k=50, min_p=0.01))

    def same(a, b):
        assert all(torch.equal(x, y) for x, y in zip(a, b, strict=True))

    want = [run(*s) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for n, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                got[n].append(run(*sets[n]))
    torch.cuda.synchronize()
    for n in range(2):
        for r in got[n]:
            same(r, want[n])

    graphs, held = [torch.cuda.CUDAGraph() for _ in sets], []
    for graph, s in zip(graphs, sets):
        with torch.cuda.graph(graph):
            held.append(run(*s))
    for _ in range(3):
        for r in held:
            for t in r:
                t.zero_()
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for r, w in zip(held, want):
            same(r, w)
        same(run(*sets[0]), want[0])
