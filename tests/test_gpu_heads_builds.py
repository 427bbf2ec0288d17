"""head_rope, cross_attention and sample at sizes that take each of their builds and launch plans: tiles of
128 rows, more blocks of keys than are listed, masks of a single row, several heads a group of lanes, sets
of rows that share a workspace, and logits that are not finite in vocabularies that are cut into parts."""
import numpy as np
import pytest

import head_reference as ref
from test_gpu_heads import check_sample, close, dev, gen, host, states

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
s3d8 = pytest.importorskip("w2_a8_matmul_amd")

BF16, F32 = torch.bfloat16, torch.float32


def wide_tiles(gpu, B, Lq, H, Hk, shared=False):
    """Whether a call takes tiles of 128 rows: where there is more than one of them for every CU."""
    pairs, rows = (1 if shared else B) * Hk, (B if shared else 1) * Lq * (H // Hk)
    return pairs * -(-rows // 128) > torch.cuda.get_device_properties(gpu).multi_processor_count


# ------------------------------------------------------------------ cross_attention
WIDE_CASES = [
    # B, Lq, Lk, H, Hk, D
    (33, 130, 65, 8, 8, 16),
    (20, 129, 133, 8, 8, 64),
    (9, 65, 191, 48, 16, 80),       # three heads a key head
    (17, 129, 200, 16, 16, 96),
    (17, 16, 1, 272, 17, 112),      # one key, sixteen heads a key head
    (5, 200, 257, 32, 8, 128),
    (33, 1, 300, 32, 8, 128),       # a token of many sequences: four rows of a tile
]


@pytest.mark.parametrize("B,Lq,Lk,H,Hk,D", WIDE_CASES)
@pytest.mark.parametrize("kind", ["all", "lens", "mask", "both"])
def test_cross_attention_tiles_of_128_rows(gpu, B, Lq, Lk, H, Hk, D, kind):
    assert wide_tiles(gpu, B, Lq, H, Hk)
    g = gen(9000, B, Lq, Lk, H, D)
    q, k, v = states(g, gpu, B, Lq, Lk, H, Hk, D, sharp=2.0)
    lens = mask = None
    if kind in ("lens", "both"):
        lens = g.integers(0, Lk + 1, B).astype(np.int32)
        lens[0], lens[1] = min(Lk, 1), 0
    if kind in ("mask", "both"):
        mask = g.random((B, Lq, Lk)) < 0.6
        mask[B // 2:, Lq // 2:, :Lk // 2] = False  # blocks that are hidden throughout
        if Lq > 1:
            mask[:, -1] = True
        mask[:, 0] &= np.arange(B)[:, None] % 2 == 1  # every other sequence's first token sees nothing
    o = s3d8.cross_attention(q, k, v, kv_lens=None if lens is None else dev(lens, gpu),
                             mask=None if mask is None else dev(mask, gpu))
    want, bound = ref.attention(host(q), host(k), host(v), D ** -0.5, lens, mask)
    close(o, want, bound)
    if lens is not None:
        assert (o[1] == 0).all()
    if mask is not None:
        assert (o[::2, 0] == 0).all()


def test_cross_attention_tiles_of_128_rows_shared(gpu):
    """Rows of several sequences in one tile."""
    B, Lq, Lk, H, Hk, D = 11, 500, 210, 8, 8, 64
    assert wide_tiles(gpu, B, Lq, H, Hk, shared=True)
    g = gen(9010)
    q, k, v = states(g, gpu, B, Lq, Lk, H, Hk, D, Bk=1)
    lens, mask = np.array([201], np.int32), g.random((B, Lq, Lk)) < 0.4
    mask[3], mask[4, :, 64:128] = False, False
    o = s3d8.cross_attention(q, k, v, kv_lens=dev(lens, gpu), mask=dev(mask, gpu))
    want, bound = ref.attention(host(q), host(k), host(v), D ** -0.5, lens, mask)
    close(o, want, bound)
    assert (o[3] == 0).all()


@pytest.mark.parametrize("B,Lq,Lk,H,Hk,D", [(1, 1, 1601, 32, 8, 128), (3, 1, 700, 15, 3, 112), (2, 1, 65, 8, 8, 96),
                                            (2, 1, 63, 4, 2, 64), (1, 1, 1, 1, 1, 16)])
@pytest.mark.parametrize("kind", ["random", "first half", "second half", "one key", "nothing"])
def test_cross_attention_mask_of_one_token(gpu, B, Lq, Lk, H, Hk, D, kind):
    """A decoded token whose mask hides blocks, whole splits of the keys, or all of them."""
    g = gen(9020, Lk, D)
    q, k, v = states(g, gpu, B, Lq, Lk, H, Hk, D, sharp=2.0)
    mask = g.random((B, Lq, Lk)) < 0.6
    if kind == "first half":
        mask[:, :, :Lk // 2] = False
    elif kind == "second half":
        mask[:, :, Lk // 2:] = False
    elif kind != "random":
        mask[:] = False
        if kind == "one key":
            mask[:, :, Lk // 3] = True
    o = s3d8.cross_attention(q, k, v, mask=dev(mask, gpu))
    want, bound = ref.attention(host(q), host(k), host(v), D ** -0.5, mask=mask)
    close(o, want, bound)
    if kind == "nothing":
        assert (o == 0).all()


@pytest.mark.parametrize("Lq,Lk", [(33000, 66100), (16000, 70000)])
def test_cross_attention_mask_of_more_blocks_than_are_listed(gpu, Lq, Lk):
    """Tiles of 128 rows on 1033 blocks of 64 keys, and of 64 rows whose two splits have 1094 blocks of 32."""
    D = 16
    assert wide_tiles(gpu, 1, Lq, 1, 1) == (Lq == 33000)
    g = gen(9030, Lq)
    q, k, v = states(g, gpu, 1, Lq, Lk, 1, 1, D, sharp=4.0)  # a row's weight is on few keys, each on others
    mask = np.repeat(g.random((1, 1, -(-Lk // 64))) < 0.5, 64, axis=2)[..., :Lk] & (g.random((1, 1, Lk)) < 0.9)
    o = s3d8.cross_attention(q, k, v, mask=dev(mask, gpu))
    some = np.unique([*g.integers(0, Lq, 300), 0, 31, 32, 63, 64, 127, 128, Lq - 1])
    want, bound = ref.attention(host(q[:, some]), host(k), host(v), D ** -0.5, mask=mask)
    close(o[:, some], want, bound)


@pytest.mark.parametrize("B,Lq,Lk,H,Hk,D,shared", [
    (1, 1, 1601, 32, 8, 128, False), (2, 140, 300, 4, 2, 80, False), (2, 33, 129, 4, 4, 48, False), (5, 20, 333, 8, 2, 96, True),
    (20, 129, 133, 8, 8, 64, False), (9, 65, 191, 48, 16, 80, False), (17, 129, 200, 16, 16, 96, False),
    (5, 200, 257, 32, 8, 128, False), (33, 1, 300, 32, 8, 128, False), (11, 500, 210, 8, 8, 64, True)])
def test_cross_attention_values_that_are_hidden_leave_the_bits(gpu, B, Lq, Lk, H, Hk, D, shared):
    """Infinities and NaN in values that a row does not see: the bits of a call with zeros there, in every build.  A row
    that sees some has their sum in their entry, and its other entries as they were."""
    g = gen(9040, B, Lq, Lk, D)
    q, k, v = states(g, gpu, B, Lq, Lk, H, Hk, D, Bk=1 if shared else None)
    mask = g.random((B, Lq, Lk)) < 0.6
    hidden = [3, 40, 41, Lk // 2, Lk - 9]
    mask[:, :, hidden] = False
    lens = np.full(1 if shared else B, Lk, np.int32)
    lens[-1] = Lk - 5
    inf, nan = float("inf"), float("nan")
    dirty_k, dirty_v, v = k.clone(), v.clone(), v.clone()
    dirty_k[:, hidden], dirty_k[-1, Lk - 5:] = nan, inf
    v[:, hidden], v[-1, Lk - 5:] = 0, 0
    dirty_v[:, hidden[0]], dirty_v[:, hidden[1:3]], dirty_v[:, hidden[3:]], dirty_v[-1, Lk - 5:] = inf, -inf, nan, nan
    extra = np.zeros((B, Lq, D))
    for key, entry, x in [(5, 0, inf), (6, 1, -inf), (7, 2, nan), (8, 3, inf), (Lk - 10, 3, -inf), (60, D - 1, inf),
                          (61, D - 1, inf), (9, 4, -inf), (10, 4, -inf), (2, 5, nan), (1, 5, inf)]:
        v[:, key, -1, entry], dirty_v[:, key, -1, entry] = 0, x
        with np.errstate(invalid="ignore"):
            extra[:, :, entry] += np.where(mask[:, :, key], x, 0)
    kw = dict(kv_lens=dev(lens, gpu), mask=dev(mask, gpu))
    want = s3d8.cross_attention(q, k, v, **kw)
    want[:, :, -(H // Hk):] += dev(extra, gpu, BF16)[:, :, None]
    got = s3d8.cross_attention(q, dirty_k, dirty_v, **kw)
    lost = torch.isnan(want)
    assert torch.equal(torch.isnan(got), lost)
    assert torch.equal(got[~lost], want[~lost])
    q[0, Lq // 2, 0] = nan  # a row of its own
    again = s3d8.cross_attention(q, dirty_k, dirty_v, **kw)
    assert torch.isnan(again[0, Lq // 2, 0]).all()
    again[0, Lq // 2, 0] = got[0, Lq // 2, 0]
    assert torch.equal(torch.isnan(again), lost) and torch.equal(again[~lost], got[~lost])


# ------------------------------------------------------------------ head_rope
@pytest.mark.parametrize("M,H,Hk,D,rot,layout,norm,dtype,out", [
    # two heads a group of lanes: heads that fill the device 6 to 20 times
    (1999, 32, 8, 128, 128, "half", True, BF16, "bf16"),      # 32 groups a workgroup
    (1300, 16, 7, 128, 64, "interleaved", True, F32, "bf16"),  # 16
    (1001, 5, 3, 10, 10, "half", True, F32, "f32"),            # 4: a pair a lane
    # four, of which the last workgroup has one left over
    (4003, 5, 3, 10, 6, "interleaved", False, F32, "f32"),
    (8193, 32, 8, 64, 64, "half", True, BF16, "bf16"),
])
def test_head_rope_heads_in_turn(gpu, M, H, Hk, D, rot, layout, norm, dtype, out):
    g = gen(9100, M, H, D, rot)
    q, k = (dev(g.standard_normal((M, n, D)).astype(np.float32), gpu, dtype) for n in (H, Hk))
    w = [dev((1 + 0.1 * g.standard_normal(D)).astype(np.float32), gpu) if norm else None for _ in range(2)]
    pos = g.integers(0, 130000, M)
    rope = s3d8.Rope(rot, layout=layout, device=gpu)
    f, factor = ref.frequencies(rot, 10000.0)
    both = s3d8.head_rope(q, k, dev(pos, gpu), rope, q_weight=w[0], k_weight=w[1], out=out)
    for x, y, weight in zip((q, k), both, w):
        want, bound = ref.head_rope(host(x), pos, f, factor, layout == "interleaved", None if weight is None else host(weight),
                                    1e-5)
        if out == "bf16":
            bound = bound + ref.HALF_BF16 * (np.abs(want) + bound)
        close(y, want, bound)


def test_head_rope_cosines_past_their_room(gpu):
    """One head of 80 a token, enough to fill the device 20 times: the cosines of the 128 tokens that a
    workgroup would take in turns of four do not fit, so it takes two.  The bits of small calls."""
    M, D = 165000, 80
    g = gen(9110)
    q = torch.randn(M, 1, D, device=gpu, generator=torch.Generator(device=gpu).manual_seed(9110)).to(BF16)
    rope, pos = s3d8.Rope(D, device=gpu), torch.arange(M, device=gpu)
    y = s3d8.head_rope(q, positions=pos, rope=rope, out="f32")
    for at in range(0, M, 4099):
        assert torch.equal(y[at:at + 4099], s3d8.head_rope(q[at:at + 4099], positions=pos[at:at + 4099], rope=rope, out="f32"))
    some = g.integers(0, M, 500)
    f, factor = ref.frequencies(D, 10000.0)
    want, bound = ref.head_rope(host(q)[some], some, f, factor, False, None, 1e-5)
    close(y[dev(some, gpu)], want, bound)


def test_head_rope_cosine_and_sine(gpu):
    """Cosine and sine themselves, as the turned pair (1, 0), in units of 2^-25, half a step of a value from 1/2 to 1.

    The rest x of at most an eighth of a turn is off by 1, its square z by 1.  Cosine: sin(x) <= 0.71 of the one and
    half of the other, the last sum's rounding 1, that of its factor (from 1/4 to 1/2, a half) times z <= 0.62, and less
    than 0.06 of what comes before: 2.6.  Sine: cos(x) <= 1 of x, the last rounding 1, z times x/6 <= 0.14, z x (half a unit)
    times 1/6, its factor (a quarter) times x^3 <= 0.49, the series' rest 0.06: 2.5.  Near an eighth of a turn the mean of 65536
    errors is that of the coefficients, 2^-30 times z^2 <= 0.39, and six times 2^-25 / sqrt(65536) at most: 2^-29.8."""
    D, M = 256, 512
    g = gen(9120)
    rope, q = s3d8.Rope(D, device=gpu), torch.zeros(M, 1, D, device=gpu)
    q[..., :D // 2] = 1

    def turned(angles):  # [M][D / 2]: a call a row, its angles as frequencies
        both = []
        for row in angles:
            rope.frequencies = dev(row, gpu)
            both.append(s3d8.head_rope(q[:1], positions=torch.ones(1, dtype=torch.int64, device=gpu), rope=rope, out="f32"))
        y = host(torch.cat(both))[:, 0]
        return y[:, :D // 2] - np.cos(angles), y[:, D // 2:] - np.sin(angles)

    for angles in (g.uniform(-20, 20, (M, D // 2)), np.pi / 4 * np.arange(-M * D // 4, M * D // 4).reshape(M, D // 2)):
        c, s = turned(angles)
        assert np.abs(c).max() <= 2.6 * 2.0 ** -25 and np.abs(s).max() <= 2.6 * 2.0 ** -25  # (either is either, by quarters)
    assert abs(turned(g.uniform(0.7, np.pi / 4, (M, D // 2)))[0].mean()) <= 2.0 ** -29.8


# ------------------------------------------------------------------ sample
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("top_k,top_p", [("rows", "rows"), (0, "rows"), (0, 1.0), (30, 0.9)])
def test_sample_sets_of_rows_share_a_workspace(gpu, dtype, top_k, top_p):
    """2500 rows in sets of 1024, 1024 and 452, rows of every kind in each: each set's result by itself, and some rows'
    against the plain form."""
    g = gen(9200)
    M, V = 2500, 4001
    logits = (3 * g.standard_normal((M, V))).astype(np.float32)
    logits[::11] = 1.5          # more equal logits than are listed
    logits[5::13] = -np.inf     # no token
    l, u = dev(logits, gpu, dtype), g.random(M, dtype=np.float32)
    T = (0.3 + g.random(M)).astype(np.float32)
    T[7::17] = 0
    k = np.array([0, 1, 50, 1000, 1024, 1025, 4000, 4001], np.int32)[np.arange(M) % 8]
    p = (0.5 + 0.6 * g.random(M)).astype(np.float32)
    k, p = k if top_k == "rows" else np.full(M, top_k, np.int32), p if top_p == "rows" else np.full(M, top_p, np.float32)

    def call(at):
        return s3d8.sample(l[at], dev(u[at], gpu), temperature=dev(T[at], gpu), min_p=1e-3,
                           top_k=dev(k[at], gpu) if top_k == "rows" else top_k,
                           top_p=dev(p[at], gpu) if top_p == "rows" else top_p)

    token, prob = call(slice(None))
    for at in (slice(0, 1024), slice(1024, 2048), slice(2048, M)):
        t, pr = call(at)
        assert torch.equal(token[at], t) and torch.equal(prob[at], pr)
    rows = l.float().cpu().numpy()
    for m in [*range(16), *range(1016, 1032), *range(2040, 2056), M - 1]:
        want, share = ref.sample(rows[m], u[m], T[m], k[m], p[m], 1e-3)
        assert int(token[m]) == want, m
        assert abs(float(prob[m]) - share) <= 2.0 ** -24 * share * 1.01 + 2.0 ** -43


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_sample_values_that_are_not_finite_in_parts(gpu, dtype):
    """Infinities and NaN first, last and between parts of rows that are cut, among finite logits and alone."""
    inf, nan = np.inf, np.nan
    g = gen(9210)
    V = 9001
    rows = (2 * g.standard_normal((10, V))).astype(np.float32)
    rows[0] = -inf
    rows[1] = nan
    rows[2] = -inf
    rows[2, [0, 4000]], rows[2, [1, V - 1]] = nan, 1.0     # two tokens, as far apart as can be
    rows[3, [17, 5000, V - 1]], rows[3, 18] = inf, nan     # three that take all
    rows[4, ::2], rows[4, 1::4] = nan, -inf
    rows[5, :8192], rows[5, 8192:] = nan, -3.0             # the last part alone
    rows[6, 0], rows[6, 4096] = 3.3e38, -3.3e38
    rows[7] = np.where(g.random(V) < 0.5, -3.3e38, -inf)
    rows[8] = np.array([1e-45, 0, -1e-45, -0.0], np.float32)[g.integers(0, 4, V)]
    rows[9, 4000:] = -inf
    for u0 in (0.0, 0.4, 0.999):
        u = np.full(len(rows), u0, np.float32)
        for args in [(1.0, 0, 1.0, 0.0), (1.0, 2, 1.0, 0.0), (1.0, 0, 0.6, 0.0), (0.0, 0, 1.0, 0.0), (1e-30, 0, 0.9, 0.1),
                     (1e30, 3, 0.9, 0.0), (0.8, 700, 0.9, 0.0), (1.0, 3000, 0.9, 0.0)]:
            check_sample(gpu, rows, u, *args, dtype)


def test_sample_limits_outside_their_range_in_parts(gpu):
    """As in a small vocabulary: values of rows outside their ranges count as the ends."""
    g = gen(9220)
    V = 5000
    logits = (2 * g.standard_normal((7, V))).astype(np.float32)
    u = np.array([0.3, 1.0, 2.0, -1.0, np.nan, 0.5, 0.999], np.float32)
    T = np.array([-1.0, 1.0, 1.0, np.nan, 1.0, 1.0, np.inf], np.float32)
    p = np.array([1.0, 1.5, 0.9, 0.9, -0.5, 0.7, 0.9], np.float32)
    mp = np.array([0, -1, 0, 0, 0, 3.0, 0], np.float32)
    for k in (np.array([-3, 0, 10, 0, 0, 2 ** 31 - 1, V], np.int32), np.zeros(7, np.int32)):
        token, prob = s3d8.sample(dev(logits, gpu), dev(u, gpu), temperature=dev(T, gpu), top_k=dev(k, gpu),
                                  top_p=dev(p, gpu), min_p=dev(mp, gpu))
        fine_u, fine_T = np.where(np.isnan(u), 0, u), np.minimum(np.where(np.isnan(T), 0, T), np.float32(2.0 ** 100))
        for m in range(7):
            want, share = ref.sample(logits[m], fine_u[m], fine_T[m], k[m], p[m], mp[m])
            assert int(token[m]) == want, m
            assert abs(float(prob[m]) - share) <= 2.0 ** -24 * share * 1.01 + 2.0 ** -43


# ------------------------------------------------------------------ buffers for results
def test_buffers_of_another_shape_are_refused(gpu):
    """A buffer with as many elements in another order of the dimensions would be filled in the wrong places; one with
    neighbouring dimensions joined takes the same bytes."""
    g = gen(9300)
    B, Lq, Lk, H, D, M = 2, 3, 20, 4, 32, 6
    q, k, v = states(g, gpu, B, Lq, Lk, H, 2, D)
    want = s3d8.cross_attention(q, k, v)
    for shape in [(B, H, Lq, D), (Lq, B, H, D), (B, Lq, D, H), (B * Lq * 2, H * D // 2), (B, Lq * 2, H, D // 2)]:
        o = torch.full(shape, 7.0, dtype=BF16, device=gpu)
        with pytest.raises(ValueError):
            s3d8.cross_attention(q, k, v, o=o)
        assert (o == 7).all()
    for shape in [(B, Lq, H * D), (B * Lq, H * D), (B * Lq, H, D), (B * Lq * H * D,)]:
        o = torch.empty(shape, dtype=BF16, device=gpu)
        assert s3d8.cross_attention(q, k, v, o=o) is o and torch.equal(o.view(q.shape), want)
    logits, u = dev(g.standard_normal((M, 50)).astype(np.float32), gpu), dev(g.random(M, dtype=np.float32), gpu)
    token, prob = s3d8.sample(logits, u)
    for bad in [(2, 3), (3, 2)]:
        with pytest.raises(ValueError):
            s3d8.sample(logits, u, token=torch.empty(bad, dtype=torch.int32, device=gpu))
        with pytest.raises(ValueError):
            s3d8.sample(logits, u, prob=torch.empty(bad, dtype=F32, device=gpu))
    column = torch.empty(M, 1, dtype=torch.int32, device=gpu)
    assert s3d8.sample(logits, u, token=column)[0] is column and torch.equal(column[:, 0], token)
    assert s3d8.sample(logits, u, token=token, prob=prob)[0] is token
