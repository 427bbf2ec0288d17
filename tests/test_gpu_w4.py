"""The 4-bit linear layer on the GPU against its plain 64-bit form."""
import numpy as np
import pytest

import block_reference as ref
import workloads

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
s3d8 = pytest.importorskip("w2_a8_matmul_amd")


def rng(*words):
    return np.random.Generator(np.random.PCG64(np.random.SeedSequence(list(words))))


def matrix(N, K, group, zeros):
    g = rng(7200, N, K, group, zeros)
    G = -(-K // group)
    q = g.integers(0, 16, (N, K), dtype=np.uint8)
    scales = ref.bf16_bits(g.lognormal(-5, 0.5, (N, G)).astype(np.float32) * np.where(g.random((N, G)) < 0.2, -1, 1))
    z = g.integers(0, 16, (N, G), dtype=np.uint8) if zeros else None
    return q, scales, z


def tiled_on(gpu, q, scales, z, group):
    return s3d8.W4Linear(ref.pack(q), scales, group, z, device=gpu)


def codes(M, K, word=0):
    g = rng(7201, M, K, word)
    return g.integers(-127, 128, (M, K), dtype=np.int8), g.lognormal(-3, 1, M).astype(np.float32)


def check(y, xq, xs, q, scales, z, group):
    y_r, size = ref.w4_linear(xq, xs, q, scales, z, group)
    err = np.abs(y.double().cpu().numpy() - y_r)
    tol = ref.w4_tolerance(y_r, size, q.shape[1], y.dtype == torch.bfloat16)
    assert (err <= tol).all(), (np.argwhere(err > tol)[:5], err.max())


def run(gpu, M, N, K, group, zeros, out="f32", word=0):
    q, scales, z = matrix(N, K, group, zeros)
    lin = tiled_on(gpu, q, scales, z, group)
    xq, xs = codes(M, K, word)
    dq, ds = torch.from_numpy(xq).to(gpu), torch.from_numpy(xs).to(gpu)
    # the output lies inside a larger buffer whose other values must survive
    dtype = torch.float32 if out == "f32" else torch.bfloat16
    pad = 4096
    buf = torch.full((M * N + 2 * pad,), 77.0, dtype=dtype, device=gpu)
    y = buf[pad:pad + M * N].view(M, N)
    assert lin.linear(dq, ds, y=y, out=out) is y
    check(y, xq, xs, q, scales, z, group)
    assert (buf[:pad] == 77).all() and (buf[pad + M * N:] == 77).all()
    again = lin.linear(dq, ds, out=out)
    assert torch.equal(again, y)  # the order of the sums is fixed


# every variant: rows (1 .. 4 .. 8 .. 16 .. more), scales per 128 columns, zero points
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 96, 128, 256])
@pytest.mark.parametrize("M", [1, 2, 4, 5, 8, 9, 16, 17, 33, 65, 130])
def test_rows_and_groups(gpu, M, group, zeros):
    run(gpu, M, 83, 656, group, zeros, "bf16" if M % 2 else "f32")


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M", [1, 3, 7, 16, 40, 300])
@pytest.mark.parametrize("N,K,group", [(1, 16, 32), (1, 4096, 64), (15, 48, 32), (16, 128, 128), (17, 144, 64),
                                       (31, 112, 64), (33, 2064, 128), (100, 240, 4096), (513, 1040, 32),
                                       (1003, 1296, 96)])
def test_ragged_shapes(gpu, N, K, group, M, zeros):
    run(gpu, M, N, K, group, zeros)


@pytest.mark.parametrize("M,N,K,group,zeros", [(1, 4096, 14336, 128, False), (8, 14336, 4096, 64, True),
                                               (256, 1280, 5120, 128, True), (512, 5120, 1280, 64, False),
                                               (515, 2500, 4096, 32, True), (1601, 700, 2064, 64, True),
                                               (1030, 1030, 528, 128, False), (2, 40000, 272, 32, False)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_larger_shapes(gpu, M, N, K, group, zeros, out):
    run(gpu, M, N, K, group, zeros, out)


# each workgroup tile of the many-row kernel (128 x 256, also with a last round in
# halves, 64 x 256, 64 x 128, 64 x 64, 32 x 128, 32 x 64 rows x channels), with 1, 2
# and 4 scales per 128 columns
@pytest.mark.parametrize("group,zeros", [(128, False), (64, False), (32, False), (128, True), (64, True), (32, True)])
@pytest.mark.parametrize("M,N,K", [(2000, 7000, 400), (1601, 5120, 272), (520, 7000, 656), (120, 14330, 1040), (50, 16000, 912),
                                   (30, 30000, 592), (40, 1000, 1296)])
def test_workgroup_tiles(gpu, M, N, K, group, zeros):
    run(gpu, M, N, K, group, zeros, "bf16" if zeros else "f32")


@pytest.mark.parametrize("M", [1, 6, 16, 20, 200])
@pytest.mark.parametrize("group,zeros", [(32, False), (64, True), (128, False), (128, True)])
def test_extremes(gpu, M, group, zeros):
    """Largest products of one sign, zero rows, zero scales, zero and largest zero points."""
    N, K = 48, 512
    G = K // group
    q = np.zeros((N, K), np.uint8)
    q[1::2] = 15
    scales = np.full((N, G), ref.bf16_bits(np.float32(1.0)), np.uint16)
    scales[3] = 0
    z = np.zeros((N, G), np.uint8) if zeros else None
    if zeros:
        z[::2] = 15
    xq = np.full((M, K), -127, np.int8)
    xq[M // 2] = 127
    xs = np.ones((M,), np.float32)
    if M > 2:
        xq[1], xs[1] = 0, 0.0
    lin = tiled_on(gpu, q, scales, z, group)
    y = lin.linear(torch.from_numpy(xq).to(gpu), torch.from_numpy(xs).to(gpu))
    y_r, _ = ref.w4_linear(xq, xs, q, scales, z, group)
    assert np.array_equal(y.double().cpu().numpy(), y_r)  # all of it small integers: exact


def test_one_hot_columns(gpu):
    """Each column alone reproduces its weight exactly: pins the layout."""
    for group, zeros in ((32, True), (64, False), (128, True)):
        N, K = 37, 272
        q, scales, z = matrix(N, K, group, zeros)
        lin = tiled_on(gpu, q, scales, z, group)
        eye = np.eye(K, dtype=np.int8)
        for rows in (slice(0, K), slice(5, 6), slice(100, 107), slice(200, 216)):
            xq = torch.from_numpy(np.ascontiguousarray(eye[rows])).to(gpu)
            y = lin.linear(xq, torch.ones(xq.shape[0], device=gpu)).cpu().numpy()
            zz = 8 if z is None else np.repeat(z, group, 1)[:, :K].astype(np.float32)
            w = (q.astype(np.float32) - zz) * ref.bf16_value(np.repeat(scales, group, 1)[:, :K])
            assert np.array_equal(y, w.T[rows])


@pytest.mark.parametrize("M", [1, 4, 19])
def test_forward_from_weights(gpu, M):
    W = workloads.gaussian_matrix([7202], 96, 320, 0.02)
    x = workloads.gaussian_matrix([7203, M], M, 320)
    for zeros in (False, True):
        lin = s3d8.W4Linear.from_weights(W, 64, zeros, device=gpu)
        q, scales, z = ref.w4_encode(W, 64, zeros)
        dx = torch.from_numpy(x).to(gpu)
        y, xq, xs = s3d8.w4_forward(dx, lin.tiled, 96, 64, zeros, return_all=True)
        cq, cs = ref.quantise(x)
        assert np.array_equal(xq.cpu().numpy(), cq) and np.array_equal(xs.cpu().numpy(), cs)
        check(y, cq, cs, q, scales, z if zeros else None, 64)
        assert torch.equal(lin(dx), y)
        # 4-bit weights: each is off by at most half a step (7.5 steps span a
        # group's largest value, its bf16 scale off by 2^-9), each code by half
        # of its step (plus fp32 rounding): a bound on the product's error
        step = ref.bf16_value(np.repeat(scales, 64, 1)[:, :320]).astype(np.float64)
        dw, da = 0.5 * step * (1 + 2.0 ** -4), 0.5 * cs.astype(np.float64)[:, None] * (1 + 2.0 ** -10)
        ax = np.abs(x).astype(np.float64)
        bound = ax @ dw.T + np.broadcast_to(da, x.shape) @ (np.abs(W) + dw).T
        assert (np.abs(y.double().cpu().numpy() - x.astype(np.float64) @ W.T.astype(np.float64)) <= bound).all()


def test_side_stream_and_two_at_once(gpu):
    q, scales, z = matrix(640, 1040, 64, True)
    lin = tiled_on(gpu, q, scales, z, 64)
    xa, sa = codes(3, 1040, 1)
    xb, sb = codes(70, 1040, 2)
    da, dsa, db, dsb = (torch.from_numpy(t).to(gpu) for t in (xa, sa, xb, sb))
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(gpu), torch.cuda.Stream(gpu)
    with torch.cuda.stream(one):
        ya = [lin.linear(da, dsa) for _ in range(4)]
    with torch.cuda.stream(two):
        yb = [lin.linear(db, dsb) for _ in range(4)]
    torch.cuda.synchronize()
    for y in ya:
        check(y, xa, sa, q, scales, z, 64)
    for y in yb:
        check(y, xb, sb, q, scales, z, 64)


def test_binding_refusals(gpu):
    q, scales, z = matrix(40, 128, 64, True)
    lin = tiled_on(gpu, q, scales, z, 64)
    xq, xs = (torch.from_numpy(t).to(gpu) for t in codes(3, 128))
    with pytest.raises(TypeError):
        lin.linear(xq, xs, y=torch.empty((3, 40), dtype=torch.bfloat16, device=gpu))
    with pytest.raises(ValueError):
        lin.linear(xq, xs, y=torch.empty((3, 39), device=gpu))
    with pytest.raises(ValueError):
        lin.linear(xq, xs[:2])
    with pytest.raises(ValueError):
        lin.linear(xq, xs, out="f16")
    with pytest.raises(TypeError):
        lin.linear(xq.cpu(), xs)
    with pytest.raises(ValueError):
        lin.linear(torch.zeros((128, 3), dtype=torch.int8, device=gpu).t(), xs)
    with pytest.raises(s3d8.S3D8Error):
        lin.linear(xq[:, :64].contiguous(), xs)  # another K: the size of the matrix does not fit
    with pytest.raises(s3d8.S3D8Error):
        s3d8.w4_linear(xq, xs, lin.tiled, 40, 64, False)
    with pytest.raises(s3d8.S3D8Error):
        s3d8.w4_linear(xq, xs, lin.tiled, 40, 48, True)
    packed = torch.from_numpy(ref.pack(q)).to(gpu)
    sc = torch.from_numpy(scales.view(np.int16)).to(gpu)
    with pytest.raises(ValueError):
        s3d8.w4_tile(packed, sc[:, :1].contiguous(), 64)
    with pytest.raises(TypeError):
        s3d8.w4_tile(packed, sc.float(), 64)
    with pytest.raises(ValueError):
        s3d8.w4_tile(packed, sc, 64, tiled=torch.empty(8, dtype=torch.uint8, device=gpu))
    with pytest.raises((ValueError, s3d8.S3D8Error)):
        s3d8.w4_tile(packed, sc, 0)
    torch.cuda.synchronize()


def test_many_rows_in_a_graph(gpu):
    """1601 rows, which may take two launches (the last row by itself), captured once and replayed."""
    M, N, K, group = 1601, 1280, 5120, 128
    q, scales, z = matrix(N, K, group, True)
    lin = tiled_on(gpu, q, scales, z, group)
    dq, ds = (torch.from_numpy(t).to(gpu) for t in codes(M, K))
    lin.linear(dq, ds)
    torch.cuda.synchronize()
    side = torch.cuda.Stream(gpu)
    side.wait_stream(torch.cuda.current_stream(gpu))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        y = lin.linear(dq, ds)
    for word in (1, 2, 3):
        xq, xs = codes(M, K, word)
        dq.copy_(torch.from_numpy(xq))
        ds.copy_(torch.from_numpy(xs))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(lin.linear(dq, ds), y)
        some = [0, 1, 63, 64, 800, 1535, 1536, 1599, 1600]
        check(y[some], xq[some], xs[some], q, scales, z, group)


@pytest.mark.parametrize("M,N,K", [(1 << 19, 20, 16), (1 << 19, 4080, 32), (16, 1 << 22, 32)])
def test_largest_sizes(gpu, M, N, K):
    """The most rows, an output of 8.6 GB, channels past 2^22: some rows and channels against the plain form."""
    q, scales, z = matrix(min(N, 4096), K, 32, False)
    times = N // q.shape[0]
    lin = tiled_on(gpu, np.tile(q, (times, 1)), np.tile(scales, (times, 1)), None, 32)
    xq, xs = codes(1024, K)
    xq, xs = xq[:M], xs[:M]
    dq, ds = torch.from_numpy(xq).to(gpu), torch.from_numpy(xs).to(gpu)
    rep = M // xq.shape[0]
    y = lin.linear(dq.repeat(rep, 1), ds.repeat(rep))
    check(y[:xq.shape[0], :q.shape[0]], xq, xs, q, scales, None, 32)
    check(y[M - xq.shape[0]:, N - q.shape[0]:], xq, xs, q, scales, None, 32)
    for a in range(0, M, max(M // 4, xq.shape[0])):
        assert torch.equal(y[a:a + xq.shape[0], :q.shape[0]], y[:xq.shape[0], :q.shape[0]])


def test_module_refuses_other_types(gpu):
    q, scales, z = matrix(40, 128, 64, True)
    for args in ((ref.pack(q), ref.bf16_value(scales), 64, z), (ref.pack(q).astype(np.int32), scales, 64, z),
                 (ref.pack(q), scales, 64, z.astype(np.float32))):
        with pytest.raises(TypeError):
            s3d8.W4Linear(*args, device=gpu)


@pytest.mark.parametrize("M", [1, 6, 12, 40, 200])
@pytest.mark.parametrize("group,zeros", [(32, False), (64, False), (128, False), (64, True)])
def test_scales_at_the_ends_of_their_range(gpu, M, group, zeros):
    """Sums close to the largest fp32 (2^126.9) and subnormal scales: what the definition says is finite or exact stays so."""
    N, K = 48, 512
    G = K // group
    q = np.zeros((N, K), np.uint8)
    q[1::2] = 15
    z = np.full((N, G), 8, np.uint8) if zeros else None
    xq = np.full((M, K), 127, np.int8)
    xq[M // 2] = -96
    # every partial sum is an integer below 2^20 times the scale: exact in fp32
    for exponent, x_exponent in ((107, -100), (-133, 60)):
        scales = np.full((N, G), ref.bf16_bits(np.float32(2.0 ** exponent)), np.uint16)
        xs = np.full((M,), 2.0 ** x_exponent, np.float32)
        lin = tiled_on(gpu, q, scales, z, group)
        y = lin.linear(torch.from_numpy(xq).to(gpu), torch.from_numpy(xs).to(gpu))
        y_r, _ = ref.w4_linear(xq, xs, q, scales, z, group)
        assert np.isfinite(y_r).all() and (np.abs(y_r) >= 2.0 ** -126).all()
        assert np.array_equal(y.double().cpu().numpy(), y_r)
    # random codes and scales, sums of up to 2^127
    g = rng(7204, M, group)
    q = g.integers(0, 16, (N, K), dtype=np.uint8)
    scales = ref.bf16_bits((g.lognormal(0, 0.3, (N, G)) * 2.0 ** 111).astype(np.float32))
    xq, _ = codes(M, K, 3)
    xs = np.full((M,), 2.0 ** -90, np.float32)
    y_r, size = ref.w4_linear(xq, xs, q, scales, z, group)
    assert (size * 2.0 ** 90 < 2.0 ** 127).all()
    lin = tiled_on(gpu, q, scales, z, group)
    check(lin.linear(torch.from_numpy(xq).to(gpu), torch.from_numpy(xs).to(gpu)), xq, xs, q, scales, z, group)


def test_module_refuses_activations_of_another_width(gpu):
    """Widths that end in the same block of 128 columns have tiled matrices of one size: the module knows its own."""
    N, K = 40, 240
    q, scales, z = matrix(N, K, 64, False)
    lin = tiled_on(gpu, q, scales, z, 64)
    for wrong in (144, 224, 256, 272):
        xq, xs = (torch.from_numpy(t).to(gpu) for t in codes(3, wrong))
        with pytest.raises(s3d8.S3D8Error):
            lin.linear(xq, xs)
        with pytest.raises(s3d8.S3D8Error):
            lin(torch.zeros((3, wrong), device=gpu))
    xq, xs = codes(3, K)
    check(lin.linear(torch.from_numpy(xq).to(gpu), torch.from_numpy(xs).to(gpu)), xq, xs, q, scales, z, 64)
    assert not lin(torch.zeros((3, K), device=gpu)).any()


def test_tile_refuses_other_shapes(gpu):
    """As many scales or zero points, but group by group instead of channel by channel; codes in three dimensions."""
    N, K, group = 48, 256, 64
    q, scales, z = matrix(N, K, group, True)
    packed, sc, zz = (torch.from_numpy(t).to(gpu) for t in (ref.pack(q), scales.view(np.int16), z))
    with pytest.raises(ValueError):
        s3d8.w4_tile(packed, sc.t().contiguous(), group, zz)
    with pytest.raises(ValueError):
        s3d8.w4_tile(packed, sc, group, zz.t().contiguous())
    with pytest.raises(ValueError):
        s3d8.w4_tile(packed.view(N, K // 4, 2), sc[:, :2].contiguous(), group, zz[:, :2].contiguous())
    with pytest.raises(ValueError):
        s3d8.W4Linear(packed, sc.t().contiguous(), group, zz)
    tiled = s3d8.w4_tile(packed, sc, group, zz)
    assert torch.equal(s3d8.w4_tile(packed, sc.flatten(), group, zz.flatten()), tiled)
    tiled = s3d8.w4_tile(packed, sc[:, :1].contiguous(), K, zz[:, :1].contiguous())  # one scale a channel
    assert torch.equal(s3d8.w4_tile(packed, sc[:, :1].reshape(1, N).contiguous(), K,
                                    zz[:, :1].reshape(1, N).contiguous()), tiled)


# every build of the kernel for few rows: tiles per group (1 up to 4096 channels on 256 CUs; 2; 4 past 12288 and 8
# rows), registers by rows (up to 4, 8, 16), scales per 128 columns and zero points
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N", [(3, 1000), (3, 4500), (7, 1000), (7, 4500), (13, 1000), (13, 4500), (13, 12500)])
def test_each_few_row_build(gpu, M, N, group, zeros):
    run(gpu, M, N, 656, group, zeros, "bf16" if zeros else "f32")


# the same with several tile groups a team, and with the columns on 4, 8 and 16 waves
@pytest.mark.parametrize("M,N,K,group,zeros", [(1, 14336, 4096, 64, False), (1, 4096, 4096, 128, True),
                                               (8, 30000, 1040, 128, False), (16, 30000, 1040, 32, True),
                                               (12, 50000, 528, 128, False), (2, 100000, 272, 64, True)])
def test_few_rows_in_rounds(gpu, M, N, K, group, zeros):
    run(gpu, M, N, K, group, zeros)
