"""MX products at sizes that take every kernel the library has for them, at and
beside the sizes where one gives way to the next, against 64 bits on the GPU."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import gemm_qgemv_amd as q
import mx_ref as ref
from test_mx_gpu import BF16, DT, E2M1, E4M3, F32, Layer, Out, dev, operand, rng_for, run_experts, run_gemm, shares, wide_values

pytestmark = pytest.mark.gpu


def check_wide(got, x, w, xfmt, silu, dtype):
    """check_product with the plain form on the GPU: |error| of a sum at most
    sums_bound of the sum of magnitudes, of the activation what its sums'
    errors make of it and 8 roundings, and the output's rounding."""
    xv, wv = wide_values(*map(dev, x), xfmt), wide_values(*map(dev, w), E2M1)
    K, M = xv.shape[1], wv.shape[0] // (1 + silu)
    want, e = xv @ wv.T.contiguous(), (xv.abs() @ wv.abs().T.contiguous()) * ref.sums_bound(K)
    if silu:
        g, u, eg, eu = want[:, :M], want[:, M:], e[:, :M], e[:, M:]
        s = g / (1 + torch.exp(-g))
        want = s * u
        e = 1.1 * eg * (u.abs() + eu) + s.abs() * eu + 8 * 2.0 ** -24 * want.abs() + 2.0 ** -126
    if dtype == BF16:
        e = e + 2.0 ** -8 * (want.abs() + e)
    assert bool(((dev(got).double() - want).abs() <= e).all())


# rows and weight rows (gate and up both): some tens of rows, 16 to a block, with 64
# weight rows a workgroup up to 16384 and 128 above; more rows, in tiles of 64, 128
# and 256; and both sides of where the smallest pieces give way
KINDS = [(17, 8210), (32, 8196), (17, 16400), (32, 17408), (33, 5480), (64, 4102), (60, 17002), (64, 16386), (65, 3290), (77, 2740), (80, 16394), (77, 17408),
         (81, 16390), (90, 3002), (96, 2736), (96, 17002), (90, 16386),
         (97, 2400), (150, 1700), (129, 2050), (250, 1030), (700, 6146), (1030, 4100), (2000, 9000), (4100, 8194), (1000, 16004), (1900, 8190),
         (64, 4096), (16, 20002), (128, 2048), (256, 1024), (1024, 256), (1030, 262)]


@pytest.mark.parametrize("N,wide", KINDS)
@pytest.mark.parametrize("xfmt", [E2M1, E4M3])
@pytest.mark.parametrize("silu", [0, 1])
def test_product_of_every_kind(N, wide, xfmt, silu):
    rng = rng_for(60, N, wide, xfmt, silu)
    M = wide // (1 + silu)
    for K in (32 * int(rng.integers(1, 9)), 32 * int(rng.integers(9, 40))):
        dtype = [F32, BF16][int(rng.integers(0, 2))]
        x, w = operand(rng, N, K, xfmt), operand(rng, M * (1 + silu), K, E2M1)
        if silu:
            x[1][:] -= 8
        check_wide(run_gemm(x, w, xfmt, M, K, N, silu, dtype), x, w, xfmt, silu, dtype)


@pytest.mark.parametrize("K", [32, 64, 96, 128, 160, 224, 256, 288, 384, 416, 512, 544, 640, 1024, 1056, 1536, 1568, 2080])
@pytest.mark.parametrize("N,M", [(20, 8210), (75, 16400), (140, 2060)])
def test_product_of_every_depth(N, M, K):
    """Lengths that end in every place of a kernel's steps, sums exact."""
    for xfmt in (E2M1, E4M3):
        rng = rng_for(61, N, K, xfmt)
        x, w = operand(rng, N, K, xfmt, True), operand(rng, M, K, E2M1, True)
        got = run_gemm(x, w, xfmt, M, K, N, 0, F32)
        want = wide_values(*map(dev, x), xfmt) @ wide_values(*map(dev, w), E2M1).T.contiguous()
        assert bool((dev(got) == want.float()).all())


@pytest.mark.parametrize("N,M", [(20, 8210), (50, 17003), (75, 16401), (90, 3010), (140, 2063), (520, 8200)])
@pytest.mark.parametrize("xfmt", [E2M1, E4M3])
def test_kinds_nan_and_what_lies_behind(N, M, xfmt):
    """A NaN block makes its row or its column NaN and nothing else, and
    what lies behind the last rows (all NaN) does not matter."""
    rng = rng_for(62, N, M, xfmt)
    K = 544
    x, w = operand(rng, N + 70, K, xfmt), operand(rng, M + 70, K, E2M1)
    for t in (x, w):
        t[1][-70:] = 255
    x[0][-70:] = 0x7F
    x[1][N // 2, K // 32 - 1] = 255
    x[0][N // 2] = 0
    w[1][M - 3, 0] = 255
    nan = np.zeros((N, M), bool)
    nan[N // 2], nan[:, M - 3] = True, True
    if xfmt == E4M3:
        x[0][N - 1, K - 1] = 0x7F
        nan[N - 1] = True
    assert np.array_equal(np.isnan(run_gemm(x, w, xfmt, M, K, N, 0, F32)), nan)


def test_kinds_scales_of_any_size():
    for N, M in ((20, 8210), (75, 16401), (140, 2063)):
        for xfmt in (E2M1, E4M3):
            rng = rng_for(63, N, xfmt)
            K = 512
            x, w = operand(rng, N, K, xfmt), operand(rng, M, K, E2M1)
            x[1][:, :K // 32] = rng.integers(77, 177, (N, K // 32))
            w[1][:, :K // 32] = rng.integers(117, 137, (M, K // 32))
            check_wide(run_gemm(x, w, xfmt, M, K, N, 0, F32), x, w, xfmt, 0, F32)
            x[1][:, :K // 32], w[1][:, :K // 32] = 0, 254
            check_wide(run_gemm(x, w, xfmt, M, K, N, 0, F32), x, w, xfmt, 0, F32)


# rows, experts, top, weight rows: averages of 17 to some hundred pairs an expert
@pytest.mark.parametrize("rows,experts,top,wide", [(300, 32, 2, 1030), (300, 32, 2, 2060), (500, 24, 2, 2050), (640, 16, 2, 1500), (700, 16, 2, 3002), (900, 8, 1, 4100),
                                                   (1200, 16, 2, 1026), (2000, 8, 2, 2050), (4000, 16, 4, 1030), (64, 128, 8, 1024)])
@pytest.mark.parametrize("kind", ["even", "skewed", "some", "one"])
def test_experts_of_every_kind(rows, experts, top, wide, kind):
    seed = (rows, experts, top, wide)
    rng = rng_for(64, *seed)
    pick = int(rng.integers(0, 16))
    xfmt, silu, dtype, gather = [E2M1, E4M3][pick & 1], pick >> 1 & 1, [F32, BF16][pick >> 2 & 1], pick >> 3
    M, K = wide // (1 + silu), 32 * int(rng.integers(3, 30))
    ids = shares(rng, rows, experts, top, kind)
    offsets, order, _ = ref.plan(ids, experts)
    x = operand(rng, rows if gather else rows * top, K, xfmt)
    w = operand(rng, experts * M * (1 + silu), K, E2M1)
    if silu:
        x[1][:] -= 8
    got, raw = run_experts(x, w, xfmt, offsets, order if gather else None, rows, experts, top, silu, dtype, M, K)
    for e in range(experts):
        a, b = offsets[e], offsets[e + 1]
        if a < b:
            at = order[a:b] // top if gather else np.arange(a, b)
            check_wide(got[a:b], [t[at] for t in x], [t[e * M * (1 + silu):(e + 1) * M * (1 + silu)] for t in w], xfmt, silu, dtype)
    assert (raw[offsets[-1]:] == 0xA5).all(), "rows behind the last are left as they were"


@pytest.mark.parametrize("xfmt", [E2M1, E4M3])
@pytest.mark.parametrize("silu", [0, 1])
@pytest.mark.parametrize("rows,experts,top,wide,K", [(4000, 16, 4, 1790, 416), (2040, 8, 2, 3070, 800), (2040, 8, 2, 3070, 256), (4001, 60, 4, 1540, 544)])
def test_experts_in_the_largest_tiles(rows, experts, top, wide, K, silu, xfmt):
    rng = rng_for(67, rows, experts, wide, K, silu, xfmt)
    M = wide // (1 + silu)
    ids = shares(rng, rows, experts, top, "skewed")
    offsets, order, _ = ref.plan(ids, experts)
    for gather in (0, 1):
        x = operand(rng, rows if gather else rows * top, K, xfmt)
        w = operand(rng, experts * M * (1 + silu), K, E2M1)
        if silu:
            x[1][:] -= 8
        got, raw = run_experts(x, w, xfmt, offsets, order if gather else None, rows, experts, top, silu, BF16, M, K)
        for e in range(experts):
            a, b = offsets[e], offsets[e + 1]
            if a < b:
                at = order[a:b] // top if gather else np.arange(a, b)
                check_wide(got[a:b], [t[at] for t in x], [t[e * M * (1 + silu):(e + 1) * M * (1 + silu)] for t in w], xfmt, silu, BF16)
        assert (raw[offsets[-1]:] == 0xA5).all()


@pytest.mark.parametrize("xfmt", [E2M1, E4M3])
@pytest.mark.parametrize("M,silu", [(1500, 0), (2100, 1)])
def test_experts_of_every_kind_with_offsets_and_order_of_any_content(xfmt, M, silu):
    """Contents that are no plan's: nothing outside y is written (the bytes around it are
    held to it), and every address is held to its buffer by the kernels' own range checks."""
    rng = rng_for(65, xfmt, M)
    for rows, experts, top in ((300, 16, 2), (1000, 8, 2)):
        K = 288
        x, w = operand(rng, rows, K, xfmt), operand(rng, experts * M * (1 + silu), K, E2M1)
        for scale in (rows // 2, rows * 3, 2 ** 31):
            offsets = rng.integers(-scale, scale, experts + 1).astype(np.int32)
            order = rng.integers(-scale, scale, rows * top).astype(np.int32)
            run_experts(x, w, xfmt, offsets, order, rows, experts, top, silu, F32, M, K)


def test_two_graphs_share_a_workspace():
    """Two layers captured on the same workspace, replayed in turn: each launch
    lays out what it reads itself."""
    a, b = Layer(300, 256, 512, 4, 2, E4M3, BF16, 11), Layer(520, 288, 640, 4, 2, E2M1, F32, 12)
    assert q.qmoe_gemm_workspace_bytes(E2M1, q.QMX_SILU_MUL, 520, 4, 2, 640, 288) > 0, "both layers work in tiles"
    assert q.qmoe_gemm_workspace_bytes(E4M3, q.QMX_SILU_MUL, 300, 4, 2, 512, 256) > 0
    a.ws = b.ws = max(a.ws, b.ws, key=lambda t: t.numel())
    graphs = []
    side = torch.cuda.Stream()
    for layer in (a, b):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            layer.step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            layer.step()
        graphs.append(graph)
    want = []
    for layer in (a, b):
        layer.step()
        want.append(layer.out.clone())
    for i in range(4):
        a.out.zero_(), b.out.zero_(), a.ws.fill_(37 * i)
        for graph in (graphs if i % 2 else graphs[::-1]):
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a.out, want[0]) and torch.equal(b.out, want[1])


def test_operands_at_the_least_alignment():
    """Codes 16 bytes, scales 4 bytes, offsets and order 4 bytes into their buffers."""
    for N, M in ((3, 100), (20, 8210), (75, 16400), (140, 2060)):
        for xfmt in (E2M1, E4M3):
            rng = rng_for(66, N, xfmt)
            K = 160
            x, w = operand(rng, N, K, xfmt, True), operand(rng, M, K, E2M1, True)

            def moved(t, by):
                buffer = torch.full((t.size + by + 64,), 0x7F, dtype=torch.uint8, device="cuda")
                buffer[by:by + t.size] = dev(t).reshape(-1)
                return buffer[by:by + t.size]

            y = Out((N, M), DT[F32])
            need = q.qmx_gemm_workspace_bytes(xfmt, 0, M, K, N)
            ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda") if need else None
            q.qmx_gemm(xfmt, moved(x[0], 16), moved(x[1], 4), moved(w[0], 16), moved(w[1], 4), 0, F32, y.t, M, K, N, ws)
            want = wide_values(*map(dev, x), xfmt) @ wide_values(*map(dev, w), E2M1).T.contiguous()
            assert bool((dev(y.check()) == want.float()).all())


def random_operand(seed, rows, K, fmt):
    """operand on the GPU, for more bytes than the host should make."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.empty(rows, ref.row_bytes(fmt, K), dtype=torch.uint8, device="cuda")
    for part in codes.split(max(1, (1 << 30) // codes.shape[1])):
        part.copy_(torch.randint(0, 126 if fmt == E4M3 else 256, part.shape, generator=g, device="cuda", dtype=torch.uint8))
    scales = torch.randint(118, 130, (rows, ref.pitch(K)), generator=g, device="cuda", dtype=torch.uint8)
    return codes, scales


@pytest.mark.parametrize("xfmt,N,M,K,ends", [(E2M1, 3, 131080, 65536, "w"), (E4M3, 40, 131080, 65536, "w"), (E2M1, 130, 131080, 65536, "w"),
                                             (E4M3, 70001, 72, 65536, "x"), (E2M1, 140001, 8200, 64, "y"), (E4M3, 20, 7000000, 64, "M")])
def test_product_behind_four_gib(xfmt, N, M, K, ends):
    """Operands or outputs of more than 4 GiB (and as many outputs a row as there may be,
    nearly): the first and the last rows and columns."""
    x, w = random_operand(1, N, K, xfmt), random_operand(2, M, K, E2M1)
    y = torch.full((N, M), float("nan"), device="cuda")
    need = q.qmx_gemm_workspace_bytes(xfmt, 0, M, K, N)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda") if need else None
    q.qmx_gemm(xfmt, *x, *w, 0, F32, y, M, K, N, ws)
    for rows in (slice(0, 70), slice(max(0, N - 70), N)):
        for columns in (slice(0, 300), slice(M - 300, M) if M > 300 else slice(0, M)):
            xv, wv = wide_values(x[0][rows], x[1][rows], xfmt), wide_values(w[0][columns], w[1][columns], E2M1)
            e = (xv.abs() @ wv.abs().T.contiguous()) * ref.sums_bound(K)
            assert bool(((y[rows, columns].double() - xv @ wv.T.contiguous()).abs() <= e).all())
    assert not bool(torch.isnan(y[:, ::997]).any()) and not bool(torch.isnan(y[::997]).any())


@pytest.mark.parametrize("rows", [5, 2100, 5000])
def test_experts_weights_behind_four_gib(rows):
    experts, top, M, K = 40, 1, 16400, 16384
    x, w = random_operand(3, rows, K, E2M1), random_operand(4, experts * M, K, E2M1)
    ids = np.full((rows, top), experts - 1, np.int32)
    ids[:rows // 2] = 35
    offsets, order, _ = ref.plan(ids, experts)
    y = torch.full((rows, M), float("nan"), device="cuda")
    need = q.qmoe_gemm_workspace_bytes(E2M1, 0, rows, experts, top, M, K)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda") if need else None
    q.qmoe_gemm(E2M1, *x, *w, dev(offsets), dev(order), rows, experts, top, 0, F32, y, M, K, ws)
    for e, some in ((35, [0, rows // 2 - 1]), (39, [rows // 2, rows - 1])):
        xv = wide_values(x[0][some], x[1][some], E2M1)
        for columns in (slice(0, 300), slice(M - 300, M)):
            at = slice(e * M + columns.start, e * M + columns.stop)
            wv = wide_values(w[0][at], w[1][at], E2M1)
            e_ = (xv.abs() @ wv.abs().T.contiguous()) * ref.sums_bound(K)
            assert bool(((y[some, columns].double() - xv @ wv.T.contiguous()).abs() <= e_).all())
    assert not bool(torch.isnan(y).any())
