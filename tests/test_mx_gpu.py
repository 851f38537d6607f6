"""The MX operators and the experts' layer on the GPU against plain forms in 64
bits (mx_ref). Tolerances come from the arithmetic: rounding to bf16 is off by
at most 2^-8 of the value, a float32 operation by 2^-24; products' sums see
mx_ref.sums_bound. Codes, scales, places and whole numbers have to be equal."""
import numpy as np
import pytest
import torch

import gemm_qgemv_amd as q
import mx_ref as ref

pytestmark = pytest.mark.gpu

F32, BF16 = q.QG_F32, q.QG_BF16
E2M1, E4M3 = q.QMX_E2M1, q.QMX_E4M3
DT = {F32: torch.float32, BF16: torch.bfloat16}
GUARD = 256                                              # elements before and behind every output


def rng_for(*key):
    return np.random.default_rng([2027, *key])


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Out:
    """An output buffer between guard bands."""

    def __init__(self, shape, dtype):
        self.n, self.shape, self.dtype = int(np.prod(shape)), shape, dtype
        size = torch.empty(0, dtype=dtype).element_size()
        self.pad = GUARD // size * size
        self.raw = torch.full(((self.n + 2 * self.pad) * size,), 0xA5, dtype=torch.uint8, device="cuda")
        self.t = self.raw.view(dtype)[self.pad:self.pad + self.n].view(shape)

    def check(self):
        size = self.t.element_size()
        torch.cuda.synchronize()
        raw = self.raw.cpu().numpy()
        assert (raw[:self.pad * size] == 0xA5).all() and (raw[(self.pad + self.n) * size:] == 0xA5).all(), "written outside"
        return self.t.float().cpu().numpy() if self.dtype == torch.bfloat16 else self.t.cpu().numpy()


def rounding(dtype, v):
    return 2.0 ** -8 * np.abs(v) if dtype == BF16 else 0.0


# ---------------------------------------------------------------------------
# Quantizer
# ---------------------------------------------------------------------------

def rows_of(rng, rows, K):
    x = (rng.standard_normal((rows, K)) * np.exp(rng.standard_normal(K) * 2)).astype(np.float32)
    b = x.reshape(-1, 32)
    for i in range(0, b.shape[0], 7):                    # ties and values beyond the largest element
        s = np.float32(2.0 ** rng.integers(-20, 20))
        b[i] = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.99, 0.0, -0.0, 17 / 16, 19 / 16, 2 ** -9, 3 * 2.0 ** -10], 32).astype(np.float32) * \
            rng.choice([-1, 1], 32).astype(np.float32) * s
        b[i, 3] = 7 * s
    return x


def run_quant(x, dtype, fmt, pad=0):
    rows, K = x.shape
    wide = torch.zeros(rows, K + pad, dtype=DT[dtype], device="cuda")
    wide[:, :K] = dev(x).to(DT[dtype])
    codes, scales = Out((rows, ref.row_bytes(fmt, K)), torch.uint8), Out((rows, ref.pitch(K)), torch.uint8)
    q.qmx_quant(dtype, wide, K + pad, rows, K, fmt, codes.t, scales.t)
    return codes.check(), scales.check(), wide[:, :K].float().cpu().numpy()


@pytest.mark.parametrize("fmt", [E2M1, E4M3])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,K,pad", [(1, 32, 0), (3, 96, 8), (64, 2048, 0), (257, 160, 16), (5, 6144, 128), (1000, 64, 0), (17, 4192, 0)])
def test_quant(fmt, dtype, rows, K, pad):
    codes, scales, x = run_quant(rows_of(rng_for(1, rows, K), rows, K), dtype, fmt, pad)
    want_codes, want_scales = ref.quantize(x, fmt)
    assert np.array_equal(scales, want_scales)
    assert np.array_equal(codes, want_codes)


@pytest.mark.parametrize("fmt", [E2M1, E4M3])
def test_quant_any_bits(fmt):
    """Any float32 bit pattern: subnormal numbers, the largest, infinities, NaN."""
    rng = rng_for(2, fmt)
    x = rng.integers(0, 2 ** 32, (512, 256), dtype=np.uint64).astype(np.uint32).view(np.float32)
    x[::3] = (rng.integers(0, 2 ** 24, x[::3].shape).astype(np.uint32) | (rng.integers(0, 2, x[::3].shape).astype(np.uint32) << 31)).view(np.float32)
    x[1::3][np.abs(x[1::3]) > 1e30] = 3.4e38
    x[1::3][np.isnan(x[1::3])] = -3.4e38
    x[5, 40], x[8, 0], x[11, 255] = np.inf, -np.inf, np.nan
    codes, scales, x = run_quant(x, F32, fmt)
    want_codes, want_scales = ref.quantize(x, fmt)
    assert np.array_equal(scales, want_scales) and np.array_equal(codes, want_codes)
    assert (scales == 255).any() and (scales == 0).any()


@pytest.mark.parametrize("fmt", [E2M1, E4M3])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_dequant_every_code_and_scale(fmt, dtype):
    K = 512
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], ref.pitch(K), axis=1)
    codes = np.tile(np.arange(ref.row_bytes(fmt, K)).astype(np.uint8), (256, 1))
    x = Out((256, K + 24), DT[dtype])
    q.qmx_dequant(fmt, dev(codes), dev(scales), 256, K, dtype, x.t, K + 24)
    got = x.check()[:, :K]
    with np.errstate(over="ignore"):
        want = torch.from_numpy(ref.values(codes, scales, fmt).astype(np.float32)).to(DT[dtype]).float().numpy()
    assert np.array_equal(got, want, equal_nan=True)
    assert np.array_equal(np.signbit(got), np.signbit(want)) or np.isnan(want).any()
    left = x.t[:, K:].contiguous().view(torch.uint8).cpu().numpy()
    assert (left == 0xA5).all()                          # what lies between rows


def test_quant_rows_behind_four_gib():
    """Offsets past 32 bits: the last rows of a tall matrix."""
    rows, K = 700_001, 4096
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")           # 5.7 GB
    tail = rows_of(rng_for(3), 3, K)
    x[-3:] = dev(tail).bfloat16()
    codes = torch.empty(rows, K, dtype=torch.uint8, device="cuda")
    scales = torch.empty(rows, K // 32, dtype=torch.uint8, device="cuda")
    q.qmx_quant(BF16, x, K, rows, K, E4M3, codes, scales)
    want = ref.quantize(x[-3:].float().cpu().numpy(), E4M3)
    assert np.array_equal(codes[-3:].cpu().numpy(), want[0]) and np.array_equal(scales[-3:].cpu().numpy(), want[1])
    assert not codes[:-3].any()
    x[-3:] = 0
    q.qmx_dequant(E4M3, codes, scales, rows, K, BF16, x, K)
    assert np.array_equal(x[-3:].float().cpu().numpy(), torch.from_numpy(ref.values(*want, E4M3)).bfloat16().float().numpy())


# ---------------------------------------------------------------------------
# Products
# ---------------------------------------------------------------------------

def operand(rng, rows, K, fmt, whole=False):
    """Random codes and scales; `whole`: scales of 1, so that sums are exact."""
    codes = rng.integers(0, 256, (rows, ref.row_bytes(fmt, K))).astype(np.uint8)
    if fmt == E4M3:
        if whole:                                        # 0, 1, .., 7 and negatives
            codes = np.array([0, 0x38, 0x40, 0x44, 0x48, 0x4a, 0x4c, 0x4e], np.uint8)[codes % 8] | (codes & 128)
        codes[(codes & 127) == 127] = 0x31
    scales = rng.integers(118, 130, (rows, ref.pitch(K))).astype(np.uint8)
    if whole:
        scales[:] = 127
    scales[:, K // 32:] = 255                            # padding may hold anything
    return codes, scales


def run_gemm(x, w, xfmt, M, K, N, silu, dtype, stream=None):
    need = q.qmx_gemm_workspace_bytes(xfmt, silu, M, K, N)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda") if need else None
    y = Out((N, M), DT[dtype])
    q.qmx_gemm(xfmt, *[dev(t) for t in x], *[dev(t) for t in w], silu, dtype, y.t, M, K, N, ws, stream=stream)
    return y.check()


def check_product(got, x, w, xfmt, silu, dtype):
    want, bound = ref.product(ref.values(*x, xfmt), ref.values(*w, E2M1), silu)
    bad = ~(np.abs(got - want) <= bound + rounding(dtype, np.abs(want) + bound))
    assert not bad.any(), (np.argwhere(bad)[:4], np.max(np.abs(got - want) / (bound + 1e-300)))


SIZES = [(1, 1, 32), (1, 6144, 2048), (2, 30, 64), (5, 100, 160), (16, 257, 544), (17, 64, 96), (33, 700, 288), (48, 1024, 1056), (64, 129, 2080),
         (65, 300, 256), (100, 1000, 512), (129, 515, 224), (200, 640, 1280), (300, 2050, 736), (31, 2048, 5120), (256, 256, 256), (13, 5001, 320)]


@pytest.mark.parametrize("silu", [0, 1])
@pytest.mark.parametrize("xfmt", [E2M1, E4M3])
@pytest.mark.parametrize("N,M,K", SIZES)
def test_product_exact_sums(N, M, K, xfmt, silu):
    """Small whole numbers: float32 sums are exact in any order, so every
    element of both operands has to be in its place."""
    rng = rng_for(10, N, M, K, xfmt, silu)
    x, w = operand(rng, N, K, xfmt, True), operand(rng, M * (1 + silu), K, E2M1, True)
    got = run_gemm(x, w, xfmt, M, K, N, silu, F32)
    xv, wv = ref.values(*x, xfmt), ref.values(*w, E2M1)
    if silu:
        check_product(got, x, w, xfmt, silu, F32)
    else:
        assert np.array_equal(got, (xv @ wv.T).astype(np.float32))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("silu", [0, 1])
@pytest.mark.parametrize("xfmt", [E2M1, E4M3])
@pytest.mark.parametrize("N,M,K", SIZES)
def test_product(N, M, K, xfmt, silu, dtype):
    rng = rng_for(11, N, M, K, xfmt, silu, dtype)
    x, w = operand(rng, N, K, xfmt), operand(rng, M * (1 + silu), K, E2M1)
    if silu:                                             # gates of a size that matters
        x[1][:] -= 8
    check_product(run_gemm(x, w, xfmt, M, K, N, silu, dtype), x, w, xfmt, silu, dtype)


@pytest.mark.parametrize("seed", range(24))
def test_product_random_sizes(seed):
    rng = rng_for(12, seed)
    N, M = int(np.exp(rng.uniform(0, np.log(700)))), int(np.exp(rng.uniform(0, np.log(3000))))
    K = 32 * int(np.exp(rng.uniform(0, np.log(120))))
    xfmt, silu, dtype = [E2M1, E4M3][seed % 2], seed // 2 % 2, [F32, BF16][seed // 4 % 2]
    x, w = operand(rng, N, K, xfmt), operand(rng, M * (1 + silu), K, E2M1)
    check_product(run_gemm(x, w, xfmt, M, K, N, silu, dtype), x, w, xfmt, silu, dtype)


def wide_values(codes, scales, fmt):
    """ref.values on the GPU, for products too large for the CPU."""
    t = torch.from_numpy(ref.E2M1_VALUES if fmt == E2M1 else ref.E4M3_VALUES).cuda()
    c = torch.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1) if fmt == E2M1 else codes
    return t[c.long()] * torch.exp2(scales[:, :c.shape[1] // 32].double() - 127).repeat_interleave(32, 1)


@pytest.mark.parametrize("xfmt,N,M,K,silu,dtype", [(E2M1, 2051, 16400, 288, 0, BF16), (E2M1, 4097, 4100, 1056, 1, F32), (E4M3, 2051, 16400, 288, 0, F32),
                                                   (E4M3, 4097, 4100, 1056, 1, BF16), (E2M1, 1500, 9000, 2048, 0, F32), (E4M3, 700, 20001, 512, 0, BF16)])
def test_product_large(xfmt, N, M, K, silu, dtype):
    rng = rng_for(13, N, M, K, xfmt, silu)
    x, w = operand(rng, N, K, xfmt), operand(rng, M * (1 + silu), K, E2M1)
    if silu:
        x[1][:] -= 8
    got = torch.from_numpy(run_gemm(x, w, xfmt, M, K, N, silu, dtype)).cuda().double()
    xv, wv = wide_values(*map(dev, x), xfmt), wide_values(*map(dev, w), E2M1)
    want, e = xv @ wv.T, (xv.abs() @ wv.abs().T) * ref.sums_bound(K)
    if silu:
        g, u, eg, eu = want[:, :M], want[:, M:], e[:, :M], e[:, M:]
        s = g / (1 + torch.exp(-g))
        want = s * u
        e = 1.1 * eg * (u.abs() + eu) + s.abs() * eu + 8 * 2.0 ** -24 * want.abs() + 2.0 ** -126
    if dtype == BF16:
        e = e + 2.0 ** -8 * (want.abs() + e)
    assert bool(((got - want).abs() <= e).all())


@pytest.mark.parametrize("N", [3, 40, 150])
@pytest.mark.parametrize("xfmt", [E2M1, E4M3])
def test_product_scales_of_any_size(N, xfmt):
    """Scales from 2^-100 to 2^100 in one row: a sum keeps 24 bits of its
    largest product; and scale 0 (2^-127) beside 254 (2^127)."""
    rng = rng_for(14, N, xfmt)
    M, K = 70, 512
    x, w = operand(rng, N, K, xfmt), operand(rng, M, K, E2M1)
    x[1][:, :K // 32] = rng.integers(77, 177, (N, K // 32))
    w[1][:, :K // 32] = rng.integers(117, 137, (M, K // 32))
    check_product(run_gemm(x, w, xfmt, M, K, N, 0, F32), x, w, xfmt, 0, F32)
    x[1][:, :K // 32], w[1][:, :K // 32] = 0, 254
    check_product(run_gemm(x, w, xfmt, M, K, N, 0, F32), x, w, xfmt, 0, F32)


@pytest.mark.parametrize("N,M", [(5, 40), (50, 300), (200, 640)])
@pytest.mark.parametrize("xfmt", [E2M1, E4M3])
def test_product_nan_blocks(N, M, xfmt):
    """A NaN block makes its row or its column NaN, and nothing else."""
    rng = rng_for(15, N, M, xfmt)
    K = 544
    x, w = operand(rng, N, K, xfmt), operand(rng, M, K, E2M1)
    x[1][N // 2, K // 32 - 1] = 255
    x[0][N // 2] = 0
    w[1][M - 3, 0] = 255
    nan = np.zeros((N, M), bool)
    nan[N // 2], nan[:, M - 3] = True, True
    if xfmt == E4M3:
        x[0][N - 1, K - 1] = 0x7F                        # an element that is NaN
        nan[N - 1] = True
    got = run_gemm(x, w, xfmt, M, K, N, 0, F32)
    assert np.array_equal(np.isnan(got), nan)


@pytest.mark.parametrize("N,M,K", [(4, 64, 96), (40, 130, 416), (150, 700, 288)])
@pytest.mark.parametrize("xfmt", [E2M1, E4M3])
def test_product_reads_nothing_behind(N, M, K, xfmt):
    """What lies behind the operands' last rows (NaN codes and scales) does not matter."""
    rng = rng_for(16, N, M, K, xfmt)
    x, w = operand(rng, N + 70, K, xfmt), operand(rng, M + 70, K, E2M1)
    for t in (x, w):
        t[1][-70:] = 255
    x[0][-70:] = 0x7F
    y = Out((N, M), torch.float32)
    need = q.qmx_gemm_workspace_bytes(xfmt, 0, M, K, N)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda") if need else None
    q.qmx_gemm(xfmt, *[dev(t) for t in x], *[dev(t) for t in w], 0, F32, y.t, M, K, N, ws)
    check_product(y.check(), [t[:N] for t in x], [t[:M] for t in w], xfmt, 0, F32)


# ---------------------------------------------------------------------------
# Router and plan
# ---------------------------------------------------------------------------

def run_plan(ids, experts):
    rows, top = ids.shape
    need = q.qmoe_plan_workspace_bytes(rows, experts, top)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda") if need else None
    o = [Out((experts + 1,), torch.int32), Out((rows * top,), torch.int32), Out((rows, top), torch.int32)]
    q.qmoe_plan(dev(ids), rows, experts, top, *[b.t for b in o], ws)
    return [b.check() for b in o]


@pytest.mark.parametrize("rows,experts,top", [(1, 1, 1), (1, 128, 8), (7, 3, 2), (64, 64, 8), (500, 1000, 4), (511, 60, 8), (513, 8, 8),
                                              (2500, 256, 6), (40000, 128, 8), (70001, 1024, 1), (3000, 7, 5)])
@pytest.mark.parametrize("kind", ["even", "skewed", "some", "one", "none"])
def test_plan(rows, experts, top, kind):
    rng = rng_for(20, rows, experts, top)
    ids = rng.integers(0, experts, (rows, top))
    if kind == "skewed":
        ids = np.minimum(ids, rng.integers(0, experts, (rows, top)) // 3)
    elif kind == "some":                                 # another GPU's experts, and none
        ids = rng.integers(-experts, 2 * experts, (rows, top))
        ids[rng.random((rows, top)) < 0.1] = -2 ** 31
        ids[rng.random((rows, top)) < 0.1] = 2 ** 31 - 1
    elif kind == "one":
        ids[:] = experts - 1
    elif kind == "none":
        ids[:] = -1
    got = run_plan(ids.astype(np.int32), experts)
    for g, w in zip(got, ref.plan(ids.astype(np.int32), experts)):
        assert np.array_equal(g, w)


def test_plan_of_no_rows():
    offsets = Out((9,), torch.int32)
    e = torch.empty(16, dtype=torch.int32, device="cuda")
    q.qmoe_plan(e, 0, 8, 2, offsets.t, e, e)
    assert not offsets.check().any()


def run_route(x, ld, rows, experts, top, renorm, dtype):
    wide = torch.full((rows, ld), float("nan"), dtype=DT[dtype], device="cuda")
    wide[:, :experts] = dev(x).to(DT[dtype])
    need = q.qmoe_plan_workspace_bytes(rows, experts, top)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda") if need else None
    ids, w = Out((rows, top), torch.int32), Out((rows, top), torch.float32)
    o = [Out((experts + 1,), torch.int32), Out((rows * top,), torch.int32), Out((rows, top), torch.int32)]
    q.qmoe_route(dtype, wide, ld, rows, experts, top, renorm, ids.t, w.t, *[b.t for b in o], ws)
    return wide[:, :experts].double().cpu().numpy(), ids.check(), w.check(), [b.check() for b in o]


@pytest.mark.parametrize("dtype,renorm", [(F32, 0), (F32, 1), (BF16, 0), (BF16, 1)])
@pytest.mark.parametrize("rows,experts,top,pad", [(1, 1, 1, 0), (1, 128, 8, 0), (5, 7, 7, 1), (64, 128, 8, 0), (33, 60, 4, 5), (17, 64, 32, 0), (100, 65, 1, 0),
                                                  (40, 256, 16, 0), (40, 257, 17, 3), (1000, 512, 10, 0), (30, 1024, 32, 0), (20, 1000, 6, 7), (600, 16, 2, 0)])
def test_route(rows, experts, top, pad, dtype, renorm):
    rng = rng_for(21, rows, experts, top)
    x = (rng.standard_normal((rows, experts)) * 2).astype(np.float32)
    if rows > 4:
        x[::3] = np.round(x[::3])                        # ties, zeros of both signs
        x[1::4][rng.random(x[1::4].shape) < 0.3] = -np.inf
        x[4, :] = -np.inf
        x[3, :] = -np.inf
        x[3, experts - 1] = -1e38
    if rows > 16:
        x[7, experts // 2], x[8, 0], x[9, -1] = np.nan, np.inf, -np.nan
        x[10] = 88.0
        x[11] *= 1e30
        x[12] *= 1e-40
    xs, ids, w, planned = run_route(x, experts + pad, rows, experts, top, renorm, dtype)
    want_ids, want_w = ref.route(xs, top, renorm)
    assert np.array_equal(ids, want_ids)
    assert np.array_equal(np.isnan(w), np.isnan(want_w))
    # the differences x - max are rounded (2^-24 of up to 104 where the exponential does not
    # vanish), an exponential is off by 2 units, sums of 16 V numbers by V + 4, quotient 2
    tol = 2.0 ** -24 * (104 + 4 + experts / 16 + 5 + top + 4) * np.abs(want_w) + 2.0 ** -126
    ok = ~np.isnan(want_w)
    assert np.all(np.abs(w - want_w)[ok] <= tol[ok])
    for g, p in zip(planned, ref.plan(want_ids, experts)):
        assert np.array_equal(g, p)


def test_route_many_rows():
    """Several runs of the sort, and their workspace."""
    rng = rng_for(22)
    rows, experts, top = 9001, 100, 6
    x = rng.standard_normal((rows, experts)).astype(np.float32)
    x[rng.random(rows) < 0.1] = -np.inf
    xs, ids, w, planned = run_route(x, experts, rows, experts, top, 1, F32)
    want_ids, want_w = ref.route(xs, top, 1)
    assert np.array_equal(ids, want_ids) and np.allclose(w, want_w, rtol=1e-5, atol=0)
    for g, p in zip(planned, ref.plan(want_ids, experts)):
        assert np.array_equal(g, p)


# ---------------------------------------------------------------------------
# Experts' products
# ---------------------------------------------------------------------------

def shares(rng, rows, experts, top, kind):
    if kind == "one":
        return np.full((rows, top), experts // 2, np.int32)
    like = rng.standard_normal(experts) * (3 if kind == "skewed" else 0.5)
    ids = np.argsort(-(rng.standard_normal((rows, experts)) + like), axis=1)[:, :top].astype(np.int32)
    if kind == "some":
        ids[rng.random((rows, top)) < 0.4] = -1
    return ids


def run_experts(x, w, xfmt, offsets, order, rows, experts, top, silu, dtype, M, K):
    need = q.qmoe_gemm_workspace_bytes(xfmt, silu, rows, experts, top, M, K)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda") if need else None
    y = Out((rows * top, M), DT[dtype])
    q.qmoe_gemm(xfmt, *[dev(t) for t in x], *[dev(t) for t in w], dev(offsets), None if order is None else dev(order), rows, experts, top,
                silu, dtype, y.t, M, K, ws)
    got = y.check()
    return got, y.t.view(torch.uint8).reshape(rows * top, -1).cpu().numpy()


@pytest.mark.parametrize("kind", ["even", "skewed", "some", "one"])
@pytest.mark.parametrize("gather", [0, 1])
@pytest.mark.parametrize("rows,experts,top,M,K", [(1, 128, 8, 64, 256), (1, 1, 1, 17, 32), (5, 8, 2, 100, 160), (64, 64, 8, 40, 96), (150, 3, 2, 130, 288),
                                                  (300, 16, 4, 66, 544), (700, 4, 3, 257, 64), (40, 300, 6, 33, 128), (1200, 8, 4, 1030, 256), (9, 1024, 32, 16, 64)])
def test_experts(rows, experts, top, M, K, gather, kind):
    seed = (rows, experts, top, M, K, gather)
    rng = rng_for(30, *seed)
    pick = int(rng.integers(0, 8))
    xfmt, silu, dtype = [E2M1, E4M3][pick & 1], pick >> 1 & 1, [F32, BF16][pick >> 2]
    ids = shares(rng, rows, experts, top, kind)
    offsets, order, _ = ref.plan(ids, experts)
    x = operand(rng, rows if gather else rows * top, K, xfmt)
    w = operand(rng, experts * M * (1 + silu), K, E2M1)
    if silu:
        x[1][:] -= 8
    got, raw = run_experts(x, w, xfmt, offsets, order if gather else None, rows, experts, top, silu, dtype, M, K)
    wide = M * (1 + silu)
    for e in range(experts):
        a, b = offsets[e], offsets[e + 1]
        if a < b:
            at = order[a:b] // top if gather else np.arange(a, b)
            check_product(got[a:b], [t[at] for t in x], [t[e * wide:(e + 1) * wide] for t in w], xfmt, silu, dtype)
    assert (raw[offsets[-1]:] == 0xA5).all(), "rows behind the last are left as they were"


@pytest.mark.parametrize("xfmt,silu", [(E2M1, 1), (E4M3, 0)])
def test_experts_large(xfmt, silu):
    """The largest tiles, every expert's weights in place."""
    rng = rng_for(31, xfmt)
    rows, experts, top, M, K = 4099, 16, 4, 1000, 512
    ids = shares(rng, rows, experts, top, "skewed")
    offsets, order, _ = ref.plan(ids, experts)
    x, w = operand(rng, rows, K, xfmt, True), operand(rng, experts * M * (1 + silu), K, E2M1, True)
    x[1][:] = 120                                        # sums exact, gates of a size that matters
    got, _ = run_experts(x, w, xfmt, offsets, order, rows, experts, top, silu, F32, M, K)
    xv, wv = wide_values(*map(dev, x), xfmt), wide_values(*map(dev, w), E2M1).reshape(experts, M * (1 + silu), K)
    got = torch.from_numpy(got).cuda()
    for e in range(experts):
        a, b = offsets[e], offsets[e + 1]
        y = xv[dev(order[a:b] // top).long()] @ wv[e].T
        if silu:
            g, u = y[:, :M], y[:, M:]
            y = g / (1 + torch.exp(-g)) * u
            assert bool(((got[a:b] - y).abs() <= 2.0 ** -20 * y.abs() + 2.0 ** -126).all())
        else:
            assert bool((got[a:b] == y.float()).all())


def test_experts_offsets_and_order_of_any_content():
    """Contents that are no plan's: nothing outside y is written, no place
    outside the inputs is read (each address is held to its buffer by the kernels' own range checks)."""
    rng = rng_for(32)
    rows, experts, top, M, K = 60, 20, 3, 70, 288
    x, w = operand(rng, rows, K, E2M1), operand(rng, experts * M, K, E2M1)
    for scale in (50, 400, 2 ** 31):
        offsets = rng.integers(-scale, scale, experts + 1).astype(np.int32)
        order = rng.integers(-scale, scale, rows * top).astype(np.int32)
        run_experts(x, w, E2M1, offsets, order, rows, experts, top, 0, F32, M, K)
    # an order that points outside stands for zeros
    offsets = np.full(experts + 1, rows * top, np.int32)
    offsets[:4] = 0
    order = np.where(rng.random(rows * top) < 0.5, rng.integers(0, rows * top, rows * top), rng.choice([-1, rows * top, 2 ** 31 - 1], rows * top)).astype(np.int32)
    got, _ = run_experts(x, w, E2M1, offsets, order, rows, experts, top, 0, F32, M, K)
    ok = (order >= 0) & (order < rows * top)
    xs = [np.where(ok[:, None], t[np.where(ok, order // top, 0)], 0) for t in x]
    check_product(got, xs, [t[3 * M:4 * M] for t in w], E2M1, 0, F32)


# ---------------------------------------------------------------------------
# Way back
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,out_dtype", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("rows,top,M", [(1, 1, 1), (1, 8, 2048), (7, 3, 30), (64, 8, 1024), (100, 5, 257), (33, 32, 40), (1000, 6, 136)])
def test_combine(rows, top, M, dtype, out_dtype):
    rng = rng_for(40, rows, top, M)
    y = dev(rng.standard_normal((rows * top, M)).astype(np.float32)).to(DT[dtype])
    slots = rng.permutation(rows * top).reshape(rows, top).astype(np.int32)
    slots[rng.random((rows, top)) < 0.2] = -1
    if rows > 5:
        slots[1, 0], slots[2, -1], slots[3, 0] = rows * top, -2 ** 31, 2 ** 31 - 1
        slots[4] = -1
        slots[5] = slots[5, 0]                           # the same row twice
    w = rng.random((rows, top)).astype(np.float32)
    out = Out((rows, M), DT[out_dtype])
    q.qmoe_combine(dtype, y, dev(slots), dev(w), rows, top, M, out_dtype, out.t)
    want, mag = ref.combine(y.double().cpu().numpy(), slots, w.astype(np.float64))
    got = out.check()
    e = (top + 1) * 2.0 ** -24 * mag
    assert np.all(np.abs(got - want) <= e + rounding(out_dtype, np.abs(want) + e))


def test_combine_nan_weights_and_dropped_rows():
    y = torch.full((8, 16), float("nan"), device="cuda")
    y[2] = 1.0
    slots = dev(np.array([[2, -1], [-1, -1], [-1, 2], [0, 2]], np.int32))
    w = dev(np.array([[0.5, 0.5], [np.nan, np.nan], [0.0, 2.0], [0.0, 1.0]], np.float32))
    out = torch.empty(4, 16, device="cuda")
    q.qmoe_combine(F32, y, slots, w, 4, 2, 16, F32, out)
    got = out.cpu().numpy()
    assert (got[0] == 0.5).all() and np.isnan(got[1]).all() and (got[2] == 2.0).all() and np.isnan(got[3]).all()


def test_combine_rows_behind_four_gib():
    rows, top, M = 300_007, 2, 4096
    y = torch.zeros(rows * top, M, dtype=torch.bfloat16, device="cuda")       # 4.9 GB
    y[-1], y[-2] = 3.0, 5.0
    slots = torch.full((rows, top), -1, dtype=torch.int32, device="cuda")
    slots[-1] = torch.tensor([rows * top - 1, rows * top - 2], dtype=torch.int32)
    w = torch.full((rows, top), 0.5, device="cuda")
    out = torch.empty(rows, M, dtype=torch.bfloat16, device="cuda")
    q.qmoe_combine(BF16, y, slots, w, rows, top, M, BF16, out)
    assert bool((out[-1] == 4.0).all()) and not out[:-1].any()


# ---------------------------------------------------------------------------
# Together
# ---------------------------------------------------------------------------

class Layer:
    """An experts' layer as a decoder runs it, all buffers allocated once."""

    def __init__(self, rows, D, I, E, top, xfmt, dtype, seed):
        self.rows, self.D, self.I, self.E, self.top, self.xfmt, self.dtype = rows, D, I, E, top, xfmt, dtype
        rng = rng_for(50, seed)
        self.router = dev((rng.standard_normal((D, E)) / np.sqrt(D)).astype(np.float32))
        self.up = self.weights(rng, E * 2 * I, D)
        self.down = self.weights(rng, E * D, I)
        P, b = rows * top, lambda *s, t=torch.uint8: torch.empty(*s, dtype=t, device="cuda")
        i32 = torch.int32
        self.h = dev(rng.standard_normal((rows, D)).astype(np.float32)).to(DT[dtype])
        self.ids, self.w = b(rows, top, t=i32), b(rows, top, t=torch.float32)
        self.offsets, self.order, self.slots = b(E + 1, t=i32), b(P, t=i32), b(rows, top, t=i32)
        self.xc, self.xs = b(rows, ref.row_bytes(xfmt, D)), b(rows, ref.pitch(D))
        self.a = torch.zeros(P, I, dtype=torch.bfloat16, device="cuda")
        self.ac, self.as_ = b(P, ref.row_bytes(xfmt, I)), b(P, ref.pitch(I))
        self.y, self.out = torch.zeros(P, D, device="cuda"), torch.empty(rows, D, dtype=DT[dtype], device="cuda")
        ws = max(q.qmoe_plan_workspace_bytes(rows, E, top), q.qmoe_gemm_workspace_bytes(xfmt, 1, rows, E, top, I, D),
                 q.qmoe_gemm_workspace_bytes(xfmt, 0, rows, E, top, D, I))
        self.ws = b(max(ws, 16))

    @staticmethod
    def weights(rng, rows, K):
        w = dev((rng.standard_normal((rows, K)) / np.sqrt(K)).astype(np.float32))
        codes = torch.empty(rows, K // 2, dtype=torch.uint8, device="cuda")
        scales = torch.empty(rows, ref.pitch(K), dtype=torch.uint8, device="cuda")
        q.qmx_quant(F32, w, K, rows, K, E2M1, codes, scales)
        return codes, scales

    def step(self):
        R, D, I, E, top = self.rows, self.D, self.I, self.E, self.top
        logits = self.h.float() @ self.router
        q.qmoe_route(F32, logits, E, R, E, top, 1, self.ids, self.w, self.offsets, self.order, self.slots, self.ws)
        q.qmx_quant(self.dtype, self.h, D, R, D, self.xfmt, self.xc, self.xs)
        q.qmoe_gemm(self.xfmt, self.xc, self.xs, *self.up, self.offsets, self.order, R, E, top, q.QMX_SILU_MUL, BF16, self.a, I, D, self.ws)
        q.qmx_quant(BF16, self.a, I, R * top, I, self.xfmt, self.ac, self.as_)
        q.qmoe_gemm(self.xfmt, self.ac, self.as_, *self.down, self.offsets, None, R, E, top, q.QMX_NONE, F32, self.y, D, I, self.ws)
        q.qmoe_combine(F32, self.y, self.slots, self.w, R, top, D, self.dtype, self.out)
        return logits

    def check(self, logits):
        """Every stage against the 64-bit form of what went into it."""
        n = lambda t: t.cpu().numpy()
        ids, w = ref.route(logits.double().cpu().numpy(), self.top, 1)
        assert np.array_equal(n(self.ids), ids) and np.allclose(n(self.w), w, rtol=1e-5, atol=0)
        offsets, order, slots = ref.plan(ids, self.E)
        assert np.array_equal(n(self.offsets), offsets) and np.array_equal(n(self.order), order) and np.array_equal(n(self.slots), slots)
        xc, xs = ref.quantize(n(self.h.float()), self.xfmt)
        assert np.array_equal(n(self.xc), xc) and np.array_equal(n(self.xs), xs)
        a = n(self.a.float())
        ac, as_ = ref.quantize(a, self.xfmt)
        assert np.array_equal(n(self.ac), ac) and np.array_equal(n(self.as_), as_)
        y = n(self.y)
        for e in range(self.E):
            lo, hi = offsets[e], offsets[e + 1]
            if lo < hi:
                at = order[lo:hi] // self.top
                check_product(a[lo:hi], (xc[at], xs[at]), [n(t[e * 2 * self.I:(e + 1) * 2 * self.I]) for t in self.up], self.xfmt, 1, BF16)
                check_product(y[lo:hi], (ac[lo:hi], as_[lo:hi]), [n(t[e * self.D:(e + 1) * self.D]) for t in self.down], self.xfmt, 0, F32)
        want, mag = ref.combine(y.astype(np.float64), slots, n(self.w).astype(np.float64))
        e = (self.top + 1) * 2.0 ** -24 * mag
        assert np.all(np.abs(n(self.out.float()) - want) <= e + rounding(self.dtype, np.abs(want) + e))


@pytest.mark.parametrize("rows,D,I,E,top,xfmt,dtype", [(1, 256, 128, 16, 4, E4M3, BF16), (37, 288, 160, 12, 3, E2M1, F32), (300, 256, 96, 8, 2, E4M3, F32),
                                                       (520, 128, 192, 4, 2, E2M1, BF16)])
def test_layer(rows, D, I, E, top, xfmt, dtype):
    layer = Layer(rows, D, I, E, top, xfmt, dtype, rows)
    layer.check(layer.step())


def test_layer_on_another_stream_repeats_its_bits():
    layer = Layer(200, 256, 128, 8, 2, E4M3, BF16, 7)
    layer.step()
    torch.cuda.synchronize()
    first = [t.clone() for t in (layer.out, layer.y, layer.a, layer.order)]
    side = torch.cuda.Stream()
    for _ in range(3):
        for t in (layer.out, layer.y, layer.a, layer.order):
            t.zero_()
        layer.ws.fill_(255)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            layer.step()
        torch.cuda.current_stream().wait_stream(side)
        for t, f in zip((layer.out, layer.y, layer.a, layer.order), first):
            assert torch.equal(t, f)


def test_layer_in_a_graph():
    """Captured once and replayed on other activations, with eager work between."""
    layer = Layer(70, 256, 128, 8, 2, E2M1, F32, 8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.step()
    g = torch.Generator(device="cuda").manual_seed(5)
    for i in range(4):
        layer.h.copy_(torch.randn(layer.h.shape, generator=g, device="cuda") * (1 + i))
        layer.ws.fill_(37 * i)
        layer.out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        replayed = layer.out.clone()
        layer.out.zero_()
        logits = layer.step()
        assert torch.equal(replayed, layer.out)
        layer.check(logits)
