"""g / (1 + exp(-g)) * u of the MX products over all of float32's range: gates and
up values that are exact sums, so that only the activation's own roundings count,
with gates so far below zero that the factor alone would vanish, beside up values
so large that the result does not."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import mx_ref as ref
from test_mx_gpu import BF16, E2M1, E4M3, F32, rng_for, run_experts, run_gemm

pytestmark = pytest.mark.gpu

K = 96
# rows, outputs: each kernel (few rows, some tens, tiles), and of few rows one wave and more
SIZES = [(1, 40), (5, 700), (40, 2750), (75, 8200), (150, 850), (300, 2060)]


def operands(rng, N, M, xfmt, kind):
    """(x, w, g, u) with g and u float64 [N][M], exact as float32: of a row's inputs
    only the first of each block is not zero, and they are alike."""
    v = np.array([1.5, 1.0, 0.5])[np.arange(N) % 3]
    table = list(ref.E2M1_VALUES[:8]) if xfmt == E2M1 else list(ref.E4M3_VALUES[:127])
    code = np.array([table.index(t) for t in v], np.uint8)
    x = [np.zeros((N, ref.row_bytes(xfmt, K)), np.uint8), np.full((N, ref.pitch(K)), 127, np.uint8)]
    x[0][:, ::ref.row_bytes(xfmt, 32)] = code[:, None]
    w = [np.zeros((2 * M, K // 2), np.uint8), np.full((2 * M, ref.pitch(K)), 127, np.uint8)]
    # gates: three numbers, of 16, 4 and 1 each
    c = rng.integers(0, 8, (M, 3))
    sign = 8 * (rng.random((M, 1)) < (0.95 if kind != "small" else 0.5)).astype(np.int64)
    w[0][:M, ::16] = np.where(c > 0, c | sign, 0)
    w[1][:M, :3] = [131, 129, 127]
    if kind == "small":                                  # |g| below 12
        w[1][:M, :3] = [128, 126, 124]
    # up: one number of any size
    w[0][M:, 0] = rng.integers(1, 8, M) | 8 * rng.integers(0, 2, M)
    size = {"large": (90, 125), "any": (-100, 125), "small": (-100, 100)}[kind]
    w[1][M:, 0] = 127 + rng.integers(*size, M)
    wv = ref.values(*w, E2M1)
    g, u = v[:, None] * wv[:M].sum(1), v[:, None] * wv[M:].sum(1)
    assert np.array_equal(g, g.astype(np.float32)) and np.array_equal(u, u.astype(np.float32))
    return x, w, g, u


def factor(g):
    """g / (1 + exp(-g)) in 64 bits."""
    t = np.exp(-np.abs(g))
    return np.where(g < 0, g * t / (1 + t), g / (1 + t))


def close(got, want, e):
    """|error| at most e; beyond float32's range (or its border) the infinity."""
    top = float(np.finfo(np.float32).max)
    with np.errstate(invalid="ignore"):
        ok = np.abs(got - want) <= e
    ok |= (np.abs(want) + e > top) & (np.isinf(got) | (np.abs(got) >= top * (1 - 2.0 ** -8))) & (np.sign(got) == np.sign(want))
    return ok


@pytest.mark.parametrize("kind", ["large", "any", "small"])
@pytest.mark.parametrize("xfmt", [E2M1, E4M3])
@pytest.mark.parametrize("N,M", SIZES)
def test_silu_float32(N, M, xfmt, kind):
    rng = rng_for(70, N, M, xfmt, len(kind))
    x, w, g, u = operands(rng, N, M, xfmt, kind)
    want = factor(g) * u
    if kind == "large" and M > 500:
        assert ((g < -44.5) & (np.abs(want) > 1e-30)).any() and ((g < -132) & (np.abs(want) > 1e-37)).any()
    # 8 roundings; what is subnormal is rounded to a multiple of 2^-149
    e = 8 * 2.0 ** -24 * np.abs(want) + 2.0 ** -149
    assert close(run_gemm(x, w, xfmt, M, K, N, 1, F32), want, e).all()


@pytest.mark.parametrize("kind", ["large", "any", "small"])
@pytest.mark.parametrize("xfmt", [E2M1, E4M3])
@pytest.mark.parametrize("N,M", SIZES)
def test_silu_bfloat16(N, M, xfmt, kind):
    rng = rng_for(72, N, M, xfmt, len(kind))
    x, w, g, u = operands(rng, N, M, xfmt, kind)
    want = factor(g) * u
    if kind == "large" and M > 500:
        assert ((g < -89) & (np.abs(want) > 1e-30)).any() and ((g < -132) & (np.abs(want) > 1e-37)).any()
    # g and u take one factor y = 1 / sqrt(1 + w^2), w = exp(-g / 2), each. The argument of
    # w = 2^a, a = -g log2(e) / 2 - 63 (w is held 2^63 smaller), is rounded, 2^-24 of up to
    # 0.72 |g| + 63, and so is the constant: (|g| + 44) 2^-24 of w, twice that of the result;
    # exponential and root a unit (2^-23) each and twice, 1 + w^2, and three products half a unit:
    # 50 units in all. y is no longer a normal number below g = -174, and 0 below -176, where
    # |g / (1 + exp(-g))| < 177 exp(-176) < 2^-246. Then the output's rounding, to a
    # multiple of 2^-133 at least.
    e = np.abs(want) * (np.abs(g) + 50) * 2.0 ** -23 + 2.0 ** -246 * np.abs(u) + 2.0 ** -149
    e = e + 2.0 ** -8 * (np.abs(want) + e) + 2.0 ** -134
    assert close(run_gemm(x, w, xfmt, M, K, N, 1, BF16), want, e).all()


@pytest.mark.parametrize("rows,experts,top,M", [(3, 4, 2, 130), (200, 8, 2, 700), (500, 4, 1, 1500)])
@pytest.mark.parametrize("xfmt", [E2M1, E4M3])
def test_silu_float32_of_experts(rows, experts, top, M, xfmt):
    rng = rng_for(71, rows, M, xfmt)
    ids = np.stack([rng.permutation(experts)[:top] for _ in range(rows)]).astype(np.int32)
    offsets, order, _ = ref.plan(ids, experts)
    x, w, g, u = operands(rng, rows, M * experts, xfmt, "large")
    # each expert's gate and up rows one behind the other
    w = [np.concatenate([t[:M * experts].reshape(experts, M, -1), t[M * experts:].reshape(experts, M, -1)], 1).reshape(2 * M * experts, -1) for t in w]
    got, _ = run_experts(x, w, xfmt, offsets, order, rows, experts, top, 1, F32, M, K)
    want = (factor(g) * u).reshape(rows, experts, M)[order // top, np.repeat(np.arange(experts), np.diff(offsets))]
    assert close(got, want, 8 * 2.0 ** -24 * np.abs(want) + 2.0 ** -149).all()


def test_silu_of_infinite_and_nan_sums():
    """Sums past float32's range: an infinite gate gives up, or NaN below zero."""
    for N, M in SIZES:
        for xfmt in (E2M1, E4M3):
            x = [np.zeros((N, ref.row_bytes(xfmt, K)), np.uint8), np.full((N, ref.pitch(K)), 127, np.uint8)]
            x[0][:, 0], x[1][:, 0] = (7 if xfmt == E2M1 else 0x7E), 254
            w = [np.zeros((2 * M, K // 2), np.uint8), np.full((2 * M, ref.pitch(K)), 127, np.uint8)]
            w[0][:M, 0], w[1][:M, 0] = np.where(np.arange(M) % 2, 7, 15), 200
            w[0][M:, 0], w[1][M:, 0] = 2, 60
            for dtype in (F32, BF16):
                got = run_gemm(x, w, xfmt, M, K, N, 1, dtype)
                assert (got[:, 1::2] == np.inf).all() and np.isnan(got[:, 0::2]).all()
