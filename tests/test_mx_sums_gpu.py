"""What the MX products' float32 sums are off by at worst: operands made so that as
many products as can be lie just where a sum drops them, and sums at the ends of
float32's range. The bound is the documented one, (K / 8 + 4) 2^-23 of the sum of
magnitudes and K 2^-148.

Its arithmetic: a block of 32 products meets the sum so far (of e4m3 rows those with
|x| >= 4, then the others). Beside a sum of exponent S products below 2^(S - 27) are
dropped, 32 of them at most 2^-22 of it, 2 units of 2^-23; beside larger products the
sum loses less than a unit; each addition rounds, half a unit. So 2.5 units a block,
of e4m3 2 + 1/2 and 1 + 1/2; the sums of waves that share K are less than 4 more. Below
2^-126 a product may lose all of 2^-149, K of them, and the roundings are 2 K / 32
halves of that."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import mx_ref as ref
from test_mx_gpu import E2M1, E4M3, F32, dev, operand, rng_for, run_gemm, wide_values

pytestmark = pytest.mark.gpu

# rows and outputs of each kernel: few rows, some tens, tiles of 64, of 128 (of e2m1
# rows) and of 256
SIZES = [(3, 200), (20, 8210), (75, 16400), (140, 2060), (130, 17000), (1030, 8200)]


def held(got, x, w, xfmt):
    """Errors in units of the bound."""
    xv, wv = wide_values(*map(dev, x), xfmt), wide_values(*map(dev, w), E2M1)
    K = xv.shape[1]
    want, a = xv @ wv.T.contiguous(), xv.abs() @ wv.abs().T.contiguous()
    return float(((dev(got).double() - want).abs() / ((K / 8 + 4) * 2.0 ** -23 * a + K * 2.0 ** -148)).max())


def alike(code, rows, K, fmt):
    c = np.broadcast_to(code, (rows, K)).astype(np.uint8)
    return c[:, 0::2] | c[:, 1::2] << 4 if fmt == E2M1 else c


@pytest.mark.parametrize("K", [64, 128, 512, 2048, 8192])
@pytest.mark.parametrize("xfmt", [E2M1, E4M3])
@pytest.mark.parametrize("N,M", SIZES)
def test_sums_beside_one_large_product(N, M, xfmt, K):
    """One product, in the first block or the last, and all others alike, from
    where each counts to where all are dropped."""
    if N * K > 1 << 21:
        K = 1024
    rng = rng_for(80, N, M, xfmt, K)
    blocks = K // 32
    if xfmt == E2M1:
        code = rng.choice([2, 3, 5, 7], (N, 1))
    else:                                                # both parts in turn, or one
        pair = rng.choice([0x38, 0x3F, 0x48, 0x4F, 0x7E], (N, 1)), rng.choice([0x38, 0x3F, 0x47, 0x48, 0x4F], (N, 1))
        code = np.where((np.arange(K) % 2 == 1) & (np.arange(N) % 2 == 1)[:, None], pair[1], pair[0])
    x = [alike(code, N, K, xfmt), np.full((N, ref.pitch(K)), 127, np.uint8)]
    el = np.broadcast_to(rng.choice([2, 3, 5, 7], (M, 1)), (M, K)).astype(np.uint8)
    ws = np.full((M, ref.pitch(K)), 127, np.uint8)
    ws[:, :blocks] = 127 - rng.integers(18, 40, (M, 1))
    for m in range(M):
        b = 0 if m % 2 else blocks - 1
        ws[m, b] = 127
        el[m, 32 * b:32 * b + 32] = 0
        el[m, 32 * b + m % 32] = 2
    w = [alike(el, M, K, E2M1), ws]
    worst = held(run_gemm(x, w, xfmt, M, K, N, 0, F32), x, w, xfmt)
    assert worst <= 1.0
    if K == 8192:
        # (of four waves that share K one has the large product)
        assert worst > 0.05, "the case is one that drops products"


@pytest.mark.parametrize("xfmt", [E2M1, E4M3])
@pytest.mark.parametrize("N,M", SIZES)
def test_sums_of_any_scales(N, M, xfmt):
    """Scales that fall, rise or jump by up to 2^30 from block to block."""
    rng = rng_for(81, N, M, xfmt)
    K = 512
    x, w = operand(rng, N, K, xfmt), operand(rng, M, K, E2M1)
    step = rng.integers(-4, 5, (M, 1)) * np.arange(K // 32)
    jump = rng.integers(0, 31, (M, K // 32))
    w[1][:, :K // 32] = np.clip(np.where(np.arange(M)[:, None] % 2, 127 + step, 100 + jump), 40, 200)
    assert held(run_gemm(x, w, xfmt, M, K, N, 0, F32), x, w, xfmt) <= 1.0


@pytest.mark.parametrize("xfmt", [E2M1, E4M3])
@pytest.mark.parametrize("N,M", SIZES)
def test_sums_at_the_ends_of_the_range(N, M, xfmt):
    rng = rng_for(82, N, M, xfmt)
    K = 512
    x, w = operand(rng, N, K, xfmt), operand(rng, M, K, E2M1)
    w[1][:, :K // 32] = 0
    for byte in (0, 90, 100, 106, 110, 117, 120, 127):       # sums of 2^-240 to 2^-110
        x[1][:, :K // 32] = byte
        assert held(run_gemm(x, w, xfmt, M, K, N, 0, F32), x, w, xfmt) <= 1.0
    w[1][:, :K // 32] = 240                                  # sums of magnitudes up to 2^127
    x[1][:, :K // 32] = 127 + (2 if xfmt == E2M1 else -4)
    got = run_gemm(x, w, xfmt, M, K, N, 0, F32)
    assert np.isfinite(got).all() and np.abs(got).max() > 2.0 ** 120
    assert held(got, x, w, xfmt) <= 1.0
