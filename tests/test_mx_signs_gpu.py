"""Signs of what the MX rows stand for: of zeros, and of numbers that vanish."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import gemm_qgemv_amd as q
import mx_ref as ref
from test_mx_gpu import BF16, DT, E2M1, E4M3, F32, Out, dev, run_quant

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [E2M1, E4M3])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_dequant_keeps_signs(fmt, dtype):
    """Every code at every scale but NaN's: equal bit by bit where it is a number."""
    K = 512
    scales = np.repeat(np.arange(255, dtype=np.uint8)[:, None], ref.pitch(K), axis=1)
    codes = np.tile(np.arange(ref.row_bytes(fmt, K)).astype(np.uint8), (255, 1))
    x = Out((255, K), DT[dtype])
    q.qmx_dequant(fmt, dev(codes), dev(scales), 255, K, dtype, x.t, K)
    got = x.check()
    with np.errstate(over="ignore"):
        want = torch.from_numpy(ref.values(codes, scales, fmt).astype(np.float32)).to(DT[dtype]).float().numpy()
    number = ~np.isnan(want)
    assert np.array_equal(np.isnan(got), ~number) and number.any()
    assert np.array_equal(got[number].view(np.uint32), want[number].view(np.uint32))
    assert (np.signbit(want) & (want == 0)).any() and (~np.signbit(want) & (want == 0)).any()


@pytest.mark.parametrize("fmt", [E2M1, E4M3])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_signs_there_and_back(fmt, dtype):
    """Zeros, and numbers that become zero at their block's scale, keep their signs."""
    K = 96
    x = np.zeros((4, K), np.float32)
    x[:, ::2] = -0.0
    x[1, 0::32] = 1024.0
    x[2] = np.where(np.arange(K) % 2, 1e-30, -1e-30)
    x[2, 0::32] = 1024.0
    x[3] = np.where(np.arange(K) % 2, 2.0 ** -133, -2.0 ** -133)     # the smallest number of bf16
    codes, scales, _ = run_quant(x, dtype, fmt)
    back = Out((4, K), torch.float32)
    q.qmx_dequant(fmt, dev(codes), dev(scales), 4, K, F32, back.t, K)
    got, want = back.check(), ref.values(*ref.quantize(x, fmt), fmt).astype(np.float32)
    assert np.array_equal(got.view(np.uint32), want.view(np.uint32))
    assert np.array_equal(np.signbit(got), np.signbit(x))
