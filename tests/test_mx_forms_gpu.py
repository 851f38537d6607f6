"""The MX products in every form of every kernel: both kinds of rows, with and
without the activation, both output types, and of experts rows gathered and in the
plan's order, against 64 bits. Sizes are chosen for the kernel that they take; experts
differ in their rows, one has none, and some pairs have no expert."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import gemm_qgemv_amd as q
import mx_ref as ref
from test_mx_gpu import BF16, E2M1, E4M3, F32, operand, rng_for, run_experts, run_gemm
from test_mx_kinds_gpu import check_wide

pytestmark = pytest.mark.gpu


def uneven(rng, rows, experts, top):
    """Experts of each row: some liked more, the one before the last not at all."""
    like = rng.standard_normal(experts) * 0.4
    like[experts - 2] = -1e9
    ids = np.argsort(-(rng.standard_normal((rows, experts)) + like), axis=1)[:, :top].astype(np.int32)
    ids[rng.random((rows, top)) < 0.02] = -1
    return ids


def check(rows, experts, top, wide, K, xfmt, silu, dtype, gather, seed):
    rng = rng_for(90, rows, experts, wide, K, xfmt, silu, dtype, gather, seed)
    M = wide // (1 + silu)
    ids = uneven(rng, rows, experts, top)
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


FORMS = [(xfmt, silu, dtype, gather) for xfmt in (E2M1, E4M3) for silu in (0, 1) for dtype in (F32, BF16) for gather in (0, 1)]
form = pytest.mark.parametrize("xfmt,silu,dtype,gather", FORMS)

# Few rows an expert. K: one, two and four waves share it, and ends of every length; wide:
# one block of outputs a wave, and (without the activation) two
FEW = [(5, 24, 4, wide, K) for wide in (198, 1300) for K in (32, 160, 512, 544, 992, 1024, 1056, 1568, 2048)]
FEW += [(1, 24, 8, 1030, 2048), (40, 24, 4, 510, 1056), (9, 20, 3, 2046, 544)]


@form
@pytest.mark.parametrize("rows,experts,top,wide,K", FEW)
def test_few_rows_an_expert(rows, experts, top, wide, K, xfmt, silu, dtype, gather):
    check(rows, experts, top, wide, K, xfmt, silu, dtype, gather, 0)


# Some tens of rows an expert: 64 weight rows a workgroup and 2, 4, 6 blocks of 16 rows,
# then 128 weight rows and 2, 4, 5 (e4m3) or 6 (e2m1)
MID = [(120, 8, 2, 798, 544), (240, 8, 2, 1022, 288), (360, 8, 2, 766, 1056), (120, 8, 2, 1402, 288), (240, 8, 2, 1398, 1056), (320, 8, 2, 1402, 544),
       (320, 8, 2, 1278, 96), (500, 20, 1, 1410, 416)]


@form
@pytest.mark.parametrize("rows,experts,top,wide,K", MID)
def test_some_tens_of_rows_an_expert(rows, experts, top, wide, K, xfmt, silu, dtype, gather):
    assert q.qmoe_gemm_workspace_bytes(xfmt, silu, rows, experts, top, wide // (1 + silu), K) == 0
    check(rows, experts, top, wide, K, xfmt, silu, dtype, gather, 1)


# Tiles of 64, 128 (of e2m1 rows) and 256 weight rows
TILES = [(500, 8, 2, 302, 544), (500, 8, 2, 1154, 96), (1000, 8, 2, 1702, 288), (1000, 8, 2, 1698, 1056), (2000, 8, 2, 2702, 160), (2000, 8, 2, 2698, 800)]


@form
@pytest.mark.parametrize("rows,experts,top,wide,K", TILES)
def test_tiles_of_experts(rows, experts, top, wide, K, xfmt, silu, dtype, gather):
    assert q.qmoe_gemm_workspace_bytes(xfmt, silu, rows, experts, top, wide // (1 + silu), K) > 0
    check(rows, experts, top, wide, K, xfmt, silu, dtype, gather, 2)


@pytest.mark.parametrize("rows,experts,top,wide,K,xfmt,silu,dtype,gather", [
    (1, 128, 8, 2048, 2048, E4M3, 1, F32, 1), (64, 128, 8, 2048, 1024, E4M3, 0, F32, 0), (64, 128, 8, 2048, 2048, E2M1, 1, BF16, 1)])
def test_decode_steps(rows, experts, top, wide, K, xfmt, silu, dtype, gather):
    check(rows, experts, top, wide, K, xfmt, silu, dtype, gather, 3)


# Products without experts: few rows (one block of outputs a wave and two; one, two and four
# waves that share K), some tens (64 weight rows a workgroup and 2, 4, 6 blocks of 16 rows,
# then 128 and 2, 4, 5 or 6), tiles of 64, 128 (of e2m1 rows) and 256
PRODUCTS = [(5, 198, 512), (5, 198, 544), (5, 198, 1056), (16, 16390, 96), (16, 16390, 544), (13, 16390, 1056), (17, 8210, 544), (33, 5480, 288),
            (65, 3290, 544), (17, 16450, 288), (64, 16386, 160), (77, 16400, 544), (90, 16386, 288), (97, 2400, 544), (700, 6146, 288), (2000, 8102, 288)]


@pytest.mark.parametrize("N,wide,K", PRODUCTS)
@pytest.mark.parametrize("xfmt", [E2M1, E4M3])
@pytest.mark.parametrize("silu", [0, 1])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_products(N, wide, K, xfmt, silu, dtype):
    rng = rng_for(91, N, wide, K, xfmt, silu, dtype)
    M = wide // (1 + silu)
    x, w = operand(rng, N, K, xfmt), operand(rng, M * (1 + silu), K, E2M1)
    if silu:
        x[1][:] -= 8
    check_wide(run_gemm(x, w, xfmt, M, K, N, silu, dtype), x, w, xfmt, silu, dtype)
