"""Refusals of the MX and experts' entry points: every argument error is found
on the host, before anything is enqueued, so no call here reaches a GPU. And
the reference forms the GPU tests compare with, held to hand-worked values."""
import numpy as np
import pytest

import gemm_qgemv_amd as q
import mx_ref as ref

A = 1 << 20    # fake, 16-byte aligned "device" addresses, far apart, never dereferenced


def at(i):
    return A + (i << 44)


def err(fn, kw, **change):
    with pytest.raises(q.QGError) as e:
        fn(**{**kw, **change}, stream=0)
    return e.value.status


QUANT = dict(dtype=q.QG_F32, x=at(1), x_stride=256, rows=4, K=256, fmt=q.QMX_E2M1, codes=at(2), scales=at(3))
GEMM = dict(xfmt=q.QMX_E2M1, x_codes=at(1), x_scales=at(2), w_codes=at(3), w_scales=at(4), act=q.QMX_NONE, dtype=q.QG_F32,
            y=at(5), M=64, K=256, N=4)
PLAN = dict(ids=at(1), rows=4, experts=8, top=2, offsets=at(2), order=at(3), slots=at(4))
ROUTE = dict(dtype=q.QG_F32, logits=at(5), ld=8, rows=4, experts=8, top=2, renorm=1, ids=at(1), weights=at(6), offsets=at(2),
             order=at(3), slots=at(4))
MOE = dict(xfmt=q.QMX_E2M1, x_codes=at(1), x_scales=at(2), w_codes=at(3), w_scales=at(4), offsets=at(6), order=at(7), rows=4,
           experts=8, top=2, act=q.QMX_NONE, dtype=q.QG_F32, y=at(5), M=64, K=256)
COMBINE = dict(dtype=q.QG_F32, y=at(1), slots=at(2), weights=at(3), rows=4, top=2, M=64, out_dtype=q.QG_F32, out=at(4))


@pytest.mark.parametrize("change,status", [
    (dict(x=None), q.QG_ERR_NULL), (dict(codes=None), q.QG_ERR_NULL), (dict(scales=None), q.QG_ERR_NULL),
    (dict(dtype=3), q.QG_ERR_FORMAT), (dict(dtype=0), q.QG_ERR_FORMAT), (dict(fmt=0), q.QG_ERR_FORMAT), (dict(fmt=3), q.QG_ERR_FORMAT),
    (dict(K=0), q.QG_ERR_SHAPE), (dict(K=16), q.QG_ERR_SHAPE), (dict(K=48), q.QG_ERR_SHAPE),
    (dict(K=q.QMX_MAX_K + 32, x_stride=1 << 22), q.QG_ERR_SHAPE), (dict(rows=-1), q.QG_ERR_SHAPE), (dict(rows=1 << 31), q.QG_ERR_SHAPE),
    (dict(x_stride=252), q.QG_ERR_SHAPE), (dict(x_stride=258), q.QG_ERR_SHAPE), (dict(x_stride=260, dtype=q.QG_BF16), q.QG_ERR_SHAPE),
    (dict(x=at(1) + 8), q.QG_ERR_ALIGN), (dict(codes=at(2) + 8), q.QG_ERR_ALIGN), (dict(scales=at(3) + 2), q.QG_ERR_ALIGN)])
def test_quant_and_dequant_refuse(change, status):
    assert err(q.qmx_quant, QUANT, **change) == status
    assert err(q.qmx_dequant, QUANT, **change) == status


def test_quant_alias():
    assert err(q.qmx_quant, QUANT, codes=at(1)) == q.QG_ERR_ALIAS
    assert err(q.qmx_quant, QUANT, codes=at(1) + 3 * 1024 + 1008) == q.QG_ERR_ALIAS          # the last row's end
    assert err(q.qmx_quant, QUANT, scales=at(2) + 508) == q.QG_ERR_ALIAS
    assert err(q.qmx_dequant, QUANT, x=at(3)) == q.QG_ERR_ALIAS


def test_quant_of_no_rows():
    q.qmx_quant(**{**QUANT, "rows": 0}, stream=0)
    q.qmx_dequant(**{**QUANT, "rows": 0}, stream=0)
    assert err(q.qmx_quant, QUANT, rows=0, x=None) == q.QG_ERR_NULL


def test_scale_pitch():
    for K, want in ((32, 4), (128, 4), (160, 8), (2048, 64), (q.QMX_MAX_K, q.QMX_MAX_K // 32)):
        assert q.qmx_scale_pitch(K) == want == ref.pitch(K)
    for K in (0, -32, 16, 33, q.QMX_MAX_K + 32):
        assert q.qmx_scale_pitch(K) == 0


PRODUCT_ERRORS = [
    (dict(x_codes=None), q.QG_ERR_NULL), (dict(x_scales=None), q.QG_ERR_NULL), (dict(w_codes=None), q.QG_ERR_NULL),
    (dict(w_scales=None), q.QG_ERR_NULL), (dict(y=None), q.QG_ERR_NULL),
    (dict(xfmt=0), q.QG_ERR_FORMAT), (dict(xfmt=3), q.QG_ERR_FORMAT), (dict(act=2), q.QG_ERR_FORMAT), (dict(act=-1), q.QG_ERR_FORMAT),
    (dict(dtype=3), q.QG_ERR_FORMAT),
    (dict(M=0), q.QG_ERR_SHAPE), (dict(M=q.QMX_MAX_M + 1), q.QG_ERR_SHAPE), (dict(K=0), q.QG_ERR_SHAPE), (dict(K=100), q.QG_ERR_SHAPE),
    (dict(K=q.QMX_MAX_K + 32), q.QG_ERR_SHAPE),
    (dict(x_codes=at(1) + 4), q.QG_ERR_ALIGN), (dict(w_codes=at(3) + 8), q.QG_ERR_ALIGN), (dict(y=at(5) + 4), q.QG_ERR_ALIGN),
    (dict(x_scales=at(2) + 1), q.QG_ERR_ALIGN), (dict(w_scales=at(4) + 2), q.QG_ERR_ALIGN),
    (dict(y=at(1)), q.QG_ERR_ALIAS), (dict(y=at(2)), q.QG_ERR_ALIAS), (dict(y=at(3) + 64 * 128 - 16), q.QG_ERR_ALIAS),
    (dict(y=at(4)), q.QG_ERR_ALIAS)]


@pytest.mark.parametrize("change,status", PRODUCT_ERRORS + [(dict(N=-1), q.QG_ERR_SHAPE), (dict(N=1 << 31), q.QG_ERR_SHAPE),
                                                            (dict(N=(1 << 31) - 1, M=1 << 20), q.QG_ERR_SHAPE)])
def test_product_refuses(change, status):
    assert err(q.qmx_gemm, GEMM, **change) == status


def test_silu_weights_are_two_matrices():
    # the second matrix's last bytes
    y = at(3) + 2 * 64 * 128 - 16
    assert err(q.qmx_gemm, GEMM, act=q.QMX_SILU_MUL, y=y) == q.QG_ERR_ALIAS
    assert err(q.qmoe_gemm, MOE, act=q.QMX_SILU_MUL, y=at(3) + 8 * 2 * 64 * 128 - 16) == q.QG_ERR_ALIAS


def test_product_of_no_rows():
    q.qmx_gemm(**{**GEMM, "N": 0}, stream=0)
    q.qmoe_gemm(**{**MOE, "rows": 0}, stream=0)
    q.qmoe_combine(**{**COMBINE, "rows": 0}, stream=0)


@pytest.mark.parametrize("change,status", PRODUCT_ERRORS + [
    (dict(offsets=None), q.QG_ERR_NULL), (dict(offsets=at(6) + 2), q.QG_ERR_ALIGN), (dict(order=at(7) + 1), q.QG_ERR_ALIGN),
    (dict(rows=-1), q.QG_ERR_SHAPE), (dict(rows=1 << 30), q.QG_ERR_SHAPE), (dict(experts=0), q.QG_ERR_SHAPE),
    (dict(experts=q.QMOE_MAX_EXPERTS + 1), q.QG_ERR_SHAPE), (dict(top=0), q.QG_ERR_SHAPE), (dict(top=9), q.QG_ERR_SHAPE),
    (dict(experts=64, top=q.QMOE_MAX_TOP + 1), q.QG_ERR_SHAPE),
    # gathered rows beyond 32-bit offsets
    (dict(rows=1 << 24, K=4096, M=16), q.QG_ERR_SHAPE),
    (dict(y=at(6)), q.QG_ERR_ALIAS), (dict(y=at(7) + 16), q.QG_ERR_ALIAS)])
def test_experts_product_refuses(change, status):
    assert err(q.qmoe_gemm, MOE, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(ids=None), q.QG_ERR_NULL), (dict(offsets=None), q.QG_ERR_NULL), (dict(order=None), q.QG_ERR_NULL), (dict(slots=None), q.QG_ERR_NULL),
    (dict(rows=-1), q.QG_ERR_SHAPE), (dict(rows=1 << 30), q.QG_ERR_SHAPE), (dict(experts=0), q.QG_ERR_SHAPE),
    (dict(experts=1025), q.QG_ERR_SHAPE), (dict(top=0), q.QG_ERR_SHAPE), (dict(top=9), q.QG_ERR_SHAPE),
    (dict(ids=at(1) + 1), q.QG_ERR_ALIGN), (dict(offsets=at(2) + 2), q.QG_ERR_ALIGN), (dict(order=at(3) + 2), q.QG_ERR_ALIGN),
    (dict(slots=at(4) + 2), q.QG_ERR_ALIGN),
    (dict(rows=1 << 20), q.QG_ERR_WORKSPACE), (dict(rows=1 << 20, ws=at(9), ws_bytes=16), q.QG_ERR_WORKSPACE),
    (dict(rows=1 << 20, ws=at(9) + 4, ws_bytes=1 << 30), q.QG_ERR_ALIGN),
    (dict(order=at(2)), q.QG_ERR_ALIAS), (dict(slots=at(3) + 28), q.QG_ERR_ALIAS),
    (dict(rows=1 << 20, ws=at(3), ws_bytes=1 << 30), q.QG_ERR_ALIAS)])
def test_plan_and_route_refuse(change, status):
    assert err(q.qmoe_plan, PLAN, **change) == status
    assert err(q.qmoe_route, ROUTE, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(logits=None), q.QG_ERR_NULL), (dict(weights=None), q.QG_ERR_NULL), (dict(dtype=0), q.QG_ERR_FORMAT), (dict(ld=7), q.QG_ERR_SHAPE),
    (dict(renorm=2), q.QG_ERR_SHAPE), (dict(logits=at(5) + 2), q.QG_ERR_ALIGN), (dict(logits=at(5) + 1, dtype=q.QG_BF16), q.QG_ERR_ALIGN),
    (dict(weights=at(6) + 2), q.QG_ERR_ALIGN), (dict(weights=at(1)), q.QG_ERR_ALIAS), (dict(ids=at(5) + 124), q.QG_ERR_ALIAS),
    (dict(weights=at(2) + 32), q.QG_ERR_ALIAS)])
def test_route_refuses(change, status):
    assert err(q.qmoe_route, ROUTE, **change) == status


def test_plan_alias_with_ids():
    assert err(q.qmoe_plan, PLAN, slots=at(1)) == q.QG_ERR_ALIAS


@pytest.mark.parametrize("change,status", [
    (dict(y=None), q.QG_ERR_NULL), (dict(slots=None), q.QG_ERR_NULL), (dict(weights=None), q.QG_ERR_NULL), (dict(out=None), q.QG_ERR_NULL),
    (dict(dtype=0), q.QG_ERR_FORMAT), (dict(out_dtype=3), q.QG_ERR_FORMAT), (dict(rows=-1), q.QG_ERR_SHAPE), (dict(rows=1 << 30), q.QG_ERR_SHAPE),
    (dict(top=0), q.QG_ERR_SHAPE), (dict(top=33), q.QG_ERR_SHAPE), (dict(M=0), q.QG_ERR_SHAPE), (dict(M=q.QMX_MAX_M + 1), q.QG_ERR_SHAPE),
    (dict(y=at(1) + 8), q.QG_ERR_ALIGN), (dict(out=at(4) + 8), q.QG_ERR_ALIGN), (dict(slots=at(2) + 1), q.QG_ERR_ALIGN),
    (dict(weights=at(3) + 1), q.QG_ERR_ALIGN), (dict(out=at(1) + 7 * 256), q.QG_ERR_ALIAS), (dict(out=at(2)), q.QG_ERR_ALIAS),
    (dict(out=at(3) + 16), q.QG_ERR_ALIAS)])
def test_combine_refuses(change, status):
    assert err(q.qmoe_combine, COMBINE, **change) == status


def test_workspace_sizes():
    for fn, good in ((q.qmoe_plan_workspace_bytes, (100, 8, 2)),):
        assert fn(*good) == 0
    assert q.qmoe_plan_workspace_bytes(1 << 20, 256, 8) > 0
    for bad in ((-1, 8, 2), (4, 0, 2), (4, 8, 9), (1 << 30, 8, 2)):
        assert q.qmoe_plan_workspace_bytes(*bad) == 0
    assert q.qmx_gemm_workspace_bytes(9, 0, 64, 256, 4) == 0
    assert q.qmx_gemm_workspace_bytes(q.QMX_E2M1, 0, 64, 100, 4) == 0
    assert q.qmoe_gemm_workspace_bytes(q.QMX_E2M1, 0, 4, 0, 2, 64, 256) == 0


LARGE = dict(M=4096, K=256, N=4096)
FAR = 1 << 40


def test_products_in_tiles_need_a_workspace():
    for xfmt in (q.QMX_E2M1, q.QMX_E4M3):
        for act in (q.QMX_NONE, q.QMX_SILU_MUL):
            need = q.qmx_gemm_workspace_bytes(xfmt, act, 4096, 256, 4096)
            assert need >= (4096 * (1 + act) + 4096) * 8        # both operands' scales
            call = dict(xfmt=xfmt, act=act, **LARGE)
            for status, more in ((q.QG_ERR_WORKSPACE, dict(ws=None, ws_bytes=need)), (q.QG_ERR_WORKSPACE, dict(ws=FAR, ws_bytes=need - 1)),
                                 (q.QG_ERR_ALIGN, dict(ws=FAR + 4, ws_bytes=need))):
                assert err(q.qmx_gemm, GEMM, **call, **more) == status
            # apart from each other, and then the workspace over each of them
            apart = dict(x_codes=FAR, x_scales=FAR + (1 << 28), w_codes=FAR + (2 << 28), w_scales=FAR + (3 << 28), y=FAR + (4 << 28))
            for name in apart:
                assert err(q.qmx_gemm, GEMM, **{**call, **apart}, ws=apart[name], ws_bytes=need) == q.QG_ERR_ALIAS


def test_experts_in_tiles_need_a_workspace():
    need = q.qmoe_gemm_workspace_bytes(q.QMX_E2M1, 0, 2048, 8, 2, 4096, 256)
    assert need >= (8 * 4096 + 4096) * 8 + 4096 * 4             # scales, and where the sorted rows begin
    call = dict(xfmt=q.QMX_E2M1, act=0, rows=2048, experts=8, top=2, M=4096, K=256)
    for status, more in ((q.QG_ERR_WORKSPACE, dict(ws=None, ws_bytes=need)), (q.QG_ERR_WORKSPACE, dict(ws=FAR, ws_bytes=need - 1)),
                         (q.QG_ERR_ALIGN, dict(ws=FAR + 8, ws_bytes=need))):
        assert err(q.qmoe_gemm, MOE, **call, **more) == status
    apart = {name: FAR + (i << 28) for i, name in enumerate(("x_codes", "x_scales", "w_codes", "w_scales", "y", "offsets", "order"))}
    for name in apart:
        assert err(q.qmoe_gemm, MOE, **call, **apart, ws=apart[name], ws_bytes=need) == q.QG_ERR_ALIAS


# ---- the reference forms --------------------------------------------------

def test_reference_quantizer_by_hand():
    # largest magnitude 7 = 1.75 * 2^2: scale 2^0; 5 and 0.25 are ties, 6.5 and 7 beyond the largest
    x = np.zeros((1, 32), np.float32)
    x[0, :8] = [7, -5, 0.25, 0.75, -0.3, 6.5, 2.4, -0.0]
    codes, scales = ref.quantize(x, ref.E2M1)
    assert list(scales[0]) == [127, 0, 0, 0]
    assert list(ref.unpack(codes, ref.E2M1)[0, :8]) == [6, -4, 0, 1, -0.5, 6, 2, 0]
    assert codes[0, 3] >> 4 == 8                        # -0 keeps its sign
    codes, scales = ref.quantize(x, ref.E4M3)
    assert scales[0, 0] == 127 + 2 - 8
    assert ref.values(codes, scales, ref.E4M3)[0, 0] == 7.0
    # 2^-6 of the largest: 0.25 is exact there
    assert ref.values(codes, scales, ref.E4M3)[0, 2] == 0.25


def test_reference_quantizer_edges():
    x = np.zeros((3, 32), np.float32)
    x[0, 5] = np.float32(2.0 ** -149)
    x[1, 3] = np.float32(3.4e38)
    x[2, 0] = np.nan
    for fmt, emax in ((ref.E2M1, 2), (ref.E4M3, 8)):
        codes, scales = ref.quantize(x, fmt)
        assert list(scales[:, 0]) == [0, 254 - emax, 255]
        assert not codes[0].any() and not codes[2].any()


def test_reference_e4m3_table():
    assert ref.E4M3_VALUES[0x7e] == 448 and ref.E4M3_VALUES[1] == 2.0 ** -9 and np.isnan(ref.E4M3_VALUES[0xff])
    assert ref.E4M3_VALUES[0x38] == 1.0


def test_reference_plan_by_hand():
    ids = np.array([[2, 0], [-1, 2], [0, 7]], np.int32)
    offsets, order, slots = ref.plan(ids, 3)
    assert list(offsets) == [0, 2, 2, 4]
    assert list(order) == [1, 4, 0, 3, -1, -1]
    assert slots.tolist() == [[2, 0], [-1, 3], [1, -1]]


def test_reference_route_by_hand():
    x = np.array([[1.0, 3.0, 3.0, -np.inf], [-np.inf] * 4, [0.0, np.nan, 1.0, 2.0]])
    ids, w = ref.route(x, 3, 1)
    assert ids.tolist() == [[1, 2, 0], [-1, -1, -1], [-1, -1, -1]]
    e = np.exp(-2.0)
    assert np.allclose(w[0], [1 / (2 + e), 1 / (2 + e), e / (2 + e)]) and not w[1].any() and np.isnan(w[2]).all()
