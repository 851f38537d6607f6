"""Arguments of the binding and of the entry points at their edges; no call
here reaches a GPU (see test_serve_abi_cpu.py)."""
import ctypes

import numpy as np
import pytest

import gemm_qgemv_amd as q
from test_serve_abi_cpu import LP, PLAN, at, cache


@pytest.mark.parametrize("host", [b"abc", "abc", bytearray(64), (ctypes.c_float * 16)(), np.zeros(16, np.float32), 1.5, [1, 2]])
def test_only_tensors_and_addresses_are_taken_as_device_memory(host):
    """What has no device pointer is refused; ctypes would pass the host
    address of some of these on."""
    c = cache()
    calls = [(q.qgemv, (q.QG_U4_G64, host, at(1), at(2), at(3), at(4), 64, 64, 1)),
             (q.qgemm, (q.QG_I8_ROW, at(1), at(2), None, host, at(4), 64, 64, 1)),
             (q.qgemv_argmax_noalloc, (q.QG_U4_G64, at(1), at(2), at(3), host, None, at(5), 64, 64, 1)),
             (q.qembed, (q.QG_U4_G64, at(1), at(2), at(3), host, at(4), 64, 64, 1)),
             (q.qkv_append, (q.QG_F32, host, 128, at(2), 128, at(3), 4, c)),
             (q.qkv_read, (q.QG_F32, c, at(3), 4, at(1), 128, host, 128))]
    for fn, args in calls:
        with pytest.raises(TypeError):
            fn(*args, stream=0)
    with pytest.raises(TypeError):
        q.qkv_plan(**dict(PLAN, slots=host), stream=0)
    with pytest.raises(TypeError):
        q.qlogprobs(**dict(LP, logits=host), stream=0)
    with pytest.raises(TypeError):
        q.KVCache(host, 8, 16, 2, 64)


def test_attention_launches_that_no_grid_holds():
    """2^24 workgroups of 256 threads are more than a launch takes."""
    from test_serve_abi_cpu import attn_err
    c = cache(pages=4, heads=257)
    most = (2 ** 24 - 1) // 257                     # requests; one workgroup a request and head
    a = dict(cache=c, q_heads=257, q_stride=257 * 64, out_stride=257 * 64, total_q=1, max_q=1, max_kv=16)
    assert attn_err(**a, batch=most + 1) == q.QG_ERR_SHAPE
    assert q.qkv_attn_workspace_bytes(c, most + 1, 1, 1, 16, 257) == 0
    # one fewer is looked at further
    assert attn_err(**dict(a, out=at(1)), batch=most) == q.QG_ERR_ALIAS


def test_rows_that_touch_each_other_are_refused():
    """Rows of one wider buffer: side by side is accepted (see the GPU tests),
    shared elements are not."""
    from test_serve_abi_cpu import ATTN, err
    c = cache()
    rd = dict(dtype=q.QG_F32, cache=c, slots=at(3), n=4, k=at(1), k_stride=256, v=at(1) + 512, v_stride=256)
    for kw in (dict(v=at(1) + 496), dict(v=at(1) + 528), dict(v=at(1) + 512, v_stride=260), dict(v=at(1)), dict(v=at(1) + 1024),
               dict(v=at(1) - 496), dict(k_stride=128, v_stride=128)):
        assert err(q.qkv_read, **dict(rd, **kw)) == q.QG_ERR_ALIAS, kw
    at_once = dict(ATTN, cache=c, q=at(1), q_stride=512, out_stride=512)
    for out in (at(1) + 1008, at(1) + 1040, at(1), at(1) + 2048):
        assert err(q.qkv_attn, **dict(at_once, out=out)) == q.QG_ERR_ALIAS, out


def test_cache_memory_is_one_piece():
    """A strided view has enough elements, but they do not lie where the
    kernels look for them."""
    import torch
    n = q.qkv_cache_bytes(cache(data=None))
    wide = torch.zeros(2 * n, dtype=torch.uint8)
    with pytest.raises(ValueError):
        q.KVCache(wide[::2], 8, 16, 2, 64)
    with pytest.raises(ValueError):
        q.KVCache(wide.view(2, n).t(), 8, 16, 2, 64)
    assert q.KVCache(wide[n:], 8, 16, 2, 64).data.numel() == n
    assert q.KVCache(wide.view(2, n), 8, 16, 2, 64).num_pages == 8


def test_the_build_refuses_kernels_that_spill():
    from gemm_qgemv_amd import build

    def remarks(name, spilled, scratch):
        at = f"serve/x.hpp:62:1: remark: "
        return "".join(f"{at}{t} [-Rpass-analysis=kernel-resource-usage]\n" for t in (
            f"Function Name: {name}", "    TotalSGPRs: 40", "    VGPRs: 168", f"    ScratchSize [bytes/lane]: {scratch}",
            "    Occupancy [waves/SIMD]: 3", "    SGPRs Spill: 2", f"    VGPRs Spill: {spilled}"))
    assert build.spilling(remarks("a", 0, 0) + remarks("b", 0, 0)) == []
    assert build.spilling(remarks("a", 0, 0) + remarks("b", 1, 8) + remarks("c", 0, 16)) == ["b", "c"]
    assert build.spilling("warning: something else\n") == []
