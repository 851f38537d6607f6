"""GPU tests of the serving-step operators at the edges of their contents and
sizes: row starts out of order, requests cut off by the call's row count, value
scales far apart, page numbers past 32-bit slots, interleaved read-back.
References and bounds are those of test_serve_gpu.py."""
import numpy as np
import pytest

import gemm_qgemv_amd as q
import serve_ref as ref
from test_serve_gpu import AttnCase, Guarded, dev, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available(), "these tests need the GPU"
    return t


# --- row starts --------------------------------------------------------------------

@pytest.mark.parametrize("cu", [[50, 100, 0, 0], [100, 0, 50, 100], [0, 100, 30, 40], [90, 80, 70, 3], [-7, 300, 20, 60]])
@pytest.mark.parametrize("G,D,kv", [(3, 64, 60), (24, 128, 60), (3, 64, 1500)])
@pytest.mark.parametrize("max_q", [1, 50])
def test_attention_row_starts_out_of_order(torch, cu, G, D, kv, max_q):
    """No place outside the rows is written (the guard bands and the gaps of a
    head's width between the rows are looked at by run), and rows before the
    least and behind the last start stay as they were."""
    say("row starts", cu, G, D, kv, max_q)
    c = AttnCase(torch, "f32", 1, G, D, 16, [(kv, 50), (40, 50), (30, 0)], pad=D)
    c.cu = np.array(cu, np.int32)
    out, lse = c.run(max_q=max_q)
    inside = [min(max(s, 0), c.total) for s in cu]
    for lo, hi in ((0, min(inside)), (max(inside), c.total)):
        assert np.all(out[lo:hi] == 77) and np.all(lse[lo:hi] == 77)
