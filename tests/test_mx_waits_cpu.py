"""The counted waits of the MX products for some tens of rows, in the code that the
compiler makes of them: loads come in order, so a wait for all but the last n of them
is one for x only if every stage asks for x (loads to LDS) before its weights and
their scales (loads to registers). Compiled as the library is, and with a scheduler
that puts the loads to registers first wherever it may."""
import os
import re
import subprocess

import pytest

from gemm_qgemv_amd import build

KERNELS = ["4, float, false, true, 2, 4", "4, float, true, false, 4, 6", "0, uint16_t, true, false, 4, 5", "0, float, false, true, 2, 2"]


def stages(body):
    """What a kernel's code does between its barriers: ((n of the wait before the
    barrier, or None), loads in order: L to LDS, r to registers)."""
    out, wait = [(None, "")], None
    for line in body.splitlines():
        t = line.strip()
        m = re.match(r"s_waitcnt vmcnt\((\d+)\) lgkmcnt\(0\)$", t)
        if m:
            wait = int(m.group(1))
        elif t.startswith("s_barrier"):
            out.append((wait, ""))
        elif t.startswith("buffer_load"):
            out[-1] = out[-1][0], out[-1][1] + ("L" if re.search(r"\blds\b", t) else "r")
    return out


@pytest.fixture(scope="module")
def source(tmp_path_factory):
    path = tmp_path_factory.mktemp("mid") / "mid.hip"
    here = os.path.join(build.HERE, "mx")
    path.write_text("".join(f'#include "{here}/{name}"\n' for name in ("mx_host.hpp", "mx_mid.hpp")) +
                    "".join(f"template __global__ void qg::mx_mid_kernel<{k}>(qg::MxGemmParams);\n" for k in KERNELS))
    return path


@pytest.mark.parametrize("scheduler", [[], ["-mllvm", "-misched=gcn-max-ilp"]])
def test_every_stage_asks_for_x_first(source, scheduler, tmp_path):
    out = tmp_path / "mid.s"
    res = subprocess.run([build.HIPCC, *build.FLAGS, *scheduler, "--cuda-device-only", "-S", str(source), "-o", str(out)],
                         capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-2000:]
    bodies = re.findall(r"^_ZN2qg13mx_mid_kernel\S*:.*?\n(.*?)s_endpgm", out.read_text(), re.S | re.M)
    assert len(bodies) == len(KERNELS)
    for body in bodies:
        code = stages(body)
        assert all(re.fullmatch("L*r*", loads) for _, loads in code), code
        # the loop's four stages: the wait before each lets the loads pass that were
        # asked for behind x's of the stage two before, and no more
        at = next(i for i in range(len(code) - 3) if all("L" in loads and "r" in loads for _, loads in code[i:i + 4]) and i > 0)
        loop = code[at:at + 4]
        for i, (wait, _) in enumerate(loop):
            assert wait == len(loop[i - 1][1]) + loop[i - 2][1].count("r"), (i, loop)
