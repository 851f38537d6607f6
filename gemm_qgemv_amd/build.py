"""Build libqg.so (the HIP kernels and the C ABI) for gfx950 with hipcc.

Run ``python -m gemm_qgemv_amd.build``; ``__graft_entry__.build()`` calls
``build()``. The library is written next to this file and loaded from there.
"""
from __future__ import annotations

import os
import re
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
# the low-bit products, and the serving-step operators
SOURCES = [os.path.join(HERE, "csrc", "qg.hip"), os.path.join(HERE, "serve", "kv.hip"),
           os.path.join(HERE, "serve", "attn.hip"), os.path.join(HERE, "serve", "logprobs.hip")]
OUT = os.path.join(HERE, "libqg.so")
PROBE_SRC = os.path.join(HERE, "csrc", "probe.hip")
PROBE_OUT = os.path.join(HERE, "libqgprobe.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-Wall",
    # IEEE float32: no fast-math, fp32 denormals kept
    "-fno-fast-math",
    "-fno-gpu-flush-denormals-to-zero",
    # no packed-FP32 instructions (plain float code only)
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # what each kernel takes, for the check below
    "-Rpass-analysis=kernel-resource-usage",
    "-I", os.path.join(ROOT, "include"),
]


def build(out: str = OUT, extra: list[str] | None = None, verbose: bool = False) -> str:
    """Build libqg.so and the measurement-only libqgprobe.so. Sources are
    compiled side by side."""
    with tempfile.TemporaryDirectory() as tmp:
        objects = [os.path.join(tmp, f"{i}.o") for i in range(len(SOURCES))]
        jobs = [(["-c", src], obj) for src, obj in zip(SOURCES, objects)]
        jobs.append((["-shared", PROBE_SRC], PROBE_OUT))
        with ThreadPoolExecutor(max_workers=len(jobs)) as pool:
            for done in [pool.submit(_hipcc, what, to, extra, verbose) for what, to in jobs]:
                done.result()
        return _hipcc(["-shared", *objects], out, extra, verbose)


def _hipcc(what: list[str], out: str, extra: list[str] | None, verbose: bool) -> str:
    tmp = out + ".tmp"
    cmd = [HIPCC, *FLAGS, *(extra or []), *what, "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"hipcc failed to build {os.path.basename(out)}")
    spills = spilling(res.stderr)
    if spills:
        raise RuntimeError(f"kernels of {' '.join(what)} keep registers in scratch memory: {', '.join(spills)}")
    errs = [l for l in res.stderr.splitlines()
            if "warning" in l and "packed-fp32-ops" not in l]
    if errs and verbose:
        sys.stderr.write("\n".join(errs) + "\n")
    os.replace(tmp, out)
    return out


def spilling(remarks: str) -> list[str]:
    """Names of the kernels that the compiler's resource remarks say spill
    vector registers or use scratch memory: none may (a variant of the attention
    kernels that spilled heavily was once seen to give wrong results, and a spill
    in a loop over tiles costs more than what it makes room for)."""
    names = []
    for kernel in re.split(r"remark:\s+Function Name: ", remarks)[1:]:
        numbers = re.findall(r"(?:VGPRs Spill|ScratchSize \[bytes/lane\]): (\d+)", kernel)
        if any(int(n) for n in numbers):
            names.append(kernel.split()[0])
    return names


if __name__ == "__main__":
    print(build(verbose=True))
