"""Build libgdn2.so in-tree with hipcc for gfx950.

    python -m gated_delta_rule_83_amd.build        # or build() from Python

Every HIP translation unit is compiled in parallel, then linked into
``gated_delta_rule_83_amd/libgdn2.so`` next to this file. The prefill kernel
template is compiled once per (dtype, d_k) so that its instances build in
parallel.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT = os.path.join(HERE, "libgdn2.so")
OBJDIR = os.path.join(HERE, "_build")

ARCH = "gfx950"
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
# Packed fp32 instructions are kept out of the generated code: hipcc forms
# them from ordinary float code otherwise.
CFLAGS = ["-O3", "-std=c++20", "-fPIC", f"--offload-arch={ARCH}", "-I", INCLUDE, "-I", CSRC,
          "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-Wall", "-Wno-unused-function"]


def _units():
    units = [("gdn2_api.cpp", "api", []), ("gdn2_operators_api.cpp", "operators_api", []),
             ("gdn2_linear.hip", "linear", []), ("gdn2_norm.hip", "norm", []),
             ("gdn2_norm.hip", "norm_backward", ["-DGDN2_NORM_BACKWARD"]), ("gdn2_state_cache.hip", "state_cache", []),
             ("gdn2_decode.hip", "decode", []),
             ("gdn2_prefill.hip", "prefill", []), ("gdn2_noalloc.hip", "noalloc", []),
             ("gdn2_backward_chunk.hip", "backward_chunk", [])]
    for bf in (1, 0):
        units.append(("gdn2_backward.hip", f"backward_{'bf16' if bf else 'f32'}", [f"-DGDN2_BWD_BF16={bf}"]))
    for dt, bf in (("bf16", 1), ("f32", 0)):
        for dk in (16, 32, 64, 128):
            fn = f"launch_prefill_{dt}_dk{dk}"
            units.append(("gdn2_prefill_inst.hip", f"prefill_{dt}_dk{dk}",
                          [f"-DGDN2_INST_DK={dk}", f"-DGDN2_INST_BF16={bf}", f"-DGDN2_INST_FN={fn}"]))
    return units


def _compile(src, tag, defs):
    obj = os.path.join(OBJDIR, tag + ".o")
    cmd = [HIPCC] + CFLAGS + defs
    if src.endswith(".cpp"):
        cmd += ["-x", "hip"]
    cmd += ["-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    # the host pass does not know the packed-fp32 target feature: drop that note
    err = "\n".join(l for l in r.stderr.splitlines() if "packed-fp32-ops" not in l)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src} ({tag}):\n{err}")
    return obj, err


def build(jobs: int = 0, verbose: bool = False) -> str:
    """Compile every HIP translation unit and link libgdn2.so. Returns its path."""
    if not os.path.exists(HIPCC) and shutil.which("hipcc") is None:
        raise RuntimeError("hipcc not found: the HIP library cannot be built")
    os.makedirs(OBJDIR, exist_ok=True)
    jobs = jobs or min(16, os.cpu_count() or 4)
    units = _units()
    objs = []
    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        futs = [ex.submit(_compile, *u) for u in units]
        for f in futs:
            obj, err = f.result()
            objs.append(obj)
            if verbose and err.strip():
                print(err, file=sys.stderr)
    tmp = OUT + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, OUT)
    return OUT


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
