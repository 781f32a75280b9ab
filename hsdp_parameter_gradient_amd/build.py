"""Build the gfx950 shared library libfsdpflat.so in-tree with hipcc.

    python -m hsdp_parameter_gradient_amd.build

Every call compiles from source (no up-to-date check); the library is
written to a temporary name and renamed into place, so a process that has
the old library loaded keeps a consistent file.  The compiler's resource
report of every kernel (registers, occupancy, LDS, private scratch) is
written beside it as kernel_resources.json.
"""

from __future__ import annotations

import json
import os
import re
import shutil
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB_DIR = os.path.join(PKG, "lib")
LIB_NAME = "libfsdpflat.so"
RESOURCES = "kernel_resources.json"
_REMARK = "kernel-resource-usage"
_FIELDS = {"VGPRs": "vgprs", "AGPRs": "agprs", "TotalSGPRs": "sgprs", "ScratchSize [bytes/lane]": "scratch_bytes",
           "Occupancy [waves/SIMD]": "waves_per_simd", "VGPRs Spill": "vgpr_spill", "SGPRs Spill": "sgpr_spill",
           "LDS Size [bytes/block]": "lds_bytes"}
SOURCES = ("fsdp_flat.cpp", "kernels.hip", "token_ops.cpp", "token_kernels.hip")

HIP_FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-Wall",
    # IEEE fp32 everywhere: keep denormals, correctly rounded division
    "-fno-gpu-flush-denormals-to-zero",
    "-fhip-fp32-correctly-rounded-divide-sqrt",
    "-ffp-contract=off",
    # no packed-fp32 instructions in device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def hipcc() -> str:
    for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("hipcc not found (ROCm is required to build libfsdpflat.so)")


def parse_resources(stderr: str) -> dict:
    """Per-kernel figures of hipcc's kernel-resource-usage remarks, keyed by
    the mangled kernel name."""
    out, cur = {}, None
    for line in stderr.splitlines():
        if _REMARK not in line:
            continue
        m = re.search(r"remark: Function Name: (\S+)", line)
        if m:
            cur = out.setdefault(m.group(1), {})
            continue
        m = re.search(r"remark:\s+(.+?): (\w+) \[", line)
        if m and cur is not None and m.group(1) in _FIELDS:
            v = m.group(2)
            cur[_FIELDS[m.group(1)]] = int(v) if v.isdigit() else v
    return out


def build(verbose: bool = False) -> str:
    os.makedirs(LIB_DIR, exist_ok=True)
    out = os.path.join(LIB_DIR, LIB_NAME)
    tmp = out + ".tmp%d" % os.getpid()

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        return subprocess.run(cmd, capture_output=True, text=True)

    with tempfile.TemporaryDirectory() as objs:
        obj = {s: os.path.join(objs, s + ".o") for s in SOURCES}
        with ThreadPoolExecutor(len(SOURCES)) as pool:  # one compiler per source
            rs = list(pool.map(lambda s: run([hipcc(), *HIP_FLAGS, "-I", os.path.join(ROOT, "include"), "-I", CSRC,
                                              "-c", os.path.join(CSRC, s), "-o", obj[s],
                                              "-Rpass-analysis=" + _REMARK]), SOURCES))
        if all(r.returncode == 0 for r in rs):
            rs.append(run([hipcc(), "--offload-arch=gfx950", "-shared", "-fPIC", *obj.values(), "-o", tmp]))
    stderr = "\n".join(r.stderr or "" for r in rs)
    # hipcc's host pass does not know the packed-fp32 feature and says so
    noise = "not a recognized feature for this target"
    warn = "\n".join(l for l in stderr.splitlines()
                     if noise not in l and "ignoring feature" not in l and _REMARK not in l)
    failed = [r for r in rs if r.returncode != 0]
    if failed:
        if os.path.exists(tmp):
            os.unlink(tmp)
        raise RuntimeError("hipcc failed (%d):\n%s\n%s" % (failed[0].returncode, failed[0].stdout, warn))
    if verbose and warn.strip():
        print(warn, file=sys.stderr)
    res = parse_resources(stderr)
    rtmp = os.path.join(LIB_DIR, RESOURCES + ".tmp%d" % os.getpid())
    with open(rtmp, "w") as f:
        json.dump(res, f, indent=1, sort_keys=True)
    os.replace(tmp, out)
    os.replace(rtmp, os.path.join(LIB_DIR, RESOURCES))
    return out


if __name__ == "__main__":
    print(build(verbose=True))
