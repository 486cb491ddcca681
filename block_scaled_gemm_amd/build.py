"""Build libfp8bs.so in-tree with hipcc for gfx950.

    python -m block_scaled_gemm_amd.build

Compiles every source under csrc/ into block_scaled_gemm_amd/libfp8bs.so.
Flags: -O3, no fast-math (IEEE divisions and no denormal flushing are part
of the quantisers' contract), hidden visibility except the C ABI, and the
packed-fp32 feature switched off for device code.
"""
import concurrent.futures
import os
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libfp8bs.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

SOURCES = ["gemm.hip", "gated.hip", "quant.hip", "norm.hip", "clip.hip", "api.cpp", "block_api.cpp"]

FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
    "-fvisibility=hidden", "-Wall",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd))
    r = subprocess.run(cmd, capture_output=True, text=True)
    # hipcc's host pass does not know the device-only feature flag and says so
    noise = "'-packed-fp32-ops' is not a recognized feature"
    err = "\n".join(l for l in r.stderr.splitlines() if noise not in l)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed ({r.returncode}):\n{err}")
    if err.strip() and verbose:
        print(err, file=sys.stderr)


def build(out=LIB, verbose=False):
    # every source on its own, side by side, then one link
    with tempfile.TemporaryDirectory() as tmp, concurrent.futures.ThreadPoolExecutor(len(SOURCES)) as pool:
        objs = [os.path.join(tmp, s + ".o") for s in SOURCES]
        jobs = [pool.submit(_run, [HIPCC, *FLAGS, "-x", "hip", "-c", os.path.join(CSRC, s), "-o", o], verbose)
                for s, o in zip(SOURCES, objs)]
        for j in jobs:
            j.result()
        _run([HIPCC, f"--offload-arch={ARCH}", "-shared", *objs, "-o", out + ".tmp"], verbose)
    os.replace(out + ".tmp", out)
    return out


if __name__ == "__main__":
    print(build(verbose=True))
