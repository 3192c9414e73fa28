"""Build libllmoe.so (the gfx950 HIP library) in-tree with hipcc.

    python combine_ll_moe_amd/build.py
"""
import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libllmoe.so")
SOURCES = ["gemm_few_int4.hip", "gemm_tile.hip", "gemm_few_fp8.hip", "gemm_few_bf16.hip",  # longest first
           "api.hip", "dispatch.hip", "combine.hip", "two_phase.hip", "receive.hip", "watch.hip",
           "probe.hip", "expert_api.hip", "norm.hip"]
ARCH = "gfx950"

FLAGS = [
    "-O3", "-std=c++17", "-fPIC", "-shared",
    f"--offload-arch={ARCH}",
    # keep the compiler away from packed fp32 instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-fno-gpu-rdc", "-Wall",
]


def build(verbose: bool = False, extra_flags=None) -> str:
    """Compile every source (a few at a time), then link."""
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    # hipcc's host pass does not know the packed-fp32 feature and says so
    noise = "'-packed-fp32-ops' is not a recognized feature"

    def run(cmd) -> None:
        if verbose:
            print(" ".join(cmd), flush=True)
        res = subprocess.run(cmd, capture_output=True, text=True)
        err = "\n".join(l for l in res.stderr.splitlines() if noise not in l)
        if res.returncode != 0:
            raise RuntimeError(f"hipcc failed ({res.returncode}):\n{err}")
        if verbose and err.strip():
            print(err, file=sys.stderr)

    flags = [*FLAGS, *(extra_flags or []), "-I", os.path.join(ROOT, "include"), "-I", CSRC]
    with tempfile.TemporaryDirectory() as tmp:
        objects = [os.path.join(tmp, s + ".o") for s in SOURCES]
        with ThreadPoolExecutor(min(6, os.cpu_count() or 1)) as pool:
            list(pool.map(run, ([hipcc, *[f for f in flags if f != "-shared"], "-c", "-o", o,
                                 os.path.join(CSRC, s)] for s, o in zip(SOURCES, objects))))
        run([hipcc, *FLAGS, *(extra_flags or []), "-o", LIB + ".tmp", *objects])
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
