"""Compile libeq.so in-tree for gfx950.

host_codec.cpp is plain C++17 (g++); decode.hip, encode.hip, rownorm.hip and
w4.hip are HIP for gfx950 only (wave64, CDNA4), built without packed-fp32
instruction selection; pipeline.hip is the host-side block schedule.
"""
import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libeq.so")
ARCH = os.environ.get("EQ_OFFLOAD_ARCH", "gfx950")

HIPCC_FLAGS = ["-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}",
               "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
               "-Wall", "-Wno-unused-command-line-argument"]


def _run(cmd, verbose):
    if verbose:
        print("+", " ".join(cmd), flush=True)
    subprocess.check_call(cmd, cwd=ROOT)


def build_library(verbose: bool = False, out: str = LIB, defines: dict | None = None,
                  build_dir: str = BUILD) -> str:
    """Build libeq.so (or a variant with extra -D defines at `out`)."""
    os.makedirs(build_dir, exist_ok=True)
    dflags = [f"-D{k}={v}" for k, v in (defines or {}).items()]
    sources = {"host_codec": ["g++", "-O2", "-std=c++17", "-fPIC", "-pthread", "-Wall", "-Wextra"],
               "decode": ["hipcc", *HIPCC_FLAGS, *dflags], "encode": ["hipcc", *HIPCC_FLAGS, *dflags],
               "rownorm": ["hipcc", *HIPCC_FLAGS, *dflags], "w4": ["hipcc", *HIPCC_FLAGS, *dflags],
               "pipeline": ["hipcc", *HIPCC_FLAGS]}
    objects = [os.path.join(build_dir, name + ".o") for name in sources]
    commands = [[*cc, "-c", os.path.join(CSRC, name + (".cpp" if cc[0] == "g++" else ".hip")), "-o", o]
                for (name, cc), o in zip(sources.items(), objects)]
    with ThreadPoolExecutor(max_workers=min(4, os.cpu_count() or 1)) as pool:
        for done in [pool.submit(_run, c, verbose) for c in commands]:
            done.result()
    tmp = out + ".tmp"
    _run(["hipcc", "-shared", f"--offload-arch={ARCH}", *objects, "-o", tmp, "-pthread"], verbose)
    os.replace(tmp, out)
    return out


if __name__ == "__main__":
    build_library(verbose=True)
