"""Build libmxq.so (the HIP kernels and their C ABI) in-tree for gfx950.

    python -m nvfp4_quantization_grouped_amd.build

Compiles every csrc/*.hip file (kernels) and csrc/*.cpp file (the host-side
C ABI) with hipcc for gfx950 and links them into
nvfp4_quantization_grouped_amd/libmxq.so.  hipcc cross-compiles, so this runs
on a machine without a GPU.
"""

import ctypes
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libmxq.so")
BUILD_DIR = os.path.join(ROOT, "_build")

ARCH = "gfx950"
HIPCC_FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
    # packed-fp32 VALU forms are left to nobody: keep plain fp32 ops
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
    "-I", os.path.join(ROOT, "include"),
]
# Flags of some files (by the start of their names).  The attention kernels' sums pass through branches and are scaled
# between products: in VGPRs they stay where they are, in AGPRs each passage copies them (64 of 430 registers at head size
# 128, and a third of the instructions).
FILE_FLAGS = {"cache_attention_": ["-mllvm", "-amdgpu-mfma-vgpr-form=1"]}


def hipcc():
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    exe = shutil.which("hipcc") or os.path.join(rocm, "bin", "hipcc")
    if not os.path.exists(exe):
        raise RuntimeError("hipcc not found (needed to build libmxq for gfx950)")
    return exe


def _compile(src, extra):
    obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
    own = [f for start, flags in FILE_FLAGS.items() if os.path.basename(src).startswith(start) for f in flags]
    cmd = [hipcc(), *HIPCC_FLAGS, *own, *extra, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    noise = "is not a recognized feature for this target"
    err = "\n".join(l for l in (r.stderr or "").splitlines() if noise not in l)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{err}")
    if err.strip():
        sys.stderr.write(err + "\n")
    return obj


def build(verbose=True, extra_flags=()):
    """Compile all csrc/*.hip and csrc/*.cpp and link libmxq.so; returns the library path."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    srcs = sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".hip", ".cpp")))
    with ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(lambda s: _compile(s, list(extra_flags)), srcs))
    tmp = LIB + ".tmp"
    cmd = [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    # an unresolved kernel stub only shows up at load time: load it here
    try:
        ctypes.CDLL(tmp)
    except OSError as e:
        os.remove(tmp)
        raise RuntimeError(f"built library does not load: {e}") from None
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build()
