"""Build libgdn.so (HIP kernels for gfx950 + the C ABI) in-tree with hipcc, and then the binding's
module _marshal with the host compiler."""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJDIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libgdn.so")

SOURCES = ["gdn_fwd.hip", "gdn_bwd.hip", "gdn_decode.hip", "gdn_conv.hip", "gdn_scratch.hip", "gdn_abi.cpp",
           "gdn_trace.cpp", "layer/conv_carry.hip", "layer/norm.hip", "layer/ssm_decode.hip", "layer/ssm_sweep.hip",
           "layer/ssm_grad.hip", "layer/layer_abi.cpp"]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"
# Packed-FP32 instructions are disabled for every device pass.
FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    f"-I{INCLUDE}", f"-I{CSRC}",
]


def _compile(src: str) -> str:
    obj = os.path.join(OBJDIR, os.path.splitext(os.path.basename(src))[0] + ".o")
    cmd = [HIPCC, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    if src.endswith(".cpp"):
        cmd.insert(1, "-xhip")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stderr}")
    return obj


def _marshal() -> None:
    """The binding's C module (no GPU code), for the interpreter that runs this: its tag is in the name."""
    out = os.path.join(PKG, "_marshal" + sysconfig.get_config_var("EXT_SUFFIX"))
    cmd = [os.environ.get("CC", "gcc"), "-O2", "-Wall", "-shared", "-fPIC", f"-I{sysconfig.get_paths()['include']}",
           os.path.join(CSRC, "layer", "marshal.c"), "-o", out + ".tmp"]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
    except OSError as e:
        raise RuntimeError(f"{cmd[0]} for marshal.c: {e} ({LIB} is built; the operators of gdn.h work without)") from e
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed for marshal.c ({LIB} is built; the operators of gdn.h work without):\n{r.stderr}")
    os.replace(out + ".tmp", out)


def build(verbose: bool = False) -> str:
    os.makedirs(OBJDIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(len(SOURCES), os.cpu_count() or 1)) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    _marshal()
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
