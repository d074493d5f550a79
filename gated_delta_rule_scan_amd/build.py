"""Build libgdn.so for gfx950 with hipcc, and, where torch, its host compiler and
the Python headers are there, the layer operators' native binding for torch
(_binding.so, host code), in-tree, no JIT cache.

Usage: ``python -m gated_delta_rule_scan_amd.build`` (or ``build()``).
"""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libgdn.so")
BINDING = os.path.join(PKG, "_binding.so")
SOURCES = ["gdn_api.hip", "gdn_prep.hip", "gdn_prep_wide.hip", "gdn_chain.hip", "gdn_colchain.hip", "gdn_epilogue.hip", "gdn_vda.hip",
           "gdn_layer.hip", "gdn_conv.hip", "gdn_ssm.hip", "gdn_rotary.hip", "gdn_step.hip", "gdn_hybrid.hip", "gdn_kv.hip",
           "gdn_attend.hip", "gdn_norm.hip"]
ARCH = "gfx950"

# -packed-fp32-ops: keep the compiler from forming packed fp32 VALU ops.
# -amdgpu-mfma-vgpr-form: matrix-core results land in ordinary VGPRs (gfx950
# has one register file for both), which saves the accumulator-register
# copies around every product whose result feeds vector code (about 100
# copies per state-chain step).
FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-mllvm", "-amdgpu-mfma-vgpr-form",
    "-Wall", "-Wno-unused-result",
    f"-I{INCLUDE}", f"-I{CSRC}",
]


def hipcc() -> str:
    return os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


def _cxx() -> str:
    return os.environ.get("CXX", "g++")


def binding_needs() -> list:
    """What the binding cannot be built without and is not here."""
    needs = []
    if importlib.util.find_spec("torch") is None:
        needs.append("torch")
    if shutil.which(_cxx()) is None:
        needs.append(f"the host compiler {_cxx()}")
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        needs.append("the Python headers")
    return needs


def binding_command() -> list:
    """The compiler line of the binding: host code against torch's headers and
    libraries; the library's entry points are bound at run time."""
    torch = importlib.util.find_spec("torch").submodule_search_locations[0]
    rocm = os.path.dirname(os.path.dirname(hipcc()))
    return [_cxx(), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__=1",
            "-DUSE_ROCM=1", f"-I{torch}/include", f"-I{torch}/include/torch/csrc/api/include", f"-I{rocm}/include",
            f"-I{sysconfig.get_paths()['include']}", f"-I{INCLUDE}", os.path.join(CSRC, "gdn_binding.cpp"), "-o",
            BINDING + ".tmp", f"-L{torch}/lib", "-lc10", "-lc10_hip", "-ltorch_cpu", "-ltorch_hip", "-ltorch_python",
            f"-Wl,-rpath,{torch}/lib"]


def _start(cmd: list) -> subprocess.Popen:
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)


def _ended_well(p: subprocess.Popen, verbose: bool) -> bool:
    out, _ = p.communicate()
    lines = [ln for ln in out.splitlines() if "packed-fp32-ops" not in ln and ln.strip()]
    if p.returncode != 0:
        print("\n".join(lines), file=sys.stderr)
    elif verbose and lines:
        print("\n".join(lines))
    return p.returncode == 0


def build(verbose: bool = False) -> str:
    """Compile every HIP source and link libgdn.so, then the binding, which the
    library does not wait for; always rebuilds."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    needs = binding_needs()
    binding = None if needs else _start(binding_command())
    procs = []
    objs = []
    for src in SOURCES:
        obj = os.path.join(BUILD_DIR, src.replace(".hip", ".o"))
        objs.append(obj)
        cmd = [hipcc(), *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((src, _start(cmd)))
    failed = [src for src, p in procs if not _ended_well(p, verbose)]
    bound = binding is not None and _ended_well(binding, verbose)
    if failed:
        raise RuntimeError(f"hipcc failed for {failed}")
    tmp = LIB + ".tmp"
    cmd = [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp]
    subprocess.check_call(cmd)
    os.replace(tmp, LIB)
    if bound:
        os.replace(BINDING + ".tmp", BINDING)
        return LIB
    if os.path.exists(BINDING):  # of another library
        os.remove(BINDING)
    if needs:
        print(f"the binding for torch is not built: it needs {' and '.join(needs)}", file=sys.stderr)
    else:
        raise RuntimeError("the binding for torch (gdn_binding.cpp) failed; libgdn.so is built")
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
