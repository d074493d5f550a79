"""Build libgdn.so for gfx950 with hipcc, and the layer operators' native
binding for torch (_binding.so, host code), in-tree, no JIT cache.

Usage: ``python -m gated_delta_rule_scan_amd.build`` (or ``build()``).
"""
from __future__ import annotations

import importlib.util
import os
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
           "gdn_layer.hip", "gdn_conv.hip", "gdn_ssm.hip", "gdn_rotary.hip", "gdn_step.hip"]
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


def binding_command() -> list:
    """The compiler line of the binding: host code against torch's headers and
    libraries; the library's entry points are bound at run time."""
    torch = importlib.util.find_spec("torch").submodule_search_locations[0]
    rocm = os.path.dirname(os.path.dirname(hipcc()))
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__=1",
            "-DUSE_ROCM=1", f"-I{torch}/include", f"-I{torch}/include/torch/csrc/api/include", f"-I{rocm}/include",
            f"-I{sysconfig.get_paths()['include']}", f"-I{INCLUDE}", os.path.join(CSRC, "gdn_binding.cpp"), "-o",
            BINDING + ".tmp", f"-L{torch}/lib", "-lc10", "-lc10_hip", "-ltorch_cpu", "-ltorch_hip", "-ltorch_python",
            f"-Wl,-rpath,{torch}/lib"]


def build(verbose: bool = False) -> str:
    """Compile every HIP source and link libgdn.so, and the binding; always
    rebuilds."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    procs = [("gdn_binding.cpp", subprocess.Popen(binding_command(), stdout=subprocess.PIPE, stderr=subprocess.STDOUT,
                                                  text=True))]
    objs = []
    for src in SOURCES:
        obj = os.path.join(BUILD_DIR, src.replace(".hip", ".o"))
        objs.append(obj)
        cmd = [hipcc(), *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        lines = [ln for ln in out.splitlines() if "packed-fp32-ops" not in ln and ln.strip()]
        if p.returncode != 0:
            failed.append(src)
            print("\n".join(lines), file=sys.stderr)
        elif verbose and lines:
            print("\n".join(lines))
    if failed:
        raise RuntimeError(f"hipcc failed for {failed}")
    tmp = LIB + ".tmp"
    cmd = [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp]
    subprocess.check_call(cmd)
    os.replace(tmp, LIB)
    os.replace(BINDING + ".tmp", BINDING)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
