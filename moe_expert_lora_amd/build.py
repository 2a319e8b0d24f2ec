"""Build libmlora.so in-tree with hipcc for gfx950.

Usage: ``python -m moe_expert_lora_amd.build`` (or ``build()`` from Python).
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libmlora.so")
SOURCES = [os.path.join(CSRC, name)
           for name in ("mlora_host.cpp", "mlora_fold.hip", "mlora_moe.hip", "mlora_w4.hip",
                       "mlora_fp8.hip", "mlora_layer.hip", "mlora_norm.hip")]
# measurement probes for bench.py (launch and read-pattern floors), a library of their own
PROBE_LIB = os.path.join(PKG, "libmlora_probe.so")
PROBE_SOURCES = [os.path.join(CSRC, "mlora_probe.hip")]
# the CPython binding of the MoE layer's operators, against libmlora.so and torch
BINDING = os.path.join(PKG, "_native" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
BINDING_SOURCE = os.path.join(CSRC, "mlora_binding.cpp")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CXX = os.environ.get("CXX", "g++")

FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-Wall",
    # keep hipcc from forming packed fp32 VALU ops (v_pk_*_f32)
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # kernel arguments that lead with plain pointers / ints arrive in SGPRs
    # (the kernel keeps a prologue that loads them where firmware does not)
    "-mllvm", "-amdgpu-kernarg-preload-count=10",
    "-I", INCLUDE,
]


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    noise = "is not a recognized feature for this target"
    err = "\n".join(l for l in (res.stderr or "").splitlines() if noise not in l)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed ({res.returncode}):\n{err}")
    if verbose and err.strip():
        print(err, file=sys.stderr)


def _compile(sources, lib, verbose):
    """Each source to an object, side by side, then one link."""
    with tempfile.TemporaryDirectory(dir=PKG, prefix="_build") as tmp:
        objs = [os.path.join(tmp, os.path.basename(src) + ".o") for src in sources]
        with ThreadPoolExecutor(4) as pool:
            list(pool.map(lambda so: _run([HIPCC, *FLAGS, "-c", so[0], "-o", so[1]], verbose),
                          zip(sources, objs)))
        out = os.path.join(tmp, os.path.basename(lib))
        _run([HIPCC, "--offload-arch=gfx950", "-shared", *objs, "-o", out], verbose)
        os.replace(out, lib)


def has_torch() -> bool:
    """Whether a PyTorch for ROCm is there to build the binding against."""
    try:
        import torch
    except ImportError:
        return False
    return torch.version.hip is not None


def _compile_binding(verbose):
    """Host code only: torch's core headers, Python's and HIP's."""
    import torch
    from torch.utils.cpp_extension import include_paths
    lib_dir = os.path.join(os.path.dirname(torch.__file__), "lib")
    system = [*include_paths(), "/opt/rocm/include", sysconfig.get_paths()["include"]]
    out = BINDING + ".tmp"
    _run([CXX, "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__=1",
          "-DUSE_ROCM=1", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
          "-I", INCLUDE, *[a for d in system for a in ("-isystem", d)], BINDING_SOURCE,
          "-L", lib_dir, "-lc10", "-lc10_hip", "-ltorch_cpu", "-ltorch_python", "-L", PKG,
          "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN", "-o", out], verbose)
    os.replace(out, BINDING)


def build(verbose: bool = False) -> str:
    """Compile moe_expert_lora_amd/libmlora.so (the fold and the MoE layer's
    operators), libmlora_probe.so (bench.py's measurement probes) and, where there
    is a PyTorch for ROCm, the CPython binding of the MoE layer's operators (the C
    interface and the host functions do without); returns libmlora.so's path."""
    _compile(SOURCES, LIB, verbose)
    _compile(PROBE_SOURCES, PROBE_LIB, verbose)
    if has_torch():
        _compile_binding(verbose)
    else:
        print("no PyTorch for ROCm: " + os.path.basename(BINDING) + " is not built",
              file=sys.stderr)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
