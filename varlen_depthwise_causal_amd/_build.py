"""Ahead-of-time build of libvdc.so for gfx950 with hipcc, and of the recurrent
layer's binding (no JIT)."""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIBRARY = os.path.join(PKG, "libvdc.so")
BINDING = os.path.join(PKG, "_vdc_torch.so")

ARCH = "gfx950"
# Packed FP32 instructions stay off: plain float code is scheduled on the
# scalar-per-lane FP32 pipes.  FMA contraction is off too: every FMA in the
# kernels is written out, so the evaluation order is exactly the source's.
DEVICE_FLAGS = ["-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
                "-ffp-contract=off"]
COMMON = ["-O3", "-std=c++17", "-fPIC", "--offload-arch=" + ARCH, "-I", INCLUDE, "-I", CSRC]

SOURCES = ("vdc_kernels.hip", "vdc_conv_state.hip", "vdc_scan.hip", "vdc_norm.hip", "vdc_recurrence.hip",
           "vdc_layer_norm.hip", "vdc_pool.hip", "vdc_api.cpp", "vdc_ssm_api.cpp", "vdc_layer_api.cpp")


def hipcc() -> str:
    path = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(path):
        raise RuntimeError("hipcc not found; ROCm is required to build libvdc.so")
    return path


def _binding_commands(torch: str, obj: str, out: str):
    """Compiles csrc/vdc_torch.cpp against the torch installed in that folder and
    links it with libvdc.so, which it finds beside itself, and torch's libraries,
    which are loaded when it is."""
    cxx = shutil.which("g++") or hipcc()
    rocm = os.path.dirname(os.path.dirname(os.path.realpath(hipcc())))
    compile_ = [cxx, "-O2", "-std=c++17", "-fPIC", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
                "-I", sysconfig.get_paths()["include"], "-I", os.path.join(torch, "include"),
                "-I", os.path.join(rocm, "include"), "-I", INCLUDE, "-c", os.path.join(CSRC, "vdc_torch.cpp"), "-o", obj]
    link = [cxx, "-shared", "-o", out, obj, "-L", PKG, "-lvdc", "-Wl,-rpath,$ORIGIN", "-L", os.path.join(torch, "lib"),
            "-ltorch_python", "-ltorch_hip", "-ltorch_cpu", "-lc10_hip", "-lc10"]
    return compile_, link


def build(verbose: bool = False) -> str:
    """Compile csrc/*.hip + csrc/*.cpp into libvdc.so, and the recurrent layer's
    binding into _vdc_torch.so (always rebuilds).  libvdc.so needs hipcc alone and
    is in place before the binding can fail; without torch there is no binding,
    and the calls of module layer raise ImportError."""
    def start(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        return cmd, subprocess.Popen(cmd)

    def finish(cmd, process):
        if process.wait():
            raise subprocess.CalledProcessError(process.returncode, cmd)

    def link(cmd, tmp, out):
        finish(*start(cmd))
        os.replace(tmp, out)

    os.makedirs(BUILD_DIR, exist_ok=True)
    cc = hipcc()
    objs, running = [], []
    for src in SOURCES:
        obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
        extra = DEVICE_FLAGS if src.endswith(".hip") else []
        running.append(start([cc, *COMMON, *extra, "-c", os.path.join(CSRC, src), "-o", obj]))
        objs.append(obj)
    torch, tmp = importlib.util.find_spec("torch"), ".tmp%d" % os.getpid()
    if torch:
        binding_compile, binding_link = _binding_commands(os.path.dirname(torch.origin),
                                                          os.path.join(BUILD_DIR, "vdc_torch.o"), BINDING + tmp)
        binding = start(binding_compile)
    for job in running:
        finish(*job)
    link([cc, "-shared", "-fPIC", "--offload-arch=" + ARCH, "-o", LIBRARY + tmp, *objs], LIBRARY + tmp, LIBRARY)
    if torch:
        finish(*binding)
        link(binding_link, BINDING + tmp, BINDING)
    else:
        print("torch not found: libvdc.so alone, without the binding of module layer", flush=True)
    return LIBRARY


if __name__ == "__main__":
    print(build(verbose=True))
