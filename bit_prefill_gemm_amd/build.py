"""Build the HIP library libbpg.so in place (gfx950), and _native.so, the
compiled Python entry points over it.

Every source is compiled with -ffp-contract=off (the quantizer must not fuse
its adds and multiplies) and with packed fp32 instructions disabled.
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libbpg.so")
NATIVE = os.path.join(HERE, "_native.so")
SOURCES = ["api.hip", "quantize.hip", "gemm.hip", "skinny.hip", "wide.hip", "strip.hip", "grouped.hip", "moe.hip",
           "norm.hip", "route.hip", "fp8_quantize.hip", "fp8_stream.hip", "fp8_tile.hip", "logprobs.hip"]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
# code-generation flags (the part of the command line that shapes the kernels;
# the include directories below are paths of this checkout)
KERNEL_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-ffp-contract=off",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # matrix-instruction results in ordinary VGPRs: the epilogues read them with
    # VALU instructions, which cannot read accumulation registers
    "-mllvm", "-amdgpu-mfma-vgpr-form",
]
FLAGS = KERNEL_FLAGS + ["-Wall", "-Wno-unused-function", "-I", INCLUDE, "-I", CSRC]


def _run(cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    # the host pass does not know the packed-fp32 feature name; that warning is harmless
    err = "\n".join(ln for ln in r.stderr.splitlines() if "packed-fp32-ops" not in ln)
    if r.returncode != 0:
        raise RuntimeError("command failed: %s\n%s" % (" ".join(cmd), err))
    return err


def _torch_dir() -> str:
    import importlib.util
    return os.path.dirname(importlib.util.find_spec("torch").origin)


def _native_commands(obj, out):
    """Compile and link commands of the Python extension (host code over libbpg.so and torch)."""
    torch_dir = _torch_dir()
    compile_cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-fvisibility=hidden",
                   "-DUSE_ROCM", "-D__HIP_PLATFORM_AMD__", "-I", INCLUDE,
                   "-isystem", os.path.join(torch_dir, "include"),
                   "-isystem", "/opt/rocm/include", "-isystem", sysconfig.get_paths()["include"],
                   "-c", os.path.join(CSRC, "native.cpp"), "-o", obj]
    link_cmd = ["g++", "-shared", obj, "-o", out, "-L", HERE, "-l:libbpg.so",
                "-L", os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu",
                "-ltorch_hip", "-lc10", "-lc10_hip", "-Wl,-rpath,$ORIGIN"]
    return compile_cmd, link_cmd


def build(verbose: bool = False) -> str:
    objdir = os.path.join(HERE, "_build")
    os.makedirs(objdir, exist_ok=True)
    objs = [os.path.join(objdir, s.replace(".hip", ".o")) for s in SOURCES]
    cmds = [[HIPCC, *FLAGS, "-c", os.path.join(CSRC, s), "-o", o] for s, o in zip(SOURCES, objs)]
    native_tmp = NATIVE + ".tmp%d" % os.getpid()
    native_cmd, native_link = _native_commands(os.path.join(objdir, "native.o"), native_tmp)
    with ThreadPoolExecutor(max_workers=len(cmds) + 1) as ex:
        outs = list(ex.map(_run, cmds + [native_cmd]))
    if verbose:
        for o in outs:
            if o.strip():
                print(o, file=sys.stderr)
    tmp = LIB + ".tmp%d" % os.getpid()
    _run([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp])
    os.replace(tmp, LIB)
    _run(native_link)
    os.replace(native_tmp, NATIVE)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
