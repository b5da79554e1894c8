"""Build libfp8gemm.so (the gfx950 kernels and their C ABI) with hipcc, and
_direct.so (Python's way to its shortest calls) with the host compiler.

The library is built in-tree, next to this file, so it travels with the
source tree.  Nothing here is needed at run time except the built library
(without _direct.so the binding makes the same calls through ctypes).
"""
from __future__ import annotations

import importlib.util
import os
import shlex
import shutil
import subprocess
import sysconfig
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libfp8gemm.so")
SOURCES = [os.path.join(CSRC, f) for f in ("fp8gemm.hip", "moe.hip", "moe_ops.hip", "w4.hip", "block_ops.hip",
                                                    "moe_few.hip", "jit.hip")]
DENSE_SOURCE = os.path.join(CSRC, "dense_launch.hip")  # once per operand-format pair, with an epilogue and without
DIRECT = os.path.join(HERE, "_direct.so")
DIRECT_SOURCE = os.path.join(CSRC, "direct.cpp")
W4_SOURCE = os.path.join(CSRC, "w4_launch.hip")  # compiled once per kind of 4-bit matrix

# Device code generation; the runtime specialisation compiles with the same.
DEVICE_FLAGS = [
    "-O3", "-std=c++17",
    # no packed-FP32 VALU ops anywhere in device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # MFMA results land in architectural VGPRs, where the promotion FMAs read them
    "-mllvm", "-amdgpu-mfma-vgpr-form",
]
LIBS: list = []
# Headers the runtime specialisation compiles (embedded in the library).
JIT_HEADERS = ["device_common.hpp", "gemm_kernel.hpp"]
_DELIM = "fp8jit"


def jit_sources_inc() -> str:
    """C++ text embedding the kernel headers and the device options."""
    out = ["// Generated by build.py: the kernel headers and device options the",
           "// runtime specialisation compiles with.", "namespace fp8g {", "namespace jit_src {",
           f"constexpr int kNumHeaders = {len(JIT_HEADERS)};",
           "const char* const kHeaderNames[] = {" + ", ".join(f'"{h}"' for h in JIT_HEADERS) + "};",
           "const char* const kHeaderTexts[] = {"]
    for h in JIT_HEADERS:
        text = open(os.path.join(CSRC, h)).read()
        if f"){_DELIM}\"" in text:
            raise RuntimeError(f"{h} contains the raw-string delimiter")
        out.append(f'R"{_DELIM}({text}){_DELIM}",')
    out += ["};", f"constexpr int kNumOptions = {len(DEVICE_FLAGS)};",
            "const char* const kOptions[] = {" + ", ".join(f'"{f}"' for f in DEVICE_FLAGS) + "};",
            "}  // namespace jit_src", "}  // namespace fp8g", ""]
    return "\n".join(out)


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found")


def _compile_jobs(gen: str, objdir: str):
    """(command, object) per translation unit: the host/grouped/cast unit, the
    MoE layout unit, the routing and combine unit, the 4-bit unit, the unit of
    norms and the epilogue's gradients, that of whole MoE layers, the
    runtime-specialisation unit, the dense GEMM instantiations once per
    operand-format pair (with and without an epilogue) and the 4-bit kernels
    once per kind of matrix."""
    base = [hipcc(), *DEVICE_FLAGS, "--offload-arch=gfx950", "-fPIC", "-c", "-I", INCLUDE, "-I", CSRC, "-I", gen]
    jobs = []
    for src in SOURCES:
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        jobs.append(([*base, src, "-o", obj], obj))
    for fmt in range(4):
        for epi in range(2):
            obj = os.path.join(objdir, f"dense_launch_fmt{fmt}_epi{epi}.o")
            jobs.append(([*base, f"-DFP8G_DENSE_FMT={fmt}", f"-DFP8G_DENSE_EPI={epi}", DENSE_SOURCE, "-o", obj], obj))
    for kind in range(3):
        obj = os.path.join(objdir, f"w4_launch_kind{kind}.o")
        jobs.append(([*base, f"-DFP8G_W4_KIND={kind}", W4_SOURCE, "-o", obj], obj))
    return jobs


def host_cxx() -> list:
    """The host compiler's command: $CXX, g++, or the ROCm compiler that hipcc runs."""
    if os.environ.get("CXX"):
        return shlex.split(os.environ["CXX"])
    return [shutil.which("g++") or os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin", "clang++")]


def _direct_command(out: str) -> list:
    """The host compiler's command for _direct.so (against the installed torch and the built library)."""
    torch_dir = os.path.dirname(importlib.util.find_spec("torch").origin)
    return [*host_cxx(), "-O2", "-std=c++17", "-shared", "-fPIC", "-I", INCLUDE,
            "-I", os.path.join(torch_dir, "include"),
            "-I", os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
            "-I", sysconfig.get_paths()["include"], DIRECT_SOURCE, "-o", out, "-L", os.path.join(torch_dir, "lib"),
            "-ltorch_python", "-ltorch_cpu", "-lc10", "-L", HERE, f"-l:{os.path.basename(LIB)}",
            "-Wl,-rpath,$ORIGIN"]


def build(verbose: bool = False) -> str:
    tmp = LIB + ".tmp"
    with tempfile.TemporaryDirectory() as gen:
        with open(os.path.join(gen, "jit_sources.inc"), "w") as f:
            f.write(jit_sources_inc())
        jobs = _compile_jobs(gen, gen)
        procs = [(subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True), obj)
                 for cmd, obj in jobs]
        errors = []
        for proc, obj in procs:
            out, err = proc.communicate()
            if proc.returncode != 0:
                errors.append(err)
            elif verbose and err:
                print(err)
        if errors:
            raise RuntimeError("hipcc failed:\n" + "\n".join(errors))
        cmd = [hipcc(), "--offload-arch=gfx950", "-shared", "-fPIC", *[obj for _, obj in jobs], "-o", tmp, *LIBS]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError("hipcc link failed:\n" + res.stderr)
    os.replace(tmp, LIB)
    tmp = DIRECT + ".tmp"
    res = subprocess.run(_direct_command(tmp), capture_output=True, text=True)
    if res.returncode != 0:
        if os.path.exists(DIRECT):  # of an earlier build, perhaps of other entry points
            os.remove(DIRECT)
        raise RuntimeError(f"building {os.path.basename(DIRECT)} failed:\n" + res.stderr)
    os.replace(tmp, DIRECT)
    return LIB


if __name__ == "__main__":
    print(build(verbose=False))
