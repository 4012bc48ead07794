"""Build in-tree: libmoe.so, the HIP kernels for gfx950 plus the host-side C
ABI, with hipcc and g++ alone; tensor_calls.so, the binding's calls on torch
tensors, with torch's headers.  ``python -m block_quantized_expert_amd.build``."""

from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "lib", "libmoe.so")
CALLS = os.path.join(PKG, "lib", "tensor_calls.so")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
HIPCC = os.path.join(ROCM, "bin", "hipcc")
ARCH = "gfx950"

HIP_SOURCES = ["moe_api.hip", "moe_route_group.hip", "moe_ffn.hip", "moe_gemm.hip", "moe_fused.hip",
               "moe_pack.hip", "moe_probe.hip", "moe_rows.hip", "moe_int8.hip", "moe_norm.hip",
               "moe_mxfp4.hip"]
HOST_SOURCES = ["moe_host.cpp", "moe_ops_host.cpp"]

COMMON = ["-O3", "-std=c++17", "-fPIC", "-Wall", "-I" + INCLUDE, "-I" + CSRC]
# Packed fp32 instructions are kept out of the device code on purpose.
HIP_FLAGS = COMMON + ["--offload-arch=" + ARCH, "-Xclang", "-target-feature",
                      "-Xclang", "-packed-fp32-ops"]
HOST_FLAGS = COMMON + ["-D__HIP_PLATFORM_AMD__", "-I" + os.path.join(ROCM, "include")]


def _run(cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    out = (r.stdout + r.stderr).strip()
    # the host pass does not know the device-only feature above
    lines = [ln for ln in out.splitlines() if "packed-fp32-ops" not in ln]
    if r.returncode != 0:
        raise RuntimeError("command failed: %s\n%s" % (" ".join(cmd), "\n".join(lines)))
    return "\n".join(lines)


def _torch_flags():
    import sysconfig

    from torch.utils import cpp_extension

    return ["-DUSE_ROCM=1", "-fvisibility=hidden"] + [
        "-isystem" + p for p in cpp_extension.include_paths() + [sysconfig.get_paths()["include"]]]


def _torch_libs():
    from torch.utils import cpp_extension

    return ["-L" + p for p in cpp_extension.library_paths()] + [
        "-lc10", "-lc10_hip", "-ltorch_cpu", "-ltorch_hip", "-ltorch_python"]


def build(verbose: bool = False) -> str:
    """Compile every source and link libmoe.so, then the calls on tensors
    (tensor_calls.so), which need torch's and Python's headers; returns the
    library's path.  Without torch only the library is built; if the calls on
    tensors do not compile, the library is in place when the error is raised."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    os.makedirs(os.path.dirname(LIB), exist_ok=True)
    jobs = []
    for src in HIP_SOURCES:
        obj = os.path.join(BUILD_DIR, src + ".o")
        jobs.append((obj, [HIPCC] + HIP_FLAGS + ["-c", os.path.join(CSRC, src), "-o", obj]))
    for src in HOST_SOURCES:
        obj = os.path.join(BUILD_DIR, src + ".o")
        jobs.append((obj, ["g++"] + HOST_FLAGS + ["-c", os.path.join(CSRC, src), "-o", obj]))
    try:
        torch_flags = _torch_flags()
    except (ImportError, OSError) as e:
        torch_flags = None
        print("tensor_calls.so is not built: %s" % e, file=sys.stderr)
        if os.path.exists(CALLS):
            os.remove(CALLS)
    calls = os.path.join(BUILD_DIR, "tensor_calls.cpp.o")
    workers = min(len(jobs) + 1, max(1, min(8, os.cpu_count() or 1)))
    with cf.ThreadPoolExecutor(workers) as ex:
        compiled = None
        if torch_flags is not None:
            compiled = ex.submit(_run, ["g++"] + HOST_FLAGS + torch_flags + [
                "-c", os.path.join(CSRC, "tensor_calls.cpp"), "-o", calls])
        logs = list(ex.map(lambda j: _run(j[1]), jobs))
        tmp = LIB + ".tmp"
        logs.append(_run([HIPCC, "-shared", "-fPIC", "--offload-arch=" + ARCH]
                         + [o for o, _ in jobs] + ["-o", tmp]))
        os.replace(tmp, LIB)
        if compiled is not None:
            logs.append(compiled.result())
            tmp = CALLS + ".tmp"
            logs.append(_run(["g++", "-shared", calls, "-o", tmp, "-L" + os.path.dirname(LIB),
                              "-l:libmoe.so", "-Wl,-rpath,$ORIGIN"] + _torch_libs()))
            os.replace(tmp, CALLS)
    if verbose:
        for log in logs:
            if log:
                print(log)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
