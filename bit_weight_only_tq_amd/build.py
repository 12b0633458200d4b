"""Build libtq.so (the HIP kernels and the C ABI) in-tree for gfx950, and
_serving.so, the Python entry of its serving operators (host code only, built
against the installed torch).

Usage: python -m bit_weight_only_tq_amd.build  (or call ``build()``).

Every HIP translation unit is compiled with hipcc for --offload-arch=gfx950
and linked into ``bit_weight_only_tq_amd/libtq.so``.  The prepare kernels
(pack.hip) are compiled with -ffp-contract=off so that their fp64 sums and
divisions are exactly the operations written.  Packed fp32 instructions are
disabled for all device code (-packed-fp32-ops); hipcc's host pass warns
that it does not know that feature, which is harmless.
"""

import os
import shutil
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libtq.so")
BINDING = os.path.join(HERE, "_serving.so")
ARCH = "gfx950"

SOURCES = {
    "pack.hip": ["-ffp-contract=off"],
    "gemv.hip": [],
    "gemm.hip": [],
    "diag.hip": [],
    "paged.hip": [],
    "attention.hip": [],
    "sample.hip": [],
    "moe.hip": [],
    "experts.hip": [],
    "lora.hip": [],
    "api.cpp": ["-x", "hip"],
    "api_serving.cpp": ["-x", "hip"],
    "api_experts.cpp": ["-x", "hip"],
}


def _hipcc():
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (set HIPCC or install ROCm)")


def _binding_command():
    """The compile and link of _serving.so, or what it lacks here (a RuntimeError's text)."""
    import sysconfig
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        raise RuntimeError("no C++ compiler (g++ or c++)")
    try:
        import torch
        from torch.utils import cpp_extension
    except ImportError as e:
        raise RuntimeError(f"torch cannot be imported ({e})")
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    python = sysconfig.get_paths()["include"]
    system = cpp_extension.include_paths() + [os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "include")]
    for header in ("Python.h", "ATen/ATen.h", "c10/hip/HIPStream.h", "torch/csrc/autograd/python_variable.h"):
        if not any(os.path.exists(os.path.join(path, header)) for path in [python] + system):
            raise RuntimeError(f"no header {header}")
    cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall",
           "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", INCLUDE, "-I", python]
    for path in system:
        cmd += ["-isystem", path]
    return cmd + [os.path.join(CSRC, "binding.cpp"), "-o", BINDING + ".tmp", "-L", HERE, "-l:libtq.so", "-L", lib,
                  "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_hip", "-Wl,-rpath,$ORIGIN"]


def _build_binding():
    """Compile and link _serving.so beside libtq.so, which it needs.

    The library and its other calls do without it, so where its compiler or
    headers are missing the build goes on: the serving calls then raise, and
    one of an earlier build, for another library, is removed."""
    try:
        cmd = _binding_command()
    except RuntimeError as e:
        if os.path.exists(BINDING):
            os.remove(BINDING)
        print(f"_serving.so not built: {e}; the serving calls will not run, libtq.so is complete", file=sys.stderr)
        return
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    if r.returncode != 0:
        raise RuntimeError(f"_serving build failed: {' '.join(cmd)}\n" + r.stdout.decode(errors="replace"))
    os.replace(BINDING + ".tmp", BINDING)


def build(verbose: bool = False, jobs: int = 4) -> str:
    """Compile all sources and link libtq.so; returns the library path."""
    hipcc = _hipcc()
    common = [
        "-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}",
        "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
        "-I", INCLUDE, "-I", CSRC, "-Wall", "-Wno-unused-function",
    ]
    with tempfile.TemporaryDirectory(prefix="tq_build_") as tmp:
        procs = []
        objs = []
        for src, extra in SOURCES.items():
            obj = os.path.join(tmp, src.replace(".", "_") + ".o")
            cmd = [hipcc] + common + extra + ["-c", os.path.join(CSRC, src), "-o", obj]
            objs.append(obj)
            procs.append((src, cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
        failed = []
        for src, cmd, p in procs:
            out = p.communicate()[0].decode(errors="replace")
            lines = [ln for ln in out.splitlines() if "packed-fp32-ops" not in ln]
            if p.returncode != 0:
                failed.append((src, " ".join(cmd), "\n".join(lines)))
            elif verbose and lines:
                print(f"[{src}]\n" + "\n".join(lines))
        if failed:
            msg = "\n\n".join(f"{s}: {c}\n{o}" for s, c, o in failed)
            raise RuntimeError(f"libtq build failed:\n{msg}")
        tmp_lib = LIB + ".tmp"
        link = [hipcc, "-shared", "-fPIC", f"--offload-arch={ARCH}", "-o", tmp_lib] + objs
        r = subprocess.run(link, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
        if r.returncode != 0:
            raise RuntimeError("libtq link failed:\n" + r.stdout.decode(errors="replace"))
        os.replace(tmp_lib, LIB)
    _build_binding()
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
