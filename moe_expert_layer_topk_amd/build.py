"""Build libmoe.so (all HIP sources, gfx950) in place with hipcc, and the
Python module _marshal.so (argument marshalling, host code) beside it."""
import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libmoe.so")
MARSHAL = os.path.join(HERE, "_marshal.so")
BUILD = os.path.join(ROOT, "_build")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"
FLAGS = ["-O3", "-fPIC", "-std=c++17", f"--offload-arch={ARCH}",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-Wno-unused-result", "-I" + os.path.join(ROOT, "include")]


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".hip"))


def _compile(src):
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [HIPCC, *FLAGS, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    err = "\n".join(ln for ln in (r.stderr or "").splitlines() if "packed-fp32-ops" not in ln)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{err}")
    return obj, err


def _compile_marshal():
    """Object file of the marshalling module and the directory of torch's libraries."""
    import torch
    tdir = os.path.dirname(torch.__file__)
    rocm = os.path.dirname(os.path.dirname(HIPCC))
    obj = os.path.join(BUILD, "marshal.cpp.o")
    cmd = ["g++", "-O2", "-fPIC", "-std=c++17", "-DUSE_ROCM", "-D__HIP_PLATFORM_AMD__",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I" + os.path.join(tdir, "include"), "-I" + os.path.join(tdir, "include", "torch", "csrc", "api", "include"),
           "-I" + sysconfig.get_paths()["include"], "-I" + os.path.join(rocm, "include"), "-w",
           "-c", os.path.join(CSRC, "marshal.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for marshal.cpp:\n{r.stderr}")
    return obj, os.path.join(tdir, "lib")


def _link(cmd, out):
    tmp = out + ".tmp"
    subprocess.run([*cmd, "-o", tmp], check=True)
    os.replace(tmp, out)


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        marshal = ex.submit(_compile_marshal)
        results = list(ex.map(_compile, sources()))
        mobj, tlib = marshal.result()
    for _, err in results:
        if verbose and err.strip():
            print(err, file=sys.stderr)
    _link([HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-Wl,-soname,libmoe.so", *[o for o, _ in results]], LIB)
    _link(["g++", "-shared", "-fPIC", mobj, LIB, "-L" + tlib, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_hip", "-lc10",
           "-lc10_hip", "-Wl,-rpath,$ORIGIN"], MARSHAL)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
