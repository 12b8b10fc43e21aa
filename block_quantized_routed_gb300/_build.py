"""In-tree build of the CUDA library (sm_103a) with nvcc: every .cu file in
csrc/ is compiled in parallel, then linked into _build/libmoe_q8k.so; beside
it the host compiler builds the tensor binding (csrc/binding.cpp) against
torch's headers into _build/moe_binding.so.  The library is C and needs no
torch: without it the binding alone is left out."""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libmoe_q8k.so")
BINDING = os.path.join(BUILD, "moe_binding.so")
INCLUDE = os.path.join(ROOT, "include")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I" + INCLUDE, "-I" + CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build block_quantized_routed_gb300")


def _sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps():
    files = _sources() + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h", ".cpp"))]
    files.append(os.path.join(INCLUDE, "moe_q8k.h"))
    return files


def _has_torch() -> bool:
    import importlib.util
    import sys
    if "torch" in sys.modules:
        return sys.modules["torch"] is not None
    return importlib.util.find_spec("torch") is not None


def up_to_date() -> bool:
    made = [LIB, BINDING] if _has_torch() else [LIB]
    if not all(os.path.exists(f) for f in made):
        return False
    t = min(os.path.getmtime(f) for f in made)
    return all(os.path.getmtime(f) <= t for f in _deps())


def _binding_commands(out: str):
    """Compile and link commands of csrc/binding.cpp; the link needs LIB."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    inc = [INCLUDE, os.path.join(cuda, "include"), sysconfig.get_paths()["include"], *cpp_extension.include_paths()]
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    obj = os.path.join(BUILD, "binding.o")
    cxx = os.environ.get("CXX") or shutil.which("g++") or "g++"
    return ([cxx, "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
             *["-I" + i for i in inc], "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj],
            [cxx, "-shared", "-o", out, obj, "-L" + BUILD, "-l:libmoe_q8k.so", "-L" + lib, "-lc10", "-lc10_cuda",
             "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN"])


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")
    return r


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    srcs = _sources()
    objs = [os.path.join(BUILD, os.path.basename(s)[:-3] + ".o") for s in srcs]

    def compile_one(pair):
        src, obj = pair
        cmd = [cc, *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and r.stderr:
            print(r.stderr)
        return obj

    btmp = BINDING + f".tmp{os.getpid()}"

    def compile_binding():
        if not _has_torch():
            return None
        bind_compile, bind_link = _binding_commands(btmp)
        _run(bind_compile, "the compilation of csrc/binding.cpp")
        return bind_link

    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 1))) as ex:
        bound = ex.submit(compile_binding)
        list(ex.map(compile_one, zip(srcs, objs)))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    bind_link = bound.result()  # (the library is there whatever becomes of the binding)
    if bind_link:
        _run(bind_link, "the link of the binding")
        os.replace(btmp, BINDING)
    return LIB


def header_functions() -> list[str]:
    """Names of the functions declared in include/moe_q8k.h."""
    import re
    src = open(os.path.join(INCLUDE, "moe_q8k.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    return re.findall(r"^\s*(?:const\s+)?[A-Za-z_][A-Za-z0-9_]*\s*\*?\s*(moe_[a-z0-9_]+)\s*\(", src, flags=re.M)
