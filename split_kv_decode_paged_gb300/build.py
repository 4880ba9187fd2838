"""Build libfd.so (the CUDA library behind include/fd_api.h) in-tree with nvcc.

One -gencode (sm_103a), translation units compiled in parallel, then linked
into split_kv_decode_paged_gb300/libfd.so.  No cmake, no torch extension
machinery: the library is plain C ABI over the CUDA runtime.  Beside it the
host compiler builds _fd_torch.so (csrc/torch_binding.cpp), the native
marshalling of the calls made once a layer and step.
"""
import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libfd.so")
BINDING = os.path.join(HERE, "_fd_torch.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
SOURCES = ["fd_api.cu", "decode_f16.cu", "decode_bf16.cu", "decode_e4m3.cu", "decode_scores_f16.cu",
           "decode_scores_bf16.cu", "decode_scores_e4m3.cu", "decode_diff_f16.cu", "decode_diff_bf16.cu",
           "decode_diff_e4m3.cu", "decode_state_f16.cu", "decode_state_bf16.cu", "decode_state_e4m3.cu", "merge.cu", "append.cu",
           "append_norm.cu", "weights.cu", "evict.cu", "noalloc.cu", "rows.cu", "rows_api.cu"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(os.path.dirname(HERE), "include", "fd_api.h"))
    return files


def build_binding() -> str:
    """Compile _fd_torch.so against the installed torch; returns its path."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    cxx = os.environ.get("CXX") or shutil.which("g++") or "c++"
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    inc = cpp_extension.include_paths() + [cuda, sysconfig.get_paths()["include"]]
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    cmd += [a for i in inc for a in ("-isystem", i)] + [os.path.join(CSRC, "torch_binding.cpp"), "-o", tmp]
    cmd += [f"-L{d}" for d in cpp_extension.library_paths()] + ["-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cxx} failed for torch_binding.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    return BINDING


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Compile every CUDA source for sm_103a and link libfd.so, and the torch
    binding beside it; returns the library's path."""
    newest = max(os.path.getmtime(f) for f in _deps())
    fresh = [os.path.exists(f) and os.path.getmtime(f) >= newest for f in (LIB, BINDING)]
    if force or verbose_ptxas:
        fresh = [False, False]
    if not fresh[0]:
        _build_lib(verbose_ptxas, binding=not fresh[1])
    elif not fresh[1]:
        _try_binding()
    return LIB


def _try_binding() -> None:
    try:
        build_binding()
    except (RuntimeError, OSError) as e:
        # the calls it serves then go the Python way, which takes longer; an
        # older binding may have other structures than the library
        if os.path.exists(BINDING):
            os.remove(BINDING)
        print(f"warning: no native torch binding: {e}", file=sys.stderr)


def _build_lib(verbose_ptxas: bool, binding: bool) -> None:
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    common = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
                     "-I", os.path.join(os.path.dirname(HERE), "include")]
    if verbose_ptxas:
        common += ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = [cc] + common + ["-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    with cf.ThreadPoolExecutor(max_workers=min(len(SOURCES) + 1, os.cpu_count() or 4)) as ex:
        native = ex.submit(_try_binding) if binding else None
        results = list(ex.map(compile_one, SOURCES))
        if native:
            native.result()
    if verbose_ptxas:
        for _, log in results:
            sys.stderr.write(log)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [cc] + ARCH + ["-shared", "-o", tmp] + [o for o, _ in results]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
