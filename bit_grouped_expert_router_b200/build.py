"""In-tree build of libmoe.so (the CUDA library behind include/moe.h) for sm_100a, and of its torch module.

Each .cu file compiles to an object in parallel; the objects link into one shared library with
the CUDA runtime linked statically, so loading the library needs no GPU driver (symbols can be
inspected on a machine without a GPU; the first CUDA call needs one).

_torch_ops is the Python module behind ops.py (csrc/torch_ops.cpp: torch tensors in, libmoe calls out);
it compiles against the installed torch and links to the libmoe.so next to it.  Its file's name has Python's tag, and it
holds the version of torch, so another Python or torch gets one of its own.  The library stands without it: where
there is no torch the module is left out, and where it does not compile a warning says why (ops.py then fails at its first
call).
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libmoe.so")
EXT = os.path.join(PKG, "_torch_ops" + sysconfig.get_config_var("EXT_SUFFIX"))
SOURCES = ["api.cu", "repack.cu", "route.cu", "router_tc.cu", "gemm.cu", "decode.cu", "decode_fused.cu", "route_static.cu",
           "ops_api.cu", "rows.cu", "norm.cu", "mx4.cu"]
NVCC_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
              "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden", "-I", INCLUDE]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


EXT_SOURCE = "torch_ops.cpp"


def _newer(target: str, sources) -> bool:
    files = [os.path.join(CSRC, f) for f in sources] + [os.path.join(INCLUDE, "moe.h"), os.path.abspath(__file__)]
    return os.path.exists(target) and all(os.path.getmtime(f) <= os.path.getmtime(target) for f in files)


def _has_torch() -> bool:
    try:
        import torch  # noqa: F401
    except ImportError:
        return False
    return True


def _lib_up_to_date() -> bool:
    return _newer(LIB, [f for f in os.listdir(CSRC) if f != EXT_SOURCE])


def built_for() -> str:
    """What the module is compiled against, as it says itself (``_torch_ops.built_for``)."""
    import torch
    return f"torch {torch.__version__}"


def _ext_up_to_date() -> bool:
    if not _has_torch():
        return True
    if not _newer(EXT, [EXT_SOURCE]):
        return False
    with open(EXT, "rb") as f:
        return built_for().encode() + b"\0" in f.read()


def up_to_date() -> bool:
    return _lib_up_to_date() and _ext_up_to_date()


# The decode GEMVs feed 4-bit codes to fp32 FMAs as IEEE subnormals (code * 2^-149, see
# csrc/decode.cu); those FMAs are written as explicit fma.rn.f32 in inline PTX so they keep
# subnormals whatever the compiler flags say, and flush-to-zero builds are refused here as well so
# no other arithmetic silently changes either.
FORBIDDEN_FLAGS = ("-ftz=true", "--ftz=true", "--use_fast_math", "-use_fast_math")


def check_flags(flags) -> None:
    bad = [f for f in flags if f in FORBIDDEN_FLAGS]
    if bad:
        raise ValueError(f"libmoe must be built without flush-to-zero / fast math (got {bad})")


# The system's g++, whatever $CXX names: the module must share the libstdc++ that torch has loaded (with one
# linked in statically, its first C++ exception ends the process).
HOST_CXX = "/usr/bin/g++" if os.path.exists("/usr/bin/g++") else "g++"


def _compile_ext(obj: str) -> None:
    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    cmd = [HOST_CXX, "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", f'-DMOE_BUILT_FOR="{built_for()}"',
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", sysconfig.get_paths()["include"],
           "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", cuda,
           "-c", os.path.join(CSRC, EXT_SOURCE), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{EXT_SOURCE} failed:\n{r.stdout}\n{r.stderr}")


def _link_ext(obj: str) -> None:
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = EXT + ".tmp"
    old = os.path.join(PKG, "_torch_ops.so")   # an earlier build's, without the tag: any Python would find it
    if os.path.exists(old):
        os.remove(old)
    cmd = [HOST_CXX, "-shared", obj, "-o", tmp, "-L", PKG, "-l:libmoe.so", "-L", lib, "-ltorch_python",
           "-ltorch_cuda", "-ltorch_cpu", "-ltorch", "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of _torch_ops failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, EXT)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    check_flags(list(NVCC_FLAGS) + list(extra_flags))
    want_lib, want_ext = force or not _lib_up_to_date(), _has_torch() if force else not _ext_up_to_date()
    if not want_lib and not want_ext:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc, *NVCC_FLAGS, *extra_flags, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and r.stderr:
            print(r.stderr, file=sys.stderr)
        return obj

    ext_obj = os.path.join(BUILD, EXT_SOURCE + ".o")
    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        ext = ex.submit(_compile_ext, ext_obj) if want_ext else None
        if want_lib:
            objs = list(ex.map(compile_one, SOURCES))
            tmp = LIB + ".tmp"
            cmd = [nvcc, "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-cudart", "static",
                   "-Xcompiler", "-fPIC", "-o", tmp, *objs]
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
            os.replace(tmp, LIB)
    if ext:
        try:
            ext.result()
            _link_ext(ext_obj)
        except RuntimeError as e:
            if os.path.exists(EXT):
                os.remove(EXT)   # of an older source: it must not pass for this one's
            warnings.warn(f"libmoe is built, _torch_ops is not: {e}", RuntimeWarning, stacklevel=2)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
