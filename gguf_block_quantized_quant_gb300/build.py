"""Builds libqg.so in-tree with nvcc for sm_103a (GB300), and the torch marshalling module beside it.

The CUDA sources are compiled in parallel: the C-ABI and decoder-layer translation units once, and
``qg_fmt.cu`` once per block format (``-DQG_FMT=<GGUF type id>``).  The library links the
shared CUDA runtime so that it shares the process's runtime state (current device,
streams) with PyTorch.  ``qg_torch.so`` (g++, against the installed torch's headers) is the Python
module that marshals torch tensors for the decoder-layer calls.  The library does not depend on it:
where it cannot be built, ``build()`` warns, and those calls say so when they are made.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(OUT_DIR, "libqg.so")
TORCH_MODULE = os.path.join(OUT_DIR, "qg_torch.so")
TORCH_STAMP = TORCH_MODULE + ".for"  # the torch and the Python that the module was built for

FORMATS = {"q4_0": 2, "q4_1": 3, "q5_0": 6, "q5_1": 7, "q8_0": 8, "q2_k": 10, "q3_k": 11, "q4_k": 12, "q5_k": 13,
           "q6_k": 14, "iq4_nl": 20, "iq4_xs": 23}
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    p = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(p):
        raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libqg")
    return p


def _cuda_lib_dir() -> str:
    nv = os.path.realpath(_nvcc())
    return os.path.join(os.path.dirname(os.path.dirname(nv)), "lib64")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")) +
                  glob.glob(os.path.join(CSRC, "*.h")) + [os.path.join(INCLUDE, "qg.h"), __file__])


def _torch_sources():
    return [os.path.join(CSRC, "qg_torch.cpp"), os.path.join(INCLUDE, "qg.h"), __file__]


def _flags(extra=()):
    return [*ARCH, "-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC,-O2",
            "-I", CSRC, "-I", INCLUDE, *extra]


def _units():
    units = [(os.path.join(CSRC, f"{u}.cu"), os.path.join(OUT_DIR, f"{u}.o"), []) for u in ("qg_chunk", "qg_attn", "qg_layer", "qg_abi")]
    for name, fid in FORMATS.items():
        units.append((os.path.join(CSRC, "qg_fmt.cu"), os.path.join(OUT_DIR, f"qg_fmt_{name}.o"),
                      [f"-DQG_FMT={fid}"]))
    return units


def _newer(out, sources) -> bool:
    return os.path.exists(out) and all(os.path.getmtime(s) <= os.path.getmtime(out) for s in sources)


def _torch_id() -> str:
    import torch
    return f"torch {torch.__version__}, {sys.implementation.cache_tag}"


def module_is_for() -> str | None:
    """The torch and Python that the module was built for (None: there is no module)."""
    if not (os.path.exists(TORCH_MODULE) and os.path.exists(TORCH_STAMP)):
        return None
    with open(TORCH_STAMP) as f:
        return f.read()


def up_to_date() -> bool:
    return _newer(LIB, _sources()) and _module_up_to_date()


def _module_up_to_date() -> bool:
    return _newer(TORCH_MODULE, _torch_sources()) and module_is_for() == _torch_id()


def _torch_commands(out):
    """Compile and link commands of the torch module (linked once libqg.so is there)."""
    import torch
    t = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    obj = os.path.join(OUT_DIR, "qg_torch.o")
    include = [os.path.join(t, "include"), os.path.join(t, "include", "torch", "csrc", "api", "include"),
               os.path.join(cuda, "include"), sysconfig.get_paths()["include"], INCLUDE]
    compile_cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-c", os.path.join(CSRC, "qg_torch.cpp"), "-o", obj,
                   f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f"-I{d}" for d in include)]
    link_cmd = ["g++", "-shared", "-o", out, obj, "-L", OUT_DIR, "-l:libqg.so", "-L", os.path.join(t, "lib"), "-lc10", "-lc10_cuda",
                "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-Wl,-rpath,$ORIGIN"]
    return compile_cmd, link_cmd


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stderr[-6000:]}")
    return r


def _build_lib(verbose, jobs):
    nvcc = _nvcc()

    def compile_one(u):
        src, obj, extra = u
        r = _run([nvcc, *_flags(extra), "-c", src, "-o", obj], f"nvcc for {os.path.basename(obj)}")
        if verbose and r.stderr.strip():
            print(r.stderr)
        return obj

    units = _units()
    workers = jobs or min(len(units), max(1, os.cpu_count() or 1))
    with cf.ThreadPoolExecutor(max_workers=workers) as ex:
        objs = list(ex.map(compile_one, units))
    tmp = LIB + f".tmp{os.getpid()}"
    _run([nvcc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs, "-Xlinker", f"-rpath,{_cuda_lib_dir()}"], "link of libqg.so")
    os.replace(tmp, LIB)


def _build_module(compiled, link_cmd, tmp):
    """Links the module once the library is there.  compiled: the future of its compilation."""
    try:
        compiled.result()
        _run(link_cmd, "link of qg_torch.so")
    except (RuntimeError, OSError) as e:
        for stale in (TORCH_MODULE, TORCH_STAMP):
            if os.path.exists(stale):
                os.remove(stale)
        warnings.warn(f"libqg.so is built, but not the module of the decoder-layer calls (qg_norm_residual, qg_rope_append, "
                      f"qg_attn_paged) for this torch; those calls will raise.  {e}", stacklevel=3)
        return
    os.replace(tmp, TORCH_MODULE)
    with open(TORCH_STAMP, "w") as f:
        f.write(_torch_id())


def build(force: bool = False, verbose: bool = False, jobs: int | None = None) -> str:
    """Compile (if needed) and return the path of libqg.so."""
    lib = force or not _newer(LIB, _sources())
    module = force or not _module_up_to_date()
    os.makedirs(OUT_DIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        if module:
            tmp = TORCH_MODULE + f".tmp{os.getpid()}"
            compile_cmd, link_cmd = _torch_commands(tmp)
            compiled = ex.submit(_run, compile_cmd, "g++ for qg_torch.o")
        if lib:
            _build_lib(verbose, jobs)
        if module:
            _build_module(compiled, link_cmd, tmp)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
