"""Build libfme.so (the CUDA library behind include/fme.h) for sm_103a with nvcc, and
the compiled half of its Python binding (csrc/binding.cpp) with the host compiler.

Every translation unit is compiled in parallel, then linked into
``fp8_moe_expert_gb300/libfme.so`` (git-ignored, rebuilt on each machine: the
object code is architecture specific and the host code is built for the host
it runs on).  Usage: ``python -m fp8_moe_expert_gb300.build``.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
import tempfile
import warnings
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
LIBRARY = os.path.join(HERE, "libfme.so")
BINDING = os.path.join(HERE, "_binding.so")
BUILD_DIR = os.path.join(HERE, "_build")
SOURCES = ["api.cu", "quant_nvfp4.cu", "quant_mxfp8.cu", "gemm.cu", "gemm_nvfp4.cu", "route.cu",
           "quant_block128.cu", "gemm_block128.cu", "gemm_bf16.cu",
           "gemv_nvfp4.cu", "activation.cu", "gate.cu"]
HEADERS = ["fme_device.cuh", "fme_launch.h", "gemm_common.cuh", "block128.cuh", "gemm_tiles.cuh", "swiglu.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libfme.so")


def _inputs() -> list[str]:
    files = [os.path.join(CSRC, f) for f in SOURCES + HEADERS]
    files.append(os.path.join(ROOT, "include", "fme.h"))
    return files


def _older(output: str, inputs: list[str]) -> bool:
    if not os.path.exists(output):
        return True
    t = os.path.getmtime(output)
    return any(os.path.getmtime(f) > t for f in inputs)


def _binding_inputs() -> list[str]:
    return [os.path.join(CSRC, "binding.cpp"), os.path.join(ROOT, "include", "fme.h")]


def binding_target() -> str:
    """What a binding is built for: it is compiled against torch's headers and Python's."""
    import torch

    return f"torch {torch.__version__}, Python {sys.version_info[0]}.{sys.version_info[1]}"


def _binding_stale() -> bool:
    if _older(BINDING, _binding_inputs()):
        return True
    try:
        target = binding_target()
    except ImportError:  # no torch: there is nothing to bind for
        return False
    with open(BINDING, "rb") as f:  # a constant of the module (built_for)
        return target.encode() not in f.read()


def stale(output: str = LIBRARY) -> bool:
    return _older(output, _inputs()) or (output == LIBRARY and _binding_stale())


def _torch_dir() -> str:
    import torch

    return os.path.dirname(torch.__file__)


def _build_binding_object(obj: str, env: dict) -> None:
    """binding.cpp against the installed torch's headers (about 20 s)."""
    include = [os.path.join(_torch_dir(), "include"), sysconfig.get_paths()["include"],
               os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-DNDEBUG",
           f'-DFME_BUILT_FOR="{binding_target()}"', *(f"-I{p}" for p in include), "-c",
           os.path.join(CSRC, "binding.cpp"), "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True, env=env)
    if res.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed on binding.cpp:\n{res.stdout}\n{res.stderr}")


def _link_binding(obj: str, env: dict) -> None:
    tmp_out = BINDING + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-shared", "-o", tmp_out, obj, LIBRARY, "-Wl,-rpath,$ORIGIN",
           "-L" + os.path.join(_torch_dir(), "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda",
           "-ltorch_python"]
    res = subprocess.run(cmd, capture_output=True, text=True, env=env)
    if res.returncode != 0:
        raise RuntimeError(f"linking the binding failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp_out, BINDING)


def _without_binding(error: Exception) -> None:
    """The library serves the C ABI and the ctypes calls without the binding, which needs a host compiler and the
    headers of Python and torch; its own calls raise until it is built, so an outdated one is taken away."""
    if os.path.exists(BINDING):
        os.remove(BINDING)
    warnings.warn(f"the compiled binding was not built, the FP8 block-128, bf16, 4-bit and router calls will "
                  f"raise: {error}",
                  RuntimeWarning, stacklevel=3)


def build_binding() -> None:
    """Compile and link the binding to the package's library."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    with tempfile.TemporaryDirectory(prefix=f"{os.getpid()}_", dir=BUILD_DIR) as tmp:
        env = dict(os.environ, TMPDIR=tmp)
        obj = os.path.join(tmp, "binding.o")
        _build_binding_object(obj, env)
        _link_binding(obj, env)


def refresh() -> str:
    """Build what is missing or out of date of the library and the binding; returns the library's path."""
    if _older(LIBRARY, _inputs()):
        return build()
    if _binding_stale():
        try:
            build_binding()
        except (ImportError, OSError, RuntimeError) as e:
            _without_binding(e)
    return LIBRARY


def build(output: str = LIBRARY, extra_flags: list[str] | None = None, verbose: bool = False) -> str:
    """Compile and link the library (and, for the package's own, the binding); returns its path.  A binding that cannot
    be built is warned of: the library is in place then."""
    binding = output == LIBRARY and _binding_stale()
    flags = NVCC_FLAGS + (extra_flags or [])
    tool = nvcc()
    # objects and nvcc's own intermediates stay inside the package tree (git-ignored)
    os.makedirs(BUILD_DIR, exist_ok=True)
    with tempfile.TemporaryDirectory(prefix=f"{os.getpid()}_", dir=BUILD_DIR) as tmp:
        env = dict(os.environ, TMPDIR=tmp)

        def compile_one(src: str) -> str:
            obj = os.path.join(tmp, os.path.splitext(src)[0] + ".o")
            cmd = [tool, *ARCH, *flags, "-I", os.path.join(ROOT, "include"), "-c",
                   os.path.join(CSRC, src), "-o", obj]
            res = subprocess.run(cmd, capture_output=True, text=True, env=env)
            if res.returncode != 0:
                raise RuntimeError(f"nvcc failed on {src}:\n{res.stdout}\n{res.stderr}")
            if verbose:
                sys.stderr.write(res.stdout + res.stderr)
            return obj

        binding_obj = os.path.join(tmp, "binding.o")
        with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as pool:
            pending = pool.submit(_build_binding_object, binding_obj, env) if binding else None
            objs = list(pool.map(compile_one, SOURCES))
            failed = pending.exception() if pending else None
        tmp_out = output + ".tmp"
        # a soname of its own: the binding, linked to the package's library, must not be given another build of it
        # that the process loaded first
        cmd = [tool, *ARCH, "-shared", "-Xlinker", f"-soname={os.path.basename(output)}", "-o", tmp_out, *objs]
        res = subprocess.run(cmd, capture_output=True, text=True, env=env)
        if res.returncode != 0:
            raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
        os.replace(tmp_out, output)
        if binding:
            try:
                if failed:
                    raise failed
                _link_binding(binding_obj, env)
            except (ImportError, OSError, RuntimeError) as e:
                _without_binding(e)
    return output


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
