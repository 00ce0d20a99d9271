"""Build of the CUDA library ``libmpgemm.so`` (in-tree, sm_103a only).

Every translation unit under ``csrc/`` is compiled by nvcc in parallel with
``-gencode arch=compute_103a,code=sm_103a`` and linked (static CUDA runtime)
into ``mixed_precision_matmul_gb300/_build/libmpgemm.so``; where torch and g++
are there, the marshalling extension of the torch forms is compiled beside it
(without it those calls are marshalled in Python).  The ptxas resource
report (``-Xptxas -v``: registers, spills, shared memory) of each unit is kept
in ``_build/ptxas.log``.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libmpgemm.so")
INCLUDE = os.path.join(ROOT, "include")

SOURCES = [
    "api.cu",
    "host_common.cu",
    "plan.cu",
    "host_api.cu",
    "attention_api.cu",
    "acc_layout.cpp",
    "aux_kernels.cu",
    "ffma.cu",
    "tc_direct.cu",
    "tc_staged.cu",
    "tc_generic.cu",
    "prepass.cu",
    "tc_pair.cu",
    "attention.cu",
    "tmem_probe.cu",
    "fp8_api.cu",
    "fp8_quant.cu",
    "fp8_gemm.cu",
    "fp8_pair.cu",
    "ortho_api.cu",
    "ortho.cu",
    "fused_plan.cu",
    "fused_plain.cu",
    "fused_gated.cu",
    "fused_gated_grad.cu",
    "fused_loss.cu",
    "few_rows.cu",
    "few_grad.cu",
    "fused_aux.cu",
    "gated_api.cu",
    "loss_api.cu",
    "clip.cu",
]
HEADERS = ["ptx.cuh", "cluster.cuh", "internal.h", "tc_gemm.cuh", "outio.cuh", "host.h", "staging.cuh",
           "fp8.h", "fp8_tc.cuh", "ortho.h", "fused.h", "fused.cuh", "fused_deal.h", "fused_gemm.cuh"]

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found; the CUDA toolkit is required to build libmpgemm")
    return cand


def _stale(target: str, deps: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src: str) -> tuple[str, str]:
    path = os.path.join(CSRC, src)
    obj = os.path.join(BUILD, src + ".o")
    deps = [path, os.path.join(INCLUDE, "mpgemm.h")] + [os.path.join(CSRC, h) for h in HEADERS]
    if not _stale(obj, deps):
        return obj, ""
    cmd = [_nvcc(), "-c", path, "-o", obj + ".tmp", "-std=c++17", "-O3", "-lineinfo",
           "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC] + ARCH
    if src.endswith(".cu"):
        cmd += ["-Xptxas", "-v", "--expt-relaxed-constexpr"]
    else:
        cmd += ["-x", "c++"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    os.replace(obj + ".tmp", obj)
    return obj, r.stderr


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile (when sources changed) and link libmpgemm.so; returns its path.
    The library needs nvcc alone; the marshalling extension of the torch forms
    is left out, with a warning, where it does not compile."""
    os.makedirs(BUILD, exist_ok=True)
    if force:
        for f in os.listdir(BUILD):
            if f.endswith(".o"):
                os.remove(os.path.join(BUILD, f))
    jobs = min(len(SOURCES) + 1, max(2, os.cpu_count() or 2))
    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        calls = ex.submit(build_torch_calls)
        results = list(ex.map(_compile, SOURCES))
    objs = [o for o, _ in results]
    logs = "".join(f"== {s}\n{log}" for s, (_, log) in zip(SOURCES, results) if log)
    if logs:
        with open(os.path.join(BUILD, "ptxas.log"), "w") as fh:
            fh.write(logs)
    if _stale(LIB, objs):
        tmp = LIB + f".{os.getpid()}.tmp"
        cmd = [_nvcc(), "-shared", "-o", tmp] + objs + ARCH + ["-cudart", "static"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    failure = calls.exception()
    if failure is not None and not isinstance(failure, ModuleNotFoundError):     # (no torch: nothing to marshal)
        warnings.warn(f"the torch forms' calls will be marshalled in Python: {failure}", RuntimeWarning)
    if verbose:
        print(f"built {LIB}", file=sys.stderr)
    return LIB


def torch_calls_path() -> str:
    """The marshalling extension, built for the torch and the Python that are running."""
    import sysconfig

    import torch
    return os.path.join(BUILD, f"_torch_calls-{torch.__version__}{sysconfig.get_config_var('EXT_SUFFIX') or '.so'}")


def build_torch_calls() -> str:
    """Compile csrc/torch_calls.cpp (host code only) against the installed torch."""
    import sysconfig

    import torch
    os.makedirs(BUILD, exist_ok=True)
    src, out = os.path.join(CSRC, "torch_calls.cpp"), torch_calls_path()
    if not _stale(out, [src, os.path.join(INCLUDE, "mpgemm.h")]):
        return out
    root = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include"), INCLUDE]
    tmp = out + f".{os.getpid()}.tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           src, "-o", tmp] + [f"-I{d}" for d in inc] + [f"-L{os.path.join(root, 'lib')}", "-ltorch_python", "-ltorch_cpu",
                                                       "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for torch_calls.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out)
    return out


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
