"""Builds libmoe_gb300.so in-tree with nvcc for sm_103a (no torch extension
machinery: the library is plain C ABI + CUDA), and beside it _moe_torch.so, the
compiled PyTorch binding of the handle-less operators (host code only; left out
where there is no PyTorch)."""
from __future__ import annotations

import os
import shutil
import subprocess
from pathlib import Path

PKG = Path(__file__).resolve().parent
ROOT = PKG.parent
CSRC = PKG / "csrc"
BUILD = PKG / "_build"
LIB = PKG / "libmoe_gb300.so"
BINDING = PKG / "_moe_torch.so"
KEY = "moe_torch.key"          # in BUILD: what the binding was built for
SOURCES = ["moe_kernels.cu", "moe_decode.cu", "moe_fp8.cu", "moe_route_ops.cu", "moe_abi.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and Path(cand).exists():
            return cand
    raise RuntimeError("nvcc not found")


def _stale(target: Path, deps) -> bool:
    if not target.exists():
        return True
    t = target.stat().st_mtime
    return any(Path(d).stat().st_mtime > t for d in deps)


def binding_key() -> str | None:
    """What the compiled binding depends on beside its sources: PyTorch's C++ interface has no stable ABI, nor
    has Python's.  None without a PyTorch that has CUDA: the C library alone is built then."""
    import sysconfig
    try:
        import torch
    except ImportError:
        return None
    root = Path(torch.__file__).resolve().parent
    if not (root / "lib" / "libc10_cuda.so").exists():
        return None
    return f"torch {torch.__version__} at {root}, C++11 ABI {int(torch._C._GLIBCXX_USE_CXX11_ABI)}, {sysconfig.get_config_var('SOABI')}"


def binding_built_for() -> str | None:
    """The key that the binding in the tree was built for."""
    key = BUILD / KEY
    return key.read_text() if BINDING.exists() and key.exists() else None


def _binding_command(obj: Path) -> list[str]:
    """Compiles the binding's object: g++ on PyTorch's and Python's headers."""
    import sysconfig
    import torch
    inc = Path(torch.__file__).resolve().parent / "include"
    cuda = Path(nvcc()).resolve().parent.parent / "include"
    dirs = [ROOT / "include", sysconfig.get_paths()["include"], inc, inc / "torch/csrc/api/include", cuda]
    return ["g++", "-std=c++17", "-O2", "-fPIC", "-fvisibility=hidden", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *[a for d in dirs for a in ("-isystem", str(d))], "-c", str(CSRC / "moe_torch.cpp"), "-o", str(obj)]


def _link_binding(obj: Path, key: str) -> None:
    import torch
    libs = Path(torch.__file__).resolve().parent / "lib"
    tmp = BINDING.with_suffix(".so.tmp%d" % os.getpid())
    (BUILD / KEY).unlink(missing_ok=True)
    subprocess.run(["g++", "-shared", "-o", str(tmp), str(obj), f"-L{libs}", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda",
                    f"-L{PKG}", f"-l:{LIB.name}", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{libs}"], check=True)
    os.replace(tmp, BINDING)
    (BUILD / KEY).write_text(key)


def build_library(force: bool = False, verbose: bool = False) -> Path:
    headers = list(CSRC.glob("*.h")) + list((ROOT / "include").glob("*.h"))
    BUILD.mkdir(exist_ok=True)
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
                    "-I", str(ROOT / "include"), "-I", str(CSRC)]
    if verbose:
        flags += ["-Xptxas", "-v"]
    procs, objs, errors = [], [], []

    def start(command: list[str], tmp: Path, obj: Path) -> None:
        procs.append((subprocess.Popen(command, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True), tmp, obj))

    try:
        for src in SOURCES:
            obj = BUILD / (Path(src).stem + ".o")
            objs.append(obj)
            if force or _stale(obj, [CSRC / src] + headers):
                tmp = obj.with_suffix(".o.tmp%d" % os.getpid())
                start([nvcc(), *flags, "-c", str(CSRC / src), "-o", str(tmp)], tmp, obj)
        binding, key = BUILD / "moe_torch.o", binding_key()
        other = key is not None and binding_built_for() != key      # also: not linked yet
        if key is None:
            print("no PyTorch with CUDA: building the C library alone, without the binding of the operators on tensors")
        elif force or other or _stale(binding, [CSRC / "moe_torch.cpp", ROOT / "include" / "moe.h"]):
            tmp = binding.with_suffix(".o.tmp%d" % os.getpid())
            start(_binding_command(tmp), tmp, binding)
    finally:
        for proc, tmp, obj in procs:      # each that was started is waited for, whatever became of the others
            out, _ = proc.communicate()
            if proc.returncode != 0:
                errors.append(out)
            else:
                os.replace(tmp, obj)
                if verbose and out:
                    print(out)
    if errors:
        raise RuntimeError("compilation failed:\n" + "\n".join(errors))
    if force or _stale(LIB, objs):
        tmp = LIB.with_suffix(".so.tmp%d" % os.getpid())
        subprocess.run([nvcc(), *ARCH, "-shared", "-o", str(tmp), *map(str, objs)], check=True)
        os.replace(tmp, LIB)
    if key is not None and (force or other or _stale(BINDING, [binding, LIB])):
        _link_binding(binding, key)
    return LIB


if __name__ == "__main__":
    import sys
    build_library(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
