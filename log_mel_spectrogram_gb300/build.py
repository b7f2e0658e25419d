"""Builds liblogmel.so, the library's C-ABI shared object, in-tree.

Each ``csrc/*.cu`` file is compiled by nvcc for sm_103a in parallel, then
linked into ``log_mel_spectrogram_gb300/_build/liblogmel.so``.  The build is
skipped when the library is newer than every source and header.

The torch binding of the decoding operations and layers, ``csrc/*.cpp``, becomes the
Python module ``_build/_decode.so`` beside it (g++, torch's headers), linked
against liblogmel.so.

``build(checked=True)`` makes the bounds-checked debug variant
``_build/checked/liblogmel_checked.so`` (-DLOGMEL_CHECKED): the same sources
with every computed global-memory index of the STFT and waveform kernels tested
against its buffer (the decoding kernels carry no such tests).
"""
from __future__ import annotations

import concurrent.futures
import os
import pathlib
import shutil
import subprocess
import sysconfig

PKG = pathlib.Path(__file__).resolve().parent
ROOT = PKG.parent
CSRC = PKG / "csrc"
INCLUDE = ROOT / "include"
OUT_DIR = PKG / "_build"
LIB = OUT_DIR / "liblogmel.so"
BINDING = OUT_DIR / "_decode.so"
CHECKED_DIR = OUT_DIR / "checked"
CHECKED_LIB = CHECKED_DIR / "liblogmel_checked.so"

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "--expt-relaxed-constexpr",
              f"-I{INCLUDE}", f"-I{CSRC}"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build liblogmel.so")
    return cand


def sources() -> list[pathlib.Path]:
    return sorted(CSRC.glob("*.cu"))


def _stale(lib: pathlib.Path = LIB) -> bool:
    if not lib.exists() or (lib == LIB and not BINDING.exists()):
        return True
    t = lib.stat().st_mtime
    deps = sources() + list(CSRC.glob("*.cpp")) + list(CSRC.glob("*.cuh")) + list(CSRC.glob("*.h")) + list(INCLUDE.glob("*.h"))
    deps.append(pathlib.Path(__file__))
    return any(d.stat().st_mtime > t for d in deps)


def _torch_dir() -> pathlib.Path:
    import torch
    return pathlib.Path(torch.__file__).resolve().parent


def _compile_binding(src: pathlib.Path, verbose: bool) -> pathlib.Path:
    """A source of the binding against torch's headers."""
    inc = _torch_dir() / "include"
    cuda = pathlib.Path(_nvcc()).resolve().parents[1] / "include"
    obj = OUT_DIR / (src.stem + ".binding.o")
    cmd = ["g++", "-std=c++17", "-O2", "-fPIC", "-fvisibility=hidden", f"-I{INCLUDE}",
           f"-I{sysconfig.get_path('include')}", "-isystem", str(inc), "-isystem",
           str(inc / "torch" / "csrc" / "api" / "include"), "-isystem", str(cuda), "-c", str(src),
           "-o", str(obj)]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {src.name}:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_binding(objs: list[pathlib.Path]) -> None:
    lib = _torch_dir() / "lib"
    cuda = pathlib.Path(_nvcc()).resolve().parents[1] / "lib64"
    tmp = OUT_DIR / f"_decode.{os.getpid()}.so"
    cmd = ["g++", "-shared", "-o", str(tmp), *map(str, objs), f"-L{lib}", "-ltorch_python", "-ltorch_cpu", "-lc10_cuda",
           "-lc10", f"-L{OUT_DIR}", "-l:liblogmel.so", f"-L{cuda}", "-lcudart", f"-Wl,-rpath,{lib}",
           "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{cuda}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of the binding failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False,
          checked: bool = False) -> pathlib.Path:
    """Compile and link liblogmel.so (or, with checked=True, the bounds-checked
    variant); returns its path."""
    lib, out_dir = (CHECKED_LIB, CHECKED_DIR) if checked else (LIB, OUT_DIR)
    if not force and not _stale(lib):
        return lib
    out_dir.mkdir(parents=True, exist_ok=True)
    nvcc = _nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_verbose else []
    if checked:
        extra.append("-DLOGMEL_CHECKED")

    def compile_one(src: pathlib.Path) -> pathlib.Path:
        obj = out_dir / (src.stem + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *extra, "-c", str(src), "-o", str(obj)]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src.name}:\n{r.stdout}\n{r.stderr}")
        if (verbose or ptxas_verbose) and r.stderr:
            print(r.stderr, flush=True)
        return obj

    bindings = [] if checked else sorted(CSRC.glob("*.cpp"))
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(sources()) + len(bindings)) as ex:
        binding = [ex.submit(_compile_binding, src, verbose) for src in bindings]
        objs = list(ex.map(compile_one, sources()))
    tmp = out_dir / f"{lib.stem}.{os.getpid()}.so"
    # (No soname: a program that links the library by its path then finds it there.)
    cmd = [nvcc, *ARCH, "-shared", "-o", str(tmp), *map(str, objs)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    if binding:
        _link_binding([b.result() for b in binding])
    return lib


if __name__ == "__main__":
    import sys
    build(force="--force" in sys.argv, verbose=True, ptxas_verbose="--ptxas" in sys.argv)
    print(LIB)
