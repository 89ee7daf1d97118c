"""Build step for the CUDA library ``libgemm_tn.so`` (sm_103a only) and the
extension modules ``_kv_cache`` (the paged cache) and ``_feed_forward``.

Each translation unit under ``csrc/`` is compiled by nvcc in parallel with one
``-gencode arch=compute_103a,code=sm_103a`` and linked into a shared object in
this package directory. Objects go to ``_build/`` at the repository root.
The CUDA runtime is linked statically, so the library only needs the driver.
The extension modules are a C++ file each over torch's headers (g++), compiled at
the same time. The library needs none of them: without a torch that has CUDA, or
where a module does not compile, it is there all the same.

    python -m dense_tiled_gemm_03_gb300.build [--force] [--ptxas-verbose]
"""
from __future__ import annotations

import argparse
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor
from pathlib import Path

PKG = Path(__file__).resolve().parent
ROOT = PKG.parent
CSRC = PKG / "csrc"
INCLUDE = ROOT / "include"
BUILD_DIR = ROOT / "_build" / "gemm_tn"
LIBRARY = PKG / "libgemm_tn.so"
BINDING_SOURCE = CSRC / "kv_cache_py.cpp"
BINDING = PKG / ("_kv_cache" + sysconfig.get_config_var("EXT_SUFFIX"))
FF_SOURCE = CSRC / "feed_forward_py.cpp"
FF_BINDING = PKG / ("_feed_forward" + sysconfig.get_config_var("EXT_SUFFIX"))

SOURCES = ["gemm_tn_api.cu", "sm103_gemm_1cta.cu", "sm103_gemm_2cta.cu", "sm103_gemm_nn.cu", "sm103_gemm_fused.cu",
           "sm103_flash_attn.cu", "repack.cu", "sm103_gemm_splitk.cu", "sm103_tree_attn.cu", "sm103_decode_attn.cu",
           "sm103_cache_weigh.cu",
           "kv_cache_ops.cu", "kv_cache_api.cu",
           "sm103_ff_gated.cu", "sm103_ff_nt.cu", "sm103_ff_e4m3.cu", "sm103_ff_skinny.cu", "ff_ops.cu", "ff_api.cu"]
GENCODE = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC",
              "-Xcompiler", "-fvisibility=hidden", "-I", str(INCLUDE), "-I", str(CSRC)]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not Path(cand).exists():
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libgemm_tn.so")
    return cand


def _inputs() -> list[Path]:
    files = [CSRC / s for s in SOURCES]
    files += sorted(CSRC.glob("*.cuh")) + sorted(CSRC.glob("*.h")) + sorted(INCLUDE.glob("*.h"))
    return files + [Path(__file__)]


def is_stale() -> bool:
    if not LIBRARY.exists():
        return True
    built = LIBRARY.stat().st_mtime
    return any(p.stat().st_mtime > built for p in _inputs())


def torch_version(torch_dir: Path) -> str:
    """The version that the torch there states of itself (torch.__version__)."""
    return re.search(r"""^__version__\s*=\s*['"]([^'"]+)""", (torch_dir / "version.py").read_text(), re.MULTILINE).group(1)


def _binding_stamp() -> Path:
    return BUILD_DIR / "binding_torch.txt"


def _ff_stamp() -> Path:
    return BUILD_DIR / "ff_binding_torch.txt"


def _is_stale(module: Path, source: Path, stamp: Path, torch_dir: Path) -> bool:
    """Whether a module is missing, older than its sources, or built against another torch."""
    if not module.exists() or not stamp.exists():
        return True
    if stamp.read_text() != f"{torch_dir} {torch_version(torch_dir)}":
        return True
    inputs = [source, CSRC / "py_args.h", Path(__file__), *INCLUDE.glob("*.h")]
    return any(p.stat().st_mtime > module.stat().st_mtime for p in inputs)


def binding_is_stale(torch_dir: Path) -> bool:
    """_is_stale of the paged cache's module."""
    return _is_stale(BINDING, BINDING_SOURCE, _binding_stamp(), torch_dir)


def ff_binding_is_stale(torch_dir: Path) -> bool:
    """_is_stale of the feed-forward operators' module."""
    return _is_stale(FF_BINDING, FF_SOURCE, _ff_stamp(), torch_dir)


def torch_dir() -> Path | None:
    """Where the installed torch lies (found, not imported); None for no torch, or one without CUDA."""
    spec = importlib.util.find_spec("torch")
    found = Path(spec.submodule_search_locations[0]) if spec is not None and spec.submodule_search_locations else None
    return found if found is not None and (found / "lib" / "libc10_cuda.so").exists() else None


def _build_module(module: Path, source: Path, stamp: Path, torch_dir: Path) -> Path:
    cuda = Path(nvcc()).resolve().parent.parent
    tmp = module.with_name(f".{module.name}.{os.getpid()}")
    version = torch_version(torch_dir)
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", str(source), "-o", str(tmp),
           f'-DBUILT_AGAINST_TORCH="{version}"',
           "-I", str(INCLUDE), "-I", str(CSRC), "-I", str(torch_dir / "include"), "-I", sysconfig.get_paths()["include"],
           "-I", str(cuda / "include"), "-L", str(torch_dir / "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed for {source.name}:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, module)
    stamp.parent.mkdir(parents=True, exist_ok=True)
    stamp.write_text(f"{torch_dir} {version}")
    return module


def build_binding(torch_dir: Path) -> Path:
    """Compile the paged cache's module against that torch."""
    return _build_module(BINDING, BINDING_SOURCE, _binding_stamp(), torch_dir)


def build_ff_binding(torch_dir: Path) -> Path:
    """Compile the feed-forward operators' module against that torch."""
    return _build_module(FF_BINDING, FF_SOURCE, _ff_stamp(), torch_dir)


def _compile(src: Path, obj: Path, verbose_ptxas: bool) -> None:
    cmd = [nvcc(), *GENCODE, *NVCC_FLAGS, "-c", str(src), "-o", str(obj)]
    if verbose_ptxas:
        cmd += ["-Xptxas", "-v"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src.name}:\n{res.stdout}\n{res.stderr}")
    if verbose_ptxas and (res.stdout or res.stderr):
        sys.stderr.write(res.stdout + res.stderr)


def _link(objs: list[Path]) -> None:
    tmp = LIBRARY.with_name(f".libgemm_tn.{os.getpid()}.so")
    cmd = [nvcc(), *GENCODE, "-shared", "-Xcompiler", "-fPIC", *map(str, objs), "-o", str(tmp)]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIBRARY)


def build(force: bool = False, verbose_ptxas: bool = False) -> Path:
    """Compile and link libgemm_tn.so and the bindings if a source changed (or if forced). Returns the library's path."""
    all_of_it = force or verbose_ptxas
    torch = torch_dir()
    if torch is None:
        sys.stderr.write("no torch with CUDA found: the Python bindings of the paged cache and the feed-forward operators are not built\n")
    with ThreadPoolExecutor(max_workers=len(SOURCES) + 2) as pool:
        bindings = []
        if torch is not None and (all_of_it or binding_is_stale(torch)):
            bindings.append(pool.submit(build_binding, torch))
        if torch is not None and (all_of_it or ff_binding_is_stale(torch)):
            bindings.append(pool.submit(build_ff_binding, torch))
        if all_of_it or is_stale():
            BUILD_DIR.mkdir(parents=True, exist_ok=True)
            objs = [BUILD_DIR / (Path(s).stem + ".o") for s in SOURCES]
            list(pool.map(lambda so: _compile(CSRC / so[0], so[1], verbose_ptxas), zip(SOURCES, objs)))
            _link(objs)
        for binding in bindings:
            binding.result()
    return LIBRARY


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--ptxas-verbose", action="store_true")
    ns = ap.parse_args()
    print(build(force=ns.force, verbose_ptxas=ns.ptxas_verbose))
