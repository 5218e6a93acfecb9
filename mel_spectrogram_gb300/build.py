"""Ahead-of-time build of libfm_mel.so for sm_103a with nvcc.

Each translation unit compiles in its own nvcc process (in parallel), then
the objects are linked into ``mel_spectrogram_gb300/libfm_mel.so`` beside this
file. Rebuilds only what changed (source or header newer than the object).
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libfm_mel.so")
# the debug build (every guarded access index-checked, see FM_IN in fm_internal.h)
BUILD_CHECK = os.path.join(PKG, "_build_check")
LIB_CHECK = os.path.join(PKG, "libfm_mel_check.so")
CHECK_FLAGS = ["-DFM_BOUNDS_CHECK"]
# the operators as functions on tensors: one C++ file against torch's headers,
# linked to libfm_mel.so beside it
TORCH_SRC = os.path.join(CSRC, "torch", "fm_torch.cpp")
TORCH_LIB = os.path.join(PKG, "_fm_torch.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
COMMON = ["-O3", "-std=c++17", "-lineinfo", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC,-O2",
          f"-I{INCLUDE}", f"-I{CSRC}"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libfm_mel.so")


def _sources(build_dir: str = BUILD) -> list[str]:
    found = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))
    if build_dir == BUILD_CHECK:  # the frame-encoder operators have no index-checked build
        found = [f for f in found if not os.path.basename(f).startswith("fm_ops_")]
    return found


def _weight(src: str) -> int:
    """A rough compile time: the attention kernels and the unrolled transforms
    take longest."""
    name = os.path.basename(src)
    return 2 if "_attn_" in name else 1 if "odd" in name or "hops" in name or "longhop" in name else 0


def _headers() -> list[str]:
    return glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(
        os.path.join(INCLUDE, "*.h"))


def _obj(src: str, build_dir: str = BUILD) -> str:
    return os.path.join(build_dir, os.path.basename(src) + ".o")


def _stale(target: str, deps: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src: str, extra: list[str], build_dir: str = BUILD) -> str:
    out = _obj(src, build_dir)
    cmd = [nvcc(), *ARCH, *COMMON, *extra, "-c", src, "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return r.stderr


def _torch_identity() -> str:
    """What the binding is built against: torch's place and version (without
    importing it) and Python's; "" where torch is not installed."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.origin:
        return ""
    with open(os.path.join(os.path.dirname(spec.origin), "version.py")) as f:
        return "\n".join([spec.origin, sys.version, f.read()])


def _torch_stale(out: str, identity: str) -> bool:
    """Whether the binding's object is missing, older than its sources or built
    against another torch."""
    try:
        with open(out + ".torch") as f:
            built = f.read()
    except OSError:
        return True
    return built != identity or _stale(out, [TORCH_SRC, *_headers(), __file__])


def _compile_torch() -> str:
    """The object of fm_torch.cpp; "" where torch is not installed."""
    identity = _torch_identity()
    if not identity:
        return ""
    out = os.path.join(BUILD, "fm_torch.cpp.o")
    if not _torch_stale(out, identity):
        return out
    import torch

    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           f"-I{INCLUDE}", f"-isystem{inc}", f"-isystem{os.path.join(inc, 'torch', 'csrc', 'api', 'include')}",
           f"-isystem{cuda}", f"-isystem{sysconfig.get_paths()['include']}", "-c", TORCH_SRC, "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for fm_torch.cpp:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    with open(out + ".torch", "w") as f:
        f.write(identity)
    return out


def _link_torch(obj: str) -> None:
    if not _stale(TORCH_LIB, [obj, LIB]):
        return
    libs = os.path.join(os.path.dirname(importlib.util.find_spec("torch").origin), "lib")
    tmp = TORCH_LIB + ".tmp"
    cmd = ["g++", "-shared", "-o", tmp, obj, f"-L{PKG}", "-l:libfm_mel.so", f"-L{libs}", "-lc10", "-lc10_cuda",
           "-ltorch_cpu", "-ltorch", "-ltorch_python", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{libs}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, TORCH_LIB)


def build(verbose: bool = False, extra: list[str] | None = None, jobs: int | None = None,
          check: bool = False) -> str:
    """Compile and link libfm_mel.so (check=True: the index-checked debug
    build libfm_mel_check.so, in its own object directory); returns its path."""
    return build_many([check], verbose, extra, jobs)[0]


def build_many(checks: list[bool], verbose: bool = False, extra: list[str] | None = None,
               jobs: int | None = None) -> list[str]:
    """Build several of the libraries (release / debug) in one pool of nvcc
    processes; returns their paths in order."""
    extra = list(extra or [])
    hdrs = _headers()
    targets = [(BUILD_CHECK, LIB_CHECK, extra + CHECK_FLAGS) if c else (BUILD, LIB, extra) for c in checks]
    todo = []
    for bdir, _, flags in targets:
        os.makedirs(bdir, exist_ok=True)
        todo += [(s, flags, bdir) for s in _sources(bdir) if extra or _stale(_obj(s, bdir), [s, *hdrs, __file__])]
    # the largest translation units first, so that none is left for the end
    todo.sort(key=lambda t: -_weight(t[0]))
    n = jobs or max(1, os.cpu_count() or 1)
    torch_obj = ""
    if todo or False in checks:
        with cf.ThreadPoolExecutor(n) as ex:
            binding = ex.submit(_compile_torch) if False in checks else None
            for (src, _, _), log in zip(todo, ex.map(lambda t: _compile(*t), todo)):
                if verbose and log.strip():
                    print(f"[{os.path.basename(src)}]\n{log}", file=sys.stderr)
            torch_obj = binding.result() if binding else ""
    for bdir, lib, _ in targets:
        objs = [_obj(s, bdir) for s in _sources(bdir)]
        if any(t[2] == bdir for t in todo) or _stale(lib, objs):
            tmp = lib + ".tmp"
            cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
            os.replace(tmp, lib)
    if torch_obj:
        _link_torch(torch_obj)
    return [lib for _, lib, _ in targets]


if __name__ == "__main__":
    v = "-v" in sys.argv
    extra = ["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else []
    print(build(verbose=v or bool(extra), extra=extra, check="--check" in sys.argv))
