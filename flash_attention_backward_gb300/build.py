"""Compile the CUDA library in-tree for sm_103a (nvcc, no cmake)."""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
import tempfile
import warnings

try:
    from ._fast_path import fast_path
except ImportError:  # run as a file, without the package (and PyTorch)
    from _fast_path import fast_path

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
LIB = os.path.join(HERE, "libfa_back.so")
FAST_SRC = os.path.join(CSRC, "py_fast.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
_fast_given_up = False  # the marshalling module could not be built in this process


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps():
    out = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh"))]
    out += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    return out


def _newer(target, deps) -> bool:
    return target is not None and os.path.exists(target) and all(os.path.getmtime(d) <= os.path.getmtime(target) for d in deps)


def up_to_date() -> bool:
    return _newer(LIB, _deps()) and (_fast_given_up or _newer(fast_path(), _fast_deps()))


def _fast_deps():
    return [FAST_SRC] + [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]


def _fast_command(out: str):
    """Compile and link the marshalling module of paged.py against this interpreter's PyTorch."""
    import torch

    root = os.path.dirname(torch.__file__)
    lib = os.path.join(root, "lib")
    inc = [a for p in (os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
                       sysconfig.get_paths()["include"], os.path.join(_cuda_home(), "include")) for a in ("-isystem", p)]
    abi = f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-nostartfiles", "-fvisibility=hidden", abi, *inc, FAST_SRC, "-o", out, "-L", lib,
            "-Wl,--no-as-needed", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", f"-Wl,-rpath,{lib}"]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if c and (os.path.isabs(c) and os.path.exists(c) or not os.path.isabs(c)):
            return c
    return "nvcc"


def _cuda_home() -> str:
    return os.path.dirname(os.path.dirname(os.path.realpath(shutil.which(nvcc()) or "/usr/local/cuda/bin/nvcc")))


def build(force: bool = False, verbose: bool = False) -> str:
    """Build libfa_back.so and the marshalling module of paged.py next to this file; returns the library's
    path.  The translation units compile in parallel (one compiler per file, objects in a temporary
    folder), then one link.  The module is optional: without g++ or PyTorch's headers a warning says so,
    and the wrappers make their calls from Python."""
    if not force and up_to_date():
        return LIB
    fast = _FastBuild() if force or not (_fast_given_up or _newer(fast_path(), _fast_deps())) else None
    try:
        if force or not _newer(LIB, _deps()):
            _build_library(verbose)
    except BaseException:
        if fast is not None:
            fast.stop()
        raise
    if fast is not None:
        fast.finish()
    return LIB


class _FastBuild:
    """The marshalling module's compiler, beside the library's.  What it was made of before goes first: a
    module of older headers would not do for the library that is built now."""

    def __init__(self):
        self.target = fast_path()
        self.tmp, self.proc, self.why = "%s.tmp%d" % (self.target, os.getpid()), None, "no PyTorch"
        if self.target is None:
            return
        if os.path.exists(self.target):
            os.remove(self.target)
        try:
            self.proc = subprocess.Popen(_fast_command(self.tmp), stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
        except (OSError, AttributeError) as e:  # no g++, no PyTorch as expected
            self.why = "%s: %s" % (type(e).__name__, e)

    def finish(self) -> None:
        global _fast_given_up
        if self.proc is not None:
            out, _ = self.proc.communicate()
            if self.proc.returncode == 0:
                os.replace(self.tmp, self.target)
                _fast_given_up = False
                paged = sys.modules.get((__package__ or "-") + ".paged")
                if paged is not None:  # imported before there was a module
                    paged.look_for_fast()
                return
            self.why = "g++ ended with %d: %s" % (self.proc.returncode, out.strip()[-500:])
        _fast_given_up = True
        self.stop()
        warnings.warn("the marshalling module _fast was not built, the wrappers make their calls from Python (%s)" % self.why,
                      RuntimeWarning, stacklevel=3)

    def stop(self) -> None:
        if self.proc is not None and self.proc.poll() is None:
            self.proc.kill()
            self.proc.communicate()
        if os.path.exists(self.tmp):
            os.remove(self.tmp)


def _build_library(verbose: bool) -> None:
    tmp = LIB + ".tmp%d" % os.getpid()
    flags = [*ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE]
    if verbose:
        flags.insert(0, "-Xptxas=-v")
    with tempfile.TemporaryDirectory(prefix="fa_back_build_") as obj_dir:
        jobs = []
        for src in sources():
            obj = os.path.join(obj_dir, os.path.basename(src) + ".o")
            cmd = [nvcc(), *flags, "-c", src, "-o", obj]
            jobs.append((obj, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
        failed = False
        for obj, proc in jobs:
            out, _ = proc.communicate()
            if proc.returncode != 0:
                failed = True
                sys.stderr.write(out)
            elif verbose:
                sys.stderr.write(out)
        if failed:
            raise RuntimeError("nvcc failed building libfa_back.so")
        r = subprocess.run([nvcc(), *ARCH, "-shared", *[o for o, _ in jobs], "-o", tmp], stdout=subprocess.PIPE,
                           stderr=subprocess.STDOUT, text=True)
        if r.returncode != 0:
            sys.stderr.write(r.stdout)
            raise RuntimeError("nvcc failed linking libfa_back.so")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
