"""Builds libgdr.so (the CUDA library behind include/gdr.h) in-tree for sm_103a,
and the operators' Python binding beside it.

Each translation unit is compiled in parallel with nvcc (the binding with the
host compiler), then linked as one shared library at
gated_delta_rule_varlen_gb300/lib/libgdr.so; the binding, which depends on the
PyTorch and the Python it was compiled against, carries both in its name.  The
library needs neither: without PyTorch it is built alone, and an error in the
binding is raised once the library is there.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIBDIR = os.path.join(HERE, "lib")
LIB = os.path.join(LIBDIR, "libgdr.so")
SOURCES = ["gdr_fwd.cu", "gdr_walk.cu", "gdr_bwd.cu", "gdr_api.cu", "gdr_sconv.cu", "gdr_ssm.cu", "gdr_ssm_tc.cu",
           "gdr_step.cu", "gdr_norm_fwd.cu", "gdr_norm_bwd.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def binding_path() -> str:
    import torch
    return os.path.join(LIBDIR, f"_gdr_ops-{torch.__version__}.{sysconfig.get_config_var('SOABI')}.so")


def _cxx(source: str, target: str):
    """The compile and the link command of the binding."""
    import torch
    cxx = os.environ.get("CXX") or "g++"
    home, cuda = os.path.dirname(torch.__file__), os.path.dirname(os.path.dirname(nvcc()))
    obj = target[:-3] + ".o"
    compile_ = [cxx, "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                f"-I{home}/include", f"-I{sysconfig.get_paths()['include']}", f"-I{cuda}/include", "-c", source, "-o", obj]
    link = [cxx, "-shared", obj, "-o", target + f".tmp{os.getpid()}", f"-L{home}/lib", "-lc10", "-lc10_cuda", "-ltorch_cpu",
            "-ltorch_python", f"-L{LIBDIR}", "-lgdr", "-Wl,-rpath,$ORIGIN"]
    return obj, compile_, link


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    os.makedirs(LIBDIR, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    headers.append(os.path.join(os.path.dirname(HERE), "include", "gdr.h"))
    objs, procs = [], []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(LIBDIR, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s] + headers):
            cmd = [nvcc()] + ARCH + FLAGS + list(extra_flags) + ["-c", s, "-o", o]
            if verbose:
                print(" ".join(cmd), file=sys.stderr)
            procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    bound = None
    try:
        binding = binding_path()
    except ImportError:
        print("PyTorch is not installed: the library is built without the operators' Python binding", file=sys.stderr)
        binding = None
    if binding:
        source = os.path.join(CSRC, "gdr_binding.cpp")
        bobj, compile_, link = _cxx(source, binding)
        if force or _stale(bobj, [source, headers[-1]]):
            bound = subprocess.Popen(compile_, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)

    def finish(src, p):
        """The compiler's complaint, or None."""
        out, _ = p.communicate()
        text = out.decode(errors="replace")
        if p.returncode != 0:
            return f"{src}:\n{text}"
        if verbose and text:
            print(text, file=sys.stderr)
        return None

    errors = [e for e in (finish(src, p) for src, p in procs) if e]
    if not errors and (force or procs or _stale(LIB, objs)):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc()] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs
        subprocess.run(cmd, check=True)
        os.replace(tmp, LIB)
    if bound:
        errors += [e for e in (finish("gdr_binding.cpp", bound),) if e]
    if errors:
        raise RuntimeError("compilation failed:\n" + "\n".join(errors))
    if binding and (force or _stale(binding, [bobj])):
        subprocess.run(link, check=True)
        os.replace(binding + f".tmp{os.getpid()}", binding)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra_flags=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else ())
