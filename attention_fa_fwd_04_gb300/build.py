"""Build libfa_gb300.so in-tree with nvcc for sm_103a, and _fa_bind.so, the
native part of the Python binding, with the host compiler.

The translation units compile in parallel; the CUDA ones link into one shared
library next to this file.  No CMake, no torch extension machinery.

The library (the C ABI) needs nvcc alone and is installed first.  The binding
needs the installed torch's headers: without torch, or where they do not
compile, it is left out with a message, and the package's calls that go through
it say so.
"""
import importlib.util
import os
import re
import subprocess
import sys
import sysconfig
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libfa_gb300.so")
SOURCES = ["fa_api.cu", "fa_prefill.cu", "fa_decode.cu", "fa_decode_noalloc.cu",
           "fa_backward.cu", "fa_host.cu", "fa_rope.cu", "fa_tree.cu", "fa_verify.cu",
           "fa_shared.cu", "fa_sample.cu", "fa_pages.cu"]
HEADERS = ["fa_ptx.cuh", "fa_tiles.cuh", "fa_exp2_table.h", "fa_shares.h", "fa_internal.h"]
BIND = os.path.join(HERE, "_fa_bind.so")
BIND_SOURCE = os.path.join(CSRC, "fa_bind.cpp")
BIND_STAMP = os.path.join(HERE, "_fa_bind.torch")  # version of the torch it was built against

NVCC = os.environ.get("NVCC", "nvcc")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", CSRC, "-I", INCLUDE]


def _inputs():
    files = [os.path.join(CSRC, s) for s in SOURCES + HEADERS]
    files.append(os.path.join(INCLUDE, "fa.h"))
    return files


def _newer(target, sources) -> bool:
    return os.path.exists(target) and all(os.path.getmtime(f) <= os.path.getmtime(target)
                                          for f in sources)


def up_to_date() -> bool:
    return _newer(LIB, _inputs())


def _torch():
    """(folder, version) of the installed torch, which is not imported; or None."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        return None
    folder = spec.submodule_search_locations[0]
    try:
        with open(os.path.join(folder, "version.py")) as f:
            m = re.search(r"^__version__\s*=\s*['\"]([^'\"]+)", f.read(), re.M)
    except OSError:
        m = None
    return folder, m.group(1) if m else ""


def _bind_up_to_date(version) -> bool:
    """Whether the binding is there, newer than its sources and this torch's."""
    if not _newer(BIND, [BIND_SOURCE, os.path.join(INCLUDE, "fa.h")]):
        return False
    try:
        with open(BIND_STAMP) as f:
            return f.read() == version
    except OSError:
        return False


def _bind_command(out, torch_dir, version):
    """The host compiler's command for the native binding: against the
    installed torch's headers and libraries, and the CUDA headers beside nvcc."""
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    lib = os.path.join(torch_dir, "lib")
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
            f'-DFA_TORCH_VERSION="{version}"', "-I", INCLUDE,
            "-I", sysconfig.get_paths()["include"], "-I", os.path.join(torch_dir, "include"),
            "-I", os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
            "-I", os.path.join(cuda, "include"), BIND_SOURCE, "-o", out, "-L", lib,
            "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10", "-lc10_cuda", f"-Wl,-rpath,{lib}"]


def _start(cmd, verbose):
    """The running command, or None where its program is missing."""
    if verbose:
        print(" ".join(cmd), flush=True)
    try:
        return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    except OSError as e:
        print(f"{cmd[0]}: {e}", file=sys.stderr, flush=True)
        return None


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    torch = _torch()
    lib_stale = force or not up_to_date()
    bind_stale = force or (lib_stale if torch is None else not _bind_up_to_date(torch[1]))
    if not lib_stale and not bind_stale:
        return LIB
    extra = ["-Xptxas", "-v"] if ptxas_info else []
    with tempfile.TemporaryDirectory(prefix="fa_build_") as tmp:
        tmp_bind = os.path.join(tmp, "_fa_bind.so")
        bind = _start(_bind_command(tmp_bind, *torch), verbose) if torch and bind_stale else None
        if lib_stale:
            procs, objs = [], []
            for s in SOURCES:
                obj = os.path.join(tmp, s.replace(".cu", ".o"))
                cmd = [NVCC] + ARCH + FLAGS + extra + ["-c", os.path.join(CSRC, s), "-o", obj]
                procs.append((s, _start(cmd, verbose)))
                objs.append(obj)
            failed = []
            for s, pr in procs:
                out = pr.communicate()[0] if pr else ""
                if out and (verbose or ptxas_info or pr.returncode):
                    sys.stdout.write(out)
                if pr is None or pr.returncode:
                    failed.append(s)
            if failed:
                if bind:
                    bind.communicate()
                raise RuntimeError(f"nvcc failed for {failed}")
            tmp_lib = os.path.join(tmp, "libfa_gb300.so")
            cmd = [NVCC] + ARCH + ["-shared", "-o", tmp_lib] + objs
            subprocess.check_call(cmd)
            os.replace(tmp_lib, LIB)
        if bind_stale:
            _install_bind(bind, tmp_bind, torch, verbose)
    return LIB


def _install_bind(proc, built, torch, verbose):
    """Installs the compiled binding; one that could not be built (of older
    sources, or for another torch) does not stay behind."""
    out = proc.communicate()[0] if proc else ""
    if out and (verbose or proc.returncode):
        sys.stdout.write(out)
    if proc and proc.returncode == 0:
        os.replace(built, BIND)
        with open(BIND_STAMP, "w") as f:
            f.write(torch[1])
        return
    for path in (BIND, BIND_STAMP):
        if os.path.exists(path):
            os.remove(path)
    why = "torch is not installed" if torch is None else f"it does not compile against torch {torch[1]}"
    print(f"{os.path.basename(BIND)} left out: {why}.  The C library is complete without it.",
          file=sys.stderr, flush=True)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                ptxas_info="--ptxas" in sys.argv))
