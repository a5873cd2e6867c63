"""Builds libssd.so in-tree with nvcc for sm_103a (GB300), and its Python binding.

Each .cu file under csrc/ is compiled in parallel to an object file, then the
objects are linked into ``state_space_model_scan_gb300/libssd.so``.  No torch
extension machinery is used: the library has a plain C ABI (include/ssd.h).
csrc/binding.cpp becomes the extension module ``_binding`` against the installed
torch's headers (g++).
"""
import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libssd.so")
BUILD_DIR = os.path.join(PKG, "_build")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _headers_mtime():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hs.append(os.path.join(ROOT, "include", "ssd.h"))
    return max(os.path.getmtime(h) for h in hs)


def _compile(src, obj, extra):
    cmd = [nvcc()] + ARCH + NVCC_FLAGS + extra + ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, " ".join(cmd), r.stdout + r.stderr))
    return r.stdout + r.stderr


BINDING = os.path.join(PKG, "_binding.so")
BUILT_FOR = os.path.join(BUILD_DIR, "_binding.txt")   # the torch and Python whose headers the binding was built with


def build_binding(force: bool = False) -> str:
    """Compile csrc/binding.cpp into the extension module _binding; returns its path.  Built again when a source is newer, or
    for another torch or Python."""
    import torch
    src, deps = os.path.join(CSRC, "binding.cpp"), [os.path.join(ROOT, "include", "ssd.h")]
    home = os.path.dirname(torch.__file__)
    built_for = "torch %s (%s) in %s, python %s" % (torch.__version__, torch.version.git_version, home, sys.version)
    if not force and os.path.exists(BINDING) and os.path.getmtime(BINDING) >= max(os.path.getmtime(f) for f in [src] + deps):
        try:
            with open(BUILT_FOR) as f:
                if f.read() == built_for:
                    return BINDING
        except OSError:
            pass
    inc = [sysconfig.get_paths()["include"], os.path.join(home, "include"),
           os.path.join(home, "include", "torch", "csrc", "api", "include"),
           os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
    tmp = BINDING + ".tmp.%d" % os.getpid()
    cmd = (["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch.compiled_with_cxx11_abi()] +
           [f for i in inc for f in ("-isystem", i)] + [src, "-o", tmp, "-L" + os.path.join(home, "lib"),
                                                        "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"])
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed for %s:\n%s\n%s" % (src, " ".join(cmd), r.stdout + r.stderr))
    os.replace(tmp, BINDING)
    os.makedirs(BUILD_DIR, exist_ok=True)
    with open(BUILT_FOR, "w") as f:
        f.write(built_for)
    return BINDING


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    """Compile csrc/*.cu and link libssd.so; build the binding beside it.  Returns the library's path."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        binding = ex.submit(build_binding, force)
        lib = _build_lib(force, verbose, extra)
        binding.result()
    return lib


def _build_lib(force, verbose, extra) -> str:
    srcs = sources()
    hm = _headers_mtime()
    jobs = []
    for s in srcs:
        o = os.path.join(BUILD_DIR, os.path.basename(s)[:-3] + ".o")
        if force or not os.path.exists(o) or os.path.getmtime(o) < max(os.path.getmtime(s), hm) or extra:
            jobs.append((s, o))
    if jobs:
        with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 4))) as ex:
            futs = [ex.submit(_compile, s, o, list(extra)) for s, o in jobs]
            for f in futs:
                out = f.result()
                if verbose and out.strip():
                    print(out, file=sys.stderr)
    objs = [os.path.join(BUILD_DIR, os.path.basename(s)[:-3] + ".o") for s in srcs]
    if force or jobs or not os.path.exists(LIB) or os.path.getmtime(LIB) < max(os.path.getmtime(o) for o in objs):
        tmp = LIB + ".tmp.%d" % os.getpid()
        cmd = [nvcc()] + ARCH + ["-shared", "-o", tmp] + objs
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("link failed:\n%s\n%s" % (" ".join(cmd), r.stdout + r.stderr))
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
