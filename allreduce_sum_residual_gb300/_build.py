"""Build libarnorm.so (the CUDA kernels and the C ABI) for sm_103a, in tree.

Each .cu file compiles to an object in parallel; the objects link into
``allreduce_sum_residual_gb300/libarnorm.so``.  Only nvcc is needed (no
cmake); the same command works on x86_64 and aarch64 hosts.  Beside it g++
builds ``_binding-<python>-<torch>.so``, the expert-layer calls on torch
tensors in one step, against the installed torch; where that cannot be built
the library stands alone and those calls go through ctypes.
"""
import concurrent.futures as cf
import glob
import importlib.util
import os
import re
import shutil
import subprocess
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJ_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libarnorm.so")
# The checking build: the same sources with device-side bounds checks
# compiled in (AR_CHECK=1); a failed check records AR_ERR_BOUNDS in the
# device status word and skips the access.  For tests, not for production.
CHECK_OBJ_DIR = os.path.join(PKG, "_build_check")
CHECK_LIB = os.path.join(PKG, "libarnorm_check.so")
CXX = "g++"
BINDING_DIR = PKG
BINDING_SRC = os.path.join(CSRC, "binding.cpp")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2",
              "-Xptxas", "-warn-spills", f"-I{INCLUDE}", f"-I{CSRC}"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libarnorm.so")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (sources() + glob.glob(os.path.join(CSRC, "*.cuh"))
            + glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)])


def up_to_date(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(d) <= t for d in _deps())


def binding_path(torch_version: str, torch_git: str) -> str:
    """The binding for this Python and that torch, whose internals it calls:
    another of either neither loads it nor takes it for up to date."""
    python = sysconfig.get_config_var("EXT_SUFFIX")[1:-len(".so")]
    return os.path.join(BINDING_DIR, f"_binding-{python}-torch{torch_version}-{torch_git[:9]}.so")


def build_binding(force: bool = False):
    """Compile the binding unless it is newer than its sources; returns its
    path, or None without a CUDA build of torch (the C library needs none)."""
    spec = importlib.util.find_spec("torch")
    torch = spec.submodule_search_locations[0] if spec else ""
    if not os.path.exists(os.path.join(torch, "lib", "libc10_cuda.so")):
        return None
    with open(os.path.join(torch, "version.py")) as f:
        said = dict(re.findall(r"^(\w+)\s*(?::[^=]*)?=\s*'([^']*)'", f.read(), re.M))
    path = binding_path(said["__version__"], said.get("git_version", ""))
    deps = [BINDING_SRC, os.path.join(INCLUDE, "ar_rmsnorm.h"), os.path.abspath(__file__)]
    if not force and os.path.exists(path) and \
            all(os.path.getmtime(d) <= os.path.getmtime(path) for d in deps):
        return path
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    tmp = path + f".tmp{os.getpid()}"
    cmd = [CXX, "-std=c++17", "-O2", "-fPIC", "-shared", f"-I{INCLUDE}",
           f"-I{sysconfig.get_paths()['include']}", "-isystem", os.path.join(torch, "include"),
           "-isystem", os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(cuda, "include"), BINDING_SRC, "-o", tmp,
           "-L" + os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-ltorch",
           "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{CXX} failed on {BINDING_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, path)
    return path


def _binding_if_possible(force: bool = False):
    """build_binding, which the library does not need: a warning where it
    fails (no g++, no Python.h, no torch headers)."""
    try:
        return build_binding(force)
    except (RuntimeError, OSError, KeyError) as e:
        warnings.warn("the expert-layer calls will go through ctypes, some 10 us a call slower: their "
                      f"binding was not built ({e})", RuntimeWarning, stacklevel=3)
        return None


def build(force: bool = False, verbose: bool = False, extra_flags=(), check: bool = False) -> str:
    """Compile and link libarnorm.so (with ``check``: libarnorm_check.so, the
    checking build) unless it is newer than every source; without ``check``
    the binding too, if it can be built."""
    lib_path, obj_dir = (CHECK_LIB, CHECK_OBJ_DIR) if check else (LIB, OBJ_DIR)
    extra_flags = tuple(extra_flags) + (("-DAR_CHECK=1",) if check else ())
    if not force and up_to_date(lib_path):
        if not check:
            _binding_if_possible()
        return lib_path
    os.makedirs(obj_dir, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(obj_dir, os.path.basename(src)[:-3] + ".o")
        cmd = [cc, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        binding = None if check else ex.submit(_binding_if_possible, force)
        objs = list(ex.map(compile_one, srcs))
    tmp = lib_path + f".tmp{os.getpid()}"
    r = subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of {os.path.basename(lib_path)} failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib_path)
    if binding is not None:
        binding.result()
    return lib_path


if __name__ == "__main__":
    import sys
    print(build(force=True, verbose="-v" in sys.argv, check="--check" in sys.argv,
                extra_flags=["-Xptxas", "-v"] if "-v" in sys.argv else []))
