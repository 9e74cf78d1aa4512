"""Build step for the CUDA library (sm_103a only).

Compiles every ``csrc/*.cu`` translation unit with nvcc in parallel and links
them into ``_build/libgdn_gb300.so``, an in-tree shared library exporting the
C ABI of ``include/gdn.h``.  The CUDA runtime is linked statically; the
library depends on the driver (libcuda) only at run time.  Beside it, with g++,
``_build/_attn_binding.so``: the CPython extension through which torch tensors
reach the attention layers' operators (``csrc/attn_binding.cpp``), compiled again when
torch or Python is another version.
"""
import concurrent.futures
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_NAME = "libgdn_gb300.so"
BINDING_NAME = "_attn_binding.so"
BINDING_SRC = os.path.join(CSRC, "attn_binding.cpp")
ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def lib_path():
    return os.path.join(BUILD_DIR, LIB_NAME)


def binding_path():
    return os.path.join(BUILD_DIR, BINDING_NAME)


def _binding_command(out):
    import torch

    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    cxx = shutil.which("g++") or "c++"
    return [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            "-I", INCLUDE, "-isystem", sysconfig.get_paths()["include"],
            "-isystem", os.path.join(base, "include"),
            "-isystem", os.path.join(base, "include", "torch", "csrc", "api", "include"),
            "-isystem", os.path.join(cuda, "include"), BINDING_SRC, "-o", out,
            "-L", os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def _binding_made_with():
    """What the extension is compiled against: another torch or Python wants another one."""
    import torch

    return "\n".join([torch.__version__, sys.version, *_binding_command(binding_path())])


def _binding_stale(headers):
    stamp = binding_path() + ".made_with"
    if _stale(binding_path(), [BINDING_SRC] + headers) or not os.path.exists(stamp):
        return True
    with open(stamp) as f:
        return f.read() != _binding_made_with()


def _nvcc():
    exe = shutil.which("nvcc")
    if exe:
        return exe
    cand = "/usr/local/cuda/bin/nvcc"
    if os.path.exists(cand):
        return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")


def _sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hs += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    return hs


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force=False, verbose=False, extra_flags=()):
    """Compile (if stale) and return the path of the shared library."""
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    headers = _headers()
    objs, jobs = [], []
    for src in _sources():
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + headers):
            cmd = [nvcc, *ARCH_FLAGS, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
            jobs.append(cmd)

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return r

    binding, binding_tmp = binding_path(), binding_path() + f".tmp{os.getpid()}"
    if force or _binding_stale(headers):
        jobs.append(_binding_command(binding_tmp))
    if jobs:
        with concurrent.futures.ThreadPoolExecutor(max_workers=min(len(jobs), os.cpu_count() or 4)) as ex:
            list(ex.map(run, jobs))
    if os.path.exists(binding_tmp):
        os.replace(binding_tmp, binding)
        with open(binding + ".made_with", "w") as f:
            f.write(_binding_made_with())
    out = lib_path()
    if force or jobs or _stale(out, objs):
        tmp = out + f".tmp{os.getpid()}"
        run([nvcc, *ARCH_FLAGS, "-shared", "-o", tmp, *objs])
        os.replace(tmp, out)
    return out


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
