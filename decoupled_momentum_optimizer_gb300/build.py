"""Build libdemo_gb300.so in-tree for sm_103a (GB300) with nvcc.

Usage: ``python -m decoupled_momentum_optimizer_gb300.build`` (or ``build()``).
The translation units compile in parallel, then link into one shared
library next to this file.  The DCT factor header is regenerated from its
generator first, so the constants always come from gen_dct_factors.py.
"""

import concurrent.futures
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
LIB_NAME = "libdemo_gb300.so"
LIB_PATH = os.path.join(HERE, LIB_NAME)
# Python's way to the norm, embedding and clipping calls, of one interpreter and one torch; which torch stands beside
# the objects.
BIND_PATH = os.path.join(HERE, "_bind_ops" + sysconfig.get_config_var("EXT_SUFFIX"))
BIND_STAMP = os.path.join(os.path.dirname(HERE), "_build", "bind_ops_torch.txt")
SOURCES = ["demo_api.cu", "demo_step.cu", "demo_encode.cu", "demo_decode.cu", "demo_decode_lanes.cu",
           "demo_decode_groups.cu", "demo_dense.cu", "demo_adamw.cu", "train_api.cu", "train_dropout.cu",
           "train_quantize.cu", "train_matmul.cu", "train_linear.cu", "train_norm.cu", "train_norm_grad.cu",
           "train_embedding.cu", "train_clip.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-fmad=false", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]


def _nvcc():
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def _regen_factors():
    gen = os.path.join(CSRC, "gen_dct_factors.py")
    out = subprocess.run([sys.executable, gen], check=True, capture_output=True, text=True).stdout
    path = os.path.join(CSRC, "dct32_factors.cuh")
    old = open(path).read() if os.path.exists(path) else None
    if old != out:
        with open(path, "w") as f:
            f.write(out)


def _compile(src, build_dir, verbose):
    obj = os.path.join(build_dir, os.path.splitext(src)[0] + ".o")
    cmd = [_nvcc()] + NVCC_FLAGS + (["-Xptxas", "-v"] if verbose else []) + ["-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj, r.stderr


def _cuda_include(nvcc):
    """The folder of CUDA's headers beside nvcc, wherever PATH finds it (a link, say); None where there is none."""
    path = shutil.which(nvcc)
    for tool in (path, os.path.realpath(path)) if path else ():
        include = os.path.join(os.path.dirname(os.path.dirname(tool)), "include")
        if os.path.exists(os.path.join(include, "cuda_runtime.h")):
            return include
    return None


def _bind(verbose):
    """Compile and link the extension module against the library and the torch that is installed."""
    import torch

    if torch.version.cuda is None:
        raise RuntimeError("the torch that is installed has no CUDA")
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BIND_PATH + ".tmp"
    headers = [h for h in (inc, os.path.join(inc, "torch", "csrc", "api", "include"), _cuda_include(_nvcc())) if h]
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", sysconfig.get_paths()["include"],
           f'-DDEMO_TORCH="{torch_tag(torch)}"', *[a for h in headers for a in ("-isystem", h)], os.path.join(CSRC, "bind_ops.cpp"), "-o", tmp, "-L", HERE,
           f"-l:{LIB_NAME}", "-Wl,-rpath,$ORIGIN", "-L", lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda",
           "-ltorch_python"]
    _forget_bind()
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"the extension module did not build:\n{r.stdout}\n{r.stderr}")
    if verbose:
        sys.stderr.write(r.stderr)
    os.replace(tmp, BIND_PATH)
    with open(BIND_STAMP, "w") as f:
        f.write(_torch())


def _forget_bind():
    for path in (BIND_STAMP, BIND_PATH):
        if os.path.exists(path):
            os.remove(path)


def _try_bind(verbose):
    """Build the extension module.  The library is complete without it (Python's calls then go through ctypes), so what
    keeps it from being built is reported and not raised; an older one does not stay beside a newer library."""
    try:
        _bind(verbose)
    except Exception as e:
        _forget_bind()
        sys.stderr.write(f"{os.path.basename(BIND_PATH)} was not built, calls go through ctypes: {e}\n")


def torch_tag(torch):
    """What names a torch whose tensors the module reads: compiled into it, and compared when it is imported."""
    return f"{torch.__version__} {torch.version.git_version}"


def _torch():
    """What the installed torch says of its version (read without importing it); None without one (the library itself does
    without)."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.origin:
        return None
    try:
        with open(os.path.join(os.path.dirname(spec.origin), "version.py")) as f:
            return f.read()
    except OSError:
        return spec.origin


def _bound():
    """The torch that the module was built against, None without one."""
    try:
        with open(BIND_STAMP) as f:
            return f.read()
    except OSError:
        return None


def build(verbose=False, force=False):
    """Compile and link the library, and the extension module where torch and g++ allow it; returns the library's path."""
    _regen_factors()
    build_dir = os.path.join(os.path.dirname(HERE), "_build")
    os.makedirs(build_dir, exist_ok=True)
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, "demo.h")]
    newest = max(os.path.getmtime(d) for d in deps)

    def current(path):
        return not force and os.path.exists(path) and os.path.getmtime(path) >= newest

    if current(LIB_PATH):
        if _torch() and (not current(BIND_PATH) or _bound() != _torch()):
            _try_bind(verbose)
        return LIB_PATH
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        results = list(ex.map(lambda s: _compile(s, build_dir, verbose), SOURCES))
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    objs = [o for o, _ in results]
    tmp = LIB_PATH + ".tmp"
    cmd = [_nvcc()] + ARCH + ["-shared", "-cudart", "shared", "-Xlinker", "-rpath,/usr/local/cuda/lib64", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    if _torch():
        _try_bind(verbose)
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, force="-f" in sys.argv))
