"""Build the in-tree CUDA library ``lib/libattn47_sm103.so`` with nvcc.

Every translation unit is compiled for sm_103a only
(``-gencode arch=compute_103a,code=sm_103a``), in parallel, then linked into
one shared object with the CUDA runtime linked statically, so that the
library loads on a machine without a GPU (e.g. to check its exported
symbols) and needs only the driver at run time.  Beside it g++ builds
``lib/_attn47_fast_<torch version>.<Python's ABI>.so``, the Python module that marshals the
usual case of the short calls (csrc/fast_calls.cpp, against torch's headers);
where that cannot be built, the library is, and those calls go another way.

Usage: ``python -m exact_attention_47_gb300.build_lib`` or ``build()``.
"""

import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_DIR = os.path.join(PKG, "lib")
LIB_NAME = "libattn47_sm103.so"
LIB_PATH = os.path.join(LIB_DIR, LIB_NAME)

SOURCES = ["api.cu", "fwd_sm103.cu", "bwd_sm103.cu", "decode_sm103.cu", "decode_kv4_sm103.cu", "decode_kv8_sm103.cu", "kv_append_sm103.cu", "rope_sm103.cu",
           "fusion_sm103.cu", "gemm_sm103.cu", "ssd_sm103.cu"]
GENCODE = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = GENCODE + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
                    "-I", INCLUDE, "-I", CSRC]

FAST_SOURCE = "fast_calls.cpp"


def _torch():
    """(version, folder) of the installed torch."""
    import torch

    return str(torch.__version__), os.path.dirname(os.path.abspath(torch.__file__))


def fast_path():
    """Where the module of the fast calls is built for the installed torch and
    this Python: it fits no other of either."""
    return os.path.join(LIB_DIR, "_attn47_fast_%s%s" % (_torch()[0], sysconfig.get_config_var("EXT_SUFFIX")))


def _fast_command(out):
    home = _torch()[1]
    include = os.path.join(home, "include")
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    return (["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", os.path.join(CSRC, FAST_SOURCE),
             "-o", out]
            + ["-I" + d for d in (INCLUDE, include, os.path.join(include, "torch", "csrc", "api", "include"),
                                  sysconfig.get_paths()["include"], os.path.join(cuda, "include"))]
            + ["-L" + os.path.join(home, "lib")]
            + ["-l" + n for n in ("torch_python", "torch_cpu", "torch_cuda", "torch", "c10", "c10_cuda")])


def _nvcc():
    exe = shutil.which("nvcc")
    if exe is None:
        cand = "/usr/local/cuda/bin/nvcc"
        if os.path.exists(cand):
            return cand
        raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build the library")
    return exe


def _run(cmd):
    proc = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if proc.returncode != 0:
        raise RuntimeError("command failed (%d): %s\n%s" % (proc.returncode, " ".join(cmd), proc.stdout))
    return proc.stdout


def _stale(obj, src):
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    deps = [src] + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    deps.append(os.path.join(INCLUDE, "attn47.h"))
    return any(os.path.getmtime(d) > t for d in deps)


def _build_fast():
    """Compile the module of the fast calls if its sources changed.  The library
    does not need it: where it cannot be built, that is said, and one from other
    sources is not left in its place."""
    fast = None
    try:
        fast = fast_path()
        if _stale(fast, os.path.join(CSRC, FAST_SOURCE)):
            _run(_fast_command(fast + ".tmp"))
            os.replace(fast + ".tmp", fast)
    except (ImportError, OSError, RuntimeError) as e:
        if fast is not None and os.path.exists(fast):
            os.remove(fast)
        sys.stderr.write("the module of the fast calls was not built (the rotary, append and 8- and 4-bit-cache calls cost "
                         "more host time without it): %s\n" % e)


def build(verbose=False, ptxas_info=False):
    """Compile (only what changed) and link; returns the library path."""
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)
    jobs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        if ptxas_info or _stale(o, s):
            cmd = [nvcc] + CFLAGS + (["-Xptxas", "-v"] if ptxas_info else []) + ["-c", s, "-o", o]
            jobs.append(cmd)
    link = bool(jobs) or not os.path.exists(LIB_PATH)
    with ThreadPoolExecutor(max_workers=max(1, min(len(jobs) + 1, os.cpu_count() or 1))) as ex:
        fast = ex.submit(_build_fast)
        outs = list(ex.map(_run, jobs))
        fast.result()
    if verbose or ptxas_info:
        for out in outs:
            sys.stdout.write(out)
    objs = [os.path.join(BUILD_DIR, s.replace(".cu", ".o")) for s in SOURCES]
    if link:
        tmp = LIB_PATH + ".tmp"
        _run([nvcc] + GENCODE + ["-shared", "-cudart", "static", "-o", tmp] + objs)
        os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose=True, ptxas_info="--ptxas" in sys.argv))
