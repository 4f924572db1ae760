"""Builds libexternd.so (sm_100a) in-tree from csrc/*.cu with nvcc, and the
native part of the Python binding (_calls.so) from csrc/calls.cpp."""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libexternd.so")
CALLS = os.path.join(HERE, "_calls.so")  # the native part of the Python binding
CALLS_STAMP = os.path.join(HERE, "_build", "_calls.interfaces")  # what it was built against
# (-static-global-template-stub=false: the sequential kernel template is
# instantiated in its own units and launched from seq_als.cu)
NVCC_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-O3", "-std=c++17",
              "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr", "-static-global-template-stub=false"]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _interfaces() -> str:
    """The torch and the Python whose interfaces _calls.so is bound to."""
    import importlib.metadata
    import sysconfig
    return f"torch {importlib.metadata.version('torch')} {sysconfig.get_config_var('SOABI')}"


def _stale_calls() -> bool:
    if not os.path.exists(CALLS_STAMP) or open(CALLS_STAMP).read() != _interfaces():
        return True
    deps = (os.path.join(CSRC, "calls.cpp"), os.path.join(HERE, "..", "include", "externd.h"))
    return not os.path.exists(CALLS) or any(os.path.getmtime(d) > os.path.getmtime(CALLS)
                                            for d in deps)


def build_calls() -> str:
    """Builds the module that marshals the 8-bit calls between torch and the C
    ABI (it is given the library's entry points when that is loaded)."""
    import sysconfig

    import torch
    base = os.path.dirname(torch.__file__)
    nvcc = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    inc = [os.path.join(base, "include"),
           os.path.join(base, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    tmp = CALLS + ".tmp"
    subprocess.run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
                    f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                    os.path.join(CSRC, "calls.cpp"), "-o", tmp, *(f"-I{i}" for i in inc),
                    "-L" + os.path.join(base, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu",
                    "-ltorch_cuda", "-ltorch", "-ltorch_python"], check=True)
    os.replace(tmp, CALLS)
    os.makedirs(os.path.dirname(CALLS_STAMP), exist_ok=True)
    with open(CALLS_STAMP, "w") as f:
        f.write(_interfaces())
    return CALLS


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))
    deps.append(os.path.join(HERE, "..", "include", "externd.h"))
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    if force or _stale_calls():
        build_calls()
    if not force and not _stale():
        return LIB
    nvcc = os.environ.get("NVCC", "nvcc")
    objdir = os.path.join(HERE, "_build")
    os.makedirs(objdir, exist_ok=True)
    objs, cmds = [], []
    for src in sources():
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        cmd = [nvcc, *NVCC_FLAGS, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        cmds.append(cmd)
        objs.append(obj)
    # the translation units are independent: compile them side by side
    from concurrent.futures import ThreadPoolExecutor
    with ThreadPoolExecutor(max_workers=min(len(cmds), os.cpu_count() or 1)) as ex:
        for r in list(ex.map(lambda c: subprocess.run(c, check=True), cmds)):
            pass
    tmp = LIB + ".tmp"
    subprocess.run([nvcc, "-gencode", "arch=compute_100a,code=sm_100a", "-shared", *objs, "-o", tmp,
                    "-lcudart"], check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose="-v" in sys.argv))


# the source files each profiled kernel is built from
KERNEL_SOURCES = {
    "seq_als_kernel": ("seq_als.cu", "seq_kernel.cuh", "seq_inst_smem_plain.cu", "common.cuh"),
    "contract_tma_kernel": ("umma_contract.cu", "umma_layout.cuh", "common.cuh"),
}


def kernel_source_hash(kernel: str) -> str:
    """Hash of the files one kernel is compiled from (identifies that kernel's
    code across unrelated changes elsewhere in the library)."""
    import hashlib
    h = hashlib.sha256()
    for name in KERNEL_SOURCES[kernel]:
        h.update(name.encode())
        h.update(open(os.path.join(CSRC, name), "rb").read())
    return h.hexdigest()[:16]


def source_hash() -> str:
    """Hash of the CUDA sources and the public header (identifies a kernel build)."""
    import hashlib
    h = hashlib.sha256()
    deps = sources() + sorted(glob.glob(os.path.join(CSRC, "*.h"))) + \
        sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + [os.path.join(HERE, "..", "include", "externd.h")]
    for d in deps:
        h.update(os.path.basename(d).encode())
        h.update(open(d, "rb").read())
    return h.hexdigest()[:16]
