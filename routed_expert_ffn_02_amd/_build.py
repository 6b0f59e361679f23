"""Build the routed-MoE C-ABI library for gfx950 with hipcc (in-tree, no JIT cache), and the
Python module that hands torch tensors to the calls around the experts.

    python routed_expert_ffn_02_amd/_build.py        # compile csrc/ -> libroutedmoe.so, _marshal.<abi>.so

The library needs neither Python's headers nor torch; where one of them is missing, it is built alone.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(os.path.dirname(HERE), "_build")
LIB = os.path.join(HERE, "libroutedmoe.so")
# the tag of the Python it is built for: another one does not load it
MARSHAL = os.path.join(HERE, "_marshal" + sysconfig.get_config_var("EXT_SUFFIX"))
ARCH = os.environ.get("RMOE_OFFLOAD_ARCH", "gfx950")

HIP_SOURCES = ["route.hip", "lookup.hip", "decode.hip", "prefill.hip", "fill.hip", "tokens.hip", "norm.hip"]
CPP_SOURCES = ["runtime.cpp", "cpu_ffn.cpp", "placement.cpp", "bank.cpp"]
MARSHAL_SOURCE = "marshal.cpp"

# Packed fp32 VALU ops are disabled for all device code (the host pass warns that it
# does not know the feature; that is harmless).
HIP_FLAGS = ["-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}", "-Xclang", "-target-feature", "-Xclang",
             "-packed-fp32-ops", "-Wno-unused-result", "-fvisibility=hidden"]
CPP_FLAGS = ["-O3", "-std=c++17", "-fPIC", "-Wno-unused-result", "-D__HIP_PLATFORM_AMD__", "-fvisibility=hidden"]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found")


def rocm_root() -> str:
    return os.path.dirname(os.path.dirname(os.path.realpath(hipcc())))


def host_cxx() -> str:
    """ROCm's clang++ for the host-only sources (runtime, CPU branch)."""
    cand = os.path.join(rocm_root(), "lib", "llvm", "bin", "clang++")
    return cand if os.path.exists(cand) else (shutil.which("clang++") or "g++")


def marshal_includes():
    """Include paths of the tensor module: torch's, Python's.  None where one has no headers here."""
    try:
        import torch
    except ImportError:
        return None
    paths = [os.path.join(os.path.dirname(torch.__file__), "include"), sysconfig.get_paths()["include"]]
    heads = ["torch/csrc/autograd/python_variable.h", "Python.h"]
    return paths if all(os.path.exists(os.path.join(p, h)) for p, h in zip(paths, heads)) else None


def _compile(src: str, flags=()) -> str:
    path = os.path.join(CSRC, src)
    obj = os.path.join(BUILD, src + ".o")
    if src.endswith(".hip"):
        cmd = [hipcc()] + HIP_FLAGS + ["-c", path, "-o", obj]
    else:
        cmd = [host_cxx()] + CPP_FLAGS + ["-I", os.path.join(rocm_root(), "include"), "-c", path, "-o", obj]
    cmd += flags
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compile failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return obj


def build(verbose: bool = True) -> str:
    """Compile every source and link libroutedmoe.so and the tensor module (always rebuilds)."""
    os.makedirs(BUILD, exist_ok=True)
    srcs = HIP_SOURCES + CPP_SOURCES
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs) + 1)) as ex:
        marshal = ex.submit(build_marshal_object)
        objs = list(ex.map(_compile, srcs))
        _link([hipcc(), "-shared", "-fPIC", f"--offload-arch={ARCH}"] + objs, LIB, ["-lpthread"])
        if verbose:
            print(f"built {LIB}")
        marshal = marshal.result()
    for old in glob.glob(os.path.join(HERE, "_marshal*.so")):
        os.remove(old)  # of an earlier source, or another Python's
    if marshal is None:
        print("no torch or no Python headers here: the calls around the experts are in the library, "
              "without their Python module", file=sys.stderr)
        return LIB
    torch_lib = os.path.join(os.path.dirname(marshal_includes()[0]), "lib")
    _link([host_cxx(), "-shared", "-fPIC", marshal, "-L", HERE, "-L", torch_lib], MARSHAL,
          ["-l:libroutedmoe.so", "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_hip", "-lamdhip64", "-Wl,-rpath,$ORIGIN"])
    if verbose:
        print(f"built {MARSHAL}")
    return LIB


def build_marshal_object():
    """The tensor module's object file, or None where it cannot be built."""
    paths = marshal_includes()
    if paths is None:
        return None
    return _compile(MARSHAL_SOURCE, ["-DUSE_ROCM"] + [f for p in paths for f in ("-I", p)])


def _link(cmd, out: str, libs) -> None:
    tmp = out + ".tmp"
    cmd = cmd + ["-o", tmp] + libs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out)


if __name__ == "__main__":
    build()
    sys.exit(0)
