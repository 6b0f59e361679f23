"""Which kernels a call of the experts' products launches, without a device: the library's entry points run as they are,
over pointers that nothing follows, and a stand-in for the runtime (native/launch_log.cpp) writes the launches down.

    launches([dict(call="glu", rows=.., E=.., K=.., N=.., fmt="bf16", ...), ...]) -> [[(kernel, ...), ...], ...]

runs them in a process of its own, whose library the stand-in serves.  A kernel is its name and its template's
arguments, such as ("product_direct", "bf16", 0, 256, 256, 128, 64, 1, 1): operand type, product (0 glu, 1 linear, 2 dx,
3 dw), tile, a wavefront's part, ..
"""
import ctypes
import json
import os
import re
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
LIB = os.path.join(os.path.dirname(HERE), "routed_expert_ffn_02_amd", "libroutedmoe.so")

FMT = {"f32": 0, "bf16": 1}
ACT = {"none": 0, "silu": 1, "gelu": 2}


class Config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("rows", "n_experts", "K", "N", "fmt", "y_fmt", "dw_fmt", "act")] + [
        (n, ctypes.c_int64) for n in ("ld_x", "ld_dx", "ld_w", "gs_w", "ld_y", "ld_residual", "ld_z")]


def parse(mangled):
    """("product_direct", "bf16", 0, ...) of a mangled name; templates of no type are left without one."""
    m = re.match(r"_ZN4rmoe(?:12_GLOBAL__N_1)?(\d+)(\w+)", mangled)
    if not m:
        return (mangled,)
    n = int(m.group(1))
    name, rest = m.group(2)[:n], m.group(2)[n:]
    out = [re.sub("_kernel$", "", name)]
    if rest.startswith("I"):
        rest = rest[1:]
        if rest[0] in "tf":
            out.append({"t": "bf16", "f": "f32"}[rest[0]])
            rest = rest[1:]
        while rest.startswith("L"):
            v = re.match(r"L[ib](\d+)E", rest)
            out.append(int(v.group(1)))
            rest = rest[v.end():]
    return tuple(out)


def _run(lib, log, c):
    """One call, and its launches.  how: rows dense, with gaps that keep 16 bytes, or starting one element off."""
    how, E = c.get("how", "dense"), c.get("E", 0)
    pad, first = {"dense": (0, 0), "gaps": (24, 8), "odd": (3, 1)}[how]
    call, n = c["call"], max(E, 1)
    glu, back = call.startswith("glu"), call.endswith("backward")
    K, N = c["K"], c["N"]
    cols = 2 * N if glu else N
    fmt, y_fmt = FMT[c["fmt"]], FMT[c.get("y", c["fmt"])]
    p = Config(c["rows"], n, K, N, fmt, y_fmt, FMT[c.get("dw", c["fmt"])], ACT[c.get("act", "silu" if glu else "none")],
               K + pad, K + pad, K + pad, cols * (K + pad), N + pad, N + pad, cols + pad)
    at = iter(range(1 << 44, 1 << 46, 1 << 41))
    eb, yb = (2 if fmt else 4), (2 if y_fmt else 4)
    row, yrow, flat = (lambda: next(at) + first * eb), (lambda: next(at) + first * yb), (lambda: next(at))
    off, out = flat() if E else None, c.get("out", ("dx", "dw", "dbias"))
    if call == "glu":
        st = lib.moe_glu(ctypes.byref(p), row(), row(), off, row(), row(), None)
    elif call == "linear":
        st = lib.moe_linear(ctypes.byref(p), row(), row(), flat(), yrow(), off, yrow(), row(), None)
    else:
        ws = flat()
        dx, dw, db = row() if "dx" in out else None, flat() if "dw" in out else None, flat() if "dbias" in out else None
        if call == "glu_backward":
            size = lib.moe_glu_workspace(c["rows"], n, K, N, fmt)
            st = lib.moe_glu_backward(ctypes.byref(p), row(), row(), row(), row(), off, dx, dw, ws, size, None)
        else:
            size = lib.moe_linear_workspace(c["rows"], n, K, N, fmt)
            st = lib.moe_linear_backward(ctypes.byref(p), yrow(), row(), row(), row(), off, dx, dw, db, ws, size, None)
    return st, [line.rsplit(" ", 4) for line in log().decode().splitlines()]


def main(stand_in):
    log = ctypes.CDLL(stand_in, mode=ctypes.RTLD_GLOBAL)
    log.launch_log.restype = log.launch_kernels.restype = ctypes.c_char_p
    lib = ctypes.CDLL(LIB)
    vp, z = ctypes.c_void_p, ctypes.c_size_t
    lib.moe_glu.argtypes = [vp] * 7
    lib.moe_linear.argtypes = [vp] * 9
    lib.moe_glu_backward.argtypes = [vp] * 9 + [z, vp]
    lib.moe_linear_backward.argtypes = [vp] * 10 + [z, vp]
    lib.moe_glu_workspace.restype = lib.moe_linear_workspace.restype = ctypes.c_int64
    calls = json.load(sys.stdin)
    json.dump({"kernels": log.launch_kernels().decode().split(), "calls": [_run(lib, log.launch_log, c) for c in calls]}, sys.stdout)


def stand_in(folder):
    """The stand-in, compiled into `folder`."""
    out = os.path.join(str(folder), "liblaunchlog.so")
    subprocess.check_call(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", os.path.join(HERE, "native", "launch_log.cpp"), "-o", out])
    return out


def launches(stand_in_path, calls):
    """([all kernels], [(status, [(kernel, grid, threads), ...]) of each call])"""
    r = subprocess.run([sys.executable, os.path.abspath(__file__), stand_in_path], input=json.dumps(calls), capture_output=True, text=True)
    if r.returncode:
        raise RuntimeError(r.stderr)
    d = json.loads(r.stdout)
    return [parse(k) for k in d["kernels"]], [
        (st, [(parse(k), tuple(int(v) for v in grid), int(threads)) for k, *grid, threads in ls]) for st, ls in d["calls"]]


if __name__ == "__main__":
    main(sys.argv[1])
