"""Python binding of the routed-MoE C-ABI library (libroutedmoe.so, HIP for gfx950).

Argument marshalling only: every function here has the name of a C entry point
declared in include/routed_moe.h and forwards to it.  Device tensors are passed
as raw pointers (torch supplies device memory and the HIP stream); every step of
the hot path runs in the library's kernels.  There is no fallback: importing
this package fails when the compiled library is missing.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch  # noqa: F401  (loads the HIP runtime the library links against)

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libroutedmoe.so")

MOE_OK, MOE_EINVAL, MOE_ENOMEM, MOE_EHIP, MOE_ESTATE, MOE_ENOPIN, MOE_ENOTSUP, MOE_ETIMEDOUT = 0, -1, -2, -3, -4, -5, -6, -7
MOE_WFMT_F32, MOE_WFMT_BF16, MOE_WFMT_FP4, MOE_WFMT_MXFP4 = 0, 1, 2, 3
MOE_AFMT_F32, MOE_AFMT_BF16 = 0, 1
MOE_MODE_FUSED, MOE_MODE_OFFLOAD, MOE_MODE_CPU, MOE_MODE_HYBRID = 0, 1, 2, 3
MOE_KIND_HIT, MOE_KIND_FILL, MOE_KIND_CPU, MOE_KIND_BUF = 0, 1, 2, 3
MOE_FLAG_PROFILE = 1
MOE_FLAG_DEVICE_FILLS = 2
MOE_FLAG_MX_PREFILL = 4

_STATUS = {0: "MOE_OK", -1: "MOE_EINVAL", -2: "MOE_ENOMEM", -3: "MOE_EHIP", -4: "MOE_ESTATE",
           -5: "MOE_ENOPIN", -6: "MOE_ENOTSUP", -7: "MOE_ETIMEDOUT"}


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str, msg: str):
        super().__init__(f"{where}: {_STATUS.get(status, status)}: {msg}")
        self.status = status


class moe_config(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int32), ("n_experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("hidden", ctypes.c_int32), ("inter", ctypes.c_int32), ("wfmt", ctypes.c_int32),
                ("afmt", ctypes.c_int32), ("renorm", ctypes.c_int32), ("max_tokens", ctypes.c_int32),
                ("mode", ctypes.c_int32), ("bw_pcie", ctypes.c_uint64), ("bw_host", ctypes.c_uint64),
                ("cpu_threads", ctypes.c_int32), ("flags", ctypes.c_int32)]


class moe_trace_rec(ctypes.Structure):
    _fields_ = [("key", ctypes.c_int32), ("kind", ctypes.c_int32), ("slot", ctypes.c_int32),
                ("evicted", ctypes.c_int32)]


class moe_stats(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint64) for n in ("decode_calls", "prefill_calls", "lookups", "hits", "fills",
                                                 "cpu_experts", "evictions", "fill_bytes")] + [
        ("phase1_ms", ctypes.c_double), ("phase2_ms", ctypes.c_double),
        ("phase1_launches", ctypes.c_uint64), ("phase2_launches", ctypes.c_uint64),
        ("phase1_bytes", ctypes.c_uint64), ("phase2_bytes", ctypes.c_uint64),
        ("gemm1_ms", ctypes.c_double), ("gemm2_ms", ctypes.c_double),
        ("gemm1_launches", ctypes.c_uint64), ("gemm2_launches", ctypes.c_uint64),
        ("gemm_flops", ctypes.c_double), ("copy_ms", ctypes.c_double), ("copy_bytes", ctypes.c_uint64),
        ("cpu_ms", ctypes.c_double)]

    def as_dict(self):
        return {n: getattr(self, n) for n, _ in self._fields_}


class moe_step_rec(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("layer", "misses", "fills", "cpu")] + [
        ("fill_ms", ctypes.c_double), ("cpu_ms", ctypes.c_double)]


MOE_PLACE_LRU, MOE_PLACE_PREFILL, MOE_PLACE_STATIC, MOE_PLACE_PINNED_RING = 0, 1, 2, 3


class moe_replay_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("n_layers", "n_experts", "pairs", "policy", "capacity",
                                              "ring_per_layer")]


class moe_replay_result(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint64) for n in ("keys", "misses", "reads")]


MOE_GATE_NONE, MOE_GATE_TOKEN, MOE_GATE_CHANNEL = 0, 1, 2


class moe_norm_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "H", "h_fmt", "y_fmt", "x_fmt", "gate_kind")] + [
        ("alpha", ctypes.c_float), ("eps", ctypes.c_float)] + [
        (n, ctypes.c_int64) for n in ("ld_h", "ld_y", "ld_x")]


class moe_bank_header(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("n_layers", "n_experts", "hidden", "inter", "wfmt", "pad")] + [
        ("record_bytes", ctypes.c_int64), ("n_records", ctypes.c_int64)]


class moe_bank_stats(ctypes.Structure):
    _fields_ = [("bytes", ctypes.c_uint64), ("seconds", ctypes.c_double), ("mode", ctypes.c_int32),
                ("threads", ctypes.c_int32), ("direct_errno", ctypes.c_int32), ("pad", ctypes.c_int32)]


BANK_READ_MODES = {0: "direct", 1: "direct_bounce", 2: "buffered"}


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python routed_expert_ffn_02_amd/_build.py` "
                          "(hipcc, gfx950).  There is no CPU fallback.")
    L = ctypes.CDLL(LIB_PATH)
    P, I32, I64, U64, VP = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64, ctypes.c_void_p
    sig = {
        "moe_create": (I32, [ctypes.POINTER(moe_config), ctypes.POINTER(P)]),
        "moe_destroy": (I32, [P]),
        "moe_last_error": (ctypes.c_char_p, [P]),
        "moe_record_bytes": (I64, [ctypes.POINTER(moe_config)]),
        "moe_pool_alloc": (I32, [P, I64, ctypes.POINTER(VP)]),
        "moe_pool_register": (I32, [P, VP, I64, I32]),
        "moe_bind": (I32, [P, VP, VP, ctypes.c_size_t, I32]),
        "moe_fused_load": (I32, [P, VP]),
        "moe_set_bandwidths": (I32, [P, U64, U64]),
        "moe_set_mode": (I32, [P, I32]),
        "moe_set_cpu_wait": (I32, [P, ctypes.c_double]),
        "moe_route": (I32, [P, I32, VP, I32, VP, VP, VP, VP, VP]),
        "moe_topk": (I32, [P, VP, I32, VP, VP, VP]),
        "expert_cache_lookup": (I32, [P, I32, VP, I32, VP, VP, VP, VP]),
        "moe_route_lookup": (I32, [P, I32, VP, I32, VP, VP, VP, VP, VP, VP, VP, VP]),
        "moe_decode_layer": (I32, [P, I32, VP, I32, VP, VP, VP, VP, VP, VP]),
        "moe_ffn_decode": (I32, [P, I32, VP, I32, VP, VP, VP, VP, VP]),
        "moe_prefill_begin": (I32, [P, VP]),
        "moe_ffn_prefill": (I32, [P, I32, VP, I32, VP, VP, VP, VP, VP, VP]),
        "moe_prefill_end": (I32, [P, VP]),
        "moe_permute": (I32, [P, VP, I32, VP, VP, VP, VP, VP]),
        "expert_cache_resize": (I32, [P, I32, VP, ctypes.c_size_t, VP]),
        "qstar_split": (I32, [I32, U64, U64, I32, I32]),
        "moe_bench_bw": (I32, [P, ctypes.POINTER(U64), ctypes.POINTER(U64)]),
        "moe_cache_snapshot": (I32, [P, VP, VP, VP, ctypes.POINTER(U64), ctypes.POINTER(I32)]),
        "moe_get_stats": (I32, [P, ctypes.POINTER(moe_stats)]),
        "moe_reset_stats": (I32, [P]),
        "moe_sync": (I32, [P, VP]),
        "moe_step_log": (I32, [P, VP, I32, ctypes.POINTER(I32)]),
        "moe_permute_noalloc": (I32, [VP, I32, I32, VP, VP, VP, VP, VP]),
        "moe_bench_hbm": (I32, [VP, ctypes.c_size_t, ctypes.c_size_t, I32, VP, VP]),
        "moe_placement_replay": (I32, [ctypes.POINTER(moe_replay_config), VP, I32, VP, I32, I32, VP,
                                       ctypes.POINTER(moe_replay_result)]),
        "moe_pool_check_f16": (I32, [ctypes.POINTER(moe_config), VP, I64, ctypes.POINTER(I64)]),
        "moe_bank_write": (I32, [ctypes.c_char_p, ctypes.POINTER(moe_config), VP, I64]),
        "moe_bank_info": (I32, [ctypes.c_char_p, ctypes.POINTER(moe_bank_header)]),
        "moe_bank_read": (I32, [ctypes.c_char_p, ctypes.POINTER(moe_config), VP, I64, I32,
                                ctypes.POINTER(moe_bank_stats)]),
        "moe_dispatch_workspace": (I64, [I32, I32, I32]),
        "moe_dispatch": (I32, [VP, I32, I32, I32, VP, I32, I32, I64, VP, VP, VP, VP, VP, ctypes.c_size_t, VP]),
        "moe_dispatch_backward": (I32, [VP, I32, VP, I32, I32, I32, VP, I32, I64, VP]),
        "moe_combine": (I32, [VP, I32, VP, VP, I32, I32, I32, VP, I32, I64, VP]),
        "moe_combine_backward": (I32, [VP, I32, I64, VP, I32, VP, VP, I32, I32, I32, VP, VP, VP]),
        "moe_topk_backward": (I32, [VP, I32, I32, VP, I32, VP, I32, VP, VP]),
        "moe_block_norm": (I32, [ctypes.POINTER(moe_norm_config), VP, VP, VP, VP, VP, VP, VP, VP]),
        "moe_block_norm_workspace": (I64, [I32, I32]),
        "moe_block_norm_backward": (I32, [ctypes.POINTER(moe_norm_config)] + [VP] * 13 + [ctypes.c_size_t, VP]),
        "moe_decode_block": (I32, [P, I32, VP, I32, VP, VP, VP, VP, VP, ctypes.POINTER(moe_norm_config), VP, VP, VP,
                                   VP, VP, VP]),
        "moe_pool_load": (I32, [P, ctypes.c_char_p, I32, ctypes.POINTER(VP), ctypes.POINTER(moe_bank_stats)]),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    return L


lib = _load()


# ---------------------------------------------------------------------------
def _ptr(t):
    """Device / host pointer of a tensor, an int address, or None."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(s):
    if s is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(s, int):
        return s
    return s.cuda_stream


class Ctx:
    """Owner of a moe_ctx handle (destroyed with moe_destroy)."""

    def __init__(self, handle: int, cfg: moe_config):
        self.handle = handle
        self.cfg = cfg
        # held here so that a context collected at interpreter exit, after the
        # module globals are cleared, can still be destroyed
        self._destroy = lib.moe_destroy

    def __del__(self):
        if getattr(self, "handle", None):
            self._destroy(self.handle)
            self.handle = None


def _check(ctx, st, where):
    if st != MOE_OK:
        msg = lib.moe_last_error(ctx.handle if isinstance(ctx, Ctx) else ctx)
        raise MoeError(st, where, msg.decode() if msg else "")


def make_config(n_layers, n_experts, top_k, hidden, inter, wfmt, afmt, max_tokens, mode, renorm=0,
                bw_pcie=0, bw_host=0, cpu_threads=0, flags=0) -> moe_config:
    return moe_config(n_layers, n_experts, top_k, hidden, inter, wfmt, afmt, renorm, max_tokens, mode,
                      bw_pcie, bw_host, cpu_threads, flags)


def moe_create(cfg: moe_config) -> Ctx:
    h = ctypes.c_void_p()
    st = lib.moe_create(ctypes.byref(cfg), ctypes.byref(h))
    if st != MOE_OK:
        raise MoeError(st, "moe_create", "invalid configuration or device error")
    return Ctx(h.value, cfg)


def moe_destroy(ctx: Ctx) -> None:
    if ctx.handle:
        _check(ctx, lib.moe_destroy(ctx.handle), "moe_destroy")
        ctx.handle = None


def moe_last_error(ctx: Ctx) -> str:
    return lib.moe_last_error(ctx.handle).decode()


def moe_record_bytes(cfg: moe_config) -> int:
    return int(lib.moe_record_bytes(ctypes.byref(cfg)))


def moe_pool_check_f16(cfg: moe_config, pool, n_records: int) -> int:
    """Lowest record index whose block scales could take an FP4 / MXFP4 prefill weight out of
    f16's normal range, or -1 when every record passes."""
    bad = ctypes.c_int64(-1)
    st = lib.moe_pool_check_f16(ctypes.byref(cfg), _ptr(pool), n_records, ctypes.byref(bad))
    if st not in (MOE_OK, MOE_EINVAL) or (st == MOE_EINVAL and bad.value < 0):
        raise MoeError(st, "moe_pool_check_f16", "bad argument")
    return int(bad.value)


def moe_pool_alloc(ctx: Ctx, n_records: int) -> int:
    p = ctypes.c_void_p()
    _check(ctx, lib.moe_pool_alloc(ctx.handle, n_records, ctypes.byref(p)), "moe_pool_alloc")
    return p.value


def moe_pool_register(ctx: Ctx, host_pool, n_records: int, pinned: int) -> None:
    _check(ctx, lib.moe_pool_register(ctx.handle, _ptr(host_pool), n_records, pinned), "moe_pool_register")


def moe_bind(ctx: Ctx, router_w, arena, arena_bytes: int, n_slots: int) -> None:
    _check(ctx, lib.moe_bind(ctx.handle, _ptr(router_w), _ptr(arena), arena_bytes, n_slots), "moe_bind")


def moe_fused_load(ctx: Ctx, stream=None) -> None:
    _check(ctx, lib.moe_fused_load(ctx.handle, _stream(stream)), "moe_fused_load")


def moe_set_bandwidths(ctx: Ctx, bw_pcie: int, bw_host: int) -> None:
    _check(ctx, lib.moe_set_bandwidths(ctx.handle, int(bw_pcie), int(bw_host)), "moe_set_bandwidths")


def moe_set_mode(ctx: Ctx, mode: int) -> None:
    _check(ctx, lib.moe_set_mode(ctx.handle, mode), "moe_set_mode")


def moe_set_cpu_wait(ctx: Ctx, timeout_ms: float) -> None:
    _check(ctx, lib.moe_set_cpu_wait(ctx.handle, float(timeout_ms)), "moe_set_cpu_wait")


def moe_route(ctx: Ctx, layer, x, T, logit_bias, logits_out, topk_idx, topk_w, stream=None) -> None:
    _check(ctx, lib.moe_route(ctx.handle, layer, _ptr(x), T, _ptr(logit_bias), _ptr(logits_out), _ptr(topk_idx),
                              _ptr(topk_w), _stream(stream)), "moe_route")


def moe_topk(ctx: Ctx, logits, T, topk_idx, topk_w, stream=None) -> None:
    _check(ctx, lib.moe_topk(ctx.handle, _ptr(logits), T, _ptr(topk_idx), _ptr(topk_w), _stream(stream)),
           "moe_topk")


def expert_cache_lookup(ctx: Ctx, layer, topk_idx, T, slot_idx, trace=None, counts=None, stream=None) -> None:
    _check(ctx, lib.expert_cache_lookup(ctx.handle, layer, _ptr(topk_idx), T, _ptr(slot_idx), _ptr(trace),
                                        _ptr(counts), _stream(stream)), "expert_cache_lookup")


def moe_route_lookup(ctx: Ctx, layer, x, T, logit_bias, logits_out, topk_idx, topk_w, slot_idx, trace=None,
                     counts=None, stream=None) -> None:
    _check(ctx, lib.moe_route_lookup(ctx.handle, layer, _ptr(x), T, _ptr(logit_bias), _ptr(logits_out), _ptr(topk_idx),
                                     _ptr(topk_w), _ptr(slot_idx), _ptr(trace), _ptr(counts), _stream(stream)),
           "moe_route_lookup")


def moe_decode_layer(ctx: Ctx, layer, x, T, logit_bias, topk_idx, topk_w, slot_idx, y, stream=None) -> None:
    _check(ctx, lib.moe_decode_layer(ctx.handle, layer, _ptr(x), T, _ptr(logit_bias), _ptr(topk_idx), _ptr(topk_w),
                                     _ptr(slot_idx), _ptr(y), _stream(stream)), "moe_decode_layer")


def moe_ffn_decode(ctx: Ctx, layer, x, T, topk_idx, topk_w, slot_idx, y, stream=None) -> None:
    _check(ctx, lib.moe_ffn_decode(ctx.handle, layer, _ptr(x), T, _ptr(topk_idx), _ptr(topk_w), _ptr(slot_idx),
                                   _ptr(y), _stream(stream)), "moe_ffn_decode")


def moe_prefill_begin(ctx: Ctx, stream=None) -> None:
    _check(ctx, lib.moe_prefill_begin(ctx.handle, _stream(stream)), "moe_prefill_begin")


def moe_ffn_prefill(ctx: Ctx, layer, x, T, topk_idx, topk_w, y, trace=None, counts=None, stream=None) -> None:
    _check(ctx, lib.moe_ffn_prefill(ctx.handle, layer, _ptr(x), T, _ptr(topk_idx), _ptr(topk_w), _ptr(y),
                                    _ptr(trace), _ptr(counts), _stream(stream)), "moe_ffn_prefill")


def moe_prefill_end(ctx: Ctx, stream=None) -> None:
    _check(ctx, lib.moe_prefill_end(ctx.handle, _stream(stream)), "moe_prefill_end")


def moe_permute(ctx: Ctx, slot_idx, T, perm, offsets, group_slot, n_groups, stream=None) -> None:
    _check(ctx, lib.moe_permute(ctx.handle, _ptr(slot_idx), T, _ptr(perm), _ptr(offsets), _ptr(group_slot),
                                _ptr(n_groups), _stream(stream)), "moe_permute")


def expert_cache_resize(ctx: Ctx, new_n_slots, new_arena=None, new_arena_bytes=0, stream=None) -> None:
    _check(ctx, lib.expert_cache_resize(ctx.handle, new_n_slots, _ptr(new_arena), new_arena_bytes,
                                        _stream(stream)), "expert_cache_resize")


def qstar_split(m: int, bw_pcie: int, bw_host: int, mode: int, evictable: int) -> int:
    return int(lib.qstar_split(m, bw_pcie, bw_host, mode, evictable))


def moe_placement_replay(n_layers: int, n_experts: int, policy: int, capacity: int, decode, calib=None,
                         ring_per_layer: int = 0, want_miss: bool = False):
    """Replay a host routing trace (decode [steps, L, T*k], calib [tokens, L, k], int32
    NumPy arrays) against one placement policy.  Returns a dict with keys, misses, reads
    and, with want_miss, the per-pair miss flags [steps, L, T*k] (uint8)."""
    import numpy as np
    dec = np.ascontiguousarray(decode, dtype=np.int32)
    steps, L, pairs = dec.shape
    cal = None if calib is None else np.ascontiguousarray(calib, dtype=np.int32)
    cfg = moe_replay_config(n_layers, n_experts, pairs, policy, capacity, ring_per_layer)
    miss = np.zeros(dec.shape, np.uint8) if want_miss else None
    res = moe_replay_result()
    st = lib.moe_placement_replay(ctypes.byref(cfg), dec.ctypes.data, steps,
                                  None if cal is None else cal.ctypes.data,
                                  0 if cal is None else cal.shape[0], 1 if cal is None else cal.shape[2],
                                  None if miss is None else miss.ctypes.data, ctypes.byref(res))
    if st != MOE_OK:
        raise MoeError(st, "moe_placement_replay", "invalid shapes, ids or capacity")
    out = {"keys": res.keys, "misses": res.misses, "reads": res.reads}
    if want_miss:
        out["miss"] = miss
    return out


def _stats_dict(st: "moe_bank_stats") -> dict:
    return {"bytes": st.bytes, "seconds": st.seconds, "mode": BANK_READ_MODES.get(st.mode, st.mode),
            "threads": st.threads, "direct_errno": st.direct_errno}


def moe_bank_write(path: str, cfg: moe_config, pool, n_records: int) -> None:
    """Write n_records records from host memory `pool` (address or NumPy array) as a bank file."""
    st = lib.moe_bank_write(os.fsencode(path), ctypes.byref(cfg), _host_ptr(pool), n_records)
    if st != MOE_OK:
        raise MoeError(st, "moe_bank_write", f"cannot write {path}")


def moe_bank_info(path: str) -> dict:
    h = moe_bank_header()
    st = lib.moe_bank_info(os.fsencode(path), ctypes.byref(h))
    if st != MOE_OK:
        raise MoeError(st, "moe_bank_info", f"{path}: missing, malformed or truncated bank file")
    return {n: getattr(h, n) for n, _ in h._fields_ if n != "pad"}


def moe_bank_read(path: str, cfg, dst, dst_bytes: int, threads: int = 8) -> dict:
    """Read a bank file's records into host memory `dst` (address or NumPy array)."""
    out = moe_bank_stats()
    st = lib.moe_bank_read(os.fsencode(path), None if cfg is None else ctypes.byref(cfg), _host_ptr(dst), dst_bytes,
                           threads, ctypes.byref(out))
    if st != MOE_OK:
        raise MoeError(st, "moe_bank_read", f"{path}: header mismatch, short buffer or read error")
    return _stats_dict(out)


def moe_pool_load(ctx: Ctx, path: str, threads: int = 8):
    """Allocate the context's page-locked pool from a bank file and fill it; returns (pool address, stats)."""
    p = ctypes.c_void_p()
    out = moe_bank_stats()
    _check(ctx, lib.moe_pool_load(ctx.handle, os.fsencode(path), threads, ctypes.byref(p), ctypes.byref(out)),
           "moe_pool_load")
    return p.value, _stats_dict(out)


def _host_ptr(a):
    if a is None or isinstance(a, int):
        return a
    return a.ctypes.data


def moe_bench_bw(ctx: Ctx):
    bp, bh = ctypes.c_uint64(), ctypes.c_uint64()
    _check(ctx, lib.moe_bench_bw(ctx.handle, ctypes.byref(bp), ctypes.byref(bh)), "moe_bench_bw")
    return bp.value, bh.value


def moe_cache_snapshot(ctx: Ctx):
    """(slot_of [L*E], key_of [n_slots], stamp [n_slots], counter) as numpy arrays / int."""
    import numpy as np
    c = ctx.cfg
    slot_of = np.empty(c.n_layers * c.n_experts, np.int32)
    n = ctypes.c_int32()
    cnt = ctypes.c_uint64()
    _check(ctx, lib.moe_cache_snapshot(ctx.handle, slot_of.ctypes.data, None, None, ctypes.byref(cnt),
                                       ctypes.byref(n)), "moe_cache_snapshot")
    key_of = np.empty(max(n.value, 1), np.int32)
    stamp = np.empty(max(n.value, 1), np.uint64)
    _check(ctx, lib.moe_cache_snapshot(ctx.handle, None, key_of.ctypes.data, stamp.ctypes.data, None, None),
           "moe_cache_snapshot")
    return slot_of, key_of[: n.value], stamp[: n.value], cnt.value


def moe_get_stats(ctx: Ctx) -> dict:
    st = moe_stats()
    _check(ctx, lib.moe_get_stats(ctx.handle, ctypes.byref(st)), "moe_get_stats")
    return st.as_dict()


def moe_reset_stats(ctx: Ctx) -> None:
    _check(ctx, lib.moe_reset_stats(ctx.handle), "moe_reset_stats")


def moe_sync(ctx: Ctx, stream=None) -> None:
    _check(ctx, lib.moe_sync(ctx.handle, _stream(stream)), "moe_sync")


def moe_step_log(ctx: Ctx, capacity: int = 1 << 20):
    """The logged steps (oldest first) as a numpy record array; clears the log."""
    import numpy as np
    buf = (moe_step_rec * capacity)()
    n = ctypes.c_int32()
    _check(ctx, lib.moe_step_log(ctx.handle, ctypes.addressof(buf), capacity, ctypes.byref(n)), "moe_step_log")
    dt = np.dtype([("layer", np.int32), ("misses", np.int32), ("fills", np.int32), ("cpu", np.int32),
                   ("fill_ms", np.float64), ("cpu_ms", np.float64)])
    return np.frombuffer(bytes(buf)[: n.value * ctypes.sizeof(moe_step_rec)], dtype=dt).copy()


def moe_bench_hbm(buf, buf_bytes: int, read_bytes: int, reps: int, stream=None):
    """Per-pass kernel seconds of reps plain reads of read_bytes from the device buffer buf."""
    import numpy as np
    out = np.zeros(reps, np.float64)
    st = lib.moe_bench_hbm(_ptr(buf), buf_bytes, read_bytes, reps, out.ctypes.data, _stream(stream))
    if st != MOE_OK:
        raise MoeError(st, "moe_bench_hbm", "bad arguments or device error")
    return out


def moe_permute_noalloc(slot_idx, P: int, n_slot_range: int, perm, offsets, group_slot, n_groups, stream=None):
    st = lib.moe_permute_noalloc(_ptr(slot_idx), P, n_slot_range, _ptr(perm), _ptr(offsets), _ptr(group_slot),
                                 _ptr(n_groups), _stream(stream))
    if st != MOE_OK:
        raise MoeError(st, "moe_permute_noalloc", "sizes out of range, null pointer or launch failure")


# ---------------------------------------------------------------------------
# Around the experts.  These take torch tensors only and read shapes, formats and row strides
# from them; a tensor the library would misread (type, shape, stride, device) is refused here.
_FMT = {torch.float32: MOE_AFMT_F32, torch.bfloat16: MOE_AFMT_BF16}
_I32_MAX = 0x7fffffff


# the current stream's handle and the current device without the objects around them
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


class _Args:
    """Checks the tensors of one call and holds the device they share.  A decode step makes these
    calls once a layer, so a check reads each property of a tensor once."""
    __slots__ = ("where", "dev")

    def __init__(self, where: str):
        self.where = where
        self.dev = None

    def refuse(self, msg: str):
        raise MoeError(MOE_EINVAL, self.where, msg)

    def place(self, name, t):
        d = t.get_device()
        if d != self.dev:
            if d < 0:
                self.refuse(f"{name} must be on the GPU")
            if self.dev is not None:
                self.refuse(f"{name} is on cuda:{d}, other tensors on cuda:{self.dev}")
            self.dev = d

    def rows(self, name, t, n_rows=None, width=None, dense=False, like=None):
        """(pointer, format, row stride, rows, H) of a [rows, H] matrix with contiguous rows."""
        try:
            fmt = _FMT[t.dtype]
            n, h = t.shape
        except (AttributeError, KeyError, ValueError):
            self.refuse(f"{name} must be a two-dimensional fp32 or bf16 tensor")
        if n < 1 or h < 1 or n > _I32_MAX or h > _I32_MAX or (n_rows is not None and n != n_rows) or (
                width is not None and h != width):
            self.refuse(f"{name} has shape {(n, h)}, not {(n_rows or 'T', width or 'H')}")
        if t.is_contiguous():
            ld = h
        else:
            ld, step = t.stride()
            if n == 1:
                ld = h
            if (step != 1 and h > 1) or ld < h or dense:
                self.refuse(f"{name} needs contiguous rows" + (" without gaps" if dense else ""))
        if like is not None and (fmt, ld) != like:
            self.refuse(f"{name} must have the type and row stride of the tensor it belongs to")
        if t.get_device() != self.dev:
            self.place(name, t)
        return t.data_ptr(), fmt, ld, n, h

    def flat(self, name, t, dtype, *shape):
        """Pointer of a dense tensor of this type and shape (one number: that many elements)."""
        try:
            ok = t.dtype is dtype and t.is_contiguous()
        except AttributeError:
            ok = False
        if not ok:
            self.refuse(f"{name} must be a contiguous {dtype} tensor")
        if t.shape != shape and not (len(shape) == 1 and t.numel() == shape[0]):
            self.refuse(f"{name} has shape {tuple(t.shape)}, not {shape}")
        if t.get_device() != self.dev:
            self.place(name, t)
        return t.data_ptr()

    def pairs(self, name, t):
        """(T, k, pointer) of an int32 [T, k] table."""
        try:
            T, k = t.shape
        except (AttributeError, ValueError):
            T = k = 0
        if not T or not k or T > _I32_MAX or k > _I32_MAX:
            self.refuse(f"{name} must be an int32 tensor [T, k]")
        return T, k, self.flat(name, t, torch.int32, T, k)

    def workspace(self, t):
        """(pointer, bytes) of the caller's workspace."""
        if t is None:
            return None, 0
        if not isinstance(t, torch.Tensor) or not t.is_contiguous():
            self.refuse("ws must be a contiguous tensor")
        n = t.numel() * t.element_size()
        if not n:
            return None, 0
        self.place("ws", t)
        return t.data_ptr(), n

    def call(self, fn, stream, *args):
        """Forward to the C entry point on `stream` (default: the current stream of the tensors' device)."""
        dev = self.dev
        if stream is None:
            s = _raw_stream(dev)
        else:
            if isinstance(stream, torch.cuda.Stream) and stream.device.index != dev:
                self.refuse(f"stream is on {stream.device}, tensors on cuda:{dev}")
            s = _stream(stream)
        if _current_device() == dev:
            st = fn(*args, s)
        else:
            with torch.cuda.device(dev):
                st = fn(*args, s)
        if st:
            raise MoeError(st, self.where, "launch failure" if st == MOE_EHIP else
                           "shape out of range, overlapping tensors, missing argument or short workspace")


def moe_dispatch_workspace(T: int, k: int, n_experts: int) -> int:
    """Bytes of workspace of moe_dispatch."""
    n = int(lib.moe_dispatch_workspace(T, k, n_experts))
    if n < 0:
        raise MoeError(MOE_EINVAL, "moe_dispatch_workspace", "shape out of range")
    return n


def moe_dispatch(topk_idx, n_experts: int, x, xs, perm, inv, offsets, ws=None, stream=None) -> None:
    """Sort the pairs of topk_idx [T,k] by expert into perm [T*k], inv [T,k] and offsets [n_experts+1], and
    move the rows of x [T,H] to xs [T*k,H] (both None: sort only).  ws: uint8 workspace."""
    a = _Args("moe_dispatch")
    T, k, idx = a.pairs("topk_idx", topk_idx)
    P = T * k
    xp = xsp = None
    fmt = H = ld = 0
    if x is not None or xs is not None:
        xp, fmt, ld, _, H = a.rows("x", x, T)
        xsp, xs_fmt, _, _, _ = a.rows("xs", xs, P, H, True)
        if xs_fmt != fmt:
            a.refuse("xs must have x's type")
    p = a.flat("perm", perm, torch.int32, P)
    i = a.flat("inv", inv, torch.int32, T, k)
    o = a.flat("offsets", offsets, torch.int32, n_experts + 1)
    w, wn = a.workspace(ws)
    a.call(lib.moe_dispatch, stream, idx, T, k, n_experts, xp, fmt, H, ld, xsp, p, i, o, w, wn)


def moe_dispatch_backward(dxs, inv, dx, stream=None) -> None:
    """dx [T,H] = the sum of each token's rows of dxs [T*k,H]."""
    a = _Args("moe_dispatch_backward")
    T, k, i = a.pairs("inv", inv)
    g, fmt, _, _, H = a.rows("dxs", dxs, T * k, None, True)
    o, o_fmt, ld, _, _ = a.rows("dx", dx, T, H)
    a.call(lib.moe_dispatch_backward, stream, g, fmt, i, T, k, H, o, o_fmt, ld)


def moe_combine(ys, inv, w, y, stream=None) -> None:
    """y [T,H] = the sum of each token's rows of ys [T*k,H] weighted by w [T,k] (fp32)."""
    a = _Args("moe_combine")
    T, k, i = a.pairs("inv", inv)
    r, fmt, _, _, H = a.rows("ys", ys, T * k, None, True)
    wp = a.flat("w", w, torch.float32, T, k)
    o, o_fmt, ld, _, _ = a.rows("y", y, T, H)
    a.call(lib.moe_combine, stream, r, fmt, i, wp, T, k, H, o, o_fmt, ld)


def moe_combine_backward(dy, ys, inv, w, dys, dw, stream=None) -> None:
    """From dy [T,H]: dys [T*k,H] (or None; may be ys) and dw [T,k] (or None, then ys may be None)."""
    a = _Args("moe_combine_backward")
    T, k, i = a.pairs("inv", inv)
    d, d_fmt, ld, _, H = a.rows("dy", dy, T)
    r = o = wp = g = None
    fmt = d_fmt
    if dys is not None:
        o, fmt, _, _, _ = a.rows("dys", dys, T * k, H, True)
        wp = a.flat("w", w, torch.float32, T, k)
    if dw is not None:
        r, r_fmt, _, _, _ = a.rows("ys", ys, T * k, H, True)
        if dys is not None and r_fmt != fmt:
            a.refuse("dys must have ys's type")
        fmt = r_fmt
        g = a.flat("dw", dw, torch.float32, T, k)
    a.call(lib.moe_combine_backward, stream, d, d_fmt, ld, r, fmt, i, wp, T, k, H, o, g)


def moe_topk_backward(logits, topk_idx, dw, renorm: int, dlogits, stream=None) -> None:
    """dlogits [T,E] from the gates' gradients dw [T,k] at the chosen experts topk_idx [T,k]."""
    a = _Args("moe_topk_backward")
    T, k, idx = a.pairs("topk_idx", topk_idx)
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2:
        a.refuse("logits must be fp32 [T, E]")
    E = logits.shape[1]
    z = a.flat("logits", logits, torch.float32, T, E)
    g = a.flat("dw", dw, torch.float32, T, k)
    o = a.flat("dlogits", dlogits, torch.float32, T, E)
    a.call(lib.moe_topk_backward, stream, z, T, E, idx, k, g, renorm, o)


# The configuration of a norm call, by its values (the library reads it during the call only).
_norm_config = functools.lru_cache(maxsize=1024)(lambda *fields: ctypes.pointer(moe_norm_config(*fields)))


def _norm_inputs(a: _Args, T, H, w_post, gate, w_pre, gate_kind):
    q = None if w_post is None else a.flat("w_post", w_post, torch.float32, H)
    p = None if w_pre is None else a.flat("w_pre", w_pre, torch.float32, H)
    if (gate is None) != (gate_kind == MOE_GATE_NONE):
        a.refuse("gate and gate_kind must go together")
    g = None if gate is None else a.flat("gate", gate, torch.float32, T if gate_kind == MOE_GATE_TOKEN else H)
    return q, g, p


def moe_block_norm(h, y=None, w_post=None, gate=None, w_pre=None, h_out=None, x_out=None,
                   gate_kind: int = MOE_GATE_NONE, alpha: float = 1.0, eps: float = 1e-6, stream=None) -> None:
    """h_out = h + alpha gate norm(y; w_post), x_out = norm(h_out; w_pre): the step between two blocks."""
    a = _Args("moe_block_norm")
    hp, h_fmt, ld_h, T, H = a.rows("h", h)
    yp = ho = xo = None
    y_fmt = x_fmt = h_fmt
    ld_y = ld_x = H
    if y is not None:
        yp, y_fmt, ld_y, _, _ = a.rows("y", y, T, H)
    if h_out is not None:
        ho = hp if h_out is h else a.rows("h_out", h_out, T, H, False, (h_fmt, ld_h))[0]
    if x_out is not None:
        xo, x_fmt, ld_x, _, _ = a.rows("x_out", x_out, T, H)
    q, g, p = _norm_inputs(a, T, H, w_post, gate, w_pre, gate_kind)
    a.call(lib.moe_block_norm, stream, _norm_config(T, H, h_fmt, y_fmt, x_fmt, gate_kind, alpha, eps, ld_h, ld_y, ld_x),
           hp, yp, q, g, p, ho, xo)


def moe_block_norm_workspace(T: int, H: int) -> int:
    """Bytes of workspace of moe_block_norm_backward."""
    n = int(lib.moe_block_norm_workspace(T, H))
    if n < 0:
        raise MoeError(MOE_EINVAL, "moe_block_norm_workspace", "shape out of range")
    return n


def moe_block_norm_backward(h_out, y, w_post, gate, w_pre, dh_out, dx, dh, dy, dw_post, dgate, dw_pre, ws=None,
                            gate_kind: int = MOE_GATE_NONE, alpha: float = 1.0, eps: float = 1e-6,
                            stream=None) -> None:
    """The gradient of moe_block_norm from dh_out and dx (either may be None); any output may be None."""
    a = _Args("moe_block_norm_backward")
    lead = dx if dh_out is None else dh_out
    if not isinstance(lead, torch.Tensor) or lead.dim() != 2:
        a.refuse("dh_out or dx must be given")
    T, H = lead.shape
    # (format, row stride) that h_out, dh_out and dh share, and y and dy
    h_like = y_like = None
    hp = yp = dhp = dxp = o_h = o_y = None
    h_fmt = y_fmt = x_fmt = 0
    ld_h = ld_y = ld_x = H
    if dh_out is not None:
        dhp, h_fmt, ld_h, _, _ = a.rows("dh_out", dh_out, T, H)
        h_like = h_fmt, ld_h
    if h_out is not None:
        hp, h_fmt, ld_h, _, _ = a.rows("h_out", h_out, T, H, False, h_like)
        h_like = h_fmt, ld_h
    if dh is not None:
        o_h, h_fmt, ld_h, _, _ = a.rows("dh", dh, T, H, False, h_like)
    if y is not None:
        yp, y_fmt, ld_y, _, _ = a.rows("y", y, T, H)
        y_like = y_fmt, ld_y
    if dy is not None:
        o_y, y_fmt, ld_y, _, _ = a.rows("dy", dy, T, H, False, y_like)
    if dx is not None:
        dxp, x_fmt, ld_x, _, _ = a.rows("dx", dx, T, H)
    q, g, p = _norm_inputs(a, T, H, w_post, gate, w_pre, gate_kind)
    dq = None if dw_post is None else a.flat("dw_post", dw_post, torch.float32, H)
    dp = None if dw_pre is None else a.flat("dw_pre", dw_pre, torch.float32, H)
    dg = None if dgate is None else a.flat("dgate", dgate, torch.float32, T if gate_kind == MOE_GATE_TOKEN else H)
    w, wn = a.workspace(ws)
    a.call(lib.moe_block_norm_backward, stream,
           _norm_config(T, H, h_fmt, y_fmt, x_fmt, gate_kind, alpha, eps, ld_h, ld_y, ld_x),
           hp, yp, q, g, p, dhp, dxp, o_h, o_y, dq, dg, dp, w, wn)


def moe_decode_block(ctx: Ctx, layer, x, T, logit_bias, topk_idx, topk_w, slot_idx, y, norm: moe_norm_config, h,
                     w_post=None, gate=None, w_pre=None, x_next=None, stream=None) -> None:
    """One decode layer step (moe_decode_layer into y) and moe_block_norm of y into h, in place, and x_next."""
    _check(ctx, lib.moe_decode_block(ctx.handle, layer, _ptr(x), T, _ptr(logit_bias), _ptr(topk_idx), _ptr(topk_w),
                                     _ptr(slot_idx), _ptr(y), ctypes.byref(norm), _ptr(h), _ptr(w_post), _ptr(gate),
                                     _ptr(w_pre), _ptr(x_next), _stream(stream)), "moe_decode_block")
