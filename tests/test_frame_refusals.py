"""Refusals of the calls around the experts, on the CPU: what the library and its binding turn away
before anything is enqueued (pointers here are never followed)."""
import ctypes

import pytest
import torch

import routed_expert_ffn_02_amd as R

L = R.lib
# far-apart addresses, 16-byte aligned
A = [0x10_0000_0000 * (i + 1) for i in range(16)]
F32, BF16 = R.MOE_AFMT_F32, R.MOE_AFMT_BF16


def dispatch(**kw):
    a = dict(idx=A[0], T=8, k=2, E=4, x=A[1], fmt=BF16, H=64, ld=0, xs=A[2], perm=A[3], inv=A[4], off=A[5], ws=A[6],
             n=1 << 20)
    a.update(kw)
    return L.moe_dispatch(*a.values(), None)


LONG = dict(T=1 << 15, k=4)   # a sort that needs a workspace


@pytest.mark.parametrize("bad", [
    dict(idx=None), dict(perm=None), dict(inv=None), dict(off=None), dict(LONG, ws=None), dict(x=None), dict(xs=None),
    dict(T=0), dict(T=-1), dict(T=(1 << 21) + 1), dict(k=0), dict(k=1025), dict(T=1 << 20, k=128), dict(E=0), dict(E=1025),
    dict(fmt=2), dict(fmt=-1), dict(H=0), dict(H=65537), dict(ld=63), dict(ld=-64), dict(ld=(1 << 36) + 1), dict(LONG, n=3), dict(x=A[1] + 1),
    dict(xs=A[2] + 1), dict(LONG, ws=A[6] + 2),
    dict(xs=A[1]), dict(xs=A[1] + 8 * 128 - 2), dict(perm=A[4]), dict(inv=A[5]), dict(inv=A[0]), dict(off=A[2]),
    dict(LONG, ws=A[3]), dict(perm=A[2] + 16 * 128 - 4)])
def test_dispatch_refuses(bad):
    assert dispatch(**bad) == R.MOE_EINVAL


def move(which, **kw):
    if which == "back":
        a = dict(dxs=A[0], fmt=BF16, inv=A[1], T=8, k=2, H=64, dx=A[2], out_fmt=F32, ld=0)
        a.update(kw)
        return L.moe_dispatch_backward(*a.values(), None)
    a = dict(ys=A[0], fmt=BF16, inv=A[1], w=A[3], T=8, k=2, H=64, y=A[2], out_fmt=F32, ld=0)
    a.update(kw)
    return L.moe_combine(*a.values(), None)


@pytest.mark.parametrize("bad", [
    dict(dxs=None), dict(inv=None), dict(dx=None), dict(fmt=3), dict(out_fmt=-1), dict(T=0), dict(k=0), dict(H=0),
    dict(ld=10), dict(dx=A[0]), dict(dx=A[1]), dict(dxs=A[0] + 1), dict(dx=A[2] + 2)])
def test_dispatch_backward_refuses(bad):
    assert move("back", **bad) == R.MOE_EINVAL


@pytest.mark.parametrize("bad", [
    dict(ys=None), dict(inv=None), dict(w=None), dict(y=None), dict(fmt=3), dict(out_fmt=7), dict(T=0), dict(k=2000),
    dict(H=1 << 20), dict(ld=1), dict(y=A[0]), dict(y=A[1]), dict(y=A[3]), dict(y=A[2] + 2)])
def test_combine_refuses(bad):
    assert move("combine", **bad) == R.MOE_EINVAL


def combine_backward(**kw):
    a = dict(dy=A[0], dfmt=F32, ld=0, ys=A[1], fmt=BF16, inv=A[2], w=A[3], T=8, k=2, H=64, dys=A[4], dw=A[5])
    a.update(kw)
    return L.moe_combine_backward(*a.values(), None)


@pytest.mark.parametrize("bad", [
    dict(dy=None), dict(inv=None), dict(dys=None, dw=None), dict(ys=None), dict(w=None), dict(dfmt=5), dict(fmt=5),
    dict(T=0), dict(H=0), dict(ld=2), dict(dys=A[0]), dict(dys=A[1] + 2), dict(dw=A[3]), dict(dw=A[4]), dict(dw=A[2]),
    dict(dys=A[4] + 1)])
def test_combine_backward_refuses(bad):
    assert combine_backward(**bad) == R.MOE_EINVAL


def topk(**kw):
    a = dict(z=A[0], T=8, E=16, idx=A[1], k=2, dw=A[2], renorm=0, dz=A[3])
    a.update(kw)
    return L.moe_topk_backward(*a.values(), None)


@pytest.mark.parametrize("bad", [
    dict(z=None), dict(idx=None), dict(dw=None), dict(dz=None), dict(T=0), dict(E=0), dict(E=1025), dict(k=0),
    dict(renorm=2), dict(renorm=-1), dict(dz=A[0] + 4), dict(dz=A[1]), dict(dz=A[2])])
def test_topk_backward_refuses(bad):
    assert topk(**bad) == R.MOE_EINVAL


def norm_cfg(**kw):
    a = dict(T=8, H=64, h=BF16, y=F32, x=BF16, gate_kind=R.MOE_GATE_CHANNEL, alpha=1.0, eps=1e-6, ld_h=0, ld_y=0, ld_x=0)
    a.update(kw)
    return R.moe_norm_config(*a.values())


BAD_CONFIG = [dict(T=0), dict(T=(1 << 21) + 1), dict(H=0), dict(H=8193), dict(h=2), dict(y=-1), dict(x=9),
              dict(gate_kind=3), dict(gate_kind=-1), dict(alpha=float("inf")), dict(alpha=float("nan")), dict(eps=0.0), dict(eps=1e-40),
              dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=2.0), dict(ld_h=63), dict(ld_h=(1 << 36) + 1), dict(ld_y=-1), dict(ld_x=1)]


def norm(cfg=None, **kw):
    a = dict(h=A[0], y=A[1], w_post=A[2], gate=A[3], w_pre=A[4], h_out=A[5], x_out=A[6])
    a.update(kw)
    return L.moe_block_norm(ctypes.byref(cfg or norm_cfg()), *a.values(), None)


@pytest.mark.parametrize("bad", BAD_CONFIG)
def test_norm_config_refused(bad):
    assert norm(norm_cfg(**bad)) == R.MOE_EINVAL
    assert norm_backward(norm_cfg(**bad)) == R.MOE_EINVAL


@pytest.mark.parametrize("bad", [
    dict(h=None), dict(y=None), dict(h_out=None), dict(gate=None), dict(w_pre=None), dict(x_out=None),
    dict(h_out=A[1]), dict(x_out=A[0]), dict(x_out=A[5]), dict(h_out=A[0] + 2), dict(h_out=A[4]), dict(x_out=A[2]),
    dict(h=A[1], h_out=A[1]), dict(h=A[0] + 1), dict(y=A[1] + 2), dict(w_post=A[2] + 2), dict(x_out=A[6] + 1)])
def test_norm_refuses(bad):
    assert norm(**bad) == R.MOE_EINVAL
    assert L.moe_block_norm(None, *A[:7], None) == R.MOE_EINVAL


def test_norm_gate_must_match_its_kind():
    assert norm(norm_cfg(gate_kind=R.MOE_GATE_NONE)) == R.MOE_EINVAL
    assert norm(y=None, w_post=None, h_out=None) == R.MOE_EINVAL          # a gate without a block's output


def norm_backward(cfg=None, **kw):
    a = dict(h_out=A[0], y=A[1], w_post=A[2], gate=A[3], w_pre=A[4], dh_out=A[5], dx=A[6], dh=A[7], dy=A[8],
             dw_post=A[9], dgate=A[10], dw_pre=A[11], ws=A[12], n=1 << 24)
    a.update(kw)
    return L.moe_block_norm_backward(ctypes.byref(cfg or norm_cfg()), *a.values(), None)


@pytest.mark.parametrize("bad", [
    dict(dh_out=None, dx=None), dict(dh=None, dy=None, dw_post=None, dgate=None, dw_pre=None), dict(h_out=None),
    dict(w_pre=None), dict(dx=None), dict(y=None), dict(w_post=None), dict(gate=None), dict(ws=None), dict(n=100),
    dict(ws=A[12] + 1), dict(dh=A[0]), dict(dh=A[5] + 2), dict(dh_out=A[1], dh=A[1]), dict(y=A[0], dy=A[0]), dict(dy=A[1] + 4), dict(dy=A[7]), dict(dgate=A[9]),
    dict(dw_pre=A[4]), dict(ws=A[8]), dict(dx=A[6] + 1)])
def test_norm_backward_refuses(bad):
    assert norm_backward(**bad) == R.MOE_EINVAL


def test_workspace_sizes():
    for bad in ((0, 1, 1), (1, 0, 1), (1, 1, 0), (1, 1, 1025), (1 << 21, 1024, 8)):
        assert L.moe_dispatch_workspace(*bad) == -1
        with pytest.raises(R.MoeError):
            R.moe_dispatch_workspace(*bad)
    assert 0 < R.moe_dispatch_workspace(1 << 20, 64, 1024) <= 4 * (1 << 26) + (1 << 21)   # a word a pair and the histograms
    assert R.moe_dispatch_workspace(LONG["T"], LONG["k"], 4) > 3
    for bad in ((0, 1), (1, 0), (1, 8193)):
        with pytest.raises(R.MoeError):
            R.moe_block_norm_workspace(*bad)
    assert R.moe_block_norm_workspace(4096, 2048) == R.moe_block_norm_workspace(1 << 21, 2048)   # bounded


# --- the binding's own checks ------------------------------------------------
def refused(f, *a, **kw):
    with pytest.raises(R.MoeError) as e:
        f(*a, **kw)
    assert e.value.status == R.MOE_EINVAL
    return str(e.value)


T, k, H, E = 4, 2, 8, 4


def i32(*s):
    return torch.zeros(s, dtype=torch.int32)


def f32(*s):
    return torch.zeros(s)


def tables():
    return [i32(T * k), i32(T, k), i32(E + 1)]


@pytest.mark.parametrize("bad,msg", [
    (dict(), "topk_idx must be on the GPU"), (dict(topk_idx=i32(T, k).long()), "int32"), (dict(topk_idx=i32(T * k)), "T, k"),
    (dict(topk_idx=i32(0, k)), "T, k"), (dict(topk_idx=i32(k, T).t()), "contiguous"), (dict(topk_idx=None), "tensor"),
    (dict(topk_idx=[[0, 1]]), "tensor"), (dict(n_experts=1 << 40), "out of range"), (dict(n_experts="4"), "integer"),
    (dict(x=f32(T, H).half()), "fp32 or bf16"), (dict(x=f32(T, H).double()), "fp32 or bf16"),
    (dict(x=f32(H)), "two-dimensional"), (dict(x=f32(H, T).t()), "contiguous rows"),
    (dict(x=f32(T, 2 * H)[:, ::2]), "contiguous rows"), (dict(x=f32(1, H).expand(T, H)), "contiguous rows"),
    (dict(x=f32(5, H)), "shape"), (dict(x=f32(T, 0)), "shape"), (dict(x=None), "x must be a tensor"),
    (dict(xs=None), "xs must be a tensor"), (dict(xs=f32(T * k, 2 * H)[:, :H]), "without gaps"), (dict(xs=f32(T * k, 9)), "shape"),
    (dict(xs=f32(T * k, H).bfloat16()), "x's type"), (dict(perm=i32(T * k + 1)), "shape"), (dict(perm=f32(T * k)), "int32"),
    (dict(inv=i32(k, T)), "shape"), (dict(offsets=i32(E)), "shape"), (dict(ws=f32(4, 2).t()), "ws must be a contiguous"),
    (dict(x=f32(T, H).to_sparse()), "strided"), (dict(topk_idx=i32(T, k).to("meta")), "on the GPU")])
def test_dispatch_binding_refuses(bad, msg):
    perm, inv, offsets = tables()
    a = dict(topk_idx=i32(T, k), n_experts=E, x=f32(T, H), xs=f32(T * k, H), perm=perm, inv=inv, offsets=offsets, ws=None)
    a.update(bad)
    assert msg in refused(R.moe_dispatch, **a)


@pytest.mark.parametrize("bad,msg", [
    (dict(), "must be on the GPU"), (dict(inv=i32(T, k).short()), "int32"), (dict(ys=f32(T * k + 1, H)), "shape"),
    (dict(w=f32(T, k).double()), "float32"), (dict(w=f32(k, T).t()), "contiguous"), (dict(w=f32(T, k + 1)), "shape"),
    (dict(w=None), "w must be a tensor"), (dict(y=f32(T, H + 1)), "shape"), (dict(y=f32(T, H).half()), "fp32 or bf16")])
def test_combine_binding_refuses(bad, msg):
    a = dict(ys=f32(T * k, H), inv=i32(T, k), w=f32(T, k), y=f32(T, H))
    a.update(bad)
    assert msg in refused(R.moe_combine, **a)
    if "w" not in bad:
        assert msg in refused(R.moe_dispatch_backward, a["ys"], a["inv"], a["y"])
        b = dict(dy=a["y"], ys=a["ys"], inv=a["inv"], w=a["w"], dys=f32(T * k, a["y"].shape[1]), dw=f32(T, k))
        if a["y"].shape == (T, H):
            assert msg in refused(R.moe_combine_backward, **b)


def test_combine_backward_binding_refuses():
    a = dict(dy=f32(T, H), ys=f32(T * k, H), inv=i32(T, k), w=f32(T, k), dys=f32(T * k, H), dw=f32(T, k))
    for bad, msg in [(dict(dys=f32(T * k, H).bfloat16()), "ys's type"), (dict(w=None), "w must be"), (dict(ys=None), "ys must be"),
                     (dict(dw=f32(T, k).bfloat16()), "float32"), (dict(dys=None, w=None), "on the GPU"),
                     (dict(dw=None, ys=None), "on the GPU")]:
        assert msg in refused(R.moe_combine_backward, **{**a, **bad})


def test_topk_backward_binding_refuses():
    a = dict(logits=f32(T, E), topk_idx=i32(T, k), dw=f32(T, k), renorm=0, dlogits=f32(T, E))
    for bad, msg in [(dict(), "on the GPU"), (dict(logits=f32(T, E).bfloat16()), "fp32"), (dict(logits=f32(T, 2 * E)[:, :E]), "gaps"),
                     (dict(logits=f32(T + 1, E)), "shape"), (dict(dlogits=f32(T, E + 1)), "shape"), (dict(renorm=None), "integer"),
                     (dict(dw=f32(T, k + 1)), "shape"), (dict(topk_idx=f32(T, k)), "int32")]:
        assert msg in refused(R.moe_topk_backward, **{**a, **bad})


def test_block_norm_binding_refuses():
    a = dict(h=f32(T, H), y=f32(T, H), w_post=f32(H), gate=f32(H), w_pre=f32(H), h_out=f32(T, H), x_out=f32(T, H),
             gate_kind=R.MOE_GATE_CHANNEL)
    wide = f32(T, 2 * H)[:, :H]
    for bad, msg in [(dict(), "on the GPU"), (dict(h_out=f32(T, H).bfloat16()), "belongs to"), (dict(h_out=wide), "belongs to"),
                     (dict(gate_kind=R.MOE_GATE_NONE), "go together"), (dict(gate=None), "go together"), (dict(y=f32(T + 1, H)), "shape"),
                     (dict(gate=f32(T), gate_kind=R.MOE_GATE_CHANNEL), "shape"), (dict(w_pre=f32(H + 1)), "shape"),
                     (dict(w_post=f32(H).bfloat16()), "float32"), (dict(alpha="a"), "number"), (dict(h=None), "h must be"),
                     (dict(gate_kind=1.5), "integer")]:
        assert msg in refused(R.moe_block_norm, **{**a, **bad})
    b = dict(h_out=f32(T, H), y=f32(T, H), w_post=f32(H), gate=f32(H), w_pre=f32(H), dh_out=f32(T, H), dx=f32(T, H), dh=f32(T, H),
             dy=f32(T, H), dw_post=f32(H), dgate=f32(H), dw_pre=f32(H), gate_kind=R.MOE_GATE_CHANNEL)
    for bad, msg in [(dict(), "on the GPU"), (dict(dh_out=None, dx=None), "dh_out or dx"), (dict(dx=f32(T, H + 1)), "shape"),
                     (dict(h_out=wide), "belongs to"), (dict(dh=wide), "belongs to"), (dict(dy=f32(T, H).bfloat16()), "belongs to"),
                     (dict(dgate=f32(T + 1)), "shape"), (dict(dw_pre=f32(H).double()), "float32"),
                     (dict(dh_out=None, h_out=None, dh=wide), "on the GPU")]:
        assert msg in refused(R.moe_block_norm_backward, **{**b, **bad})
    with pytest.raises(TypeError):
        R._marshal.combine(1, 2)


def test_side_by_side_blocks_of_one_buffer_are_told_apart():
    """Two halves of rows of one [8, 128] bf16 buffer: no shared byte, so no refusal for overlap: the
    call goes on to its launch, which fails here without a device and is refused for nothing else."""
    if torch.cuda.is_available():
        pytest.skip("the pointers are not memory: this runs where nothing can be launched")
    cfg = norm_cfg(y=BF16, ld_h=128, ld_x=128)
    assert norm(cfg, x_out=A[5] + 128) == R.MOE_EHIP          # h_out and x_out side by side
    assert norm(cfg, x_out=A[5] + 126) == R.MOE_EINVAL        # one element shared
    assert norm(norm_cfg(y=BF16, ld_h=128, ld_x=256), x_out=A[5] + 128) == R.MOE_EINVAL
    assert norm(cfg, x_out=A[5] + 8 * 256) == R.MOE_EHIP      # behind the last row
