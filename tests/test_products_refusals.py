"""Refusals of the experts' products, on the CPU: what the library and its binding turn away before anything
is enqueued (pointers here are never followed)."""
import ctypes

import pytest
import torch

import routed_expert_ffn_02_amd as R

L = R.lib
# far-apart addresses, 16-byte aligned
A = [0x10_0000_0000 * (i + 1) for i in range(16)]
F32, BF16 = R.MOE_AFMT_F32, R.MOE_AFMT_BF16
BIG = 1 << 30


def config(**kw):
    a = dict(rows=40, n_experts=4, K=64, N=32, fmt=BF16, y_fmt=BF16, dw_fmt=BF16, act=R.MOE_ACT_SILU, ld_x=0, ld_dx=0, ld_w=0,
             gs_w=0, ld_y=0, ld_residual=0, ld_z=0)
    a.update(kw)
    return R.moe_product_config(*a.values())


def glu(cfg=None, **kw):
    a = dict(x=A[0], w=A[1], off=A[2], a=A[3], gu=A[4])
    a.update(kw)
    return L.moe_glu(ctypes.byref(cfg or config()), *a.values(), None)


def glu_backward(cfg=None, **kw):
    a = dict(da=A[0], gu=A[1], x=A[2], w=A[3], off=A[4], dx=A[5], dw=A[6], ws=A[7], n=BIG)
    a.update(kw)
    return L.moe_glu_backward(ctypes.byref(cfg or config()), *a.values(), None)


def linear(cfg=None, **kw):
    a = dict(x=A[0], w=A[1], bias=A[2], residual=A[3], off=A[4], y=A[5], z=A[6])
    a.update(kw)
    return L.moe_linear(ctypes.byref(cfg or config()), *a.values(), None)


def linear_backward(cfg=None, **kw):
    a = dict(dy=A[0], z=A[1], x=A[2], w=A[3], off=A[4], dx=A[5], dw=A[6], db=A[7], ws=A[8], n=BIG)
    a.update(kw)
    return L.moe_linear_backward(ctypes.byref(cfg or config()), *a.values(), None)


CALLS = [glu, glu_backward, linear, linear_backward]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("bad", [
    dict(rows=0), dict(rows=-1), dict(rows=(1 << 26) + 1), dict(n_experts=0), dict(n_experts=1025), dict(K=0), dict(K=65537),
    dict(N=0), dict(N=-4), dict(N=65537), dict(fmt=2), dict(fmt=-1), dict(y_fmt=2), dict(dw_fmt=7), dict(act=3), dict(act=-1),
    dict(ld_x=63), dict(ld_x=(1 << 36) + 1), dict(ld_dx=1), dict(ld_w=63), dict(ld_w=-64), dict(gs_w=31 * 64 + 63), dict(gs_w=-1),
    dict(gs_w=(1 << 36) + 1), dict(ld_y=31), dict(ld_y=-32), dict(ld_z=31), dict(ld_residual=31)])
def test_config_refused(call, bad):
    assert call(config(**bad)) == R.MOE_EINVAL


@pytest.mark.parametrize("call", CALLS)
def test_experts_need_offsets_and_products_a_config(call):
    assert call(off=None) == R.MOE_EINVAL
    f = getattr(L, "moe_" + call.__name__)
    assert f(None, *A[:len(f.argtypes) - 2 - (ctypes.c_size_t in f.argtypes)], *([BIG] if ctypes.c_size_t in f.argtypes else []), None) == R.MOE_EINVAL


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(w=None), dict(a=None), dict(x=A[0] + 1), dict(w=A[1] + 1), dict(a=A[3] + 1), dict(gu=A[4] + 1), dict(off=A[2] + 2),
    dict(a=A[0]), dict(a=A[1] + 4 * 64 * 64 * 2 - 2), dict(a=A[2]), dict(gu=A[0] + 40 * 128 - 2), dict(gu=A[3]), dict(gu=A[1])])
def test_glu_refuses(bad):
    assert glu(**bad) == R.MOE_EINVAL


@pytest.mark.parametrize("bad", [
    dict(da=None), dict(gu=None), dict(x=None), dict(w=None), dict(dx=None, dw=None), dict(ws=None), dict(n=100), dict(da=A[0] + 1),
    dict(gu=A[1] + 1), dict(x=A[2] + 1), dict(w=A[3] + 1), dict(dx=A[5] + 1), dict(dw=A[6] + 1), dict(off=A[4] + 1), dict(dx=A[0]),
    dict(dx=A[2]), dict(dw=A[3]), dict(dw=A[5]), dict(ws=A[1]), dict(ws=A[5] - 8), dict(dx=A[4])])
def test_glu_backward_refuses(bad):
    assert glu_backward(**bad) == R.MOE_EINVAL


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(w=None), dict(y=None), dict(x=A[0] + 1), dict(w=A[1] + 1), dict(bias=A[2] + 2), dict(residual=A[3] + 1),
    dict(off=A[4] + 2), dict(y=A[5] + 1), dict(z=A[6] + 1), dict(y=A[0]), dict(y=A[1]), dict(y=A[2]), dict(y=A[3] + 64), dict(y=A[4]),
    dict(z=A[5]), dict(z=A[3]), dict(z=A[0])])
def test_linear_refuses(bad):
    assert linear(**bad) == R.MOE_EINVAL


def test_linear_in_place_needs_one_stride():
    assert linear(config(ld_residual=64), residual=A[5]) == R.MOE_EINVAL


@pytest.mark.parametrize("bad", [
    dict(dy=None), dict(z=None), dict(x=None), dict(w=None), dict(dx=None, dw=None, db=None), dict(ws=None), dict(n=100),
    dict(dy=A[0] + 1), dict(z=A[1] + 1), dict(x=A[2] + 1), dict(w=A[3] + 1), dict(dx=A[5] + 1), dict(dw=A[6] + 1), dict(db=A[7] + 2),
    dict(off=A[4] + 2), dict(dx=A[0]), dict(dx=A[3]), dict(dw=A[2]), dict(db=A[4]), dict(db=A[6]), dict(ws=A[7]), dict(dw=A[1])])
def test_linear_backward_refuses(bad):
    assert linear_backward(**bad) == R.MOE_EINVAL


def test_workspaces():
    for f in (R.moe_glu_workspace, R.moe_linear_workspace):
        for bad in ((0, 1, 8, 8, F32), (8, 0, 8, 8, F32), (8, 1025, 8, 8, F32), (8, 1, 0, 8, F32), (8, 1, 8, 0, F32), (8, 1, 8, 8, 2),
                    ((1 << 26) + 1, 1, 8, 8, F32), (8, 1, 65537, 8, F32), (8, 1, 8, 65537, F32), (1 << 40, 1, 8, 8, F32)):
            with pytest.raises(R.MoeError):
                f(*bad)
        assert f(1 << 26, 1024, 1 << 16, 1 << 16, F32) > 1 << 43   # no overflow
        assert f(1, 1, 1, 1, BF16) > 0
    # d of both projections, and of one
    assert R.moe_glu_workspace(1000, 8, 64, 96, BF16) >= 1000 * 192 * 2
    assert R.moe_linear_workspace(1000, 8, 64, 96, F32) >= 1000 * 96 * 4
    # sums of a long k in parts: of dw [64, 48] over many rows, of dx [3, 48] over many outputs; some MB at most
    for rows, n in ((8192, 64), (3, 8192)):
        d = rows * n * 4
        assert d + 4 * min(rows, 64) * 48 <= R.moe_linear_workspace(rows, 1, 48, n, F32) <= d + (10 << 20)


def test_too_many_tiles():
    assert glu(config(rows=1 << 26, N=65536), a=A[3], gu=None, w=1 << 50, x=1 << 52) == R.MOE_EINVAL


@pytest.mark.parametrize("out", ["dx", "dw"])
@pytest.mark.parametrize("fmt", [BF16, F32])
def test_too_many_tiles_of_a_gradient(fmt, out):
    """Refused before anything is enqueued: a launch would fail here, and say so with another error."""
    c = config(rows=1 << 26, n_experts=1, K=65536, N=64, fmt=fmt) if out == "dx" else config(rows=8, n_experts=1024, K=65536, N=65536, fmt=fmt)
    far = dict(x=1 << 50, w=1 << 52, ws=1 << 54, n=1 << 50, dx=None, dw=None)
    far[out] = 1 << 56
    assert glu_backward(c, da=1 << 44, gu=1 << 48, off=None if out == "dx" else A[4], **far) == R.MOE_EINVAL
    assert linear_backward(c, dy=1 << 44, z=1 << 48, off=None if out == "dx" else A[4], **{**far, "db": 1 << 40}) == R.MOE_EINVAL


# --- the binding's own checks ------------------------------------------------
def refused(f, *a, **kw):
    with pytest.raises(R.MoeError) as e:
        f(*a, **kw)
    assert e.value.status == R.MOE_EINVAL
    return str(e.value)


T, E, H, I = 6, 3, 8, 4


def f32(*s):
    return torch.zeros(s)


def off():
    return torch.zeros(E + 1, dtype=torch.int32)


@pytest.mark.parametrize("bad,msg", [
    (dict(), "on the GPU"), (dict(x=f32(H)), "two-dimensional"), (dict(x=f32(T, H).half()), "fp32 or bf16"), (dict(x=None), "tensor"),
    (dict(x=f32(T, 0)), "shape"), (dict(x=f32(H, T).t()), "contiguous rows"), (dict(w=None), "w must be"), (dict(w=f32(2 * I)), "three-dimensional"),
    (dict(w=f32(E, 2 * I, H).double()), "fp32 or bf16"), (dict(w=f32(E, 2 * I, H).bfloat16()), "operands' type"),
    (dict(w=f32(E + 1, 2 * I, H)), "shape"), (dict(w=f32(E, 2 * I + 1, H)), "shape"), (dict(w=f32(E, 2 * I, H + 1)), "shape"),
    (dict(w=f32(2 * I, H)), "shape"), (dict(w=f32(E, H, 2 * I).transpose(1, 2)), "contiguous rows"), (dict(w=f32(E, 0, H)), "size may be 0"),
    (dict(w=f32(1, 2 * I, H).expand(E, 2 * I, H)), "one after the other"), (dict(w=f32(E, 1, H).expand(E, 2 * I, H)), "contiguous rows"),
    (dict(a=f32(T, I + 1)), "shape"), (dict(a=f32(T + 1, I)), "shape"), (dict(a=f32(T, I).bfloat16()), "operands' type"), (dict(a=None), "tensor"),
    (dict(gu=f32(T, I)), "shape"), (dict(gu=f32(T, 2 * I).bfloat16()), "operands' type"), (dict(offsets=off().long()), "int32"),
    (dict(offsets=off()[:1]), "experts + 1"), (dict(offsets=off().view(2, 2)), "experts + 1"), (dict(offsets=None), "shape"),
    (dict(act="silu"), "integer"), (dict(x=[1]), "tensor"), (dict(x=f32(T, H).to_sparse()), "strided")])
def test_glu_binding_refuses(bad, msg):
    a = dict(x=f32(T, H), w=f32(E, 2 * I, H), a=f32(T, I), gu=f32(T, 2 * I), offsets=off())
    a.update(bad)
    assert msg in refused(R.moe_glu, **a)


@pytest.mark.parametrize("bad,msg", [
    (dict(), "on the GPU"), (dict(da=None), "tensor"), (dict(gu=None), "tensor"), (dict(gu=f32(T, I)), "shape"),
    (dict(gu=f32(T, 2 * I).bfloat16()), "operands' type"), (dict(w=None), "dx needs w"), (dict(w=f32(E, I, H)), "shape"),
    (dict(x=None), "x must be"), (dict(x=f32(T, H + 1)), "shape"), (dict(x=f32(T, H).bfloat16()), "operands' type"),
    (dict(dx=f32(T, H + 1)), "shape"), (dict(dx=f32(T, H).bfloat16()), "operands' type"), (dict(dx=None, dw=None), "must be given"),
    (dict(dw=f32(E, I, H)), "shape"), (dict(dw=f32(E, 2 * I, H).half()), "fp32 or bf16"), (dict(dw=f32(E, 2 * I, 2 * H)[:, :, :H]), "contiguous"),
    (dict(dw=f32(2 * I, H)), "shape"), (dict(dw=f32(E, 2 * I, H).bfloat16()), "on the GPU"), (dict(dx=None, w=None), "on the GPU"),
    (dict(dw=None, x=None), "on the GPU"), (dict(ws=f32(4, 2).t()), "ws must be"), (dict(act=None), "integer")])
def test_glu_backward_binding_refuses(bad, msg):
    a = dict(da=f32(T, I), gu=f32(T, 2 * I), x=f32(T, H), w=f32(E, 2 * I, H), dx=f32(T, H), dw=f32(E, 2 * I, H), ws=f32(100), offsets=off())
    a.update(bad)
    assert msg in refused(R.moe_glu_backward, **a)


@pytest.mark.parametrize("bad,msg", [
    (dict(), "on the GPU"), (dict(w=f32(E, I, H + 1)), "shape"), (dict(y=f32(T, I + 1)), "shape"), (dict(y=f32(T, I).half()), "fp32 or bf16"),
    (dict(y=f32(T, I).bfloat16()), "y's type"), (dict(bias=f32(I)), "shape"), (dict(bias=f32(E, I).bfloat16()), "float32"),
    (dict(bias=f32(I, E).t()), "contiguous"), (dict(residual=f32(T, I).bfloat16()), "y's type"), (dict(residual=f32(T + 1, I)), "shape"),
    (dict(z=f32(T, I).bfloat16()), "operands' type"), (dict(z=f32(T, I + 1)), "shape"), (dict(offsets=None), "shape"),
    (dict(y=f32(T, I).bfloat16(), residual=None), "on the GPU")])
def test_linear_binding_refuses(bad, msg):
    a = dict(x=f32(T, H), w=f32(E, I, H), y=f32(T, I), bias=f32(E, I), residual=f32(T, I), z=f32(T, I), offsets=off())
    a.update(bad)
    assert msg in refused(R.moe_linear, **a)


@pytest.mark.parametrize("bad,msg", [
    (dict(), "on the GPU"), (dict(dy=None), "tensor"), (dict(z=None), "z must be"), (dict(z=f32(T, I + 1)), "shape"),
    (dict(z=f32(T, I).bfloat16()), "operands' type"), (dict(z=None, act=R.MOE_ACT_NONE), "on the GPU"), (dict(w=None), "dx needs w"),
    (dict(x=None), "x must be"), (dict(x=f32(T, H).bfloat16()), "operands' type"), (dict(dx=None, dw=None, dbias=None), "must be given"),
    (dict(dbias=f32(E, I).double()), "float32"), (dict(dbias=f32(I)), "shape"), (dict(dw=f32(E, H, I)), "shape"),
    (dict(dy=f32(T, I).bfloat16()), "on the GPU"), (dict(offsets=None), "shape")])
def test_linear_backward_binding_refuses(bad, msg):
    a = dict(dy=f32(T, I), z=f32(T, I), x=f32(T, H), w=f32(E, I, H), dx=f32(T, H), dw=f32(E, I, H), dbias=f32(E, I), ws=f32(100),
             offsets=off(), act=R.MOE_ACT_SILU)
    a.update(bad)
    assert msg in refused(R.moe_linear_backward, **a)


def test_what_is_taken_goes_on_to_its_launch():
    """Calls that nothing refuses end at the launch, which fails here without a device."""
    if torch.cuda.is_available():
        pytest.skip("the pointers are not memory: this runs where nothing can be launched")
    assert glu() == glu(gu=None) == R.MOE_EHIP
    assert glu(config(n_experts=1), off=None) == R.MOE_EHIP
    assert glu(config(ld_y=64, ld_z=64), gu=A[3] + 5 * 40 * 128) == R.MOE_EHIP
    assert linear(residual=A[5]) == linear(bias=None, residual=None, z=None) == R.MOE_EHIP
    assert linear(config(ld_x=96, ld_y=96), y=A[0] + 128) == R.MOE_EHIP      # side by side in one buffer's rows
    assert linear(config(ld_x=96, ld_y=96), y=A[0] + 126) == R.MOE_EINVAL
    assert glu_backward() == glu_backward(dx=None, w=None) == glu_backward(dw=None, x=None) == R.MOE_EHIP
    assert linear_backward() == linear_backward(dx=None, w=None, dw=None, x=None) == R.MOE_EHIP
    assert linear_backward(config(act=R.MOE_ACT_NONE), z=None, ws=A[8] + 3) == R.MOE_EHIP
    n = R.moe_glu_workspace(40, 4, 64, 32, BF16)
    assert glu_backward(n=n) == R.MOE_EHIP and glu_backward(n=n - 1) == R.MOE_EINVAL


def test_struct_layout():
    assert ctypes.sizeof(R.moe_product_config) == 8 * 4 + 7 * 8
