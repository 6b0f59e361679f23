"""GPU: every way to name a stream of the tensors' device leads to the same call."""
import pytest
import torch

from test_gpu_tokens import R

pytestmark = pytest.mark.gpu


def buffers():
    inv = torch.tensor([[0, 1], [3, 2]], dtype=torch.int32, device="cuda:0")
    return torch.randn(4, 33, device="cuda:0"), inv, torch.rand(2, 2, device="cuda:0")


def test_handles_of_the_tensors_device():
    """The null stream, the legacy one and the thread's own by their handles, a stream's handle and object."""
    r = R()
    ys, inv, w = buffers()
    h, wp, z = torch.randn(3, 40, device="cuda:0"), torch.rand(40, device="cuda:0"), torch.randn(2, 4, device="cuda:0")
    side = torch.cuda.Stream(device=0)
    want = None
    for stream in (None, 0, side.cuda_stream, side, torch.cuda.ExternalStream(side.cuda_stream), 2, 1):
        out = [torch.zeros(n, 33, device="cuda:0") for n in (2, 2, 4)]
        tables = [torch.zeros(n, dtype=torch.int32, device="cuda:0") for n in (4, (2, 2), 5)]
        dw, dz, x, dh, dwp = (torch.zeros(s, device="cuda:0") for s in ((2, 2), (2, 4), (3, 40), (3, 40), 40))
        ws = torch.empty(r.moe_block_norm_workspace(3, 40), dtype=torch.uint8, device="cuda:0")
        torch.cuda.synchronize()
        r.moe_combine(ys, inv, w, out[0], stream=stream)
        r.moe_dispatch_backward(ys, inv, out[1], stream=stream)
        r.moe_combine_backward(out[0], ys, inv, w, out[2], dw, stream=stream)
        r.moe_dispatch(inv, 4, None, None, *tables, stream=stream)
        r.moe_topk_backward(z, inv, w, 1, dz, stream=stream)
        r.moe_block_norm(h, None, None, None, wp, None, x, stream=stream)
        r.moe_block_norm_backward(h, None, None, None, wp, None, x, dh, None, None, None, dwp, ws, stream=stream)
        torch.cuda.synchronize()
        got = out + tables + [dw, dz, x, dh, dwp]
        want = want or got
        assert all(torch.equal(a, b) for a, b in zip(got, want)), stream


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs a second device")
def test_handles_of_another_device():
    ys, inv, w = buffers()
    y = torch.zeros(2, 33, device="cuda:0")
    other = torch.cuda.Stream(device=1)
    for stream in (other, other.cuda_stream):
        with pytest.raises(R().MoeError, match="stream is on cuda:1"):
            R().moe_combine(ys, inv, w, y, stream=stream)
    want = torch.empty_like(y)
    R().moe_combine(ys, inv, w, want)
    with torch.cuda.device(1):              # the tensors' device counts, not the current one
        R().moe_combine(ys, inv, w, y)
        assert torch.cuda.current_device() == 1
    torch.cuda.synchronize(0)
    assert torch.equal(y, want)
