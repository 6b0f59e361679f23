"""GPU: the sort without rows (x = xs = NULL) in each of its forms, eager, captured and with values in
the arguments that it does not use, against the sort with rows."""
import numpy as np
import pytest
import torch

from test_gpu_tokens import R, check_dispatch, dev, routing, run_dispatch

pytestmark = pytest.mark.gpu

# one launch; two; three (chunks of 1024 pairs, and of more), with few and many experts
FORMS = [(3, 5, 7), (128, 8, 256), (2000, 4, 33), (16384, 1, 1024), (5000, 8, 256), (17, 1000, 1000), (150000, 2, 3), (70000, 4, 1000)]


@pytest.mark.parametrize("T,k,E", FORMS)
@pytest.mark.parametrize("unused", [(0, 0, 0), (-7, 2 ** 31 - 1, -1), (1, -(2 ** 31), 2 ** 62), (5, 65536, 3)])
def test_sort_alone(T, k, E, unused):
    r = R()
    idx = routing(T, k, E, 0.1)
    x = torch.arange(T, device="cuda", dtype=torch.float32)[:, None]
    want = run_dispatch(idx, E, x)
    check_dispatch(idx, E, x, want)
    ids = dev(idx)
    perm, inv, off = (torch.full(s, -7, dtype=torch.int32, device="cuda") for s in ((T * k,), (T, k), (E + 1,)))
    ws = torch.empty(r.moe_dispatch_workspace(T, k, E), dtype=torch.uint8, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    assert r.lib.moe_dispatch(ids.data_ptr(), T, k, E, None, *unused, None, perm.data_ptr(), inv.data_ptr(), off.data_ptr(),
                              ws.data_ptr() or None, ws.numel(), s) == r.MOE_OK
    for got, ref in zip((perm, inv, off), want[1:]):
        assert torch.equal(got, ref)


@pytest.mark.parametrize("T,k,E", [(128, 8, 256), (2000, 4, 33), (5000, 8, 256)])
def test_captured(T, k, E):
    r = R()
    g = torch.Generator(device="cuda").manual_seed(T)
    idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
    tables = [[torch.full(s, -7, dtype=torch.int32, device="cuda") for s in ((T * k,), (T, k), (E + 1,))] for _ in range(2)]
    ws = [torch.empty(r.moe_dispatch_workspace(T, k, E), dtype=torch.uint8, device="cuda") for _ in range(2)]
    idx.copy_(torch.randint(0, E, (T, k), device="cuda", generator=g))
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            r.moe_dispatch(idx, E, None, None, *tables[0], ws[0])
    for _ in range(3):
        idx.copy_(torch.randint(0, E, (T, k), device="cuda", generator=g))      # every pair kept: perm is written whole
        torch.cuda.synchronize()
        graph.replay()
        r.moe_dispatch(idx, E, None, None, *tables[1], ws[1])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(*tables))
        order = np.argsort(idx.cpu().numpy().reshape(-1), kind="stable")
        assert np.array_equal(tables[0][0].cpu().numpy(), order)
