"""GPU: a projection's bias gradient without the others, with the workspace of its sizes."""
import pytest
import torch

from oracle import products
from test_gpu_products import B, F, FILL, R, act_kind, dev, f64, fmt_of, uneven, within

pytestmark = pytest.mark.gpu


# wide products, which are not split along the k, so that their workspace holds no parts of sums; dy in fp32 where the
# operands are bf16
@pytest.mark.parametrize("act,y_dtype", [("none", B), ("none", F), ("gelu", B), ("gelu", F)])
@pytest.mark.parametrize("rows,E,K,N", [(777, 0, 1000, 1001), (2048, 0, 2048, 512), (1500, 4, 1024, 640)])
def test_bias_alone(rows, E, K, N, act, y_dtype):
    L = R()
    g = torch.Generator(device="cuda").manual_seed(rows + N)
    rnd = lambda dt, *s: torch.randn(*s, device="cuda", generator=g).to(dt)  # noqa: E731
    off, n = uneven(rows, E, 5) if E else None, max(E, 1)
    dy, z, x, w = rnd(y_dtype, rows, N), rnd(B, rows, N) if act != "none" else None, rnd(B, rows, K), rnd(B, n, N, K)
    ws = torch.full((L.moe_linear_workspace(rows, n, K, N, fmt_of(B)),), 255, dtype=torch.uint8, device="cuda")
    db, all_db = (torch.full((n, N), FILL, device="cuda") for _ in range(2))
    L.moe_linear_backward(dy, z, None, None, None, None, db, ws, dev(off), act=act_kind(act))
    dx, dw = torch.empty(rows, K, dtype=B, device="cuda"), torch.empty(n, N, K, dtype=B, device="cuda")
    L.moe_linear_backward(dy, z, x, w, dx, dw, all_db, ws, dev(off), act=act_kind(act))
    assert torch.equal(db, all_db)
    thin = torch.zeros(rows, 1).double().numpy(), torch.zeros(n, N, 1).double().numpy()   # the bias knows neither x nor w
    ref, _ = products.linear_backward(f64(dy), f64(z), *thin, off, act)
    within("dbias", db, ref["dbias"], F)
