"""GPU: where moe_decode_block may write.  Every refusal comes from the host before anything is
enqueued: outputs and residency tables stay as they were."""
import numpy as np
import pytest
import torch

from test_gpu_tokens import B, F, R

pytestmark = pytest.mark.gpu

EPS = 1e-6


class Step:
    """One step of a small context, all its memory in one buffer (fp32 words) so that any two blocks
    can be laid over each other inside it."""

    def __init__(self, wl, T):
        from moe_harness import Harness
        r = R()
        self.h = Harness(wl, r.MOE_MODE_OFFLOAD, n_slots=wl.n_experts)
        self.wl, self.T, self.H, self.k = wl, T, wl.hidden, wl.top_k
        self.act = F if wl.afmt == r.MOE_AFMT_F32 else B
        n = T * self.H
        self.words = 8 * n + 3 * T * self.k + T * wl.n_experts + 4 * self.H
        self.buf = torch.zeros(self.words, device="cuda")
        self.base, self.at, next_ = self.buf.data_ptr(), {}, 0
        for name, words in dict(x=2 * n, h=2 * n, y=n, xn=3 * n, idx=T * self.k, w=T * self.k, slot=T * self.k,
                                bias=T * wl.n_experts, w_post=self.H, w_pre=self.H).items():
            self.at[name] = self.base + 4 * next_
            next_ += words
        self.buf[: 2 * n].view(self.act)[:n].normal_()
        for name in ("w_post", "w_pre"):
            i = (self.at[name] - self.base) // 4
            self.buf[i:i + self.H] = 1.0

    def run(self, h_fmt=F, x_fmt=None, ld_h=0, ld_x=0, gate=None, kind=0, **at):
        r = R()
        p = {**self.at, **at}
        f = lambda t: r.MOE_AFMT_BF16 if t is B else r.MOE_AFMT_F32  # noqa: E731
        cfg = r.moe_norm_config(self.T, self.H, f(h_fmt), r.MOE_AFMT_F32, f(x_fmt or self.act), kind, 1.0, EPS, ld_h, 0, ld_x)
        r.moe_decode_block(self.h.ctx, 0, p["x"], self.T, p["bias"], p["idx"], p["w"], p["slot"], p["y"], cfg, p["h"],
                           p["w_post"], gate, p["w_pre"], p["xn"])

    def refused(self, **kw):
        torch.cuda.synchronize()
        before, tables = self.buf.clone(), self.h.snapshot()
        with pytest.raises(R().MoeError) as e:
            self.run(**kw)
        assert e.value.status == R().MOE_EINVAL and "norm" in str(e.value)
        torch.cuda.synchronize()
        assert torch.equal(self.buf, before) and all(np.array_equal(p, q) for p, q in zip(tables, self.h.snapshot()))


@pytest.mark.parametrize("T", [1, 3])
@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_outputs_stay_out_of_the_step(act, T):
    import workloads as W
    wl = W.TINY if act == "f32" else W.A3B_DECODE.with_(name="block", n_layers=1, n_experts=8, top_k=2, hidden=256, inter=128)
    s = Step(wl, T)
    a, H = s.at, s.H
    wrong = B if s.act is F else F
    eb = 4 if s.act is F else 2
    s.refused(xn=a["x"], x_fmt=wrong)                                   # fp32 over bf16 x writes past its end
    s.refused(xn=a["x"] + 4)
    s.refused(h=a["x"], h_fmt=wrong, xn=a["xn"])
    s.refused(h=a["x"] + 4 * (T * H * eb // 4 - 1))
    if T > 1:
        s.refused(xn=a["x"], ld_x=H + 8)                                # x has dense rows
    for name in ("idx", "w", "slot", "bias", "y"):
        s.refused(xn=a[name])
        s.refused(h=a[name])
        if name != "y":
            s.refused(xn=a[name] - 4 * (T * H * eb // 4) + 4)           # ends inside it
    s.refused(xn=s.h.arena.data_ptr())
    s.refused(h=s.h.arena.data_ptr())
    s.refused(xn=s.h.router.data_ptr())
    s.refused(w_post=a["y"])
    s.refused(w_pre=a["y"] + 4 * (T * H - 1))
    s.refused(gate=a["y"], kind=R().MOE_GATE_TOKEN)
    # the same step as documented: x_next in x's place, x_next elsewhere, h in x's place
    n = T * H
    x0 = s.buf[: 2 * n].clone()
    outs = []
    for xn in (a["xn"], a["x"]):
        s.buf[: 2 * n] = x0
        s.buf[2 * n: 4 * n] = 0.5
        s.run(xn=xn)
        torch.cuda.synchronize()
        i = (xn - s.base) // 4
        outs.append((s.buf[2 * n: 4 * n].clone(), s.buf[4 * n: 5 * n].clone(), s.buf[i: i + n].view(s.act)[:n].clone()))
    assert all(torch.equal(p, q) for p, q in zip(*outs)) and outs[0][2].float().abs().sum() > 0
    s.buf[: 2 * n] = x0
    s.buf[2 * n: 4 * n].view(s.act)[:n] = x0.view(s.act)[:n]
    s.run(h_fmt=s.act)
    torch.cuda.synchronize()
    apart = s.buf[2 * n: 4 * n].view(s.act)[:n].clone()
    s.run(h_fmt=s.act, h=a["x"])
    torch.cuda.synchronize()
    assert torch.equal(s.buf[: 2 * n].view(s.act)[:n], apart)
