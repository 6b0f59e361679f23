"""The experts' products and their gradients, as measured cases.

A case names one pass: the gated half of a feed-forward block (``glu``: both projections, the activation
and their product), a projection with bias, activation and residual (``linear``), and the gradients of
both, over rows sorted by expert (``E`` of them, ``offsets`` as a dispatch leaves them) or, with E = 0, over
all rows with one weight.

``run`` computes a pass with the library's entry points where ``own`` is true, and in its plain form
(elementary torch operations in fp32, rounded once at the end) where it is false.  ``exact`` gives the
same outputs in 64 bits.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
NBYTES = {"f32": 4, "bf16": 2}


# ---------------------------------------------------------------------------
# cases
#   glu, glu_backward:        x [R,H], w [E,2I,H] (gate rows, then up rows), a [R,I], gu [R,2I]
#   linear, linear_backward:  x [R,H], w [E,I,H], y [R,I]

def listed():
    return [
        # the gated half
        # one token through a shared expert of the A3B shape: launch and one round trip of memory
        {"name": "glu token", "op": "glu", "R": 1, "E": 0, "H": 2048, "I": 512, "fmt": "bf16", "act": "silu",
         "save": False, "drop": 0.0},
        # a decode step of four tokens over the A3B experts: thirty experts' weights, about one row each
        {"name": "glu decode experts", "op": "glu", "R": 32, "E": 256, "H": 2048, "I": 512, "fmt": "bf16",
         "act": "silu", "save": False, "drop": 0.0},
        # the A3B prompt: 4096 tokens of eight experts, 1.07 GB of weights read once
        {"name": "glu prompt experts", "op": "glu", "R": 32768, "E": 256, "H": 2048, "I": 512, "fmt": "bf16",
         "act": "silu", "save": False, "drop": 0.0},
        # training a shared expert of the DSV4 shape: both projections kept for the gradient
        {"name": "glu training shared", "op": "glu", "R": 4096, "E": 0, "H": 4096, "I": 2048, "fmt": "bf16",
         "act": "silu", "save": True, "drop": 0.0},
        # its gradient over a share of the A3B experts (one of eight GPUs), one pair in twenty dropped
        {"name": "glu_backward experts", "op": "glu_backward", "R": 16384, "E": 32, "H": 2048, "I": 512, "fmt": "bf16",
         "act": "silu", "drop": 0.05},
        # and of a shared expert of the DSV4 shape, a ragged batch
        {"name": "glu_backward shared R3001", "op": "glu_backward", "R": 3001, "E": 0, "H": 4096, "I": 2048,
         "fmt": "bf16", "act": "silu", "drop": 0.0},
        # a small model in fp32 with sizes that nothing divides
        {"name": "glu_backward odd f32", "op": "glu_backward", "R": 333, "E": 7, "H": 999, "I": 257, "fmt": "f32",
         "act": "gelu", "drop": 0.1},
        # the projection
        # one token's way back from the shared expert, added to the routed experts' sum in fp32
        {"name": "linear token residual", "op": "linear", "R": 1, "E": 0, "H": 512, "I": 2048, "fmt": "bf16",
         "y": "f32", "act": "none", "bias": False, "residual": True, "save": False, "drop": 0.0},
        # the A3B prompt's down projections
        {"name": "linear prompt experts", "op": "linear", "R": 32768, "E": 256, "H": 512, "I": 2048, "fmt": "bf16",
         "y": "bf16", "act": "none", "bias": False, "residual": False, "save": False, "drop": 0.0},
        # an adapter in fp32 with everything in its epilogue, a ragged batch
        {"name": "linear gelu residual f32", "op": "linear", "R": 1531, "E": 0, "H": 2048, "I": 1024, "fmt": "f32",
         "y": "f32", "act": "gelu", "bias": True, "residual": True, "save": True, "drop": 0.0},
        # training the down projections of a share of the DSV4 experts: 1024 tokens of six
        {"name": "linear_backward experts", "op": "linear_backward", "R": 6144, "E": 32, "H": 2048, "I": 4096,
         "fmt": "bf16", "y": "bf16", "act": "none", "bias": False, "drop": 0.02},
        # a projection with bias and activation whose rows start anywhere
        {"name": "linear_backward gelu odd", "op": "linear_backward", "R": 777, "E": 0, "H": 1000, "I": 1001,
         "fmt": "bf16", "y": "bf16", "act": "gelu", "bias": True, "drop": 0.0},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A size of the model: usually a multiple of 64, sometimes of 8, sometimes any."""
    n = _log_int(rng, lo, hi)
    step = rng.choice((64, 64, 8, 1))
    return max(lo, n // step * step)


def draw(rng):
    op = rng.choice(("glu", "glu_backward", "linear", "linear_backward"))
    fmt = rng.choice(("bf16", "bf16", "f32"))
    E = rng.choice((0, 1)) and _log_int(rng, 2, 256)
    H, I = _width(rng, 64, 4096), _width(rng, 64, 4096)
    N = 2 * I if op.startswith("glu") else I
    # no more weights than 256 experts of the A3B shape, a quarter of that with a gradient; no more products
    # than the A3B prompt, half of that with a gradient; fp32 half as much
    less = (2 if op.endswith("backward") else 1) * (2 if fmt == "f32" else 1)
    E = min(E, 256 * 1024 * 2048 // (less * less * N * H)) if E else 0
    E = 0 if E < 2 else E
    most = max(1, min(32768, 32768 * 1024 * 2048 // (less * N * H), 32768 * 4096 // (N + H)))
    c = {"op": op, "R": _log_int(rng, 1, most), "E": E, "H": H, "I": I, "fmt": fmt,
         "drop": rng.choice((0.0, 0.05, 0.3)) if E else 0.0}
    if op.startswith("glu"):
        c["act"] = rng.choice(("silu", "silu", "gelu"))
    else:
        c.update(act=rng.choice(("none", "none", "silu", "gelu")), bias=rng.random() < 0.5,
                 y=rng.choice((fmt, "f32")) if op == "linear" else fmt)
        if op == "linear":
            c["residual"] = rng.random() < 0.5
    if not op.endswith("backward"):
        c["save"] = rng.random() < 0.5
    return c


# ---------------------------------------------------------------------------
# inputs

def prepare(case, seed):
    c = case
    op, R, E, H, I = c["op"], c["R"], c["E"], c["H"], c["I"]
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, glu, back = DT[c["fmt"]], op.startswith("glu"), op.endswith("backward")
    rnd = lambda dtype, *shape: torch.randn(*shape, device="cuda", generator=g).to(dtype)  # noqa: E731
    new = lambda dtype, *shape: torch.zeros(*shape, device="cuda", dtype=dtype)  # noqa: E731
    N = 2 * I if glu else I
    s = dict(c)
    s["offsets"], s["cap"] = None, R
    if E:
        # rows of uneven experts, the dropped ones behind the last
        kept = max(1, int(round(R * (1.0 - c["drop"]))))
        p = torch.exp(0.5 * torch.randn(E, device="cuda", generator=g))
        counts = torch.bincount(torch.multinomial(p, kept, replacement=True, generator=g), minlength=E)
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["cap"] = int(counts.max())
    # rows as a norm leaves them, weights that keep a projection's outputs about 1
    s["in_x"] = rnd(dt, R, H)
    w = torch.empty(*((E, N, H) if E else (N, H)), device="cuda", dtype=dt)
    s["w"] = w.normal_(0.0, 1.0 / math.sqrt(H), generator=g)
    if glu:
        if back:
            s["in_gu"], s["in_da"] = rnd(dt, R, 2 * I), rnd(dt, R, I)
            s["out"] = {"dx": new(dt, R, H), "dw": torch.zeros_like(w)}
        else:
            s["out"] = {"a": new(dt, R, I)}
            if c["save"]:
                s["out"]["gu"] = new(dt, R, 2 * I)
        return s
    yt = DT[c["y"]]
    shape = (E, I) if E else (I,)
    s["bias"] = 0.1 * rnd(torch.float32, *shape) if c["bias"] else None
    if back:
        s["in_dy"], s["in_z"] = rnd(yt, R, I), rnd(dt, R, I) if c["act"] != "none" else None
        s["out"] = {"dx": new(dt, R, H), "dw": torch.zeros_like(w)}
        if c["bias"]:
            s["out"]["dbias"] = new(torch.float32, *shape)
    else:
        s["in_residual"] = rnd(yt, R, I) if c["residual"] else None
        s["out"] = {"y": new(yt, R, I)}
        if c["save"]:
            s["out"]["z"] = new(dt, R, I)
    return s


# ---------------------------------------------------------------------------
# one pass

def run(state):
    return (_own if own else _plain)[state["op"]](state)


def _experts(s):
    """The expert of each row (E behind the last) and the row's place among its expert's rows."""
    pos = torch.arange(s["R"], device="cuda")
    off = s["offsets"].long()
    e = torch.searchsorted(off[1:], pos, right=True)
    return e, pos - off[e.clamp_max(s["E"] - 1)]


def _pad(v, s, at):
    """Rows [R,n] in fp32 as [E,cap,n], zeros where an expert has fewer; rows without an expert are left out."""
    e, i = at
    n = s["E"] * s["cap"]
    out = torch.zeros(n + 1, v.shape[1], device=v.device)
    out[torch.where(e < s["E"], e * s["cap"] + i, n)] = v.float()
    return out[:n].view(s["E"], s["cap"], -1)


def _unpad(p, s, at):
    e, i = at
    rows = p.flatten(0, 1)[torch.where(e < s["E"], e * s["cap"] + i, 0)]
    return torch.where((e < s["E"])[:, None], rows, 0.0)


def _times(v, w, s):
    """v [R,n] times its expert's w^T, w [E,m,n] or [m,n], in fp32; zeros for rows without an expert."""
    if not s["E"]:
        return v.float() @ w.float().T
    at = _experts(s)
    if s["R"] <= s["E"]:  # fewer rows than experts: each row's own weights
        e = at[0]
        rows = (w[e.clamp_max(s["E"] - 1)].float() @ v.float()[:, :, None])[:, :, 0]
        return torch.where((e < s["E"])[:, None], rows, 0.0)
    wt = w.transpose(1, 2).to(torch.float32, memory_format=torch.contiguous_format)
    return _unpad(torch.bmm(_pad(v, s, at), wt), s, at)


def _outer(d, v, s):
    """The weights' gradient [E,m,n] of d [R,m] and v [R,n]."""
    if not s["E"]:
        return d.float().T @ v.float()
    at = _experts(s)
    return torch.bmm(_pad(d, s, at).transpose(1, 2).contiguous(), _pad(v, s, at))


def _act(z, kind):
    if kind == "none":
        return z
    if kind == "silu":
        return z / (1.0 + torch.exp(-z))
    return 0.5 * z * (1.0 + torch.tanh(0.7978845608028654 * (z + 0.044715 * z * z * z)))


def _act_grad(z, kind):
    if kind == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    t = torch.tanh(0.7978845608028654 * (z + 0.044715 * z * z * z))
    return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * 0.7978845608028654 * (1.0 + 0.134145 * z * z)


def _plain_glu(s):
    gu = _times(s["in_x"], s["w"], s)
    g, u = gu.chunk(2, dim=1)
    out = {"a": (_act(g, s["act"]) * u).to(DT[s["fmt"]])}
    if s["save"]:
        out["gu"] = gu.to(DT[s["fmt"]])
    return out


def _gradients(d, s):
    back = s["w"].transpose(-1, -2)
    return {"dx": _times(d, back, s).to(DT[s["fmt"]]), "dw": _outer(d, s["in_x"], s).to(DT[s["fmt"]])}


def _plain_glu_backward(s):
    g, u = s["in_gu"].float().chunk(2, dim=1)
    da = s["in_da"].float()
    return _gradients(torch.cat([da * u * _act_grad(g, s["act"]), da * _act(g, s["act"])], dim=1), s)


def _kept(s):
    """[R,1]: the row has an expert."""
    if not s["E"]:
        return torch.ones(s["R"], 1, device="cuda", dtype=torch.bool)
    return (_experts(s)[0] < s["E"])[:, None]


def _plain_linear(s):
    z = _times(s["in_x"], s["w"], s)
    if s["bias"] is not None:
        z = z + (s["bias"][_experts(s)[0].clamp_max(s["E"] - 1)] if s["E"] else s["bias"])
    y = _act(z, s["act"])
    if s["in_residual"] is not None:
        y = y + s["in_residual"].float()
    kept = _kept(s)
    out = {"y": torch.where(kept, y, 0.0).to(DT[s["y"]])}
    if s["save"]:
        out["z"] = torch.where(kept, z, 0.0).to(DT[s["fmt"]])
    return out


def _plain_linear_backward(s):
    d = s["in_dy"].float()
    if s["act"] != "none":
        d = d * _act_grad(s["in_z"].float(), s["act"])
    out = _gradients(d, s)
    if s["bias"] is not None:
        out["dbias"] = _pad(d, s, _experts(s)).sum(1) if s["E"] else d.sum(0)
    return out


_plain = {"glu": _plain_glu, "glu_backward": _plain_glu_backward, "linear": _plain_linear,
          "linear_backward": _plain_linear_backward}


def _lib():
    import routed_expert_ffn_02_amd as R
    return R


def _act_kind(R, s):
    return {"none": R.MOE_ACT_NONE, "silu": R.MOE_ACT_SILU, "gelu": R.MOE_ACT_GELU}[s["act"]]


def _workspace(s, size):
    """The pass's workspace, made by the first pass on a state and kept with it, as a program keeps its own."""
    if "ws" not in s:
        s["ws"] = torch.empty(size(), dtype=torch.uint8, device="cuda")
    return s["ws"]


def _own_glu(s):
    R, o = _lib(), s["out"]
    R.moe_glu(s["in_x"], s["w"], o["a"], o.get("gu"), s["offsets"], act=_act_kind(R, s))
    return o


def _own_glu_backward(s):
    R, o = _lib(), s["out"]
    ws = _workspace(s, lambda: R.moe_glu_workspace(s["R"], s["E"] or 1, s["H"], s["I"], _fmt(R, s["fmt"])))
    R.moe_glu_backward(s["in_da"], s["in_gu"], s["in_x"], s["w"], o["dx"], o["dw"], ws, s["offsets"],
                       act=_act_kind(R, s))
    return o


def _own_linear(s):
    R, o = _lib(), s["out"]
    R.moe_linear(s["in_x"], s["w"], o["y"], s["bias"], s["in_residual"], o.get("z"), s["offsets"],
                 act=_act_kind(R, s))
    return o


def _own_linear_backward(s):
    R, o = _lib(), s["out"]
    ws = _workspace(s, lambda: R.moe_linear_workspace(s["R"], s["E"] or 1, s["H"], s["I"], _fmt(R, s["fmt"])))
    R.moe_linear_backward(s["in_dy"], s["in_z"], s["in_x"], s["w"], o["dx"], o["dw"], o.get("dbias"), ws, s["offsets"],
                          act=_act_kind(R, s))
    return o


def _fmt(R, name):
    return R.MOE_AFMT_BF16 if name == "bf16" else R.MOE_AFMT_F32


_own = {"glu": _own_glu, "glu_backward": _own_glu_backward, "linear": _own_linear,
        "linear_backward": _own_linear_backward}


# ---------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    """Inputs read once, outputs written once; dropped rows are neither, and an expert without a row is not read."""
    c = case
    R, E, H, I, b = c["R"] * (1.0 - c["drop"]), c["E"], c["H"], c["I"], NBYTES[c["fmt"]]
    glu, back = c["op"].startswith("glu"), c["op"].endswith("backward")
    N = 2 * I if glu else I
    weights = b * N * H * (E * (1.0 - (1.0 - 1.0 / E) ** R) if E else 1)
    index, product = 4 * (E + 1), 2 * R * N * H
    if back:
        rows = (2 * H + 3 * I) * b if glu else 2 * H * b + I * (NBYTES[c["y"]] + (b if c["act"] != "none" else 0))
        bias = 0 if glu or not c["bias"] else 4 * I * max(E, 1)
        return {"bytes": int(R * rows + weights + b * N * H * max(E, 1) + bias + index), "flops": int(2 * product)}
    if glu:
        rows = (H + I + (2 * I if c["save"] else 0)) * b
        return {"bytes": int(R * rows + weights + index), "flops": int(product)}
    rows = H * b + I * (NBYTES[c["y"]] * (2 if c["residual"] else 1) + (b if c["save"] else 0))
    return {"bytes": int(R * rows + weights + (4 * I * max(E, 1) if c["bias"] else 0) + index), "flops": int(product)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits, expert by expert

def _sigmoid64(z):
    return 0.5 + 0.5 * torch.tanh(0.5 * z)


def _act64(z, kind):
    """(the activation, its derivative): silu is z s(z); gelu in its tanh form is z s(2 p(z)) with the cubic p,
    since (1 + tanh p) / 2 = s(2 p)."""
    if kind == "none":
        return z, torch.ones_like(z)
    c = math.sqrt(2.0 / math.pi)
    q, dq = (z, torch.ones_like(z)) if kind == "silu" else (2 * c * (z + 0.044715 * z ** 3), 2 * c * (1 + 3 * 0.044715 * z ** 2))
    sg = _sigmoid64(q)
    return z * sg, sg + z * sg * _sigmoid64(-q) * dq


def exact(case, seed):
    s = prepare(case, seed)
    op, E, R, I = case["op"], case["E"], case["R"], case["I"]
    bounds = s["offsets"].tolist() if E else [0, R]
    out = {k: torch.zeros(v.shape, dtype=torch.float64, device="cuda") for k, v in s["out"].items()}
    for e in range(max(E, 1)):
        lo, hi = bounds[e], bounds[e + 1]
        if lo == hi:
            continue
        part = {k: (v[e] if k in ("dw", "dbias") and E else v if k in ("dw", "dbias") else v[lo:hi]) for k, v in out.items()}
        x = s["in_x"][lo:hi].double()
        w = (s["w"][e] if E else s["w"]).double()
        if op in ("glu", "linear"):
            z = x @ w.T
            if op == "glu":
                if "gu" in part:
                    part["gu"].copy_(z)
                part["a"].copy_(_act64(z[:, :I], case["act"])[0] * z[:, I:])
                continue
            if s["bias"] is not None:
                z = z + (s["bias"][e] if E else s["bias"]).double()
            if "z" in part:
                part["z"].copy_(z)
            y = _act64(z, case["act"])[0]
            part["y"].copy_(y if s["in_residual"] is None else y + s["in_residual"][lo:hi].double())
            continue
        if op == "glu_backward":
            gu, da = s["in_gu"][lo:hi].double(), s["in_da"][lo:hi].double()
            v, dv = _act64(gu[:, :I], case["act"])
            d = torch.cat([da * gu[:, I:] * dv, da * v], dim=1)
        else:
            d = s["in_dy"][lo:hi].double()
            if case["act"] != "none":
                d = d * _act64(s["in_z"][lo:hi].double(), case["act"])[1]
            if "dbias" in part:
                part["dbias"].copy_(d.sum(0))
        part["dx"].copy_(d @ w)
        part["dw"].copy_(d.T @ x)
    return out
