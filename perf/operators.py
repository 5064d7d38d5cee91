"""Cases and plain forms of the dense feed-forward operators.

Three operators, forward and backward, that together make the dense (not
routed) feed-forward sub-layer beside the MoE layer -- a leading dense layer,
or the shared expert kept in bf16:

  layer_norm     y = (s - mean(s)) / sqrt(var(s) + eps) * gamma + beta over the
                 columns of s = x + residual; backward: dx (plus the gradient
                 that reaches s along the residual path), dgamma, dbeta
  gated_linear   a = act(x Wg^T) * (x Wu^T) with W13 = [Wg; Wu], keeping
                 h = x W13^T for the backward; backward: dx, dW13
  linear         y = act(x W^T + bias) + residual, keeping
                 z = x W^T + bias for the backward; backward: dx, dW, dbias

The plain forms below are float32 torch operations; `exact` evaluates the
definitions in float64.  `own` selects the library's kernels instead.
"""

import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
DTYPES = {"bf16": BF16, "f32": F32}
EPS = 1e-5


# ---------------------------------------------------------------------------
# Cases.  M: tokens; H, I: hidden and intermediate sizes (7168 and 2048 are the
# MoE layer's); N, K: output and input features of a linear layer; pad: extra
# elements between the rows of the activations (a slice of a wider buffer).
# ---------------------------------------------------------------------------

def listed():
    return [
        # the norm before the feed-forward layer, one sequence being decoded:
        # a single token, where the launch is what counts
        {"name": "norm_one_token", "op": "layer_norm", "M": 1, "H": 7168, "dtype": "bf16", "residual": True, "pad": 0},
        # the same norm over the largest batch of the framework's workloads
        {"name": "norm_32768", "op": "layer_norm", "M": 32768, "H": 7168, "dtype": "bf16", "residual": True, "pad": 0},
        # its backward on a training micro-batch, with the residual gradient
        {"name": "norm_bwd_4096", "op": "layer_norm_backward", "M": 4096, "H": 7168, "dtype": "bf16", "residual": True,
         "pad": 0},
        # float32 activations of an odd width, rows of a wider buffer
        {"name": "norm_bwd_ragged_f32", "op": "layer_norm_backward", "M": 1037, "H": 1001, "dtype": "f32",
         "residual": False, "pad": 3},
        # the down projection of one token being decoded: one read of the weight
        {"name": "linear_one_token", "op": "linear", "M": 1, "N": 7168, "K": 2048, "act": "none", "bias": False,
         "residual": True, "save": False, "out": "bf16", "pad": 0},
        # the down projection of a prefill batch, residual in the epilogue
        {"name": "linear_4096", "op": "linear", "M": 4096, "N": 7168, "K": 2048, "act": "none", "bias": True,
         "residual": True, "save": False, "out": "bf16", "pad": 0},
        # a small projection with sizes of no alignment, float32 result, the
        # pre-activation kept for training
        {"name": "linear_ragged_gelu", "op": "linear", "M": 777, "N": 1003, "K": 515, "act": "gelu", "bias": True,
         "residual": True, "save": True, "out": "f32", "pad": 0},
        # the down projection's gradients on a training micro-batch (float32
        # weight gradient, as an optimizer accumulates it)
        {"name": "linear_bwd_4096", "op": "linear_backward", "M": 4096, "N": 7168, "K": 2048, "act": "none",
         "bias": True, "dw": "f32", "pad": 0},
        # gate and up projections of a decode batch: bound by the weight
        {"name": "gated_decode_64", "op": "gated_linear", "M": 64, "H": 7168, "I": 2048, "act": "silu", "save": False,
         "pad": 0},
        # gate and up projections of the largest batch, in training
        {"name": "gated_32768", "op": "gated_linear", "M": 32768, "H": 7168, "I": 2048, "act": "silu", "save": True,
         "pad": 0},
        # their gradients on a training micro-batch
        {"name": "gated_bwd_4096", "op": "gated_linear_backward", "M": 4096, "H": 7168, "I": 2048, "act": "silu",
         "dw": "bf16", "pad": 0},
        # a small model's gradients on the ragged end of a data set
        {"name": "gated_bwd_ragged", "op": "gated_linear_backward", "M": 333, "H": 1000, "I": 343, "act": "gelu",
         "dw": "bf16", "pad": 5},
    ]


def _size(rng, lo, hi):
    """A size spread over the logarithm of [lo, hi]: a third as it falls, a
    third a multiple of 8, a third a multiple of 128 (of 8 below 128)."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    step = rng.choice((1, 8, 128))
    if step > 1:
        step = step if v >= step else 8 if v >= 8 else 1
        v = max(step, v // step * step)
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(("layer_norm", "layer_norm_backward", "linear", "linear_backward", "gated_linear",
                     "gated_linear_backward"))
    pad = rng.choice((0, 0, 0, 8, 3))
    while True:
        if op.startswith("layer_norm"):
            c = {"op": op, "M": _size(rng, 1, 32768), "H": _size(rng, 32, 8192), "dtype": rng.choice(("bf16", "f32")),
                 "residual": rng.random() < 0.5, "pad": pad}
        elif op.startswith("linear"):
            c = {"op": op, "M": _size(rng, 1, 32768), "N": _size(rng, 64, 8192), "K": _size(rng, 64, 8192),
                 "act": rng.choice(("none", "none", "silu", "gelu", "relu")), "bias": rng.random() < 0.5, "pad": pad}
            if op == "linear":
                c |= {"residual": rng.random() < 0.5, "save": c["act"] != "none" and rng.random() < 0.5,
                      "out": rng.choice(("bf16", "bf16", "f32"))}
            else:
                # a float32 weight gradient of exact products needs dz = dy
                c |= {"dw": rng.choice(("bf16", "f32")) if c["act"] == "none" else "bf16"}
        else:
            c = {"op": op, "M": _size(rng, 1, 32768), "H": _size(rng, 64, 8192), "I": _size(rng, 64, 4096),
                 "act": rng.choice(("silu", "silu", "gelu")), "pad": pad}
            c |= {"save": rng.random() < 0.5} if op == "gated_linear" else {"dw": "bf16"}
        w = work(c)
        if w["flops"] <= 1.2e12 and w["bytes"] <= 2.0e9:
            return c


def work(case):
    c, op, M = case, case["op"], case["M"]
    if op.startswith("layer_norm"):
        e, H = (2 if c["dtype"] == "bf16" else 4), c["H"]
        if op == "layer_norm":  # x, residual in; y, sum, mean, rstd out
            return {"bytes": M * H * e * (4 if c["residual"] else 2) + 2 * H * e + 8 * M, "flops": 8 * M * H}
        # dy, x, dsum in; dx, dgamma, dbeta out
        return {"bytes": M * H * e * (4 if c["residual"] else 3) + H * e + 8 * H + 8 * M, "flops": 14 * M * H}
    if op.startswith("linear"):
        N, K = c["N"], c["K"]
        if op == "linear":
            o = 4 if c["out"] == "f32" else 2
            return {"bytes": 2 * (M * K + N * K) + o * M * N * (1 + c["residual"] + c["save"]) + (2 * N if c["bias"] else 0),
                    "flops": 2 * M * N * K}
        z = 2 * M * N if c["act"] != "none" else 0
        return {"bytes": 2 * (M * N + 2 * M * K + N * K) + z + (4 if c["dw"] == "f32" else 2) * N * K + (4 * N if c["bias"] else 0),
                "flops": 4 * M * N * K}
    H, I = c["H"], c["I"]
    if op == "gated_linear":
        return {"bytes": 2 * (M * H + 2 * I * H + M * I * (3 if c["save"] else 1)), "flops": 4 * M * H * I}
    return {"bytes": 2 * (M * I + 2 * M * I + 2 * M * H + 2 * I * H) + 2 * 2 * I * H, "flops": 8 * M * H * I}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

class _Inputs:
    """Seeded tensors on the GPU."""

    def __init__(self, seed, pad):
        self.g = torch.Generator(device="cuda").manual_seed(int(seed))
        self.pad = pad

    def normal(self, rows, cols, std, dtype=BF16, pad=None):
        pad = self.pad if pad is None else pad
        t = torch.empty((rows, cols + pad), dtype=dtype, device="cuda")
        for r0 in range(0, rows, 8192):  # bounds the float32 temporaries
            r1 = min(rows, r0 + 8192)
            t[r0:r1] = torch.randn((r1 - r0, cols + pad), generator=self.g, device="cuda") * std
        return t[:, :cols]

    def vector(self, n, std, mean=0.0, dtype=BF16):
        return (torch.randn((n,), generator=self.g, device="cuda") * std + mean).to(dtype)


def prepare(case, seed):
    c, op, M = dict(case), case["op"], case["M"]
    r = _Inputs(seed, c["pad"])
    s = {"case": c}
    if op.startswith("layer_norm"):
        H, dt = c["H"], DTYPES[c["dtype"]]
        # hidden states: channels of uneven scale, a few large ones, a mean off 0
        x = r.normal(M, H, 1.0, dt)
        scale = torch.exp(r.vector(H, 0.5, dtype=F32))
        scale[:: max(1, H // 5)] *= 20.0
        x.mul_(scale.to(dt)).add_(0.1)
        s["gamma"], s["beta"] = r.vector(H, 0.1, 1.0, dt), r.vector(H, 0.1, 0.0, dt)
        if op == "layer_norm":
            s["x"], s["residual"] = x, (r.normal(M, H, 1.0, dt) if c["residual"] else None)
        else:
            s["x"] = x
            s["mean"] = torch.empty((M,), device="cuda")
            s["rstd"] = torch.empty((M,), device="cuda")
            for r0 in range(0, M, 4096):
                v = x[r0:r0 + 4096].float()
                s["mean"][r0:r0 + 4096] = v.mean(1)
                s["rstd"][r0:r0 + 4096] = 1.0 / torch.sqrt(v.var(1, correction=0) + EPS)
            s["dy"] = r.normal(M, H, 1e-3, dt)
            s["dsum"] = r.normal(M, H, 1e-3, dt) if c["residual"] else None
        return s
    if op.startswith("linear"):
        N, K = c["N"], c["K"]
        s["x"] = r.normal(M, K, 1.0)
        s["w"] = r.normal(N, K, 0.02, pad=0)
        s["bias"] = r.vector(N, 0.1) if c["bias"] else None
        if op == "linear":
            s["residual"] = r.normal(M, N, 1.0, DTYPES[c["out"]]) if c["residual"] else None
        else:
            s["dy"] = r.normal(M, N, 1e-2)
            s["z"] = r.normal(M, N, 0.02 * math.sqrt(K)) if c["act"] != "none" else None
        return s
    H, I = c["H"], c["I"]
    s["x"] = r.normal(M, H, 1.0)
    s["w13"] = r.normal(2 * I, H, 0.02, pad=0)
    if op == "gated_linear_backward":
        s["h"] = r.normal(M, 2 * I, 0.02 * math.sqrt(H))
        s["da"] = r.normal(M, I, 1e-2)
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _act(z, act):
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "relu":
        return z * (z > 0)
    return z


def _act_grad(z, act):
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    if act == "relu":
        return (z > 0).to(z.dtype)
    return torch.ones_like(z)


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "layer_norm":
        dt = DTYPES[c["dtype"]]
        v = s["x"].float()
        if s["residual"] is not None:
            v = v + s["residual"].float()
        mean = v.mean(1)
        d = v - mean[:, None]
        rstd = 1.0 / torch.sqrt((d * d).mean(1) + EPS)
        y = d * rstd[:, None] * s["gamma"].float() + s["beta"].float()
        out = {"y": y.to(dt), "mean": mean, "rstd": rstd}
        if s["residual"] is not None:
            out["sum"] = v.to(dt)
        return out
    if op == "layer_norm_backward":
        dt = DTYPES[c["dtype"]]
        dy = s["dy"].float()
        xhat = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
        g = dy * s["gamma"].float()
        dx = s["rstd"][:, None] * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
        if s["dsum"] is not None:
            dx = dx + s["dsum"].float()
        return {"dx": dx.to(dt), "dgamma": (dy * xhat).sum(0), "dbeta": dy.sum(0)}
    if op == "linear":
        dt = DTYPES[c["out"]]
        z = s["x"].float() @ s["w"].float().t()
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = _act(z, c["act"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return {"y": y.to(dt), "z": z.to(dt)} if c["save"] else {"y": y.to(dt)}
    if op == "linear_backward":
        dz = s["dy"].float()
        if c["act"] != "none":
            dz = dz * _act_grad(s["z"].float(), c["act"])
        out = {"dx": (dz @ s["w"].float()).to(BF16), "dw": (dz.t() @ s["x"].float()).to(DTYPES[c["dw"]])}
        if c["bias"]:
            out["dbias"] = dz.sum(0)
        return out
    I = c["I"]
    if op == "gated_linear":
        h = s["x"].float() @ s["w13"].float().t()
        a = (_act(h[:, :I], c["act"]) * h[:, I:]).to(BF16)
        return {"a": a, "h": h.to(BF16)} if c["save"] else {"a": a}
    g, u, da = s["h"][:, :I].float(), s["h"][:, I:].float(), s["da"].float()
    dh = torch.cat([da * u * _act_grad(g, c["act"]), da * _act(g, c["act"])], 1)
    return {"dx": (dh @ s["w13"].float()).to(BF16), "dw13": (dh.t() @ s["x"].float()).to(DTYPES[c["dw"]])}


def run(state):
    if not own:
        return _plain(state)
    import fp8_block_scaled_dsmoe_amd as d
    s, c = state, state["case"]
    op = c["op"]
    if op == "layer_norm":
        y, mean, rstd, total = d.layer_norm(s["x"], s["gamma"], s["beta"], eps=EPS, residual=s["residual"])
        out = {"y": y, "mean": mean, "rstd": rstd}
        if total is not None:
            out["sum"] = total
        return out
    if op == "layer_norm_backward":
        dx, dgamma, dbeta = d.layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["gamma"], dsum=s["dsum"])
        return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
    if op == "linear":
        y, z = d.linear(s["x"], s["w"], s["bias"], act=c["act"], residual=s["residual"], out_dtype=DTYPES[c["out"]],
                        save_z=c["save"])
        return {"y": y, "z": z} if c["save"] else {"y": y}
    if op == "linear_backward":
        dx, dw, dbias = d.linear_backward(s["dy"], s["x"], s["w"], z=s["z"], act=c["act"], dw_dtype=DTYPES[c["dw"]],
                                          need_dbias=c["bias"])
        return {"dx": dx, "dw": dw, "dbias": dbias} if c["bias"] else {"dx": dx, "dw": dw}
    if op == "gated_linear":
        a, h = d.gated_linear(s["x"], s["w13"], act=c["act"], save_h=c["save"])
        return {"a": a, "h": h} if c["save"] else {"a": a}
    dx, dw13 = d.gated_linear_backward(s["da"], s["x"], s["w13"], s["h"], act=c["act"], dw_dtype=DTYPES[c["dw"]])
    return {"dx": dx, "dw13": dw13}


# ---------------------------------------------------------------------------
# The definitions in float64, row by row or by blocks of columns
# ---------------------------------------------------------------------------

def _phi(t):
    return 0.5 * torch.special.erfc(-t / math.sqrt(2.0))


def _f64(act, t):
    """(act(t), act'(t)) in float64."""
    if act == "none":
        return t, torch.ones_like(t)
    if act == "relu":
        return torch.clamp(t, min=0.0), torch.where(t > 0, 1.0, 0.0).double()
    if act == "silu":
        p = torch.sigmoid(t)
        return t * p, p + t * p * torch.sigmoid(-t)
    return t * _phi(t), _phi(t) + t * torch.exp(-t * t / 2.0) / math.sqrt(2.0 * math.pi)


def exact(case, seed):
    s, c, op = prepare(case, seed), case, case["op"]
    v = {k: t.double() for k, t in s.items() if isinstance(t, torch.Tensor)}
    if op == "layer_norm":
        total = v["x"] if v.get("residual") is None else v["x"] + v["residual"]
        mu = total.sum(1) / c["H"]
        var = ((total * total).sum(1) - c["H"] * mu * mu) / c["H"]
        inv = (var + EPS).rsqrt()
        a = inv[:, None] * v["gamma"][None]
        out = {"y": total * a + (v["beta"][None] - mu[:, None] * a), "mean": mu, "rstd": inv}
        if c["residual"]:
            out["sum"] = total
        return out
    if op == "layer_norm_backward":
        H, inv = c["H"], v["rstd"][:, None]
        n = v["x"] * inv - v["mean"][:, None] * inv
        dn = v["gamma"][None] * v["dy"]
        dx = inv / H * (H * dn - dn.sum(1, keepdim=True) - n * (dn * n).sum(1, keepdim=True))
        ones = torch.ones((1, c["M"]), dtype=torch.float64, device="cuda")
        return {"dx": dx + v["dsum"] if c["residual"] else dx, "dgamma": torch.einsum("mh,mh->h", v["dy"], n),
                "dbeta": (ones @ v["dy"])[0]}
    if op == "linear":
        z = torch.addmm(v["bias"], v["x"], v["w"].t()) if c["bias"] else torch.mm(v["x"], v["w"].t())
        y = _f64(c["act"], z)[0]
        y = y + v["residual"] if c["residual"] else y
        return {"y": y, "z": z} if c["save"] else {"y": y}
    if op == "linear_backward":
        dz = v["dy"] if c["act"] == "none" else v["dy"] * _f64(c["act"], v["z"])[1]
        out = {"dx": torch.mm(dz, v["w"]), "dw": torch.mm(v["x"].t(), dz).t().contiguous()}
        if c["bias"]:
            out["dbias"] = torch.mv(dz.t(), torch.ones(c["M"], dtype=torch.float64, device="cuda"))
        return out
    I = c["I"]
    if op == "gated_linear":
        g, u = torch.mm(v["x"], v["w13"][:I].t()), torch.mm(v["x"], v["w13"][I:].t())
        a = _f64(c["act"], g)[0] * u
        return {"a": a, "h": torch.cat((g, u), 1)} if c["save"] else {"a": a}
    f, df = _f64(c["act"], v["h"][:, :I])
    dg, du = v["da"] * v["h"][:, I:] * df, v["da"] * f
    return {"dx": torch.mm(dg, v["w13"][:I]) + torch.mm(du, v["w13"][I:]),
            "dw13": torch.cat((torch.mm(dg.t(), v["x"]), torch.mm(du.t(), v["x"])), 0)}
