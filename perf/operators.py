"""The dense-layer operators, as cases that can be timed and checked.

The operators are those of a per-Gaussian attribute head (a residual MLP whose last layer adds
to the Gaussians' records before they are projected) and of the image-token block that conditions
it: the linear layer ``y = act(x W^T + b) + r`` and layer normalisation, each forward and backward.

``run`` computes a case in plain torch operations in 32 bits when ``own`` is false and through
``gaussian_splatting_gb300.dense`` when it is true; ``exact`` gives the definition in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

EPS = 1e-5
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
ACTS = ("none", "relu", "gelu", "silu")


# ------------------------------------------------------------------ cases
def _linear(name, op, rows, n_in, n_out, dtype, act, bias, residual, train=True):
    return {"name": name, "op": op, "rows": rows, "in": n_in, "out": n_out, "dtype": dtype, "act": act, "bias": bias,
            "residual": residual, "train": train}


def _norm(name, op, rows, width, dtype, skip=False):
    return {"name": name, "op": op, "rows": rows, "width": width, "dtype": dtype, "skip": skip}


def listed():
    return [
        # one embedding per view of a batch of 16 (the 4K workload's batch): latency alone counts
        _linear("views-16 embed f32", "linear_fwd", 16, 32, 128, "f32", "gelu", True, False),
        # a hidden layer of the head over the 300K-Gaussian object scene, training (z is kept)
        _linear("object-300k hidden bf16", "linear_fwd", 300_000, 256, 256, "bf16", "gelu", True, True),
        # its last layer: 59 outputs (the Gaussian record) added to the stored record, f32, rendering only
        _linear("object-300k record f32", "linear_fwd", 300_000, 128, 59, "f32", "none", True, True, False),
        # the wide half of a token block: one token per 8x8 block of a 1236x820 view
        _linear("tokens-15965 wide bf16", "linear_fwd", 15_965, 1024, 4096, "bf16", "gelu", True, False),
        # backward of a small scene's hidden layer (2,048 Gaussians)
        _linear("tiny-2k hidden f32 bwd", "linear_bwd", 2_048, 64, 64, "f32", "relu", True, False),
        # backward of the same hidden, record and wide layers
        _linear("object-300k hidden bf16 bwd", "linear_bwd", 300_000, 256, 256, "bf16", "gelu", True, True),
        _linear("object-300k record f32 bwd", "linear_bwd", 300_000, 128, 59, "f32", "none", True, True),
        _linear("tokens-15965 wide bf16 bwd", "linear_bwd", 15_965, 1024, 4096, "bf16", "gelu", True, False),
        # the head's normalisation over a small scene (latency) and over the 3M-Gaussian scene (bandwidth)
        _norm("tiny-2k norm f32", "layernorm_fwd", 2_048, 64, "f32"),
        _norm("unbounded-3m norm bf16", "layernorm_fwd", 3_000_000, 128, "bf16"),
        # backward of the token block's normalisation, with the gradient of the residual path added
        _norm("tokens-15965 norm bf16 bwd", "layernorm_bwd", 15_965, 1024, "bf16", True),
        # backward over the 3M-Gaussian scene in f32
        _norm("unbounded-3m norm f32 bwd", "layernorm_bwd", 3_000_000, 128, "f32", True),
    ]


_MOST_FLOPS = 2.5e11   # of the largest listed product
_MOST_BYTES = 6.0e9    # of the largest listed pass over memory


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """A case of the listed ones' ranges: 1 to 3M rows, 1 to 4096 features, both types, every activation."""
    while True:
        op = rng.choice(["linear_fwd", "linear_fwd", "linear_bwd", "linear_bwd", "layernorm_fwd", "layernorm_bwd"])
        dtype = rng.choice(["f32", "bf16"])
        rows = _log_int(rng, 1, 3_000_000)
        if op.startswith("linear"):
            # most programs keep their widths at multiples of 8; one in three is any number
            n_in, n_out = _log_int(rng, 8, 4096), _log_int(rng, 1, 4096)
            if rng.random() < 0.67:
                n_in, n_out = max(8, n_in // 8 * 8), max(8, n_out // 8 * 8)
            c = _linear("", op, rows, n_in, n_out, dtype, rng.choice(ACTS), rng.random() < 0.8, rng.random() < 0.5,
                        op == "linear_bwd" or rng.random() < 0.5)
        else:
            c = _norm("", op, rows, _log_int(rng, 8, 4096), dtype, op == "layernorm_bwd" and rng.random() < 0.5)
        del c["name"]
        w = work(c)
        # products in f32 cost several in bf16
        flops = w["flops"] * (8 if dtype == "f32" else 1)
        if flops <= _MOST_FLOPS and w["bytes"] <= _MOST_BYTES and 3072 not in c.values():
            return c


# ------------------------------------------------------------------ inputs
def _gradient(shape, g):
    """A loss gradient per Gaussian: its length spans decades, and it is zero where no view saw the Gaussian."""
    rows = shape[0]
    scale = torch.pow(10.0, torch.rand((rows, 1), generator=g, device="cuda") * 2.0 - 6.0)
    scale *= (torch.rand((rows, 1), generator=g, device="cuda") < 0.7)
    if rows <= 16:
        scale = torch.full_like(scale, 1e-5)
    return torch.randn(shape, generator=g, device="cuda") * scale


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device="cuda").mul_(std)

    rows = case["rows"]
    s = {"case": dict(case)}
    if case["op"].startswith("linear"):
        n_in, n_out = case["in"], case["out"]
        s["x"] = normal(rows, n_in).to(t)  # normalised features
        s["w"] = normal(n_out, n_in, std=1.0 / math.sqrt(n_in)).to(t)
        s["b"] = normal(n_out, std=0.1).to(t) if case["bias"] else None
        if case["op"] == "linear_fwd":
            s["r"] = normal(rows, n_out).to(t) if case["residual"] else None
        else:
            s["dy"] = _gradient((rows, n_out), g).to(t)
            s["z"] = None
            if case["act"] != "none":  # what the forward pass kept
                z = s["x"].float() @ s["w"].float().t()
                s["z"] = (z if s["b"] is None else z.add_(s["b"].float())).to(t)
                del z
    else:
        n = case["width"]
        x = normal(rows, n) * (0.5 + torch.rand((1, n), generator=g, device="cuda")) + normal(1, n, std=0.5)
        s["x"] = x.to(t)
        s["gamma"] = (1.0 + normal(n, std=0.1)).to(t)
        s["beta"] = normal(n, std=0.1).to(t)
        if case["op"] == "layernorm_bwd":
            s["dy"] = _gradient((rows, n), g).to(t)
            s["skip"] = _gradient((rows, n), g).to(t) if case["skip"] else None
            xf = s["x"].float()
            s["mean"] = xf.mean(1)
            xf.sub_(s["mean"][:, None])
            s["rstd"] = torch.rsqrt(xf.square_().mean(1) + EPS)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    from gaussian_splatting_gb300 import dense
    c = s["case"]
    op = c["op"]
    if op == "linear_fwd":
        y, z = dense.linear_fwd(s["x"], s["w"], s["b"], s["r"], act=c["act"], keep_z=c["train"])
        return {"y": y, "z": z}
    if op == "linear_bwd":
        dx, dw, db = dense.linear_bwd(s["dy"], s["x"], s["w"], z=s["z"], act=c["act"], bias=c["bias"])
        return {"dx": dx, "dw": dw, "db": db}
    if op == "layernorm_fwd":
        y, mean, rstd = dense.layernorm_fwd(s["x"], s["gamma"], s["beta"], eps=EPS)
        return {"y": y, "mean": mean, "rstd": rstd}
    dx, dgamma, dbeta = dense.layernorm_bwd(s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"], skip=s["skip"])
    return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}


def _act(z, act):
    if act == "relu":
        return z * (z > 0)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "silu":
        return z * (1.0 / (1.0 + torch.exp(-z)))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    sig = 1.0 / (1.0 + torch.exp(-z))
    return sig * (1.0 + z * (1.0 - sig))


def _run_plain(s):
    c = s["case"]
    op, t = c["op"], s["x"].dtype
    x = s["x"].float()
    if op == "linear_fwd":
        z = x @ s["w"].float().t()
        if s["b"] is not None:
            z = z + s["b"].float()
        y = _act(z, c["act"])
        if s["r"] is not None:
            y = y + s["r"].float()
        return {"y": y.to(t), "z": z.to(t) if c["train"] else None}
    if op == "linear_bwd":
        dz = s["dy"].float()
        if s["z"] is not None:
            dz = dz * _act_slope(s["z"].float(), c["act"])
        return {"dx": (dz @ s["w"].float()).to(t), "dw": (dz.t() @ x).to(t), "db": dz.sum(0).to(t) if c["bias"] else None}
    gamma = s["gamma"].float()
    if op == "layernorm_fwd":
        mean = x.mean(1, keepdim=True)
        d = x - mean
        rstd = 1.0 / torch.sqrt((d * d).mean(1, keepdim=True) + EPS)
        return {"y": (d * rstd * gamma + s["beta"].float()).to(t), "mean": mean[:, 0], "rstd": rstd[:, 0]}
    dy = s["dy"].float()
    xhat = (x - s["mean"][:, None]) * s["rstd"][:, None]
    gy = dy * gamma
    dx = (gy - gy.mean(1, keepdim=True) - xhat * (gy * xhat).mean(1, keepdim=True)) * s["rstd"][:, None]
    if s["skip"] is not None:
        dx = dx + s["skip"].float()
    return {"dx": dx.to(t), "dgamma": (dy * xhat).sum(0).to(t), "dbeta": dy.sum(0).to(t)}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    x, act = d["x"], case.get("act")
    if case["op"] == "linear_fwd":
        z = torch.matmul(x, d["w"].mT)
        if "b" in d:
            z += d["b"]
        if act == "relu":
            y = z.clamp(min=0.0)
        elif act == "gelu":
            y = z * 0.5 * torch.erfc(-z / math.sqrt(2.0))
        elif act == "silu":
            y = z / (1.0 + torch.exp(-z))
        else:
            y = z.clone()
        if "r" in d:
            y += d["r"]
        return {"y": y, "z": z if case["train"] else None}
    if case["op"] == "linear_bwd":
        z, dz = d.get("z"), d["dy"]
        if act == "relu":
            dz = torch.where(z > 0, dz, torch.zeros_like(dz))
        elif act == "gelu":
            dz = dz * (0.5 * torch.erfc(-z / math.sqrt(2.0)) + z * torch.exp(-z * z / 2.0) / math.sqrt(2.0 * math.pi))
        elif act == "silu":
            e = torch.exp(-z)
            dz = dz * ((1.0 + e + z * e) / (1.0 + e) ** 2)
        return {"dx": torch.matmul(dz, d["w"]), "dw": torch.matmul(dz.mT, x), "db": dz.sum(dim=0) if case["bias"] else None}
    if case["op"] == "layernorm_fwd":
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = (var + EPS) ** -0.5
        return {"y": torch.addcmul(d["beta"], (x - mean[:, None]) * rstd[:, None], d["gamma"]), "mean": mean, "rstd": rstd}
    h = (x - d["mean"][:, None]) * d["rstd"][:, None]
    n = x.shape[1]
    g = d["dy"] * d["gamma"]
    along = torch.einsum("ij,ij->i", g, h) / n
    dx = d["rstd"][:, None] * (g - g.sum(dim=1, keepdim=True) / n - along[:, None] * h)
    if "skip" in d:
        dx += d["skip"]
    return {"dx": dx, "dgamma": torch.einsum("ij,ij->j", d["dy"], h), "dbeta": d["dy"].sum(dim=0)}


# ------------------------------------------------------------------ what one pass cannot do without
def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    rows = case["rows"]
    if case["op"].startswith("linear"):
        n_in, n_out = case["in"], case["out"]
        weights = n_in * n_out + (n_out if case["bias"] else 0)
        if case["op"] == "linear_fwd":
            values = rows * n_in + weights + rows * n_out * (1 + int(case["residual"]) + int(case["train"]))
            return {"bytes": size * values, "flops": 2.0 * rows * n_in * n_out}
        values = rows * (2 * n_in + n_out * (1 if case["act"] == "none" else 2)) + n_in * n_out + weights
        return {"bytes": size * values, "flops": 4.0 * rows * n_in * n_out}
    n = case["width"]
    if case["op"] == "layernorm_fwd":
        return {"bytes": size * (2 * rows * n + 2 * n) + 8 * rows, "flops": 8.0 * rows * n}
    values = rows * n * (3 + int(case["skip"])) + 3 * n
    return {"bytes": size * values + 8 * rows, "flops": 14.0 * rows * n}
