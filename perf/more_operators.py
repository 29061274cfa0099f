"""Operators around the dense layers, as cases that can be timed and checked.

They are what a per-Gaussian attribute head needs beside its linear layers and its layer norm when it learns from
images: the lookup of learned codes (a code per view, per Gaussian or per cluster of Gaussians) with its gradient
summed over sorted indices, group normalisation with an activation over channels-last feature maps of the views with
its gradient, and the AdamW step that updates the head's tensors and its code tables, with moments in 32 or in 8 bits.

``run`` computes a case in plain torch operations when ``own`` is false and through
``gaussian_splatting_gb300.dense`` when it is true; ``exact`` gives the definition in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

EPS = 1e-5
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
ACTS = ("none", "relu", "gelu", "silu")
BETAS, ADAM_EPS, LR, DECAY = (0.9, 0.999), 1e-8, 1e-3, 1e-2
BLOCK = 256  # values that share a scale where moments are held in 8 bits
TOP = 448.0  # the largest value of float8_e4m3fn
SEED = 7     # of the rounding of 8-bit moments


# ------------------------------------------------------------------ cases
def _codes(name, op, rows, n, width, dtype, scale, skew, gaps=0.0, index="i32"):
    """``rows`` lookups in a table of ``n`` codes; ``skew``: some codes are much more common than others; ``gaps``:
    the share of rows that have no code (index -1)."""
    return {"name": name, "op": op, "rows": rows, "n": n, "width": width, "dtype": dtype, "scale": scale, "skew": skew,
            "gaps": gaps, "index": index}


def _norm(name, op, samples, rows, width, groups, dtype, act, skip=False):
    """``samples`` feature maps of ``rows`` pixels each."""
    return {"name": name, "op": op, "samples": samples, "rows": rows, "width": width, "groups": groups, "dtype": dtype,
            "act": act, "skip": skip}


def _adamw(name, hidden, blocks, table, bits, grads, copies):
    """The tensors of a residual head of ``blocks`` blocks (59 outputs, 24 inputs) and a table of ``table`` values."""
    return {"name": name, "op": "adamw", "hidden": hidden, "blocks": blocks, "table": table, "bits": bits, "grads": grads,
            "copies": copies}


def listed():
    return [
        # a learned code for each view of a batch of 16, out of a capture's 311 views: latency alone counts
        _codes("views-16 codes f32", "embedding_fwd", 16, 311, 32, "f32", 1.0, False),
        # a codebook of 65,536 entries read by the 10M Gaussians of a city scene, a few without an entry
        _codes("city-10m codebook bf16", "embedding_fwd", 10_000_000, 65_536, 64, "bf16", 8.0, True, 0.05),
        # gradient of a small scene's anchors: 2,048 Gaussians of 500 anchors, an odd width
        _codes("tiny-2k anchors f32 bwd", "embedding_bwd", 2_048, 500, 27, "f32", 1.0, False),
        # gradient of a codebook that the object scene shares, a few entries very common
        _codes("object-300k codebook bf16 bwd", "embedding_bwd", 300_000, 4_096, 64, "bf16", 8.0, True, 0.05),
        # gradient of 2M anchors that the 11M Gaussians of an unbounded scene hang on
        _codes("unbounded-11m anchors f32 bwd", "embedding_bwd", 11_000_000, 2_000_000, 32, "f32", 1.0, False),
        # small feature maps of 16 views: latency
        _norm("maps-16 32x32 f32", "groupnorm_fwd", 16, 1_024, 64, 8, "f32", "silu"),
        # one token per 8x8 block of 16 views at 1236x820
        _norm("maps-16 155x103 bf16", "groupnorm_fwd", 16, 15_965, 256, 32, "bf16", "silu"),
        # backward of odd maps and groups in f32, with the gradient of the residual path
        _norm("maps-4 77x51 f32 bwd", "groupnorm_bwd", 4, 3_927, 200, 20, "f32", "gelu", True),
        # backward over whole images: four views at 1236x820
        _norm("images-4 1236x820 bf16 bwd", "groupnorm_bwd", 4, 1_013_520, 64, 8, "bf16", "silu"),
        # a small head's update: 18 tensors, 21,000 parameters: latency
        _adamw("head f32", 64, 2, 0, 32, "f32", False),
        # a wide head that computes in bfloat16 (its gradients and working copies) with 8-bit moments
        _adamw("wide head bf16, 8 bits", 1_024, 8, 0, 8, "bf16", True),
        # a head and a table of 16 values for each of 11M Gaussians, whose moments would take 1.4 GB in 32 bits
        _adamw("head and 11m codes, 8 bits", 128, 2, 176_000_000, 8, "f32", False),
    ]


_MOST_BYTES = 2.8e9  # of the largest listed pass


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """A case of the listed ones' ranges: 1 to 11M lookups of 1 to 4M codes, feature maps of 1 to 1M pixels and 4 to 1024
    channels, 100 to 176M parameters; both types, every activation."""
    while True:
        op = rng.choice(["embedding_fwd", "embedding_bwd", "groupnorm_fwd", "groupnorm_bwd", "adamw"])
        dtype = rng.choice(["f32", "bf16"])
        if op.startswith("embedding"):
            width = _log_int(rng, 4, 1024)
            if rng.random() < 0.67:  # most programs keep their widths at multiples of 8
                width = max(8, width // 8 * 8)
            c = _codes("", op, _log_int(rng, 1, 11_000_000), _log_int(rng, 1, 4_000_000), width, dtype,
                       rng.choice([1.0, 8.0, math.sqrt(width)]), rng.random() < 0.5, rng.choice([0.0, 0.05]),
                       rng.choice(["i32", "i64"]))
        elif op.startswith("groupnorm"):
            per = rng.choice([1, 2, 3, 4, 8, 8, 10, 16, 16, 24, 32])
            groups = _log_int(rng, max(1, 4 // per), max(1, 1024 // per))
            c = _norm("", op, _log_int(rng, 1, 16), _log_int(rng, 1, 1_013_520), per * groups, groups, dtype,
                      rng.choice(ACTS), op == "groupnorm_bwd" and rng.random() < 0.5)
        else:
            c = _adamw("", _log_int(rng, 4, 1024), rng.randint(0, 8), rng.choice([0, _log_int(rng, 100, 176_000_000)]),
                       rng.choice([8, 32]), dtype, rng.random() < 0.5)
        del c["name"]
        if work(c)["bytes"] <= _MOST_BYTES:
            return c


# ------------------------------------------------------------------ inputs
def _gradient(rows, width, g):
    """A loss gradient per Gaussian: its length spans decades, and it is zero where no view saw the Gaussian."""
    scale = torch.pow(10.0, torch.rand((rows, 1), generator=g, device="cuda") * 2.0 - 6.0)
    scale *= torch.rand((rows, 1), generator=g, device="cuda") < 0.7
    if rows <= 16:
        scale = torch.full_like(scale, 1e-5)
    return torch.randn((rows, width), generator=g, device="cuda").mul_(scale)


def _head_shapes(c):
    """Shapes of the tensors that an AdamW case updates: the head's, then the table."""
    h = c["hidden"]
    shapes = [(h, 24), (h,)]
    for _ in range(c["blocks"]):
        shapes += [(h,), (h,), (h, h), (h,), (h, h), (h,)]
    shapes += [(h,), (h,), (59, h), (59,)]
    return shapes + ([(c["table"], 1)] if c["table"] else [])


def _pieces(c):
    """(start, length, decayed) of each tensor in the flat buffers: each starts at a multiple of BLOCK values."""
    at, got = 0, []
    for s in _head_shapes(c):
        n = math.prod(s)
        got.append((at, n, len(s) == 2))
        at += -(-n // BLOCK) * BLOCK
    return got, at


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c = dict(case)
    s = {"case": c}

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device="cuda").mul_(std)

    if c["op"].startswith("embedding"):
        t = DTYPES[c["dtype"]]
        u = torch.rand(c["rows"], generator=g, device="cuda", dtype=torch.float64)
        idx = (u ** 3 if c["skew"] else u).mul_(c["n"]).long().clamp_(max=c["n"] - 1)
        if c["gaps"]:
            idx[torch.rand(c["rows"], generator=g, device="cuda") < c["gaps"]] = -1
        s["idx"] = idx.int() if c["index"] == "i32" else idx
        if c["op"] == "embedding_fwd":
            s["table"] = normal(c["n"], c["width"], std=0.1).to(t)
        else:
            s["dy"] = _gradient(c["rows"], c["width"], g).to(t)
        return s
    if c["op"].startswith("groupnorm"):
        t, rows, n = DTYPES[c["dtype"]], c["samples"] * c["rows"], c["width"]
        x = normal(rows, n).mul_(0.5 + torch.rand((1, n), generator=g, device="cuda")).add_(normal(1, n, std=0.5))
        s["x"] = x.to(t)
        s["gamma"] = (1.0 + normal(n, std=0.1)).to(t)
        s["beta"] = normal(n, std=0.1).to(t)
        if c["op"] == "groupnorm_bwd":
            del x
            s["dy"] = _gradient(rows, n, g).to(t)
            s["skip"] = _gradient(rows, n, g).to(t) if c["skip"] else None
            xg = s["x"].float().view(c["samples"], c["rows"], c["groups"], -1)  # what the forward pass kept
            s["mean"] = xg.mean((1, 3))
            xg = xg - s["mean"][:, None, :, None]
            s["rstd"] = torch.rsqrt(xg.square_().mean((1, 3)) + EPS)
        return s
    pieces, total = _pieces(c)
    flat = {"p": normal(total, std=0.1), "g": _gradient(-(-total // 16), 16, g).view(-1)[:total].to(DTYPES[c["grads"]])}
    if c["bits"] == 32:
        flat["m"], flat["v"] = normal(total, std=1e-5), normal(total, std=1e-5).square_()
    else:  # moments as an earlier step left them: each block's largest at the top of the type
        for k in ("m", "v"):
            q = normal(total // BLOCK, BLOCK)
            q = q if k == "m" else q.abs_()
            q *= TOP / q.abs().amax(1, keepdim=True)
            flat[k] = (q if k == "m" else q.clamp_(min=2.0 ** -9)).view(-1).to(torch.float8_e4m3fn)
            flat[k + "_scale"] = torch.pow(10.0, torch.rand(total // BLOCK, generator=g, device="cuda") * 2.0 - 9.0)
    keep = torch.zeros(total, dtype=torch.bool, device="cuda")
    for at, n, _ in pieces:
        keep[at:at + n] = True
    for k in ("p", "g", "m", "v"):  # nothing between the tensors
        flat[k].view(torch.uint8 if flat[k].element_size() == 1 else torch.int16 if flat[k].element_size() == 2
                     else torch.int32).mul_(keep)
    if c["copies"]:
        flat["copy"] = torch.zeros(total, dtype=torch.bfloat16, device="cuda")
    shapes = _head_shapes(c)
    s["flat"] = flat
    for k, v in flat.items():  # the tensors as the program has them: views of the buffers
        s[k] = [v[at // BLOCK:at // BLOCK - (-n // BLOCK)] if k.endswith("scale") else v[at:at + n].view(shape)
                for (at, n, _), shape in zip(pieces, shapes)]
    s["decay"] = [DECAY if d else 0.0 for _, _, d in pieces]
    s["decay_of"] = torch.tensor(s["decay"], dtype=torch.float64, device="cuda")
    s["spans"] = torch.tensor([-(-n // BLOCK) * BLOCK for _, n, _ in pieces], device="cuda")
    s["step"] = 1000  # steps taken so far
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    from gaussian_splatting_gb300 import dense
    c = s["case"]
    op = c["op"]
    if op == "embedding_fwd":
        return {"y": dense.embedding_fwd(s["table"], s["idx"], c["scale"])}
    if op == "embedding_bwd":
        return {"dtable": dense.embedding_bwd(s["dy"], s["idx"], c["n"], c["scale"])}
    if op == "groupnorm_fwd":
        y, mean, rstd = dense.groupnorm_fwd(s["x"], s["gamma"], s["beta"], c["groups"], samples=c["samples"],
                                            act=c["act"], eps=EPS)
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "groupnorm_bwd":
        dx, dgamma, dbeta = dense.groupnorm_bwd(s["dy"], s["x"], s["gamma"], s["beta"], s["mean"], s["rstd"],
                                                act=c["act"], skip=s["skip"])
        return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
    s["step"] += 1
    scales = (s["m_scale"], s["v_scale"]) if c["bits"] == 8 else None
    dense.adamw(s["p"], s["g"], s["m"], s["v"], s["step"], lr=LR, betas=BETAS, eps=ADAM_EPS, weight_decay=s["decay"],
                scales=scales, copies=s.get("copy"), seed=SEED)
    return dict(s["flat"], g=None)


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
    op = c["op"]
    if op == "embedding_fwd":
        at = s["idx"].long()
        there = (at >= 0) & (at < c["n"])
        y = s["table"][at * there].float() * c["scale"]
        return {"y": (y * there[:, None]).to(s["table"].dtype)}
    if op == "embedding_bwd":
        # sums of up to millions of rows: in 64 bits; one row more takes what has no code
        at = s["idx"].long()
        at = torch.where((at >= 0) & (at < c["n"]), at, c["n"])
        sums = torch.zeros((c["n"] + 1, c["width"]), dtype=torch.float64, device="cuda")
        sums.index_add_(0, at, s["dy"].double())
        return {"dtable": (sums[:-1] * c["scale"]).to(s["dy"].dtype)}
    if op.startswith("groupnorm"):
        return _plain_norm(s)
    s["step"] += 1
    return _plain_adamw(s)


def _plain_norm(s):
    c, t = s["case"], s["x"].dtype
    x = s["x"].float().view(c["samples"], c["rows"], c["groups"], -1)
    gamma, beta = s["gamma"].float().view(c["groups"], -1), s["beta"].float().view(c["groups"], -1)
    if c["op"] == "groupnorm_fwd":
        mean = x.mean((1, 3), keepdim=True)
        d = x - mean
        rstd = 1.0 / torch.sqrt((d * d).mean((1, 3), keepdim=True) + EPS)
        y = _act(d * rstd * gamma + beta, c["act"])
        return {"y": y.to(t).view(s["x"].shape), "mean": mean[:, 0, :, 0], "rstd": rstd[:, 0, :, 0]}
    rstd = s["rstd"][:, None, :, None]
    h = (x - s["mean"][:, None, :, None]) * rstd
    dz = s["dy"].float().view(x.shape)
    if c["act"] != "none":
        dz = dz * _act_slope(h * gamma + beta, c["act"])
    dgamma, dbeta = (dz * h).sum((0, 1)), dz.sum((0, 1))
    dz = dz * gamma
    dx = (dz - dz.mean((1, 3), keepdim=True) - h * (dz * h).mean((1, 3), keepdim=True)) * rstd
    dx = dx.view(s["x"].shape)
    if s["skip"] is not None:
        dx = dx + s["skip"].float()
    return {"dx": dx.to(t), "dgamma": dgamma.view(-1).to(t), "dbeta": dbeta.view(-1).to(t)}


def _noise(n, step):
    """32 random bits for each value of the call, of its number, the seed and the step."""
    low = 0xFFFFFFFF
    h = torch.arange(n, device="cuda") * 0x9E3779B1 + (SEED * 0x6A09E667 + step * 0xBB67AE85) & low
    h = ((h ^ (h >> 16)) * 0x6A09E667) & low
    h = ((h ^ (h >> 15)) * 0xBB67AE85) & low
    return h ^ (h >> 16)


def _to_8_bits(x, noise):
    """x [blocks, BLOCK] as float8 values and a scale per block.  16 random bits decide whether a value's bits beyond
    the type's four significant ones round it up."""
    top = x.abs().amax(1, keepdim=True)
    top = top * (top >= 2.0 ** -100)
    q = (x * torch.where(top > 0, top.reciprocal() * TOP, top)).clamp(-TOP, TOP)
    bits = q.view(torch.int32) + (noise.view(x.shape) << 4).int()
    return (bits & -0x100000).view(torch.float32), (top * (1.0 / TOP))[:, 0]


def _plain_adamw(s):
    c, f, t = s["case"], s["flat"], s["step"]
    b1, b2 = BETAS
    g = f["g"].float()
    m, v = f["m"].float(), f["v"].float()
    if c["bits"] == 8:
        m = (m.view(-1, BLOCK) * f["m_scale"][:, None]).view(-1)
        v = (v.view(-1, BLOCK) * f["v_scale"][:, None]).view(-1)  # the root of the second moment
        v = v * v
    m = m * b1 + g * (1.0 - b1)
    v = v * b2 + (g * g) * (1.0 - b2)
    root = torch.sqrt(v)
    keep = torch.repeat_interleave((1.0 - LR * s["decay_of"]).float(), s["spans"], output_size=g.numel())
    p = f["p"] * keep - m * (LR / (1.0 - b1 ** t)) / (root * (1.0 / math.sqrt(1.0 - b2 ** t)) + ADAM_EPS)
    f["p"].copy_(p)
    if c["copies"]:
        f["copy"].copy_(p)
    if c["bits"] == 32:
        f["m"].copy_(m)
        f["v"].copy_(v)
    else:
        noise = _noise(g.numel(), t)
        q, scale = _to_8_bits(m.view(-1, BLOCK), noise & 0xFFFF)
        f["m"].copy_(q.view(-1))
        f["m_scale"].copy_(scale)
        q, scale = _to_8_bits(root.view(-1, BLOCK), noise >> 16)
        # what is not zero stays so: the next step divides by it
        q = torch.where((root.view(-1, BLOCK) > 0) & (scale[:, None] > 0), q.clamp(min=2.0 ** -9), q)
        f["v"].copy_(q.view(-1))
        f["v_scale"].copy_(scale)
    return dict(f, g=None)


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "embedding_fwd":
        padded = torch.cat([s["table"].double() * c["scale"], torch.zeros((1, c["width"]), dtype=torch.float64, device="cuda")])
        return {"y": padded[s["idx"].long()]}  # -1 is the row of zeros
    if c["op"] == "embedding_bwd":
        # differences of running sums over the sorted rows
        at, order = s["idx"].long().sort()
        total = torch.nn.functional.pad(s["dy"][order].t().double(), (1, 0)).cumsum(1)
        ends = torch.searchsorted(at, torch.arange(c["n"] + 1, device="cuda"))
        return {"dtable": (total[:, ends[1:]] - total[:, ends[:-1]]).t() * c["scale"]}
    if c["op"].startswith("groupnorm"):
        return _exact_norm(s)
    return _exact_adamw(s)


def _exact_norm(s):
    c = s["case"]
    n, r, k, w = c["samples"], c["rows"], c["groups"], c["width"] // c["groups"]
    gamma, beta = (s[k_].double().view(k, 1, w) for k_ in ("gamma", "beta"))
    out = {}
    parts = {"dgamma": 0.0, "dbeta": 0.0}
    per_sample = {"y": [], "mean": [], "rstd": [], "dx": []}
    for i in range(n):  # sample by sample: 64 bits of all of them would not fit three times
        x = s["x"][i * r:(i + 1) * r].double().view(r, k, w).transpose(0, 1)
        if c["op"] == "groupnorm_fwd":
            var, mean = torch.var_mean(x, dim=(1, 2), correction=0)
            rstd = (var + EPS) ** -0.5
        else:
            mean, rstd = s["mean"][i].double(), s["rstd"][i].double()
        h = (x - mean[:, None, None]) * rstd[:, None, None]
        z = torch.addcmul(beta, h, gamma)
        if c["op"] == "groupnorm_fwd":
            if c["act"] == "relu":
                z = z.clamp(min=0.0)
            elif c["act"] == "gelu":
                z = z * 0.5 * torch.erfc(-z / math.sqrt(2.0))
            elif c["act"] == "silu":
                z = z / (1.0 + torch.exp(-z))
            per_sample["y"].append(z.transpose(0, 1).reshape(r, -1))
            per_sample["mean"].append(mean)
            per_sample["rstd"].append(rstd)
            continue
        d = s["dy"][i * r:(i + 1) * r].double().view(r, k, w).transpose(0, 1)
        if c["act"] == "relu":
            d = torch.where(z > 0, d, torch.zeros_like(d))
        elif c["act"] == "gelu":
            d = d * (0.5 * torch.erfc(-z / math.sqrt(2.0)) + z * torch.exp(-z * z / 2.0) / math.sqrt(2.0 * math.pi))
        elif c["act"] == "silu":
            e = torch.exp(-z)
            d = d * ((1.0 + e + z * e) / (1.0 + e) ** 2)
        parts["dbeta"] = parts["dbeta"] + d.sum(dim=1)
        parts["dgamma"] = parts["dgamma"] + torch.einsum("grc,grc->gc", d, h)
        a = d * gamma
        along = torch.einsum("grc,grc->g", a, h) / (r * w)
        dx = rstd[:, None, None] * (a - a.sum(dim=(1, 2))[:, None, None] / (r * w) - along[:, None, None] * h)
        dx = dx.transpose(0, 1).reshape(r, -1)
        if s["skip"] is not None:
            dx += s["skip"][i * r:(i + 1) * r].double()
        per_sample["dx"].append(dx)
    if c["op"] == "groupnorm_fwd":
        return {"y": torch.cat(per_sample["y"]), "mean": torch.stack(per_sample["mean"]), "rstd": torch.stack(per_sample["rstd"])}
    out["dx"] = torch.cat(per_sample["dx"])
    return dict(out, dgamma=parts["dgamma"].reshape(-1), dbeta=parts["dbeta"].reshape(-1))


def _exact_adamw(s):
    """Moments in 8 bits are rounded at random: they have no value of their own here, their scales have."""
    c, f = s["case"], s["flat"]
    t = s["step"] + 1
    out = {"p": torch.zeros_like(f["p"], dtype=torch.float64), "g": None}
    for k in ("m", "v"):
        out[k] = None if c["bits"] == 8 else torch.zeros_like(f["p"], dtype=torch.float64)
        if c["bits"] == 8:
            out[k + "_scale"] = torch.zeros_like(f[k + "_scale"], dtype=torch.float64)
    for (at, n, decayed), g in zip(_pieces(c)[0], s["g"]):
        g, span, blocks = g.double().reshape(-1), slice(at, at + n), slice(at // BLOCK, at // BLOCK - (-n // BLOCK))
        m, v = f["m"][span].double(), f["v"][span].double()
        if c["bits"] == 8:
            m *= f["m_scale"][blocks].double().repeat_interleave(BLOCK)[:n]
            v = (v * f["v_scale"][blocks].double().repeat_interleave(BLOCK)[:n]) ** 2
        m, v = torch.lerp(g, m, BETAS[0]), torch.lerp(g * g, v, BETAS[1])
        p = f["p"][span].double()
        step = (m / (1.0 - BETAS[0] ** t)) / ((v / (1.0 - BETAS[1] ** t)) ** 0.5 + ADAM_EPS)
        out["p"][span] = p - LR * ((DECAY if decayed else 0.0) * p + step)
        for k, x in (("m", m), ("v", v if c["bits"] == 32 else v ** 0.5)):
            if c["bits"] == 32:
                out[k][span] = x
            else:
                x = torch.nn.functional.pad(x.abs(), (0, -n % BLOCK))
                out[k + "_scale"][blocks] = x.view(-1, BLOCK).max(dim=1).values / TOP
    if c["copies"]:
        out["copy"] = out["p"]
    return out


# ------------------------------------------------------------------ what one pass cannot do without
def work(case):
    c = case
    if c["op"] == "adamw":
        # parameters, moments: read and written; gradients read; the copies written
        n = sum(math.prod(s) for s in _head_shapes(c))
        states = 16.0 if c["bits"] == 32 else 4.0 + 16.0 / BLOCK
        return {"bytes": n * (8.0 + states + (4 if c["grads"] == "f32" else 2) + (2 if c["copies"] else 0)), "flops": 16.0 * n}
    size = 4 if c["dtype"] == "f32" else 2
    if c["op"].startswith("embedding"):
        index = (4 if c["index"] == "i32" else 8) * c["rows"]
        if c["op"] == "embedding_fwd":  # of the table what the rows can reach
            return {"bytes": size * c["width"] * (min(c["n"], c["rows"]) + c["rows"]) + index, "flops": 1.0 * c["rows"] * c["width"]}
        return {"bytes": size * c["width"] * (c["n"] + c["rows"]) + index, "flops": 1.0 * c["rows"] * c["width"]}
    values, sums = c["samples"] * c["rows"] * c["width"], 8 * c["samples"] * c["groups"]
    if c["op"] == "groupnorm_fwd":
        return {"bytes": size * (2 * values + 2 * c["width"]) + sums, "flops": 12.0 * values}
    return {"bytes": size * (values * (3 + int(c["skip"])) + 4 * c["width"]) + sums, "flops": 24.0 * values}
