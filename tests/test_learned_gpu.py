"""Code lookup, group norm and AdamW (gs_embedding_*, gs_groupnorm_*, gs_adamw) against the same formulas in 64 bits.

Tolerances are derived from the arithmetic, elementwise.  With u = 2^-24 (a 32-bit rounding):
 - a sum of k terms whose signs vary: (8 + 2 sqrt(k)) u times the sum of the terms' absolute values;
 - the type's own rounding of a stored value: 2^-8 (bfloat16) or 2^-24 (float32) of it;
 - group norm adds no more than CHAIN terms one after the other (a thread's rows, a lane's share of a block's threads, its
   share of the chunks); the variance is taken about pivots among the values, so its error is that of a mean of squares of at
   most D^2, D the largest distance of two values;
 - the activations are evaluated to a few u of their argument (slopes at most 1.13, second derivatives at most 0.8).
"""
import math
import os
import sys

import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a CUDA device", allow_module_level=True)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

from gaussian_splatting_gb300 import dense  # noqa: E402

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, BF16, F8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
ROUND = {F32: 2.0 ** -24, BF16: 2.0 ** -8}
TINY = 2.0 ** -126
CHAIN = 600
ACTS = ["none", "relu", "gelu", "silu"]
both = pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])


def _sum_u(k):
    return (8 + 2 * math.sqrt(k)) * U


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rand(shape, dtype, seed, std=1.0, pad=0, shift=0, mean=0.0):
    """A normal matrix or vector; `pad` extra elements between rows, `shift` elements off the allocation."""
    v = (torch.randn(shape, generator=_gen(seed), device="cuda") * std + mean).to(dtype)
    if not pad and not shift:
        return v
    width = shape[-1] + (pad if len(shape) > 1 else 0)
    out = torch.zeros(math.prod(shape[:-1]) * width + shift, dtype=dtype, device="cuda")[shift:]
    out = out.view(*shape[:-1], width)[..., :shape[-1]]
    out.copy_(v)
    return out


def _close(got, want, tol, what):
    off = (got.double() - want).abs()
    assert torch.isfinite(got.double()).all(), f"{what}: not finite"
    out = int((~(off <= tol)).sum())
    assert out == 0, f"{what}: {out} of {off.numel()} out, worst ratio {(off / tol).max().item():.3g}"


# ------------------------------------------------------------------ code lookup
def _indices(rows, n, kind, seed, dtype=torch.int32):
    u = torch.rand(rows, generator=_gen(seed), device="cuda", dtype=torch.float64)
    if kind == "one":
        idx = torch.full((rows,), n - 1, device="cuda")
    elif kind == "sorted":
        idx = (u * n).long().sort().values
    else:
        idx = ((u ** 4 if kind == "skewed" else u) * n).long()
    idx = idx.clamp(0, max(n - 1, 0)).to(dtype)
    if kind == "gaps":
        idx[torch.rand(rows, generator=_gen(seed + 1), device="cuda") < 0.3] = -1
        idx[::7] = n
        idx[::11] = torch.iinfo(dtype).min
        idx[3::13] = torch.iinfo(dtype).max
    if kind == "none":
        idx[:] = -1
    return idx


def _lookup(table, idx, scale):
    at = idx.long()
    there = (at >= 0) & (at < table.shape[0])
    return torch.cat([table.double(), torch.zeros_like(table[:1]).double()])[torch.where(there, at, table.shape[0])] * scale


def _gradient(dy, idx, n, scale):
    """The sums, and the sums of absolute values with the counts."""
    at = idx.long()
    at = torch.where((at >= 0) & (at < n), at, n)
    out = []
    for t in (dy.double(), dy.double().abs()):
        out.append(torch.zeros((n + 1, dy.shape[1]), dtype=torch.float64, device="cuda").index_add_(0, at, t)[:n] * scale)
    return out[0], out[1].abs(), torch.bincount(at, minlength=n + 1)[:n]


def _check_embedding(rows, n, width, dtype, kind, scale=1.0, idx_dtype=torch.int32, pad=0, shift=0, seed=1):
    idx = _indices(rows, n, kind, seed, idx_dtype)
    scale = float(torch.tensor(scale, dtype=F32))
    table = _rand((n, width), dtype, seed + 2, 1.0, pad, shift)
    y = dense.embedding_fwd(table, idx, scale)
    want = _lookup(table, idx, scale)
    assert y.dtype == dtype and y.shape == (rows, width)
    _close(y, want, 1.01 * ROUND[dtype] * want.abs() + TINY, "y")
    dy = _rand((rows, width), dtype, seed + 3, 1e-3, pad, shift)
    out = _rand((n, width), dtype, seed + 4, 1.0, pad, shift)  # overwritten, what lies between its rows is not
    full = out.as_strided((n, width + pad), (width + pad, 1))[:-1] if pad else None
    between = full[:, width:].clone() if pad else None
    got = dense.embedding_bwd(dy, idx, n, scale, dtable=out)
    assert got.data_ptr() == out.data_ptr()
    want, mag, counts = _gradient(dy, idx, n, scale)
    tol = (8 + 2 * counts.double().sqrt())[:, None] * U * mag + 1.01 * ROUND[dtype] * want.abs() + TINY
    _close(got, want, tol, "dtable")
    assert not got[counts == 0].any()
    if pad:
        assert torch.equal(full[:, width:], between)
    again = dense.embedding_bwd(dy, idx, n, scale)
    if not pad and not shift:
        assert torch.equal(again, got)
    return got


# rows, codes, width: one of everything, tiles' and parts' edges, one to four digits of sorting, odd widths
LOOKUPS = [(1, 1, 1), (1, 5, 3), (7, 1, 8), (16, 311, 32), (33, 2, 27), (255, 256, 4), (256, 255, 5), (1000, 40, 130),
           (2048, 500, 27), (4095, 17, 16), (4097, 65_536, 12), (5000, 3, 1), (9001, 70_000, 7), (20_000, 300, 64),
           (70_000, 1_000_000, 2), (300_000, 4096, 9), (123_457, 12_345, 31), (3000, 1 << 25, 1)]


@both
@pytest.mark.parametrize("shape", LOOKUPS, ids=str)
def test_embedding(shape, dtype):
    rows, n, width = shape
    kinds = ["uniform", "skewed", "gaps", "one", "sorted", "none"]
    k = LOOKUPS.index(shape)
    for i, kind in enumerate(kinds):
        if n > 1 << 22 and i % 3:
            continue
        _check_embedding(rows, n, width, dtype, kind, scale=[1.0, 8.0, -0.3][(i + k) % 3],
                         idx_dtype=[torch.int32, torch.int64][(i + k) % 2], seed=10 * i + k)


@both
@pytest.mark.parametrize("width,pad,shift", [(64, 8, 0), (64, 4, 0), (64, 3, 1), (24, 2, 0), (256, 0, 0), (300, 0, 4),
                                             (513, 0, 0), (1024, 0, 0), (1030, 2, 0)])
def test_embedding_strides_and_widths(width, pad, shift, dtype):
    _check_embedding(3001, 77, width, dtype, "skewed", 2.0, pad=pad, shift=shift)
    _check_embedding(500, 2000, width, dtype, "gaps", 2.0, pad=pad, shift=shift)


@both
def test_embedding_codes_of_many_rows(dtype):
    """Codes whose rows fill several blocks, next to each other and at both ends."""
    for rows, n, kind in ((1_000_000, 1, "one"), (1_000_000, 3, "uniform"), (500_000, 5000, "skewed")):
        _check_embedding(rows, n, 20, dtype, kind)


# many rows, which go to buckets of codes: one code a bucket, several, as many as fit, too many (again the sort); a common
# bucket and a common code, which take several parts; rows of few and of many vectors
MANY = [(1_600_000, 257, 3, "uniform"), (1_600_000, 300, 8, "skewed"), (1_700_000, 5000, 40, "skewed"),
        (1_600_001, 70_001, 16, "gaps"), (2_000_000, 1_000_000, 24, "uniform"), (1_573_000, 1 << 22, 4, "skewed"),
        (3_000_000, 4099, 5, "one"), (1_600_000, 3_000_000, 2, "sorted"), (1_600_000, 40_000, 300, "skewed"),
        (1_600_000, (1 << 22) + 1, 3, "uniform"), (1_600_000, 1000, 6, "none"),
        (1 << 20, 65_536, 12, "skewed"), ((1 << 20) - 1, 65_536, 12, "uniform")]


@both
@pytest.mark.parametrize("case", MANY, ids=str)
def test_embedding_many_rows(case, dtype):
    rows, n, width, kind = case
    k = MANY.index(case)
    _check_embedding(rows, n, width, dtype, kind, [1.0, -3.0][k % 2], [torch.int32, torch.int64][k // 2 % 2], seed=50 + k)
    if width % 8 == 0:  # rows apart and off 16 bytes
        _check_embedding(rows, n, width, dtype, kind, 1.0, pad=5, shift=1, seed=70 + k)


def test_embedding_many_rows_infinities_stay_in_their_code():
    rows, n = 1_600_000, 2000
    idx = _indices(rows, n, "skewed", 3)
    dy = _rand((rows, 16), F32, 4)
    clean = dense.embedding_bwd(dy, idx, n)
    dy[idx == 0] = float("inf")
    dy[idx == 77] = float("nan")
    got = dense.embedding_bwd(dy, idx, n)
    assert torch.isinf(got[0]).all() and torch.isnan(got[77]).all()
    others = torch.ones(n, dtype=torch.bool, device="cuda")
    others[[0, 77]] = False
    assert torch.equal(got[others], clean[others])


def test_embedding_with_nothing_to_do():
    table = _rand((5, 6), F32, 1)
    none = torch.zeros(0, dtype=torch.int64, device="cuda")
    assert dense.embedding_fwd(table, none).shape == (0, 6)
    assert not dense.embedding_bwd(table[:0], none, 5, dtable=torch.ones((5, 8), device="cuda")[:, :6]).any()
    idx = torch.zeros(4, dtype=torch.int32, device="cuda")
    assert not dense.embedding_fwd(table[:0], idx, out=torch.ones((4, 6), device="cuda")).any()
    assert dense.embedding_bwd(_rand((4, 6), F32, 2), idx, 0).shape == (0, 6)


def test_embedding_infinities_stay_in_their_code():
    """A row without a code, and the codes of other rows, see nothing of them."""
    dy = _rand((6000, 10), F32, 3)
    idx = _indices(6000, 50, "uniform", 4)
    dy[idx == 7] = math.inf
    dy[idx == 9] = math.nan
    dy[::50] = math.nan
    idx[::50] = -1
    got = dense.embedding_bwd(dy, idx, 50)
    fine = torch.ones(50, dtype=torch.bool, device="cuda")
    fine[7] = fine[9] = False
    assert torch.isfinite(got[fine]).all() and torch.isinf(got[7]).all() and torch.isnan(got[9]).all()
    table = _rand((50, 10), F32, 5)
    table[0] = math.nan
    assert torch.isfinite(dense.embedding_fwd(table, torch.full((9,), -1, dtype=torch.int32, device="cuda"))).all()


def test_embedding_offsets_past_2_to_31():
    """Rows far apart, and an output of more than 2^31 values."""
    far = torch.empty((3, 1 << 30), dtype=BF16, device="cuda")[:, :40]
    far.copy_(_rand((3, 40), BF16, 6))
    idx = _indices(500, 3, "uniform", 7)
    assert torch.equal(dense.embedding_fwd(far, idx), far[idx.long()])
    dy = _rand((500, 40), BF16, 8)
    got = dense.embedding_bwd(dy, idx, 3, dtable=far)
    assert torch.equal(got, dense.embedding_bwd(dy, idx, 3))
    table, idx = _rand((100, 256), BF16, 9), _indices(9_000_000, 100, "uniform", 10)
    y = dense.embedding_fwd(table, idx)
    for part in (slice(0, 1000), slice(8_388_000, 8_390_000), slice(-1000, None)):
        assert torch.equal(y[part], table[idx[part].long()])
    dy = y[-500_000:]
    far = dense.embedding_bwd(y, torch.where(torch.arange(9_000_000, device="cuda") >= 8_500_000, idx, -1), 100)
    want, mag, counts = _gradient(dy, idx[-500_000:], 100, 1.0)
    _close(far, want, (8 + 2 * counts.double().sqrt())[:, None] * U * mag + 1.01 * ROUND[BF16] * want.abs(), "dtable")


# ------------------------------------------------------------------ group norm
def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2.0))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def _slope(z, act):
    if act == "relu":
        return (z > 0).double()
    if act == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2.0)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


def _norm_case(samples, rows, width, groups, dtype, seed=1, pad=0, shift=0, mean=0.5):
    x = _rand((samples * rows, width), dtype, seed, 1.5, pad, shift, mean)
    gamma, beta = _rand((width,), dtype, seed + 1, 0.3, 0, shift, 1.0), _rand((width,), dtype, seed + 2, 0.3, 0, shift)
    return x, gamma, beta


def _check_norm_fwd(samples, rows, groups, x, gamma, beta, act, eps, got):
    y, mean, rstd = got
    width = x.shape[1]
    X = x.double().reshape(samples, rows, groups, -1)
    mu = X.mean((1, 3), keepdim=True)
    var = (X - mu).square().mean((1, 3), keepdim=True)
    D = X.amax((1, 3), keepdim=True) - X.amin((1, 3), keepdim=True)
    r = (var + eps) ** -0.5
    emu = _sum_u(CHAIN) * (mu.abs() + D)
    er = (0.5 * (_sum_u(CHAIN) * D * D + emu * emu) / (var + eps) + 4 * U) * r
    if mean is not None:
        _close(mean, mu[:, 0, :, 0], emu[:, 0, :, 0], "mean")
        _close(rstd, r[:, 0, :, 0], er[:, 0, :, 0], "rstd")
    G, B = gamma.double().view(groups, -1), beta.double().view(groups, -1)
    h = (X - mu) * r
    z = h * G + B
    ez = (emu * r + (X - mu).abs() * er) * G.abs() + 4 * U * ((h * G).abs() + B.abs())
    want = _act(z, act).reshape(-1, width)
    tol = (1.13 * ez + 8 * U * z.abs()).reshape(-1, width) + 1.01 * ROUND[x.dtype] * want.abs() + TINY
    _close(y, want, tol, f"y {act}")


# maps, rows, channels, groups: one of everything, groups of one channel, one group, odd groups, rows at chunks' edges
NORMS = [(1, 1, 1, 1), (1, 1, 8, 2), (3, 1, 64, 8), (1, 7, 5, 5), (2, 33, 6, 3), (16, 1024, 64, 8), (4, 257, 200, 20),
         (1, 5000, 32, 1), (5, 100, 96, 96), (2, 4096, 24, 2), (3, 77, 1030, 10), (1, 300, 2048, 4), (2, 64, 4100, 2),
         (300, 9, 16, 4), (1, 100_000, 8, 2), (7, 1000, 59, 1), (2, 500, 100, 25), (1, 40, 9000, 3)]


@both
@pytest.mark.parametrize("shape", NORMS, ids=str)
def test_groupnorm_forward(shape, dtype):
    samples, rows, width, groups = shape
    x, gamma, beta = _norm_case(samples, rows, width, groups, dtype, NORMS.index(shape))
    for act in ACTS:
        got = dense.groupnorm_fwd(x, gamma, beta, groups, samples, act, 1e-5, stats=act != "relu")
        assert (got[1] is None) == (act == "relu") == (got[2] is None)
        _check_norm_fwd(samples, rows, groups, x, gamma, beta, act, 1e-5, got)
    again = dense.groupnorm_fwd(x, gamma, beta, groups, samples, act, 1e-5)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


# maps whose groups a block holds, at the edges of that: as many rows as fit (512 threads, 8 vectors of 16 bytes or 32 shorter
# ones each) and one more, groups as wide as the block and wider, next to 16 MB, next to 6,080 blocks, mean and rstd either way
SMALL = [(2, 2048, 16, 2), (2, 2049, 16, 2), (1, 4096, 16, 4), (3, 5461, 9, 3), (3, 5462, 9, 3), (1, 8, 4096, 1), (2, 3, 8192, 2),
         (1, 33, 1028, 2), (16, 1024, 256, 32), (17, 1024, 256, 32), (380, 3, 32, 16), (381, 3, 32, 16), (7, 100, 30, 3),
         (1, 4095, 32, 1)]


@both
@pytest.mark.parametrize("shape", SMALL, ids=str)
def test_groupnorm_small_maps(shape, dtype):
    samples, rows, width, groups = shape
    for act, pad, shift in (("silu", 0, 0), ("gelu", 3, 1)):
        x, gamma, beta = _norm_case(samples, rows, width, groups, dtype, 60 + SMALL.index(shape), pad, shift, 3.0)
        got = dense.groupnorm_fwd(x, gamma, beta, groups, samples, act, 1e-5)
        _check_norm_fwd(samples, rows, groups, x, gamma, beta, act, 1e-5, got)
        y, mean, rstd = dense.groupnorm_fwd(x, gamma, beta, groups, samples, act, 1e-5, stats=False)
        assert mean is None and rstd is None and torch.equal(y, got[0])
        out = x.clone()
        assert torch.equal(dense.groupnorm_fwd(out, gamma, beta, groups, samples, act, 1e-5, out=out)[0],
                           dense.groupnorm_fwd(x.clone(), gamma, beta, groups, samples, act, 1e-5)[0])


@both
@pytest.mark.parametrize("mean", [0.0, 30.0, -1000.0])
def test_groupnorm_far_from_zero(mean, dtype):
    """A mean of many times the spread costs the mean's own rounding, not the variance's digits."""
    x, gamma, beta = _norm_case(3, 3000, 40, 5, dtype, 3, mean=mean)
    _check_norm_fwd(3, 3000, 5, x, gamma, beta, "none", 1e-5, dense.groupnorm_fwd(x, gamma, beta, 5, 3))


def _norm_grads(samples, groups, dy, x, gamma, beta, mean, rstd, act, skip):
    rows, width = x.shape[0] // samples, x.shape[1]
    X, DY = (t.double().reshape(samples, rows, groups, -1) for t in (x, dy))
    G, B = gamma.double().view(groups, -1), beta.double().view(groups, -1)
    m, r = mean.double()[:, None, :, None], rstd.double()[:, None, :, None]
    h = (X - m) * r
    z = h * G + B
    ez = 4 * U * ((h * G).abs() + B.abs())
    if act == "none":
        dz, ed = DY, torch.zeros_like(DY)
    else:
        dz = DY * _slope(z, act)
        ed = DY.abs() * (16 * U * (1 + z.abs()) + 0.8 * ez)
        if act == "relu":
            ed = 2 * U * dz.abs() + DY.abs() * (z.abs() <= ez)  # the slope jumps there
    g, eg = dz * G, ed * G.abs() + 2 * U * (dz * G).abs()
    avg = lambda t: t.mean((1, 3), keepdim=True)  # noqa: E731
    m1, m2 = avg(g), avg(g * h)
    e1 = avg(eg) + _sum_u(CHAIN) * avg(g.abs())
    e2 = avg((eg + 4 * U * g.abs()) * h.abs()) + _sum_u(CHAIN) * avg((g * h).abs())
    dx = r * (g - m1 - h * m2)
    edx = r * (eg + e1 + h.abs() * e2 + 6 * U * (g.abs() + m1.abs() + (h * m2).abs()))
    dx, edx = dx.reshape(x.shape), edx.reshape(x.shape)
    if skip is not None:
        dx, edx = dx + skip.double(), edx + 2 * U * (dx.abs() + skip.double().abs())
    over = lambda t: t.sum((0, 1)).reshape(-1)  # noqa: E731
    v = ROUND[x.dtype]
    dg, db = over(dz * h), over(dz)
    out = {"dx": (dx, edx), "dgamma": (dg, over((ed + 4 * U * dz.abs()) * h.abs()) + _sum_u(CHAIN) * over((dz * h).abs())),
           "dbeta": (db, over(ed) + _sum_u(CHAIN) * over(dz.abs()))}
    return {k: (w, e + 1.01 * v * w.abs() + TINY) for k, (w, e) in out.items()}


@both
@pytest.mark.parametrize("shape", NORMS, ids=str)
def test_groupnorm_backward(shape, dtype):
    samples, rows, width, groups = shape
    k = NORMS.index(shape)
    x, gamma, beta = _norm_case(samples, rows, width, groups, dtype, k)
    _, mean, rstd = dense.groupnorm_fwd(x, gamma, beta, groups, samples)
    dy, skip = _rand(x.shape, dtype, k + 30, 1e-3), _rand(x.shape, dtype, k + 31, 1e-3)
    for i, act in enumerate(ACTS):
        s = skip if (i + k) % 2 else None
        got = dense.groupnorm_bwd(dy, x, gamma, beta, mean, rstd, act=act, skip=s)
        want = _norm_grads(samples, groups, dy, x, gamma, beta, mean, rstd, act, s)
        for name, v in zip(("dx", "dgamma", "dbeta"), got):
            _close(v, *want[name], f"{name} {act}")
    dx = dense.groupnorm_bwd(dy, x, gamma, beta, mean, rstd, act=act, skip=s, need_dparams=False)
    assert torch.equal(dx[0], got[0]) and dx[1] is None and dx[2] is None
    sums = dense.groupnorm_bwd(dy, x, gamma, beta, mean, rstd, act=act, skip=s, need_dx=False)
    assert sums[0] is None and torch.equal(sums[1], got[1]) and torch.equal(sums[2], got[2])


@both
@pytest.mark.parametrize("pad,shift", [(8, 0), (4, 0), (2, 0), (1, 0), (8, 1), (0, 3), (0, 8)])
def test_groupnorm_strides(pad, shift, dtype):
    samples, rows, width, groups = 3, 211, 48, 6
    x, gamma, beta = _norm_case(samples, rows, width, groups, dtype, 5, pad, shift)
    dy, skip = _rand(x.shape, dtype, 40, 1e-3, pad, shift), _rand(x.shape, dtype, 41, 1e-3, pad + 8, 0)
    out = _rand(x.shape, dtype, 42, 1.0, pad + 1, shift)
    wide = out.as_strided((samples * rows - 1, width + pad + 1), out.stride())
    between = wide[:, width:].clone()
    got = dense.groupnorm_fwd(x, gamma, beta, groups, samples, "silu", out=out)
    assert got[0].data_ptr() == out.data_ptr()
    _check_norm_fwd(samples, rows, groups, x, gamma, beta, "silu", 1e-5, got)
    mean, rstd = got[1:]
    got = dense.groupnorm_bwd(dy, x, gamma, beta, mean, rstd, act="silu", skip=skip, dx=out)
    want = _norm_grads(samples, groups, dy, x, gamma, beta, mean, rstd, "silu", skip)
    for name, v in zip(("dx", "dgamma", "dbeta"), got):
        _close(v, *want[name], name)
    assert torch.equal(wide[:, width:], between)


@both
def test_groupnorm_in_place(dtype):
    x, gamma, beta = _norm_case(2, 3000, 64, 8, dtype, 6)
    dy, skip = _rand(x.shape, dtype, 50), _rand(x.shape, dtype, 51)
    y, mean, rstd = dense.groupnorm_fwd(x, gamma, beta, 8, 2, "gelu")
    dx, dg, db = dense.groupnorm_bwd(dy, x, gamma, beta, mean, rstd, act="gelu", skip=skip)
    for reuse in (dy, skip):
        given = {"dy": dy.clone(), "skip": skip.clone()}
        into = given["dy" if reuse is dy else "skip"]
        got = dense.groupnorm_bwd(given["dy"], x, gamma, beta, mean, rstd, act="gelu", skip=given["skip"], dx=into)
        assert got[0].data_ptr() == into.data_ptr()
        assert torch.equal(got[0], dx) and torch.equal(got[1], dg) and torch.equal(got[2], db)
    same = x.clone()
    assert torch.equal(dense.groupnorm_fwd(same, gamma, beta, 8, 2, "gelu", out=same)[0], y)


def test_groupnorm_with_nothing_to_do():
    gamma, beta = _rand((6,), F32, 1), _rand((6,), F32, 2)
    none = torch.zeros((0, 6), device="cuda")
    y, mean, rstd = dense.groupnorm_fwd(none, gamma, beta, 3, samples=2, eps=0.25)
    assert y.shape == (0, 6) and mean.tolist() == [[0.0] * 3] * 2 and rstd.tolist() == [[2.0] * 3] * 2
    dx, dg, db = dense.groupnorm_bwd(none, none, gamma, beta, mean, rstd, act="silu")
    assert dx.shape == (0, 6) and not dg.any() and not db.any()
    y, mean, rstd = dense.groupnorm_fwd(none, gamma, beta, 3, samples=0)
    assert mean.shape == (0, 3)


def test_groupnorm_constant_maps():
    """No spread at all: h is zero, rstd eps^-1/2."""
    x = torch.full((300, 12), 7.25, device="cuda")
    gamma, beta = _rand((12,), F32, 1), _rand((12,), F32, 2)
    y, mean, rstd = dense.groupnorm_fwd(x, gamma, beta, 4, samples=3, eps=1e-6)
    assert torch.equal(mean, torch.full_like(mean, 7.25)) and torch.allclose(rstd, torch.full_like(rstd, 1e3), rtol=1e-6)
    assert torch.equal(y, beta.expand(300, 12))


def test_groupnorm_nan_stays_in_its_group():
    x, gamma, beta = _norm_case(3, 400, 24, 4, F32, 7)
    x[450, 7] = math.nan   # map 1, group 1
    x[820, 23] = math.inf  # map 2, group 3
    y, mean, rstd = dense.groupnorm_fwd(x, gamma, beta, 4, 3, "silu")
    bad = torch.isnan(y.view(3, 400, 4, 6)).any(3).any(1)
    want = torch.zeros((3, 4), dtype=torch.bool, device="cuda")
    want[1, 1] = want[2, 3] = True
    assert torch.equal(bad, want) and torch.equal(torch.isnan(rstd), want)


def test_groupnorm_gradient_against_differences():
    """The 64-bit formulas that the kernels are held to, against central differences of the forward formula."""
    samples, rows, width, groups, eps = 2, 5, 6, 2, 1e-5
    x, gamma, beta = (t.double() for t in _norm_case(samples, rows, width, groups, F32, 8))
    dy = _rand(x.shape, F32, 60).double()

    def loss(x, gamma, beta, act):
        X = x.view(samples, rows, groups, -1)
        mu = X.mean((1, 3), keepdim=True)
        r = ((X - mu).square().mean((1, 3), keepdim=True) + eps) ** -0.5
        z = (X - mu) * r * gamma.view(groups, -1) + beta.view(groups, -1)
        return (_act(z, act).reshape(x.shape) * dy).sum()

    X = x.view(samples, rows, groups, -1)
    mean = X.mean((1, 3))
    rstd = ((X - mean[:, None, :, None]).square().mean((1, 3)) + eps) ** -0.5
    ROUND[torch.float64] = 0.0
    try:
        for act in ACTS:
            want = _norm_grads(samples, groups, dy, x, gamma, beta, mean, rstd, act, None)
            for name, t in (("dx", x), ("dgamma", gamma), ("dbeta", beta)):
                for i in range(0, t.numel(), 3):
                    d = torch.zeros_like(t).view(-1)
                    d[i] = 1e-6
                    d = d.view(t.shape)
                    args = {"dx": (x, gamma, beta), "dgamma": (x, gamma, beta), "dbeta": (x, gamma, beta)}[name]
                    up = [a + d if a is t else a for a in args]
                    down = [a - d if a is t else a for a in args]
                    slope = (loss(*up, act) - loss(*down, act)) / 2e-6
                    # differences: 1e-12 of the loss's curvature, 1e-16 of the loss over 1e-6
                    assert abs(slope - want[name][0].reshape(-1)[i]) <= 1e-7, (act, name, i)
    finally:
        del ROUND[torch.float64]


# ------------------------------------------------------------------ AdamW
BETAS, EPS = (0.9, 0.999), 1e-8


def _tensors(sizes, grad_type, seed, shift=0, bits=32):
    """Parameters, gradients and moments, each `shift` values off an allocation."""
    def one(n, dtype, seed, std, positive=False):
        t = _rand((n,), F32, seed, std)
        t = (t.abs() if positive else t)
        if dtype == F8:
            t = (t * 100).clamp(-448, 448)
            raw = torch.zeros(n + shift, dtype=torch.uint8, device="cuda")
            raw[shift:] = (t.clamp(min=2.0 ** -9) if positive else t).to(F8).view(torch.uint8)
            return raw.view(F8)[shift:]
        out = torch.zeros(n + shift, dtype=dtype, device="cuda")[shift:]
        out.copy_(t)
        return out

    p = [one(n, F32, seed + i, 0.5) for i, n in enumerate(sizes)]
    g = [one(n, grad_type, seed + 100 + i, 1e-3) for i, n in enumerate(sizes)]
    if bits == 32:
        m = [one(n, F32, seed + 200 + i, 1e-3) for i, n in enumerate(sizes)]
        v = [one(n, F32, seed + 300 + i, 1e-6, True) for i, n in enumerate(sizes)]
        return p, g, m, v, None
    m, v = ([one(n, F8, seed + k + i, 1.0, k == 300) for i, n in enumerate(sizes)] for k in (200, 300))
    scales = tuple([_rand(((n + 255) // 256,), F32, seed + k + i, 1e-6).abs() + 1e-7 for i, n in enumerate(sizes)]
                   for k in (400, 500))
    return p, g, m, v, scales


def _decode(q, scale):
    return q.double() * scale.double().repeat_interleave(256)[:q.numel()]


def _adamw_64(p, g, m, v, t, lr, wd):
    """New values with tolerances of m, v and p; m and v are given in 64 bits."""
    b1, b2 = BETAS
    g = g.double()
    tm, tv = 4 * U * ((b1 * m).abs() + ((1 - b1) * g).abs()), 6 * U * (b2 * v + (1 - b2) * g * g)
    m, v = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    den = (v / (1 - b2 ** t)).sqrt() + EPS
    step = lr / (1 - b1 ** t) * m / den
    # the root has half of v's error, the quotient two units in the last place
    tp = lr / (1 - b1 ** t) * tm / den + 16 * U * step.abs() + 4 * U * p.double().abs() + TINY
    return p.double() * (1 - lr * wd) - step, m, v, tp, tm + TINY, tv + TINY


SIZES = [[1], [3, 0, 256], [255, 257, 4, 2048, 2049], [64 * 24, 64, 64, 64, 64 * 64, 5], [1_000_003, 17, 300_000],
         [31] * 45, [9] * 700]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{s[0]}")
@pytest.mark.parametrize("grad_type", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shift", [0, 1, 4])
def test_adamw_32_bits(sizes, grad_type, shift):
    p, g, m, v, _ = _tensors(sizes, grad_type, 1, shift)
    copies = [torch.zeros(n + shift, dtype=BF16, device="cuda")[shift:] for n in sizes] if shift != 1 else None
    lr = [1e-3 * (1 + i % 3) for i in range(len(sizes))]
    wd = [0.1 * (i % 2) for i in range(len(sizes))]
    want = [_adamw_64(*(t.clone() for t in (p[i], g[i])), m[i].double(), v[i].double(), 7, lr[i], wd[i]) for i in range(len(sizes))]
    assert dense.adamw(p, g, m, v, 7, lr, BETAS, EPS, wd, copies=copies) is None
    for i, (wp, wm, wv, tp, tm, tv) in enumerate(want):
        _close(m[i], wm, tm, f"m {i}")
        _close(v[i], wv, tv, f"v {i}")
        _close(p[i], wp, tp, f"p {i}")
        if copies:
            assert torch.equal(copies[i], p[i].to(BF16))


def _noise(count, seed, step):
    low = 0xFFFFFFFF
    h = (torch.arange(count, device="cuda") * 0x9E3779B1 + seed * 0x6A09E667 + step * 0xBB67AE85) & low
    h = ((h ^ (h >> 16)) * 0x6A09E667) & low
    h = ((h ^ (h >> 15)) * 0xBB67AE85) & low
    return h ^ (h >> 16)


def _round_at_random(x, bits16):
    """x (padded to whole runs) as codes and scales, in single precision as the header describes it."""
    x = x.view(-1, 256)
    top = x.abs().amax(1, keepdim=True)
    top = top * (top >= 2.0 ** -100)
    q = (x * torch.where(top > 0, top.reciprocal() * 448.0, top)).clamp(-448.0, 448.0)
    bits = (q.view(torch.int32) + (bits16.view(x.shape) << 4).int()) & -0x100000
    return bits.view(F32), (top * (1.0 / 448.0))[:, 0]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{s[0]}")
@pytest.mark.parametrize("grad_type", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shift", [0, 1, 4])
def test_adamw_8_bits(sizes, grad_type, shift):
    p, g, m, v, scales = _tensors(sizes, grad_type, 2, shift, 8)
    b1, b2 = BETAS
    want, codes, place = [], [], 0
    runs = sum((n + 255) // 256 for n in sizes)
    noise = _noise(runs * 256, 5, 9)
    for i, n in enumerate(sizes):
        want.append(_adamw_64(p[i].clone(), g[i], _decode(m[i], scales[0][i]), _decode(v[i], scales[1][i]).square(), 9, 2e-3, 0.05))
        # the moments' bits, in single precision
        r = (n + 255) // 256
        grow = lambda t: torch.nn.functional.pad(t.float(), (0, r * 256 - n))  # noqa: E731
        of_run = lambda t: t.repeat_interleave(256)  # noqa: E731
        mf = grow(m[i]) * of_run(scales[0][i]) * b1 + grow(g[i]) * (1 - b1)
        vf = grow(v[i]) * of_run(scales[1][i])
        vf = (vf * vf) * b2 + (grow(g[i]) * grow(g[i])) * (1 - b2)
        bits = noise[place:place + r * 256]
        root = torch.sqrt(vf)
        q, ms = _round_at_random(mf, bits & 0xFFFF)
        s, vs = _round_at_random(root, bits >> 16)
        s = torch.where((root.view(-1, 256) > 0) & (vs[:, None] > 0), s.clamp(min=2.0 ** -9), s)
        codes.append((q.reshape(-1)[:n].to(F8), s.reshape(-1)[:n].to(F8), ms, vs, mf[:n], root[:n]))
        place += r * 256
    copies = [torch.zeros(n + shift, dtype=BF16, device="cuda")[shift:] for n in sizes] if shift != 1 else None
    dense.adamw(p, g, m, v, 9, 2e-3, BETAS, EPS, 0.05, scales=scales, copies=copies, seed=5)
    for i, (wp, wm, wv, tp, tm, tv) in enumerate(want):
        _close(p[i], wp, tp, f"p {i}")
        q, s, ms, vs, mf, root = codes[i]
        assert torch.equal(scales[0][i], ms) and torch.equal(scales[1][i], vs), i
        assert torch.equal(m[i].view(torch.uint8), q.view(torch.uint8)) and torch.equal(v[i].view(torch.uint8), s.view(torch.uint8)), i
        # and against 64 bits: what is rounded is x / scale, with 2^e <= |x / scale| < 2^(e + 1): a step of four significant
        # bits there is 2^(e - 3), times the scale; below 2^-6 the type's own steps are 2^-9, of which half is added
        for got, scale, x, off in ((m[i], scales[0][i], wm, tm), (v[i], scales[1][i], wv.sqrt(), 4 * U * wv.sqrt())):
            unit = scale.double().repeat_interleave(256)[:x.numel()]
            step = unit * torch.exp2(torch.floor(torch.log2((x.abs() / unit).clamp(min=1e-300)))) / 8 * 1.001
            tol = torch.maximum(step, torch.where(x.abs() < unit * 2.0 ** -6, 1.5 * unit * 2.0 ** -9, 0.0)) + off
            _close(got.double() * unit, x, tol, f"moment {i}")
        if copies:
            assert torch.equal(copies[i], p[i].to(BF16))


def test_adamw_8_bits_rounds_without_bias_and_lets_moments_fade():
    """With zero gradients the expected root shrinks by beta2^1/2 a step, though its change (5e-4) is far below half a
    step of the type (3e-2 at least).  Each step's rounding is off by at most half a step's width in standard deviation (a
    sixteenth of the value), independently: over N values and k steps the mean is off by sqrt(k / N) / 16 of the root mean
    square at one standard deviation; six of them are allowed."""
    n, steps = 1 << 20, 200
    p, g = [torch.zeros(n, device="cuda")], [_rand((n,), F32, 3)]
    m, v, scales = dense.adamw_state(p, bits=8)
    dense.adamw(p, g, m, v, 1, 0.0, BETAS, EPS, 0.0, scales=scales)
    m0, v0 = _decode(m[0], scales[0][0]), _decode(v[0], scales[1][0])
    exact = g[0].double().abs() * (1 - BETAS[1]) ** 0.5
    rms = exact.square().mean().sqrt()
    # (the first rounding, by itself: a 32nd of its value's bias would show)
    assert abs(v0.mean() - exact.mean()) <= 6 / 16 / math.sqrt(n) * rms + 2.0 ** -10 * scales[1][0].double().mean()
    assert abs((m0 - (1 - BETAS[0]) * g[0].double()).mean()) <= 6 / 16 / math.sqrt(n) * 0.1
    g[0].zero_()
    for t in range(steps):
        dense.adamw(p, g, m, v, 2 + t, 0.0, BETAS, EPS, 0.0, scales=scales)
    faded = _decode(v[0], scales[1][0])
    want = v0.mean() * BETAS[1] ** (steps / 2)
    # (values below 2^-6 of the scale round to the nearest of the type, at most 2^-10 of the scale off each step: they are
    # one in 10^4 of these)
    assert abs(faded.mean() - want) <= 6 * math.sqrt(steps / n) / 16 * rms + 1e-4 * rms
    assert (faded > 0)[v0 > 0].all()


def test_adamw_state_starts_at_zero():
    p, g = [torch.zeros(1000, device="cuda"), torch.zeros((7, 5), device="cuda")], [_rand((1000,), F32, 1), _rand((7, 5), F32, 2)]
    after = []
    for bits in (32, 8):
        q = [t.clone() for t in p]
        m, v, scales = dense.adamw_state(q, bits)
        assert m[1].shape == (7, 5) and m[0].dtype == (F32 if bits == 32 else F8)
        dense.adamw(q, g, m, v, 1, 1e-2, weight_decay=0.0, scales=scales)
        after.append(q)
    # the first step moves every value by lr (eps is 1e-5 of the smallest root here)
    for a, b, d in zip(*after, g):
        assert torch.equal(a, b)
        assert torch.allclose(a, -1e-2 * d.sign(), rtol=1e-4)
    with pytest.raises(ValueError, match="bits"):
        dense.adamw_state(p, 4)


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_nan_and_tiny_values(bits):
    """A NaN gradient stays in its value (its run of 256 where moments share a scale); moments that 8 bits cannot scale
    become zeros."""
    p, g, m, v, scales = _tensors([1024], F32, 4, 0, bits)
    g[0][300] = math.nan
    dense.adamw(p, g, m, v, 2, 1e-3, scales=scales)
    assert torch.isnan(p[0]).sum() == 1 and torch.isnan(p[0][300])
    bad = torch.isnan(m[0].float() * (1.0 if bits == 32 else scales[0][0].repeat_interleave(256)))
    if bits == 32:
        assert bad.sum() == 1
    else:
        assert bad[256:512].all() and bad.sum() == 256
    p, g = [torch.ones(512, device="cuda")], [torch.full((512,), 1e-38, device="cuda")]
    m, v, scales = dense.adamw_state(p, bits)
    dense.adamw(p, g, m, v, 1, 1e-3, weight_decay=0.0, scales=scales)
    assert torch.isfinite(p[0]).all() and torch.isfinite(m[0].float()).all()
    if bits == 8:
        assert not scales[0][0].any() and not m[0].float().any() and not v[0].float().any()


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_skips_by_status(bits):
    p, g, m, v, scales = _tensors([500, 70], F32, 5, 0, bits)
    everything = [*p, *[t.view(torch.uint8) for t in (*m, *v)], *(scales[0] + scales[1] if scales else [])]
    before = [t.clone() for t in everything]
    counts = torch.zeros((3, 2), dtype=torch.int64, device="cuda")
    counts[1, 1] = 4
    dense.adamw(p, g, m, v, 3, scales=scales, counts=counts)
    assert all(torch.equal(a, b) for a, b in zip(before, everything))
    counts.zero_()
    counts[:, 0] = 9  # (the first words are counts)
    dense.adamw(p, g, m, v, 3, scales=scales, counts=counts)
    assert not torch.equal(before[0], p[0])
    q, h, m2, v2, s2 = _tensors([500, 70], F32, 5, 0, bits)
    dense.adamw(q, h, m2, v2, 3, scales=s2)
    assert torch.equal(q[0], p[0]) and torch.equal(q[1], p[1])


def test_adamw_seed_and_step_decide_the_bits():
    def once(seed, step):
        p, g, m, v, scales = _tensors([5000], F32, 6, 0, 8)
        dense.adamw(p, g, m, v, step, scales=scales, seed=seed)
        return m[0].view(torch.uint8).clone()

    a = once(1, 4)
    assert torch.equal(a, once(1, 4)) and not torch.equal(a, once(2, 4)) and torch.equal(a, once(1 + (1 << 32), 4))


# ------------------------------------------------------------------ together
def _step_of_all(p, views, at, pixel, maps, want, groups, scale):
    """A head's training step: codes and normalised image features into two linear layers, a loss, every gradient.
    p: table, gamma, beta, w1, b1, w2, b2."""
    table, gamma, beta, w1, b1, w2, b2 = p
    f, mean, rstd = dense.groupnorm_fwd(maps, gamma, beta, groups, views, "silu")
    e = dense.embedding_fwd(table, at, scale)
    q = dense.embedding_fwd(f, pixel)  # the pixel's features; zeros where no view saw the Gaussian
    h, z = dense.linear_fwd(e, w1, b1, q, "gelu", keep_z=True)
    out, _ = dense.linear_fwd(h, w2, b2)
    dout = out - want  # of half the squared distance
    dh, dw2, db2 = dense.linear_bwd(dout, h, w2)
    de, dw1, db1 = dense.linear_bwd(dh, e, w1, z, "gelu")
    df = dense.embedding_bwd(dh, pixel, f.shape[0])  # the residual's gradient is dh
    dmaps, dgamma, dbeta = dense.groupnorm_bwd(df, maps, gamma, beta, mean, rstd, "silu")
    return out, [dense.embedding_bwd(de, at, table.shape[0], scale), dgamma, dbeta, dw1, db1, dw2, db2], dmaps


def _step_of_all_64(p, views, at, pixel, maps, want, groups, scale):
    p = [t.double().requires_grad_() for t in p]
    maps = maps.double().requires_grad_()
    table, gamma, beta, w1, b1, w2, b2 = p
    x = maps.view(views, -1, groups, maps.shape[1] // groups)
    mu = x.mean((1, 3), keepdim=True)
    h = (x - mu) * ((x - mu).square().mean((1, 3), keepdim=True) + 1e-5) ** -0.5
    f = _act(h.view(maps.shape) * gamma + beta, "silu")

    def rows(t, idx, by):
        i = idx.long()
        there = (i >= 0) & (i < t.shape[0])
        return t[torch.where(there, i, 0)] * there[:, None] * by

    e, q = rows(table, at, scale), rows(f, pixel, 1.0)
    h = _act(e @ w1.t() + b1, "gelu") + q
    out = h @ w2.t() + b2
    (0.5 * (out - want.double()).square().sum()).backward()
    return out.detach(), [t.grad for t in p], maps.grad


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("gaussians,codes,views,pixels", [(3000, 200, 5, 150), (1, 1, 1, 1), (9001, 70_000, 2, 1537)])
def test_codes_norm_layers_and_update_together(gaussians, codes, views, pixels, bits):
    width, groups, outs, scale = 32, 4, 11, 2.0
    p = [_rand((codes, width), F32, 80, 0.3), _rand((width,), F32, 81, 0.1, mean=1.0), _rand((width,), F32, 82, 0.1),
         _rand((width, width), F32, 83, 0.2), _rand((width,), F32, 84, 0.1), _rand((outs, width), F32, 85, 0.2),
         _rand((outs,), F32, 86, 0.1)]
    maps = _rand((views * pixels, width), F32, 87)
    at, pixel = _indices(gaussians, codes, "skewed", 88), _indices(gaussians, views * pixels, "gaps", 89)
    want = _rand((gaussians, outs), F32, 90)
    m, v, scales = dense.adamw_state(p, bits)
    for step in (1, 2, 3):
        out, grads, dmaps = _step_of_all(p, views, at, pixel, maps, want, groups, scale)
        out64, grads64, dmaps64 = _step_of_all_64(p, views, at, pixel, maps, want, groups, scale)
        # Each of at most ten stages is off by 2^-17 of its output's norm or less (128 roundings of 2^-24 in a row, more than
        # any of its sums takes one after the other), and hands an error on no more than four times as large.
        for got, ref in zip([out, *grads, dmaps], [out64, *grads64, dmaps64]):
            assert (got - ref).norm() <= 40 * 2.0 ** -17 * ref.norm() + TINY
        before = [t.clone() for t in p]
        state = [[_decode(t.view(-1), s).view(t.shape) for t, s in zip(x, scales[k])] if bits == 8 else [t.double() for t in x]
                 for k, x in enumerate((m, v))]
        dense.adamw(p, grads, m, v, step, 1e-2, BETAS, EPS, 0.05, scales=scales, seed=4)
        for new, old, g, m0, v0 in zip(p, before, grads, *state):
            wp, _, _, tp, _, _ = _adamw_64(old, g, m0, v0.square() if bits == 8 else v0, step, 1e-2, 0.05)
            _close(new, wp, tp, f"step {step}")


# ------------------------------------------------------------------ streams, graphs
def _everything(seed):
    """One call of each operator on inputs of its own; the inputs, and what the calls return."""
    table, idx = _rand((300, 24), F32, seed), _indices(5000, 300, "skewed", seed)
    gamma, beta = _rand((24,), F32, seed + 1, 0.1, mean=1.0), _rand((24,), F32, seed + 2)
    state = _tensors([300 * 24, 24, 24], F32, seed + 3, 0, 8)

    def calls(stream=None):
        y = dense.embedding_fwd(table, idx, 2.0, stream=stream)
        z, mean, rstd = dense.groupnorm_fwd(y, gamma, beta, 4, 5, "silu", stream=stream)
        dx, dg, db = dense.groupnorm_bwd(z, y, gamma, beta, mean, rstd, act="silu", stream=stream)
        dt = dense.embedding_bwd(dx, idx, 300, 2.0, stream=stream)
        p, _, m, v, scales = state
        dense.adamw(p, [dt.view(-1), dg, db], m, v, 5, scales=scales, stream=stream)
        return [y, z, mean, rstd, dx, dg, db, dt, *p, *[t.view(torch.uint8) for t in (*m, *v)]]

    return (table, idx, state), calls


def test_calls_on_other_streams():
    _, calls = _everything(20)
    want = [t.clone() for t in calls()]
    _, calls = _everything(20)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = calls(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    # two at once
    pairs = [_everything(20), _everything(20)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [calls(s) for (_, calls), s in zip(pairs, streams)]
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(want, g))


def _live(state):
    """The arrays that an update changes."""
    p, _, m, v, scales = state
    return [*p, *[t.view(torch.uint8) for t in (*m, *v)], *scales[0], *scales[1]]


def test_calls_in_graphs():
    """Two graphs that share a pool of memory, captured, and replayed in turn on the inputs of other seeds."""
    pool, graphs, inputs, outs = torch.cuda.graph_pool_handle(), [], [], []
    _everything(29)[1]()  # (loads the kernels)
    torch.cuda.synchronize()
    for seed in (30, 40):
        held, calls = _everything(seed)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, pool=pool):
            outs.append(calls())
        graphs.append(graph), inputs.append(held)
    for seed in (30, 50, 60):
        for graph, (table, idx, state), out in zip(graphs, inputs, outs):
            (new_table, new_idx, new_state), calls = _everything(seed)
            # (gamma and beta stay the captured seed's: the group norm's outputs are compared in the first round only)
            table.copy_(new_table), idx.copy_(new_idx)
            for a, b in zip(_live(state), _live(new_state)):
                a.copy_(b)
            want = calls()
            graph.replay()
            torch.cuda.synchronize()
            same = len(want) if seed == 30 and graph is graphs[0] else 1
            assert all(torch.equal(a, b) for a, b in zip(want[:same], out[:same]))
