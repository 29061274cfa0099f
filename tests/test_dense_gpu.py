"""The dense-layer entry points (gs_linear_*, gs_layernorm_*) against the same formulas in 64 bits.

Tolerances are derived from the arithmetic, elementwise.  With u = 2^-24 (32-bit rounding):
 - a sum of k terms whose signs vary: each of the k additions is off by at most 2u of the partial sum,
   which grows as sqrt(k): (8 + 2 sqrt(k)) u times the sum of the terms' absolute values covers it, even
   where every addition rounds the same way;
 - the type's own rounding of a stored value: v = 2^-8 (bfloat16: 8 significant bits, half a unit of the last) or 2^-24 (float32) of it;
 - the activations are evaluated to a few u of their argument (their slopes are at most 1.13);
 - in bfloat16 a linear layer's dz is rounded once more where it enters the products (when there is
   an activation): v times the products' absolute values.
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

from gaussian_splatting_gb300 import _native as N  # noqa: E402
from gaussian_splatting_gb300 import dense  # noqa: E402

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16
ROUND = {F32: 2.0 ** -24, BF16: 2.0 ** -8}
ACTS = ["none", "relu", "gelu", "silu"]


def _sum_u(k):
    return (8 + 2 * math.sqrt(k)) * U


def _rand(shape, dtype, seed, std=1.0, pad=0, shift=0):
    """A normal matrix or vector; `pad` extra elements between rows, `shift` elements off the allocation."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    v = (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)
    if not pad and not shift:
        return v
    if len(shape) == 1:
        out = torch.zeros(shape[0] + shift, dtype=dtype, device="cuda")[shift:]
    else:
        out = torch.zeros(shape[0] * (shape[1] + pad) + shift, dtype=dtype, device="cuda")[shift:].view(
            shape[0], shape[1] + pad)[:, :shape[1]]
    out.copy_(v)
    return out


def _twin(t):
    """A copy with the same strides and alignment (another layout may sum in another order)."""
    return torch.empty(0, dtype=t.dtype, device=t.device).set_(t.untyped_storage().clone(), t.storage_offset(), t.size(),
                                                               t.stride())


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


def _close(got, want, tol, what):
    off = (got.double() - want).abs()
    assert torch.isfinite(got.double()).all(), f"{what}: not finite"
    worst = (off - tol).max().item() if off.numel() else -1.0
    assert worst <= 0, f"{what}: {int((off > tol).sum())} of {off.numel()} out, worst ratio {(off / tol).max().item():.3g}"


def _linear_tolerances(x, w, b, r, act):
    X, W = x.double(), w.double()
    z = X @ W.T
    mag = X.abs() @ W.abs().T
    if b is not None:
        z = z + b.double()
        mag = mag + b.double().abs()
    ez = _sum_u(x.shape[1]) * mag
    y = _act(z, act)
    ey = 1.13 * ez + 8 * U * z.abs() + 4 * U * y.abs()
    if r is not None:
        ey = ey + 2 * U * (y.abs() + r.double().abs())
        y = y + r.double()
    v = ROUND[x.dtype]
    tiny = 2.0 ** -126
    return y, ey + 1.01 * v * y.abs() + tiny, z, ez + 1.01 * v * z.abs() + tiny


# rows, in, out: one of everything, widths around the tiles' edges, odd ones, a long reduction, few
# rows with many features (split reductions), many rows with few
SHAPES = [(1, 1, 1), (1, 8, 8), (1, 64, 64), (2, 1024, 512), (3, 5, 7), (16, 32, 128), (17, 4096, 40), (64, 64, 1),
          (127, 129, 65), (128, 64, 256), (129, 256, 59), (300, 45, 3), (1000, 1, 33), (257, 1100, 17), (2048, 64, 64),
          (77, 513, 300), (640, 256, 264), (5000, 128, 128), (1111, 72, 520)]


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_linear_forward(shape, dtype):
    rows, n_in, n_out = shape
    k = SHAPES.index(shape)
    for i, act in enumerate(ACTS):
        has_b, has_r, keep = (k + i) % 3 != 0, (k + i) % 2 == 0, (k + i) % 4 != 1
        x, w = _rand((rows, n_in), dtype, 1), _rand((n_out, n_in), dtype, 2, 1 / math.sqrt(n_in))
        b = _rand((n_out,), dtype, 3, 0.3) if has_b else None
        r = _rand((rows, n_out), dtype, 4) if has_r else None
        y, z = dense.linear_fwd(x, w, b, r, act=act, keep_z=keep)
        Y, ey, Z, ez = _linear_tolerances(x, w, b, r, act)
        _close(y, Y, ey, f"y {act} bias={has_b} residual={has_r}")
        assert (z is not None) == keep
        if keep:
            _close(z, Z, ez, f"z {act}")


def _linear_grads(dy, x, w, z, act):
    DY, X, W = dy.double(), x.double(), w.double()
    if act == "none":
        s, d = torch.ones_like(DY), DY
    else:
        s = _slope(z.double(), act)
        d = DY * s
    v = ROUND[dy.dtype]
    ed = 0 * d if act == "none" else 16 * U * (DY * (1 + z.double().abs())).abs()  # the slope's evaluation
    ein = ed + (1.01 * v * d.abs() if act != "none" and dy.dtype == BF16 else 0)
    tiny = 2.0 ** -126
    out = {}
    out["dx"] = (d @ W, ein @ W.abs() + _sum_u(dy.shape[1]) * (d.abs() @ W.abs()))
    out["dw"] = (d.T @ X, ein.T @ X.abs() + _sum_u(dy.shape[0]) * (d.abs().T @ X.abs()))
    out["db"] = (d.sum(0), ed.sum(0) + _sum_u(dy.shape[0]) * d.abs().sum(0))
    return {k: (g, e + 1.01 * v * g.abs() + tiny) for k, (g, e) in out.items()}


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_linear_backward(shape, dtype):
    rows, n_in, n_out = shape
    for act in ACTS:
        dy, x = _rand((rows, n_out), dtype, 5, 1e-3), _rand((rows, n_in), dtype, 6)
        w = _rand((n_out, n_in), dtype, 7, 1 / math.sqrt(n_in))
        z = None if act == "none" else _rand((rows, n_out), dtype, 8)
        dx, dw, db = dense.linear_bwd(dy, x, w, z, act=act)
        want = _linear_grads(dy, x, w, z, act)
        _close(dx, *want["dx"], f"dx {act}")
        _close(dw, *want["dw"], f"dw {act}")
        _close(db, *want["db"], f"db {act}")


# a few rows (odd numbers of them, one, the most that count as few, one more), long and short sums, any width
FEW = [(1, 7, 9), (7, 2048, 96), (8, 40, 1000), (15, 1023, 77), (16, 4096, 256), (9, 300, 2050), (17, 96, 64), (33, 64, 64),
       (500, 60, 64), (3000, 33, 17), (700, 200, 130), (40_000, 64, 64)]


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", FEW, ids=str)
def test_linear_small_calls(shape, dtype):
    rows, n_in, n_out = shape
    for act, has_r, keep, pad in (("gelu", True, True, 0), ("none", False, False, 3), ("silu", True, False, 8)):
        x, w = _rand((rows, n_in), dtype, 1, 1.0, pad), _rand((n_out, n_in), dtype, 2, 1 / math.sqrt(n_in), pad)
        b, r = _rand((n_out,), dtype, 3, 0.3), _rand((rows, n_out), dtype, 4, 1.0, pad) if has_r else None
        y, z = dense.linear_fwd(x, w, b, r, act=act, keep_z=keep)
        Y, ey, Z, ez = _linear_tolerances(x, w, b, r, act)
        _close(y, Y, ey, f"y {act}")
        if keep:
            _close(z, Z, ez, f"z {act}")
        dy = _rand((rows, n_out), dtype, 5, 1e-3, pad)
        z = None if act == "none" else _rand((rows, n_out), dtype, 8, 1.0, pad)
        full = dense.linear_bwd(dy, x, w, z, act=act)
        want = _linear_grads(dy, x, w, z, act)
        for k, v in zip(("dx", "dw", "db"), full):
            _close(v, *want[k], f"{k} {act}")
        for kw, kept in ((dict(need_dx=False), (1, 2)), (dict(need_dw=False), (0, 2)), (dict(bias=False), (0, 1))):
            part = dense.linear_bwd(dy, x, w, z, act=act, **kw)
            for i in range(3):
                assert (part[i] is not None) == (i in kept)
                assert i not in kept or torch.equal(part[i], full[i])


# thin layers over more rows than the small backward takes: one entry, odd widths, the widest, one wider
THIN = [(40_000, 1, 1), (33_001, 9, 5), (50_000, 16, 16), (200_000, 3, 16), (170_001, 16, 1), (40_000, 17, 4)]


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", THIN, ids=str)
def test_linear_thin_layers(shape, dtype):
    test_linear_small_calls(shape, dtype)


def test_a_backward_without_dw_does_not_read_x():
    for rows, n in ((2000, 40), (40_000, 9), (8, 24), (40_000, 72)):
        dy, w = _rand((rows, n), F32, 1), _rand((n, n), F32, 2)
        want, _, wb = dense.linear_bwd(dy, dy, w, need_dw=False)
        d = N.LinearDesc()
        d.rows, d.in_features, d.out_features, d.dtype, d.act = rows, n, n, N.GS_F32, N.GS_ACT_NONE
        d.ldx = d.ldw = d.ldy = d.lddx = d.lddw = n
        dx, db = torch.empty_like(dy), torch.empty(n, device="cuda")
        need = N.gs_linear_bwd_workspace_size(d)
        ws = torch.empty(max(1, need), dtype=torch.uint8, device="cuda")
        N.gs_linear_bwd(d, dy, None, w, None, dx, None, db, ws, need)
        torch.cuda.synchronize()
        assert torch.equal(dx, want) and torch.equal(db, wb)


# enough tiles for every kernel's persistent walk to take several, ranges of k in the weight gradient, ragged
# last tiles in each direction, widths on and off 16-byte rows
MANY = [(33_000, 136, 264), (20_011, 256, 200), (40_000, 64, 59), (25_000, 59, 61), (19_999, 520, 131), (16_500, 264, 512)]


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", MANY, ids=str)
def test_linear_with_many_rows(shape, dtype):
    rows, n_in, n_out = shape
    for act, has_r, keep in (("gelu", True, True), ("none", True, False), ("relu", False, False), ("silu", False, True)):
        x, w = _rand((rows, n_in), dtype, 1), _rand((n_out, n_in), dtype, 2, 1 / math.sqrt(n_in))
        b, r = _rand((n_out,), dtype, 3, 0.3), _rand((rows, n_out), dtype, 4) if has_r else None
        y, z = dense.linear_fwd(x, w, b, r, act=act, keep_z=keep)
        Y, ey, Z, ez = _linear_tolerances(x, w, b, r, act)
        _close(y, Y, ey, f"y {act}")
        if keep:
            _close(z, Z, ez, f"z {act}")
        dy = _rand((rows, n_out), dtype, 5, 1e-3)
        z = None if act == "none" else _rand((rows, n_out), dtype, 8)
        dx, dw, db = dense.linear_bwd(dy, x, w, z, act=act)
        want = _linear_grads(dy, x, w, z, act)
        for k, v in (("dx", dx), ("dw", dw), ("db", db)):
            _close(v, *want[k], f"{k} {act}")


# several rounds of tiles by pairs of blocks, the last one short, with columns of its tiles outside
ROUNDS = [(13_100, 520, 600), (13_100, 600, 520), (13_057, 1024, 768), (4_900, 640, 2064)]


@pytest.mark.parametrize("shape", ROUNDS, ids=str)
def test_linear_with_a_short_last_round(shape):
    test_linear_with_many_rows(shape, BF16)


# narrow layers, whose dz and dx come out of one pass: a tile, a row more, one and two buffers of dz, widths
# that end inside blocks of 64 and of 16, the widest, one column of vectors
NARROW = [(128, 256, 256), (129, 72, 8), (1, 256, 256), (20_000, 256, 256), (25_001, 8, 248), (40_000, 200, 128), (33_333, 128, 72),
          (19_500, 40, 24), (3000, 250, 256)]


@pytest.mark.parametrize("pad", [0, 8])
@pytest.mark.parametrize("shape", NARROW, ids=str)
def test_narrow_backward(shape, pad):
    rows, n_in, n_out = shape
    for act in ACTS:
        dy, x = _rand((rows, n_out), BF16, 5, 1e-3, pad), _rand((rows, n_in), BF16, 6, 1.0, pad)
        w = _rand((n_out, n_in), BF16, 7, 1 / math.sqrt(n_in), pad)
        z = None if act == "none" else _rand((rows, n_out), BF16, 8, 1.0, pad)
        out = torch.full((rows, n_in + 24), 7.0, dtype=BF16, device="cuda")
        full = dense.linear_bwd(dy, x, w, z, act=act, dx=out[:, 8:8 + n_in])
        assert (out[:, :8] == 7).all() and (out[:, 8 + n_in:] == 7).all()
        want = _linear_grads(dy, x, w, z, act)
        for k, v in zip(("dx", "dw", "db"), full):
            _close(v, *want[k], f"{k} {act}")
        for kw, kept in ((dict(need_dx=False), (1, 2)), (dict(need_dw=False), (0, 2)), (dict(bias=False), (0, 1)),
                         (dict(need_dx=False, need_dw=False), (2,))):
            part = dense.linear_bwd(dy, x, w, z, act=act, **kw)
            for i in kept:
                assert torch.equal(part[i], full[i])


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("pad,shift", [(8, 0), (24, 8), (1, 0), (3, 1), (2, 0)])
def test_linear_takes_any_stride_and_alignment_and_leaves_the_gaps(dtype, pad, shift):
    rows, n_in, n_out = 389, 136, 72
    x = _rand((rows, n_in), dtype, 1, 1.0, pad, shift)
    w = _rand((n_out, n_in), dtype, 2, 0.1, pad, shift)
    b = _rand((n_out,), dtype, 3, 0.3, 0, shift)
    r = _rand((rows, n_out), dtype, 4, 1.0, pad, shift)

    def canvas(m, n):
        full = torch.full((m * (n + pad) + shift,), 7.0, dtype=dtype, device="cuda")
        return full, full[shift:].view(m, n + pad)[:, :n]

    def gaps_kept(full, m, n):
        body = full[shift:].view(m, n + pad)
        assert (full[:shift] == 7).all() and (body[:, n:] == 7).all()

    fy, y = canvas(rows, n_out)
    fz, z = canvas(rows, n_out)
    dense.linear_fwd(x, w, b, r, act="gelu", out=y, z=z)
    Y, ey, Z, ez = _linear_tolerances(x, w, b, r, "gelu")
    _close(y, Y, ey, "y")
    _close(z, Z, ez, "z")
    gaps_kept(fy, rows, n_out)
    gaps_kept(fz, rows, n_out)
    fdx, dx = canvas(rows, n_in)
    fdw, dw = canvas(n_out, n_in)
    dy = _rand((rows, n_out), dtype, 5, 1e-2, pad, shift)
    _, _, db = dense.linear_bwd(dy, x, w, z, act="gelu", dx=dx, dw=dw)
    want = _linear_grads(dy, x, w, z, "gelu")
    for k, v in (("dx", dx), ("dw", dw), ("db", db)):
        _close(v, *want[k], k)
    gaps_kept(fdx, rows, n_in)
    gaps_kept(fdw, n_out, n_in)


def _view(m, n, ld, dtype, fill, seed=None, std=1.0):
    """(whole, view): an [m, n] view of rows of ld elements whose other elements are `fill`."""
    whole = torch.full((m, ld), fill, dtype=dtype, device="cuda")
    view = whole[:, :n]
    if seed is not None:
        view.copy_(_rand((m, n), dtype, seed, std))
    return whole, view


# widths that end inside a 16-byte unit of rows that start on one, few rows and many, every kernel
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", [(9, 61, 59), (300, 57, 62), (40_000, 59, 61), (20_000, 125, 258), (9000, 270, 35)], ids=str)
def test_what_lies_between_the_rows_is_neither_read_nor_written(shape, dtype):
    rows, n_in, n_out = shape
    up = lambda n: (n + 7) // 8 * 8 + 8  # noqa: E731
    nan = math.nan
    _, x = _view(rows, n_in, up(n_in), dtype, nan, 1)
    _, w = _view(n_out, n_in, up(n_in), dtype, nan, 2, 1 / math.sqrt(n_in))
    _, r = _view(rows, n_out, up(n_out), dtype, nan, 4)
    _, dy = _view(rows, n_out, up(n_out), dtype, nan, 5, 1e-3)
    b = _rand((n_out,), dtype, 3, 0.3)

    def kept(whole, n):
        assert (whole[:, n:] == 7).all()

    for act in ("none", "gelu"):
        wy, y = _view(rows, n_out, up(n_out), dtype, 7)
        wz, z = _view(rows, n_out, up(n_out), dtype, 7)
        dense.linear_fwd(x, w, b, r, act=act, out=y, z=z)
        Y, ey, Z, ez = _linear_tolerances(x, w, b, r, act)
        _close(y, Y, ey, "y")
        _close(z, Z, ez, "z")
        kept(wy, n_out)
        kept(wz, n_out)
        wz[:, n_out:] = nan
        wdx, dx = _view(rows, n_in, up(n_in), dtype, 7)
        wdw, dw = _view(n_out, n_in, up(n_in), dtype, 7)
        _, _, db = dense.linear_bwd(dy, x, w, z, act=act, dx=dx, dw=dw)
        want = _linear_grads(dy, x, w, z, act)
        for k, v in (("dx", dx), ("dw", dw), ("db", db)):
            _close(v, *want[k], k)
        kept(wdx, n_in)
        kept(wdw, n_in)
    gamma, beta = _rand((n_in,), dtype, 6), _rand((n_in,), dtype, 7)
    wy, y = _view(rows, n_in, up(n_in), dtype, 7)
    _, mean, rstd = dense.layernorm_fwd(x, gamma, beta, out=y)
    small, m2, r2 = dense.layernorm_fwd(x.contiguous(), gamma, beta)
    assert torch.isfinite(y.float()).all() and torch.allclose(y.float(), small.float(), rtol=2e-2, atol=2e-2)
    kept(wy, n_in)
    wdx, dx = _view(rows, n_in, up(n_in), dtype, 7)
    _, dg, db = dense.layernorm_bwd(x, x, gamma, mean, rstd, skip=x, dx=dx)
    assert all(torch.isfinite(t.float()).all() for t in (dx, dg, db))
    kept(wdx, n_in)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_linear_residual_in_place_and_partial_outputs(dtype):
    rows, n = 1500, 96
    x, w, r = _rand((rows, n), dtype, 1), _rand((n, n), dtype, 2, 0.1), _rand((rows, n), dtype, 3)
    y, _ = dense.linear_fwd(x, w, None, r, act="silu")
    h = r.clone()
    out, _ = dense.linear_fwd(x, w, None, h, act="silu", out=h)
    assert out is h and torch.equal(h, y)
    dy, z = _rand((rows, n), dtype, 4, 1e-3), _rand((rows, n), dtype, 5)
    full = dense.linear_bwd(dy, x, w, z, act="silu")
    for kw, kept in ((dict(need_dx=False), (1, 2)), (dict(need_dw=False), (0, 2)), (dict(bias=False), (0, 1)),
                     (dict(need_dx=False, need_dw=False), (2,))):
        part = dense.linear_bwd(dy, x, w, z, act="silu", **kw)
        for i in range(3):
            assert (part[i] is not None) == (i in kept)
            if i in kept:
                assert torch.equal(part[i], full[i])


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_no_rows(dtype):
    x, w = torch.empty((0, 24), dtype=dtype, device="cuda"), _rand((16, 24), dtype, 1)
    y, z = dense.linear_fwd(x, w, None, None, act="relu", keep_z=True)
    assert y.shape == (0, 16) and z.shape == (0, 16)
    wide = torch.full((16, 40), 7.0, dtype=dtype, device="cuda")
    dx, dw, db = dense.linear_bwd(y, x, w, z, act="relu", dw=wide[:, :24])
    assert dx.shape == (0, 24) and not dw.any() and not db.any() and (wide[:, 24:] == 7).all()
    y, mean, rstd = dense.layernorm_fwd(x, w[0].contiguous(), w[1].contiguous())
    assert y.shape == (0, 24) and mean.shape == (0,)
    dx, dg, db = dense.layernorm_bwd(y, x, w[0].contiguous(), mean, rstd)
    assert dx.shape == (0, 24) and not dg.any() and not db.any()


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", [(640, 256, 256), (640, 75, 35), (5, 256, 64)], ids=str)
def test_what_is_not_finite_stays_in_its_row(dtype, shape):
    """A row of x (or dy) with an infinity or a NaN makes that row of y (dx) not finite and leaves the bits of
    every other row."""
    rows, n_in, n_out = shape
    x, w = _rand((rows, n_in), dtype, 1), _rand((n_out, n_in), dtype, 2, 0.1)
    y, _ = dense.linear_fwd(x, w, act="gelu")
    bad = x.clone()
    bad[1, 3], bad[4, 0], bad[rows - 2, n_in - 1] = math.inf, math.nan, -math.inf
    yb, zb = dense.linear_fwd(bad, w, act="gelu", keep_z=True)
    hit = torch.zeros(rows, dtype=torch.bool, device="cuda")
    hit[[1, 4, rows - 2]] = True
    assert torch.equal(yb[~hit], y[~hit])
    assert not torch.isfinite(zb[hit].float()).any()
    dy = _rand((rows, n_out), dtype, 3, 1e-3)
    dx, _, _ = dense.linear_bwd(dy, x, w)
    dy[4, n_out - 1] = math.nan
    dxb, dwb, dbb = dense.linear_bwd(dy, x, w)
    keep = torch.arange(rows, device="cuda") != 4
    assert torch.equal(dxb[keep], dx[keep]) and torch.isnan(dxb[4].float()).all()
    assert torch.isnan(dwb[n_out - 1].float()).all() and torch.isfinite(dwb[:n_out - 1].float()).all()
    assert torch.isnan(dbb[n_out - 1].float()) and torch.isfinite(dbb[:n_out - 1].float()).all()


# widths: every form (part of a warp, a warp, a block, wider than its registers), odd ones
WIDTHS = [1, 2, 7, 8, 24, 64, 100, 128, 256, 257, 500, 512, 1000, 1024, 2048, 2049, 4096, 6000, 8192, 20000, 70001]


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("width", WIDTHS)
def test_layernorm_forward_and_backward(width, dtype):
    for rows, pad, shift in ((1, 0, 0), (37, 8, 0), (301, 3, 1)):
        _check_norm(rows, width, dtype, pad, shift)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows,width", [(40_000, 64), (30_001, 96), (12_345, 129), (9_000, 1024)])
def test_layernorm_with_many_rows(rows, width, dtype):
    _check_norm(rows, width, dtype, 0, 0)


def _check_norm(rows, width, dtype, pad, shift):
    eps, v = 1e-5, ROUND[dtype]
    x = _rand((rows, width), dtype, 1, 1.5, pad, shift)
    x += 2.0  # a mean that a one-pass variance would lose digits to
    gamma, beta = _rand((width,), dtype, 2, 0.3) + 1, _rand((width,), dtype, 3, 0.3)
    y, mean, rstd = dense.layernorm_fwd(x, gamma, beta, eps=eps)
    X, G, B = x.double(), gamma.double(), beta.double()
    m = X.mean(1, keepdim=True)
    var = (X - m).square().mean(1, keepdim=True)
    rs = (var + eps) ** -0.5
    h = (X - m) * rs
    su = _sum_u(width)
    em = su * X.abs().mean(1, keepdim=True)
    ers = rs * (su + 4 * U) + 0.5 * rs ** 3 * (2 * em * (X - m).abs().mean(1, keepdim=True) + em * em)  # of rstd
    eh = rs * (em + 2 * U * (X.abs() + m.abs())) + (X - m).abs() * ers
    _close(mean, m[:, 0], em[:, 0] + U * m[:, 0].abs(), "mean")
    _close(rstd, rs[:, 0], ers[:, 0], "rstd")
    Y = h * G + B
    _close(y, Y, G.abs() * eh + 4 * U * (h.abs() * G.abs() + B.abs()) + 1.01 * v * Y.abs(), "y")
    # backward, from the stored statistics
    dy, skip = _rand((rows, width), dtype, 4, 1e-3, pad, shift), _rand((rows, width), dtype, 5, 1e-3, pad, shift)
    D, M, R = dy.double(), mean.double()[:, None], rstd.double()[:, None]
    H = (X - M) * R
    eH = 4 * U * R * (X.abs() + M.abs())
    g = D * G
    s1, s2 = g.mean(1, keepdim=True), (g * H).mean(1, keepdim=True)
    es1 = (su + 2 * U) * g.abs().mean(1, keepdim=True)
    es2 = (su + 2 * U) * (g * H).abs().mean(1, keepdim=True) + (g.abs() * eH).mean(1, keepdim=True)
    dxx = R * (g - s1 - H * s2)
    edx = R * (es1 + H.abs() * es2 + eH * s2.abs() + 4 * U * (g.abs() + s1.abs() + (H * s2).abs()))
    DG, DB = (D * H).sum(0), D.sum(0)
    rsum = _sum_u(rows)
    edg = (D.abs() * eH).sum(0) + (rsum + 2 * U) * (D * H).abs().sum(0) + 1.01 * v * DG.abs()
    edb = rsum * D.abs().sum(0) + 1.01 * v * DB.abs()
    for sk in (None, skip):
        want = dxx if sk is None else dxx + skip.double()
        e = edx + 2 * U * want.abs() + (0 if sk is None else 2 * U * (skip.double().abs() + dxx.abs()))
        dx, dgamma, dbeta = dense.layernorm_bwd(dy, x, gamma, mean, rstd, skip=sk)
        _close(dx, want, e + 1.01 * v * want.abs(), "dx")
        _close(dgamma, DG, edg, "dgamma")
        _close(dbeta, DB, edb, "dbeta")
    # in place of dy, and each output alone
    own = _twin(dy)
    dx2, none, _ = dense.layernorm_bwd(own, x, gamma, mean, rstd, skip=skip, dx=own, need_dparams=False)
    assert none is None and torch.equal(dx2, dx)
    none, dg2, db2 = dense.layernorm_bwd(dy, x, gamma, mean, rstd, need_dx=False)
    assert none is None and torch.equal(dg2, dgamma) and torch.equal(db2, dbeta)
    xi = _twin(x)
    yi, _, _ = dense.layernorm_fwd(xi, gamma, beta, eps=eps, out=xi, stats=False)
    assert torch.equal(yi, y)


def test_layernorm_of_constant_and_extreme_rows():
    x = torch.zeros((6, 48), device="cuda")
    x[1] = 3.0
    x[2] = 1e18
    x[3, 5] = math.inf
    x[4, 7] = math.nan
    x[5] = torch.arange(48, device="cuda") * 1e-30
    gamma, beta = _rand((48,), F32, 1) + 1, _rand((48,), F32, 2)
    y, mean, rstd = dense.layernorm_fwd(x, gamma, beta)
    assert torch.equal(y[0], beta) and torch.allclose(y[1], beta, atol=1e-3) and rstd[0].item() == pytest.approx(1e-5 ** -0.5)
    assert mean[2].item() == pytest.approx(1e18, rel=1e-6) and torch.isfinite(y[5]).all()
    assert torch.isnan(y[3]).all() and torch.isnan(y[4]).all()


@pytest.mark.parametrize("act", ACTS)
def test_gradients_against_differences(act):
    """The directional derivative of sum(c * y), y = linear(layernorm(x)) + x, by central differences of the
    64-bit forward, against the kernels' gradients (float32).  Step 1e-5: the differences are good to about
    1e-9 of the terms, the kernels to the bounds above; 2e-5 of the sum of the terms' absolute values covers both."""
    rows, n = 53, 40
    x, gamma, beta = _rand((rows, n), F32, 1), _rand((n,), F32, 2, 0.2) + 1, _rand((n,), F32, 3, 0.2)
    w, b, c = _rand((n, n), F32, 4, 0.3), _rand((n,), F32, 5, 0.3), _rand((rows, n), F32, 6)
    h, mean, rstd = dense.layernorm_fwd(x, gamma, beta)
    y, z = dense.linear_fwd(h, w, b, x, act=act, keep_z=True)
    dh, dw, db = dense.linear_bwd(c, h, w, z, act=act)
    dx, dg, dbeta = dense.layernorm_bwd(dh, x, gamma, mean, rstd, skip=c)

    def loss(p):
        X, G, B, W, b_ = p
        m = X.mean(1, keepdim=True)
        hh = (X - m) * ((X - m).square().mean(1, keepdim=True) + 1e-5) ** -0.5 * G + B
        return ((_act(hh @ W.T + b_, act) + X) * c.double()).sum()

    p = [t.double() for t in (x, gamma, beta, w, b)]
    grads = (dx, dg, dbeta, dw, db)
    for i, g in enumerate(grads):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(100 + i)
        v = torch.randn(p[i].shape, generator=gen, device="cuda", dtype=torch.float64)
        e = 1e-5 if act != "relu" else 1e-7  # a kink within the step would show
        lo, hi = list(p), list(p)
        lo[i], hi[i] = p[i] - e * v, p[i] + e * v
        num = (loss(hi) - loss(lo)) / (2 * e)
        ours = (g.double() * v).sum()
        assert abs(num - ours) <= 2e-5 * (g.double() * v).abs().sum(), (i, float(num), float(ours))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_the_same_call_gives_the_same_bits(dtype):
    dy, x = _rand((20_000, 72), dtype, 1, 1e-3), _rand((20_000, 200), dtype, 2)
    w, z = _rand((72, 200), dtype, 3, 0.1), _rand((20_000, 72), dtype, 4)
    first = dense.linear_bwd(dy, x, w, z, act="silu")
    gamma = _rand((200,), dtype, 5)
    _, mean, rstd = dense.layernorm_fwd(x, gamma, gamma)
    n1 = dense.layernorm_bwd(x, x, gamma, mean, rstd)
    for _ in range(3):
        for a, b in zip(first, dense.linear_bwd(dy, x, w, z, act="silu")):
            assert torch.equal(a, b)
        for a, b in zip(n1, dense.layernorm_bwd(x, x, gamma, mean, rstd)):
            assert torch.equal(a, b)


def test_calls_run_on_the_stream_they_are_given():
    """Work behind a long copy on a side stream: the results are there once that stream is done, and the
    outputs' memory is not handed out early."""
    s = torch.cuda.Stream()
    big = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    x, w = _rand((5000, 64), BF16, 1), _rand((64, 64), BF16, 2, 0.1)
    want, wz = dense.linear_fwd(x, w, act="gelu", keep_z=True)
    wdx, wdw, wdb = dense.linear_bwd(want, x, w, wz, act="gelu")
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(8):
            big.add_(1)
        late = x.clone()
    for st in (s, s.cuda_stream):
        y, z = dense.linear_fwd(late, w, act="gelu", keep_z=True, stream=st)
        dx, dw, db = dense.linear_bwd(y, late, w, z, act="gelu", stream=st)
        n, mean, rstd = dense.layernorm_fwd(y, w[0], w[1], stream=st)
        dense.layernorm_bwd(y, y, w[0], mean, rstd, stream=st)
        s.synchronize()
        assert torch.equal(y, want) and torch.equal(dx, wdx) and torch.equal(dw, wdw) and torch.equal(db, wdb)


def _chain(x, w, wide, gamma, back):
    """Calls of every kind, each on what the one before it wrote, the buffers of some written again at once."""
    n, mean, rstd = dense.layernorm_fwd(x, gamma, gamma)
    y, z = dense.linear_fwd(n, w, gamma, residual=n, act="gelu", keep_z=True)
    dy, _ = dense.linear_fwd(y, wide)
    dy, _ = dense.linear_fwd(dy, back)
    dx, dw, db = dense.linear_bwd(dy, n, w, z, act="gelu")
    dense.linear_fwd(dx, w, out=dy)
    dn, dg, dbeta = dense.layernorm_bwd(dy, x, gamma, mean, rstd)
    few, _ = dense.linear_fwd(dn[:5], w, act="silu")
    small, _ = dense.linear_fwd(dn[:2000], w[:40])
    dense.linear_fwd(dn, w, out=dx)
    return y, dx, dw, db, dy, dn, dg, dbeta, few, small


@pytest.mark.parametrize("width", [64, 59])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_calls_follow_each_other_and_are_captured(dtype, width):
    """A kernel may be set up while the one before it ends: what a chain of calls returns does not depend
    on whether the host waits between them, nor on their being replayed as a graph on other inputs."""
    w, back = _rand((width, width), dtype, 1, 0.1), _rand((width, 200), dtype, 2, 0.1)
    wide, gamma = _rand((200, width), dtype, 3, 0.1), _rand((width,), dtype, 4)
    inputs = [_rand((30_001, width), dtype, 5 + i) for i in range(3)]
    x = inputs[0].clone()
    names = ["layernorm_fwd", "layernorm_bwd", "linear_fwd", "linear_bwd"]
    plain = {n: getattr(dense, n) for n in names}
    want = []
    try:
        for n in names:
            def waiting(*a, _call=plain[n], **k):
                r = _call(*a, **k)
                torch.cuda.synchronize()
                return r
            setattr(dense, n, waiting)
        for v in inputs:
            want.append(_chain(v, w, wide, gamma, back))
    finally:
        for n in names:
            setattr(dense, n, plain[n])
    for v, expect in zip(inputs, want):
        for _ in range(4):
            assert all(torch.equal(a, b) for a, b in zip(_chain(v, w, wide, gamma, back), expect))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        _chain(x, w, wide, gamma, back)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = _chain(x, w, wide, gamma, back)
    for v, expect in zip(inputs, want):
        x.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, expect))


def test_offsets_beyond_32_bits():
    """Arrays of more than 2^31 elements (rows far apart): the last rows are read and written in place."""
    rows, n, ld = 70_000, 64, 40_000
    big = torch.zeros((rows, ld), dtype=BF16, device="cuda")
    x = big[:, 128:128 + n]
    x.copy_(_rand((rows, n), BF16, 1))
    out = big[:, 256:256 + n]
    small = x.contiguous()
    w = _rand((n, n), BF16, 2, 0.1)
    y, _ = dense.linear_fwd(x, w, None, x, act="relu", out=out)
    want, _ = dense.linear_fwd(small, w, None, small, act="relu")
    assert torch.equal(y, want)
    got = dense.linear_bwd(out, x, w, out, act="relu", dx=big[:, 512:512 + n])
    for a, b in zip(got, dense.linear_bwd(want, small, w, want, act="relu")):
        assert torch.equal(a, b)
    y, m, r = dense.layernorm_fwd(x, w[0], w[1], out=out)
    want, m2, r2 = dense.layernorm_fwd(small, w[0], w[1])
    assert torch.equal(y, want) and torch.equal(m, m2)
    a = dense.layernorm_bwd(out, x, w[0], m, r, skip=x, dx=big[:, 512:512 + n])
    for p, q in zip(a, dense.layernorm_bwd(want, small, w[0], m, r, skip=small)):
        assert torch.equal(p, q)
    assert not big[:, :128].any() and not big[:, 1024:1032].any()


def test_status_stays_clear():
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    x, w = _rand((3000, 64), BF16, 1), _rand((64, 64), BF16, 2)
    y, _ = dense.linear_fwd(x, w, status=status)
    dense.linear_bwd(y, x, w, status=status)
    assert status.item() == 0


@pytest.mark.parametrize("case", ["f32", "f32 residual", "bf16", "bf16 pair", "bf16 residual", "bf16 unaligned"])
def test_a_wait_that_runs_out_sets_the_status_and_leaves_the_device_usable(case):
    """A product whose operands never arrive (a test hook): every role gives up after 2 ms, the status word says
    so, and the next call is right."""
    dtype = F32 if case.startswith("f32") else BF16
    rows, n_in, n_out = (20_000, 1024, 512) if "pair" in case else (3000, 304 if "unaligned" not in case else 301, 136)
    x, w = _rand((rows, n_in), dtype, 1), _rand((n_out, n_in), dtype, 2, 0.05)
    r = _rand((rows, n_out), dtype, 3) if "residual" in case else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want, _ = dense.linear_fwd(x, w, None, r, status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    lib = N.load()
    try:
        lib.gs_debug_set_wait_limit(2000)
        lib.gs_debug_drop_publish(3)
        dense.linear_fwd(x, w, None, r, status=status)
        torch.cuda.synchronize()
    finally:
        lib.gs_debug_set_wait_limit(0)
        lib.gs_debug_drop_publish(0)
    assert status.item() == 2
    status.zero_()
    y, _ = dense.linear_fwd(x, w, None, r, status=status)
    assert status.item() == 0 and torch.equal(y, want)


@pytest.mark.parametrize("width", [256, 40])
def test_a_wait_that_runs_out_in_a_narrow_backward(width):
    """The same for the pass that forms dz: w never arrives, dz and dx wait for it in vain."""
    x, w = _rand((60_000, width), BF16, 1), _rand((width, width), BF16, 2, 0.05)
    z, status = _rand((60_000, width), BF16, 3), torch.zeros(1, dtype=torch.int32, device="cuda")
    want = dense.linear_bwd(x, x, w, z, act="gelu", status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    lib = N.load()
    try:
        lib.gs_debug_set_wait_limit(2000)
        lib.gs_debug_drop_publish(3)
        dense.linear_bwd(x, x, w, z, act="gelu", status=status)
        torch.cuda.synchronize()
    finally:
        lib.gs_debug_set_wait_limit(0)
        lib.gs_debug_drop_publish(0)
    assert status.item() == 2
    status.zero_()
    for a, b in zip(dense.linear_bwd(x, x, w, z, act="gelu", status=status), want):
        assert torch.equal(a, b)
    assert status.item() == 0


# rows of 59 columns without gaps, which the two warps of a quadrant write together: few tiles, and enough of them for
# the weights to stay in shared memory
@pytest.mark.parametrize("rows", [20_000, 60_000])
@pytest.mark.parametrize("with_r,keep_z", [(True, False), (False, True), (True, True)])
def test_a_wait_that_runs_out_where_warps_write_rows_together(rows, with_r, keep_z):
    """Warps that meet at a barrier of their own agree on whether a wait ran out: no one is left waiting there."""
    x, w = _rand((rows, 128), F32, 1), _rand((59, 128), F32, 2, 0.1)
    r = _rand((rows, 59), F32, 3) if with_r else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want, wz = dense.linear_fwd(x, w, None, r, act="gelu", keep_z=keep_z, status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    lib = N.load()
    try:
        lib.gs_debug_set_wait_limit(2000)
        lib.gs_debug_drop_publish(3)
        dense.linear_fwd(x, w, None, r, act="gelu", keep_z=keep_z, status=status)
        torch.cuda.synchronize()
    finally:
        lib.gs_debug_set_wait_limit(0)
        lib.gs_debug_drop_publish(0)
    assert status.item() == 2
    status.zero_()
    y, z = dense.linear_fwd(x, w, None, r, act="gelu", keep_z=keep_z, status=status)
    assert status.item() == 0 and torch.equal(y, want) and (not keep_z or torch.equal(z, wz))


# bfloat16 off 16-byte rows: widths that end inside the first 32 columns of a warp's share of a tile, in it and at its end;
# rows that end inside a warp's
@pytest.mark.parametrize("shape", [(40_001, 59, 131), (40_010, 61, 97), (20_031, 73, 257), (39_999, 65, 160), (700, 130, 65)], ids=str)
def test_unaligned_widths_that_end_inside_a_warps_columns(shape):
    test_linear_with_many_rows(shape, BF16)


# a product for every float32 kernel: few rows, tiles of 64 columns and of 128, operands by TMA and by words, whole rows
# written together, ranges of k
LIMITS = [(12, 40, 33), (640, 40, 33), (700, 300, 59), (20_000, 128, 200), (40_000, 128, 59), (9000, 270, 35), (200, 4096, 40),
          (2000, 520, 264)]


@pytest.mark.parametrize("shape", LIMITS, ids=str)
def test_float32_infinities_and_the_largest_values_give_the_definitions(shape):
    """Sums with an infinity are that infinity (or NaN: against a zero weight or the other infinity), the largest
    finite values give finite sums, and all other rows keep their bits, whichever kernel takes the call."""
    rows, n_in, n_out = shape
    big = torch.finfo(F32).max
    x, w = _rand((rows, n_in), F32, 1), _rand((n_out, n_in), F32, 2, 0.1)
    w.clamp_(-0.45, 0.45)  # twice the largest value by a weight stays in range
    w[1, 3] = 0.0
    _, clean = dense.linear_fwd(x, w, keep_z=True)
    bad = x.clone()
    bad[0, 3], bad[1, 3], bad[2, 3] = math.inf, -math.inf, math.nan
    bad[3, 3], bad[3, 5] = math.inf, -math.inf
    bad[4, 3], bad[5, 3], bad[6, 3] = big, -big, 3.4e38
    bad[7, 3], bad[7, 5] = big, -big
    bad[rows - 1, n_in - 1] = -big
    hit = torch.zeros(rows, dtype=torch.bool, device="cuda")
    hit[:8] = hit[rows - 1] = True
    _, ey, Z, ez = _linear_tolerances(bad, w, None, None, "none")
    for act in ("none", "relu"):
        y, z = dense.linear_fwd(bad, w, act=act, keep_z=True)
        Y = Z if act == "none" else Z.clamp(min=0)  # (a NaN stays NaN)
        for got, want, what in ((z, Z, "z"), (y, Y, "y")):
            finite = torch.isfinite(want)
            assert torch.equal(torch.isnan(got), torch.isnan(want)), what
            assert torch.equal(got[~finite & ~torch.isnan(want)].double(), want[~finite & ~torch.isnan(want)]), what
            _close(got[finite], want[finite], ez[finite], what)
        assert torch.equal(z[~hit], clean[~hit])
    alone, _ = dense.linear_fwd(bad, w)  # without z
    finite = torch.isfinite(Z)
    assert torch.equal(torch.isnan(alone), torch.isnan(Z))
    _close(alone[finite], Z[finite], ez[finite], "y alone")
    # and the gradients
    dy = _rand((rows, n_out), F32, 3, 1e-3)
    good = dense.linear_bwd(dy, x, w)
    dy[0, 1], dy[4, 2], dy[5, 0], dy[rows - 1, n_out - 1] = math.inf, big, -big, math.nan
    x.clamp_(-0.9, 0.9)
    want = _linear_grads(dy, x, w, None, "none")
    for got, (g, e), what in zip(dense.linear_bwd(dy, x, w), (want["dx"], want["dw"], want["db"]), ("dx", "dw", "db")):
        finite = torch.isfinite(g)
        assert torch.equal(torch.isnan(got), torch.isnan(g)), what
        assert torch.equal(got[~finite & ~torch.isnan(g)].double(), g[~finite & ~torch.isnan(g)]), what
        _close(got[finite], g[finite], e[finite], what)
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[[0, 4, 5, rows - 1]] = False
    assert torch.equal(dense.linear_bwd(dy, x, w)[0][keep], good[0][keep])


# narrow layers whose dx or w TMA cannot move, aligned ones, thin ones, others; dx into rows at odd distances
ALONE = [(3000, 250, 256), (40_000, 252, 64), (30_000, 20, 40), (5000, 72, 72), (40_000, 8, 16), (40_000, 16, 8), (40_000, 9, 5),
         (2000, 40, 24), (9000, 300, 264)]


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", ALONE, ids=str)
def test_the_bias_gradient_does_not_depend_on_the_other_outputs(shape, dtype):
    """Columns of dy that add up to almost nothing: another order of the sum would show even in bfloat16."""
    rows, n_in, n_out = shape
    half = _rand((rows // 2, n_out), dtype, 1)
    perm = torch.randperm(rows // 2, generator=torch.Generator().manual_seed(2)).cuda()
    dy = torch.cat([half, -half[perm]])
    x, w = _rand((rows, n_in), dtype, 3), _rand((n_out, n_in), dtype, 4, 0.1)
    strided = torch.zeros((rows, n_in + 1), dtype=dtype, device="cuda")[:, :n_in]
    for act in ("none", "relu"):
        z = None if act == "none" else torch.ones_like(dy)  # slope 1
        dx, dw, db = dense.linear_bwd(dy, x, w, z, act=act)
        for kw in (dict(need_dx=False), dict(need_dw=False), dict(need_dx=False, need_dw=False), dict(dx=strided)):
            other = dense.linear_bwd(dy, x, w, z, act=act, **kw)
            assert torch.equal(other[2], db), (act, kw.keys())
            assert other[1] is None or torch.equal(other[1], dw)
            assert "dx" in kw or other[0] is None or torch.equal(other[0], dx)
        assert torch.equal(strided, dx) or dtype == BF16  # (another kernel: the last bit)


# one more row than the few-rows kernels take and up to many, widths of one column to several tiles, thin layers
SMALL = [(17, 1, 1), (17, 256, 300), (40, 3, 5), (64, 64, 3), (333, 8, 8), (1000, 65, 129), (2048, 128, 128), (5000, 16, 9), (30_000, 64, 3),
         (100_000, 8, 1), (25, 200, 4100)]


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", SMALL, ids=str)
def test_small_forward_products(shape, dtype):
    rows, n_in, n_out = shape
    for act, has_r, keep, pad in (("gelu", True, True, 0), ("none", False, False, 5), ("relu", True, False, 8)):
        x, w = _rand((rows, n_in), dtype, 1, 1.0, pad), _rand((n_out, n_in), dtype, 2, 1 / math.sqrt(n_in), pad)
        b, r = _rand((n_out,), dtype, 3, 0.3), _rand((rows, n_out), dtype, 4, 1.0, pad) if has_r else None
        y, z = dense.linear_fwd(x, w, b, r, act=act, keep_z=keep)
        Y, ey, Z, ez = _linear_tolerances(x, w, b, r, act)
        _close(y, Y, ey, f"y {act}")
        if keep:
            _close(z, Z, ez, f"z {act}")


# calls at either side of the forward's choice of a kernel: rows, inputs, columns and blocks that just fit, and do not
EDGES = [(1, 4096, 33), (1, 4104, 33), (1, 8192, 70), (2, 1024, 64), (3, 1024, 64), (8, 256, 300), (8, 520, 40), (128, 256, 256), (136, 256, 256),
         (512, 64, 64), (520, 64, 64), (1024, 32, 128), (4, 255, 257), (512, 9, 5), (4900, 9, 5), (8, 2048, 8200), (9, 2048, 8200),
         (64, 60, 64), (16, 8, 16), (16, 1024, 1024), (5, 4096, 4096)]


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", EDGES, ids=str)
def test_forward_products_of_few_rows(shape, dtype):
    test_small_forward_products(shape, dtype)


# backwards of few rows at either side of their choice of kernels
FEW_BACK = [(1, 4096, 4096), (2, 1000, 4100), (8, 4100, 1030), (16, 520, 512), (16, 256, 256), (16, 264, 264), (9, 4096, 900), (4, 1024, 1024),
            (5, 2000, 1024), (1, 8200, 2048), (2, 8200, 64), (16, 1024, 8), (16, 1032, 8), (1, 16400, 40), (1, 64, 8200), (3, 255, 1400)]


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", FEW_BACK, ids=str)
def test_backwards_of_few_rows(shape, dtype):
    rows, n_in, n_out = shape
    for act, pad in (("none", 0), ("gelu", 8), ("silu", 3)):
        dy, x = _rand((rows, n_out), dtype, 5, 1e-3, pad), _rand((rows, n_in), dtype, 6, 1.0, pad)
        w = _rand((n_out, n_in), dtype, 7, 1 / math.sqrt(n_in), pad)
        z = None if act == "none" else _rand((rows, n_out), dtype, 8, 1.0, pad)
        full = dense.linear_bwd(dy, x, w, z, act=act)
        want = _linear_grads(dy, x, w, z, act)
        for k, v in zip(("dx", "dw", "db"), full):
            _close(v, *want[k], f"{k} {act}")
        for kw, kept in ((dict(need_dx=False), (1, 2)), (dict(need_dw=False), (0, 2)), (dict(bias=False), (0, 1))):
            part = dense.linear_bwd(dy, x, w, z, act=act, **kw)
            assert all(torch.equal(part[i], full[i]) for i in kept)


# narrow backwards at either side of their choice of kernels: the last row of one round of tiles and the next, the widest
# thin layers, one wider
NARROW_BACK = [(17, 16, 16), (4864, 64, 64), (4865, 64, 64), (4865, 16, 16), (4864, 9, 5), (4865, 9, 5), (32_000, 16, 16), (40_000, 8, 8),
               (9000, 3, 16), (9000, 17, 16), (9000, 16, 17), (6000, 64, 3), (5000, 1, 1)]


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", NARROW_BACK, ids=str)
def test_narrow_backwards_at_the_limits_of_their_kernels(shape, dtype):
    test_linear_small_calls(shape, dtype)
