"""Code lookup, group norm and AdamW where their arithmetic is at its ends, past 2^31 elements, and in graphs that are replayed
on inputs of their own.

u = 2^-24 (a 32-bit rounding); what each tolerance counts stands at its test.
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
sys.path.insert(0, os.path.join(ROOT, "tests"))

from gaussian_splatting_gb300 import dense  # noqa: E402
from gaussian_splatting_gb300._native import GSError  # noqa: E402
from test_learned_gpu import (BF16, CHAIN, F32, ROUND, TINY, U, _check_norm_fwd, _close, _gen, _gradient, _indices,  # noqa: E402
                              _norm_case, _norm_grads, _rand, _sum_u, _tensors)

pytestmark = pytest.mark.gpu
both = pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
# rows of a map: a block holds a group, or two passes do; rows on 16 bytes, or one value a thread
forms = pytest.mark.parametrize("rows", [50, 20_011], ids=["one-kernel", "two-passes"])
vectors = pytest.mark.parametrize("pad,shift", [(0, 0), (2, 2), (1, 1)], ids=["whole", "pairs", "single"])


# ------------------------------------------------------------------ code lookup
# codes that have rows, out of n: buckets of little more rows than a block takes at once, of many times as many, some of either
FULL = [(1_600_000, 1_000_000, 204_800, 32), (1_600_000, 1_000_000, 204_800, 9), (1_700_000, 1 << 22, 600_000, 12),
        (1_700_000, 1 << 22, 400_000, 20), (26_000_000, 1_000_000, 1_000_000, 8), (2_000_000, 1_000_000, 3, 64),
        (12_000_000, 2000, 2000, 40), (8_000_000, 300, 280, 40)]


@both
@pytest.mark.parametrize("case", FULL, ids=str)
def test_embedding_buckets_of_more_parts_than_places(case, dtype):
    """Parts' sums have places for a part of each bucket and a few more: with indices that make most buckets take two, or few
    buckets hundreds, blocks take several runs of rows in turn."""
    rows, n, used, width = case
    idx = (torch.rand(rows, generator=_gen(5), device="cuda", dtype=torch.float64) * used).int().clamp(max=used - 1)
    idx[::1000] = n - 1 - idx[::1000]
    idx[7::5003] = -1
    dy = _rand((rows, width), dtype, 6, 1e-3)
    got = dense.embedding_bwd(dy, idx, n, -2.0, dtable=torch.ones((n, width), dtype=dtype, device="cuda"))
    want, mag, counts = _gradient(dy, idx, n, -2.0)
    _close(got, want, (8 + 2 * counts.double().sqrt())[:, None] * U * mag + 1.01 * ROUND[dtype] * want.abs() + TINY, "dtable")
    assert not got[counts == 0].any()
    assert torch.equal(dense.embedding_bwd(dy, idx, n, -2.0), got)


# ------------------------------------------------------------------ group norm
# next to each other: z at every distance below zero
FAR = [-1e4, 0.5, -1e18, -1e38, -50.0, -1e4, 2.0, -1e30, -45.0, -41.0, -1e20, -43.0, 0.0, -80.0, -1e38, -1e38]


@both
@forms
@vectors
def test_groupnorm_silu_far_below_zero(rows, pad, shift, dtype):
    """z / (1 + exp(-z)) and its slope vanish with exp(z).  Forward, at -110 and below both are less than 2^-126; above, z is
    off by ez (its two roundings, and those of h), the exponential's argument by 4 u |z| more, so that the value is off by
    twice their sum relative to itself, and below -87, where 1 / (1 + exp(-z)) is flushed to zero, by 2^-126 |z|.  Backward, such channels' gradients are those of a channel at -200."""
    samples, groups, width = 2, 4, len(FAR)
    x, gamma, _ = _norm_case(samples, rows, width, groups, dtype, 3, pad, shift)
    beta = _rand((width,), dtype, 4, 0.0, 0, shift)
    beta.copy_(torch.tensor(FAR))
    y, mean, rstd = dense.groupnorm_fwd(x, gamma, beta, groups, samples, "silu")
    X = x.double().reshape(samples, rows, groups, -1)
    G, B = gamma.double().view(groups, -1), beta.double().view(groups, -1)
    h = (X - mean.double()[:, None, :, None]) * rstd.double()[:, None, :, None]
    z = h * G + B
    want = (z * torch.sigmoid(z)).reshape(-1, width)
    emu = U * (mean.double().abs() + 8)[:, None, :, None]  # what the block's own mean and rstd may differ by
    ez = 4 * U * ((h * G).abs() + B.abs()) + (emu + 8 * U * h.abs()) * G.abs() * rstd.double()[:, None, :, None].clamp(min=1)
    z, ez = z.reshape(-1, width), ez.reshape(-1, width)
    near = z > -110
    tol = torch.where(near, 2 * (ez + 4 * U * z.abs()) * want.abs() + 1.13 * ez * (z > -20) + 1.01 * ROUND[dtype] * want.abs() + 128 * TINY, 0.0)
    _close(y, want, tol + TINY, "y")
    dy = _rand(x.shape, dtype, 5, 1e-3, pad, shift)
    got = dense.groupnorm_bwd(dy, x, gamma, beta, mean, rstd, act="silu")
    there = torch.where(beta < -110, -200.0, beta.double())
    grads = _norm_grads(samples, groups, dy, x, gamma, there, mean, rstd, "silu", None)
    for name, v in zip(("dx", "dgamma", "dbeta"), got):
        _close(v, *grads[name], name)
    gone = beta < -110
    assert (got[1][gone].abs() <= TINY).all() and (got[2][gone].abs() <= TINY).all()


@both
@forms
@vectors
def test_groupnorm_silu_infinities_and_nan_stay_in_their_channel(rows, pad, shift, dtype):
    """Others keep their values.  Two that share a reciprocal do so by the rounded product (u) of their denominators, its
    reciprocal (2 u) and two more products (2 u): with another neighbour the result may change by 10 u, and by two roundings
    of the type."""
    samples, groups, width = 2, 2, 16
    x, gamma, beta = _norm_case(samples, rows, width, groups, dtype, 5, pad, shift)
    clean = dense.groupnorm_fwd(x, gamma, beta, groups, samples, "silu")[0].clone()
    beta[3], beta[8], beta[14] = -math.inf, math.nan, math.inf
    y = dense.groupnorm_fwd(x, gamma, beta, groups, samples, "silu")[0]
    others = [i for i in range(width) if i not in (3, 8, 14)]
    want = clean[:, others].double()
    _close(y[:, others], want, (10.1 * U + 2.02 * ROUND[dtype]) * want.abs() + TINY, "others")
    assert torch.isnan(y[:, [3, 8]]).all() and (y[:, 14] == math.inf).all()


@both
@forms
@vectors
@pytest.mark.parametrize("value", [1000.1, 12345.678, -99999.9])
def test_groupnorm_constant_maps_whose_sums_round(value, rows, pad, shift, dtype):
    """No spread at all, and sums that 32 bits do not hold: h is zero all the same."""
    samples, groups, width = 3, 2, 16
    x = _rand((samples * rows, width), dtype, 1, 0.0, pad, shift, value)
    gamma, beta = _rand((width,), dtype, 2, 0.3, 0, shift, 1.0), _rand((width,), dtype, 3, 0.3, 0, shift)
    y, mean, rstd = dense.groupnorm_fwd(x, gamma, beta, groups, samples, eps=1e-6)
    assert torch.equal(mean, torch.full_like(mean, x[0, 0].item()))
    assert torch.allclose(rstd, torch.full_like(rstd, 1e3), rtol=1e-6)
    assert torch.equal(y, beta.expand(samples * rows, width))


@vectors
@pytest.mark.parametrize("mean", [3e3, -1e5])
def test_groupnorm_small_maps_far_from_zero(mean, pad, shift):
    """Distances from a value of the group are exact here (of neighbours in a factor of two), their mean is off by
    _sum_u(CHAIN) D, D the largest distance of two values; the mean as it is kept has its own rounding besides."""
    samples, rows, width, groups = 3, 300, 40, 5
    x, gamma, beta = _norm_case(samples, rows, width, groups, F32, 6, pad, shift, mean)
    y, mu, rstd = dense.groupnorm_fwd(x, gamma, beta, groups, samples)
    X = x.double().reshape(samples, rows, groups, -1)
    want = X.mean((1, 3), keepdim=True)
    var = (X - want).square().mean((1, 3), keepdim=True)
    D = X.amax((1, 3), keepdim=True) - X.amin((1, 3), keepdim=True)
    r = (var + 1e-5) ** -0.5
    emu = _sum_u(CHAIN) * D
    er = (0.5 * (_sum_u(CHAIN) * D * D + emu * emu) / (var + 1e-5) + 4 * U) * r
    _close(mu, want[:, 0, :, 0], (emu + U * want.abs())[:, 0, :, 0], "mean")
    _close(rstd, r[:, 0, :, 0], er[:, 0, :, 0], "rstd")
    G, B = gamma.double().view(groups, -1), beta.double().view(groups, -1)
    h = (X - want) * r
    ez = (emu * r + (X - want).abs() * er) * G.abs() + 4 * U * ((h * G).abs() + B.abs())
    _close(y, (h * G + B).reshape(x.shape), ez.reshape(x.shape) + TINY, "y")


@vectors
def test_groupnorm_small_maps_whose_first_value_is_far(pad, shift):
    """A value far from all others, among which the spread of a channel is small: their distances from the mean, which is
    next to them, are off by 4 u of themselves and of the mean, whatever the first value is."""
    samples, rows, width, groups = 3, 300, 40, 5
    x, gamma, beta = _norm_case(samples, rows, width, groups, F32, 6, pad, shift, 0.0)
    beta.zero_()
    x.view(samples, rows, width)[:, 0, ::width // groups] = 1e4 if not pad else -1e6
    y, mu, rstd = dense.groupnorm_fwd(x, gamma, beta, groups, samples)
    X = x.double().reshape(samples, rows, groups, -1)
    want = X.mean((1, 3), keepdim=True)
    var = (X - want).square().mean((1, 3), keepdim=True)
    _close(mu, want[:, 0, :, 0], 8 * U * X.abs().mean((1, 3)), "mean")
    _close(rstd.double() ** -2 - 1e-5, var[:, 0, :, 0], 32 * U * var[:, 0, :, 0], "variance")
    h = (X - want) * (var + 1e-5) ** -0.5 * gamma.double().view(groups, -1)
    off = (16 * U * X.abs().mean((1, 3), keepdim=True)) * (var + 1e-5) ** -0.5 * gamma.double().abs().view(groups, -1)
    _close(y, h.reshape(x.shape), (off + 24 * U * h.abs()).reshape(x.shape) + TINY, "y")


@pytest.mark.parametrize("shape", [(1, 600_000, 8, 1), (2, 200_000, 24, 3), (40, 15_000, 64, 32)], ids=str)
def test_groupnorm_first_rows_unlike_the_others(shape):
    """A strip of a map far from the rest of it (less than a chunk of rows): the variance to 128 u of itself.  Of that 57 u are
    _sum_u(600) for a sum of squares, twice 4 u the roundings of a chunk's mean of like values and of its distance from the
    joint mean, which is itself off by less than 57 u of the distances' mean; the rest is room."""
    samples, rows, width, groups = shape
    x = _rand((samples * rows, width), F32, 7, 0.5)
    strip = 64
    x.view(samples, rows, width)[:, :strip] = 900.1 + _rand((samples, strip, width), F32, 8, 1e-3)
    _, mean, rstd = dense.groupnorm_fwd(x, torch.ones(width, device="cuda"), torch.zeros(width, device="cuda"), groups, samples)
    X = x.double().view(samples, rows, groups, -1)
    var = X.var((1, 3), correction=0)
    _close(rstd.double() ** -2 - 1e-5, var, 128 * U * var, "variance")
    _close(mean, X.mean((1, 3)), 57 * U * X.abs().mean((1, 3)), "mean")


@pytest.mark.parametrize("act", ["none", "silu"])
def test_groupnorm_offsets_past_2_to_31(act):
    """Rows far apart: the same results as from their copies."""
    samples, rows, width, groups = 2, 40, 48, 3
    far = [torch.empty((samples * rows, 1 << 26), dtype=BF16, device="cuda")[:, :width] for _ in range(2)]
    near, gamma, beta = _norm_case(samples, rows, width, groups, BF16, 9)
    dy = _rand(near.shape, BF16, 10)
    far[0].copy_(near)
    want = dense.groupnorm_fwd(near, gamma, beta, groups, samples, act)
    got = dense.groupnorm_fwd(far[0], gamma, beta, groups, samples, act, out=far[1])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    grads = dense.groupnorm_bwd(dy, near, gamma, beta, *want[1:], act=act, skip=dy)
    far[1].copy_(dy)
    got = dense.groupnorm_bwd(far[1], far[0], gamma, beta, *want[1:], act=act, skip=far[1], dx=far[1])
    assert all(torch.equal(a, b) for a, b in zip(got, grads))
    del far, got
    # more than 2^31 values
    x = torch.empty((2, 1 << 21, 520), dtype=BF16, device="cuda")
    x[:] = _rand((1 << 10, 520), BF16, 11).repeat(1 << 11, 1)
    gamma, beta = _rand((520,), BF16, 12, 0.1, mean=1.0), _rand((520,), BF16, 13)
    few = x[0, :1 << 10].contiguous()
    y, mean, rstd = dense.groupnorm_fwd(x.view(-1, 520), gamma, beta, 65, 2, act)
    _check_norm_fwd(1, 1 << 10, 65, few, gamma, beta, act, 1e-5, (y[-(1 << 10):], mean[1:], rstd[1:]))
    assert torch.equal(y[:1 << 10], y[-(1 << 10):]) and torch.equal(mean[0], mean[1])
    dx, _, _ = dense.groupnorm_bwd(x.view(-1, 520), x.view(-1, 520), gamma, beta, mean, rstd, act=act, need_dparams=False)
    want = _norm_grads(1, 65, few, few, gamma, beta, mean[:1], rstd[:1], act, None)["dx"]
    _close(dx[-(1 << 10):], *want, "dx")
    assert torch.equal(dx[:1 << 10], dx[-(1 << 10):])


def test_groupnorm_refuses_more_maps_than_it_can_number():
    """Before anything is allocated for them."""
    x, v = torch.zeros((0, 64), device="cuda"), torch.zeros(64, device="cuda")
    with pytest.raises(ValueError, match="maps"):
        dense.groupnorm_fwd(x, v, v, 64, samples=1 << 40)
    assert dense.groupnorm_fwd(x, v, v, 64, samples=3)[1].shape == (3, 64)


# ------------------------------------------------------------------ AdamW
def _off(n, dtype, shift):
    return torch.zeros(n + shift, dtype=dtype, device="cuda")[shift:]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("decay", [1e-7, 2e-8, 3e-6, 1e-3, 0.3, 0.5, 0.9990001, 1.0, 1.7, -1e-7])
def test_adamw_decay_is_not_rounded(decay, bits, shift):
    """p (1 - lr weight_decay) - step is off by half a unit in the last place (the rounding of p), by what two floats leave
    of the factor (2^-48) and by 16 u of the step, which at the first one is lr."""
    n, lr = 5001, 1e-6
    for moves in (False, True):
        p, g = _off(n, F32, shift), _off(n, F32, shift)
        p.copy_(_rand((n,), F32, 1))
        if moves:
            g.copy_(_rand((n,), F32, 2))
        step = lr * g.double() / (g.double().abs() + 1e-8)
        want = p.double() * (1 - lr * (decay / lr)) - step
        unit = torch.exp2(torch.floor(torch.log2(want.abs().clamp(min=1e-30))) - 23)
        last = 0.5 * unit + 2.0 ** -48 * p.double().abs() + 16 * U * lr * moves + TINY
        m, v, scales = dense.adamw_state([p], bits)
        dense.adamw([p], [g], m, v, 1, lr, weight_decay=decay / lr, scales=scales)
        _close(p, want, last, f"p {moves}")


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("decay", [0.0, 1e-7, 1e-3, 0.25, 1.5])
def test_adamw_leaves_the_ends_of_the_range(decay, bits):
    """Parameters that are infinite, zero, or among the smallest and largest floats, without gradients."""
    tiny, most = torch.finfo(F32).smallest_normal, torch.finfo(F32).max
    p = torch.tensor([math.inf, -math.inf, 0.0, -0.0, tiny, -tiny, 2.0 ** -149, most, -most, 1.0], device="cuda").repeat(60)
    before = p.double()
    m, v, scales = dense.adamw_state([p], bits)
    dense.adamw([p], [torch.zeros_like(p)], m, v, 1, 1e-3, weight_decay=decay / 1e-3, scales=scales)
    keep = 1 - 1e-3 * (decay / 1e-3)
    assert torch.equal(p.isinf(), before.isinf()) and (p[:2] == before[:2].float() * (1 if keep > 0 else -1)).all()
    finite = ~before.isinf()
    want = before[finite] * keep
    _close(p[finite], want, 1.0001 * U * want.abs() + 2.0 ** -149, "p")
    if decay == 0.0:
        assert torch.equal(p, before.float())


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [1e-46, 1e-40, 1.1e-38, 1e-30])
def test_adamw_smallest_eps(eps, bits):
    """A value that no gradient has reached yet stays where it is, and others move by lr at the first step."""
    p, g = [_rand((600,), F32, 1)], [_rand((600,), F32, 2)]
    g[0][::3] = 0.0
    before = p[0].clone()
    m, v, scales = dense.adamw_state(p, bits)
    dense.adamw(p, g, m, v, 1, 1e-3, eps=eps, weight_decay=0.0, scales=scales)
    assert torch.equal(p[0][::3], before[::3])
    _close(p[0], before.double() - 1e-3 * g[0].sign().double(), 16 * U * 1e-3 + 2 * U * before.double().abs(), "p")


def test_adamw_refuses_arrays_that_overlap():
    def args(**kw):
        a = dict(params=[torch.zeros(900, device="cuda") for _ in range(2)], grads=[torch.zeros(900, device="cuda") for _ in range(2)],
                 exp_avg=[torch.zeros(900, device="cuda") for _ in range(2)],
                 exp_avg_sq=[torch.zeros(900, device="cuda") for _ in range(2)])
        return {**a, **kw}

    dense.adamw(**args(), step=1)
    one = torch.zeros(2000, device="cuda")
    a = args()
    bad = [args(exp_avg=a["exp_avg"], exp_avg_sq=a["exp_avg"]), args(exp_avg=[one[:900], one[899:1799]]),
           args(grads=[one[:900], one[900:1800]], exp_avg=[one[1000:1900], a["exp_avg"][0]]),
           args(params=a["params"], grads=[a["params"][1], a["grads"][0]]), args(params=[one[:900], one[1:901]])]
    for b in bad:
        with pytest.raises(GSError, match="overlap"):
            dense.adamw(**b, step=1)
    # a gradient is only read: two tensors may share one; what lies side by side does not overlap
    dense.adamw(**args(grads=[one[:900], one[:900]]), step=1)
    dense.adamw(**args(params=[one[:900], one[900:1800]]), step=1)


@pytest.mark.parametrize("shift", [0, 1])
def test_adamw_offsets_past_2_to_31(shift):
    """More than 2^31 values in a tensor: the first and the last of them as a tensor of their own."""
    n, run = (1 << 31) + 5_000, 256
    p, g = _off(n, F32, shift), _off(n, BF16, shift)
    (m,), (v,), scales = dense.adamw_state([p], 8)
    few = {}
    for at in (0, (n - 4_000) // run * run):
        part = slice(at, at + 4_000)
        p[part], g[part] = _rand((p[part].numel(),), F32, 2), _rand((g[part].numel(),), BF16, 3)
        few[at] = (part, p[part].clone(), g[part].clone())
    dense.adamw([p], [g], [m], [v], 1, weight_decay=0.1, scales=scales)
    for at, (part, q, h) in few.items():
        m2, v2, s2 = dense.adamw_state([q], 8)
        dense.adamw([q], [h], m2, v2, 1, weight_decay=0.1, scales=s2)
        assert torch.equal(q, p[part]) and (q != 0).any()
        assert torch.equal(s2[0][0][:15], scales[0][0][at // run:at // run + 15])
    assert not p[5_000:1 << 20].any() and not p[-(1 << 20):-5_000].any()


# ------------------------------------------------------------------ graphs
def _inputs(seed):
    return [_rand((300, 24), F32, seed), _indices(5000, 300, "skewed", seed), _rand((24,), F32, seed + 1, 0.1, mean=1.0),
            _rand((24,), F32, seed + 2)], _tensors([300 * 24, 24, 24], F32, seed + 3, 0, 8)


def _live(state):
    p, _, m, v, scales = state
    return [*p, *[t.view(torch.uint8) for t in (*m, *v)], *scales[0], *scales[1]]


def _calls(inputs, state, step):
    table, idx, gamma, beta = inputs
    y = dense.embedding_fwd(table, idx, 2.0)
    z, mean, rstd = dense.groupnorm_fwd(y, gamma, beta, 4, 5, "silu")
    dx, dg, db = dense.groupnorm_bwd(z, y, gamma, beta, mean, rstd, act="silu")
    dt = dense.embedding_bwd(dx, idx, 300, 2.0)
    p, _, m, v, scales = state
    dense.adamw(p, [dt.view(-1), dg, db], m, v, step, scales=scales)
    return [y, z, mean, rstd, dx, dg, db, dt]


def test_graphs_replayed_on_new_inputs():
    """Two graphs that share a pool of memory, replayed in turn on inputs that they were not captured with: every output and
    every state that a replay leaves is that of plain calls."""
    pool, graphs = torch.cuda.graph_pool_handle(), []
    _calls(*_inputs(29), 5)  # (loads the kernels)
    torch.cuda.synchronize()
    for seed in (30, 40):
        inputs, state = _inputs(seed)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, pool=pool):
            out = _calls(inputs, state, 5)
        graphs.append((graph, inputs, state, out))
    for seed in (30, 50, 60, 50):
        for graph, inputs, state, out in graphs:
            fresh, fresh_state = _inputs(seed)
            for a, b in zip(inputs + _live(state), fresh + _live(fresh_state)):
                a.copy_(b)
            want = _calls(fresh, fresh_state, 5)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(want + _live(fresh_state), out + _live(state)))
