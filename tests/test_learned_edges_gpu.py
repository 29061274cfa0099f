"""Code lookup, group norm and AdamW where their arithmetic is at its ends.

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
from test_learned_gpu import BF16, F32, ROUND, TINY, U, _close, _norm_case, _norm_grads, _rand  # noqa: E402

pytestmark = pytest.mark.gpu
both = pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
# rows of a map: a block holds a group, or two passes do; rows on 16 bytes, or one value a thread
forms = pytest.mark.parametrize("rows", [50, 20_011], ids=["one-kernel", "two-passes"])
vectors = pytest.mark.parametrize("pad,shift", [(0, 0), (2, 2), (1, 1)], ids=["whole", "pairs", "single"])


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
