"""Refusals of the dense-layer entry points, on the host (no GPU needed): bad sizes, types, strides,
alignments and missing arrays are errors before anything is enqueued."""
import ctypes as C
import os
import sys

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

from gaussian_splatting_gb300 import _native as N  # noqa: E402
from gaussian_splatting_gb300 import dense  # noqa: E402


@pytest.fixture(scope="module")
def lib():
    from gaussian_splatting_gb300 import build
    build.build()
    return N.load()


P = 1 << 20  # an address that is never followed: the checks come first


def _linear(**kw):
    d = N.LinearDesc()
    d.rows, d.in_features, d.out_features, d.dtype, d.act = 10, 8, 6, N.GS_F32, N.GS_ACT_NONE
    d.ldx = d.ldw = d.lddx = d.lddw = 8
    d.ldy = d.ldr = d.ldz = 6
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def _fwd(lib, d, x=P, w=P, bias=None, residual=None, y=P, z=None, ws=P, n=1 << 40):
    return lib.gs_linear_fwd(C.addressof(d) if d else None, x, w, bias, residual, y, z, ws, n, None, None)


def _bwd(lib, d, dy=P, x=P, w=P, z=None, dx=P, dw=P, dbias=P, ws=P, n=1 << 40):
    return lib.gs_linear_bwd(C.addressof(d) if d else None, dy, x, w, z, dx, dw, dbias, ws, n, None, None)


BAD_SIZES = [dict(rows=-1), dict(rows=1 << 31), dict(in_features=0), dict(out_features=0), dict(in_features=-4),
             dict(out_features=(1 << 20) + 1), dict(dtype=2), dict(dtype=-1), dict(act=4), dict(act=-1)]


@pytest.mark.parametrize("bad", BAD_SIZES, ids=str)
def test_linear_refuses_bad_descriptors(lib, bad):
    assert _fwd(lib, _linear(**bad)) == N.GS_ERR_INVALID
    assert _bwd(lib, _linear(**bad)) == N.GS_ERR_INVALID
    d = _linear(**bad)
    assert lib.gs_linear_fwd_workspace_size(C.addressof(d)) == 0
    assert lib.gs_linear_bwd_workspace_size(C.addressof(d)) == 0


def test_linear_refuses_missing_misaligned_and_overlapping_arrays(lib):
    d = _linear()
    assert _fwd(lib, None) == N.GS_ERR_INVALID and _bwd(lib, None) == N.GS_ERR_INVALID
    for name in ("x", "w", "y"):
        assert _fwd(lib, d, **{name: None}) == N.GS_ERR_INVALID
        assert name.encode() in lib.gs_last_error()
        assert _fwd(lib, d, **{name: P + 2}) == N.GS_ERR_INVALID
    for name in ("bias", "residual", "z"):
        assert _fwd(lib, d, **{name: P + 1}) == N.GS_ERR_INVALID
    for name in ("dy", "x", "w"):
        assert _bwd(lib, d, **{name: None}) == N.GS_ERR_INVALID
    for name in ("dx", "dw", "dbias"):
        assert _bwd(lib, d, **{name: P + 2}) == N.GS_ERR_INVALID
    # an activation's gradient needs z
    assert _bwd(lib, _linear(act=N.GS_ACT_GELU)) == N.GS_ERR_INVALID
    assert b"z" in lib.gs_last_error()
    # rows that overlap
    for f in ("ldx", "ldw"):
        assert _fwd(lib, _linear(**{f: 7})) == N.GS_ERR_INVALID
    assert _fwd(lib, _linear(ldy=5)) == N.GS_ERR_INVALID
    assert _fwd(lib, _linear(ldr=5), residual=P) == N.GS_ERR_INVALID
    assert _fwd(lib, _linear(ldz=5), z=P) == N.GS_ERR_INVALID
    assert _bwd(lib, _linear(lddx=7)) == N.GS_ERR_INVALID
    assert _bwd(lib, _linear(lddw=7)) == N.GS_ERR_INVALID


def test_linear_refuses_a_workspace_that_is_missing_small_or_misaligned(lib):
    d = _linear(rows=300_000, in_features=64, out_features=64, ldx=64, ldw=64, ldy=64, lddx=64, lddw=64)
    need = lib.gs_linear_bwd_workspace_size(C.addressof(d))
    assert need > 0
    assert _bwd(lib, d, ws=None, n=0) == N.GS_ERR_INVALID
    assert _bwd(lib, d, n=need - 1) == N.GS_ERR_INVALID
    assert _bwd(lib, d, ws=P + 4) == N.GS_ERR_INVALID


def test_calls_with_nothing_to_do_succeed_without_touching_memory(lib):
    assert _fwd(lib, _linear(rows=0), x=None, w=None, y=None, ws=None, n=0) == N.GS_OK
    assert _bwd(lib, _linear(), dy=None, x=None, w=None, dx=None, dw=None, dbias=None, ws=None, n=0) == N.GS_OK
    assert _bwd(lib, _linear(rows=0), dy=None, x=None, w=None, dw=None, dbias=None, ws=None, n=0) == N.GS_OK
    d = _linear(rows=0)
    assert lib.gs_linear_fwd_workspace_size(C.addressof(d)) == 0


def _norm(**kw):
    d = N.LayerNormDesc()
    d.rows, d.width, d.dtype, d.eps = 10, 8, N.GS_F32, 1e-5
    d.ldx = d.ldy = d.lddy = d.ldskip = d.lddx = 8
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def _nfwd(lib, d, x=P, gamma=P, beta=P, y=P):
    return lib.gs_layernorm_fwd(C.addressof(d) if d else None, x, gamma, beta, y, None, None, None)


def _nbwd(lib, d, dy=P, x=P, gamma=P, mean=P, rstd=P, skip=None, dx=P, dgamma=P, dbeta=P, ws=P, n=1 << 40):
    return lib.gs_layernorm_bwd(C.addressof(d) if d else None, dy, x, gamma, mean, rstd, skip, dx, dgamma, dbeta, ws, n,
                                None)


def test_layernorm_refusals(lib):
    assert _nfwd(lib, None) == N.GS_ERR_INVALID and _nbwd(lib, None) == N.GS_ERR_INVALID
    for bad in (dict(rows=-1), dict(width=0), dict(width=(1 << 24) + 1), dict(dtype=7)):
        assert _nfwd(lib, _norm(**bad)) == N.GS_ERR_INVALID
        assert _nbwd(lib, _norm(**bad)) == N.GS_ERR_INVALID
    assert _nfwd(lib, _norm(eps=-1.0)) == N.GS_ERR_INVALID
    assert _nfwd(lib, _norm(eps=float("nan"))) == N.GS_ERR_INVALID
    for name in ("x", "gamma", "beta", "y"):
        assert _nfwd(lib, _norm(), **{name: None}) == N.GS_ERR_INVALID
        assert _nfwd(lib, _norm(), **{name: P + 2}) == N.GS_ERR_INVALID
    for name in ("dy", "x", "gamma", "mean", "rstd"):
        assert _nbwd(lib, _norm(), **{name: None}) == N.GS_ERR_INVALID
    for name in ("skip", "dx", "dgamma", "dbeta"):
        assert _nbwd(lib, _norm(), **{name: P + 1}) == N.GS_ERR_INVALID
    for f in ("ldx", "ldy"):
        assert _nfwd(lib, _norm(**{f: 7})) == N.GS_ERR_INVALID
    for f in ("ldx", "lddy", "lddx"):
        assert _nbwd(lib, _norm(**{f: 7})) == N.GS_ERR_INVALID
    assert _nbwd(lib, _norm(ldskip=7), skip=P) == N.GS_ERR_INVALID
    d = _norm()
    need = lib.gs_layernorm_bwd_workspace_size(C.addressof(d))
    assert need > 0
    assert _nbwd(lib, _norm(), n=need - 1) == N.GS_ERR_INVALID
    assert _nbwd(lib, _norm(), ws=None) == N.GS_ERR_INVALID
    assert _nfwd(lib, _norm(rows=0), x=None, gamma=None, beta=None, y=None) == N.GS_OK
    assert _nbwd(lib, _norm(), dx=None, dgamma=None, dbeta=None) == N.GS_OK


def test_tensor_functions_refuse_what_the_library_cannot_take(lib):
    x, w = torch.zeros(4, 8), torch.zeros(6, 8)
    with pytest.raises(ValueError, match="CUDA"):
        dense.linear_fwd(x, w)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        dense.linear_fwd(x.double(), w.double())
    with pytest.raises(ValueError, match="matrix"):
        dense.layernorm_fwd(torch.zeros(8), torch.zeros(8), torch.zeros(8))
    # shapes, types and strides of the other arguments
    like = x
    for bad in (torch.zeros(4, 7), torch.zeros(5, 8), torch.zeros(4, 8, 1), torch.zeros(4, 8).bfloat16(),
                torch.zeros(8, 4).t(), torch.zeros(1, 8).expand(4, 8)):
        with pytest.raises(ValueError):
            dense._matrix(bad, "a", 4, 8, like)
    assert dense._matrix(torch.zeros(4, 12)[:, :8], "a", 4, 8, like) == 12
    assert dense._matrix(torch.zeros(1, 8), "a", 1, 8, like) == 8
    for bad in (torch.zeros(7), torch.zeros(1, 8), torch.zeros(16)[::2], torch.zeros(8).bfloat16()):
        with pytest.raises(ValueError):
            dense._vector(bad, "a", 8, like)


@pytest.mark.parametrize("act", ["tanh", "", None, 2, ["relu"]])
def test_tensor_functions_refuse_an_activation_that_there_is_not(lib, act):
    x, w = torch.zeros(4, 8), torch.zeros(6, 8)
    with pytest.raises(ValueError, match="act must be one of none, relu, gelu, silu"):
        dense.linear_fwd(x, w, act=act)
    with pytest.raises(ValueError, match="act must be one of"):
        dense.linear_bwd(torch.zeros(4, 6), x, w, act=act)
