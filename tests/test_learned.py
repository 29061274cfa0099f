"""Refusals of code lookup, group norm and AdamW, on the host (no GPU needed): bad sizes, types, strides, alignments and
missing arrays are errors before anything is enqueued."""
import ctypes as C
import math
import os
import sys

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

from gaussian_splatting_gb300 import _native as N  # noqa: E402
from gaussian_splatting_gb300 import dense  # noqa: E402

P = 1 << 20  # an address that is never followed: the checks come first


@pytest.fixture(scope="module")
def lib():
    from gaussian_splatting_gb300 import build
    build.build()
    return N.load()


def _with(d, fields):
    for k, v in fields.items():
        setattr(d, k, v)
    return d


def _codes(**kw):
    return _with(N.EmbeddingDesc(10, 20, 8, 8, 8, N.GS_F32, 32, 1.0), kw)


def _size(size, d):
    return size(C.addressof(d))


def _look(lib, d, table=P, idx=P, y=P):
    return lib.gs_embedding_fwd(C.addressof(d) if d else None, table, idx, y, None)


def _grad(lib, d, dy=P, idx=P, dtable=P, ws=P, n=1 << 40):
    return lib.gs_embedding_bwd(C.addressof(d) if d else None, dy, idx, dtable, ws, n, None)


@pytest.mark.parametrize("bad", [dict(rows=-1), dict(rows=(1 << 31) - 1), dict(n=-1), dict(n=(1 << 31) - 1), dict(width=0),
                                 dict(width=(1 << 20) + 1), dict(dtype=2), dict(index_bits=16), dict(index_bits=0),
                                 dict(ldt=7), dict(ldy=7)], ids=str)
def test_embedding_refuses_bad_descriptors(lib, bad):
    assert _look(lib, _codes(**bad)) == N.GS_ERR_INVALID
    assert _grad(lib, _codes(**bad)) == N.GS_ERR_INVALID
    if not {"ldt", "ldy"} & set(bad):
        assert _size(lib.gs_embedding_bwd_workspace_size, _codes(**bad)) == 0


def test_embedding_refuses_missing_and_misaligned_arrays(lib):
    assert _look(lib, None) == N.GS_ERR_INVALID and _grad(lib, None) == N.GS_ERR_INVALID
    for name in ("table", "idx", "y"):
        for at in (None, P + 2):
            assert _look(lib, _codes(), **{name: at}) == N.GS_ERR_INVALID
            assert name.encode() in lib.gs_last_error()
    for name in ("dy", "idx", "dtable"):
        for at in (None, P + 2):
            assert _grad(lib, _codes(), **{name: at}) == N.GS_ERR_INVALID
            assert name.encode() in lib.gs_last_error()
    assert _look(lib, _codes(index_bits=64), idx=P + 4) == N.GS_ERR_INVALID
    assert _size(lib.gs_embedding_bwd_workspace_size, _codes()) == 0  # few rows need none
    for many in (dict(rows=20_000), dict(rows=2_000_000, n=5000)):
        need = _size(lib.gs_embedding_bwd_workspace_size, _codes(**many))
        assert need > 0
        assert _grad(lib, _codes(**many), n=need - 1) == N.GS_ERR_INVALID
        assert _grad(lib, _codes(**many), ws=None) == N.GS_ERR_INVALID
        assert _grad(lib, _codes(**many), ws=P + 16) == N.GS_ERR_INVALID
    # nothing to do
    assert _look(lib, _codes(rows=0), table=None, idx=None, y=None) == N.GS_OK
    assert _grad(lib, _codes(n=0), dy=None, idx=None, dtable=None, ws=None, n=0) == N.GS_OK


def _norm(**kw):
    return _with(N.GroupNormDesc(2, 5, 8, 8, 8, 8, 8, 8, 4, N.GS_F32, N.GS_ACT_SILU, 1e-5), kw)


def _nfwd(lib, d, x=P, gamma=P, beta=P, y=P, mean=None, rstd=None, ws=P, n=1 << 40):
    return lib.gs_groupnorm_fwd(C.addressof(d) if d else None, x, gamma, beta, y, mean, rstd, ws, n, None)


def _nbwd(lib, d, dy=P, x=P, gamma=P, beta=P, mean=P, rstd=P, skip=None, dx=P, dgamma=P, dbeta=P, ws=P, n=1 << 40):
    return lib.gs_groupnorm_bwd(C.addressof(d) if d else None, dy, x, gamma, beta, mean, rstd, skip, dx, dgamma, dbeta, ws,
                                n, None)


@pytest.mark.parametrize("bad", [dict(samples=-1), dict(rows=-1), dict(samples=1 << 20, rows=1 << 12), dict(samples=1 << 40),
                                 dict(rows=1 << 62, samples=4), dict(width=0), dict(width=(1 << 20) + 8), dict(groups=0),
                                 dict(groups=3), dict(groups=16), dict(dtype=2), dict(act=4), dict(act=-1), dict(ldx=7)], ids=str)
def test_groupnorm_refuses_bad_descriptors(lib, bad):
    assert _nfwd(lib, _norm(**bad)) == N.GS_ERR_INVALID
    assert _nbwd(lib, _norm(**bad)) == N.GS_ERR_INVALID
    if "ldx" not in bad:
        assert _size(lib.gs_groupnorm_fwd_workspace_size, _norm(**bad)) == 0
        assert _size(lib.gs_groupnorm_bwd_workspace_size, _norm(**bad)) == 0


def test_groupnorm_refuses_missing_and_misaligned_arrays(lib):
    assert _nfwd(lib, None) == N.GS_ERR_INVALID and _nbwd(lib, None) == N.GS_ERR_INVALID
    for eps in (-1.0, math.nan):
        assert _nfwd(lib, _norm(eps=eps)) == N.GS_ERR_INVALID
    for name in ("x", "gamma", "beta", "y"):
        for at in (None, P + 2):
            assert _nfwd(lib, _norm(), **{name: at}) == N.GS_ERR_INVALID
    for name in ("mean", "rstd"):
        assert _nfwd(lib, _norm(), **{name: P + 1}) == N.GS_ERR_INVALID
    for name in ("dy", "x", "gamma", "beta", "mean", "rstd"):
        for at in (None, P + 2):
            assert _nbwd(lib, _norm(), **{name: at}) == N.GS_ERR_INVALID
    for name in ("skip", "dx", "dgamma", "dbeta"):
        assert _nbwd(lib, _norm(), **{name: P + 1}) == N.GS_ERR_INVALID
    assert _nfwd(lib, _norm(ldy=7)) == N.GS_ERR_INVALID
    for f in ("lddy", "lddx"):
        assert _nbwd(lib, _norm(**{f: 7})) == N.GS_ERR_INVALID
    assert _nbwd(lib, _norm(ldskip=7), skip=P) == N.GS_ERR_INVALID
    for call, size in ((_nfwd, lib.gs_groupnorm_fwd_workspace_size), (_nbwd, lib.gs_groupnorm_bwd_workspace_size)):
        need = _size(size, _norm())
        if need:
            assert call(lib, _norm(), n=need - 1) == N.GS_ERR_INVALID
            assert call(lib, _norm(), ws=None) == N.GS_ERR_INVALID
            assert call(lib, _norm(), ws=P + 4) == N.GS_ERR_INVALID
    assert _nfwd(lib, _norm(rows=0), x=None, gamma=None, beta=None, y=None) == N.GS_OK
    assert _nbwd(lib, _norm(), dx=None, dgamma=None, dbeta=None) == N.GS_OK


def _step(lib, tensors, bits=32, counts=None, n_counts=0, **kw):
    d = _with(N.AdamWDesc(0.9, 0.999, 1e-8, 1, N.GS_F32, bits, 0), kw)
    arr = (N.AdamWTensor * max(1, len(tensors)))(*tensors)
    return lib.gs_adamw(C.addressof(d), C.addressof(arr), len(tensors), counts, n_counts, None)


def _member(k=0, scales=False, **kw):
    s = P if scales else None
    return _with(N.AdamWTensor(P + 4096 * k, P, P, P, s, s, None, 1000, 1e-3, 0.01), kw)


def test_adamw_refusals(lib):
    d = N.AdamWDesc()
    assert lib.gs_adamw(None, None, 0, None, 0, None) == N.GS_ERR_INVALID
    assert lib.gs_adamw(C.addressof(d), None, 1, None, 0, None) == N.GS_ERR_INVALID
    for bad in (dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=math.nan), dict(eps=-1e-8), dict(eps=math.nan),
                dict(step=0), dict(step=-3), dict(grad_dtype=2), dict(bits=16), dict(n_counts=-1), dict(n_counts=1),
                dict(n_counts=1, counts=P + 4)):
        assert _step(lib, [_member()], **bad) == N.GS_ERR_INVALID, bad
    for bad in (dict(param=None), dict(grad=None), dict(exp_avg=None), dict(exp_avg_sq=None), dict(param=P + 2),
                dict(grad=P + 2), dict(exp_avg=P + 1), dict(exp_avg_sq=P + 2), dict(copy=P + 1), dict(n=-1), dict(n=1 << 42),
                dict(lr=math.inf), dict(weight_decay=math.nan)):
        assert _step(lib, [_member(), _member(1, **bad)]) == N.GS_ERR_INVALID, bad
        assert b"tensor 1" in lib.gs_last_error()
    # 8-bit moments need scales; 8-bit codes any address
    assert _step(lib, [_member()], bits=8) == N.GS_ERR_INVALID
    assert _step(lib, [_member(scales=True, exp_avg_scale=P + 2)], bits=8) == N.GS_ERR_INVALID
    # the same values twice, or in part
    for twin in (_member(0), _member(0, n=1), _member(0, param=P + 3996)):
        assert _step(lib, [_member(0), _member(3), twin]) == N.GS_ERR_INVALID
        assert b"overlap" in lib.gs_last_error()
    # nothing to do
    assert _step(lib, []) == N.GS_OK
    assert _step(lib, [_member(n=0, param=None, grad=None)] * 3) == N.GS_OK


def test_tensor_functions_refuse_what_the_library_cannot_take(lib):
    x, v = torch.zeros(6, 8), torch.zeros(8)
    idx = torch.zeros(6, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        dense.embedding_fwd(x, idx)
    with pytest.raises(ValueError, match="CUDA"):
        dense.groupnorm_fwd(x, v, v, 2)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        dense.embedding_bwd(x.half(), idx, 3)
    with pytest.raises(ValueError, match="act must be one of"):
        dense.groupnorm_fwd(x, v, v, 2, act="tanh")
    with pytest.raises(ValueError, match="act must be one of"):
        dense.groupnorm_bwd(x, x, v, v, v, v, act=None)
    with pytest.raises(ValueError, match="CUDA"):
        dense.adamw([x], [x], [x], [x], 1)
    with pytest.raises(ValueError, match="params"):
        dense.adamw([x.bfloat16()], [x], [x], [x], 1)
    with pytest.raises(ValueError, match="must have 1 entries"):
        dense.adamw([x], [x, x], [x], [x], 1)
    with pytest.raises(ValueError, match="sequence"):
        dense.adamw(None, 3, [x], [x], 1)
    with pytest.raises(ValueError, match="params must be a sequence"):
        dense.adamw(3, [x], [x], [x], 1)
    assert dense.adamw([], [], [], [], 1) is None
    m, s, scales = dense.adamw_state([x, torch.zeros(300)], bits=8)
    assert m[0].dtype == s[1].dtype == torch.float8_e4m3fn and [t.numel() for t in scales[0]] == [1, 2]
    assert dense.adamw_state([x])[2] is None
