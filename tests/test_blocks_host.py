"""Refusals of the gated delta rule and the norms at the C boundary, without
a GPU: no call here reaches a kernel (FAKE addresses are never read)."""
import ctypes

import pytest
import torch

import selective_state_space_24_b200 as ssm
from selective_state_space_24_b200 import build as ssm_build

FAKE = 0x7F0000000000
OK, INVALID, SHAPE, MISALIGNED, DTYPE, WORKSPACE = 0, 1, 2, 3, 4, 5
ref = ctypes.byref


@pytest.fixture(scope="module")
def lib():
    ssm_build.build()
    return ssm.load()


def dims(B=2, L=8, Hk=2, Hv=4, K=128, V=64, dt=ssm.SSM_BF16):
    return ssm.gdr_dims(B, L, Hk, Hv, K, V, dt)


def inputs(**kw):
    f = dict(q=FAKE, k=FAKE, v=FAKE, delta=FAKE, delta_bias=None, A=FAKE, beta=FAKE, scale=1.0)
    f.update(kw)
    return ssm.gdr_inputs(**f)


def fwd(lib, d, i, init=None, out=FAKE, last=None, ws=None, n=0):
    return lib.gdr_chunk_fwd(ref(d) if d else None, ref(i) if i else None, init, out, last, ws, n, None)


def test_gdr_refusals(lib):
    assert fwd(lib, None, inputs()) == INVALID
    assert fwd(lib, dims(), None) == INVALID
    for name in ("q", "k", "v", "delta", "A", "beta"):
        assert fwd(lib, dims(), inputs(**{name: None})) == INVALID
        assert fwd(lib, dims(), inputs(**{name: FAKE + 2})) == MISALIGNED
    assert fwd(lib, dims(), inputs(), out=None) == INVALID
    assert fwd(lib, dims(), inputs(scale=float("nan"))) == INVALID
    assert fwd(lib, dims(), inputs(), init=FAKE + 4) == MISALIGNED
    assert fwd(lib, dims(), inputs(), last=FAKE + 8) == MISALIGNED
    for bad in (dict(B=-1), dict(L=-1), dict(Hk=-2), dict(K=-64)):
        assert fwd(lib, dims(**bad), inputs()) == INVALID
    for bad in (dict(K=96), dict(V=32), dict(K=256), dict(V=0), dict(Hv=3), dict(Hk=0), dict(L=2 ** 31),
                dict(B=2 ** 31 - 1), dict(Hv=2 ** 28, Hk=1)):
        assert fwd(lib, dims(**bad), inputs()) == SHAPE, bad
    assert fwd(lib, dims(dt=ssm.SSM_F32), inputs()) == DTYPE
    assert fwd(lib, dims(dt=9), inputs()) == DTYPE
    assert lib.gdr_chunk_workspace_size(None) == 0
    assert lib.gdr_chunk_workspace_size(ref(dims(K=96))) == 0
    need = lib.gdr_chunk_workspace_size(ref(dims(L=4096)))
    if need:
        assert fwd(lib, dims(L=4096), inputs()) == WORKSPACE
        assert fwd(lib, dims(L=4096), inputs(), ws=FAKE, n=need - 1) == WORKSPACE
        assert fwd(lib, dims(L=4096), inputs(), ws=FAKE + 4, n=need) == MISALIGNED


def test_gdr_step_refusals(lib):
    step = lambda d, i, st=FAKE, out=FAKE: lib.gdr_step(ref(d), ref(i), st, out, None)   # noqa: E731
    assert step(dims(L=2), inputs()) == SHAPE
    assert step(dims(L=1), inputs(), st=None) == INVALID
    assert step(dims(L=1), inputs(), out=None) == INVALID
    assert step(dims(L=1), inputs(), st=FAKE + 4) == MISALIGNED
    assert step(dims(L=1, dt=7), inputs()) == DTYPE
    assert step(dims(L=1, dt=ssm.SSM_F32), inputs(q=None)) == INVALID
    assert step(dims(B=0, L=1), inputs(q=None), st=None) == OK


def test_gdr_bwd_refusals(lib):
    need = lib.gdr_chunk_bwd_workspace_size(ref(dims()))
    assert need > 0
    names = ("dq", "dk", "dv", "ddelta", "dbeta", "dA")

    def call(d=dims(), i=inputs(), dout=FAKE, ws=FAKE, n=need, grads=True, **kw):
        g = ssm.gdr_grads(**{**{m: FAKE for m in names}, **kw})
        return lib.gdr_chunk_bwd(ref(d), ref(i), None, dout, None, ref(g) if grads else None, ws, n, None)

    assert call(grads=False) == INVALID
    assert call(dout=None) == INVALID
    for m in names:
        assert call(**{m: None}) == INVALID
        assert call(**{m: FAKE + 2}) == MISALIGNED
    assert call(i=inputs(delta_bias=FAKE)) == INVALID     # its gradient has no place
    assert call(n=need - 1) == WORKSPACE and call(ws=None) == WORKSPACE
    assert call(ws=FAKE + 8) == MISALIGNED
    assert call(d=dims(Hv=5)) == SHAPE


def nd(rows=4, dim=64, group=None, eps=1e-5, dt=ssm.SSM_BF16):
    return ssm.norm_dims(rows, dim, dim if group is None else group, eps, dt)


def test_gated_norm_refusals(lib):
    f = lambda d, x=FAKE, z=None, w=FAKE, out=FAKE: lib.gated_norm_fwd(ref(d), x, z, w, 0, out, None)   # noqa: E731
    assert f(nd(), x=None) == INVALID and f(nd(), w=None) == INVALID and f(nd(), out=None) == INVALID
    assert f(nd(), z=FAKE + 8) == MISALIGNED
    assert f(nd(rows=-1)) == INVALID and f(nd(eps=-1.0)) == INVALID and f(nd(eps=float("nan"))) == INVALID
    assert f(nd(dt=5)) == DTYPE
    assert f(nd(dim=64, group=24)) == SHAPE and f(nd(dim=16384)) == SHAPE and f(nd(dim=0)) == SHAPE
    assert f(nd(dim=60)) == MISALIGNED and f(nd(dim=64, group=4)) == MISALIGNED
    assert f(nd(dim=64, group=4, dt=ssm.SSM_F32), x=None) == INVALID   # fp32 may take groups of 4
    assert f(nd(rows=0), x=None, w=None, out=None) == OK
    need = lib.gated_norm_bwd_workspace_size(ref(nd()))
    b = lambda dz=None, z=None, ws=FAKE, n=need, dw=FAKE: lib.gated_norm_bwd(   # noqa: E731
        ref(nd()), FAKE, z, FAKE, 0, FAKE, FAKE, dz, dw, ws, n, None)
    assert b(n=need - 1) == WORKSPACE and b(ws=None) == WORKSPACE
    assert b(z=FAKE) == INVALID and b(dw=None) == INVALID and b(dz=FAKE + 4, z=FAKE) == MISALIGNED


def test_residual_norm_refusals(lib):
    def p(**kw):
        return ssm.residual_norm_params(**{**dict(weight=FAKE, samples=1, alpha=1.0), **kw})

    f = lambda d=nd(), q=p(), x=FAKE, r=FAKE, ro=FAKE, out=FAKE: lib.residual_norm_fwd(   # noqa: E731
        ref(d), ref(q) if q else None, x, r, ro, out, None)
    assert f(q=None) == INVALID and f(q=p(weight=None)) == INVALID and f(q=p(samples=0)) == INVALID
    assert f(q=p(alpha=float("inf"))) == INVALID
    assert f(x=None) == INVALID and f(ro=None) == INVALID and f(out=None) == INVALID
    assert f(d=nd(dim=64, group=32)) == SHAPE and f(q=p(samples=3)) == SHAPE
    assert f(q=p(scale=FAKE + 4)) == MISALIGNED and f(r=FAKE + 2) == MISALIGNED
    q = p(scale=FAKE, samples=2)
    need = lib.residual_norm_bwd_workspace_size(ref(nd()), ref(q))

    def b(q=q, x=FAKE, ws=FAKE, n=need, **kw):
        g = ssm.residual_norm_grads(**{**dict(dx=FAKE, dweight=FAKE, dscale=FAKE), **kw})
        return lib.residual_norm_bwd(ref(nd()), ref(q), x, FAKE, FAKE, None, ref(g), ws, n, None)

    assert b(x=None) == INVALID and b(dscale=None) == INVALID and b(dx=None) == INVALID and b(dweight=None) == INVALID
    assert b(n=need - 1) == WORKSPACE and b(ws=FAKE + 4) == MISALIGNED
    assert b(q=p(bias=FAKE)) == INVALID and b(q=p(post_weight=FAKE)) == INVALID
    assert lib.residual_norm_bwd_workspace_size(ref(nd(dim=60)), ref(q)) == 0


def test_gdr_forward_needs_no_workspace(lib):
    """Sizes of every kind; so none can be too small or misaligned."""
    for d in (dims(), dims(L=1), dims(L=100000, K=64), dims(B=300, Hv=96, Hk=1, V=128), dims(B=0), dims(L=0)):
        assert lib.gdr_chunk_workspace_size(ref(d)) == 0
    assert fwd(lib, dims(L=0), inputs(q=None), out=None, ws=FAKE + 4, n=3) == OK
    assert fwd(lib, dims(L=4096), inputs(), out=None) == INVALID   # the first that it finds wrong without one


def test_python_refusals():
    """The binding says what is wrong with CPU tensors before any library call."""
    t = torch.zeros(1, 4, 1, 64, dtype=torch.bfloat16)
    g = torch.zeros(1, 4, 1, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        ssm.gdr_chunk_fwd(t, t, t, g, torch.zeros(1), g)
    with pytest.raises(ValueError, match="CUDA"):
        ssm.gated_norm_fwd(t, torch.ones(64))
