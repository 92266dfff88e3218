"""The norms around a block on the GPU against the float64 oracle.

Tolerances, fixed before the first run: a bf16 result is rounded once (half a
step, 2^-8 of its value) on top of float32 arithmetic; float32 arithmetic is
sums of at most 8192 products per row in a tree (a few steps of 2^-24) and
reciprocal roots and exponentials within a few steps, some 2e-6 of
max(|o|, rms) -- 1e-5 is asked.  Column sums add up to 4000 rows: 1e-5 in the
2-norm.
"""
import pytest
import torch

import selective_state_space_24_b200 as ssm
from oracle import blocks as ob

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def close(got, want, sums=False):
    g, o = got.detach().double().cpu(), want.detach()
    assert g.shape == o.shape and bool(torch.isfinite(g).all())
    if sums:
        assert float((g - o).norm()) <= 1e-5 * float(o.norm()) + 1e-30
        return
    rms = float(o.pow(2).mean().sqrt())
    step = 2 ** -8 if got.dtype == BF16 else 0.0
    # values below the smallest normal float32, 2^-126, are zero on the device
    # (and rounded by up to 2^-150 where they are kept)
    assert bool(((g - o).abs() <= step * o.abs() * (1 + 2 ** -6) + 1e-5 * o.abs().clamp(min=rms) + 2 ** -126).all())


def r(gen, *s, dtype=F32, std=1.0):
    return (std * torch.randn(*s, generator=gen)).to(dtype)


GATED = [(1, 8, 8), (3, 64, 64), (5, 128, 32), (257, 128, 128), (33, 96, 24), (7, 1000, 200), (2, 2048, 2048),
         (600, 1536, 512), (3, 8192, 8192), (4, 4096, 1024), (1500, 40, 40), (9, 4104, 4104)]


@pytest.mark.parametrize("size", GATED, ids=str)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gate,first", [(False, False), (True, False), (True, True)])
def test_gated(cuda_device, size, dtype, gate, first):
    rows, dim, group = size
    gen = torch.Generator().manual_seed(rows + dim)
    x, w, dy = r(gen, rows, dim, dtype=dtype), r(gen, dim).abs() + 0.5, r(gen, rows, dim, dtype=dtype)
    z = r(gen, rows, dim, dtype=dtype, std=2.0) if gate else None
    kw = dict(group=group, norm_before_gate=first)
    cz = None if z is None else z.cuda()
    y = ssm.gated_norm_fwd(x.cuda(), w.cuda(), z=cz, **kw)
    g = ssm.gated_norm_bwd(x.cuda(), w.cuda(), dy.cuda(), z=cz, **kw)
    t = {n: ob.f64(v, True) for n, v in (("x", x), ("weight", w), ("z", z)) if v is not None}
    o = ob.gated_norm(**t, **kw)
    close(y, o)
    ref = torch.autograd.grad(o, list(t.values()), dy.double())
    assert set(g) == {"d" + n for n in t}
    for n, want in zip(t, ref):
        close(g["d" + n], want, n == "weight")


def test_gated_values(cuda_device):
    """Rows of zeros, of huge and tiny values, gates far out; in place."""
    x = torch.zeros(6, 64)
    x[1] = 1e15
    x[2] = 1e-15
    x[3, 0] = 1.0
    x[4] = torch.arange(64.0)
    x[5] = 1.0
    z = torch.linspace(-120, 120, 64).expand(6, 64).contiguous()
    w = torch.ones(64)
    for first in (False, True):
        o = ob.gated_norm(ob.f64(x), ob.f64(w), z=ob.f64(z), norm_before_gate=first)
        xc = x.cuda()
        y = ssm.gated_norm_fwd(xc, w.cuda(), z=z.cuda(), norm_before_gate=first, out=xc)
        assert y is xc
        for k in range(6):
            close(y[k], o[k])


RESID = [(1, 1, 8), (1, 5, 64), (1, 600, 384), (2, 66, 200), (1, 3, 8192), (4, 100, 1024), (1, 333, 40), (3, 3, 2056),
         (1, 2500, 128)]
KINDS = [dict(), dict(bias=True, layer=True), dict(scale=True), dict(post=True), dict(first=True, scale=True, post=True),
         dict(bias=True, layer=True, scale=True, post=True, alpha=0.5), dict(bias=True, res="same")]


@pytest.mark.parametrize("size", RESID, ids=str)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", range(len(KINDS)))
def test_residual(cuda_device, size, dtype, kind):
    samples, rows, dim = size
    kind = KINDS[kind]
    rows -= rows % samples
    gen = torch.Generator().manual_seed(rows + dim)
    rt = dtype if kind.get("res") == "same" else F32
    x, dy, w = r(gen, rows, dim, dtype=dtype), r(gen, rows, dim, dtype=dtype), r(gen, dim).abs() + 0.5
    res = None if kind.get("first") else r(gen, rows, dim, dtype=rt, std=2.0) + 1.0
    dres = r(gen, rows, dim, dtype=rt)
    par = dict(bias=r(gen, dim) if kind.get("bias") else None, scale=r(gen, samples, dim) if kind.get("scale") else None,
               post_weight=r(gen, dim).abs() + 0.5 if kind.get("post") else None)
    c = {n: None if v is None else v.cuda() for n, v in par.items()}
    kw = dict(alpha=kind.get("alpha", 1.0), layer_norm=bool(kind.get("layer")))
    y, ro = ssm.residual_norm_fwd(x.cuda(), w.cuda(), residual=None if res is None else res.cuda(),
                                  residual_f32=rt == F32, **c, **kw)
    assert ro.dtype == rt and y.dtype == dtype
    t = {n: ob.f64(v, True) for n, v in (("x", x), ("residual", res), ("scale", par["scale"]),
                                         ("post_weight", par["post_weight"])) if v is not None}
    stream = ob.residual_update(**t, alpha=kw["alpha"])
    close(ro, stream)
    # the next norm reads the stream as it is stored
    s = ob.f64(ro, True)
    n = {"weight": ob.f64(w, True)}
    if par["bias"] is not None:
        n["bias"] = ob.f64(par["bias"], True)
    o = ob.norm(s, **n, layer_norm=kw["layer_norm"])
    close(y, o)
    g = ssm.residual_norm_bwd(x.cuda(), ro, w.cuda(), dy.cuda(), dresidual_out=dres.cuda(),
                              need_dresidual=res is not None, **c, **kw)
    got = torch.autograd.grad(o, [s] + list(n.values()), dy.double())
    ref = dict(zip(n, got[1:])) | dict(zip(t, torch.autograd.grad(stream, list(t.values()), got[0] + dres.double())))
    assert set(g) == {"d" + m for m in ref}
    for m, want in ref.items():
        close(g["d" + m], want, m not in ("x", "residual"))


def test_residual_in_place_and_without_later_uses(cuda_device):
    gen = torch.Generator().manual_seed(0)
    x, res, w = r(gen, 10, 64, dtype=BF16).cuda(), r(gen, 10, 64).cuda(), r(gen, 64).cuda()
    y, ro = ssm.residual_norm_fwd(x, w, residual=res)
    keep = res.clone()
    y2, ro2 = ssm.residual_norm_fwd(x, w, residual=res, residual_out=res)
    assert ro2 is res and torch.equal(ro2, ro) and torch.equal(y2, y) and not torch.equal(res, keep)
    dy = r(gen, 10, 64, dtype=BF16).cuda()
    a = ssm.residual_norm_bwd(x, ro, w, dy)
    b = ssm.residual_norm_bwd(x, ro, w, dy, dresidual_out=torch.zeros_like(ro))
    for n in a:
        assert torch.equal(a[n], b[n]), n


def test_layer_norm_far_from_zero(cuda_device):
    gen = torch.Generator().manual_seed(1)
    x = r(gen, 50, 512) + 1000.0
    w = torch.ones(512)
    y, ro = ssm.residual_norm_fwd(x.cuda(), w.cuda(), layer_norm=True)
    close(y, ob.norm(ob.f64(ro), ob.f64(w), layer_norm=True))


def test_norms_repeat_and_capture(cuda_device):
    gen = torch.Generator().manual_seed(2)
    x, z, w = (r(gen, 700, 256, dtype=BF16).cuda(), r(gen, 700, 256, dtype=BF16).cuda(), r(gen, 256).cuda())
    dy = r(gen, 700, 256, dtype=BF16).cuda()
    a = ssm.gated_norm_bwd(x, w, dy, z=z, group=64)
    b = ssm.gated_norm_bwd(x, w, dy, z=z, group=64)
    assert all(torch.equal(a[n], b[n]) for n in a)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = ssm.gated_norm_bwd(x, w, dy, z=z, group=64)
        y = ssm.gated_norm_fwd(x, w, z=z, group=64)
    x.copy_(x.flip(0))
    graph.replay()
    d = ssm.gated_norm_bwd(x, w, dy, z=z, group=64)
    assert all(torch.equal(c[n], d[n]) for n in c) and torch.equal(y, ssm.gated_norm_fwd(x, w, z=z, group=64))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_no_eps(cuda_device, dtype):
    """eps = 0, and fewer rows than a block works on at a time."""
    gen = torch.Generator().manual_seed(6)
    x, dy, w = r(gen, 3, 64, dtype=dtype), r(gen, 3, 64, dtype=dtype), r(gen, 64)
    a, b = ob.f64(x, True), ob.f64(w, True)
    dx, dw = torch.autograd.grad(ob.gated_norm(a, b, eps=0.0), [a, b], dy.double())
    g = ssm.gated_norm_bwd(x.cuda(), w.cuda(), dy.cuda(), eps=0.0)
    close(g["dx"], dx)
    close(g["dweight"], dw, True)
    for layer in (False, True):
        dx, dw = torch.autograd.grad(ob.norm(a, b, layer_norm=layer, eps=0.0), [a, b], dy.double())
        g = ssm.residual_norm_bwd(x.cuda(), x.cuda(), w.cuda(), dy.cuda(), layer_norm=layer, eps=0.0)
        close(g["dx"], dx)
        close(g["dweight"], dw, True)


def test_more_samples_than_blocks_in_a_column(cuda_device):
    gen = torch.Generator().manual_seed(7)
    n = 70000
    x, dy, w, s = (r(gen, n, 8).cuda(), r(gen, n, 8).cuda(), r(gen, 8).cuda(), r(gen, n, 8).cuda())
    y, ro = ssm.residual_norm_fwd(x, w, scale=s)
    assert torch.equal(ro, x * s)
    zero = torch.zeros_like(w)   # without the norm, the gradients are those of x scale
    g = ssm.residual_norm_bwd(x, ro, zero, dy, dresidual_out=dy, scale=s)
    assert torch.equal(g["dx"], dy * s) and torch.equal(g["dscale"], dy * x)


def test_empty_rows(cuda_device):
    x, w = torch.zeros(0, 64, device="cuda"), torch.ones(64, device="cuda")
    assert ssm.gated_norm_fwd(x, w).shape == (0, 64)
    assert not ssm.gated_norm_bwd(x, w, x)["dweight"].any()
    y, ro = ssm.residual_norm_fwd(x, w, residual=x)
    assert y.shape == ro.shape == (0, 64)
    g = ssm.residual_norm_bwd(x, ro, w, x, scale=w, bias=w, post_weight=w)
    assert not any(g[n].any() for n in ("dweight", "dbias", "dscale", "dpost_weight"))


def test_python_refusals(cuda_device):
    x, w = torch.zeros(4, 64, device="cuda"), torch.ones(64, device="cuda")
    for kw in (dict(z=x[:2]), dict(z=x.to(BF16)), dict(z=x.cpu()), dict(out=torch.zeros(64, 4, device="cuda").t())):
        with pytest.raises((ValueError, TypeError)):
            ssm.gated_norm_fwd(x, w, **kw)
    with pytest.raises(ssm.SSMError, match="UNSUPPORTED_SHAPE"):
        ssm.gated_norm_fwd(x, w, group=24)
    with pytest.raises(ssm.SSMError, match="UNSUPPORTED_SHAPE"):
        ssm.residual_norm_fwd(x, w, scale=torch.ones(3, 64, device="cuda"))
    with pytest.raises((ValueError, TypeError)):
        ssm.residual_norm_fwd(x, w, residual=x.to(BF16))


@pytest.mark.parametrize("dim", [8, 200, 384, 1000, 5000, 8192])
@pytest.mark.parametrize("eps", [1e-5, 1e-12])
def test_layer_norm_of_constant_rows(cuda_device, dim, eps):
    """A row of one value, however large, is zero after its mean is taken off: bias is left, finite gradients,
    and nothing in the sums over rows that the other rows did not put there."""
    gen = torch.Generator().manual_seed(dim)
    value = torch.tensor([0.0, 3.0, -0.1, 1e3, 12345.678, 1.7e6, -2.24e8, 2.24e8, 1.23e9, 7.7e12, -3.3e17, 2.0])
    x = value[:, None].expand(-1, dim).contiguous()
    x[-1] = r(gen, dim)
    w, b, dy = r(gen, dim).abs() + 0.5, r(gen, dim), r(gen, len(value), dim)
    y, ro = ssm.residual_norm_fwd(x.cuda(), w.cuda(), bias=b.cuda(), layer_norm=True, eps=eps)
    assert torch.equal(ro.cpu(), x) and bool((y[:-1] == b.cuda()).all())
    s, ws = ob.f64(x, True), ob.f64(w, True)
    o = ob.norm(s, ws, bias=ob.f64(b), layer_norm=True, eps=eps)
    close(y, o)
    g = ssm.residual_norm_bwd(x.cuda(), ro, w.cuda(), dy.cuda(), bias=b.cuda(), layer_norm=True, eps=eps)
    assert all(bool(torch.isfinite(t).all()) for t in g.values())
    only = ssm.residual_norm_bwd(x[-1:].cuda(), ro[-1:].contiguous(), w.cuda(), dy[-1:].cuda(), bias=b.cuda(), layer_norm=True,
                                 eps=eps)
    assert torch.equal(g["dweight"], only["dweight"])
    dx, _ = torch.autograd.grad(o, [s, ws], dy.double())
    for k in range(len(value)):
        close(g["dx"][k], dx[k])


def test_layer_norm_of_nearly_constant_rows(cuda_device):
    """Rows that vary by a few steps of their values: the variance is that of the values, not of the mean's rounding."""
    gen = torch.Generator().manual_seed(9)
    for dim in (200, 1000, 5000):
        x = 2.24e8 + 16.0 * torch.randint(-3, 4, (20, dim), generator=gen)
        w, dy = r(gen, dim).abs() + 0.5, r(gen, 20, dim)
        y, ro = ssm.residual_norm_fwd(x.cuda(), w.cuda(), layer_norm=True)
        s, ws = ob.f64(ro, True), ob.f64(w, True)
        o = ob.norm(s, ws, layer_norm=True)
        close(y, o)
        g = ssm.residual_norm_bwd(x.cuda(), ro, w.cuda(), dy.cuda(), layer_norm=True)
        dx, dw = torch.autograd.grad(o, [s, ws], dy.double())
        close(g["dx"], dx)
        close(g["dweight"], dw, True)
