"""The gated delta rule on the GPU against the float64 oracle.

Tolerances, fixed before the first run.  bf16 results: the library's bar of
2e-2 of max(|o|, rms), and in the 2-norm 2^-7: one rounding of the result and
two of each product's operands, each at most half a step (2^-8) and about
2^-9 in the mean square, the products' energy at most twice the sum's.
float32 results: operands carry at least 16 bits (2^-17 each, three of them
per product, the products' energy at most twice the sum's) and the scalars a
few float32 steps: 2e-5 in the 2-norm, 1e-4 of max(|o|, rms) for the largest
of up to 1e6 elements (five standard deviations).
"""
import pytest
import torch

import selective_state_space_24_b200 as ssm
from gpu_util import host, rel_err
from oracle import blocks as ob

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def make(B, L, Hk, Hv, K, V, seed=0, dtype=BF16, init=False, A=None, beta=None, delta=None, step=False):
    gen = torch.Generator().manual_seed(seed)
    lead = (B,) if step else (B, L)
    r = lambda *s: torch.randn(*s, generator=gen)   # noqa: E731
    x = dict(q=r(*lead, Hk, K), k=r(*lead, Hk, K), v=r(*lead, Hv, V), delta=0.5 * r(*lead, Hv), beta=r(*lead, Hv))
    x = {n: t.to(dtype) for n, t in x.items()}
    if delta is not None:
        x["delta"] = torch.full_like(x["delta"], delta)
    if beta is not None:
        x["beta"] = torch.full_like(x["beta"], beta)
    x["A"] = -(1 + 15 * torch.rand(Hv, generator=gen)) if A is None else torch.full((Hv,), float(A))
    x["delta_bias"] = -3.0 + r(Hv)
    x["initial_state"] = 0.3 * r(B, Hv, V, K) if init or step else None
    return x


def cuda(x):
    return {n: t.cuda() if isinstance(t, torch.Tensor) else t for n, t in x.items()}


def f64(x, grad=False):
    return {n: ob.f64(t, grad) if isinstance(t, torch.Tensor) else t for n, t in x.items()}


def close(got, want, f32, spread=1.0):
    """spread: how much larger the root of the products' energy is, relative to the sum's, than twice (see above)."""
    g, o = host(got), want.detach().numpy()
    assert g.shape == o.shape
    if o.size == 0:
        return
    n = float((o * o).sum()) ** 0.5
    two = float(((g - o) ** 2).sum()) ** 0.5
    assert two <= (2e-5 if f32 else 2 ** -7) * spread * n + 1e-30, (two, n)
    assert rel_err(g, o) <= (1e-4 if f32 else 2e-2) * spread


def run_fwd(x, flags):
    c = cuda(x)
    B, Hv, V, K = x["v"].shape[0], x["v"].shape[2], x["v"].shape[3], x["q"].shape[3]
    last = torch.full((B, Hv, V, K), 7.0, device="cuda")
    args = [c.pop(n) for n in ("q", "k", "v", "delta", "A", "beta")]
    out = ssm.gdr_chunk_fwd(*args, last_state=last, **c, **flags)
    torch.cuda.synchronize()
    ssm.check_device()
    return out, last


FLAGS = [dict(), dict(beta_sigmoid=False, delta_softplus=False, scale=0.5), dict(qk_l2norm=False)]


def condition(x, flags):
    """Inputs a flag asks for: unit keys without the norm, strengths and steps in range without the maps."""
    if flags.get("qk_l2norm") is False:
        for n in ("q", "k"):
            x[n] = (x[n].float() / x[n].float().norm(dim=-1, keepdim=True)).to(x[n].dtype)
    if flags.get("beta_sigmoid") is False:
        x["beta"] = torch.sigmoid(x["beta"].float()).to(x["beta"].dtype)
    if flags.get("delta_softplus") is False:
        x["delta"] = (0.05 * torch.sigmoid(x["delta"].float())).to(x["delta"].dtype)
        x["delta_bias"] = None
    return x


SIZES = [(1, 1, 1, 1, 64, 64), (2, 2, 1, 2, 128, 128), (1, 15, 2, 2, 64, 128), (1, 63, 2, 4, 128, 64),
         (2, 64, 1, 1, 64, 64), (1, 65, 1, 3, 128, 128), (2, 130, 2, 2, 64, 64), (1, 200, 2, 4, 128, 128),
         (3, 256, 1, 1, 128, 64), (1, 1000, 1, 2, 64, 128)]


@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("flags", range(len(FLAGS)))
@pytest.mark.parametrize("init", [False, True])
def test_forward(cuda_device, size, flags, init):
    flags = FLAGS[flags]
    x = condition(make(*size, seed=sum(size), init=init), flags)
    out, last = run_fwd(x, flags)
    ro, rs = ob.gdr(**f64(x), **flags)
    close(out, ro, False)
    close(last, rs, True)


HARD = {
    "no decay": dict(A=0.0), "strong decay": dict(A=-16.0, delta=4.0), "decay to nothing": dict(A=-1e4, delta=4.0),
    "writes nothing": dict(beta=-100.0), "writes all": dict(beta=100.0),
}


@pytest.mark.parametrize("name", HARD)
def test_forward_ranges(cuda_device, name):
    x = make(1, 150, 1, 2, 128, 128, seed=3, init=True, **HARD[name])
    out, last = run_fwd(x, {})
    ro, rs = ob.gdr(**f64(x))
    close(out, ro, False)
    if float(rs.abs().max()) > 1e-30:
        close(last, rs, True)


@pytest.mark.parametrize("L", [96, 500])
def test_forward_same_key_again(cuda_device, L):
    """One key for every step, full strength: (I + A) is all ones below the diagonal.
    The state is then the last value alone, but a chunk adds it up from 64
    terms v_j - v_(j-1) of twice that energy: 128 times the sum's where two
    are assumed above, so the state may be off by the root of 64 times as much."""
    x = make(1, L, 1, 1, 128, 64, seed=5, beta=100.0, A=-0.01)
    x["k"][:] = x["k"][:, :1]
    x["q"][:] = x["k"]
    out, last = run_fwd(x, {})
    ro, rs = ob.gdr(**f64(x))
    close(out, ro, False)
    close(last, rs, True, spread=8.0)


def test_forward_zero_vectors(cuda_device):
    x = make(1, 100, 1, 1, 64, 64, seed=6)
    x["k"][:, 10:70] = 0
    x["q"][:, 5:20] = 0
    out, last = run_fwd(x, {})
    ro, rs = ob.gdr(**f64(x))
    close(out, ro, False)
    close(last, rs, True)


def test_forward_in_place_pieces_and_repeat(cuda_device):
    """A sequence in pieces with the state updated in place gives the whole's results; twice the same gives the same bits."""
    x = make(2, 300, 1, 2, 128, 128, seed=7, init=True)
    out, last = run_fwd(x, {})
    again, last2 = run_fwd(x, {})
    assert torch.equal(out, again) and torch.equal(last, last2)
    c = cuda(x)
    st = c.pop("initial_state").clone()
    outs = []
    for a, b in ((0, 70), (70, 71), (71, 199), (199, 300)):
        p = {n: t if n in ("A", "delta_bias") else t[:, a:b].contiguous() for n, t in c.items()}
        outs.append(ssm.gdr_chunk_fwd(*[p.pop(n) for n in ("q", "k", "v", "delta", "A", "beta")], initial_state=st,
                                      last_state=st, **p))
    ro, rs = ob.gdr(**f64(x))
    close(torch.cat(outs, 1), ro, False)
    close(st, rs, True)


def test_forward_padded_positions_leave_the_state(cuda_device):
    x = make(1, 200, 1, 1, 64, 64, seed=8, init=True)
    x["delta_bias"] = None
    x["delta"] = x["delta"].abs()
    x["beta"] = torch.sigmoid(x["beta"].float()).to(BF16)
    x["delta"][:, 130:] = 0
    x["beta"][:, 130:] = 0
    kw = dict(delta_softplus=False, beta_sigmoid=False)
    _, padded = run_fwd(x, kw)
    cut = {n: t[:, :130].contiguous() if n in ("q", "k", "v", "delta", "beta") else t for n, t in x.items()}
    close(padded, ob.gdr(**f64(cut), **kw)[1], True)


def test_empty_calls(cuda_device):
    x = make(2, 0, 1, 2, 64, 64, init=True)
    out, last = run_fwd(x, {})
    assert out.shape == (2, 0, 2, 64) and torch.equal(last.cpu(), x["initial_state"])
    x["initial_state"] = None
    assert not run_fwd(x, {})[1].any()
    g = run_bwd(make(1, 0, 1, 2, 64, 64, init=True), torch.zeros(1, 0, 2, 64, dtype=BF16), torch.ones(1, 2, 64, 64))
    assert not g["dA"].any() and not g["ddelta_bias"].any() and bool((g["dinitial_state"] == 1).all())


def test_no_value_heads(cuda_device):
    x = make(2, 70, 2, 0, 64, 64)
    g = run_bwd(x, torch.zeros(2, 70, 0, 64, dtype=BF16))
    assert g["dq"].shape == (2, 70, 2, 64) and not g["dq"].any() and not g["dk"].any()


def test_state_and_streams(cuda_device):
    """Another stream, and a captured call replayed on new inputs."""
    x = cuda(make(1, 150, 2, 2, 64, 64, seed=9))
    args = [x.pop(n) for n in ("q", "k", "v", "delta", "A", "beta")]
    x.pop("initial_state")
    want = ssm.gdr_chunk_fwd(*args, **x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = ssm.gdr_chunk_fwd(*args, **x, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ssm.gdr_chunk_fwd(*args, **x)
    args[2].copy_(torch.randn_like(args[2].float()).to(BF16))
    graph.replay()
    assert torch.equal(out, ssm.gdr_chunk_fwd(*args, **x))


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("size", [(1, 1, 1, 64, 64), (3, 2, 6, 128, 128), (5, 1, 1, 128, 64), (2, 3, 3, 64, 128)], ids=str)
@pytest.mark.parametrize("flags", range(len(FLAGS)))
def test_step(cuda_device, dtype, size, flags):
    flags = FLAGS[flags]
    B, Hk, Hv, K, V = size
    x = condition(make(B, 1, Hk, Hv, K, V, seed=sum(size), dtype=dtype, step=True), flags)
    c = cuda(x)
    state = c.pop("initial_state")
    want = f64(x)
    st = want.pop("initial_state")
    for _ in range(3):
        out = ssm.gdr_step(*[c[n] for n in ("q", "k", "v", "delta", "A", "beta")], state, delta_bias=c["delta_bias"],
                           **flags)
        ro, st = ob.gdr(**{n: t if n in ("A", "delta_bias") or t is None else t.unsqueeze(1) for n, t in want.items()},
                        initial_state=st, **flags)
    close(out, ro[:, 0], dtype == torch.float32)
    close(state, st, True)


def run_bwd(x, dout, dlast=None, flags={}):
    c = cuda(x)
    args = [c.pop(n) for n in ("q", "k", "v", "delta", "A", "beta")]
    g = ssm.gdr_chunk_bwd(*args, dout.cuda(), dlast_state=None if dlast is None else dlast.cuda(), **c, **flags)
    torch.cuda.synchronize()
    ssm.check_device()
    return g


def check_bwd(x, flags, seed=1, dlast=False, spread=1.0):
    gen = torch.Generator().manual_seed(seed)
    dout = torch.randn(x["v"].shape, generator=gen).to(BF16)
    B, _, Hv, V = x["v"].shape
    dl = 0.2 * torch.randn(B, Hv, V, x["q"].shape[3], generator=gen) if dlast else None
    g = run_bwd(x, dout, dl, flags)
    t = f64(x, grad=True)
    out, S = ob.gdr(**t, **flags)
    total = (out * dout.double()).sum() + (0 if dl is None else (S * dl.double()).sum())
    names = {"dq": "q", "dk": "k", "dv": "v", "ddelta": "delta", "dbeta": "beta", "dA": "A",
             "ddelta_bias": "delta_bias", "dinitial_state": "initial_state"}
    names = {n: m for n, m in names.items() if t[m] is not None}
    assert set(g) == set(names)
    ref = dict(zip(names, torch.autograd.grad(total, [t[m] for m in names.values()])))
    for n in names:
        assert torch.isfinite(g[n]).all(), n
        try:
            close(g[n], ref[n], g[n].dtype == torch.float32, spread=spread if g[n].dtype == torch.float32 else 1.0)
        except AssertionError as e:
            raise AssertionError(f"{n}: {e}") from e


@pytest.mark.parametrize("size", SIZES[:8], ids=str)
@pytest.mark.parametrize("flags", range(len(FLAGS)))
@pytest.mark.parametrize("init", [False, True])
def test_backward(cuda_device, size, flags, init):
    flags = FLAGS[flags]
    check_bwd(condition(make(*size, seed=sum(size), init=init), flags), flags, dlast=init)


@pytest.mark.parametrize("name", ["no decay", "strong decay", "writes all"])
def test_backward_ranges(cuda_device, name):
    check_bwd(make(1, 150, 1, 2, 128, 128, seed=3, init=True, **HARD[name]), {})


def _packed(seed):
    """Three sequences in one: a step so long that nothing stays starts the second and the third.
    Log2 decays then reach 2 * 150 within a chunk; each of their sums' up to 7 additions is off by at
    most half a step there, 2^-16, and a decay is the difference of two: 14 * 2^-16 ln 2 = 1.5e-4
    relative, 7.4 times the 2e-5 above, on top of it."""
    x = make(2, 150, 1, 2, 128, 128, seed=seed, init=True)
    x["delta"][:, [70, 101]] = 1e4
    return x


def test_forward_packed_sequences(cuda_device):
    x = _packed(8)
    out, last = run_fwd(x, {})
    ro, rs = ob.gdr(**f64(x))
    close(out, ro, False)
    close(last, rs, True, spread=8.4)
    own, _ = run_fwd({n: t[:, 101:].contiguous() if isinstance(t, torch.Tensor) and t.dim() > 2 and n != "initial_state"
                      else t for n, t in x.items()}, {})
    close(out[:, 101:], own.double().cpu(), False)


def test_backward_packed_sequences(cuda_device):
    x = _packed(9)
    check_bwd(x, {}, spread=8.4)
    dout = torch.zeros(x["v"].shape, dtype=BF16)
    dout[:, 101:] = 1.0
    g = run_bwd(x, dout)
    assert not any(g[n][:, :101].any() for n in ("dq", "dk", "dv", "ddelta", "dbeta")) and not g["dinitial_state"].any()


def test_backward_repeats(cuda_device):
    x = make(2, 200, 2, 4, 64, 128, seed=4, init=True)
    dout = torch.randn(2, 200, 4, 128, generator=torch.Generator().manual_seed(2)).to(BF16)
    a, b = run_bwd(x, dout), run_bwd(x, dout)
    for n in a:
        assert torch.equal(a[n], b[n]), n


def test_python_refusals(cuda_device):
    x = cuda(make(1, 8, 1, 1, 64, 64))
    args = [x.pop(n) for n in ("q", "k", "v", "delta", "A", "beta")]
    bad = lambda i, t: [t if j == i else a for j, a in enumerate(args)]   # noqa: E731
    for i, t in ((1, args[1][:, :4]), (2, args[2].float()), (3, args[3][..., None]), (4, args[4].double()),
                 (5, args[5].cpu()), (0, args[0].transpose(1, 2))):
        with pytest.raises((ValueError, TypeError)):
            ssm.gdr_chunk_fwd(*bad(i, t))
    wide = torch.zeros(1, 8, 1, 96, device="cuda", dtype=BF16)
    with pytest.raises(ssm.SSMError, match="UNSUPPORTED_SHAPE"):
        ssm.gdr_chunk_fwd(wide, wide, *args[2:])
    with pytest.raises((ValueError, TypeError)):
        ssm.gdr_chunk_fwd(*args, initial_state=torch.zeros(1, 1, 64, 64, device="cuda", dtype=BF16))


@pytest.mark.parametrize("every", [4, 8, 23])
def test_many_short_packed_sequences(cuda_device, every):
    """A step that forgets everything every few steps: log decays that have reached thousands leave the
    decays between neighbours their low bits, and the tolerances stay as they are."""
    x = make(1, 200, 1, 2, 128, 128, seed=every, init=True)
    x["delta"][:, every::every] = 1e4
    out, last = run_fwd(x, {})
    ro, rs = ob.gdr(**f64(x))
    close(out, ro, False)
    close(last, rs, True)
    check_bwd(x, {})


@pytest.mark.parametrize("size", [(1, 320, 4, 8, 128, 128), (2, 200, 8, 8, 64, 64)], ids=str)
def test_sums_over_steps_keep_float32(cuda_device, size):
    """dA and ddelta_bias to 1e-6 in the 2-norm.  Two tf32 parts, the first rounded, leave at most 2^-11 and then
    2^-22 of the value, about 2^-24 in the mean square; the product of two second parts, which is left out, is
    2^-22 at most and as much in the mean.  With float32's own additions some 1.5e-7 a product,
    without a sign of its own, and ten products in a row from the inputs to these sums: 5e-7; twice that is asked."""
    x = make(*size, seed=21, init=True)
    gen = torch.Generator().manual_seed(3)
    dout = torch.randn(x["v"].shape, generator=gen).to(BF16)
    g = run_bwd(x, dout)
    t = f64(x, grad=True)
    out, _ = ob.gdr(**t)
    for n, w in zip(("dA", "ddelta_bias"), torch.autograd.grad((out * dout.double()).sum(), [t["A"], t["delta_bias"]])):
        far = float((g[n].double().cpu() - w).norm() / w.norm())
        assert far <= 1e-6, (n, far)


@pytest.mark.parametrize("softplus", [True, False])
def test_infinite_step_between_packed_sequences(cuda_device, softplus):
    """delta = inf forgets like any other step that leaves nothing: the bits of 1e4, in the sums over steps too."""
    x = make(1, 150, 1, 2, 128, 64, seed=12, init=True)
    x["delta"] = x["delta"].abs()
    if not softplus:   # dt = delta, not negative
        x["delta_bias"] = None
    flags = dict(delta_softplus=softplus)
    dout = torch.randn(x["v"].shape, generator=torch.Generator().manual_seed(2)).to(BF16)
    got = []
    for step in (1e4, float("inf")):
        x["delta"][:, [70, 101]] = step
        got.append(run_bwd(x, dout, flags=flags) | dict(zip(("out", "last"), run_fwd(x, flags))))
    for n in got[0]:
        assert torch.isfinite(got[1][n]).all(), n
        assert torch.equal(got[0][n], got[1][n]), n


@pytest.mark.parametrize("K", [64, 128])
@pytest.mark.parametrize("chunk", [0, 2, 4])
def test_device_timeout_is_reported_and_the_next_call_is_clean(cuda_device, K, chunk):
    """A bounded wait that runs out: the gates of one chunk are never signalled (nothing else gives that signal),
    and every wait ends after 4096 polls.  The call completes: it waits for the copies and products that it issued
    and frees its tensor memory.  ssm_check_device reports it once, and the next call gives the bits of the one before."""
    lib = ssm.capi()
    x = make(2, 320, 1, 3, K, 128, seed=31, init=True)
    want = run_fwd(x, {})
    c = cuda(x)
    args = [c.pop(n) for n in ("q", "k", "v", "delta", "A", "beta")]
    last = torch.full((2, 3, 128, K), 7.0, device="cuda")
    lib.ssm_debug_gdr_stall(chunk, 1 << 12)
    try:
        ssm.gdr_chunk_fwd(*args, last_state=last, **c)
        status = lib.ssm_check_device(torch.cuda.current_stream().cuda_stream)
    finally:
        lib.ssm_debug_gdr_stall(-1, 0)
    assert status == 7, ssm.STATUS.get(status, status)
    assert lib.ssm_check_device(torch.cuda.current_stream().cuda_stream) == 0   # cleared
    assert bool((last == 7.0).all())
    out, again = run_fwd(x, {})
    assert torch.equal(out, want[0]) and torch.equal(again, want[1])


@pytest.mark.parametrize("L", [10, 11, 13, 14, 15, 25, 26, 27])
@pytest.mark.parametrize("heads", [3, 40])
def test_forward_lengths_around_the_step_by_step_limits(cuda_device, L, heads):
    """Few and many blocks of state rows, on both sides of where the chunks begin."""
    for K in (64, 128):
        x = make(1, L, 1, heads, K, 128, seed=L, init=True)
        out, last = run_fwd(x, {})
        ro, rs = ob.gdr(**f64(x))
        close(out, ro, False)
        close(last, rs, True)
