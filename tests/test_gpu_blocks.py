"""The gated delta rule and the norms together, as a block uses them: forward
and backward through residual norm, projections, delta rule, gated norm and
the next residual norm; a prompt, then tokens; calls on two streams at once.

Tolerance of the whole block, fixed before the first run: every value between
two operators is rounded to bf16 (half a step 2^-8, about 2^-9 in the mean
square); a gradient passes up to 16 such roundings, whose errors add up to at
most 16 2^-9 = 2^-5 in the 2-norm.
"""
import pytest
import torch

import selective_state_space_24_b200 as ssm
from oracle import blocks as ob

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
B, L, D, HK, HV, K, V = 2, 100, 256, 2, 4, 64, 64
SPLIT = [HK * K, HK * K, HV * V, HV, HV, HV * V]   # q, k, v, delta, beta, z


def _weights(gen):
    r = lambda *s, std=1.0: std * torch.randn(*s, generator=gen)   # noqa: E731
    w = dict(x=r(B, L, D).to(BF16), res=r(B, L, D), w1=1 + 0.1 * r(D), win=r(D, sum(SPLIT), std=D ** -0.5).to(BF16),
             A=-(1 + 15 * torch.rand(HV, generator=gen)), bias=r(HV) - 3, wn=1 + 0.1 * r(V), wo=r(HV * V, D, std=D ** -0.5).to(BF16),
             scale=0.5 + 0.1 * r(D), w2=1 + 0.1 * r(D))
    return w, r(B, L, D).to(BF16), r(B, L, D)


def _heads(t, b=B, l=L):
    q, k, v, delta, beta, z = t.split(SPLIT, -1)
    return (q.reshape(b, l, HK, K), k.reshape(b, l, HK, K), v.reshape(b, l, HV, V), delta, beta, z.reshape(b, l, HV, V))


def _oracle(w):
    """The block on float64 tensors: the next block's input and the stream."""
    r1 = ob.residual_update(w["x"], residual=w["res"])
    q, k, v, delta, beta, z = _heads(ob.norm(r1, w["w1"]) @ w["win"])
    o, _ = ob.gdr(q, k, v, delta, w["A"], beta, delta_bias=w["bias"])
    y = ob.gated_norm(o, w["wn"], z=z, norm_before_gate=True)
    r2 = ob.residual_update(y.reshape(B, L, -1) @ w["wo"], residual=r1, scale=w["scale"])
    return ob.norm(r2, w["w2"]), r2


def _far(got, want):
    g, o = got.detach().double().cpu(), want.detach()
    assert g.shape == o.shape and bool(torch.isfinite(g).all())
    return float((g - o).norm() / o.norm())


def test_block_forward_and_backward(cuda_device):
    w, dh2, dr2 = _weights(torch.Generator().manual_seed(0))
    c = {n: t.cuda() for n, t in w.items()}
    c64 = lambda t: t.contiguous()   # noqa: E731
    h1, r1 = ssm.residual_norm_fwd(c["x"], c["w1"], residual=c["res"])
    q, k, v, delta, beta, z = (c64(t) for t in _heads(h1 @ c["win"]))
    o = ssm.gdr_chunk_fwd(q, k, v, delta, c["A"], beta, delta_bias=c["bias"])
    y = ssm.gated_norm_fwd(o, c["wn"], z=z, norm_before_gate=True)
    p = y.view(B, L, -1) @ c["wo"]
    h2, r2 = ssm.residual_norm_fwd(p, c["w2"], residual=r1, scale=c["scale"])

    g2 = ssm.residual_norm_bwd(p, r2, c["w2"], dh2.cuda(), dresidual_out=dr2.cuda(), scale=c["scale"])
    dy = (g2["dx"] @ c["wo"].t()).view(y.shape)
    gn = ssm.gated_norm_bwd(o, c["wn"], dy, z=z, norm_before_gate=True)
    gd = ssm.gdr_chunk_bwd(q, k, v, delta, c["A"], beta, gn["dx"], delta_bias=c["bias"])
    flat = torch.cat([t.reshape(B, L, -1) for t in (gd["dq"], gd["dk"], gd["dv"], gd["ddelta"], gd["dbeta"], gn["dz"])], -1)
    g1 = ssm.residual_norm_bwd(c["x"], r1, c["w1"], flat @ c["win"].t(), dresidual_out=g2["dresidual"])
    got = dict(x=g1["dx"], res=g1["dresidual"], w1=g1["dweight"], A=gd["dA"], bias=gd["ddelta_bias"], wn=gn["dweight"],
               scale=g2["dscale"], w2=g2["dweight"], wo=y.view(B * L, -1).t() @ g2["dx"].view(B * L, -1),
               win=h1.view(B * L, -1).t() @ flat.view(B * L, -1))
    torch.cuda.synchronize()
    ssm.check_device()

    t = {n: ob.f64(x, True) for n, x in w.items()}
    ro, rr = _oracle(t)
    assert _far(h2, ro) <= 2 ** -5 and _far(r2, rr) <= 2 ** -5
    total = (ro * dh2.double()).sum() + (rr * dr2.double()).sum()
    for n, want in zip(t, torch.autograd.grad(total, list(t.values()))):
        assert _far(got[n], want) <= 2 ** -5, n


@pytest.mark.parametrize("prompt", [1, 5, 64, 90])
def test_prompt_then_tokens(cuda_device, prompt):
    """A prompt's last state goes on token by token: the whole sequence's outputs and state."""
    gen = torch.Generator().manual_seed(prompt)
    n = prompt + 6
    r = lambda *s: torch.randn(*s, generator=gen)   # noqa: E731
    x = dict(q=r(B, n, HK, K).to(BF16), k=r(B, n, HK, K).to(BF16), v=r(B, n, HV, V).to(BF16), delta=r(B, n, HV).to(BF16),
             beta=r(B, n, HV).to(BF16), A=-(1 + 15 * torch.rand(HV, generator=gen)))
    bias = r(HV) - 3
    c = {m: t.cuda() for m, t in x.items()}
    part = lambda a, b: [c[m] if m == "A" else c[m][:, a:b].contiguous() for m in ("q", "k", "v", "delta", "A", "beta")]   # noqa: E731
    state = torch.zeros(B, HV, V, K, device="cuda")
    out = [ssm.gdr_chunk_fwd(*part(0, prompt), delta_bias=bias.cuda(), initial_state=state, last_state=state)]
    for t in range(prompt, n):
        tok = [p if p.dim() == 1 else p[:, 0] for p in part(t, t + 1)]
        out.append(ssm.gdr_step(*tok, state, delta_bias=bias.cuda()).unsqueeze(1))
    ro, rs = ob.gdr(**{m: ob.f64(t) for m, t in x.items()}, delta_bias=ob.f64(bias))
    assert _far(torch.cat(out, 1), ro) <= 2 ** -7 and _far(state, rs) <= 2e-5


def _bwd_args(seed):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)   # noqa: E731
    return [t.cuda() for t in (r(1, 150, HK, K).to(BF16), r(1, 150, HK, K).to(BF16), r(1, 150, HV, V).to(BF16),
                               r(1, 150, HV).to(BF16), -(1 + torch.rand(HV, generator=gen)), r(1, 150, HV).to(BF16),
                               r(1, 150, HV, V).to(BF16))]


def test_two_streams_at_once(cuda_device):
    """Calls on two streams, forward and backward, overlap without touching one another."""
    args = [_bwd_args(s) for s in (1, 2)]
    want = [(ssm.gdr_chunk_fwd(*a[:6]), ssm.gdr_chunk_bwd(*a)) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append((ssm.gdr_chunk_fwd(*args[i][:6]), ssm.gdr_chunk_bwd(*args[i])))
    torch.cuda.synchronize()
    for i in range(2):
        for o, g in got[i]:
            assert torch.equal(o, want[i][0])
            for n in g:
                assert torch.equal(g[n], want[i][1][n]), n


def test_backward_captured_and_replayed(cuda_device):
    a = _bwd_args(3)
    ssm.gdr_chunk_bwd(*a)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g = ssm.gdr_chunk_bwd(*a)
    a[2].copy_(a[2].flip(1))
    a[6].copy_(a[6].flip(1))
    graph.replay()
    want = ssm.gdr_chunk_bwd(*a)
    for n in g:
        assert torch.equal(g[n], want[n]), n


def test_explicit_stream_keeps_its_memory(cuda_device):
    """Results and workspaces made for another stream are not handed out again before it is done with them."""
    a = _bwd_args(4)
    want = ssm.gdr_chunk_bwd(*a)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(5):
        g = ssm.gdr_chunk_bwd(*a, stream=s)
        for _ in range(3):   # would land in a freed workspace
            torch.full((1 << 20,), float("nan"), device="cuda")
        s.synchronize()
        for n in g:
            assert torch.equal(g[n], want[n]), n


def test_explicit_stream_and_memory_still_in_use(cuda_device):
    """Memory that the current stream has freed but not finished with is not used on the other stream."""
    a = _bwd_args(6)
    want = ssm.gdr_chunk_bwd(*a)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    torch.cuda._sleep(40_000_000)   # some 20 ms
    for n in (1 << 18, 1 << 20, 1 << 22, 1 << 24):
        torch.full((n,), float("nan"), device="cuda")
    g = ssm.gdr_chunk_bwd(*a, stream=s)
    torch.cuda.synchronize()
    for n in g:
        assert torch.equal(g[n], want[n]), n


def test_unit_scale_zero_and_shared_inputs(cuda_device):
    """q and k the same tensor; a zero scale gives zero outputs and finite gradients."""
    a = _bwd_args(5)
    a[1] = a[0]
    o = ssm.gdr_chunk_fwd(*a[:6], scale=0.0)
    assert not o.any()
    g = ssm.gdr_chunk_bwd(*a, scale=0.0)
    assert not g["dq"].any() and all(bool(torch.isfinite(t).all()) for t in g.values())


# ---- more than 2^31 elements: the last part against a call of its own

def _tail(x, lo, hi):
    return x[lo:hi].clone()   # not a view: a state is updated in place


def test_long_sequences_beyond_32_bit_offsets(cuda_device):
    B, L, Hk, Hv, K, V = 3, 64 * 2750, 1, 64, 64, 64   # v: 2.16e9 elements
    gen = torch.Generator(device="cuda").manual_seed(11)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=BF16)   # noqa: E731
    x = [r(B, L, Hk, K), r(B, L, Hk, K), r(B, L, Hv, V), r(B, L, Hv), -1 - torch.rand(Hv, device="cuda", generator=gen),
         r(B, L, Hv)]
    assert x[2].numel() > 2 ** 31
    last = torch.empty(B, Hv, V, K, device="cuda")
    out = ssm.gdr_chunk_fwd(*x, last_state=last)
    own = torch.empty(1, Hv, V, K, device="cuda")
    want = ssm.gdr_chunk_fwd(*(t if t.dim() == 1 else _tail(t, B - 1, B) for t in x), last_state=own)
    assert torch.equal(out[B - 1:], want) and torch.equal(last[B - 1:], own)
    ssm.check_device()


def test_backward_workspace_beyond_32_bit_offsets(cuda_device):
    B, L, Hk, Hv, K, V = 3, 64 * 800, 2, 16, 128, 128   # 38400 chunks and heads of 61,696 floats
    gen = torch.Generator(device="cuda").manual_seed(12)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=BF16)   # noqa: E731
    x = [r(B, L, Hk, K), r(B, L, Hk, K), r(B, L, Hv, V), r(B, L, Hv), -1 - torch.rand(Hv, device="cuda", generator=gen),
         r(B, L, Hv), r(B, L, Hv, V)]
    g = ssm.gdr_chunk_bwd(*x)
    w = ssm.gdr_chunk_bwd(*(t if t.dim() == 1 else _tail(t, B - 1, B) for t in x))
    for n in ("dq", "dk", "dv", "ddelta", "dbeta"):
        assert torch.equal(g[n][B - 1:], w[n]), n


def test_states_beyond_32_bit_offsets(cuda_device):
    B, Hk, Hv, K, V = 1040, 8, 128, 128, 128   # 2.18e9 state elements
    gen = torch.Generator(device="cuda").manual_seed(13)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=BF16)   # noqa: E731
    x = [r(B, Hk, K), r(B, Hk, K), r(B, Hv, V), r(B, Hv), -torch.ones(Hv, device="cuda"), r(B, Hv)]
    state = torch.randn(B, Hv, V, K, generator=gen, device="cuda")
    own = _tail(state, B - 8, B)
    out = ssm.gdr_step(*x, state)
    want = ssm.gdr_step(*(t if t.dim() == 1 else _tail(t, B - 8, B) for t in x), own)
    assert torch.equal(out[B - 8:], want) and torch.equal(state[B - 8:], own)


def test_norms_beyond_32_bit_offsets(cuda_device):
    rows, dim = (1 << 20) + 64, 2048
    gen = torch.Generator(device="cuda").manual_seed(14)
    x = torch.randn(rows, dim, generator=gen, device="cuda", dtype=BF16)
    w = torch.rand(dim, device="cuda") + 0.5
    z, end = x.flip(1), slice(rows - 64, rows)
    y = ssm.gated_norm_fwd(x, w, z=z, group=256)
    assert torch.equal(y[end], ssm.gated_norm_fwd(x[end].contiguous(), w, z=z[end].contiguous(), group=256))
    g = ssm.gated_norm_bwd(x, w, y, z=z, group=256)
    own = ssm.gated_norm_bwd(x[end].contiguous(), w, y[end].contiguous(), z=z[end].contiguous(), group=256)
    assert torch.equal(g["dx"][end], own["dx"]) and torch.equal(g["dz"][end], own["dz"])
    del g, z
    y, ro = ssm.residual_norm_fwd(x, w, layer_norm=True)
    y2, ro2 = ssm.residual_norm_fwd(x[end].contiguous(), w, layer_norm=True)
    assert torch.equal(y[end], y2) and torch.equal(ro[end], ro2)
    g = ssm.residual_norm_bwd(x, ro, w, y, layer_norm=True)
    own = ssm.residual_norm_bwd(x[end].contiguous(), ro2, w, y2, layer_norm=True)
    assert torch.equal(g["dx"][end], own["dx"]) and torch.equal(g["dresidual"][end], own["dresidual"])
