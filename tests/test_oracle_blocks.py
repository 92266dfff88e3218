"""Pins of the float64 oracle of the gated delta rule and the block norms
(oracle/blocks.py): closed forms, special cases, differences."""
import math

import pytest
import torch

from oracle import blocks as ob

F64 = torch.float64


def _rand(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=F64)


def _inputs(B=1, L=5, Hk=1, Hv=2, K=3, V=2, seed=0):
    return dict(q=_rand(B, L, Hk, K, seed=seed), k=_rand(B, L, Hk, K, seed=seed + 1), v=_rand(B, L, Hv, V, seed=seed + 2),
                delta=_rand(B, L, Hv, seed=seed + 3), A=-_rand(Hv, seed=seed + 4).abs(),
                beta=_rand(B, L, Hv, seed=seed + 5))


def test_delta_rule_by_hand():
    # K = V = 1, one head: s = a s; s += b (v - s k) k; out = s q
    one = lambda *x: torch.tensor(x, dtype=F64).view(1, -1, 1, 1)   # noqa: E731
    per = lambda *x: torch.tensor(x, dtype=F64).view(1, -1, 1)      # noqa: E731
    out, S = ob.gdr(one(2, 1), one(1, 2), one(3, 5), per(1, 2), torch.tensor([-math.log(2)], dtype=F64), per(0.5, 1.0),
                    delta_softplus=False, beta_sigmoid=False, qk_l2norm=False, scale=1.0,
                    initial_state=torch.full((1, 1, 1, 1), 4.0, dtype=F64))
    # s = 2, s += .5 (3 - 2) = 2.5, out 5;  s = .625, s += (5 - 1.25) 2 = 8.125
    assert out.flatten().tolist() == pytest.approx([5.0, 8.125])
    assert S.item() == pytest.approx(8.125)


def test_full_strength_write_returns_its_value():
    # b = 1, unit keys: right after a write the state returns v for k
    x = _inputs(L=7, K=4)
    k = x["k"] / x["k"].norm(dim=-1, keepdim=True)
    out, _ = ob.gdr(k, k, x["v"], x["delta"], x["A"], torch.ones_like(x["beta"]), beta_sigmoid=False, qk_l2norm=False,
                    scale=1.0)
    assert torch.allclose(out, x["v"], atol=1e-12)


def test_orthogonal_keys_make_it_the_plain_decaying_sum():
    # with orthonormal keys the delta term only meets what decayed: without
    # decay out_t for q = k_s (s <= t) is b_s v_s
    L = 4
    k = torch.eye(L, dtype=F64).view(1, L, 1, L)
    v, b = _rand(1, L, 1, 3), torch.rand(1, L, 1, dtype=F64)
    for s in range(L):
        q = k[:, s:s + 1].expand(1, L, 1, L)
        out, _ = ob.gdr(q, k, v, torch.zeros(1, L, 1, dtype=F64), torch.zeros(1, dtype=F64), b, delta_softplus=False,
                        beta_sigmoid=False, qk_l2norm=False, scale=1.0)
        assert torch.allclose(out[0, s:, 0], (b[0, s, 0] * v[0, s, 0]).expand(L - s, 3))
        assert torch.equal(out[0, :s], torch.zeros(s, 1, 3, dtype=F64))


def test_pieces_chain_and_heads_share():
    x = _inputs(L=9, Hk=2, Hv=4)
    out, S = ob.gdr(**x)
    cut = lambda a, b: {n: t if n == "A" else t[:, a:b] for n, t in x.items()}   # noqa: E731
    o1, S1 = ob.gdr(**cut(0, 4))
    o2, S2 = ob.gdr(**cut(4, 9), initial_state=S1)
    assert torch.allclose(torch.cat((o1, o2), 1), out) and torch.allclose(S2, S)
    full = dict(x, q=x["q"].repeat_interleave(2, 2), k=x["k"].repeat_interleave(2, 2))
    assert torch.allclose(ob.gdr(**full)[0], out)


def test_closed_step_leaves_the_state():
    x = _inputs(L=3)
    S0 = _rand(1, 2, 2, 3, seed=9)
    _, S = ob.gdr(x["q"], x["k"], x["v"], torch.zeros_like(x["delta"]), x["A"], torch.zeros_like(x["beta"]),
                  delta_softplus=False, beta_sigmoid=False, initial_state=S0)
    assert torch.equal(S, S0)


def test_gradients_against_differences():
    x = _inputs(L=4)
    names = list(x)
    assert torch.autograd.gradcheck(lambda *t: ob.gdr(**dict(zip(names, t))), [t.requires_grad_(True) for t in x.values()])


def test_norms_by_hand():
    x = torch.tensor([[3.0, 4.0, 0.0, 2.0]], dtype=F64)
    w = torch.tensor([1.0, 2.0, 3.0, 4.0], dtype=F64)
    r = 1 / math.sqrt(12.5)
    assert torch.allclose(ob.gated_norm(x, w, group=2, eps=0.0),
                          torch.tensor([[3 * r, 8 * r, 0.0, 4 * math.sqrt(2)]], dtype=F64))
    z = torch.full_like(x, 1e3)   # silu(z) = z: a common factor that the norm takes out again
    assert torch.allclose(ob.gated_norm(x, w, z=z, group=2, eps=0.0), ob.gated_norm(x, w, group=2, eps=0.0))
    assert torch.allclose(ob.gated_norm(x, w, z=z, group=2, eps=0.0, norm_before_gate=True),
                          1e3 * ob.gated_norm(x, w, group=2, eps=0.0))
    y = ob.norm(x, torch.ones(4, dtype=F64), layer_norm=True, eps=0.0)
    assert abs(y.mean()) < 1e-12 and y.pow(2).mean().item() == pytest.approx(1.0)
    t = ob.residual_update(x.expand(4, 4), residual=torch.ones(4, 4, dtype=F64), alpha=0.5,
                           scale=torch.tensor([[1.0] * 4, [2.0] * 4], dtype=F64))
    assert torch.allclose(t, 0.5 + x * torch.tensor([[1.0], [1.0], [2.0], [2.0]], dtype=F64))
