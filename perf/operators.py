"""The gated delta rule and the norms around a block: what they compute, at
the sizes they are used at.

Operators (entry points of selective_state_space_24_b200):

* ``gdr_chunk_fwd`` / ``gdr_chunk_bwd``  the gated delta rule over sequences
  and its gradients.  Per value head, with state S (dv, dk):
      dt = softplus(delta + bias), a = exp(dt A), b = sigmoid(beta)
      S  = a S;  S = S + b (v - S k) k^T;  out = S (scale q)
  (q, k divided by their 2-norms first where ``l2norm`` is set)
* ``gdr_step``  the same for one token, the stored state updated in place
* ``gated_norm_fwd`` / ``_bwd``  RMS norm of groups of channels with a SiLU
  gate before or after it
* ``residual_norm_fwd`` / ``_bwd``  residual stream update with a block's
  output (normed, scaled) and the next block's norm

``own`` False: elementary torch operations in 32 bits.  True: the calls a
user makes.  A case is a dict of plain values (see ``listed``).
"""
import math

import torch

own = False

CHUNK = 64
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
L2_EPS = 1e-6


# ---------------------------------------------------------------- the cases

def _gdr(name, op, B, L, Hk, Hv, dk, dv, dtype="bf16", init=False, l2norm=True, sigmoid=True, softplus=True):
    return dict(name=name, op=op, B=B, L=L, Hk=Hk, Hv=Hv, dk=dk, dv=dv, dtype=dtype, init=init, l2norm=l2norm,
                sigmoid=sigmoid, softplus=softplus)


def _gated(name, op, rows, dim, group, dtype, gate, norm_first):
    return dict(name=name, op=op, rows=rows, dim=dim, group=group, dtype=dtype, gate=gate, norm_first=norm_first)


def _resid(name, op, samples, rows, dim, dtype, res32, first, layer, scale, post, alpha=1.0):
    return dict(name=name, op=op, samples=samples, rows=rows, dim=dim, dtype=dtype, res32=res32, first=first,
                layer=layer, scale=scale, post=post, alpha=alpha)


def listed():
    return [
        # a short continued prompt of one user: latency of a few chunks from a stored state
        _gdr("prompt", "chunk_fwd", 1, 197, 16, 32, 128, 128, init=True),
        # one long prompt, two value heads to each key head: few sequences, a long chain
        _gdr("prefill", "chunk_fwd", 1, 4096, 16, 32, 128, 128),
        # a training batch at the Mamba2 workload's batch, length and heads
        _gdr("train", "chunk_fwd", 4, 8192, 32, 32, 128, 128),
        # gradients of a small odd-length batch (the image models' 197 tokens)
        _gdr("grad-small", "chunk_bwd", 2, 197, 6, 6, 64, 64, init=True),
        # gradients of a training micro-batch with shared key heads
        _gdr("grad-train", "chunk_bwd", 2, 2048, 8, 16, 128, 128),
        # one token for one user, and for a full serving batch
        _gdr("token", "step", 1, 1, 16, 32, 128, 128, dtype="bf16"),
        _gdr("tokens", "step", 256, 1, 16, 32, 128, 128, dtype="bf16"),
        # the output norm of the heads (norm, then gate) of a training batch
        _gated("head-norm", "gated_fwd", 8192 * 32, 128, 128, "bf16", True, True),
        # gradients of the Mamba2 output norm (gate, then norm over all of d_inner = 2048)
        _gated("mix-norm-grad", "gated_bwd", 16384, 2048, 2048, "bf16", True, False),
        # a decode batch's residual update and next norm
        _resid("token-resid", "resid_fwd", 1, 16, 1024, "bf16", True, False, False, False, False),
        # Vision-Mamba tokens (64 images of 197): layer scale, layer norm
        _resid("image-resid", "resid_fwd", 1, 64 * 197, 384, "bf16", True, False, True, True, False),
        # gradients with a norm after the block, a gate per sample and the next block's norm
        _resid("block-grad", "resid_bwd", 4, 4 * 4096, 1024, "bf16", True, False, False, True, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["chunk_fwd", "chunk_fwd", "chunk_bwd", "step", "gated_fwd", "gated_bwd", "resid_fwd",
                     "resid_bwd"])
    if op in ("chunk_fwd", "chunk_bwd", "step"):
        Hk = _log(rng, 1, 16)
        Hv = Hk * rng.choice([1, 1, 2, 3, 4])
        dk, dv = rng.choice([64, 128]), rng.choice([64, 128])
        dtype = rng.choice(["bf16", "f32"]) if op == "step" else "bf16"
        most = {"chunk_fwd": 4 * 8192 * 32, "chunk_bwd": 2 * 2048 * 16, "step": 256 * 32}[op]
        L = 1 if op == "step" else _log(rng, 1, 8192 if op == "chunk_fwd" else 2048)
        B = _log(rng, 1, max(1, min(256 if op == "step" else 16, most // (L * Hv))))
        while B * L * Hv > most and L > 1:
            L = max(1, most // (B * Hv))
        return dict(op=op, B=B, L=L, Hk=Hk, Hv=Hv, dk=dk, dv=dv, dtype=dtype, init=rng.random() < 0.5,
                    l2norm=rng.random() < 0.75, sigmoid=rng.random() < 0.75, softplus=rng.random() < 0.75)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("gated_fwd", "gated_bwd"):
        group = 8 * _log(rng, 4, 512)
        dim = group * rng.choice([1, 1, 2, 3, 8])
        rows = _log(rng, 1, max(1, 2 ** 24 // dim))
        return dict(op=op, rows=rows, dim=dim, group=group, dtype=dtype, gate=rng.random() < 0.8,
                    norm_first=rng.random() < 0.5)
    dim = 8 * _log(rng, 4, 512)
    samples = rng.choice([1, 1, 2, 5, 16])
    rows = samples * _log(rng, 1, max(1, 2 ** 23 // (dim * samples)))
    return dict(op=op, samples=samples, rows=rows, dim=dim, dtype=dtype, res32=rng.random() < 0.6,
                first=rng.random() < 0.2, layer=rng.random() < 0.4, scale=rng.random() < 0.6,
                post=rng.random() < 0.4, alpha=rng.choice([1.0, 1.0, 0.5]))


# --------------------------------------------------------------- the inputs

def prepare(case, seed):
    c = dict(case)
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = DTYPES[c["dtype"]]

    def normal(*shape, std=1.0, dtype=dt):
        return (torch.randn(*shape, generator=gen, device=dev) * std).to(dtype)

    def uniform(lo, hi, *shape):
        return torch.rand(*shape, generator=gen, device=dev) * (hi - lo) + lo

    s = {"case": c}
    if c["op"] in ("chunk_fwd", "chunk_bwd", "step"):
        B, L, Hk, Hv, dk, dv = (c[n] for n in ("B", "L", "Hk", "Hv", "dk", "dv"))
        lead = (B,) if c["op"] == "step" else (B, L)
        # activations after a short convolution and SiLU are of order one; without the
        # operator's own norm a user's program hands over unit vectors
        for n in ("q", "k"):
            t = normal(*lead, Hk, dk, dtype=torch.float32)
            if not c["l2norm"]:
                t = t / t.square().sum(-1, keepdim=True).sqrt()
            s[n] = t.to(dt)
        s["v"] = normal(*lead, Hv, dv)
        s["A"] = -uniform(1.0, 16.0, Hv)
        # time steps log-uniform in 1e-3 .. 1e-1 through the softplus, as the scans' workloads
        step = torch.exp(uniform(math.log(1e-3), math.log(1e-1), Hv))
        if c["softplus"]:
            s["delta"] = normal(*lead, Hv, std=0.5)
            s["delta_bias"] = step + torch.log(-torch.expm1(-step))
        else:
            s["delta"] = (step * uniform(0.5, 1.5, *lead, Hv)).to(dt)
            s["delta_bias"] = None
        s["beta"] = normal(*lead, Hv) if c["sigmoid"] else uniform(0.0, 1.0, *lead, Hv).to(dt)
        s["state"] = normal(B, Hv, dv, dk, std=0.3, dtype=torch.float32) if c["init"] or c["op"] == "step" else None
        if c["op"] == "chunk_bwd":
            s["dout"] = normal(B, L, Hv, dv)
            s["dlast"] = normal(B, Hv, dv, dk, std=0.1, dtype=torch.float32) if c["init"] else None
        return s
    rows, dim = c["rows"], c["dim"]
    s["x"] = normal(rows, dim)
    s["weight"] = uniform(0.5, 1.5, dim)
    if c["op"] in ("gated_fwd", "gated_bwd"):
        s["z"] = normal(rows, dim) if c["gate"] else None
    else:
        rt = torch.float32 if c["res32"] else dt
        s["residual"] = None if c["first"] else normal(rows, dim, std=2.0, dtype=rt)
        s["bias"] = uniform(-0.5, 0.5, dim) if c["layer"] else None
        s["scale"] = uniform(0.1, 1.0, c["samples"], dim) if c["scale"] else None
        s["post"] = uniform(0.5, 1.5, dim) if c["post"] else None
        if c["op"] == "resid_bwd":
            # what the forward call left: the updated residual stream
            s["stream"] = _stream(c, s, torch.float32).to(rt)
            s["dstream"] = normal(rows, dim, dtype=rt)
    if c["op"].endswith("_bwd"):
        s["dout"] = normal(rows, dim)
    return s


# ----------------------------------------------------------- the plain forms

def _softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-torch.abs(x)))


def _silu(x):
    return x / (1 + torch.exp(-x))


def _expand(t, groups):
    """(.., Hk, d) to one row per value head."""
    return t.unsqueeze(-2).expand(*t.shape[:-1], groups, t.shape[-1]).reshape(*t.shape[:-2], -1, t.shape[-1])


def _gdr_terms(c, q, k, delta, bias, A, beta):
    """q, k of every value head (normed, q scaled), the log decay and b, in q's type."""
    if c["l2norm"]:
        q = q / torch.sqrt(q.square().sum(-1, keepdim=True) + L2_EPS)
        k = k / torch.sqrt(k.square().sum(-1, keepdim=True) + L2_EPS)
    q = q * c["dk"] ** -0.5
    r = c["Hv"] // c["Hk"]
    dt = delta if bias is None else delta + bias
    if c["softplus"]:
        dt = _softplus(dt)
    b = 1 / (1 + torch.exp(-beta)) if c["sigmoid"] else beta
    return _expand(q, r), _expand(k, r), dt * A, b


def _tri_inverse(a):
    """(I + a)^-1 of strictly lower triangular a, halves at a time."""
    n = a.shape[-1]
    if n == 1:
        return torch.ones_like(a)
    h = n // 2
    x = _tri_inverse(torch.stack((a[..., :h, :h], a[..., h:, h:])))
    low = -(x[1] @ a[..., h:, :h] @ x[0])
    return torch.cat((torch.cat((x[0], torch.zeros_like(low)), -1), torch.cat((low, x[1]), -1)), -2)


def _gdr_chunked(c, q, k, v, delta, bias, A, beta, state):
    """out (B, L, Hv, dv) and the last state, chunk by chunk."""
    q, k, g, b = _gdr_terms(c, q, k, delta, bias, A, beta)
    B, L, H, n = c["B"], c["L"], c["Hv"], -(-c["L"] // CHUNK)
    fill = n * CHUNK - L

    def cut(t):   # (B, L, H, ..) -> (B, H, n, CHUNK, ..), zeros behind the end
        t = torch.cat((t, t.new_zeros(B, fill, *t.shape[2:])), 1) if fill else t
        return t.transpose(1, 2).reshape(B, H, n, CHUNK, *t.shape[3:])

    q, k, v, g, b = (cut(t) for t in (q, k, v, g, b))
    cs = torch.cumsum(g.double(), -1)
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=q.device).tril()
    between = torch.exp(torch.where(low, cs.unsqueeze(-1) - cs.unsqueeze(-2), -torch.inf)).to(q.dtype)
    to_end = torch.exp(cs[..., -1:] - cs).to(q.dtype)
    since = torch.exp(cs).to(q.dtype)
    kT = k.transpose(-1, -2)
    inv = _tri_inverse((b.unsqueeze(-1) * between * (k @ kT)).tril(-1))
    u = inv @ (b.unsqueeze(-1) * v)
    w = inv @ ((b * since).unsqueeze(-1) * k)
    p = between * (q @ kT)
    qd, kd = q * since.unsqueeze(-1), k * to_end.unsqueeze(-1)
    S = torch.zeros(B, H, c["dv"], c["dk"], dtype=q.dtype, device=q.device) if state is None else state
    out = []
    for i in range(n):
        St = S.transpose(-1, -2)
        new = u[:, :, i] - w[:, :, i] @ St
        out.append(qd[:, :, i] @ St + p[:, :, i] @ new)
        S = since[:, :, i, -1, None, None] * S + new.transpose(-1, -2) @ kd[:, :, i]
    out = torch.stack(out, 2).reshape(B, H, n * CHUNK, -1)[:, :, :L].transpose(1, 2)
    return out, S


def _gdr_one(c, q, k, v, delta, bias, A, beta, S):
    q, k, g, b = _gdr_terms(c, q, k, delta, bias, A, beta)
    S = torch.exp(g)[..., None, None] * S
    u = v - (S * k.unsqueeze(-2)).sum(-1)
    S = S + (b.unsqueeze(-1) * u).unsqueeze(-1) * k.unsqueeze(-2)
    return (S * q.unsqueeze(-2)).sum(-1), S


GRADS = ("q", "k", "v", "delta", "delta_bias", "A", "beta", "state")


def _plain_gdr(c, s):
    t = {n: None if s[n] is None else s[n].float() for n in GRADS}
    dt = DTYPES[c["dtype"]]
    if c["op"] == "step":
        out, S = _gdr_one(c, *(t[n] for n in GRADS))
        return {"out": out.to(dt), "state": s["state"].copy_(S)}   # the stored state moves on in place
    if c["op"] == "chunk_fwd":
        out, S = _gdr_chunked(c, *(t[n] for n in GRADS))
        return {"out": out.to(dt), "last_state": S}
    with torch.enable_grad():
        on = [n for n in GRADS if t[n] is not None]
        for n in on:
            t[n] = t[n].detach().requires_grad_(True)
        out, S = _gdr_chunked(c, *(t[n] for n in GRADS))
        total = (out * s["dout"].float()).sum()
        if s["dlast"] is not None:
            total = total + (S * s["dlast"]).sum()
        g = torch.autograd.grad(total, [t[n] for n in on])
    return {"d" + n: x.to(s[n].dtype) for n, x in zip(on, g)}


def _rms(x, eps):
    return 1 / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)


EPS = 1e-5


def _plain_gated(c, s):
    dt = DTYPES[c["dtype"]]
    shape = (c["rows"], c["dim"] // c["group"], c["group"])
    x, w = s["x"].float().view(shape), s["weight"].view(shape[1:])
    z = None if s["z"] is None else s["z"].float().view(shape)
    gate = None if z is None else _silu(z)
    u = x if gate is None or c["norm_first"] else x * gate
    r = _rms(u, EPS)
    n = u * r
    if c["op"] == "gated_fwd":
        y = n * w if gate is None or not c["norm_first"] else n * w * gate
        return {"out": y.view(c["rows"], c["dim"]).to(dt)}
    dy = s["dout"].float().view(shape)
    out = {}
    dn = dy * gate if gate is not None and c["norm_first"] else dy
    out["dweight"] = (dn * n).sum(0).view(-1)
    dn = dn * w
    du = r * (dn - n * (dn * n).mean(-1, keepdim=True))
    if gate is not None:
        sig = 1 / (1 + torch.exp(-z))
        dgate = dy * n * w if c["norm_first"] else du * x
        out["dz"] = (dgate * (sig * (1 + z * (1 - sig)))).view(c["rows"], c["dim"]).to(dt)
    dx = du if gate is None or c["norm_first"] else du * gate
    out["dx"] = dx.view(c["rows"], c["dim"]).to(dt)
    return out


def _rows_of(c, t):
    """(samples, dim) to one row per row, as a broadcast view."""
    return t.to(t.dtype).unsqueeze(1).expand(-1, c["rows"] // c["samples"], -1).reshape(c["rows"], c["dim"])


def _stream(c, s, dtype):
    x = s["x"].to(dtype)
    if s["post"] is not None:
        x = x * _rms(x, EPS) * s["post"].to(dtype)
    if s["scale"] is not None:
        x = x * _rows_of(c, s["scale"].to(dtype))
    return x if s["residual"] is None else c["alpha"] * s["residual"].to(dtype) + x


def _plain_resid(c, s):
    dt = DTYPES[c["dtype"]]
    rt = torch.float32 if c["res32"] else dt
    w = s["weight"]
    r = _stream(c, s, torch.float32) if c["op"] == "resid_fwd" else s["stream"].float()
    if c["op"] == "resid_fwd" and rt != torch.float32:
        r = r.to(rt).float()   # the stream as it is stored is what the next norm reads
    m = r - r.mean(-1, keepdim=True) if c["layer"] else r
    k = _rms(m, EPS)
    n = m * k
    if c["op"] == "resid_fwd":
        y = n * w
        return {"out": (y if s["bias"] is None else y + s["bias"]).to(dt), "residual": r.to(rt)}
    dy = s["dout"].float()
    out = {"dweight": (dy * n).sum(0)}
    if s["bias"] is not None:
        out["dbias"] = dy.sum(0)
    dn = dy * w
    dr = dn - n * (dn * n).mean(-1, keepdim=True)
    if c["layer"]:
        dr = dr - dn.mean(-1, keepdim=True)
    dr = s["dstream"].float() + k * dr
    if s["residual"] is not None:
        out["dresidual"] = (c["alpha"] * dr).to(rt)
    x = s["x"].float()
    if s["post"] is not None:
        px = _rms(x, EPS)
        pn = x * px
        x = pn * s["post"]
    d = dr
    if s["scale"] is not None:
        out["dscale"] = (dr * x).view(c["samples"], -1, c["dim"]).sum(1)
        d = dr * _rows_of(c, s["scale"])
    if s["post"] is not None:
        out["dpost_weight"] = (d * pn).sum(0)
        d = d * s["post"]
        d = px * (d - pn * (d * pn).mean(-1, keepdim=True))
    out["dx"] = d.to(dt)
    return out


# ------------------------------------------------------------- the user's calls

def _own(c, s):
    import selective_state_space_24_b200 as ssm
    op = c["op"]
    if op in ("chunk_fwd", "chunk_bwd", "step"):
        kw = dict(delta_bias=s["delta_bias"], delta_softplus=c["softplus"], beta_sigmoid=c["sigmoid"],
                  qk_l2norm=c["l2norm"])
        args = [s[n] for n in ("q", "k", "v", "delta", "A", "beta")]
        if op == "step":
            return {"out": ssm.gdr_step(*args, s["state"], **kw), "state": s["state"]}   # updated in place
        if op == "chunk_fwd":
            last = torch.empty(c["B"], c["Hv"], c["dv"], c["dk"], device=s["q"].device)
            out = ssm.gdr_chunk_fwd(*args, initial_state=s["state"], last_state=last, **kw)
            return {"out": out, "last_state": last}
        g = ssm.gdr_chunk_bwd(*args, s["dout"], initial_state=s["state"], dlast_state=s["dlast"], **kw)
        if "dinitial_state" in g:
            g["dstate"] = g.pop("dinitial_state")
        return g
    if op in ("gated_fwd", "gated_bwd"):
        kw = dict(z=s["z"], group=c["group"], eps=EPS, norm_before_gate=c["norm_first"])
        if op == "gated_fwd":
            return {"out": ssm.gated_norm_fwd(s["x"], s["weight"], **kw)}
        return ssm.gated_norm_bwd(s["x"], s["weight"], s["dout"], **kw)
    kw = dict(scale=s["scale"], post_weight=s["post"], alpha=c["alpha"], eps=EPS, layer_norm=c["layer"])
    if op == "resid_fwd":
        out, r = ssm.residual_norm_fwd(s["x"], s["weight"], residual=s["residual"], bias=s["bias"],
                                       residual_f32=c["res32"], **kw)
        return {"out": out, "residual": r}
    return ssm.residual_norm_bwd(s["x"], s["stream"], s["weight"], s["dout"], dresidual_out=s["dstream"],
                                 need_dresidual=s["residual"] is not None, bias=s["bias"], **kw)


def run(state):
    c = state["case"]
    if own:
        return _own(c, state)
    if c["op"] in ("chunk_fwd", "chunk_bwd", "step"):
        return _plain_gdr(c, state)
    return _plain_gated(c, state) if c["op"].startswith("gated") else _plain_resid(c, state)


# ------------------------------------------------------------------- the work

def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"] in ("chunk_fwd", "chunk_bwd", "step"):
        tok = c["B"] * c["L"]
        qk, v, head = tok * c["Hk"] * c["dk"], tok * c["Hv"] * c["dv"], tok * c["Hv"]
        S = c["B"] * c["Hv"] * c["dv"] * c["dk"]
        if c["op"] == "chunk_bwd":   # q k v dout delta beta in, five gradients out
            b = e * (4 * qk + 3 * v + 4 * head) + 4 * (3 * S if c["init"] else 0)
            return {"bytes": b, "flops": 18 * head * c["dk"] * c["dv"]}
        reads = S if c["init"] or c["op"] == "step" else 0
        b = e * (2 * qk + 2 * v + 2 * head) + 4 * (reads + S)
        return {"bytes": b, "flops": 6 * head * c["dk"] * c["dv"]}
    n = c["rows"] * c["dim"]
    if c["op"] == "gated_fwd":
        return {"bytes": e * n * (2 + c["gate"]), "flops": 8 * n}
    if c["op"] == "gated_bwd":
        return {"bytes": e * n * (3 + 2 * c["gate"]), "flops": 20 * n}
    r = 4 if c["res32"] else e
    if c["op"] == "resid_fwd":
        return {"bytes": n * (2 * e + (r if c["first"] else 2 * r)), "flops": 8 * n}
    # the block's output is needed only where a scale or a norm follows it
    x = e if c["scale"] or c["post"] else 0
    return {"bytes": n * (2 * e + x + 2 * r + (0 if c["first"] else r)), "flops": 20 * n}


# ----------------------------------------------------- the definition, 64 bits

def _exact_gdr(c, s):
    f = lambda n: None if s[n] is None else s[n].double()   # noqa: E731
    q0, k0, v, delta, bias, A, beta, S = (f(n) for n in ("q", "k", "v", "delta", "delta_bias", "A", "beta", "state"))
    if c["op"] == "step":
        q0, k0, v, delta, beta = (t.unsqueeze(1) for t in (q0, k0, v, delta, beta))
    B, L, Hk, Hv, dk, dv = q0.shape[0], q0.shape[1], c["Hk"], c["Hv"], c["dk"], c["dv"]
    r = Hv // Hk
    nq = torch.sqrt((q0 * q0).sum(-1, keepdim=True) + L2_EPS) if c["l2norm"] else torch.ones_like(q0[..., :1])
    nk = torch.sqrt((k0 * k0).sum(-1, keepdim=True) + L2_EPS) if c["l2norm"] else torch.ones_like(k0[..., :1])
    uq, uk = q0 / nq, k0 / nk
    head = torch.arange(Hv, device=q0.device) // r
    q, k = uq[:, :, head] / math.sqrt(dk), uk[:, :, head]
    pre = delta if bias is None else delta + bias
    dt = torch.logaddexp(pre, torch.zeros_like(pre)) if c["softplus"] else pre
    b = torch.sigmoid(beta) if c["sigmoid"] else beta
    a = torch.exp(dt * A)
    S = torch.zeros(B, Hv, dv, dk, dtype=torch.float64, device=q.device) if S is None else S
    back = c["op"] == "chunk_bwd"
    kept, us, outs = [S], [], []
    for t in range(L):
        S = S * a[:, t, :, None, None]
        u = v[:, t] - torch.einsum("bhvk,bhk->bhv", S, k[:, t])
        S = torch.addcmul(S, (b[:, t, :, None] * u).unsqueeze(-1), k[:, t].unsqueeze(-2))
        if back:
            kept.append(S)
            us.append(u)
        else:
            outs.append(torch.einsum("bhvk,bhk->bhv", S, q[:, t]))
    if c["op"] == "step":
        return {"out": outs[0], "state": S}
    if not back:
        return {"out": torch.stack(outs, 1), "last_state": S}
    do = s["dout"].double()
    G = torch.zeros_like(S) if s["dlast"] is None else s["dlast"].double()
    dq, dk_, dv_, db, da = (torch.zeros_like(t) for t in (q, k, v, b, a))
    for t in range(L - 1, -1, -1):
        G = G + do[:, t].unsqueeze(-1) * q[:, t].unsqueeze(-2)
        dq[:, t] = torch.einsum("bhvk,bhv->bhk", kept[t + 1], do[:, t])
        u, kt = us[t], k[:, t]
        w = torch.einsum("bhvk,bhk->bhv", G, kt)
        db[:, t] = (u * w).sum(-1)
        du = b[:, t, :, None] * w
        dv_[:, t] = du
        before = kept[t] * a[:, t, :, None, None]
        dk_[:, t] = b[:, t, :, None] * torch.einsum("bhvk,bhv->bhk", G, u) - torch.einsum("bhvk,bhv->bhk", before, du)
        G = G - du.unsqueeze(-1) * kt.unsqueeze(-2)
        da[:, t] = (G * kept[t]).sum((-1, -2))
        G = G * a[:, t, :, None, None]
    dg = da * a

    def unnorm(d, unit, norm):   # through the 2-norm, value heads of a key head summed
        d = d.view(B, L, Hk, r, dk).sum(3)
        return (d - unit * (unit * d).sum(-1, keepdim=True)) / norm if c["l2norm"] else d

    ddt = dg * A
    pre_d = ddt * torch.sigmoid(pre) if c["softplus"] else ddt
    out = {"dq": unnorm(dq / math.sqrt(dk), uq, nq), "dk": unnorm(dk_, uk, nk), "dv": dv_, "ddelta": pre_d,
           "dA": (dg * dt).sum((0, 1)), "dbeta": db * b * (1 - b) if c["sigmoid"] else db}
    if bias is not None:
        out["ddelta_bias"] = pre_d.sum((0, 1))
    if s["state"] is not None:
        out["dstate"] = G
    return out


def _exact_norms(c, s):
    D = lambda n: None if s.get(n) is None else s[n].double().requires_grad_(True)   # noqa: E731
    F = torch.nn.functional
    x, w = D("x"), D("weight")
    with torch.enable_grad():
        if c["op"].startswith("gated"):
            z = D("z")
            shape = (c["rows"], -1, c["group"])
            y = x if z is None or c["norm_first"] else x * F.silu(z)
            y = F.rms_norm(y.view(shape), (c["group"],), None, EPS).reshape(x.shape) * w
            if z is not None and c["norm_first"]:
                y = y * F.silu(z)
            if c["op"] == "gated_fwd":
                return {"out": y.detach()}
            names = {"dx": x, "dweight": w} | ({} if z is None else {"dz": z})
            return dict(zip(names, torch.autograd.grad(y, list(names.values()), s["dout"].double())))
        bias, scale, post, res = D("bias"), D("scale"), D("post"), D("residual")
        t = x if post is None else F.rms_norm(x, (c["dim"],), post, EPS)
        if scale is not None:
            t = t * scale.repeat_interleave(c["rows"] // c["samples"], 0)
        t = t if res is None else t + c["alpha"] * res
        rt = torch.float32 if c["res32"] else DTYPES[c["dtype"]]
        # the stored stream is what the norm reads: its value is given in the backward pass
        stored = t.detach().to(rt).double() if c["op"] == "resid_fwd" else s["stream"].double()
        r = (stored if rt != torch.float32 or c["op"] == "resid_bwd" else t.detach()).requires_grad_(True)
        y = F.layer_norm(r, (c["dim"],), w, bias, EPS) if c["layer"] else F.rms_norm(r, (c["dim"],), w, EPS)
        if c["op"] == "resid_fwd":
            return {"out": y.detach(), "residual": t.detach()}
        names = {"dweight": w} | ({} if bias is None else {"dbias": bias})
        got = torch.autograd.grad(y, [r] + list(names.values()), s["dout"].double())
        dr = got[0] + s["dstream"].double()
        out = dict(zip(names, got[1:]))
        names = {"dx": x} | {n: v for n, v in (("dresidual", res), ("dscale", scale), ("dpost_weight", post))
                             if v is not None}
        return out | dict(zip(names, torch.autograd.grad(t, list(names.values()), dr)))


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    with torch.no_grad():
        return _exact_gdr(c, s) if c["op"] in ("chunk_fwd", "chunk_bwd", "step") else _exact_norms(c, s)
