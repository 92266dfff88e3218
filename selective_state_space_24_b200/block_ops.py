"""The gated delta rule and the norms around a block: binding of
gdr_chunk_fwd, gdr_chunk_bwd, gdr_step, gated_norm_fwd / _bwd and
residual_norm_fwd / _bwd (include/ssm.h; names as there).

Tensors are contiguous, on one CUDA device, which need not be the current
one; shapes and types are checked before the call.  Work runs on ``stream``
(default: the current stream of the tensors' device).  What the call
allocates (results not passed in, the workspace) is that stream's memory and
kept alive for the current stream too.
"""
from __future__ import annotations

import ctypes

from . import SSM_BF16, SSM_F32, SSMError, _torch, capi

__all__ = ["gdr_chunk_fwd", "gdr_chunk_bwd", "gdr_step", "gated_norm_fwd", "gated_norm_bwd", "residual_norm_fwd",
           "residual_norm_bwd", "gdr_dims", "gdr_inputs", "gdr_grads", "norm_dims", "residual_norm_params",
           "residual_norm_grads"]

_vp, _i64, _i32, _f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
_sz, _int, _ref = ctypes.c_size_t, ctypes.c_int, ctypes.byref


class gdr_dims(ctypes.Structure):
    _fields_ = [("batch", _i64), ("seqlen", _i64), ("nheads_k", _i64), ("nheads_v", _i64), ("headdim_k", _i64),
                ("headdim_v", _i64), ("dtype", _i32)]


class gdr_inputs(ctypes.Structure):
    _fields_ = [("q", _vp), ("k", _vp), ("v", _vp), ("delta", _vp), ("delta_bias", _vp), ("A", _vp), ("beta", _vp),
                ("scale", _f32), ("delta_softplus", _i32), ("beta_sigmoid", _i32), ("qk_l2norm", _i32)]


class gdr_grads(ctypes.Structure):
    _fields_ = [("dq", _vp), ("dk", _vp), ("dv", _vp), ("ddelta", _vp), ("dbeta", _vp), ("dA", _vp),
                ("ddelta_bias", _vp), ("dinitial_state", _vp)]


class norm_dims(ctypes.Structure):
    _fields_ = [("rows", _i64), ("dim", _i64), ("group", _i64), ("eps", _f32), ("dtype", _i32)]


class residual_norm_params(ctypes.Structure):
    _fields_ = [("weight", _vp), ("bias", _vp), ("scale", _vp), ("post_weight", _vp), ("samples", _i64),
                ("alpha", _f32), ("layer_norm", _i32), ("residual_f32", _i32)]


class residual_norm_grads(ctypes.Structure):
    _fields_ = [("dx", _vp), ("dresidual", _vp), ("dweight", _vp), ("dbias", _vp), ("dscale", _vp),
                ("dpost_weight", _vp)]


_P = ctypes.POINTER
SIGNATURES = {
    "gdr_chunk_workspace_size": (_sz, [_P(gdr_dims)]),
    "gdr_chunk_fwd": (_int, [_P(gdr_dims), _P(gdr_inputs), _vp, _vp, _vp, _vp, _sz, _vp]),
    "gdr_step": (_int, [_P(gdr_dims), _P(gdr_inputs), _vp, _vp, _vp]),
    "gdr_chunk_bwd_workspace_size": (_sz, [_P(gdr_dims)]),
    "gdr_chunk_bwd": (_int, [_P(gdr_dims), _P(gdr_inputs), _vp, _vp, _vp, _P(gdr_grads), _vp, _sz, _vp]),
    "gated_norm_fwd": (_int, [_P(norm_dims), _vp, _vp, _vp, _int, _vp, _vp]),
    "gated_norm_bwd_workspace_size": (_sz, [_P(norm_dims)]),
    "gated_norm_bwd": (_int, [_P(norm_dims), _vp, _vp, _vp, _int, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "residual_norm_fwd": (_int, [_P(norm_dims), _P(residual_norm_params), _vp, _vp, _vp, _vp, _vp]),
    "residual_norm_bwd_workspace_size": (_sz, [_P(norm_dims), _P(residual_norm_params)]),
    "residual_norm_bwd": (_int, [_P(norm_dims), _P(residual_norm_params), _vp, _vp, _vp, _vp,
                                 _P(residual_norm_grads), _vp, _sz, _vp]),
}


class _Torch:
    """What every call needs of torch, looked up once."""
    torch = None

    @classmethod
    def load(cls):
        torch = _torch()
        cls.codes = {torch.float32: SSM_F32, torch.bfloat16: SSM_BF16}
        cls.f32, cls.empty_like = torch.float32, torch.empty_like
        cls.current_device = torch.cuda.current_device
        # the handle of a device's current stream, without building a Stream object
        cls.stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                             lambda index: torch.cuda.current_stream(index).cuda_stream)
        cls.torch = torch


class _Call:
    """One call's device, stream and temporaries."""

    def __init__(self, x, name, stream):
        if _Torch.torch is None:
            _Torch.load()
        self.index = x.get_device()
        if self.index < 0:
            raise ValueError(f"{name}: tensors must be on a CUDA device")
        self.dtype = x.dtype
        self.code = _Torch.codes.get(self.dtype)
        if self.code is None:
            raise TypeError(f"{name}: unsupported dtype {x.dtype}")
        self.torch, self.f32 = _Torch.torch, _Torch.f32
        self.name, self.device, self.stream = name, x.device, stream
        self.made = []   # allocated on an explicit stream, to be kept for the current one, which will use them

    def ptr(self, t, what, shape, dtype):
        """The address of t after its checks (None for None)."""
        if t is None:
            return None
        if t.dtype is dtype and t.shape == shape and t.get_device() == self.index and t.is_contiguous():
            return t.data_ptr()
        if t.dtype != dtype:
            raise TypeError(f"{self.name}: {what} must be {dtype}, got {t.dtype}")
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{self.name}: {what} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        if t.device != self.device:
            raise ValueError(f"{self.name}: {what} must be on {self.device}, got {t.device}")
        raise ValueError(f"{self.name}: {what} must be contiguous")

    # Memory is the stream's that the call runs on: other streams are done with it.

    def like(self, t):
        if self.stream is None:
            return _Torch.empty_like(t)
        with self.torch.cuda.stream(self.stream):
            t = _Torch.empty_like(t)
        self.made.append(t)
        return t

    def new(self, shape, dtype):
        if self.stream is not None:
            with self.torch.cuda.stream(self.stream):
                t = self.torch.empty(shape, dtype=dtype, device=self.device)
            self.made.append(t)
            return t
        return self.torch.empty(shape, dtype=dtype, device=self.device)

    def workspace(self, need, ws):
        """(address, bytes) of a workspace of at least `need` bytes."""
        if need == 0:
            return None, 0
        if ws is None:
            ws = self.new((need,), self.torch.uint8)
        elif ws.device != self.device or not ws.is_contiguous():
            raise ValueError(f"{self.name}: ws must be contiguous and on {self.device}")
        return ws.data_ptr(), ws.numel() * ws.element_size()

    def run(self, fn, *args):
        """fn(*args, stream) on the tensors' device; raises on an error."""
        if self.index != _Torch.current_device():
            with self.torch.cuda.device(self.device):
                return self._run(fn, args)
        return self._run(fn, args)

    def _run(self, fn, args):
        here = _Torch.stream(self.index)
        s = here if self.stream is None else self.stream.cuda_stream
        status = fn(*args, s)
        if s != here:
            for t in self.made:
                t.record_stream(self.torch.cuda.current_stream(self.index))
        if status != 0:
            raise SSMError(status, self.name)


def _gdr(call, q, k, v, delta, A, beta, delta_bias, delta_softplus, beta_sigmoid, qk_l2norm, scale, step):
    """dims, inputs and the state's shape."""
    qs, vs = q.shape, v.shape
    want = 3 if step else 4
    if len(qs) != want or len(vs) != want:
        raise ValueError(f"{call.name}: q, k and v must have {want} dimensions")
    if step:
        (B, Hk, K), L, (Hv, V) = qs, 1, vs[1:]
        vs_want, per = (B, Hv, V), (B, Hv)
    else:
        (B, L, Hk, K), (Hv, V) = qs, vs[2:]
        vs_want, per = (B, L, Hv, V), (B, L, Hv)
    ptr, f32, dt, head = call.ptr, call.f32, call.dtype, (Hv,)
    dims = gdr_dims(B, L, Hk, Hv, K, V, call.code)
    inp = gdr_inputs(ptr(q, "q", qs, dt), ptr(k, "k", qs, dt), ptr(v, "v", vs_want, dt), ptr(delta, "delta", per, dt),
                     ptr(delta_bias, "delta_bias", head, f32), ptr(A, "A", head, f32), ptr(beta, "beta", per, dt),
                     K ** -0.5 if scale is None else scale, 1 if delta_softplus else 0, 1 if beta_sigmoid else 0,
                     1 if qk_l2norm else 0)
    return dims, inp, (B, Hv, V, K)


def gdr_chunk_fwd(q, k, v, delta, A, beta, *, delta_bias=None, delta_softplus=True, beta_sigmoid=True,
                  qk_l2norm=True, scale=None, initial_state=None, out=None, last_state=None, ws=None, stream=None):
    """Gated delta rule over sequences: q, k (B, L, Hk, K), v (B, L, Hv, V),
    delta, beta (B, L, Hv) bfloat16, A, delta_bias (Hv) float32; returns out
    (B, L, Hv, V).  initial_state and last_state (B, Hv, V, K) float32 may be
    the same tensor.  scale defaults to K ** -0.5.  ws is not needed."""
    call = _Call(q, "gdr_chunk_fwd", stream)
    dims, inp, st = _gdr(call, q, k, v, delta, A, beta, delta_bias, delta_softplus, beta_sigmoid, qk_l2norm,
                               scale, False)
    if out is None:
        out = call.like(v)
    f32 = call.f32
    call.run(capi().gdr_chunk_fwd, _ref(dims), _ref(inp), call.ptr(initial_state, "initial_state", st, f32),
             call.ptr(out, "out", v.shape, call.dtype), call.ptr(last_state, "last_state", st, f32), None, 0)
    return out


def gdr_step(q, k, v, delta, A, beta, state, *, delta_bias=None, delta_softplus=True, beta_sigmoid=True,
             qk_l2norm=True, scale=None, out=None, stream=None):
    """One decode step: q, k (B, Hk, K), v (B, Hv, V), delta, beta (B, Hv),
    float32 or bfloat16; state (B, Hv, V, K) float32 updated in place.
    Returns out (B, Hv, V)."""
    call = _Call(q, "gdr_step", stream)
    dims, inp, st = _gdr(call, q, k, v, delta, A, beta, delta_bias, delta_softplus, beta_sigmoid, qk_l2norm,
                               scale, True)
    if out is None:
        out = call.like(v)
    call.run(capi().gdr_step, _ref(dims), _ref(inp), call.ptr(state, "state", st, call.f32),
             call.ptr(out, "out", v.shape, call.dtype))
    return out


def gdr_chunk_bwd(q, k, v, delta, A, beta, dout, *, delta_bias=None, delta_softplus=True, beta_sigmoid=True,
                  qk_l2norm=True, scale=None, initial_state=None, dlast_state=None, ws=None, stream=None):
    """Gradients of gdr_chunk_fwd for dout (B, L, Hv, V) and, where given,
    dlast_state (B, Hv, V, K) float32: a dict of dq, dk, dv, ddelta, dbeta in
    the inputs' type, dA and (with delta_bias) ddelta_bias float32, and with
    initial_state its gradient dinitial_state."""
    call = _Call(q, "gdr_chunk_bwd", stream)
    dims, inp, st = _gdr(call, q, k, v, delta, A, beta, delta_bias, delta_softplus, beta_sigmoid, qk_l2norm,
                               scale, False)
    f32 = call.f32
    g = {"dq": call.like(q), "dk": call.like(k), "dv": call.like(v), "ddelta": call.like(delta),
         "dbeta": call.like(beta), "dA": call.like(A)}
    if delta_bias is not None:
        g["ddelta_bias"] = call.like(delta_bias)
    if initial_state is not None:
        g["dinitial_state"] = call.like(initial_state)
    out = gdr_grads(**{n: t.data_ptr() for n, t in g.items()})
    lib = capi()
    w, n = call.workspace(lib.gdr_chunk_bwd_workspace_size(_ref(dims)), ws)
    call.run(lib.gdr_chunk_bwd, _ref(dims), _ref(inp), call.ptr(initial_state, "initial_state", st, f32),
             call.ptr(dout, "dout", v.shape, call.dtype), call.ptr(dlast_state, "dlast_state", st, f32),
             _ref(out), w, n)
    return g


def _rows(call, x, weight, group, eps):
    """norm_dims for x (.., dim)."""
    if x.dim() < 1 or weight.dim() != 1 or weight.shape[0] != x.shape[-1]:
        raise ValueError(f"{call.name}: weight must have the length of x's last dimension")
    dim = x.shape[-1]
    return norm_dims(x.numel() // dim if dim else 0, dim, dim if group is None else group, eps, call.code)


def gated_norm_fwd(x, weight, *, z=None, group=None, eps=1e-5, norm_before_gate=False, out=None, stream=None):
    """RMS norm of groups of `group` channels (default: all) of x (.., dim)
    with the gate silu(z): norm(x silu(z)) weight, or with norm_before_gate
    norm(x) weight silu(z).  weight (dim) float32; x, z, out float32 or
    bfloat16.  out may be x or z."""
    call = _Call(x, "gated_norm_fwd", stream)
    dims = _rows(call, x, weight, group, eps)
    if out is None:
        out = call.like(x)
    shape = x.shape
    call.run(capi().gated_norm_fwd, _ref(dims), call.ptr(x, "x", shape, call.dtype), call.ptr(z, "z", shape, call.dtype),
             call.ptr(weight, "weight", shape[-1:], call.f32), int(bool(norm_before_gate)),
             call.ptr(out, "out", shape, call.dtype))
    return out


def gated_norm_bwd(x, weight, dout, *, z=None, group=None, eps=1e-5, norm_before_gate=False, ws=None, stream=None):
    """Gradients of gated_norm_fwd: a dict of dx, dz (with z) in x's type and
    dweight float32."""
    call = _Call(x, "gated_norm_bwd", stream)
    dims = _rows(call, x, weight, group, eps)
    shape, dt = x.shape, call.dtype
    g = {"dx": call.like(x), "dweight": call.like(weight)}
    if z is not None:
        g["dz"] = call.like(z)
    lib = capi()
    w, n = call.workspace(lib.gated_norm_bwd_workspace_size(_ref(dims)), ws)
    call.run(lib.gated_norm_bwd, _ref(dims), call.ptr(x, "x", shape, dt), call.ptr(z, "z", shape, dt),
             call.ptr(weight, "weight", shape[-1:], call.f32), int(bool(norm_before_gate)),
             call.ptr(dout, "dout", shape, dt), g["dx"].data_ptr(), None if z is None else g["dz"].data_ptr(),
             g["dweight"].data_ptr(), w, n)
    return g


def _residual(call, x, weight, bias, scale, post_weight, alpha, layer_norm, residual_f32, eps):
    dims = _rows(call, x, weight, None, eps)
    one, f32 = x.shape[-1:], call.f32
    samples = 1
    if scale is not None:
        if scale.dim() == 1:
            scale = scale.unsqueeze(0)
        samples = scale.shape[0]
    p = residual_norm_params(call.ptr(weight, "weight", one, f32), call.ptr(bias, "bias", one, f32),
                             call.ptr(scale, "scale", (samples, *one), f32),
                             call.ptr(post_weight, "post_weight", one, f32), samples, alpha, int(bool(layer_norm)),
                             int(bool(residual_f32)))
    return dims, p, f32 if residual_f32 else call.dtype


def residual_norm_fwd(x, weight, *, residual=None, bias=None, scale=None, post_weight=None, alpha=1.0,
                      layer_norm=False, eps=1e-5, residual_f32=True, out=None, residual_out=None, stream=None):
    """The residual stream takes a block's output and the next block's norm
    follows: residual_out = alpha residual + scale t, t = x or, with
    post_weight, the RMS norm of x times it; out = norm(residual_out) weight
    (+ bias), the RMS or the layer norm.  x (.., dim); residual and
    residual_out float32, or x's type with residual_f32 False, and may be one
    tensor; scale (dim) or (samples, dim), the leading dimensions of x cut
    into `samples` equal runs.  Returns (out, residual_out)."""
    call = _Call(x, "residual_norm_fwd", stream)
    dims, p, rt = _residual(call, x, weight, bias, scale, post_weight, alpha, layer_norm, residual_f32, eps)
    shape, dt = x.shape, call.dtype
    if out is None:
        out = call.like(x)
    if residual_out is None:
        residual_out = call.like(x if rt == dt else residual) if rt == dt or residual is not None else call.new(shape, rt)
    call.run(capi().residual_norm_fwd, _ref(dims), _ref(p), call.ptr(x, "x", shape, dt),
             call.ptr(residual, "residual", shape, rt), call.ptr(residual_out, "residual_out", shape, rt),
             call.ptr(out, "out", shape, dt))
    return out, residual_out


def residual_norm_bwd(x, residual_out, weight, dout, *, dresidual_out=None, need_dresidual=True, bias=None,
                      scale=None, post_weight=None, alpha=1.0, layer_norm=False, eps=1e-5, ws=None, stream=None):
    """Gradients of residual_norm_fwd from the residual_out it returned, for
    dout and (where given) dresidual_out: a dict of dx, dresidual (unless
    need_dresidual is False: the call had no residual), dweight and, where
    given, dbias, dscale, dpost_weight (float32, in their inputs' shapes)."""
    call = _Call(x, "residual_norm_bwd", stream)
    if residual_out.dtype not in (call.f32, call.dtype):
        raise TypeError(f"{call.name}: residual_out must be float32 or {call.dtype}, got {residual_out.dtype}")
    dims, p, rt = _residual(call, x, weight, bias, scale, post_weight, alpha, layer_norm,
                            residual_out.dtype == call.f32, eps)
    shape, dt = x.shape, call.dtype
    g = {"dx": call.like(x), "dweight": call.like(weight)}
    if need_dresidual:
        g["dresidual"] = call.like(residual_out)
    for name, t in (("dbias", bias), ("dscale", scale), ("dpost_weight", post_weight)):
        if t is not None:
            g[name] = call.like(t)
    c = residual_norm_grads(**{n: t.data_ptr() for n, t in g.items()})
    lib = capi()
    w, n = call.workspace(lib.residual_norm_bwd_workspace_size(_ref(dims), _ref(p)), ws)
    call.run(lib.residual_norm_bwd, _ref(dims), _ref(p), call.ptr(x, "x", shape, dt),
             call.ptr(residual_out, "residual_out", shape, rt), call.ptr(dout, "dout", shape, dt),
             call.ptr(dresidual_out, "dresidual_out", shape, rt), _ref(c), w, n)
    return g
