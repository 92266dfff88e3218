// block_capi.cu -- the extern "C" boundary of the gated delta rule and of the
// norms around a block (declared in include/ssm.h): argument validation,
// workspace sizing, dispatch.  Every check runs before anything is launched.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "../../include/ssm.h"
#include "gdr.h"
#include "norm.h"

namespace {

bool any_misaligned(const void *const *p, int n)
{
    for (int i = 0; i < n; i++)
        if (reinterpret_cast<uintptr_t>(p[i]) & 15u)
            return true;
    return false;
}
template <int N> ssm_status aligned(const void *const (&p)[N])
{
    return any_misaligned(p, N) ? SSM_ERR_MISALIGNED : SSM_OK;
}

ssm_status check_workspace(const void *ws, size_t have, size_t need)
{
    if (need == 0)
        return SSM_OK;
    if (!ws || have < need)
        return SSM_ERR_WORKSPACE_TOO_SMALL;
    return any_misaligned(&ws, 1) ? SSM_ERR_MISALIGNED : SSM_OK;
}

ssm_status status(cudaError_t e) { return e == cudaSuccess ? SSM_OK : SSM_ERR_CUDA; }

ssm_status zero_f32(float *p, size_t n, cudaStream_t st)
{
    return !p || n == 0 ? SSM_OK : status(cudaMemsetAsync(p, 0, n * sizeof(float), st));
}

// ------------------------------------------------------------ delta rule

ssm_status check_gdr_dims(const gdr_dims *d, bool step)
{
    if (!d || d->batch < 0 || d->seqlen < 0 || d->nheads_k < 0 || d->nheads_v < 0 || d->headdim_k < 0 ||
        d->headdim_v < 0)
        return SSM_ERR_INVALID_ARG;
    if (d->dtype != SSM_BF16 && !(step && d->dtype == SSM_F32))
        return SSM_ERR_UNSUPPORTED_DTYPE;
    if ((d->headdim_k != 64 && d->headdim_k != 128) || (d->headdim_v != 64 && d->headdim_v != 128))
        return SSM_ERR_UNSUPPORTED_SHAPE;
    if (step && d->seqlen != 1)
        return SSM_ERR_UNSUPPORTED_SHAPE;
    if (d->nheads_k == 0 ? d->nheads_v != 0 : d->nheads_v % d->nheads_k != 0)
        return SSM_ERR_UNSUPPORTED_SHAPE;
    // 32-bit sizes and block counts inside the kernels
    if (d->batch > INT32_MAX || d->seqlen > INT32_MAX - 64 || d->nheads_v > INT32_MAX / 128 ||
        d->nheads_k > INT32_MAX / 128)
        return SSM_ERR_UNSUPPORTED_SHAPE;
    const int64_t chunks = (d->seqlen + 63) / 64;
    const int64_t heads = d->batch * d->nheads_v;   // below 2^55
    const int64_t most = INT32_MAX / 4;
    if (heads > most || (chunks > 0 && heads > most / chunks))
        return SSM_ERR_UNSUPPORTED_SHAPE;
    return SSM_OK;
}

bool empty_gdr(const gdr_dims *d)
{
    return d->batch == 0 || d->seqlen == 0 || d->nheads_v == 0;
}

size_t state_floats(const gdr_dims *d)
{
    return (size_t)d->batch * d->nheads_v * d->headdim_v * d->headdim_k;
}

ssm::GdrArgs gdr_args(const gdr_dims *d, const gdr_inputs *in)
{
    ssm::GdrArgs a;
    memset(&a, 0, sizeof(a));
    a.Bsz = (int)d->batch;
    a.L = (int)d->seqlen;
    a.Hk = (int)d->nheads_k;
    a.Hv = (int)d->nheads_v;
    a.K = (int)d->headdim_k;
    a.V = (int)d->headdim_v;
    a.dtype = d->dtype == SSM_F32 ? 0 : 1;
    if (in) {
        a.softplus = in->delta_softplus ? 1 : 0;
        a.sigmoid = in->beta_sigmoid ? 1 : 0;
        a.l2norm = in->qk_l2norm ? 1 : 0;
        a.scale = in->scale;
        a.q = in->q;
        a.k = in->k;
        a.v = in->v;
        a.delta = in->delta;
        a.beta = in->beta;
        a.bias = in->delta_bias;
        a.A = in->A;
    }
    return a;
}

ssm_status check_gdr_inputs(const gdr_inputs *in)
{
    if (!in || !in->q || !in->k || !in->v || !in->delta || !in->A || !in->beta || !isfinite(in->scale))
        return SSM_ERR_INVALID_ARG;
    const void *p[] = {in->q, in->k, in->v, in->delta, in->delta_bias, in->A, in->beta};
    return aligned(p);
}

// an empty sequence: the state passes through
ssm_status pass_state(const gdr_dims *d, const float *from, float *to, cudaStream_t st)
{
    const size_t n = state_floats(d);
    if (!to || n == 0 || from == to)
        return SSM_OK;
    if (!from)
        return zero_f32(to, n, st);
    return status(cudaMemcpyAsync(to, from, n * sizeof(float), cudaMemcpyDeviceToDevice, st));
}

// ----------------------------------------------------------------- norms

ssm_status check_norm_dims(const norm_dims *d)
{
    if (!d || d->rows < 0 || d->dim < 0 || d->group < 0 || !(d->eps >= 0.f) || !isfinite(d->eps))
        return SSM_ERR_INVALID_ARG;
    if (d->dtype != SSM_F32 && d->dtype != SSM_BF16)
        return SSM_ERR_UNSUPPORTED_DTYPE;
    if (d->group < 1 || d->group > 8192 || d->dim < 1 || d->dim % d->group != 0)
        return SSM_ERR_UNSUPPORTED_SHAPE;
    // block counts and column indices of the kernels are 32 bits
    if (d->rows > INT32_MAX || d->dim > INT32_MAX / 16)
        return SSM_ERR_UNSUPPORTED_SHAPE;
    const int64_t vec = d->dtype == SSM_F32 ? 4 : 8;
    return d->dim % vec || d->group % vec ? SSM_ERR_MISALIGNED : SSM_OK;
}

ssm_status check_residual(const norm_dims *d, const residual_norm_params *p)
{
    const ssm_status s = check_norm_dims(d);
    if (s != SSM_OK)
        return s;
    if (d->group != d->dim)
        return SSM_ERR_UNSUPPORTED_SHAPE;
    if (!p || !p->weight || p->samples < 1 || !isfinite(p->alpha))
        return SSM_ERR_INVALID_ARG;
    if (d->rows % p->samples != 0)
        return SSM_ERR_UNSUPPORTED_SHAPE;
    const void *q[] = {p->weight, p->bias, p->scale, p->post_weight};
    return aligned(q);
}

ssm::ResidualArgs residual_args(const norm_dims *d, const residual_norm_params *p)
{
    ssm::ResidualArgs a;
    memset(&a, 0, sizeof(a));
    a.rows = d->rows;
    a.samples = p->samples;
    a.dim = (int)d->dim;
    a.fdim = (float)d->dim;
    a.eps = d->eps;
    a.alpha = p->alpha;
    a.dtype = d->dtype == SSM_F32 ? 0 : 1;
    a.layer = p->layer_norm ? 1 : 0;
    a.res32 = d->dtype == SSM_F32 || p->residual_f32;
    a.weight = p->weight;
    a.bias = p->bias;
    a.scale = p->scale;
    a.post = p->post_weight;
    return a;
}

}  // namespace

extern "C" {

size_t gdr_chunk_workspace_size(const gdr_dims *) { return 0; }

ssm_status gdr_chunk_fwd(const gdr_dims *dims, const gdr_inputs *in, const float *initial_state, void *out,
                         float *last_state, void *, size_t, void *stream)
{
    ssm_status s = check_gdr_dims(dims, false);
    if (s != SSM_OK)
        return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const void *own[] = {initial_state, out, last_state};
    if ((s = aligned(own)) != SSM_OK)
        return s;
    if (empty_gdr(dims))
        return pass_state(dims, initial_state, last_state, st);
    if ((s = check_gdr_inputs(in)) != SSM_OK)
        return s;
    if (!out)
        return SSM_ERR_INVALID_ARG;
    ssm::GdrArgs a = gdr_args(dims, in);
    a.init = initial_state;
    a.out = out;
    a.last = last_state;
    return status(ssm::launch_gdr_chunk(a, st));
}

ssm_status gdr_step(const gdr_dims *dims, const gdr_inputs *in, float *state, void *out, void *stream)
{
    ssm_status s = check_gdr_dims(dims, true);
    if (s != SSM_OK)
        return s;
    if (empty_gdr(dims))
        return SSM_OK;
    if ((s = check_gdr_inputs(in)) != SSM_OK)
        return s;
    if (!state || !out)
        return SSM_ERR_INVALID_ARG;
    const void *own[] = {state, out};
    if ((s = aligned(own)) != SSM_OK)
        return s;
    ssm::GdrArgs a = gdr_args(dims, in);
    a.init = state;
    a.last = state;
    a.out = out;
    return status(ssm::launch_gdr_recurrent(a, static_cast<cudaStream_t>(stream)));
}

size_t gdr_chunk_bwd_workspace_size(const gdr_dims *dims)
{
    if (check_gdr_dims(dims, false) != SSM_OK || empty_gdr(dims))
        return 0;
    return ssm::gdr_bwd_ws_bytes(gdr_args(dims, nullptr));
}

ssm_status gdr_chunk_bwd(const gdr_dims *dims, const gdr_inputs *in, const float *initial_state,
                         const void *dout, const float *dlast_state, const gdr_grads *grads, void *workspace,
                         size_t workspace_bytes, void *stream)
{
    ssm_status s = check_gdr_dims(dims, false);
    if (s != SSM_OK)
        return s;
    if (!grads)
        return SSM_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const void *own[] = {initial_state, dout,      dlast_state,  grads->dq,          grads->dk,
                         grads->dv,     grads->ddelta, grads->dbeta, grads->dA, grads->ddelta_bias,
                         grads->dinitial_state};
    if ((s = aligned(own)) != SSM_OK)
        return s;
    if (empty_gdr(dims)) {   // sums over nothing
        if ((s = zero_f32(grads->dA, dims->nheads_v, st)) != SSM_OK ||
            (s = zero_f32(grads->ddelta_bias, dims->nheads_v, st)) != SSM_OK)
            return s;
        const size_t qk = (size_t)dims->batch * dims->seqlen * dims->nheads_k * dims->headdim_k / 2;   // in floats
        if ((s = zero_f32(static_cast<float *>(grads->dq), qk, st)) != SSM_OK ||
            (s = zero_f32(static_cast<float *>(grads->dk), qk, st)) != SSM_OK)
            return s;
        return pass_state(dims, dlast_state, grads->dinitial_state, st);
    }
    if ((s = check_gdr_inputs(in)) != SSM_OK)
        return s;
    if (!dout || !grads->dq || !grads->dk || !grads->dv || !grads->ddelta || !grads->dbeta || !grads->dA ||
        (in->delta_bias && !grads->ddelta_bias))
        return SSM_ERR_INVALID_ARG;
    ssm::GdrBwdArgs g;
    g.f = gdr_args(dims, in);
    if ((s = check_workspace(workspace, workspace_bytes, ssm::gdr_bwd_ws_bytes(g.f))) != SSM_OK)
        return s;
    g.f.init = initial_state;
    g.f.workspace = workspace;
    g.dout = dout;
    g.dlast = dlast_state;
    g.dq = grads->dq;
    g.dk = grads->dk;
    g.dv = grads->dv;
    g.ddelta = grads->ddelta;
    g.dbeta = grads->dbeta;
    g.dA = grads->dA;
    g.dbias = in->delta_bias ? grads->ddelta_bias : nullptr;
    g.dinit = grads->dinitial_state;
    return status(ssm::launch_gdr_bwd(g, st));
}

ssm_status gated_norm_fwd(const norm_dims *dims, const void *x, const void *z, const float *weight,
                          int norm_before_gate, void *out, void *stream)
{
    ssm_status s = check_norm_dims(dims);
    if (s != SSM_OK)
        return s;
    if (dims->rows == 0)
        return SSM_OK;
    if (!x || !weight || !out)
        return SSM_ERR_INVALID_ARG;
    const void *p[] = {x, z, weight, out};
    if ((s = aligned(p)) != SSM_OK)
        return s;
    ssm::GatedArgs a;
    memset(&a, 0, sizeof(a));
    a.rows = dims->rows;
    a.dim = (int)dims->dim;
    a.group = (int)dims->group;
    a.eps = dims->eps;
    a.dtype = dims->dtype == SSM_F32 ? 0 : 1;
    a.norm_first = norm_before_gate ? 1 : 0;
    a.x = x;
    a.z = z;
    a.weight = weight;
    a.out = out;
    return status(ssm::launch_gated_fwd(a, static_cast<cudaStream_t>(stream)));
}

size_t gated_norm_bwd_workspace_size(const norm_dims *dims)
{
    if (check_norm_dims(dims) != SSM_OK || dims->rows == 0)
        return 0;
    return ssm::gated_bwd_workspace(dims->rows, (int)dims->dim, (int)dims->group);
}

ssm_status gated_norm_bwd(const norm_dims *dims, const void *x, const void *z, const float *weight,
                          int norm_before_gate, const void *dout, void *dx, void *dz, float *dweight,
                          void *workspace, size_t workspace_bytes, void *stream)
{
    ssm_status s = check_norm_dims(dims);
    if (s != SSM_OK)
        return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const void *p[] = {x, z, weight, dout, dx, dz, dweight};
    if ((s = aligned(p)) != SSM_OK)
        return s;
    if (dims->rows == 0)
        return zero_f32(dweight, dims->dim, st);
    if (!x || !weight || !dout || !dx || !dweight || (z && !dz))
        return SSM_ERR_INVALID_ARG;
    if ((s = check_workspace(workspace, workspace_bytes, gated_norm_bwd_workspace_size(dims))) != SSM_OK)
        return s;
    ssm::GatedArgs a;
    memset(&a, 0, sizeof(a));
    a.rows = dims->rows;
    a.dim = (int)dims->dim;
    a.group = (int)dims->group;
    a.eps = dims->eps;
    a.dtype = dims->dtype == SSM_F32 ? 0 : 1;
    a.norm_first = norm_before_gate ? 1 : 0;
    a.x = x;
    a.z = z;
    a.dout = dout;
    a.weight = weight;
    a.dx = dx;
    a.dz = z ? dz : nullptr;
    a.dweight = dweight;
    a.parts = static_cast<float *>(workspace);
    return status(ssm::launch_gated_bwd(a, st));
}

ssm_status residual_norm_fwd(const norm_dims *dims, const residual_norm_params *p, const void *x,
                             const void *residual, void *residual_out, void *out, void *stream)
{
    ssm_status s = check_residual(dims, p);
    if (s != SSM_OK)
        return s;
    if (dims->rows == 0)
        return SSM_OK;
    if (!x || !residual_out || !out)
        return SSM_ERR_INVALID_ARG;
    const void *q[] = {x, residual, residual_out, out};
    if ((s = aligned(q)) != SSM_OK)
        return s;
    ssm::ResidualArgs a = residual_args(dims, p);
    a.x = x;
    a.residual = residual;
    a.res_out = residual_out;
    a.out = out;
    return status(ssm::launch_residual_fwd(a, static_cast<cudaStream_t>(stream)));
}

size_t residual_norm_bwd_workspace_size(const norm_dims *dims, const residual_norm_params *p)
{
    if (check_residual(dims, p) != SSM_OK || dims->rows == 0)
        return 0;
    return ssm::residual_bwd_workspace(dims->rows, p->samples, (int)dims->dim, p->bias != nullptr,
                                       p->scale != nullptr, p->post_weight != nullptr);
}

ssm_status residual_norm_bwd(const norm_dims *dims, const residual_norm_params *p, const void *x,
                             const void *residual_out, const void *dout, const void *dresidual_out,
                             const residual_norm_grads *grads, void *workspace, size_t workspace_bytes,
                             void *stream)
{
    ssm_status s = check_residual(dims, p);
    if (s != SSM_OK)
        return s;
    if (!grads || !grads->dweight || (p->bias && !grads->dbias) || (p->scale && !grads->dscale) ||
        (p->post_weight && !grads->dpost_weight))
        return SSM_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const void *q[] = {x, residual_out, dout, dresidual_out, grads->dx, grads->dresidual, grads->dweight,
                       grads->dbias, grads->dscale, grads->dpost_weight};
    if ((s = aligned(q)) != SSM_OK)
        return s;
    if (dims->rows == 0) {
        if ((s = zero_f32(grads->dweight, dims->dim, st)) != SSM_OK ||
            (s = zero_f32(p->bias ? grads->dbias : nullptr, dims->dim, st)) != SSM_OK ||
            (s = zero_f32(p->scale ? grads->dscale : nullptr, (size_t)p->samples * dims->dim, st)) != SSM_OK)
            return s;
        return zero_f32(p->post_weight ? grads->dpost_weight : nullptr, dims->dim, st);
    }
    if (!residual_out || !dout || !grads->dx || ((p->scale || p->post_weight) && !x))
        return SSM_ERR_INVALID_ARG;
    if ((s = check_workspace(workspace, workspace_bytes, residual_norm_bwd_workspace_size(dims, p))) != SSM_OK)
        return s;
    ssm::ResidualArgs a = residual_args(dims, p);
    a.x = x;
    a.res_out = const_cast<void *>(residual_out);
    a.dout = dout;
    a.dres_out = dresidual_out;
    a.dx = grads->dx;
    a.dres = grads->dresidual;
    a.dweight = grads->dweight;
    a.dbias = grads->dbias;
    a.dscale = grads->dscale;
    a.dpost = grads->dpost_weight;
    a.parts = static_cast<float *>(workspace);
    return status(ssm::launch_residual_bwd(a, st));
}

}  // extern "C"
