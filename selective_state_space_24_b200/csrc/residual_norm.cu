// residual_norm.cu -- the residual stream between two blocks and the next
// block's norm, and its gradients.  Per row:
//     t = x, or x p post with p = (mean x^2 + eps)^-1/2
//     r = alpha residual + scale t   (rounded to the stream's type)
//     out = n(r) weight + bias,   n(r) = (r - m) k,  k = (mean (r - m)^2 + eps)^-1/2
// with m = mean(r) for the layer norm, 0 for the RMS norm.  Backward, from
// g = dout weight and y = n(r):
//     dr = dres_out + k (g - y mean(g y) [- mean(g)]),  dresidual = alpha dr
//     dscale = sum dr t,  dt = dr scale
//     dpost = sum dt x p, e = dt post,  dx = p (e - x p mean(e x p))   (dx = dt without post)
//     dweight = sum dout y, dbias = sum dout
//
// Bound by HBM: one pass, a row stays in registers through up to four
// dependent sums (the mean is taken off before the squares, which keeps the
// variance exact for rows far from zero).  Thread layout and column sums as
// in gated_norm.cu; with a scale per sample a block's rows are of one sample.
// residual_out is rounded once to its type and the norm reads that value, so
// the backward pass, which gets residual_out, differentiates what was computed.
//
// Measured on B200, bf16 with a float32 stream: forward, 16 rows of 1024 (a
// decode batch) 14.5 us a call, launch and host; 12608 rows of 384, layer norm,
// 14.2 us on the device (4.1 TB/s), 16.6 a call, the RMS norm 10.1.  Backward
// of 16384 rows of 1024 with post-norm and scale per sample 82 us (3.7 TB/s, 0.56 of a
// copy): three dependent row sums, each a barrier of the row's warps, between a
// row's loads and stores; without either 50 us (0.82).  float32: 72 and 65 us (0.86,
// 0.79).  Rows above 4096 spill (norm_threads): 4096 rows of 8192, with both, bf16
// 243 us (0.38), float32 300 (0.41).
#include <type_traits>

#include "norm_common.cuh"

namespace ssm {
namespace {

// The sets of rows that never share a block: the samples where a scale's
// gradient is summed over each of them, else all rows are one.
int64_t row_sets(int64_t samples, bool has_scale) { return has_scale ? samples : 1; }

// A row's (mean square + eps)^-1/2 from its registers, with LAYER after the
// mean is taken off in place.  The float32 mean of a row far from zero is off
// by some steps of that mean; the sum of the centred values (exact differences,
// so the product is rounded before it is taken off) shows by how much, and the
// squares are summed when that is off too.  Both in one sum, off^2 taken off the
// mean square afterwards, saves 1 us of 14.5 (12608 rows of 384), but leaves
// rows that vary by less than that error, or not at all, a variance of rounding
// errors, which may be negative.
template <bool LAYER, int NV, int E>
__device__ __forceinline__ float norm_stats(float (&r)[NV][E], const bool (&in)[NV], float n, float inv, float eps,
                                            int tpr, RedSmem &red, int &turn)
{
    if (LAYER)
#pragma unroll
        for (int pass = 0; pass < 2; pass++) {   // the mean, then what its rounding left
            float m[1] = {0.f};
#pragma unroll
            for (int v = 0; v < NV; v++)
#pragma unroll
                for (int e = 0; e < E; e++)
                    m[0] += r[v][e];   // zero outside the row
            row_sum<1>(m, tpr, red, turn);
            m[0] = pass == 0 ? __fmul_rn(m[0], inv) : mean_of(m[0], n, inv);
#pragma unroll
            for (int v = 0; v < NV; v++)
#pragma unroll
                for (int e = 0; e < E; e++)
                    r[v][e] = in[v] ? r[v][e] - m[0] : 0.f;
        }
    float s[1] = {0.f};
#pragma unroll
    for (int v = 0; v < NV; v++)
#pragma unroll
        for (int e = 0; e < E; e++)
            s[0] = fmaf(r[v][e], r[v][e], s[0]);
    row_sum<1>(s, tpr, red, turn);
    return rsqrtf(s[0] * inv + eps);
}

template <typename R> __device__ __forceinline__ float rounded(float v);
template <> __device__ __forceinline__ float rounded<float>(float v) { return v; }
template <> __device__ __forceinline__ float rounded<__nv_bfloat16>(float v)
{
    return __bfloat162float(__float2bfloat16_rn(v));
}

template <typename T, typename R, int ELEMS, bool LAYER>
__global__ void __launch_bounds__(512) residual_fwd_kernel(const ResidualArgs a, int tpr, int rpb)
{
    constexpr int E = Vec<T>::N, NV = ELEMS / E;
    __shared__ RedSmem red;
    const int lane_r = threadIdx.x % tpr, sub = threadIdx.x / tpr;
    const int nv = a.dim / E;
    const T *x = static_cast<const T *>(a.x);
    const R *res = static_cast<const R *>(a.residual);
    const float inv = 1.f / (float)a.dim;
    const int64_t per = a.rows / a.samples;
    int turn = 0;
    bool in[NV];
#pragma unroll
    for (int v = 0; v < NV; v++)
        in[v] = lane_r + v * tpr < nv;
    Raw<T, NV, E> xr;   // of the next row
    Raw<R, NV, E> rr;
    auto fetch = [&](int64_t r0) {
        const bool live = r0 + sub < a.rows;
        const int64_t base = live ? (r0 + sub) * a.dim : 0;
        xr.load(x + base, lane_r, tpr, in, live);
        if (res)
            rr.load(res + base, lane_r, tpr, in, live);
    };
    const int64_t stride = (int64_t)gridDim.x * rpb;
    fetch((int64_t)blockIdx.x * rpb);
    for (int64_t r0 = (int64_t)blockIdx.x * rpb; r0 < a.rows; r0 += stride) {
        const int64_t row = r0 + sub;
        const bool live = row < a.rows;
        float t[NV][E], rv[NV][E];
        xr.get(t);
        if (res)
            rr.get(rv);
        if (r0 + stride < a.rows)
            fetch(r0 + stride);
        if (a.post) {
            float s[1] = {0.f};
#pragma unroll
            for (int v = 0; v < NV; v++)
#pragma unroll
                for (int e = 0; e < E; e++)
                    s[0] = fmaf(t[v][e], t[v][e], s[0]);
            row_sum<1>(s, tpr, red, turn);
            const float p = rsqrtf(s[0] * inv + a.eps);
#pragma unroll
            for (int v = 0; v < NV; v++)
                if (in[v]) {
                    float w[E];
                    load_f32<E>(a.post + (lane_r + v * tpr) * E, w);
#pragma unroll
                    for (int e = 0; e < E; e++)
                        t[v][e] *= p * w[e];
                }
        }
#pragma unroll
        for (int v = 0; v < NV; v++) {
            if (a.scale && live && in[v]) {
                float w[E];
                load_f32<E>(a.scale + (a.samples == 1 ? 0 : row / per) * a.dim + (lane_r + v * tpr) * E, w);
#pragma unroll
                for (int e = 0; e < E; e++)
                    t[v][e] *= w[e];
            }
#pragma unroll
            for (int e = 0; e < E; e++)
                rv[v][e] = rounded<R>(res ? fmaf(a.alpha, rv[v][e], t[v][e]) : t[v][e]);
            if (live && in[v])
                store_row<R, E>(static_cast<R *>(a.res_out) + row * a.dim + (lane_r + v * tpr) * E, rv[v]);
        }
        const float k = norm_stats<LAYER>(rv, in, a.fdim, inv, a.eps, tpr, red, turn);
#pragma unroll
        for (int v = 0; v < NV; v++)
            if (live && in[v]) {
                const int c = (lane_r + v * tpr) * E;
                float w[E], b[E], o[E];
                load_f32<E>(a.weight + c, w);
#pragma unroll
                for (int e = 0; e < E; e++)
                    b[e] = 0.f;
                if (a.bias)
                    load_f32<E>(a.bias + c, b);
#pragma unroll
                for (int e = 0; e < E; e++)
                    o[e] = fmaf(rv[v][e] * k, w[e], b[e]);
                store_row<T, E>(static_cast<T *>(a.out) + row * a.dim + c, o);
            }
    }
}

// A variant for each set of column sums (registers for the others are not kept).
template <typename T, typename R, int ELEMS, bool LAYER, bool BIAS, bool SCALE, bool POST>
__global__ void __launch_bounds__(512) residual_bwd_kernel(const ResidualArgs a, int tpr, int rpb, int parts)
{
    constexpr int E = Vec<T>::N, NV = ELEMS / E;
    __shared__ RedSmem red;
    extern __shared__ float cols[];   // (dim)
    const int lane_r = threadIdx.x % tpr, sub = threadIdx.x / tpr;
    const int nv = a.dim / E;
    const int64_t set = blockIdx.x / parts;
    const int part = blockIdx.x % parts;
    const int64_t per = SCALE ? a.rows / a.samples : a.rows;
    const int64_t row_end = (set + 1) * per;
    const float inv = 1.f / (float)a.dim;
    int turn = 0;
    bool in[NV];
    float dw[NV][E], db[BIAS ? NV : 1][E], dsc[SCALE ? NV : 1][E], dpo[POST ? NV : 1][E];
#pragma unroll
    for (int v = 0; v < NV; v++) {
        in[v] = lane_r + v * tpr < nv;
#pragma unroll
        for (int e = 0; e < E; e++) {
            dw[v][e] = 0.f;
            if (BIAS)
                db[v][e] = 0.f;
            if (SCALE)
                dsc[v][e] = 0.f;
            if (POST)
                dpo[v][e] = 0.f;
        }
    }
    Raw<R, NV, E> yr, sr;   // of the next row
    Raw<T, NV, E> gr, xr;
    auto fetch = [&](int64_t r0) {
        const bool live = r0 + sub < row_end;
        const int64_t base = live ? (r0 + sub) * a.dim : 0;
        yr.load(static_cast<const R *>(a.res_out) + base, lane_r, tpr, in, live);
        gr.load(static_cast<const T *>(a.dout) + base, lane_r, tpr, in, live);
        if (a.dres_out)
            sr.load(static_cast<const R *>(a.dres_out) + base, lane_r, tpr, in, live);
        if (SCALE || POST)
            xr.load(static_cast<const T *>(a.x) + base, lane_r, tpr, in, live);
    };
    const int64_t stride = (int64_t)parts * rpb;
    fetch(set * per + (int64_t)part * rpb);
    for (int64_t r0 = set * per + (int64_t)part * rpb; r0 < row_end; r0 += stride) {
        const int64_t row = r0 + sub;
        const bool live = row < row_end;
        float y[NV][E], g[NV][E];   // the stream (then its norm), dout weight (then dr)
        float d[NV][E], t[NV][E];   // the gradient of the stream's later uses, x
        const Raw<T, NV, E> gc = gr;
        yr.get(y);
#pragma unroll
        for (int v = 0; v < NV; v++)
#pragma unroll
            for (int e = 0; e < E; e++)
                d[v][e] = 0.f;
        if (a.dres_out)
            sr.get(d);
        if (SCALE || POST)
            xr.get(t);
        if (r0 + stride < row_end)
            fetch(r0 + stride);
        // the sums that need nothing else go together: of r^2, g r and x^2; for
        // the layer norm of r, g and x^2, then of what the mean left of r (as in
        // norm_stats), then of r^2 and g r
#pragma unroll
        for (int v = 0; v < NV; v++) {
            gc.get(v, g[v]);
            float w[E];
#pragma unroll
            for (int e = 0; e < E; e++)
                w[e] = 0.f;
            if (in[v])
                load_f32<E>(a.weight + (lane_r + v * tpr) * E, w);
#pragma unroll
            for (int e = 0; e < E; e++)
                g[v][e] *= w[e];
        }
        float sx = 0.f, mg = 0.f;
        if (POST)
#pragma unroll
            for (int v = 0; v < NV; v++)
#pragma unroll
                for (int e = 0; e < E; e++)
                    sx = fmaf(t[v][e], t[v][e], sx);
        if (LAYER) {
            float m[3] = {0.f, 0.f, sx}, off[1] = {0.f};
#pragma unroll
            for (int v = 0; v < NV; v++)
#pragma unroll
                for (int e = 0; e < E; e++) {
                    m[0] += y[v][e];
                    m[1] += g[v][e];
                }
            row_sum<3>(m, tpr, red, turn);
            const float mean = __fmul_rn(m[0], inv);
            mg = m[1] * inv;
            sx = m[2];
#pragma unroll
            for (int v = 0; v < NV; v++)
#pragma unroll
                for (int e = 0; e < E; e++) {
                    y[v][e] = in[v] ? y[v][e] - mean : 0.f;
                    off[0] += y[v][e];
                }
            row_sum<1>(off, tpr, red, turn);
            off[0] = mean_of(off[0], a.fdim, inv);
#pragma unroll
            for (int v = 0; v < NV; v++)
#pragma unroll
                for (int e = 0; e < E; e++)
                    y[v][e] -= in[v] ? off[0] : 0.f;
        }
        float s[3] = {0.f, 0.f, sx};
#pragma unroll
        for (int v = 0; v < NV; v++)
#pragma unroll
            for (int e = 0; e < E; e++) {
                s[0] = fmaf(y[v][e], y[v][e], s[0]);
                s[1] = fmaf(g[v][e], y[v][e], s[1]);
            }
        row_sum<LAYER ? 2 : 3>(s, tpr, red, turn);
        if (!LAYER)
            sx = s[2];
        // behind the last row 0, so that eps = 0 leaves no 0 / 0 in dweight
        const float k = live ? rsqrtf(s[0] * inv + a.eps) : 0.f;
        const float mgy = k * (s[1] * inv);   // mean(g y)
#pragma unroll
        for (int v = 0; v < NV; v++)
            if (in[v]) {
                float o[E];   // dout
                gc.get(v, o);
#pragma unroll
                for (int e = 0; e < E; e++) {
                    y[v][e] *= k;
                    dw[v][e] = fmaf(o[e], y[v][e], dw[v][e]);
                    if (BIAS)
                        db[v][e] += o[e];
                }
            }
#pragma unroll
        for (int v = 0; v < NV; v++)
            if (live && in[v]) {
                const int64_t at = row * a.dim + (lane_r + v * tpr) * E;
                float o[E];
#pragma unroll
                for (int e = 0; e < E; e++) {
                    g[v][e] = fmaf(k, fmaf(-y[v][e], mgy, g[v][e] - mg), d[v][e]);
                    o[e] = a.alpha * g[v][e];
                }
                if (a.dres)
                    store_row<R, E>(static_cast<R *>(a.dres) + at, o);
            }
        if (SCALE || POST) {
            const float p = POST ? rsqrtf(sx * inv + a.eps) : 1.f;
            float se[1] = {0.f};   // sum of e x p
#pragma unroll
            for (int v = 0; v < NV; v++)
                if (live && in[v]) {
                    const int c = (lane_r + v * tpr) * E;
                    float w[E];
                    if (POST) {
                        load_f32<E>(a.post + c, w);
#pragma unroll
                        for (int e = 0; e < E; e++)
                            t[v][e] *= p;
                    }
                    if (SCALE) {
                        float sc[E];
                        load_f32<E>(a.scale + set * a.dim + c, sc);
#pragma unroll
                        for (int e = 0; e < E; e++) {
                            dsc[v][e] = fmaf(g[v][e], POST ? t[v][e] * w[e] : t[v][e], dsc[v][e]);
                            g[v][e] *= sc[e];
                        }
                    }
                    if (POST)
#pragma unroll
                        for (int e = 0; e < E; e++) {
                            dpo[v][e] = fmaf(g[v][e], t[v][e], dpo[v][e]);
                            g[v][e] *= w[e];
                            se[0] = fmaf(g[v][e], t[v][e], se[0]);
                        }
                }
            if (POST) {
                row_sum<1>(se, tpr, red, turn);
                const float me = se[0] * inv;
#pragma unroll
                for (int v = 0; v < NV; v++)
#pragma unroll
                    for (int e = 0; e < E; e++)
                        g[v][e] = p * fmaf(-t[v][e], me, g[v][e]);
            }
        }
#pragma unroll
        for (int v = 0; v < NV; v++)
            if (live && in[v])
                store_row<T, E>(static_cast<T *>(a.dx) + row * a.dim + (lane_r + v * tpr) * E, g[v]);
    }
    // partial column sums: kind after kind, (sets, parts, dim) each
    float *out = a.parts + (size_t)blockIdx.x * a.dim;
    const size_t kind = (size_t)gridDim.x * a.dim;
    auto put = [&](const float(&d)[NV][E]) {
        for (int s = 0; s < rpb; s++) {
            if (s == sub)
#pragma unroll
                for (int v = 0; v < NV; v++)
                    if (in[v])
#pragma unroll
                        for (int e = 0; e < E; e++) {
                            const int c = (lane_r + v * tpr) * E + e;
                            cols[c] = s == 0 ? d[v][e] : cols[c] + d[v][e];
                        }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < a.dim; c += blockDim.x)
            out[c] = cols[c];
        __syncthreads();
        out += kind;
    };
    put(dw);
    if constexpr (BIAS)
        put(db);
    if constexpr (SCALE)
        put(dsc);
    if constexpr (POST)
        put(dpo);
}

template <typename T, typename R> cudaError_t fwd_typed(const ResidualArgs &a, cudaStream_t st)
{
    const NormPlan p = norm_threads(a.dim);
    auto go = [&](auto kernel) {
        const int64_t n = parts_for(a.rows, 1, p, resident_blocks(kernel, p.threads, 0));
        kernel<<<(unsigned)n, p.threads, 0, st>>>(a, p.tpr, p.rows_at_once);
    };
    if (p.elems == 8)
        a.layer ? go(residual_fwd_kernel<T, R, 8, true>) : go(residual_fwd_kernel<T, R, 8, false>);
    else
        a.layer ? go(residual_fwd_kernel<T, R, 16, true>) : go(residual_fwd_kernel<T, R, 16, false>);
    return cudaGetLastError();
}

template <typename T, typename R> cudaError_t bwd_typed(const ResidualArgs &a, cudaStream_t st)
{
    const int64_t sets = row_sets(a.samples, a.scale != nullptr);
    const NormPlan p = norm_threads(a.dim);
    const size_t smem = a.dim * sizeof(float);
    unsigned blocks = 0;
    auto go = [&](auto elems, auto layer, auto bias, auto scale, auto post) {
        auto kernel = residual_bwd_kernel<T, R, elems.value, layer.value, bias.value, scale.value, post.value>;
        const int parts = (int)parts_for(a.rows / sets, sets, p, resident_blocks(kernel, p.threads, smem));
        blocks = (unsigned)(sets * parts);
        kernel<<<blocks, p.threads, smem, st>>>(a, p.tpr, p.rows_at_once, parts);
    };
    const std::true_type yes;
    const std::false_type no;
    auto post = [&](auto n, auto l, auto b, auto s) { a.post ? go(n, l, b, s, yes) : go(n, l, b, s, no); };
    auto scale = [&](auto n, auto l, auto b) { a.scale ? post(n, l, b, yes) : post(n, l, b, no); };
    auto bias = [&](auto n, auto l) { a.bias ? scale(n, l, yes) : scale(n, l, no); };
    auto layer = [&](auto n) { a.layer ? bias(n, yes) : bias(n, no); };
    p.elems == 8 ? layer(std::integral_constant<int, 8>()) : layer(std::integral_constant<int, 16>());
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    PartSum sums[kMaxSums];
    int n = 0;
    auto sum = [&](float *out, int64_t of) {   // per set of rows, or over all of them
        sums[n] = PartSum{a.parts + (size_t)n * blocks * a.dim, out, of, (int)(blocks / of)};
        n++;
    };
    sum(a.dweight, 1);
    if (a.bias)
        sum(a.dbias, 1);
    if (a.scale)
        sum(a.dscale, sets);
    if (a.post)
        sum(a.dpost, 1);
    return launch_part_sums(sums, n, a.dim, st);
}

}  // namespace

size_t residual_bwd_workspace(int64_t rows, int64_t samples, int dim, bool has_bias, bool has_scale, bool has_post)
{
    const int64_t sets = row_sets(samples, has_scale);
    const size_t kinds = 1 + has_bias + has_scale + has_post;
    const NormPlan p = norm_threads(dim);
    return kinds * (size_t)sets * parts_for(rows / sets, sets, p, (int64_t)kSMs * (2048 / p.threads)) * dim * sizeof(float);
}

cudaError_t launch_residual_fwd(const ResidualArgs &a, cudaStream_t st)
{
    if (a.dtype == 0)
        return fwd_typed<float, float>(a, st);
    return a.res32 ? fwd_typed<__nv_bfloat16, float>(a, st) : fwd_typed<__nv_bfloat16, __nv_bfloat16>(a, st);
}

cudaError_t launch_residual_bwd(const ResidualArgs &a, cudaStream_t st)
{
    if (a.dtype == 0)
        return bwd_typed<float, float>(a, st);
    return a.res32 ? bwd_typed<__nv_bfloat16, float>(a, st) : bwd_typed<__nv_bfloat16, __nv_bfloat16>(a, st);
}

}  // namespace ssm
