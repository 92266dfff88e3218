// gdr_bwd.cu -- gradients of the gated delta rule, chunk by chunk.
//
// With q~ = scale q / |q|, k^ = k / |k| and, per chunk of 64 steps,
// cs = the inclusive sum of the log decays, G_ij = exp(cs_i - cs_j),
// e_j = exp(cs_end - cs_j), c_i = exp(cs_i), the forward pass is
//     A_ij = b_i G_ij k^_i.k^_j (j < i),  T = (I + A)^-1,  P = G o (Q~ K^T) (j <= i)
//     W = T diag(b c) K^,  U = T diag(b) V,  N = U - W S0^T
//     O = diag(c) Q~ S0^T + P N,  S1 = c_end S0 + N^T diag(e) K^
// The states S0 of all chunks are recomputed forward, then in reverse
//     dN = P^T dO + diag(e) K^ dS1^T
//     dS0 = c_end dS1 - dN^T W + dO^T diag(c) Q~
// and every chunk's gradients follow independently from S0, dS1, N and dN:
//     R' = T^T dN,  dA = -tril(R' N^T, -1),  dP = tril(dO N^T)
//     dQ~ = diag(c) dO S0 + (dP o G) K^
//     dK^ = diag(b) Y + Z,   Y = (dA o G) K^ - diag(c) R' S0
//         Z = diag(e) N dS1 + (dP o G)^T Q~ + (dA o b G)^T K^
//     dV = diag(b) R',   db_i = sum_v R'_iv v_iv + k^_i.Y_i
// A step's log decay g_t scales every path that crosses it: from a column j < t
// to a row i >= t, from the entering state to a row i >= t, from a column
// j < t to the leaving state, and from state to state:
//     dg_t = sum_{i >= t > j} E_ij + sum_{i >= t} s_i + sum_{j < t} z_j + c_end <dS1, S0>
//     E = dP o P + dA o A,  s_i = c_i (q~_i.(dO S0)_i - b_i k^_i.(R' S0)_i),  z_j = e_j k^_j.(N dS1)_j
// Taken so, nothing is added that has to cancel (row sums minus column sums
// of E would: its diagonal, and all that does not cross t).
// Sums over batch and length (dA, ddelta_bias) go through one partial sum per
// chunk, added in a fixed order; the value heads of a key head are added in
// one block.  All arithmetic is float32.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdr_math.cuh"

namespace ssm {
namespace {

constexpr int kC = 64;         // steps per chunk
constexpr int kThreads = 256;
constexpr int kSlice = 32;     // state rows of one chain block

using bf16 = __nv_bfloat16;

// What one (chunk, value head) keeps in the workspace, in floats.
struct Layout {
    int K, V, NC;
    int64_t heads;   // B Hv
    __host__ __device__ size_t per() const
    {
        return (size_t)6 * kC + 2 * kC * kC + (size_t)kC * K + 3 * (size_t)kC * V + 2 * (size_t)V * K;
    }
    __host__ __device__ size_t base(int64_t bh, int n) const { return ((size_t)bh * NC + n) * per(); }
    __host__ __device__ size_t cs() const { return 0; }                 // base-2 log decays, summed; then b
    __host__ __device__ size_t rk() const { return 2 * kC; }            // factor of a row of k
    __host__ __device__ size_t rq() const { return 3 * kC; }            // and of q (scale in it)
    __host__ __device__ size_t T() const { return 6 * kC; }
    __host__ __device__ size_t P() const { return T() + kC * kC; }
    __host__ __device__ size_t W() const { return P() + kC * kC; }
    __host__ __device__ size_t U() const { return W() + (size_t)kC * K; }
    __host__ __device__ size_t N() const { return U() + (size_t)kC * V; }
    __host__ __device__ size_t dN() const { return N() + (size_t)kC * V; }
    __host__ __device__ size_t S0() const { return dN() + (size_t)kC * V; }
    __host__ __device__ size_t dS() const { return S0() + (size_t)V * K; }
};

// acc[i][j] += sum_k a(ty + 16 i, k) b(k, tx + 16 j)
template <int RI, int RJ, class FA, class FB>
__device__ __forceinline__ void mm(float (&acc)[RI][RJ], int n, FA a, FB b)
{
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    for (int k = 0; k < n; k++) {
        float av[RI], bv[RJ];
#pragma unroll
        for (int i = 0; i < RI; i++)
            av[i] = a(ty + 16 * i, k);
#pragma unroll
        for (int j = 0; j < RJ; j++)
            bv[j] = b(k, tx + 16 * j);
#pragma unroll
        for (int i = 0; i < RI; i++)
#pragma unroll
            for (int j = 0; j < RJ; j++)
                acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
    }
}
template <int RI, int RJ> __device__ __forceinline__ void zero(float (&acc)[RI][RJ])
{
#pragma unroll
    for (int i = 0; i < RI; i++)
#pragma unroll
        for (int j = 0; j < RJ; j++)
            acc[i][j] = 0.f;
}
template <int RI, int RJ, class F> __device__ __forceinline__ void each(float (&acc)[RI][RJ], F f)
{
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
#pragma unroll
    for (int i = 0; i < RI; i++)
#pragma unroll
        for (int j = 0; j < RJ; j++)
            f(ty + 16 * i, tx + 16 * j, acc[i][j]);
}

// 64 rows of `cols` elements into shared memory (pitch cols + 1), zero from
// row `valid` on
__device__ __forceinline__ void load_rows(float *dst, const bf16 *src, size_t stride, int valid, int cols)
{
    for (int x = threadIdx.x; x < kC * cols; x += kThreads) {
        const int r = x / cols, c = x - r * cols;
        dst[r * (cols + 1) + c] = r < valid ? __bfloat162float(src[r * stride + c]) : 0.f;
    }
}
__device__ __forceinline__ void load_f(float *dst, const float *src, int rows, int cols, int pitch, int ld)
{
    for (int x = threadIdx.x; x < rows * cols; x += kThreads) {
        const int r = x / cols, c = x - r * cols;
        dst[r * pitch + c] = src[(size_t)r * ld + c];
    }
}

struct Where {
    int64_t b, bh;
    int h, hk, n, t0, valid;
};
__device__ __forceinline__ Where where(const GdrArgs &a, int NC, int64_t bh, int n)
{
    Where w;
    w.bh = bh;
    w.b = bh / a.Hv;
    w.h = (int)(bh % a.Hv);
    w.hk = w.h / (a.Hv / a.Hk);
    w.n = n;
    w.t0 = n * kC;
    w.valid = a.L - w.t0 < kC ? a.L - w.t0 : kC;
    return w;
}

// ---- 1. per chunk and value head: the scalars, T, P, W, U
__global__ void __launch_bounds__(kThreads) prep_kernel(const GdrArgs a, const Layout lay)
{
    extern __shared__ float sm[];
    const int K = a.K, V = a.V, pk = K + 1, pv = V + 1;
    const Where w = where(a, lay.NC, blockIdx.x / lay.NC, blockIdx.x % lay.NC);
    float *ws = static_cast<float *>(a.workspace) + lay.base(w.bh, w.n);
    float *Ks = sm, *Qs = Ks + kC * pk, *Vs = Qs + kC * pk, *As = Vs + kC * pv, *Ts = As + kC * 65, *vec = Ts + kC * 65;
    float *cs = vec, *bb = vec + kC, *rk = vec + 2 * kC, *rq = vec + 3 * kC;
    const size_t tok = (size_t)w.b * a.L + w.t0;
    load_rows(Ks, static_cast<const bf16 *>(a.k) + (tok * a.Hk + w.hk) * K, (size_t)a.Hk * K, w.valid, K);
    load_rows(Qs, static_cast<const bf16 *>(a.q) + (tok * a.Hk + w.hk) * K, (size_t)a.Hk * K, w.valid, K);
    load_rows(Vs, static_cast<const bf16 *>(a.v) + (tok * a.Hv + w.h) * V, (size_t)a.Hv * V, w.valid, V);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == 0) {
        const float bias = a.bias ? a.bias[w.h] : 0.f, Ah = a.A[w.h] * kLog2e;
        float g[2];
        for (int i = 0; i < 2; i++) {
            const int r = 2 * lane + i;
            g[i] = 0.f;
            bb[r] = 0.f;
            if (r < w.valid) {
                g[i] = gdr_dt(gdr_ld(static_cast<const bf16 *>(a.delta), (tok + r) * a.Hv + w.h), bias, a.softplus) * Ah;
                const float be = gdr_ld(static_cast<const bf16 *>(a.beta), (tok + r) * a.Hv + w.h);
                bb[r] = a.sigmoid ? gdr_sigmoid(be) : be;
            }
        }
        float incl = g[0] + g[1];
        for (int o = 1; o < 32; o <<= 1) {
            const float v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o)
                incl += v;
        }
        cs[2 * lane] = incl - g[1];
        cs[2 * lane + 1] = incl;
    }
    __syncthreads();
    for (int r = warp; r < kC; r += kThreads / 32) {
        float kk = 0.f, qq = 0.f;
        for (int c = lane; c < K; c += 32) {
            kk = fmaf(Ks[r * pk + c], Ks[r * pk + c], kk);
            qq = fmaf(Qs[r * pk + c], Qs[r * pk + c], qq);
        }
        kk = warp_sum(kk);
        qq = warp_sum(qq);
        if (lane == 0) {
            rk[r] = a.l2norm ? rsqrtf(kk + kL2Eps) : 1.f;
            rq[r] = a.scale * (a.l2norm ? rsqrtf(qq + kL2Eps) : 1.f);
        }
    }
    __syncthreads();
    {
        float kk[4][4], qk[4][4];
        zero(kk);
        zero(qk);
        mm(kk, K, [&](int i, int k) { return Ks[i * pk + k]; }, [&](int k, int j) { return Ks[j * pk + k]; });
        mm(qk, K, [&](int i, int k) { return Qs[i * pk + k]; }, [&](int k, int j) { return Ks[j * pk + k]; });
        each(kk, [&](int i, int j, float v) {
            As[i * 65 + j] = j < i ? bb[i] * ex2_mufu(cs[i] - cs[j]) * rk[i] * rk[j] * v : 0.f;
            Ts[i * 65 + j] = 0.f;
        });
        each(qk, [&](int i, int j, float v) {
            ws[lay.P() + i * kC + j] = j <= i ? ex2_mufu(cs[i] - cs[j]) * rq[i] * rk[j] * v : 0.f;
        });
    }
    __syncthreads();
    // (I + A)^-1 by forward substitution, a thread per column
    if (threadIdx.x < kC) {
        const int j = threadIdx.x;
        for (int i = j; i < kC; i++) {
            float v = i == j ? 1.f : 0.f;
            for (int k = j; k < i; k++)
                v = fmaf(-As[i * 65 + k], Ts[k * 65 + j], v);
            Ts[i * 65 + j] = v;
        }
    }
    __syncthreads();
    for (int x = threadIdx.x; x < kC * kC; x += kThreads)
        ws[lay.T() + x] = Ts[(x >> 6) * 65 + (x & 63)];
    for (int x = threadIdx.x; x < 4 * kC; x += kThreads)
        ws[x] = vec[x];
    for (int c0 = 0; c0 < K; c0 += 64) {
        float acc[4][4];
        zero(acc);
        mm(acc, kC, [&](int i, int k) { return Ts[i * 65 + k] * (bb[k] * ex2_mufu(cs[k]) * rk[k]); },
           [&](int k, int j) { return Ks[k * pk + c0 + j]; });
        each(acc, [&](int i, int j, float v) { ws[lay.W() + i * K + c0 + j] = v; });
    }
    for (int c0 = 0; c0 < V; c0 += 64) {
        float acc[4][4];
        zero(acc);
        mm(acc, kC, [&](int i, int k) { return Ts[i * 65 + k] * bb[k]; }, [&](int k, int j) { return Vs[k * pv + c0 + j]; });
        each(acc, [&](int i, int j, float v) { ws[lay.U() + i * V + c0 + j] = v; });
    }
}

// ---- 2. forward over the chunks, 32 state rows per block: S0 and N
template <int K> __global__ void __launch_bounds__(kThreads) chain_kernel(const GdrArgs a, const Layout lay)
{
    extern __shared__ float sm[];
    constexpr int pk = K + 1, ps = kSlice + 1;
    const int slices = a.V / kSlice;
    const int64_t bh = blockIdx.x / slices;
    const int v0 = (blockIdx.x % slices) * kSlice;
    float *Ws = sm, *Ke = Ws + kC * pk, *Ss = Ke + kC * pk, *Ns = Ss + kSlice * pk;
    for (int x = threadIdx.x; x < kSlice * K; x += kThreads)
        Ss[(x / K) * pk + x % K] = a.init ? a.init[((size_t)bh * a.V + v0) * K + x] : 0.f;
    for (int n = 0; n < lay.NC; n++) {
        const Where w = where(a, lay.NC, bh, n);
        float *ws = static_cast<float *>(a.workspace) + lay.base(bh, n);
        __syncthreads();
        load_f(Ws, ws + lay.W(), kC, K, pk, K);
        load_rows(Ke, static_cast<const bf16 *>(a.k) + (((size_t)w.b * a.L + w.t0) * a.Hk + w.hk) * K,
                  (size_t)a.Hk * K, w.valid, K);
        for (int x = threadIdx.x; x < kSlice * K; x += kThreads)
            ws[lay.S0() + (size_t)v0 * K + x] = Ss[(x / K) * pk + x % K];
        __syncthreads();
        const float end = ws[lay.cs() + kC - 1];
        float acc[4][2];
        zero(acc);
        mm(acc, K, [&](int i, int k) { return Ws[i * pk + k]; }, [&](int k, int j) { return Ss[j * pk + k]; });
        each(acc, [&](int i, int j, float v) {
            const float x = ws[lay.U() + i * a.V + v0 + j] - v;
            ws[lay.N() + i * a.V + v0 + j] = x;
            Ns[i * ps + j] = x * ws[lay.rk() + i] * ex2_mufu(end - ws[lay.cs() + i]);
        });
        __syncthreads();
        float up[2][K / 16];
        zero(up);
        mm(up, kC, [&](int i, int k) { return Ns[k * ps + i]; }, [&](int k, int j) { return Ke[k * pk + j]; });
        const float dec = ex2_mufu(end);
        each(up, [&](int i, int j, float v) { Ss[i * pk + j] = fmaf(dec, Ss[i * pk + j], v); });
    }
}

// ---- 3. in reverse: dS1 and dN
template <int K> __global__ void __launch_bounds__(kThreads) reverse_kernel(const GdrBwdArgs g, const Layout lay)
{
    extern __shared__ float sm[];
    const GdrArgs &a = g.f;
    constexpr int pk = K + 1, ps = kSlice + 1;
    const int slices = a.V / kSlice;
    const int64_t bh = blockIdx.x / slices;
    const int v0 = (blockIdx.x % slices) * kSlice;
    float *Ws = sm, *Ks = Ws + kC * pk, *Qs = Ks + kC * pk, *Gs = Qs + kC * pk, *Ns = Gs + kSlice * pk,
          *Os = Ns + kC * ps, *Ps = Os + kC * ps;
    for (int x = threadIdx.x; x < kSlice * K; x += kThreads)
        Gs[(x / K) * pk + x % K] = g.dlast ? g.dlast[((size_t)bh * a.V + v0) * K + x] : 0.f;
    for (int n = lay.NC - 1; n >= 0; n--) {
        const Where w = where(a, lay.NC, bh, n);
        float *ws = static_cast<float *>(a.workspace) + lay.base(bh, n);
        const size_t tok = (size_t)w.b * a.L + w.t0;
        __syncthreads();
        load_f(Ws, ws + lay.W(), kC, K, pk, K);
        load_f(Ps, ws + lay.P(), kC, kC, 65, kC);
        load_rows(Ks, static_cast<const bf16 *>(a.k) + (tok * a.Hk + w.hk) * K, (size_t)a.Hk * K, w.valid, K);
        load_rows(Qs, static_cast<const bf16 *>(a.q) + (tok * a.Hk + w.hk) * K, (size_t)a.Hk * K, w.valid, K);
        load_rows(Os, static_cast<const bf16 *>(g.dout) + (tok * a.Hv + w.h) * a.V + v0, (size_t)a.Hv * a.V, w.valid,
                  kSlice);
        for (int x = threadIdx.x; x < kSlice * K; x += kThreads)
            ws[lay.dS() + (size_t)v0 * K + x] = Gs[(x / K) * pk + x % K];
        __syncthreads();
        const float end = ws[lay.cs() + kC - 1];
        float acc[4][2];
        zero(acc);
        mm(acc, K, [&](int i, int k) { return Ks[i * pk + k]; }, [&](int k, int j) { return Gs[j * pk + k]; });
        each(acc, [&](int i, int, float &v) { v *= ws[lay.rk() + i] * ex2_mufu(end - ws[lay.cs() + i]); });
        mm(acc, kC, [&](int i, int k) { return Ps[k * 65 + i]; }, [&](int k, int j) { return Os[k * ps + j]; });
        each(acc, [&](int i, int j, float v) {
            ws[lay.dN() + i * a.V + v0 + j] = v;
            Ns[i * ps + j] = -v;
        });
        __syncthreads();
        for (int x = threadIdx.x; x < kC * kSlice; x += kThreads) {
            const int i = x / kSlice;
            Os[i * ps + x % kSlice] *= ws[lay.rq() + i] * ex2_mufu(ws[lay.cs() + i]);
        }
        __syncthreads();
        float up[2][K / 16];
        zero(up);
        mm(up, kC, [&](int i, int k) { return Ns[k * ps + i]; }, [&](int k, int j) { return Ws[k * pk + j]; });
        mm(up, kC, [&](int i, int k) { return Os[k * ps + i]; }, [&](int k, int j) { return Qs[k * pk + j]; });
        const float dec = ex2_mufu(end);
        each(up, [&](int i, int j, float v) { Gs[i * pk + j] = fmaf(dec, Gs[i * pk + j], v); });
    }
    __syncthreads();
    if (g.dinit)
        for (int x = threadIdx.x; x < kSlice * K; x += kThreads)
            g.dinit[((size_t)bh * a.V + v0) * K + x] = Gs[(x / K) * pk + x % K];
}

// ---- 4. per chunk and key head: every gradient
template <int K, int V>
__global__ void __launch_bounds__(kThreads, 1) grad_kernel(const GdrBwdArgs g, const Layout lay, float *parts)
{
    extern __shared__ float sm[];
    const GdrArgs &a = g.f;
    constexpr int pk = K + 1, pv = V + 1, RK = K / 16, RV = V / 16;
    const int per_k = a.Hv / a.Hk;
    const int64_t bhk = blockIdx.x / lay.NC;
    const int n = blockIdx.x % lay.NC;
    const int64_t b = bhk / a.Hk;
    const int hk = (int)(bhk % a.Hk);
    float *Ks = sm, *Qs = Ks + kC * pk, *Ns = Qs + kC * pk, *Rs = Ns + kC * pv, *Os = Rs + kC * pv, *Xs = Os + kC * pv,
          *vec = Xs + kC * 65;
    float *cs = vec, *bb = vec + kC, *rk = vec + 2 * kC, *rq = vec + 3 * kC, *dcs = vec + 4 * kC, *db = vec + 5 * kC,
          *sv = vec + 6 * kC, *zv = vec + 7 * kC, *red = vec + 8 * kC;   // red: one value per warp
    const int t0 = n * kC, valid = a.L - t0 < kC ? a.L - t0 : kC;
    const size_t tok = (size_t)b * a.L + t0;
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    const bf16 *kp = static_cast<const bf16 *>(a.k) + (tok * a.Hk + hk) * K;
    const bf16 *qp = static_cast<const bf16 *>(a.q) + (tok * a.Hk + hk) * K;
    float dK[4][RK], dQ[4][RK];
    zero(dK);
    zero(dQ);
    // sums over a row's 16 threads of this row layout (lanes of a half warp)
    auto row_add = [&](float v) {
#pragma unroll
        for (int o = 8; o > 0; o >>= 1)
            v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    };
    for (int hh = 0; hh < per_k; hh++) {
        const int h = hk * per_k + hh;
        const int64_t bh = b * a.Hv + h;
        const float *ws = static_cast<const float *>(a.workspace) + lay.base(bh, n);
        const float *S0 = ws + lay.S0(), *dS = ws + lay.dS();
        const bf16 *vp = static_cast<const bf16 *>(a.v) + (tok * a.Hv + h) * V;
        __syncthreads();
        for (int x = threadIdx.x; x < 4 * kC; x += kThreads)
            vec[x] = ws[x];
        load_rows(Ks, kp, (size_t)a.Hk * K, valid, K);
        load_rows(Qs, qp, (size_t)a.Hk * K, valid, K);
        load_rows(Os, static_cast<const bf16 *>(g.dout) + (tok * a.Hv + h) * V, (size_t)a.Hv * V, valid, V);
        load_f(Ns, ws + lay.N(), kC, V, pv, V);
        load_f(Rs, ws + lay.dN(), kC, V, pv, V);
        load_f(Xs, ws + lay.T(), kC, kC, 65, kC);
        __syncthreads();
        for (int x = threadIdx.x; x < kC * K; x += kThreads) {
            const int r = x / K, c = x % K;
            Ks[r * pk + c] *= rk[r];
            Qs[r * pk + c] *= rq[r];
        }
        const float end = cs[kC - 1];
        // R' = T^T dN
        float r[4][RV];
        zero(r);
        mm(r, kC, [&](int i, int k) { return Xs[k * 65 + i]; }, [&](int k, int j) { return Rs[k * pv + j]; });
        __syncthreads();
        each(r, [&](int i, int j, float v) { Rs[i * pv + j] = v; });
        float dbr[4] = {};
        each(r, [&](int i, int j, float v) {
            if (i < valid) {
                static_cast<bf16 *>(g.dv)[((tok + i) * a.Hv + h) * V + j] = __float2bfloat16_rn(bb[i] * v);
                dbr[(i - ty) >> 4] = fmaf(v, __bfloat162float(vp[(size_t)i * a.Hv * V + j]), dbr[(i - ty) >> 4]);
            }
        });
        __syncthreads();
        // (dA o G) and (dP o G)
        float xa[4][4], xp[4][4];
        zero(xa);
        zero(xp);
        mm(xa, V, [&](int i, int k) { return Rs[i * pv + k]; }, [&](int k, int j) { return Ns[j * pv + k]; });
        mm(xp, V, [&](int i, int k) { return Os[i * pv + k]; }, [&](int k, int j) { return Ns[j * pv + k]; });
        each(xa, [&](int i, int j, float &v) { v = j < i ? -v * ex2_mufu(cs[i] - cs[j]) : 0.f; });
        each(xp, [&](int i, int j, float &v) { v = j <= i ? v * ex2_mufu(cs[i] - cs[j]) : 0.f; });
        __syncthreads();
        // E = dP o P + dA o A below the diagonal, then its sums along rows up
        // to each column (thread i: row i)
        {
            float kk[4][4], qk[4][4];
            zero(kk);
            zero(qk);
            mm(kk, K, [&](int i, int k) { return Ks[i * pk + k]; }, [&](int k, int j) { return Ks[j * pk + k]; });
            mm(qk, K, [&](int i, int k) { return Qs[i * pk + k]; }, [&](int k, int j) { return Ks[j * pk + k]; });
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const int row = ty + 16 * i, col = tx + 16 * j;
                    Xs[row * 65 + col] =
                        col < row ? fmaf(xp[i][j], qk[i][j], bb[row] * xa[i][j] * kk[i][j]) : 0.f;
                }
        }
        __syncthreads();
        if (threadIdx.x < kC) {
            float run = 0.f;
            for (int j = 0; j < kC; j++) {
                const float e = Xs[threadIdx.x * 65 + j];
                Xs[threadIdx.x * 65 + j] = run;   // the sum of columns < j
                run += e;
            }
        }
        __syncthreads();
        if (threadIdx.x < kC) {
            float d = 0.f;
            for (int i = threadIdx.x; i < kC; i++)
                d += Xs[i * 65 + threadIdx.x];
            dcs[threadIdx.x] = d;
        }
        __syncthreads();
        each(xa, [&](int i, int j, float v) { Xs[i * 65 + j] = v; });
        __syncthreads();
        float Y[4][RK], Z[4][RK], q[4][RK], ss[4], zz[4];
        zero(Y);
        zero(Z);
        zero(q);
        // sum over the row's threads of k^ or q~ times a row of products
        auto row_dot = [&](const float *M, const float (&m)[RK], int row) {
            float v = 0.f;
#pragma unroll
            for (int j = 0; j < RK; j++)
                v = fmaf(M[row * pk + tx + 16 * j], m[j], v);
            return row_add(v);
        };
        // Y = (dA o G) K^ - c R' S0
        mm(Y, V, [&](int i, int k) { return Rs[i * pv + k]; }, [&](int k, int j) { return S0[(size_t)k * K + j]; });
        each(Y, [&](int i, int, float &v) { v *= -ex2_mufu(cs[i]); });
#pragma unroll
        for (int i = 0; i < 4; i++)
            ss[i] = bb[ty + 16 * i] * row_dot(Ks, Y[i], ty + 16 * i);
        mm(Y, kC, [&](int i, int k) { return Xs[i * 65 + k]; }, [&](int k, int j) { return Ks[k * pk + j]; });
        // Z = e N dS1 + (dA o b G)^T K^ + (dP o G)^T Q~
        mm(Z, V, [&](int i, int k) { return Ns[i * pv + k]; }, [&](int k, int j) { return dS[(size_t)k * K + j]; });
        each(Z, [&](int i, int, float &v) { v *= ex2_mufu(end - cs[i]); });
#pragma unroll
        for (int i = 0; i < 4; i++)
            zz[i] = row_dot(Ks, Z[i], ty + 16 * i);
        mm(Z, kC, [&](int i, int k) { return bb[k] * Xs[k * 65 + i]; }, [&](int k, int j) { return Ks[k * pk + j]; });
        __syncthreads();
        each(xp, [&](int i, int j, float v) { Xs[i * 65 + j] = v; });
        __syncthreads();
        mm(Z, kC, [&](int i, int k) { return Xs[k * 65 + i]; }, [&](int k, int j) { return Qs[k * pk + j]; });
        mm(q, V, [&](int i, int k) { return Os[i * pv + k]; }, [&](int k, int j) { return S0[(size_t)k * K + j]; });
        each(q, [&](int i, int, float &v) { v *= ex2_mufu(cs[i]); });
#pragma unroll
        for (int i = 0; i < 4; i++)
            ss[i] += row_dot(Qs, q[i], ty + 16 * i);
        mm(q, kC, [&](int i, int k) { return Xs[i * 65 + k]; }, [&](int k, int j) { return Ks[k * pk + j]; });
        // c_end <dS1, S0>
        const float dec = ex2_mufu(end);
        float through = 0.f;
        for (int x = threadIdx.x; x < V * K; x += kThreads)
            through = fmaf(dec * dS[x], S0[x], through);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int row = ty + 16 * i;
#pragma unroll
            for (int j = 0; j < RK; j++) {
                dK[i][j] += fmaf(bb[row], Y[i][j], Z[i][j]);
                dQ[i][j] += q[i][j];
            }
            const float ky = row_dot(Ks, Y[i], row), dbv = row_add(dbr[i]);
            if (tx == 0) {
                sv[row] = ss[i];
                zv[row] = zz[i];
                db[row] = dbv + ky;
            }
        }
        through = warp_sum(through);
        if ((threadIdx.x & 31) == 0)
            red[threadIdx.x >> 5] = through;
        __syncthreads();
        if (threadIdx.x < 32) {
            const int lane = threadIdx.x;
            float all = 0.f;
            for (int k = 0; k < kThreads / 32; k++)
                all += red[k];
            // sums of s from each step on, of z before each step
            const float s0 = sv[2 * lane], s1 = sv[2 * lane + 1], z0 = zv[2 * lane], z1 = zv[2 * lane + 1];
            float down = s0 + s1, up = z0 + z1;
            for (int o = 1; o < 32; o <<= 1) {
                const float v = __shfl_down_sync(0xffffffffu, down, o), u = __shfl_up_sync(0xffffffffu, up, o);
                if (lane + o < 32)
                    down += v;
                if (lane >= o)
                    up += u;
            }
            const float nd = __shfl_down_sync(0xffffffffu, down, 1), pu = __shfl_up_sync(0xffffffffu, up, 1);
            const float after = lane < 31 ? nd : 0.f, before = lane > 0 ? pu : 0.f;
            const float dg[2] = {dcs[2 * lane] + down + before + all, dcs[2 * lane + 1] + s1 + after + before + z0 + all};
            const float bias = a.bias ? a.bias[h] : 0.f, Ah = a.A[h];
            float sA = 0.f, sb = 0.f;
            for (int i = 0; i < 2; i++) {
                const int row = 2 * lane + i;
                if (row < valid) {
                    const size_t at = (tok + row) * a.Hv + h;
                    const float raw = gdr_ld(static_cast<const bf16 *>(a.delta), at);
                    sA = fmaf(dg[i], gdr_dt(raw, bias, a.softplus), sA);
                    const float dd = dg[i] * Ah * (a.softplus ? gdr_sigmoid(raw + bias) : 1.f);
                    sb += dd;
                    gdr_st(static_cast<bf16 *>(g.ddelta), at, dd);
                    gdr_st(static_cast<bf16 *>(g.dbeta), at, db[row] * (a.sigmoid ? bb[row] * (1.f - bb[row]) : 1.f));
                }
            }
            sA = warp_sum(sA);
            sb = warp_sum(sb);
            if (lane == 0) {   // parts: (2, B NC, Hv)
                const size_t at = ((size_t)b * lay.NC + n) * a.Hv + h;
                parts[at] = sA;
                parts[(size_t)a.Bsz * lay.NC * a.Hv + at] = sb;
            }
        }
    }
    // through the norms: d k = rk (dk^ - k^ (k^ . dk^))
    const float inv = a.l2norm ? 1.f / a.scale : 0.f;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int row = ty + 16 * i;
        float kd = 0.f, qd = 0.f;
#pragma unroll
        for (int j = 0; j < RK; j++) {
            kd = fmaf(Ks[row * pk + tx + 16 * j], dK[i][j], kd);
            qd = fmaf(Qs[row * pk + tx + 16 * j], dQ[i][j], qd);
        }
        kd = a.l2norm ? row_add(kd) : 0.f;
        qd = a.l2norm ? row_add(qd) * inv * inv : 0.f;   // Qs holds scale q^
        if (row < valid)
#pragma unroll
            for (int j = 0; j < RK; j++) {
                const int c = tx + 16 * j;
                const size_t at = ((tok + row) * a.Hk + hk) * K + c;
                static_cast<bf16 *>(g.dk)[at] = __float2bfloat16_rn(rk[row] * fmaf(-Ks[row * pk + c], kd, dK[i][j]));
                static_cast<bf16 *>(g.dq)[at] = __float2bfloat16_rn(rq[row] * fmaf(-Qs[row * pk + c], qd, dQ[i][j]));
            }
    }
}

// ---- 5. dA and ddelta_bias: sums over batch and chunks, a warp per head
__global__ void __launch_bounds__(32) head_sum_kernel(const float *parts, int64_t n, int Hv, float *dA, float *dbias)
{
    const int h = blockIdx.x;
    float s[2] = {0.f, 0.f};
    for (int64_t k = threadIdx.x; k < n; k += 32)
        for (int i = 0; i < 2; i++)
            s[i] += parts[((size_t)i * n + k) * Hv + h];
    const float x = warp_sum(s[0]), y = warp_sum(s[1]);
    if (threadIdx.x == 0) {
        dA[h] = x;
        if (dbias)
            dbias[h] = y;
    }
}

Layout layout(const GdrArgs &a)
{
    Layout l;
    l.K = a.K;
    l.V = a.V;
    l.NC = (a.L + kC - 1) / kC;
    l.heads = (int64_t)a.Bsz * a.Hv;
    return l;
}

template <class Kern, class... Args>
cudaError_t go(Kern kernel, int64_t blocks, size_t floats, cudaStream_t st, Args... args)
{
    const size_t bytes = floats * sizeof(float);
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess)
        return e;
    kernel<<<(unsigned)blocks, kThreads, bytes, st>>>(args...);
    return cudaGetLastError();
}

}  // namespace

size_t gdr_bwd_ws_bytes(const GdrArgs &a)
{
    const Layout l = layout(a);
    return ((size_t)l.heads * l.NC * l.per() + 2 * (size_t)l.heads * l.NC) * sizeof(float);
}

cudaError_t launch_gdr_bwd(const GdrBwdArgs &g, cudaStream_t st)
{
    const GdrArgs &a = g.f;
    const Layout l = layout(a);
    float *parts = static_cast<float *>(a.workspace) + (size_t)l.heads * l.NC * l.per();
    const size_t pk = a.K + 1, pv = a.V + 1, ps = kSlice + 1;
    cudaError_t e = go(prep_kernel, l.heads * l.NC, 2 * kC * pk + kC * pv + 2 * kC * 65 + 4 * kC, st, a, l);
    const int64_t chains = l.heads * (a.V / kSlice);
    const size_t cf = 2 * kC * pk + kSlice * pk + kC * ps;
    if (e == cudaSuccess)
        e = a.K == 128 ? go(chain_kernel<128>, chains, cf, st, a, l) : go(chain_kernel<64>, chains, cf, st, a, l);
    const size_t rf = 3 * kC * pk + kSlice * pk + 2 * kC * ps + kC * 65;
    if (e == cudaSuccess)
        e = a.K == 128 ? go(reverse_kernel<128>, chains, rf, st, g, l) : go(reverse_kernel<64>, chains, rf, st, g, l);
    const int64_t blocks = (int64_t)a.Bsz * a.Hk * l.NC;
    const size_t gf = 2 * kC * pk + 3 * kC * pv + kC * 65 + 8 * kC + 16;
    if (e == cudaSuccess) {
        if (a.K == 128)
            e = a.V == 128 ? go(grad_kernel<128, 128>, blocks, gf, st, g, l, parts)
                           : go(grad_kernel<128, 64>, blocks, gf, st, g, l, parts);
        else
            e = a.V == 128 ? go(grad_kernel<64, 128>, blocks, gf, st, g, l, parts)
                           : go(grad_kernel<64, 64>, blocks, gf, st, g, l, parts);
    }
    if (e != cudaSuccess)
        return e;
    head_sum_kernel<<<a.Hv, 32, 0, st>>>(parts, (int64_t)a.Bsz * l.NC, a.Hv, g.dA, g.dbias);
    return cudaGetLastError();
}

}  // namespace ssm
