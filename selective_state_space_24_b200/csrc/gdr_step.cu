// gdr_step.cu -- the gated delta rule step by step with the state in
// registers: one decode token (gdr_step), and sequences too short for the
// chunked kernel.  Per value head and step, S (V, K):
//     S = a S;  u = v - S k;  S = S + b u k^T;  out = S q~
// As out = a (S q~) + b u (k . q~), both products with the old state are
// taken together and the state is passed over once.
//
// The state is the only large operand (V K float32 per head, read and
// written once per call), so a single step is bound by HBM.  A warp owns
// kRows rows of one head's state, its lanes the columns (512 or 256
// contiguous bytes a row); all rows are loaded before anything else.  The
// 2 kRows row sums go through a butterfly that halves the values at each
// exchange (16 shuffles for 16 sums instead of 80).
//
// Measured on B200, K = V = 128, 32 heads, bf16: batch 256 160-165 us, 1.08 GB
// of states and operands at 6.6 TB/s, the rate of a copy; batch 1 4 us on the
// device, of some 14 us a call.  A sequence costs 0.54 us a step.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdr_math.cuh"

namespace ssm {
namespace {

constexpr int kRows = 8;      // state rows per warp
constexpr int kWarps = 4;     // 32 rows per block

template <int C> struct Lanes;   // C consecutive elements of a lane
template <> struct Lanes<4> {
    static __device__ __forceinline__ void load(const float *p, float (&f)[4])
    {
        const float4 v = *reinterpret_cast<const float4 *>(p);
        f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
    }
    static __device__ __forceinline__ void load(const __nv_bfloat16 *p, float (&f)[4])
    {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        f[0] = __uint_as_float(v.x << 16), f[1] = __uint_as_float(v.x & 0xffff0000u);
        f[2] = __uint_as_float(v.y << 16), f[3] = __uint_as_float(v.y & 0xffff0000u);
    }
    static __device__ __forceinline__ void store(float *p, const float (&f)[4])
    {
        *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
    }
};
template <> struct Lanes<2> {
    static __device__ __forceinline__ void load(const float *p, float (&f)[2])
    {
        const float2 v = *reinterpret_cast<const float2 *>(p);
        f[0] = v.x, f[1] = v.y;
    }
    static __device__ __forceinline__ void load(const __nv_bfloat16 *p, float (&f)[2])
    {
        const uint32_t v = *reinterpret_cast<const uint32_t *>(p);
        f[0] = __uint_as_float(v << 16), f[1] = __uint_as_float(v & 0xffff0000u);
    }
    static __device__ __forceinline__ void store(float *p, const float (&f)[2])
    {
        *reinterpret_cast<float2 *>(p) = make_float2(f[0], f[1]);
    }
};

template <typename T, int K>
__global__ void __launch_bounds__(kWarps * 32) gdr_recurrent_kernel(const GdrArgs a)
{
    constexpr int C = K / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int slices = a.V / (kRows * kWarps);
    const int64_t bh = blockIdx.x / slices;
    const int v0 = ((int)(blockIdx.x % slices) * kWarps + warp) * kRows;
    const int h = (int)(bh % a.Hv), hk = h / (a.Hv / a.Hk);
    const int64_t b = bh / a.Hv;

    float S[kRows][C];
    const size_t srow = ((size_t)bh * a.V + v0) * K + lane * C;
#pragma unroll
    for (int r = 0; r < kRows; r++) {
        if (a.init)
            Lanes<C>::load(a.init + srow + (size_t)r * K, S[r]);
        else
#pragma unroll
            for (int c = 0; c < C; c++)
                S[r][c] = 0.f;
    }
    const float Ah = a.A[h] * kLog2e, bias = a.bias ? a.bias[h] : 0.f;
    const T *qp = static_cast<const T *>(a.q), *kp = static_cast<const T *>(a.k), *vp = static_cast<const T *>(a.v);
    const T *dp = static_cast<const T *>(a.delta), *bp = static_cast<const T *>(a.beta);
    T *op = static_cast<T *>(a.out);

    // the butterfly leaves lane l with the sum of row (l >> 1) & 7 of S k
    // (lanes 0..15) or S q~ (lanes 16..31), low bit shared
    const int mine = (lane >> 1) & 7;
    float k[C], q[C], kn[C], qn[C], vv, vn, dl, dn, be, bn;
    auto fetch = [&](int t, float (&kk)[C], float (&qq)[C], float &v1, float &d1, float &b1) {
        const size_t tok = (size_t)b * a.L + t;
        Lanes<C>::load(kp + (tok * a.Hk + hk) * K + lane * C, kk);
        Lanes<C>::load(qp + (tok * a.Hk + hk) * K + lane * C, qq);
        v1 = gdr_ld(vp, (tok * a.Hv + h) * a.V + v0 + mine);
        d1 = gdr_ld(dp, tok * a.Hv + h);
        b1 = gdr_ld(bp, tok * a.Hv + h);
    };
    fetch(0, k, q, vv, dl, be);
    for (int t = 0; t < a.L; t++) {
        if (t + 1 < a.L)
            fetch(t + 1, kn, qn, vn, dn, bn);   // the next step's, in flight during this one
        const float dec = ex2_mufu(gdr_dt(dl, bias, a.softplus) * Ah);
        const float wb = a.sigmoid ? sigmoid_mufu(be) : be;
        float kk = 0.f, qq = 0.f, kq = 0.f;
#pragma unroll
        for (int c = 0; c < C; c++) {
            kk = fmaf(k[c], k[c], kk);
            qq = fmaf(q[c], q[c], qq);
            kq = fmaf(k[c], q[c], kq);
        }
        float sum[2 * kRows];
#pragma unroll
        for (int r = 0; r < kRows; r++) {
            sum[r] = sum[kRows + r] = 0.f;
#pragma unroll
            for (int c = 0; c < C; c++) {
                sum[r] = fmaf(S[r][c], k[c], sum[r]);
                sum[kRows + r] = fmaf(S[r][c], q[c], sum[kRows + r]);
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            kk += __shfl_xor_sync(0xffffffffu, kk, o);
            qq += __shfl_xor_sync(0xffffffffu, qq, o);
            kq += __shfl_xor_sync(0xffffffffu, kq, o);
        }
#pragma unroll
        for (int n = kRows, o = 16; n > 0; n >>= 1, o >>= 1) {
            const bool up = lane & o;
#pragma unroll
            for (int i = 0; i < n; i++) {
                const float send = up ? sum[i] : sum[i + n], keep = up ? sum[i + n] : sum[i];
                sum[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
            }
        }
        sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], 1);
        const float rk = a.l2norm ? rsqrtf(kk + kL2Eps) : 1.f;
        const float rq = a.scale * (a.l2norm ? rsqrtf(qq + kL2Eps) : 1.f);
        // lanes 0..15: u = v - a rk (S k) of row `mine`, and b u rk for the update
        const float u = wb * fmaf(-dec * rk, sum[0], vv);
        const float uk = __shfl_sync(0xffffffffu, u, lane & 15);   // the same row's u in lanes 16..31
        if (lane >= 16 && !(lane & 1))
            gdr_st(op, ((((size_t)b * a.L + t) * a.Hv + h) * a.V) + v0 + mine,
                   rq * fmaf(dec, sum[0], uk * rk * kq));
#pragma unroll
        for (int r = 0; r < kRows; r++) {
            const float ur = rk * __shfl_sync(0xffffffffu, u, 2 * r);
#pragma unroll
            for (int c = 0; c < C; c++)
                S[r][c] = fmaf(ur, k[c], dec * S[r][c]);
        }
#pragma unroll
        for (int c = 0; c < C; c++)
            k[c] = kn[c], q[c] = qn[c];
        vv = vn, dl = dn, be = bn;
    }
    if (a.last)
#pragma unroll
        for (int r = 0; r < kRows; r++)
            Lanes<C>::store(a.last + srow + (size_t)r * K, S[r]);
}

}  // namespace

cudaError_t launch_gdr_recurrent(const GdrArgs &a, cudaStream_t st)
{
    const unsigned grid = (unsigned)((int64_t)a.Bsz * a.Hv * (a.V / (kRows * kWarps)));
    auto go = [&](auto kernel) { kernel<<<grid, kWarps * 32, 0, st>>>(a); };
    if (a.dtype == 0)
        a.K == 128 ? go(gdr_recurrent_kernel<float, 128>) : go(gdr_recurrent_kernel<float, 64>);
    else
        a.K == 128 ? go(gdr_recurrent_kernel<__nv_bfloat16, 128>) : go(gdr_recurrent_kernel<__nv_bfloat16, 64>);
    return cudaGetLastError();
}

}  // namespace ssm
