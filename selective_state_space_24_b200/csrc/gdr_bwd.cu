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
// one block.
//
// Products run on the tensor cores as tf32 (mma.sync m16n8k8).  dA and
// ddelta_bias are sums in which much cancels, so everything on the way to a
// log decay's gradient keeps float32's precision: an operand is hi + lo, both
// tf32 (11 bits each), and a product is hi hi + hi lo + lo hi; K, Q, V and dO
// as they came are bf16 and exact in hi alone.  What only reaches bf16
// results (dP, dA times K and Q) takes one tf32 part; K K^T and Q K^T are bf16
// products.  (Pairs of bf16 leave dA up to 3e-5 off where the terms cancel.)
//
// Three launches and a small sum: 1 prepares every chunk by itself, 2 and 3 walk
// the chunks with 32 state rows a block, forward and in reverse side by side on
// an SM, 4 takes every chunk by itself again.  What passes between them (T, W,
// U, P^T dO, the states: 250 KB a chunk and head for K = V = 128) goes through
// the workspace in float32.
//
// Bound by mma.sync (tf32 takes 8 clocks an instruction and SM quarter, three
// per two-part product) and the instructions that feed it: in the chains the
// tensor pipe is 41% busy and 52% of the issue slots are taken on average, 56%
// and 70% on the SMs with two blocks; HBM 13%.  Measured on B200, 2 x 2048, 8 key and 16 value heads,
// K = V = 128: 687 us (preparation 89, the chains 313, the gradients 296, the sum
// 4); 2 x 197, 6 heads of 64: 60 us, the latency of four launches.  On the way:
// 3780 us with FMA units, 890 with two-part tf32, 756 with the parts taken by
// integer operations instead of cvt.tf32 (4 clocks against 2), 711 with two
// preparation blocks per SM, 703 (and 72 -> 59 us) with the chains together: by
// themselves, with two buffers a tile, they took 135 and 174 us; 666 with V,
// delta and the second reading of S0 brought in by asynchronous copies ahead of
// their use in the gradients; 669 with the log decays as pairs, 687 with the first
// parts rounded, which halves what dA is off.  512 threads a block for the gradients were slower
// (registers), the next head's tiles brought into L2 ahead no faster.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdr_math.cuh"
#include "tc100.cuh"

namespace ssm {
namespace {

constexpr int kC = 64;         // steps per chunk
constexpr int kThreads = 256;  // eight warps: 2 x 4 over a 64-row tile
constexpr int kSlice = 32;     // state rows of one chain block

using bf16 = __nv_bfloat16;

constexpr int kScalars = 5;
// What one (chunk, value head) keeps in the workspace, in floats.
struct Layout {
    int K, V, NC;
    int64_t heads;   // B Hv
    __host__ __device__ size_t per() const { return dS() + (size_t)V * K; }
    __host__ __device__ size_t base(int64_t bh, int n) const { return ((size_t)bh * NC + n) * per(); }
    // five scalars a step: log decays (base 2), summed, as hi, b, factors of a row of k and of q, and lo
    __host__ __device__ size_t cs() const { return 0; }
    __host__ __device__ size_t rk() const { return 2 * kC; }  // factor of a row of k
    __host__ __device__ size_t rq() const { return 3 * kC; }  // and of q (scale in it)
    __host__ __device__ size_t cl() const { return 4 * kC; }
    __host__ __device__ size_t T() const { return kScalars * kC; }
    __host__ __device__ size_t W() const { return T() + kC * kC; }
    __host__ __device__ size_t U() const { return W() + (size_t)kC * K; }    // T diag(b) V, then N
    __host__ __device__ size_t dN() const { return U() + (size_t)kC * V; }   // P^T dO, then dN
    __host__ __device__ size_t S0() const { return dN() + (size_t)kC * V; }
    __host__ __device__ size_t dS() const { return S0() + (size_t)V * K; }
};

// Pitches of shared tiles (in elements).  A fragment's lanes read pairs of
// neighbouring k, either along eight rows (64 or, for bf16, 32 bits a lane) or
// down eight columns: free of bank conflicts for the way named.
constexpr int pr(int n) { return n + 8; }   // float32, k along the row
constexpr int pc(int n) { return n + 4; }   // float32, k down the column
constexpr int ph(int n) { return n + 8; }   // bf16
constexpr int kPX = pc(kC), kPN = pc(kSlice);

// An operand: the values of k and k + 1 (k even) for index i of its other dimension.
struct RowF {   // float32, k along the row
    const float *p;
    int pitch;
    __device__ __forceinline__ float2 operator()(int i, int k) const
    {
        return *reinterpret_cast<const float2 *>(p + i * pitch + k);
    }
};
struct ColF {   // float32, k down the column
    const float *p;
    int pitch;
    __device__ __forceinline__ float2 operator()(int i, int k) const
    {
        return make_float2(p[k * pitch + i], p[(k + 1) * pitch + i]);
    }
};
struct RowH {   // the same for bf16
    const __nv_bfloat16 *p;
    int pitch;
    __device__ __forceinline__ float2 operator()(int i, int k) const
    {
        const uint32_t u = *reinterpret_cast<const uint32_t *>(p + i * pitch + k);
        return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    }
};
struct ColH {
    const __nv_bfloat16 *p;
    int pitch;
    __device__ __forceinline__ float2 operator()(int i, int k) const
    {
        return make_float2(__bfloat162float(p[k * pitch + i]), __bfloat162float(p[(k + 1) * pitch + i]));
    }
};
template <class F> struct Scaled {   // times a factor of k
    F f;
    const float *v;
    __device__ __forceinline__ float2 operator()(int i, int k) const
    {
        const float2 x = f(i, k), y = *reinterpret_cast<const float2 *>(v + k);
        return make_float2(x.x * y.x, x.y * y.y);
    }
};
template <class F> __device__ __forceinline__ Scaled<F> scaled(F f, const float *v) { return Scaled<F>{f, v}; }

__device__ __forceinline__ float bf(const bf16 *p) { return __bfloat162float(*p); }

// tf32 keeps the upper 19 bits of a float32, and the product cuts off the
// rest.  The first part is rounded, so that the second has either sign and its
// cutting no bias (both cut, every operand is a little small, and dA and
// ddelta_bias are 1e-6 off instead of 4e-7; rounding the second part too
// changes nothing).  (Integer operations: the conversion instruction runs on
// the slow pipe and bounded the products.)  tf32_up leaves what will be cut.
__device__ __forceinline__ uint32_t tf32_up(float x) { return __float_as_uint(x) + 0x1000u; }
__device__ __forceinline__ uint32_t tf32_round(float x) { return tf32_up(x) & 0xffffe000u; }
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2])
{
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// How an operand enters a product: two tf32 parts, one exact part (its values
// are bf16), or one rounded part.
enum Part { kTwo, kExact, kOne };

template <Part P, int N> __device__ __forceinline__ void parts(const float (&x)[N], uint32_t (&hi)[N], uint32_t (&lo)[N])
{
#pragma unroll
    for (int i = 0; i < N; i++) {
        hi[i] = P == kExact ? __float_as_uint(x[i]) : P == kOne ? tf32_up(x[i]) : tf32_round(x[i]);
        lo[i] = P == kTwo ? __float_as_uint(x[i] - __uint_as_float(hi[i])) : 0u;
    }
}

// A warp's tile: acc += sum over k of a(m0 + .., k) b(n0 + .., k), MT x 16
// rows, NT x 8 columns.  (The tensor core's slots t and t + 4 of k take k
// = 2 t and 2 t + 1 of both operands: the order within a sum is free, and so a
// lane's two values are neighbours.)  Element e of acc[m][n] is row m0 + 16 m + lane / 4 + 8 (e / 2),
// column n0 + 8 n + 2 (lane mod 4) + e mod 2.  The products of one part go
// over the whole tile before those of the next, so that an accumulator is not
// waited for; tiles of few accumulators keep one set for each part.
template <Part PA, Part PB, int MT, int NT, class FA, class FB>
__device__ __forceinline__ void mm(float (&acc)[MT][NT][4], int m0, int n0, int kdim, FA a, FB b)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    constexpr bool kApart = MT * NT <= 4;
    float other[2][kApart ? MT : 1][kApart ? NT : 1][4];
    if (kApart)
#pragma unroll
        for (int s = 0; s < 2; s++)
#pragma unroll
            for (int m = 0; m < MT; m++)
#pragma unroll
                for (int n = 0; n < NT; n++)
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        other[s][m * kApart][n * kApart][e] = 0.f;
#pragma unroll 4
    for (int k = 0; k < kdim; k += 8) {
        uint32_t ah[MT][4], al[MT][4], bh[NT][2], bl[NT][2];
#pragma unroll
        for (int m = 0; m < MT; m++) {
            const int r = m0 + 16 * m + g;
            const float2 u = a(r, k + 2 * t), v = a(r + 8, k + 2 * t);
            const float x[4] = {u.x, v.x, u.y, v.y};
            parts<PA>(x, ah[m], al[m]);
        }
#pragma unroll
        for (int n = 0; n < NT; n++) {
            const float2 u = b(n0 + 8 * n + g, k + 2 * t);
            const float y[2] = {u.x, u.y};
            parts<PB>(y, bh[n], bl[n]);
        }
        if (PB == kTwo)
#pragma unroll
            for (int m = 0; m < MT; m++)
#pragma unroll
                for (int n = 0; n < NT; n++)
                    mma(kApart ? other[0][m * kApart][n * kApart] : acc[m][n], ah[m], bl[n]);
        if (PA == kTwo)
#pragma unroll
            for (int m = 0; m < MT; m++)
#pragma unroll
                for (int n = 0; n < NT; n++)
                    mma(kApart ? other[1][m * kApart][n * kApart] : acc[m][n], al[m], bh[n]);
#pragma unroll
        for (int m = 0; m < MT; m++)
#pragma unroll
            for (int n = 0; n < NT; n++)
                mma(acc[m][n], ah[m], bh[n]);
    }
    if (kApart)
#pragma unroll
        for (int m = 0; m < MT; m++)
#pragma unroll
            for (int n = 0; n < NT; n++)
#pragma unroll
                for (int e = 0; e < 4; e++)
                    acc[m][n][e] += other[0][m * kApart][n * kApart][e] + other[1][m * kApart][n * kApart][e];
}
// The same for bf16 tiles in shared memory (one part each), 16 of k at a time:
// A[m][k] of pitch pa, B[n][k] of pitch pb; NT even.
template <int MT, int NT>
__device__ __forceinline__ void mm16(float (&acc)[MT][NT][4], int m0, int n0, int kdim, const bf16 *A, int pa, const bf16 *B,
                                     int pb)
{
    const int lane = threadIdx.x & 31, r = lane & 7, q = lane >> 3;   // row of the 8 x 8 block q
    const uint32_t a0 = tc::smem_u32(A), b0 = tc::smem_u32(B);
#pragma unroll 2
    for (int k = 0; k < kdim; k += 16) {
        uint32_t a[MT][4];
#pragma unroll
        for (int m = 0; m < MT; m++) {
            // blocks in the order (m, k), (m + 8, k), (m, k + 8), (m + 8, k + 8)
            const int mm_ = m0 + 16 * m + 8 * (q & 1), kk = k + 8 * (q >> 1);
            tc::ldsm(a0 + 2 * ((mm_ + r) * pa + kk), a[m]);
        }
#pragma unroll
        for (int n = 0; n < NT; n += 2) {
            // (n, k), (n, k + 8), (n + 8, k), (n + 8, k + 8)
            const int nn = n0 + 8 * n + 8 * (q >> 1), kk = k + 8 * (q & 1);
            uint32_t b[4];
            tc::ldsm(b0 + 2 * ((nn + r) * pb + kk), b);
#pragma unroll
            for (int m = 0; m < MT; m++) {
                tc::mma16816(acc[m][n], a[m], b[0], b[1]);
                tc::mma16816(acc[m][n + 1], a[m], b[2], b[3]);
            }
        }
    }
}
template <int MT, int NT> __device__ __forceinline__ void zero(float (&acc)[MT][NT][4])
{
#pragma unroll
    for (int m = 0; m < MT; m++)
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
            for (int e = 0; e < 4; e++)
                acc[m][n][e] = 0.f;
}
// f(row, column, element) of every element this thread holds
template <int MT, int NT, class F> __device__ __forceinline__ void each(float (&acc)[MT][NT][4], int m0, int n0, F f)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int m = 0; m < MT; m++)
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
            for (int e = 0; e < 4; e++)
                f(m0 + 16 * m + g + 8 * (e >> 1), n0 + 8 * n + 2 * t + (e & 1), acc[m][n][e]);
}
// the same for pairs of neighbouring columns: f(row, column, first, second)
template <int MT, int NT, class F> __device__ __forceinline__ void pairs(float (&acc)[MT][NT][4], int m0, int n0, F f)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int m = 0; m < MT; m++)
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
            for (int h = 0; h < 2; h++)
                f(m0 + 16 * m + g + 8 * h, n0 + 8 * n + 2 * t, acc[m][n][2 * h], acc[m][n][2 * h + 1]);
}

// Parts of the dot products of a tile's rows with rows of M: v[2 m + h] for row
// m0 + 16 m + lane / 4 + 8 h.
template <int NT, class F> __device__ __forceinline__ void dots(const float (&acc)[2][NT][4], int m0, int n0, F M, float (&v)[4])
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int m = 0; m < 2; m++)
#pragma unroll
        for (int q = 0; q < NT; q++)
#pragma unroll
            for (int e = 0; e < 4; e++)
                v[2 * m + (e >> 1)] =
                    fmaf(acc[m][q][e], M(m0 + 16 * m + g + 8 * (e >> 1), n0 + 8 * q + 2 * t + (e & 1)), v[2 * m + (e >> 1)]);
}

// 64 rows of N bf16 into shared memory, zero from row `valid` on (16 bytes at
// a time; complete after cp_wait and a barrier)
template <int N> __device__ __forceinline__ void load_rows(bf16 *dst, const bf16 *src, size_t stride, int valid)
{
    constexpr int Q = N / 8;
    for (int x = threadIdx.x; x < kC * Q; x += kThreads) {
        const int r = x / Q, c = (x % Q) * 8;
        const uint32_t to = (uint32_t)__cvta_generic_to_shared(dst + r * ph(N) + c);
        const bool in = r < valid;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(in ? src + r * stride + c : src),
                     "r"(in ? 16 : 0)
                     : "memory");
    }
}
// ROWS rows of N floats of a dense array
template <int ROWS, int N> __device__ __forceinline__ void load_f(float *dst, const float *src, int pitch)
{
    constexpr int Q = N / 4;
    for (int x = threadIdx.x; x < ROWS * Q; x += kThreads) {
        const int r = x / Q, c = (x % Q) * 4;
        const uint32_t to = (uint32_t)__cvta_generic_to_shared(dst + r * pitch + c);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(src + (size_t)r * N + c) : "memory");
    }
}
// 64 rows of `kSlice` floats, ld apart, and the scalars of every step
__device__ __forceinline__ void load_slice(float *dst, const float *src, int ld)
{
    for (int x = threadIdx.x; x < kC * kSlice / 4; x += kThreads) {
        const int r = x / (kSlice / 4), c = (x % (kSlice / 4)) * 4;
        const uint32_t to = (uint32_t)__cvta_generic_to_shared(dst + r * kPN + c);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(src + (size_t)r * ld + c) : "memory");
    }
}
__device__ __forceinline__ void load_scalars(float *dst, const float *src)
{
    static_assert(kScalars * kC / 4 <= kThreads, "16 bytes a thread");
    if (threadIdx.x < kScalars * kC / 4) {
        const uint32_t to = (uint32_t)__cvta_generic_to_shared(dst + 4 * threadIdx.x);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(src + 4 * threadIdx.x) : "memory");
    }
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void st2(float *p, float a, float b) { *reinterpret_cast<float2 *>(p) = make_float2(a, b); }

struct Where {
    int64_t b, bh;
    int h, hk, t0, valid;
    size_t tok;
};
__device__ __forceinline__ Where where(const GdrArgs &a, int64_t bh, int n)
{
    Where w;
    w.bh = bh;
    w.b = bh / a.Hv;
    w.h = (int)(bh % a.Hv);
    w.hk = w.h / (a.Hv / a.Hk);
    w.t0 = n * kC;
    w.valid = a.L - w.t0 < kC ? a.L - w.t0 : kC;
    w.tok = (size_t)w.b * a.L + w.t0;
    return w;
}

// ---- 1. per chunk and value head: the scalars, T, W, U = T diag(b) V and P^T dO
template <int K, int V> struct PrepSmem {
    bf16 k[kC * ph(K)], v[kC * ph(V)], o[kC * ph(V)];
    union {   // P takes Q's place: two blocks fit on an SM
        bf16 q[kC * ph(K)];
        float p[kC * kPX];
    };
    float a[kC * kPX], t[kC * kPX];
    float cs[kC], cl[kC], b[kC], rk[kC], rq[kC], wf[kC];   // wf: b c / |k|
};
template <int K, int V>
__global__ void __launch_bounds__(kThreads, 2) prep_kernel(const GdrBwdArgs g, const Layout lay)
{
    extern __shared__ __align__(16) uint8_t raw[];
    PrepSmem<K, V> &s = *reinterpret_cast<PrepSmem<K, V> *>(raw);
    const GdrArgs &a = g.f;
    const int n = blockIdx.x % lay.NC;
    const Where w = where(a, blockIdx.x / lay.NC, n);
    float *ws = static_cast<float *>(a.workspace) + lay.base(w.bh, n);
    load_rows<K>(s.k, static_cast<const bf16 *>(a.k) + (w.tok * a.Hk + w.hk) * K, (size_t)a.Hk * K, w.valid);
    load_rows<K>(s.q, static_cast<const bf16 *>(a.q) + (w.tok * a.Hk + w.hk) * K, (size_t)a.Hk * K, w.valid);
    load_rows<V>(s.v, static_cast<const bf16 *>(a.v) + (w.tok * a.Hv + w.h) * V, (size_t)a.Hv * V, w.valid);
    load_rows<V>(s.o, static_cast<const bf16 *>(g.dout) + (w.tok * a.Hv + w.h) * V, (size_t)a.Hv * V, w.valid);
    cp_commit();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == 0) {
        const float bias = a.bias ? a.bias[w.h] : 0.f, Ah = a.A[w.h] * kLog2e;
        float gl[2];
        for (int i = 0; i < 2; i++) {
            const int r = 2 * lane + i;
            gl[i] = 0.f;
            s.b[r] = 0.f;
            if (r < w.valid) {
                const float de = gdr_ld(static_cast<const bf16 *>(a.delta), (w.tok + r) * a.Hv + w.h);
                gl[i] = gdr_log_decay(gdr_dt(de, bias, a.softplus), Ah);
                const float be = gdr_ld(static_cast<const bf16 *>(a.beta), (w.tok + r) * a.Hv + w.h);
                s.b[r] = a.sigmoid ? sigmoid_mufu(be) : be;
            }
        }
        float2 sum[2];
        gdr_log_sums(gl, sum);
        for (int i = 0; i < 2; i++) {
            s.cs[2 * lane + i] = sum[i].x;
            s.cl[2 * lane + i] = sum[i].y;
        }
    }
    cp_wait<0>();
    __syncthreads();
    for (int r = warp; r < kC; r += kThreads / 32) {
        float kk = 0.f, qq = 0.f;
        for (int c = lane; c < K; c += 32) {
            const float x = bf(&s.k[r * ph(K) + c]), y = bf(&s.q[r * ph(K) + c]);
            kk = fmaf(x, x, kk);
            qq = fmaf(y, y, qq);
        }
        kk = warp_sum(kk);
        qq = warp_sum(qq);
        if (lane == 0) {
            s.rk[r] = a.l2norm ? rsqrtf(kk + kL2Eps) : 1.f;
            s.wf[r] = s.b[r] * ex2_mufu(s.cs[r]) * s.rk[r];
            s.rq[r] = a.scale * (a.l2norm ? rsqrtf(qq + kL2Eps) : 1.f);
        }
    }
    __syncthreads();
    const int m0 = 32 * (warp >> 2), wn = warp & 3;
    {
        float kk[2][2][4], qk[2][2][4];
        zero(kk);
        zero(qk);
        mm16(kk, m0, 16 * wn, K, s.k, ph(K), s.k, ph(K));
        mm16(qk, m0, 16 * wn, K, s.q, ph(K), s.k, ph(K));
        __syncthreads();   // Q is done with
        each(kk, m0, 16 * wn, [&](int i, int j, float v) {
            s.a[i * kPX + j] = j < i ? s.b[i] * gdr_between(s.cs[i], s.cl[i], s.cs[j], s.cl[j]) * s.rk[i] * s.rk[j] * v : 0.f;
            s.t[i * kPX + j] = 0.f;
        });
        each(qk, m0, 16 * wn, [&](int i, int j, float v) {
            s.p[i * kPX + j] = j <= i ? gdr_between(s.cs[i], s.cl[i], s.cs[j], s.cl[j]) * s.rq[i] * s.rk[j] * v : 0.f;
        });
    }
    __syncthreads();
    // T = (I + A)^-1: the 16 x 16 diagonal blocks by substitution from the
    // right (thread = row, the block's other rows by shuffles), then the
    // 16 x 16 blocks beside them and the 32 x 32 block below: T21 = -T22 A21 T11
    if (warp < 2) {
        const int i = 32 * warp + lane, il = lane & 15, c0 = i - il;
        float d[16], x[16];
#pragma unroll
        for (int j = 0; j < 16; j++) {
            d[j] = s.a[i * kPX + c0 + j];
            x[j] = 0.f;
        }
#pragma unroll
        for (int k = 15; k >= 0; k--) {
            x[k] = k == il ? 1.f : x[k];
#pragma unroll
            for (int j = 0; j < k; j++)
                x[j] = fmaf(-x[k], __shfl_sync(0xffffffffu, d[j], (lane & 16) | k), x[j]);
        }
#pragma unroll
        for (int j = 0; j < 16; j++)
            s.t[i * kPX + c0 + j] = x[j];
    }
    __syncthreads();
    // blocks as left operands (k along the row) and right ones (k down the column)
    auto Tl = [&](int r0, int c0) { return RowF{s.t + r0 * kPX + c0, kPX}; };
    auto Al = [&](int r0, int c0) { return RowF{s.a + r0 * kPX + c0, kPX}; };
    auto Tr = [&](int r0, int c0) { return ColF{s.t + r0 * kPX + c0, kPX}; };
    auto Ar = [&](int r0, int c0) { return ColF{s.a + r0 * kPX + c0, kPX}; };
    if (warp < 4) {   // A21 T11 of both pairs of 16 blocks, in the place of A21
        const int r0 = 32 * (warp >> 1) + 16, c0 = r0 - 16, n0 = 8 * (warp & 1);
        float x[1][1][4];
        zero(x);
        mm<kTwo, kTwo>(x, 0, n0, 16, Al(r0, c0), Tr(c0, c0));
        __syncwarp();
        asm volatile("bar.sync %0, 64;" ::"r"(1 + (warp >> 1)) : "memory");   // both warps have read A21
        each(x, 0, n0, [&](int i, int j, float v) { s.a[(r0 + i) * kPX + c0 + j] = v; });
    }
    __syncthreads();
    if (warp < 4) {
        const int r0 = 32 * (warp >> 1) + 16, c0 = r0 - 16, n0 = 8 * (warp & 1);
        float x[1][1][4];
        zero(x);
        mm<kTwo, kTwo>(x, 0, n0, 16, Tl(r0, r0), Ar(r0, c0));
        each(x, 0, n0, [&](int i, int j, float v) { s.t[(r0 + i) * kPX + c0 + j] = -v; });
    }
    __syncthreads();
    {   // 32 x 32: warps 2 (rows) x 4 (columns of 8)
        float x[1][1][4];
        zero(x);
        mm<kTwo, kTwo>(x, m0 / 2, 8 * wn, 32, Al(32, 0), Tr(0, 0));
        __syncthreads();
        each(x, m0 / 2, 8 * wn, [&](int i, int j, float v) { s.a[(32 + i) * kPX + j] = v; });
        __syncthreads();
        zero(x);
        mm<kTwo, kTwo>(x, m0 / 2, 8 * wn, 32, Tl(32, 32), Ar(32, 0));
        each(x, m0 / 2, 8 * wn, [&](int i, int j, float v) { s.t[(32 + i) * kPX + j] = -v; });
    }
    __syncthreads();
    for (int x = threadIdx.x; x < kC * kC; x += kThreads)
        ws[lay.T() + x] = s.t[(x >> 6) * kPX + (x & 63)];
    if (threadIdx.x < kC) {
        const int i = threadIdx.x;
        ws[lay.cs() + i] = s.cs[i];
        ws[lay.cs() + kC + i] = s.b[i];
        ws[lay.cl() + i] = s.cl[i];
        ws[lay.rk() + i] = s.rk[i];
        ws[lay.rq() + i] = s.rq[i];
    }
    {
        float acc[2][K / 32][4];
        zero(acc);
        mm<kTwo, kExact>(acc, m0, K / 4 * wn, kC, scaled(RowF{s.t, kPX}, s.wf), ColH{s.k, ph(K)});
        pairs(acc, m0, K / 4 * wn, [&](int i, int j, float x, float y) { st2(ws + lay.W() + i * K + j, x, y); });
    }
    float acc[2][V / 32][4];
    zero(acc);
    mm<kTwo, kExact>(acc, m0, V / 4 * wn, kC, scaled(RowF{s.t, kPX}, s.b), ColH{s.v, ph(V)});
    pairs(acc, m0, V / 4 * wn, [&](int i, int j, float x, float y) { st2(ws + lay.U() + i * V + j, x, y); });
    zero(acc);
    mm<kTwo, kExact>(acc, m0, V / 4 * wn, kC, ColF{s.p, kPX}, ColH{s.o, ph(V)});
    pairs(acc, m0, V / 4 * wn, [&](int i, int j, float x, float y) { st2(ws + lay.dN() + i * V + j, x, y); });
}

// ---- 2. forward over the chunks (S0, and N in U's place) and 3. in reverse (dS1,
// and dN in the place of P^T dO): neither needs the other, so one launch takes
// both, 32 state rows per block, one block of each kind to an SM.  Tiles have
// one buffer each; a phase's next tiles are fetched while the other phase runs.
template <int K> struct ChainSmem {
    float w[kC * pr(K)];
    bf16 k[kC * ph(K)];
    float u[kC * kPN], v[kScalars * kC];   // U; cs, b, 1 / |k|, scale / |q|, cs's lo
    float s[kSlice * pr(K)], n[kC * kPN];
};
template <int K> __device__ __forceinline__ void forward_chain(const GdrArgs &a, const Layout &lay, ChainSmem<K> &s, int64_t bh, int v0)
{
    const int warp = threadIdx.x >> 5;
    float *base = static_cast<float *>(a.workspace);
    auto fetch1 = [&](int n) {   // for S W^T
        if (n < lay.NC) {
            const float *ws = base + lay.base(bh, n);
            load_f<kC, K>(s.w, ws + lay.W(), pr(K));
            load_slice(s.u, ws + lay.U() + v0, a.V);
            load_scalars(s.v, ws);
        }
        cp_commit();
    };
    auto fetch2 = [&](int n) {   // for N^T K
        if (n < lay.NC) {
            const Where w = where(a, bh, n);
            load_rows<K>(s.k, static_cast<const bf16 *>(a.k) + (w.tok * a.Hk + w.hk) * K, (size_t)a.Hk * K, w.valid);
        }
        cp_commit();
    };
    fetch1(0);
    fetch2(0);
    for (int x = threadIdx.x; x < kSlice * K; x += kThreads)
        s.s[(x / K) * pr(K) + x % K] = a.init ? a.init[((size_t)bh * a.V + v0) * K + x] : 0.f;
    const int mN = 16 * (warp >> 1), nN = 16 * (warp & 1);   // N: 64 x 32 as 4 x 2 warps
    constexpr int NT = K / 64;                               // the state: 32 x K as 1 x 8
    for (int n = 0; n < lay.NC; n++) {
        float *ws = base + lay.base(bh, n);
        cp_wait<1>();
        __syncthreads();
        for (int x = threadIdx.x * 4; x < kSlice * K; x += kThreads * 4)
            *reinterpret_cast<float4 *>(ws + lay.S0() + (size_t)v0 * K + x) =
                *reinterpret_cast<const float4 *>(&s.s[(x / K) * pr(K) + x % K]);
        const float *cs = s.v, *rk = s.v + 2 * kC, *cl = s.v + 4 * kC;
        const float end = cs[kC - 1], endl = cl[kC - 1], dec = ex2_mufu(end);
        float acc[1][2][4];
        zero(acc);
        mm<kTwo, kTwo>(acc, mN, nN, K, RowF{s.w, pr(K)}, RowF{s.s, pr(K)});
        {
            const int i0 = mN + ((threadIdx.x & 31) >> 2);
            const float e[2] = {rk[i0] * gdr_between(end, endl, cs[i0], cl[i0]),
                                rk[i0 + 8] * gdr_between(end, endl, cs[i0 + 8], cl[i0 + 8])};
            pairs(acc, mN, nN, [&](int i, int j, float x, float y) {
                const float2 u = *reinterpret_cast<const float2 *>(&s.u[i * kPN + j]);
                x = u.x - x, y = u.y - y;
                st2(ws + lay.U() + i * a.V + v0 + j, x, y);
                const float f = e[(i - i0) >> 3];
                st2(&s.n[i * kPN + j], x * f, y * f);
            });
        }
        __syncthreads();
        fetch1(n + 1);
        cp_wait<1>();
        __syncthreads();
        float up[2][NT][4];
        zero(up);
        mm<kTwo, kExact>(up, 0, 8 * NT * warp, kC, ColF{s.n, kPN}, ColH{s.k, ph(K)});
        each(up, 0, 8 * NT * warp, [&](int i, int j, float v) {
            float *p = &s.s[i * pr(K) + j];
            *p = fmaf(dec, *p, v);
        });
        __syncthreads();
        fetch2(n + 1);
    }
}

template <int K> struct ReverseSmem {
    float w[kC * pc(K)];
    bf16 k[kC * ph(K)], q[kC * ph(K)], o[kC * ph(kSlice)];
    float u[kC * kPN], v[kScalars * kC];   // P^T dO; scalars
    float g[kSlice * pr(K)], n[kC * kPN];
    float f[kC];
};
template <int K> __device__ __forceinline__ void reverse_chain(const GdrBwdArgs &ga, const Layout &lay, ReverseSmem<K> &s, int64_t bh, int v0)
{
    const GdrArgs &a = ga.f;
    const int warp = threadIdx.x >> 5;
    float *base = static_cast<float *>(a.workspace);
    auto fetch1 = [&](int n) {   // for K dS^T
        if (n >= 0) {
            const Where w = where(a, bh, n);
            const float *ws = base + lay.base(bh, n);
            load_rows<K>(s.k, static_cast<const bf16 *>(a.k) + (w.tok * a.Hk + w.hk) * K, (size_t)a.Hk * K, w.valid);
            load_slice(s.u, ws + lay.dN() + v0, a.V);
            load_scalars(s.v, ws);
        }
        cp_commit();
    };
    auto fetch2 = [&](int n) {   // for dN^T W and dO^T Q
        if (n >= 0) {
            const Where w = where(a, bh, n);
            load_f<kC, K>(s.w, base + lay.base(bh, n) + lay.W(), pc(K));
            load_rows<K>(s.q, static_cast<const bf16 *>(a.q) + (w.tok * a.Hk + w.hk) * K, (size_t)a.Hk * K, w.valid);
            load_rows<kSlice>(s.o, static_cast<const bf16 *>(ga.dout) + (w.tok * a.Hv + w.h) * a.V + v0, (size_t)a.Hv * a.V,
                              w.valid);
        }
        cp_commit();
    };
    fetch1(lay.NC - 1);
    fetch2(lay.NC - 1);
    for (int x = threadIdx.x; x < kSlice * K; x += kThreads)
        s.g[(x / K) * pr(K) + x % K] = ga.dlast ? ga.dlast[((size_t)bh * a.V + v0) * K + x] : 0.f;
    const int mN = 16 * (warp >> 1), nN = 16 * (warp & 1);
    constexpr int NT = K / 64;
    for (int n = lay.NC - 1; n >= 0; n--) {
        float *ws = base + lay.base(bh, n);
        cp_wait<1>();
        __syncthreads();
        const float *cs = s.v, *rk = s.v + 2 * kC, *rq = s.v + 3 * kC, *cl = s.v + 4 * kC;
        const float end = cs[kC - 1], endl = cl[kC - 1], dec = ex2_mufu(end);
        if (threadIdx.x < kC)
            s.f[threadIdx.x] = rq[threadIdx.x] * ex2_mufu(cs[threadIdx.x]);
        for (int x = threadIdx.x * 4; x < kSlice * K; x += kThreads * 4)
            *reinterpret_cast<float4 *>(ws + lay.dS() + (size_t)v0 * K + x) =
                *reinterpret_cast<const float4 *>(&s.g[(x / K) * pr(K) + x % K]);
        float acc[1][2][4];
        zero(acc);
        mm<kExact, kTwo>(acc, mN, nN, K, RowH{s.k, ph(K)}, RowF{s.g, pr(K)});
        {
            const int i0 = mN + ((threadIdx.x & 31) >> 2);
            const float e[2] = {rk[i0] * gdr_between(end, endl, cs[i0], cl[i0]),
                                rk[i0 + 8] * gdr_between(end, endl, cs[i0 + 8], cl[i0 + 8])};
            pairs(acc, mN, nN, [&](int i, int j, float x, float y) {
                const float2 u = *reinterpret_cast<const float2 *>(&s.u[i * kPN + j]);
                const float f = e[(i - i0) >> 3];
                x = fmaf(f, x, u.x), y = fmaf(f, y, u.y);
                st2(ws + lay.dN() + i * a.V + v0 + j, x, y);
                st2(&s.n[i * kPN + j], -x, -y);
            });
        }
        __syncthreads();
        fetch1(n - 1);
        cp_wait<1>();
        __syncthreads();
        float up[2][NT][4];
        zero(up);
        mm<kTwo, kTwo>(up, 0, 8 * NT * warp, kC, ColF{s.n, kPN}, ColF{s.w, pc(K)});
        mm<kTwo, kExact>(up, 0, 8 * NT * warp, kC, scaled(ColH{s.o, ph(kSlice)}, s.f), ColH{s.q, ph(K)});
        each(up, 0, 8 * NT * warp, [&](int i, int j, float v) {
            float *p = &s.g[i * pr(K) + j];
            *p = fmaf(dec, *p, v);
        });
        __syncthreads();
        fetch2(n - 1);
    }
    if (ga.dinit)
        for (int x = threadIdx.x; x < kSlice * K; x += kThreads)
            ga.dinit[((size_t)bh * a.V + v0) * K + x] = s.g[(x / K) * pr(K) + x % K];
}

template <int K> constexpr size_t chains_smem()
{
    return sizeof(ReverseSmem<K>) > sizeof(ChainSmem<K>) ? sizeof(ReverseSmem<K>) : sizeof(ChainSmem<K>);
}
template <int K> __global__ void __launch_bounds__(kThreads, 2) chains_kernel(const GdrBwdArgs g, const Layout lay, int chains)
{
    extern __shared__ __align__(16) uint8_t raw[];
    const int slices = g.f.V / kSlice;
    // blocks 0 .. chains - 1 run forward, the others in reverse: dealt out to
    // the SMs in turn, both kinds are spread evenly
    const bool reverse = (int)blockIdx.x >= chains;
    const int at = reverse ? blockIdx.x - chains : blockIdx.x;
    const int64_t bh = at / slices;
    const int v0 = (at % slices) * kSlice;
    if (reverse)
        reverse_chain<K>(g, lay, *reinterpret_cast<ReverseSmem<K> *>(raw), bh, v0);
    else
        forward_chain<K>(g.f, lay, *reinterpret_cast<ChainSmem<K> *>(raw), bh, v0);
}

// ---- 4. per chunk and key head: every gradient
template <int K, int V> struct GradSmem {
    bf16 k[kC * ph(K)], q[kC * ph(K)], o[kC * ph(V)], v[kC * ph(V)];
    float n[kC * pr(V)], r[kC * pr(V)], x[kC * kPX];
    float t[kC * kPX], m[2][kSlice * pc(K)];   // T; 32 rows of a state, the next 32
    float cs[kScalars * kC], brk[kC];   // cs, b, rk, rq, cs's lo as in the workspace; b rk
    float delta[kC], dcs[kC], sum[6][4][kC], red[8];   // sum: row sums of each column of warps
};
template <int K, int V>
__global__ void __launch_bounds__(kThreads, 1) grad_kernel(const GdrBwdArgs ga, const Layout lay, float *partial)
{
    extern __shared__ __align__(16) uint8_t raw[];
    GradSmem<K, V> &s = *reinterpret_cast<GradSmem<K, V> *>(raw);
    const GdrArgs &a = ga.f;
    constexpr int NK = K / 32, NV = V / 32;
    const int per_k = a.Hv / a.Hk, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t bhk = blockIdx.x / lay.NC;
    const int n = blockIdx.x % lay.NC;
    const int64_t b = bhk / a.Hk;
    const int hk = (int)(bhk % a.Hk);
    const float *cs = s.cs, *bb = s.cs + kC, *rk = s.cs + 2 * kC, *rq = s.cs + 3 * kC, *cl = s.cs + 4 * kC;
    const int t0 = n * kC, valid = a.L - t0 < kC ? a.L - t0 : kC;
    const size_t tok = (size_t)b * a.L + t0;
    const int m0 = 32 * (warp >> 2), wn = warp & 3, gq = lane >> 2, tq = lane & 3;
    const int nK = K / 4 * wn, nV = V / 4 * wn, nC = 16 * wn;   // this warp's columns
    load_rows<K>(s.k, static_cast<const bf16 *>(a.k) + (tok * a.Hk + hk) * K, (size_t)a.Hk * K, valid);
    load_rows<K>(s.q, static_cast<const bf16 *>(a.q) + (tok * a.Hk + hk) * K, (size_t)a.Hk * K, valid);
    auto Kt = [&](int i, int k) { return bf(&s.k[i * ph(K) + k]); };
    auto Qt = [&](int i, int k) { return bf(&s.q[i * ph(K) + k]); };
    float dK[2][NK][4], dQ[2][NK][4];   // of the unit rows (scale q^ for q), all value heads
    zero(dK);
    zero(dQ);
    // this thread's rows: m0 + 16 m + gq + 8 h
    auto row_of = [&](int x) { return m0 + 16 * (x >> 1) + gq + 8 * (x & 1); };
    // rows' sums over the warp's columns, from each thread's part, to sum[which]
    auto put_rows = [&](int which, const float (&v)[4]) {
#pragma unroll
        for (int x = 0; x < 4; x++) {
            float r = v[x];
            r += __shfl_xor_sync(0xffffffffu, r, 1);
            r += __shfl_xor_sync(0xffffffffu, r, 2);
            if (tq == 0)
                s.sum[which][wn][row_of(x)] = r;
        }
    };
    auto all = [&](int which, int row) {
        return (s.sum[which][0][row] + s.sum[which][1][row]) + (s.sum[which][2][row] + s.sum[which][3][row]);
    };
    for (int hh = 0; hh < per_k; hh++) {
        const int h = hk * per_k + hh;
        const int64_t bh = b * a.Hv + h;
        const float *ws = static_cast<const float *>(a.workspace) + lay.base(bh, n);
        const float *S0 = ws + lay.S0(), *dS = ws + lay.dS();
        __syncthreads();
        for (int x = threadIdx.x; x < kScalars * kC; x += kThreads)
            s.cs[x] = ws[x];
        if (threadIdx.x < valid)
            s.delta[threadIdx.x] = gdr_ld(static_cast<const bf16 *>(a.delta), (tok + threadIdx.x) * a.Hv + h);
        load_rows<V>(s.o, static_cast<const bf16 *>(ga.dout) + (tok * a.Hv + h) * V, (size_t)a.Hv * V, valid);
        load_rows<V>(s.v, static_cast<const bf16 *>(a.v) + (tok * a.Hv + h) * V, (size_t)a.Hv * V, valid);
        load_f<kC, V>(s.n, ws + lay.U(), pr(V));
        load_f<kC, V>(s.r, ws + lay.dN(), pr(V));
        load_f<kC, kC>(s.t, ws + lay.T(), kPX);
        cp_commit();
        // S0 and then dS1, 32 rows at a time, two pieces on their way; beside
        // dS1's those of S0 again, in the places of T and R', done with by then
        constexpr int kPieces = V / kSlice;
        static_assert(kPieces % 2 == 0 && sizeof(s.t) >= sizeof(s.m[0]) && sizeof(s.r) >= sizeof(s.m[0]), "room for a piece");
        auto beside = [&](int i) { return i & 1 ? s.r : s.t; };
        auto fetch = [&](int i) {
            if (i < 2 * kPieces)
                load_f<kSlice, K>(s.m[i & 1], (i < kPieces ? S0 : dS - (size_t)V * K) + (size_t)i * kSlice * K, pc(K));
            if (i >= kPieces && i < 2 * kPieces)
                load_f<kSlice, K>(beside(i), S0 + (size_t)(i - kPieces) * kSlice * K, pc(K));
            cp_commit();
        };
        fetch(0);
        fetch(1);
        cp_wait<2>();
        __syncthreads();
        if (threadIdx.x < kC)   // read much later
            s.brk[threadIdx.x] = bb[threadIdx.x] * rk[threadIdx.x];
        const float end = cs[kC - 1], endl = cl[kC - 1];
        // R' = T^T dN
        {
            float r[2][NV][4];
            zero(r);
            mm<kTwo, kTwo>(r, m0, nV, kC, ColF{s.t, kPX}, ColF{s.r, pr(V)});
            __syncthreads();
            float dbr[4] = {};
#pragma unroll
            for (int m = 0; m < 2; m++)
#pragma unroll
                for (int q = 0; q < NV; q++)
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        const int i = m0 + 16 * m + gq + 8 * e, j = nV + 8 * q + 2 * tq;
                        const float x = r[m][q][2 * e], y = r[m][q][2 * e + 1];
                        st2(&s.r[i * pr(V) + j], x, y);
                        if (i < valid) {
                            const __nv_bfloat162 vv = *reinterpret_cast<const __nv_bfloat162 *>(&s.v[i * ph(V) + j]);
                            dbr[2 * m + e] = fmaf(x, __low2float(vv), fmaf(y, __high2float(vv), dbr[2 * m + e]));
                            *reinterpret_cast<__nv_bfloat162 *>(static_cast<bf16 *>(ga.dv) + ((tok + i) * a.Hv + h) * V + j) =
                                __floats2bfloat162_rn(bb[i] * x, bb[i] * y);
                        }
                    }
            put_rows(0, dbr);
        }
        __syncthreads();
        // dA o G and dP o G, and with them E
        float xp[2][2][4], xa[2][2][4];
        {
            zero(xa);
            zero(xp);
            mm<kTwo, kTwo>(xa, m0, nC, V, RowF{s.r, pr(V)}, RowF{s.n, pr(V)});
            mm<kExact, kTwo>(xp, m0, nC, V, RowH{s.o, ph(V)}, RowF{s.n, pr(V)});
#pragma unroll
            for (int m = 0; m < 2; m++)
#pragma unroll
                for (int q = 0; q < 2; q++)
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const int i = m0 + 16 * m + gq + 8 * (e >> 1), j = nC + 8 * q + 2 * tq + (e & 1);
                        const float G = gdr_between(cs[i], cl[i], cs[j], cl[j]);
                        xa[m][q][e] = j < i ? -xa[m][q][e] * G : 0.f;
                        xp[m][q][e] = j <= i ? xp[m][q][e] * G : 0.f;
                    }
            float kk[2][2][4], qk[2][2][4];
            zero(kk);
            zero(qk);
            mm16(kk, m0, nC, K, s.k, ph(K), s.k, ph(K));
            mm16(qk, m0, nC, K, s.q, ph(K), s.k, ph(K));
#pragma unroll
            for (int m = 0; m < 2; m++)
#pragma unroll
                for (int q = 0; q < 2; q++)
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const int i = m0 + 16 * m + gq + 8 * (e >> 1), j = nC + 8 * q + 2 * tq + (e & 1);
                        const float pa = bb[i] * rk[i] * xa[m][q][e] * kk[m][q][e];
                        s.x[i * kPX + j] = j < i ? rk[j] * fmaf(rq[i] * xp[m][q][e], qk[m][q][e], pa) : 0.f;
                    }
        }
        __syncthreads();
        // sums of E over i >= t > j: along each row first (four threads a row), then down
        {
            const int i = threadIdx.x >> 2, part = threadIdx.x & 3;
            float v[16], run = 0.f;
#pragma unroll
            for (int j = 0; j < 16; j++) {
                v[j] = run;   // the sum of this part's columns before j
                run += s.x[i * kPX + 16 * part + j];
            }
            float before = run;   // of the parts to the left
            const float u1 = __shfl_up_sync(0xffffffffu, run, 1), u2 = __shfl_up_sync(0xffffffffu, run, 2),
                        u3 = __shfl_up_sync(0xffffffffu, run, 3);
            before = (part > 2 ? u3 : 0.f) + (part > 1 ? u2 : 0.f) + (part > 0 ? u1 : 0.f);
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 16; j++)
                s.x[i * kPX + 16 * part + j] = before + v[j];
        }
        __syncthreads();
        {
            const int t = threadIdx.x >> 2, part = threadIdx.x & 3;
            float d = 0.f;
            for (int i = t + part; i < kC; i += 4)
                d += s.x[i * kPX + t];
            d += __shfl_xor_sync(0xffffffffu, d, 1);
            d += __shfl_xor_sync(0xffffffffu, d, 2);
            if (part == 0)
                s.dcs[t] = d;
        }
        __syncthreads();
        each(xa, m0, nC, [&](int i, int j, float v) { s.x[i * kPX + j] = v; });
        // Y = -c R' S0 and q = c dO S0, 32 rows of S0 at a time
        float Y[2][NK][4], q[2][NK][4];
        zero(Y);
        zero(q);
        for (int i = 0; i < kPieces; i++) {
            const int v0 = i * kSlice;
            const float *St = s.m[i & 1];
            cp_wait<1>();
            __syncthreads();
            mm<kTwo, kTwo>(Y, m0, nK, kSlice, RowF{s.r + v0, pr(V)}, ColF{St, pc(K)});
            mm<kExact, kTwo>(q, m0, nK, kSlice, RowH{s.o + v0, ph(V)}, ColF{St, pc(K)});
            __syncthreads();
            fetch(i + 2);
        }
        {
            each(Y, m0, nK, [&](int i, int, float &v) { v *= -ex2_mufu(cs[i]); });
            each(q, m0, nK, [&](int i, int, float &v) { v *= ex2_mufu(cs[i]); });
            float ky[4] = {}, qq[4] = {};
            dots(Y, m0, nK, Kt, ky);
            dots(q, m0, nK, Qt, qq);
#pragma unroll
            for (int x = 0; x < 4; x++) {
                const int i = row_of(x);
                qq[x] = fmaf(rq[i], qq[x], bb[i] * rk[i] * ky[x]);
            }
            put_rows(1, qq);   // s
        }
        // the rest of Y, and of q: one part is enough for their bf16 results
        mm<kOne, kExact>(Y, m0, nK, kC, scaled(RowF{s.x, kPX}, rk), ColH{s.k, ph(K)});
        {
            float ky[4] = {};
            dots(Y, m0, nK, Kt, ky);
#pragma unroll
            for (int x = 0; x < 4; x++)
                ky[x] *= rk[row_of(x)];
            put_rows(2, ky);
            each(Y, m0, nK, [&](int i, int, float &v) { v *= bb[i]; });
#pragma unroll
            for (int m = 0; m < 2; m++)
#pragma unroll
                for (int p = 0; p < NK; p++)
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        dK[m][p][e] += Y[m][p][e];
        }
        // Z = e N dS1 + ..., in Y's registers
        zero(Y);
        float through = 0.f;
        const float dec = ex2_mufu(end);
        for (int i = kPieces; i < 2 * kPieces; i++) {
            const int v0 = (i - kPieces) * kSlice;
            const float *St = s.m[i & 1];
            cp_wait<1>();
            __syncthreads();
            mm<kTwo, kTwo>(Y, m0, nK, kSlice, RowF{s.n + v0, pr(V)}, ColF{St, pc(K)});
            for (int x = threadIdx.x * 4; x < kSlice * K; x += kThreads * 4) {   // c_end <dS1, S0>
                const int at = (x / K) * pc(K) + x % K;
                const float4 f = *reinterpret_cast<const float4 *>(&beside(i)[at]);
                const float4 d = *reinterpret_cast<const float4 *>(&St[at]);
                through = fmaf(dec * d.x, f.x, fmaf(dec * d.y, f.y, fmaf(dec * d.z, f.z, fmaf(dec * d.w, f.w, through))));
            }
            __syncthreads();
            fetch(i + 2);
        }
        each(Y, m0, nK, [&](int i, int, float &v) { v *= gdr_between(end, endl, cs[i], cl[i]); });
        {
            float kz[4] = {};
            dots(Y, m0, nK, Kt, kz);
#pragma unroll
            for (int x = 0; x < 4; x++)
                kz[x] *= rk[row_of(x)];
            put_rows(3, kz);   // z
        }
        mm<kOne, kExact>(Y, m0, nK, kC, scaled(ColF{s.x, kPX}, s.brk), ColH{s.k, ph(K)});
        __syncthreads();
        each(xp, m0, nC, [&](int i, int j, float v) { s.x[i * kPX + j] = v; });
        through = warp_sum(through);
        if (lane == 0)
            s.red[warp] = through;
        __syncthreads();
        mm<kOne, kExact>(Y, m0, nK, kC, scaled(ColF{s.x, kPX}, rq), ColH{s.q, ph(K)});
        mm<kOne, kExact>(q, m0, nK, kC, scaled(RowF{s.x, kPX}, rk), ColH{s.k, ph(K)});
#pragma unroll
        for (int m = 0; m < 2; m++)
#pragma unroll
            for (int p = 0; p < NK; p++)
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    dK[m][p][e] += Y[m][p][e];
                    dQ[m][p][e] += q[m][p][e];
                }
        if (warp == 0) {
            float thr = 0.f;
            for (int k = 0; k < 8; k++)
                thr += s.red[k];
            // sums of s from each step on, of z before each step
            const float s0 = all(1, 2 * lane), s1 = all(1, 2 * lane + 1), z0 = all(3, 2 * lane), z1 = all(3, 2 * lane + 1);
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
            const float dg[2] = {s.dcs[2 * lane] + down + before + thr, s.dcs[2 * lane + 1] + s1 + after + before + z0 + thr};
            const float bias = a.bias ? a.bias[h] : 0.f, Ah = a.A[h];
            float sA = 0.f, sb = 0.f;
            for (int i = 0; i < 2; i++) {
                const int row = 2 * lane + i;
                if (row < valid) {
                    const size_t at = (tok + row) * a.Hv + h;
                    const float pre = s.delta[row];
                    // a step that leaves nothing has no gradient, not 0 times an infinite dt either
                    sA = dg[i] != 0.f ? fmaf(dg[i], gdr_dt(pre, bias, a.softplus), sA) : sA;
                    const float dd = dg[i] * Ah * (a.softplus ? sigmoid_mufu(pre + bias) : 1.f);
                    sb += dd;
                    gdr_st(static_cast<bf16 *>(ga.ddelta), at, dd);
                    const float db = all(0, row) + all(2, row);
                    gdr_st(static_cast<bf16 *>(ga.dbeta), at, db * (a.sigmoid ? bb[row] * (1.f - bb[row]) : 1.f));
                }
            }
            sA = warp_sum(sA);
            sb = warp_sum(sb);
            if (lane == 0) {   // (2, B NC, Hv)
                const size_t at = ((size_t)b * lay.NC + n) * a.Hv + h;
                partial[at] = sA;
                partial[(size_t)a.Bsz * lay.NC * a.Hv + at] = sb;
            }
        }
    }
    // through the norms: d k = rk (dk^ - k^ (k^ . dk^))
    float kd[4] = {}, qd[4] = {};
    dots(dK, m0, nK, Kt, kd);
    dots(dQ, m0, nK, Qt, qd);
    put_rows(4, kd);
    put_rows(5, qd);
    __syncthreads();
#pragma unroll
    for (int m = 0; m < 2; m++)
#pragma unroll
        for (int e = 0; e < 2; e++) {
            const int row = m0 + 16 * m + gq + 8 * e;
            if (row >= valid)
                continue;
            const float r = rk[row], f = rq[row], inv = a.scale != 0.f ? f / a.scale : 0.f;   // 1 / |k|, scale / |q|, 1 / |q|
            const float ck = a.l2norm ? r * r * all(4, row) : 0.f, cq = a.l2norm ? inv * inv * all(5, row) : 0.f;
#pragma unroll
            for (int p = 0; p < NK; p++) {
                const int j = nK + 8 * p + 2 * tq;
                const size_t at = ((tok + row) * a.Hk + hk) * K + j;
                *reinterpret_cast<__nv_bfloat162 *>(static_cast<bf16 *>(ga.dk) + at) = __floats2bfloat162_rn(
                    r * fmaf(-Kt(row, j), ck, dK[m][p][2 * e]), r * fmaf(-Kt(row, j + 1), ck, dK[m][p][2 * e + 1]));
                *reinterpret_cast<__nv_bfloat162 *>(static_cast<bf16 *>(ga.dq) + at) = __floats2bfloat162_rn(
                    f * fmaf(-Qt(row, j), cq, dQ[m][p][2 * e]), f * fmaf(-Qt(row, j + 1), cq, dQ[m][p][2 * e + 1]));
            }
        }
}

// ---- 5. dA and ddelta_bias: sums over batch and chunks, a warp per head
__global__ void __launch_bounds__(32) head_sum_kernel(const float *partial, int64_t n, int Hv, float *dA, float *dbias)
{
    const int h = blockIdx.x;
    float s[2] = {0.f, 0.f};
    for (int64_t k = threadIdx.x; k < n; k += 32)
        for (int i = 0; i < 2; i++)
            s[i] += partial[((size_t)i * n + k) * Hv + h];
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
cudaError_t go(Kern kernel, int64_t blocks, size_t bytes, cudaStream_t st, Args... args)
{
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess)
        return e;
    kernel<<<(unsigned)blocks, kThreads, bytes, st>>>(args...);
    return cudaGetLastError();
}

template <int K, int V> cudaError_t launch(const GdrBwdArgs &g, cudaStream_t st)
{
    static_assert(sizeof(GradSmem<K, V>) <= 227 * 1024 && sizeof(PrepSmem<K, V>) <= 227 * 1024 &&
                      2 * (chains_smem<K>() + 1024) <= 228 * 1024,
                  "shared memory of one block");
    const GdrArgs &a = g.f;
    const Layout l = layout(a);
    float *partial = static_cast<float *>(a.workspace) + (size_t)l.heads * l.NC * l.per();
    const int64_t chains = l.heads * (V / kSlice);
    cudaError_t e = go(prep_kernel<K, V>, l.heads * l.NC, sizeof(PrepSmem<K, V>), st, g, l);
    if (e == cudaSuccess)
        e = go(chains_kernel<K>, 2 * chains, chains_smem<K>(), st, g, l, (int)chains);
    if (e == cudaSuccess)
        e = go(grad_kernel<K, V>, (int64_t)a.Bsz * a.Hk * l.NC, sizeof(GradSmem<K, V>), st, g, l, partial);
    if (e != cudaSuccess)
        return e;
    head_sum_kernel<<<a.Hv, 32, 0, st>>>(partial, (int64_t)a.Bsz * l.NC, a.Hv, g.dA, g.dbias);
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
    if (g.f.K == 128)
        return g.f.V == 128 ? launch<128, 128>(g, st) : launch<128, 64>(g, st);
    return g.f.V == 128 ? launch<64, 128>(g, st) : launch<64, 64>(g, st);
}

}  // namespace ssm
