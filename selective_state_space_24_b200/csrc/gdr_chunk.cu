// gdr_chunk.cu -- the gated delta rule over sequences, chunk by chunk on the
// tensor cores (tcgen05, TMA, tensor memory).
//
// With q~ = scale q / |q|, k^ = k / |k| and, in a chunk of 64 steps,
// cs = the inclusive sum of the log decays (base 2), G_ij = 2^(cs_i - cs_j),
// c_i = 2^cs_i, e_j = 2^(cs_end - cs_j), the steps of a chunk together are
//     A_ij = b_i G_ij k^_i.k^_j  (j < i),   T = (I + A)^-1,   P = G o (Q~ K^T)  (j <= i)
//     N = T diag(b) (V - diag(c) K^ S^T)
//     O = diag(c) Q~ S^T + P N
//     S = c_end S + N^T diag(e) K^
// One block owns one (batch, value head) and walks its chunks; only S passes
// on.  Everything is kept transposed, value channels down: lane v of tensor
// memory and of the state's threads is row v of S (V, K), so S, N^T and O^T
// go from one product to the next as A operands in tensor memory, written by
// the thread that read their accumulator, with no exchange between threads.
// The norms of q and k, b and all decays are scalars of a row or column and
// stay outside the products: K, Q and V are read as they came.
//
// Roundings: K, Q are exact bf16; S, diag(b)(V - ..), N diag(e), N, T and P
// enter their products as bf16 pairs hi + lo (at least 16 bits, off by up to
// 2^-17), two products with K or Q, three (hi hi, hi lo, lo hi) where both
// factors are pairs.  So the state, float32 in registers between chunks, is
// 3.8e-6 off the definition in the 2-norm (3.2 to 5.2e-6 over the shapes), where
// float32 products leave 2e-7: a choice for the chain's length (a third part is
// half as many products again, and tensor memory is full).  gdr_step is float32
// throughout, gdr_chunk_bwd's products carry 21 bits.  Outputs are rounded to bf16,
// 1.7e-3.  T is inverted with float32 in its 16 x 16 diagonal blocks and bf16
// pairs between them.  Log decays are summed as float pairs (gdr_math.cuh).
//
// Per chunk the state's dependence runs S -> S K^T -> (V - ..) -> T .. -> N ->
// N^T K -> S: three products of the tensor core with a pass of the state's
// sixteen warps (a lane's row in quarters) after each.  The two halves of S's
// columns (K = 128) are handed on one by one, so their passes overlap with
// products.  Beside it, for the chunks ahead, two teams of four warps in turn
// build P and T from K K^T and Q K^T (one product), one warp brings the tiles
// of K and Q (TMA, three stages) and the log decays, one those of V, and the
// outputs of a chunk are read and written while T's product of the next runs.
//
// Bound by the latency of that dependence: three products, three passes
// through tensor memory and the barriers between them, 3.7-3.8 us a chunk,
// whatever HBM and the tensor cores could do.  So one block of 28 warps per
// SM, a role each, and nothing but the dependence between two chunks' states.
// Measured on B200, K = V = 128: 1 x 4096, 32 heads 233 us; 4 x 8192, 32
// heads (128 blocks for 148 SMs) 541 to 553 us on different GPUs, 0.30 of the
// rate of a copy.  Steps on the way, 4 x 8192: 9650 us on
// FMA units, 620 with the chain on the tensor cores, 576 with the outputs
// behind T's product, 540 with the scalars laid out for packed arithmetic and
// waits that poll less, then K K^T of the chunk after next issued behind T's
// product.  (Log decays as float pairs cost 0.5 to 1% of these.)
//
// The size of the code counts too.  Seven loops run on an SM at once, and
// where more than about 14 SMs of a GPC run them their instruction cache
// misses: 3.7 us a chunk with 112 blocks, 4.7 with 148, a third of the warps'
// stalls "no instruction" (before what follows).  So what appeared twice appears once and products are
// issued from loops over 64 columns: 128 blocks 4.16 -> 3.77 us a chunk, 148
// 4.70 -> 4.15 (4.17 now).  (One code for all rows of T saves another 4 KB, 148 blocks
// 3.80 us, but lengthens T's latency: 128 blocks 3.95; loops of single products
// issue too slowly: 16 blocks 3.47 -> 3.65.)
#include <atomic>
#include <type_traits>

#include "gdr_math.cuh"
#include "tc100.cuh"

namespace ssm {

__device__ unsigned g_gdr_error;   // a bounded wait gave up

namespace {

using bf16 = __nv_bfloat16;

constexpr int kC = 64;                        // steps per chunk
constexpr int kTile = kC * 128;               // 64 rows of 64 bf16
// shared memory.  K, Q: three stages (first halves, then second halves of the
// rows); V, later the outputs in its place: two; P and T as bf16 pairs
// hi, lo, rows K-major: three and two (T: A left of the diagonal before it);
// the scalars of four chunks
constexpr int kKQ = 3, kP = 3, kVecs = 4;
constexpr int kAhead = 2;   // chunks between a tile's prefetch into L2 and its load
constexpr int kOffV = kKQ * 4 * kTile;
constexpr int kOffP = kOffV + 2 * 2 * kTile;
constexpr int kOffT = kOffP + kP * 2 * kTile;
constexpr int kOffVec = kOffT + 2 * 2 * kTile;
struct Vec {               // of one chunk
    float ncs[kC], ncl[kC]; // -cs as hi + lo
    float rk[kC];          // 2^-lo / |k| (each array apart: neighbours make pairs for packed arithmetic)
    float4 bg[kC / 2];     // b of two steps, their -b c / |k|
    float gq[kC];          // c scale / |q| (first 1 / |q|)
    float ek[kC];          // e / |k|
    float b[kC];
    float dec;             // 2^cs_end
    float pad[3];
};
struct Bars {
    uint64_t full[kKQ], empty[kKQ], scal[kVecs], vfull[2], out[2], ready[2], kk[2], o[2], s[2], x[2], team[2][3];
    uint64_t ks, d, t, n, qs, oread, kkread, done;
    uint32_t tmem;
    int abort;
};
constexpr int kOffBars = kOffVec + kVecs * (int)sizeof(Vec);
constexpr int kSmem = kOffBars + (int)sizeof(Bars);
static_assert(kSmem <= 227 * 1024, "shared memory of one block");

// tensor memory columns.  S: per 16 columns of the state 8 of bf16 pairs hi
// and 8 lo, in place of the 16 float32 that N^T K leaves there
constexpr uint32_t kColS = 0;      // 128
constexpr uint32_t kColKS = 128;   // 64: S K^T, then N
constexpr uint32_t kColQS = 192;   // 64
constexpr uint32_t kColPN = 256;   // 64
constexpr uint32_t kColKK = 320;   // 64: lanes 0..63 K K^T, 64..127 Q K^T
constexpr uint32_t kColX = 384;    // 64: hi 32, lo 32 of diag(b)(V - ..), then of N diag(e)
constexpr uint32_t kColN = 448;    // 64: hi 32, lo 32 of N
constexpr int kTmemCols = 512;

constexpr int kStateWarps = 16, kTeamWarp = 16, kMmaWarp = 24, kLoadWarp = 25, kValueWarp = 26, kThreads = 28 * 32;
// Registers: launched with 72 a thread (64,512 in all), which the state's
// sixteen warps keep; the last four (products, loads, values, one idle) give
// up 32 x 128, the two teams take 16 x 256.
constexpr int kRegsTeam = 88, kRegsIssue = 40;

// STALL: the same kernel for the test of its waits' end, with their limit and a
// chunk to withhold from the arguments (read in every call, they cost 11%).
template <int K, bool STALL>
__global__ void __launch_bounds__(kThreads, 1)
    gdr_chunk_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapK,
                     const __grid_constant__ CUtensorMap mapV, const __grid_constant__ CUtensorMap mapO, const GdrArgs a, const int nch)
{
    using namespace tc;
    constexpr int KQ = K / 4;             // columns of S of one quarter of the state's threads
    constexpr int kSteps = K / 16;
    // used as declared (no arithmetic on its address), so that the compiler
    // knows every access for one to shared memory
    extern __shared__ __align__(1024) uint8_t sm[];
    Bars &bars = *reinterpret_cast<Bars *>(sm + kOffBars);

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);   // known to be the same for the warp
    const int64_t bh = blockIdx.x;
    const int h = (int)(bh % a.Hv), hk = h / (a.Hv / a.Hk);
    const int b = (int)(bh / a.Hv);
    const int L = a.L, V = a.V;

    if (tid == 0) {
        for (int i = 0; i < kKQ; i++) {
            bar_init(&bars.full[i], 1);
            bar_init(&bars.empty[i], 1);
        }
        for (int i = 0; i < kVecs; i++)
            bar_init(&bars.scal[i], 32);
        for (int i = 0; i < 2; i++) {
            bar_init(&bars.vfull[i], 1);
            bar_init(&bars.out[i], kStateWarps);
            bar_init(&bars.ready[i], 4);
            bar_init(&bars.kk[i], 1);
            bar_init(&bars.o[i], 1);
            bar_init(&bars.s[i], kStateWarps / 2);
            bar_init(&bars.x[i], 1);
            for (int j = 0; j < 3; j++)
                bar_init(&bars.team[i][j], 4);
        }
        bar_init(&bars.ks, 1);
        bar_init(&bars.d, kStateWarps);
        bar_init(&bars.t, 1);
        bar_init(&bars.n, kStateWarps);
        bar_init(&bars.qs, 1);
        bar_init(&bars.oread, kStateWarps);
        bar_init(&bars.kkread, 4);
        bar_init(&bars.done, 1);
        bars.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0)
        tmem_alloc(&bars.tmem, kTmemCols);
    // P and T stay zero right of their diagonal blocks
    for (int i = tid; i < (kOffVec - kOffP) / 16; i += kThreads)
        reinterpret_cast<uint4 *>(sm + kOffP)[i] = make_uint4(0, 0, 0, 0);
    fence_smem();
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tm = __shfl_sync(0xffffffffu, bars.tmem, 0);
    volatile int *abort = &bars.abort;
    bool failed = false;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (warp_wait(bar, parity, abort, STALL ? a.wait_limit : kWaitLimit))
            return true;
        failed = true;
        return false;
    };
    auto stage = [&](int c) { return sm + (c % kKQ) * 4 * kTile; };   // K, Q
    auto vtile = [&](int c) { return sm + kOffV + (c & 1) * 2 * kTile; };
    auto vec = [&](int c) { return reinterpret_cast<Vec *>(sm + kOffVec) + c % kVecs; };
    auto phase = [](int c) { return (uint32_t)((c / kKQ) & 1); };     // of the stages
    auto phase2 = [](int c) { return (uint32_t)((c >> 1) & 1); };     // of what there are two of
    auto arrive1 = [&](uint64_t *bar) {   // one arrival of this warp, after all its lanes
        __syncwarp();
        if (lane == 0)
            bar_arrive(bar);
    };

    if (warp < kStateWarps) {
        // ---- the state's threads: lane row v, a quarter of K's columns and of a chunk's steps
        const int quarter = warp >> 2, half = quarter >> 1, v = (warp & 3) * 32 + lane;
        const bool live = (warp & 3) * 32 < V;   // V = 64: half of the warps only keep step
        const uint32_t tl = tm + ((uint32_t)((warp & 3) * 32) << 16);
        float S[KQ];
        const size_t srow = ((size_t)bh * V + v) * K + quarter * KQ;
        if (live && a.init) {
#pragma unroll
            for (int i = 0; i < KQ; i += 4) {
                const float4 f = *reinterpret_cast<const float4 *>(a.init + srow + i);
                S[i] = f.x, S[i + 1] = f.y, S[i + 2] = f.z, S[i + 3] = f.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < KQ; i++)
                S[i] = 0.f;
        }
        auto put_S = [&](int p) {   // 16 columns of S as an operand
            uint32_t hi[8], lo[8];
#pragma unroll
            for (int i = 0; i < 8; i++)
                split(S[16 * p + 2 * i], S[16 * p + 2 * i + 1], hi[i], lo[i]);
            tmem_st(tl + kColS + quarter * KQ + 16 * p, hi);
            tmem_st(tl + kColS + quarter * KQ + 16 * p + 8, lo);
        };
        if (live) {
#pragma unroll
            for (int p = 0; p < KQ / 16; p++)
                put_S(p);
            tmem_wait_st();
        }
        fence_before();
        arrive1(&bars.s[half]);
        // outputs of a quarter of chunk c's steps, in the place of its V
        auto outputs = [&](int c) {
            if (!wait(&bars.o[c & 1], phase2(c)))
                return false;
            fence_after();
            if (live) {
                const Vec *ve = vec(c);
                const uint32_t vpitch = 2 * V;
                uint8_t *ot = vtile(c) + 16 * quarter * vpitch + 2 * v;
                uint32_t q[16], p[16];
                tmem_ld(tl + kColQS + 16 * quarter, q);
                tmem_ld(tl + kColPN + 16 * quarter, p);
                tmem_wait(q);
                tmem_wait(p);
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    const float2 g = *reinterpret_cast<const float2 *>(&ve->gq[16 * quarter + e]);
                    const float2 y = __ffma2_rn(g, make_float2(__uint_as_float(q[e]), __uint_as_float(q[e + 1])),
                                                make_float2(__uint_as_float(p[e]), __uint_as_float(p[e + 1])));
                    const uint32_t w = pack(y.x, y.y);
                    *reinterpret_cast<uint16_t *>(ot + e * vpitch) = (uint16_t)w;
                    *reinterpret_cast<uint16_t *>(ot + (e + 1) * vpitch) = (uint16_t)(w >> 16);
                }
            }
            fence_before();
            arrive1(&bars.oread);
            fence_smem();
            arrive1(&bars.out[c & 1]);
            return true;
        };
        for (int c = 0; c <= nch; c++) {
            const Vec *ve = vec(c);
            const bool more = c < nch;   // else only the last chunk's outputs are left
            // 1. diag(b)(V - diag(c) K^ S^T), this quarter's 16 steps
            if (more && (!wait(&bars.vfull[c & 1], phase2(c)) || !wait(&bars.ready[c & 1], phase2(c)) || !wait(&bars.ks, c & 1)))
                break;
            fence_after();
            if (more && live) {
                const uint32_t vpitch = 2 * V;
                const uint8_t *vt = vtile(c) + 16 * quarter * vpitch + 2 * v;
                uint32_t r[16], hi[8], lo[8];
                tmem_ld(tl + kColKS + 16 * quarter, r);
                tmem_wait(r);
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    const float4 bg = ve->bg[8 * quarter + i];
                    const float v0 = __bfloat162float(*reinterpret_cast<const bf16 *>(vt + 2 * i * vpitch));
                    const float v1 = __bfloat162float(*reinterpret_cast<const bf16 *>(vt + (2 * i + 1) * vpitch));
                    const float2 x = __ffma2_rn(make_float2(bg.z, bg.w),
                                                make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])),
                                                __fmul2_rn(make_float2(bg.x, bg.y), make_float2(v0, v1)));
                    split(x.x, x.y, hi[i], lo[i]);
                }
                tmem_st(tl + kColX + 8 * quarter, hi);
                tmem_st(tl + kColX + 32 + 8 * quarter, lo);
                tmem_wait_st();
            }
            fence_before();
            if (more)
                arrive1(&bars.d);
            // 2. N for the outputs, N diag(e) for the state (the last chunk's outputs
            // while T's product runs)
            if ((c > 0 && !outputs(c - 1)) || !more || !wait(&bars.t, c & 1))
                break;
            fence_after();
            if (live) {
                uint32_t r[16], hi[8], lo[8];
                tmem_ld(tl + kColKS + 16 * quarter, r);
                tmem_wait(r);
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    const float2 e = *reinterpret_cast<const float2 *>(&ve->ek[16 * quarter + 2 * i]);
                    const float2 ne =
                        __fmul2_rn(make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), e);
                    split(ne.x, ne.y, hi[i], lo[i]);
                }
                tmem_st(tl + kColX + 8 * quarter, hi);
                tmem_st(tl + kColX + 32 + 8 * quarter, lo);
#pragma unroll
                for (int i = 0; i < 8; i++)
                    split(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]), hi[i], lo[i]);
                tmem_st(tl + kColN + 8 * quarter, hi);
                tmem_st(tl + kColN + 32 + 8 * quarter, lo);
                tmem_wait_st();
            }
            fence_before();
            arrive1(&bars.n);
            // 3. S = c_end S + N^T diag(e) K^, this quarter's columns
            if (!wait(&bars.x[half], c & 1))
                break;
            fence_after();
            if (live) {
                const float dec = ve->dec;
#pragma unroll
                for (int p = 0; p < KQ / 16; p++) {
                    uint32_t r[16];
                    tmem_ld(tl + kColS + quarter * KQ + 16 * p, r);
                    tmem_wait(r);
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        const float2 x = __ffma2_rn(make_float2(dec, dec), make_float2(S[16 * p + i], S[16 * p + i + 1]),
                                                    make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])));
                        S[16 * p + i] = x.x;
                        S[16 * p + i + 1] = x.y;
                    }
                    put_S(p);
                }
                tmem_wait_st();
            }
            fence_before();
            arrive1(&bars.s[half]);
        }
        if (live && a.last && !failed && !*abort) {
#pragma unroll
            for (int i = 0; i < KQ; i += 4)
                *reinterpret_cast<float4 *>(a.last + srow + i) = make_float4(S[i], S[i + 1], S[i + 2], S[i + 3]);
        }
    } else if (warp < kMmaWarp) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsTeam));
        // ---- the teams that build P, T and the scalars: thread = row of K (0..63) or of Q
        const int team = (warp - kTeamWarp) >> 2, pw = warp & 3;
        const int row = pw * 32 + lane;          // lane of tensor memory
        const bool isq = pw >= 2;
        const int i = row & 63;                  // step in the chunk
        const uint32_t tl = tm + ((uint32_t)(pw * 32) << 16);
        int turn = 0;
        for (int c = team; c < nch; c += 2, turn++) {
            Vec *ve = vec(c);
            const uint8_t *st = stage(c);
            uint8_t *Pb = sm + kOffP + (c % kP) * 2 * kTile, *Tb = sm + kOffT + team * 2 * kTile;
            const uint32_t tb = smem_u32(Tb);
            if (!wait(&bars.scal[c % kVecs], (c / kVecs) & 1) || !wait(&bars.full[c % kKQ], phase(c)))
                break;
            if (a.l2norm) {
                // squares of 16 rows of K and of Q: the diagonal of their products with themselves
                float acc[2][2][4] = {};
#pragma unroll 2
                for (int k = 0; k < kSteps; k++)
#pragma unroll
                    for (int m = 0; m < 2; m++) {
                        uint32_t r[4];
                        ldsm(smem_u32(st) + ((k >> 2) * 2 + m) * kTile +
                                 sw128(16 * pw + (lane & 7) + ((lane >> 3) & 1) * 8, 2 * (k & 3) + (lane >> 4)),
                             r);
                        mma16816(acc[m][0], r, r[0], r[2]);
                        mma16816(acc[m][1], r, r[1], r[3]);
                    }
                if ((lane & 3) == lane >> 3) {   // columns 2 t, 2 t + 1 hold the diagonal of row lane / 4
                    const int r0 = 16 * pw + (lane >> 2);
#pragma unroll
                    for (int m = 0; m < 2; m++) {
                        float *n = m ? ve->gq : ve->rk;
                        const float w = m ? 0.f : 1.f;
                        n[r0] = rsqrtf(((lane >> 2) & 1 ? acc[m][0][1] : acc[m][0][0]) + kL2Eps) * gdr_rest(w, ve->ncl[r0]);
                        n[r0 + 8] =
                            rsqrtf(((lane >> 2) & 1 ? acc[m][1][3] : acc[m][1][2]) + kL2Eps) * gdr_rest(w, ve->ncl[r0 + 8]);
                    }
                }
            } else if (!isq) {
                ve->rk[i] = gdr_rest(1.f, ve->ncl[i]);
            } else {
                ve->gq[i] = 1.f;
            }
            arrive1(&bars.team[team][0]);
            if (!wait(&bars.team[team][0], turn & 1) || !wait(&bars.kk[team], turn & 1))
                break;
            fence_after();
            // the row's factor, 2^lo in it; a column's, rk, has 2^-lo
            const float csi = -ve->ncs[i], nl = ve->ncl[i];
            const float f = isq ? a.scale * ve->gq[i] * gdr_rest(-1.f, nl) : ve->rk[i] * ve->b[i] * gdr_rest(-2.f, nl);
            const int last = isq ? i : i - 1, blk = i >> 4, il = i & 15;
            // rows of 16 as bf16 pairs: of P; of A left of the diagonal block, that block's inverse in it
            auto put = [&](uint8_t *to, int at_blk, const float (&x)[16]) {
                uint32_t hi[8], lo[8];
#pragma unroll
                for (int e = 0; e < 8; e++)
                    split(x[2 * e], x[2 * e + 1], hi[e], lo[e]);
#pragma unroll
                for (int q = 0; q < 2; q++) {
                    const uint32_t at = sw128(i, 2 * at_blk + q);
                    *reinterpret_cast<uint4 *>(to + at) = make_uint4(hi[4 * q], hi[4 * q + 1], hi[4 * q + 2], hi[4 * q + 3]);
                    *reinterpret_cast<uint4 *>(to + kTile + at) = make_uint4(lo[4 * q], lo[4 * q + 1], lo[4 * q + 2], lo[4 * q + 3]);
                }
            };
            float d[16];   // this row of the diagonal block of A
#pragma unroll
            for (int j = 0; j < 16; j++)
                d[j] = 0.f;
            const int reach = 2 * (pw & 1) + 1;   // last block of columns that some row of the warp reaches
#pragma unroll 1
            for (int p = 0; p <= reach; p++) {
                float w[16];
                uint32_t r[16];
                tmem_ld(tl + kColKK + 16 * p, r);
                tmem_wait(r);
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                    const float4 nc = *reinterpret_cast<const float4 *>(&ve->ncs[16 * p + j]);
                    const float4 rk = *reinterpret_cast<const float4 *>(&ve->rk[16 * p + j]);
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        const float2 e = __fadd2_rn(make_float2(csi, csi), h ? make_float2(nc.z, nc.w) : make_float2(nc.x, nc.y));
                        const float2 g = __fmul2_rn(make_float2(ex2_mufu(e.x), ex2_mufu(e.y)),
                                                    h ? make_float2(rk.z, rk.w) : make_float2(rk.x, rk.y));
                        const float2 x = __fmul2_rn(make_float2(__uint_as_float(r[j + 2 * h]), __uint_as_float(r[j + 2 * h + 1])),
                                                    make_float2(f, f));
                        const float2 y = __fmul2_rn(g, x);
                        w[j + 2 * h] = y.x;
                        w[j + 2 * h + 1] = y.y;
                    }
                }
                if (p >= reach - 1) {   // the warp's diagonal: zeros right of it
                    const int n = last - 16 * p;
#pragma unroll
                    for (int j = 0; j < 16; j++)
                        w[j] = j <= n ? w[j] : 0.f;
                }
                if (isq || p < blk) {
                    put(isq ? Pb : Tb, p, w);
                } else if (p == blk) {
#pragma unroll
                    for (int j = 0; j < 16; j++)
                        d[j] = w[j];
                }
            }
            fence_before();
            arrive1(&bars.kkread);
            if (!isq) {
                float x[16];
#pragma unroll
                for (int j = 0; j < 16; j++)
                    x[j] = 0.f;
                // row il of the inverse of I + D from the right: x_k is final once all
                // later ones are, then leaves -x_k D_kj in the columns j < k
#pragma unroll
                for (int k = 15; k >= 0; k--) {
                    x[k] = k == il ? 1.f : x[k];
#pragma unroll
                    for (int j = 0; j < k; j++)
                        x[j] = fmaf(-x[k], __shfl_sync(0xffffffffu, d[j], (lane & 16) | k), x[j]);
                }
                put(Tb, blk, x);
            }
            arrive1(&bars.team[team][1]);
            if (!wait(&bars.team[team][1], turn & 1))
                break;
            // block row pw of T: T_ij = -(sum_{j < k <= i} T_ik A_kj) T_jj, as A operands of the next sums
            uint32_t th[4][4], tlo[4][4];
            const uint32_t aoff = (lane & 7) + ((lane >> 3) & 1) * 8;
            auto load_a = [&](int bi, int bj, uint32_t (&hi)[4], uint32_t (&lo)[4]) {
                const uint32_t at = tb + sw128(16 * bi + aoff, 2 * bj + (lane >> 4));
                ldsm(at, hi);
                ldsm(at + kTile, lo);
            };
            auto load_b = [&](int bi, int bj, uint32_t (&hi)[4], uint32_t (&lo)[4]) {
                const uint32_t at = tb + sw128(16 * bi + aoff, 2 * bj + (lane >> 4));
                ldsm_t(at, hi);
                ldsm_t(at + kTile, lo);
            };
            auto prod = [&](float (&acc)[2][4], const uint32_t (&ah)[4], const uint32_t (&al)[4], const uint32_t (&bh_)[4],
                            const uint32_t (&bl)[4]) {
#pragma unroll
                for (int n = 0; n < 2; n++) {
                    mma16816(acc[n], ah, bh_[2 * n], bh_[2 * n + 1]);
                    mma16816(acc[n], ah, bl[2 * n], bl[2 * n + 1]);
                    mma16816(acc[n], al, bh_[2 * n], bh_[2 * n + 1]);
                }
            };
            auto as_a = [&](const float (&acc)[2][4], float sign, uint32_t (&hi)[4], uint32_t (&lo)[4]) {
                split(sign * acc[0][0], sign * acc[0][1], hi[0], lo[0]);
                split(sign * acc[0][2], sign * acc[0][3], hi[1], lo[1]);
                split(sign * acc[1][0], sign * acc[1][1], hi[2], lo[2]);
                split(sign * acc[1][2], sign * acc[1][3], hi[3], lo[3]);
            };
            auto row_of_T = [&](auto I) {
                constexpr int bi = decltype(I)::value;
                load_a(bi, bi, th[bi], tlo[bi]);
#pragma unroll
                for (int j = bi - 1; j >= 0; j--) {
                    float acc[2][4] = {}, res[2][4] = {};
                    uint32_t bh_[4], bl[4], mh[4], ml[4];
#pragma unroll
                    for (int k = bi; k > j; k--) {
                        load_b(k, j, bh_, bl);
                        prod(acc, th[k], tlo[k], bh_, bl);
                    }
                    as_a(acc, -1.f, mh, ml);
                    load_b(j, j, bh_, bl);
                    prod(res, mh, ml, bh_, bl);
                    as_a(res, 1.f, th[j], tlo[j]);
                }
            };
            if (pw == 0) {   // no blocks left of the first: the scalars instead
                const float end = -ve->ncs[kC - 1], rest = gdr_rest(-1.f, ve->ncl[kC - 1]);
#pragma unroll
                for (int s = 0; s < 2; s++) {
                    const int at = lane + 32 * s;
                    const float nc = ve->ncs[at], rk = ve->rk[at], bb = ve->b[at];
                    float *bg = reinterpret_cast<float *>(&ve->bg[at / 2]) + (at & 1);
                    bg[0] = bb;
                    bg[2] = -bb * ex2_mufu(-nc) * rk;   // c to 2^-24 |cs| (lo, and rk's), as it is 2^cs
                    ve->ek[at] = ex2_mufu(end + nc) * rest * rk;
                }
                if (lane == 0)
                    ve->dec = ex2_mufu(end);
            } else if (pw == 1) {
                row_of_T(std::integral_constant<int, 1>());
            } else if (pw == 2) {
                row_of_T(std::integral_constant<int, 2>());
            } else {
                row_of_T(std::integral_constant<int, 3>());
            }
            if (isq)
                ve->gq[i] = ex2_mufu(csi) * f;
            arrive1(&bars.team[team][2]);
            if (!wait(&bars.team[team][2], turn & 1))   // nobody reads A any more
                break;
#pragma unroll
            for (int j = 0; j < 3; j++)
                if (j < pw)
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const uint32_t at = sw128(16 * pw + (lane >> 2) + 8 * (e & 1), 2 * j + (e >> 1)) + (lane & 3) * 4;
                        *reinterpret_cast<uint32_t *>(Tb + at) = th[j][e];
                        *reinterpret_cast<uint32_t *>(Tb + kTile + at) = tlo[j][e];
                    }
            fence_smem();
            arrive1(&bars.ready[team]);
        }
    } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    if (warp == kMmaWarp) {
        // ---- one lane issues every product of the chain
        constexpr uint32_t id64 = idesc(128, 64, 0, 0);       // B: rows of 64 steps, K-major
        constexpr uint32_t idUp = idesc(128, 64, 0, 1);       // B: K itself, steps along K
        auto issue_kk = [&](int c) {
            const uint64_t s = operand(smem_u32(stage(c)));
            if (elect()) {
                fence_after();
#pragma unroll 1
                for (int f = 0; f < K / 64; f++)
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        const uint64_t o = s + ((f * 2 * kTile + k * 32) >> 4);
                        mma_ss(tm + kColKK, o, o, id64, f + k > 0);
                    }
                commit(&bars.kk[c & 1]);
            }
            __syncwarp();
        };
        bool ok = true;
        int next_kk = 0;   // the next chunk whose K K^T is to be issued
        auto kk_blocking = [&] {
            if (next_kk >= nch)
                return true;
            if (!wait(&bars.full[next_kk % kKQ], phase(next_kk)) ||
                (next_kk > 0 && !wait(&bars.kkread, (next_kk - 1) & 1)))
                return false;
            issue_kk(next_kk++);
            return true;
        };
        // the same if its tiles are here and the last one is read
        auto kk_if_ready = [&](int c) {
            if (next_kk == c && c < nch &&
                __all_sync(0xffffffffu, bar_test(&bars.full[c % kKQ], phase(c)) && bar_test(&bars.kkread, (c - 1) & 1)))
                issue_kk(next_kk++);
        };
#pragma unroll 1
        for (int i = 0; i < 2 && ok; i++)
            ok = kk_blocking();
        for (int c = 0; c < nch && ok; c++) {
            const uint64_t s = operand(smem_u32(stage(c)));
            const uint64_t T = operand(smem_u32(sm + kOffT + (c & 1) * 2 * kTile));
            const uint64_t P = operand(smem_u32(sm + kOffP + (c % kP) * 2 * kTile));
            // S K^T (hi + lo), a half of S's columns at a time
#pragma unroll 1
            for (int half = 0; half < 2; half++) {
                ok = wait(&bars.s[half], c & 1);
                if (!ok)
                    break;
                if (elect()) {
                    fence_after();
#pragma unroll
                    for (int i = 0; i < kSteps / 2; i++) {
                        const int k = half * (kSteps / 2) + i;
                        const uint64_t kd = s + (((k >> 2) * 2 * kTile + (k & 3) * 32) >> 4);
                        mma_ts(tm + kColKS, tm + kColS + 16 * k, kd, id64, k > 0);
                        mma_ts(tm + kColKS, tm + kColS + 16 * k + 8, kd, id64, true);
                    }
                    if (half == 1)
                        commit(&bars.ks);
                }
                __syncwarp();
            }
            if (!ok)
                break;
            if (next_kk == c + 1 && !kk_blocking())
                break;
            // N = T (..): hi hi, hi lo, lo hi
            if (!wait(&bars.ready[c & 1], phase2(c)) || !wait(&bars.d, c & 1))
                break;
            if (elect()) {
                fence_after();
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    mma_ts(tm + kColKS, tm + kColX + 8 * k, T + 2 * k, id64, k > 0);
                    mma_ts(tm + kColKS, tm + kColX + 8 * k, T + (kTile >> 4) + 2 * k, id64, true);
                    mma_ts(tm + kColKS, tm + kColX + 32 + 8 * k, T + 2 * k, id64, true);
                }
                commit(&bars.t);
            }
            __syncwarp();
            // for the chunk after next, if its tiles are here (else further on):
            // its team may overwrite T now, and has that much more time
            kk_if_ready(c + 2);
            // Q~ S^T, once the last chunk's outputs are read; done before S makes way
            if (c > 0 && !wait(&bars.oread, (c - 1) & 1))
                break;
            if (elect()) {
                fence_after();
#pragma unroll 1
                for (int f = 0; f < K / 64; f++)
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        const uint64_t qd = s + (((f * 2 + 1) * kTile + k * 32) >> 4);
                        mma_ts(tm + kColQS, tm + kColS + 64 * f + 16 * k, qd, id64, f + k > 0);
                        mma_ts(tm + kColQS, tm + kColS + 64 * f + 16 * k + 8, qd, id64, true);
                    }
                commit(&bars.qs);
            }
            __syncwarp();
            if (!wait(&bars.qs, c & 1) || !wait(&bars.n, c & 1))
                break;
            if (elect()) {
                fence_after();
#pragma unroll 1
                for (int f = 0; f < K / 64; f++) {   // 64 columns of N^T diag(e) K^ (hi + lo) in S's place
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        const uint64_t kd = s + ((f * 2 * kTile + k * 2048) >> 4);
                        mma_ts(tm + kColS + 64 * f, tm + kColX + 8 * k, kd, idUp, k > 0);
                        mma_ts(tm + kColS + 64 * f, tm + kColX + 32 + 8 * k, kd, idUp, true);
                    }
                    commit(&bars.x[f]);
                }
                if (K == 64)
                    commit(&bars.x[1]);
#pragma unroll
                for (int k = 0; k < 4; k++) {   // P N: hi hi, hi lo, lo hi
                    mma_ts(tm + kColPN, tm + kColN + 8 * k, P + 2 * k, id64, k > 0);
                    mma_ts(tm + kColPN, tm + kColN + 8 * k, P + (kTile >> 4) + 2 * k, id64, true);
                    mma_ts(tm + kColPN, tm + kColN + 32 + 8 * k, P + 2 * k, id64, true);
                }
                commit(&bars.o[c & 1]);
                commit(&bars.empty[c % kKQ]);
            }
            __syncwarp();
            kk_if_ready(c + 2);
        }
        if (elect()) {
            commit(&bars.done);
            drain(&bars.done, 0, &g_gdr_error);
        }
        __syncwarp();
    } else if (warp == kLoadWarp) {
        // ---- K, Q, the log decays and b, up to three chunks ahead
        const float bias = a.bias ? a.bias[h] : 0.f, Ah = a.A[h] * kLog2e;
        const bf16 *dp = static_cast<const bf16 *>(a.delta) + (size_t)b * L * a.Hv + h;
        const bf16 *bp = static_cast<const bf16 *>(a.beta) + (size_t)b * L * a.Hv + h;
        int issued = -1;
        float dl[2], be[2];
        auto fetch = [&](int c) {
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const int t = c * kC + 2 * lane + e;
                dl[e] = c < nch && t < L ? gdr_ld(dp, (size_t)t * a.Hv) : 0.f;
                be[e] = c < nch && t < L ? gdr_ld(bp, (size_t)t * a.Hv) : 0.f;
            }
        };
        fetch(0);
        for (int c = 0; c < nch; c++) {
            float g[2], bb[2];
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const bool in = c * kC + 2 * lane + e < L;
                g[e] = in ? gdr_log_decay(gdr_dt(dl[e], bias, a.softplus), Ah) : 0.f;
                bb[e] = in ? (a.sigmoid ? sigmoid_mufu(be[e]) : be[e]) : 0.f;
            }
            fetch(c + 1);
            float2 cs[2];
            gdr_log_sums(g, cs);
            if (c >= kKQ && !wait(&bars.empty[c % kKQ], phase(c - kKQ)))
                break;
            if (__any_sync(0xffffffffu, *abort))
                break;
            if (elect()) {
                uint8_t *st = stage(c);
                uint64_t *bar = &bars.full[c % kKQ];
                bar_expect(bar, 2 * (K / 64) * kTile);
#pragma unroll
                for (int f = 0; f < K / 64; f++) {
                    tma_4d(st + 2 * f * kTile, &mapK, 64 * f, hk, c * kC, b, bar);
                    tma_4d(st + (2 * f + 1) * kTile, &mapQ, 64 * f, hk, c * kC, b, bar);
                }
                if (c + kAhead < nch) {   // DRAM's latency is longer than the stages reach
#pragma unroll
                    for (int f = 0; f < K / 64; f++) {
                        tma_prefetch_4d(&mapK, 64 * f, hk, (c + kAhead) * kC, b);
                        tma_prefetch_4d(&mapQ, 64 * f, hk, (c + kAhead) * kC, b);
                    }
                    tma_prefetch_4d(&mapV, 0, h, (c + kAhead) * kC, b);
                }
            }
            issued = c;
            Vec *ve = vec(c);
            *reinterpret_cast<float2 *>(&ve->ncs[2 * lane]) = make_float2(-cs[0].x, -cs[1].x);
            *reinterpret_cast<float2 *>(&ve->ncl[2 * lane]) = make_float2(-cs[0].y, -cs[1].y);
            ve->b[2 * lane] = bb[0];
            ve->b[2 * lane + 1] = bb[1];
            if (!STALL || c != a.withhold_chunk)
                bar_arrive(&bars.scal[c % kVecs]);
        }
        if (lane == 0)
            for (int c = max(0, issued - kKQ + 1); c <= issued; c++)
                drain(&bars.full[c % kKQ], phase(c), &g_gdr_error);
        __syncwarp();
    } else if (warp == kValueWarp) {
        // ---- V, and the outputs from its place
        int issued = -1;
        auto load = [&](int c) {
            if (elect()) {
                bar_expect(&bars.vfull[c & 1], V * kC * 2);
                tma_4d(vtile(c), &mapV, 0, h, c * kC, b, &bars.vfull[c & 1]);
            }
            __syncwarp();
            issued = c;
        };
        for (int c = 0; c < 2 && c < nch; c++)
            load(c);
        for (int c = 0; c < nch; c++) {
            if (!wait(&bars.out[c & 1], phase2(c)))
                break;
            if (elect()) {
                tma_store_4d(&mapO, vtile(c), 0, h, c * kC, b);
                tma_store_wait();
            }
            __syncwarp();
            if (c + 2 < nch)
                load(c + 2);
        }
        if (lane == 0)
            for (int c = max(0, issued - 1); c <= issued; c++)
                drain(&bars.vfull[c & 1], phase2(c), &g_gdr_error);
        __syncwarp();
    }
    }
    if (failed)
        gave_up(abort, &g_gdr_error);
    fence_before();
    __syncthreads();
    if (warp == 0)
        tmem_free(tm, kTmemCols);
}

template <int K, bool STALL> cudaError_t launch(const GdrArgs &a, cudaStream_t st)
{
    CUtensorMap q, k, v, o;
    if (!tc::head_map(&q, a.q, a.Bsz, a.L, a.Hk, a.K, true) || !tc::head_map(&k, a.k, a.Bsz, a.L, a.Hk, a.K, true) ||
        !tc::head_map(&v, a.v, a.Bsz, a.L, a.Hv, a.V, false) || !tc::head_map(&o, a.out, a.Bsz, a.L, a.Hv, a.V, false))
        return cudaErrorInvalidValue;
    const cudaError_t e = cudaFuncSetAttribute(gdr_chunk_kernel<K, STALL>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess)
        return e;
    gdr_chunk_kernel<K, STALL><<<(unsigned)((int64_t)a.Bsz * a.Hv), kThreads, kSmem, st>>>(q, k, v, o, a, (a.L + kC - 1) / kC);
    return cudaGetLastError();
}

}  // namespace

static std::atomic<int> g_withhold_chunk{-1};
static std::atomic<unsigned> g_wait_limit{0};

void gdr_stall_set(int withhold_chunk, unsigned wait_limit)
{
    g_withhold_chunk.store(withhold_chunk);
    g_wait_limit.store(wait_limit);
}

namespace {

// Sequences this short go step by step: one chunk takes 16.5 us (K = 128; 11
// us for K = 64) however little of it is filled, the recurrent kernel 2 us and
// 0.54 us a step while its blocks (of 32 state rows) are at most one per SM,
// 1.0 us a step with 3.5 of them, 0.8 us a step for K = 64.  Measured on B200,
// chunked / recurrent: 32 heads L 24 16.7 / 15.1 us, L 32 16.7 / 19.6; 128
// heads L 12 17.3 / 15.3, L 16 17.3 / 19.5; 1024 heads L 12 121 / 96, L 16
// 121 / 124; K = V = 64, 32 heads L 8 10.9 / 8.1, L 12 10.9 / 11.6.
int recurrent_limit(const GdrArgs &a)
{
    if (a.K == 64)
        return 10;
    return (int64_t)a.Bsz * a.Hv * (a.V / 32) <= 148 ? 26 : 14;
}

}  // namespace

cudaError_t launch_gdr_chunk(const GdrArgs &a, cudaStream_t st)
{
    if (a.L <= recurrent_limit(a))
        return launch_gdr_recurrent(a, st);
    const unsigned limit = g_wait_limit.load();
    const int chunk = g_withhold_chunk.load();
    if (limit || chunk >= 0) {
        GdrArgs b = a;
        b.wait_limit = limit ? limit : tc::kWaitLimit;
        b.withhold_chunk = chunk;
        return a.K == 128 ? launch<128, true>(b, st) : launch<64, true>(b, st);
    }
    return a.K == 128 ? launch<128, false>(a, st) : launch<64, false>(a, st);
}

cudaError_t read_and_clear_gdr_error(unsigned *value, cudaStream_t stream)
{
    cudaError_t e = cudaStreamSynchronize(stream);
    if (e == cudaSuccess)
        e = cudaMemcpyFromSymbol(value, g_gdr_error, sizeof(unsigned));
    const unsigned zero = 0;
    return e == cudaSuccess ? cudaMemcpyToSymbol(g_gdr_error, &zero, sizeof(unsigned)) : e;
}

}  // namespace ssm
