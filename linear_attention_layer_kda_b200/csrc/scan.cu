// scan.cu -- the recurrence over whole sequences: forward (formulas in scan.cuh).
//
//   k_scan_plan    first chunk of every sequence of a ragged batch (one block)
//   k_scan_prep    per chunk and head: Kx, Uv, W, g q, M (and X for the backward pass)
//   k_scan_state   per sequence, head and slice of value columns: U and the states, chunk by chunk;
//                  the same kernel run backwards carries the gradient of the states
//   k_scan_out     per chunk and head: o
//   k_scan_tokens  short sequences (a decode step): the recurrence as written, state in registers
#include "scan_ops.cuh"

namespace kda {
namespace scan {
namespace {

__global__ void __launch_bounds__(1024) k_scan_plan(Args a, int *pre)
{
    // chunk counts of 1024 sequences at a time, summed by a block scan; the total never exceeds the
    // chunks that the workspace holds, whatever cu says
    __shared__ int warps[32];
    __shared__ int base;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) base = 0;
    __syncthreads();
    for (int s0 = 0; s0 < a.nseq; s0 += 1024) {
        const int s = s0 + tid;
        int n = 0;
        if (s < a.nseq) {
            const long long c = (seq_end(a, s) - seq_start(a, s) + kC - 1) / kC;
            n = c > a.max_chunks ? a.max_chunks : (int)c;
        }
        int x = n;  // inclusive sum; saturates, so that repeated ranges cannot overflow
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x = min(x + y, a.max_chunks);
        }
        if (lane == 31) warps[warp] = x;
        __syncthreads();
        int before = base;
        for (int w = 0; w < warp; ++w) before = min(before + warps[w], a.max_chunks);
        x = min(x + before, a.max_chunks);
        if (s < a.nseq) pre[s + 1] = x;
        __syncthreads();
        if (tid == 1023) base = x;
        __syncthreads();
    }
    if (tid == 0) pre[0] = 0;
}

// ---------------------------------------------------------------- preparation

template <int DK, int DV>
struct PrepSmem {
    static constexpr int KH = 0, QS = KH + kC * DK;
    static constexpr int LG = QS + kC * (DK > DV ? DK : DV);  // q, then V
    static constexpr int A = LG + kC * DK, X = A + kC * kC;
    static constexpr int TOT = X + kC * kC, BETA = TOT + kNB * DK, INV = BETA + kC, WIDE = INV + kC;
    static constexpr size_t bytes = (size_t)(WIDE + kNB) * 4;
};

// k^_t or q_t times exp(LG_t - ref): rows of the left factor of a block product.
template <int DK>
struct OpLeft {
    const float *x, *lg, *ref;  // ref: the block's middle row values, or null (0)
    __device__ __forceinline__ void load(int m0, int k0, int g, int t, float &x0, float &x1) const
    {
        const tile::Op<DK, false> ox{x}, ol{lg};
        float l0, l1;
        ox.load(m0, k0, g, t, x0, x1);
        ol.load(m0, k0, g, t, l0, l1);
        if (ref) l0 -= ref[k0 + t], l1 -= ref[k0 + t + 4];
        x0 *= expf(l0);
        x1 *= expf(l1);
    }
};

// A block (I, J), I >= J, of P and M: rows 16 I .., columns 16 J ..
template <int DK>
__device__ __forceinline__ void pair_block(const Gates<DK> &G, int I, int J, float *mid, float *A, float *M)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    float p[1][2][4], m[1][2][4];
    tile::zero(p);
    tile::zero(m);
    if (I == J && G.wide[I]) {
        // a channel's decay may not be split into two factors: pair by pair, lanes over channels
        for (int i = 0; i < kSub; ++i)
            for (int s = i; s < kSub; ++s) {
                const int ri = I * kSub + i, rs = I * kSub + s;
                float kk = 0.f, kq = 0.f;
                for (int d = lane; d < DK; d += 32) {
                    const float e = G.kh[tile::at<DK>(ri, d)] * expf(G.lg[tile::at<DK>(rs, d)] - G.lg[tile::at<DK>(ri, d)]);
                    kk = fmaf(e, G.kh[tile::at<DK>(rs, d)], kk);
                    kq = fmaf(e, G.qs[tile::at<DK>(rs, d)], kq);
                }
                kk = warp_sum(kk);
                kq = warp_sum(kq);
                const int e = (s >> 3) * 2 + (i & 1);
                if (g == (s & 7) && t == ((i & 7) >> 1)) {
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            if (j == (i >> 3) && x == e) p[0][j][x] = kk, m[0][j][x] = kq;
                }
            }
    } else {
        // the right factor's reference: the middle row of the block, or the end of block I - 1
        const float *ref = nullptr;
        if (I == J) {
            for (int d = lane; d < DK; d += 32) mid[d] = G.lg[tile::at<DK>(I * kSub + kSub / 2 - 1, d)];
            __syncwarp();
            ref = mid;
        } else {
            for (int d = lane; d < DK; d += 32) mid[d] = between<DK>(G.tot, J + 1, I, d);
            __syncwarp();
        }
        const OpLeft<DK> OK{G.kh, G.lg, ref}, OQ{G.qs, G.lg, ref};
        struct Right {
            const float *kh, *lg, *mid, *tot;
            __device__ __forceinline__ void load(int n0, int k0, int g, int t, float &x0, float &x1) const
            {
                const tile::Op<DK, false> ox{kh}, ol{lg};
                float l0, l1;
                ox.load(n0, k0, g, t, x0, x1);
                ol.load(n0, k0, g, t, l0, l1);
                if (tot) {
                    l0 = (tot[k0 + t] - l0) + mid[k0 + t];
                    l1 = (tot[k0 + t + 4] - l1) + mid[k0 + t + 4];
                } else {
                    l0 = mid[k0 + t] - l0;
                    l1 = mid[k0 + t + 4] - l1;
                }
                x0 *= expf(l0);
                x1 *= expf(l1);
            }
        };
        const Right R{G.kh, G.lg, mid, I == J ? nullptr : G.tot + J * DK};
        tile::mma<1, 2>(p, OK, I * kSub, R, J * kSub, 0, DK);
        tile::mma<1, 2>(m, OQ, I * kSub, R, J * kSub, 0, DK);
        __syncwarp();
    }
    tile::each(p, I * kSub, J * kSub, [&](int r, int c, float x, float y) {
        const float b = G.beta[r];
        *reinterpret_cast<float2 *>(A + tile::at<kC>(r, c)) = make_float2(c < r ? b * x : 0.f, c + 1 < r ? b * y : 0.f);
    });
    tile::each(m, I * kSub, J * kSub, [&](int r, int c, float x, float y) {
        *reinterpret_cast<float2 *>(M + tile::at<kC>(r, c)) = make_float2(c <= r ? x : 0.f, c + 1 <= r ? y : 0.f);
    });
}

// X = (I + A)^-1 for the unit lower triangular I + A, by blocks of 16.
__device__ __forceinline__ void invert(const float *A, float *X)
{
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (warp < kNB) {  // the diagonal blocks by forward substitution, a lane per column
        const int b0 = warp * kSub;
        float x[kSub];
        if (lane < kSub) {
#pragma unroll
            for (int r = 0; r < kSub; ++r) {
                float s = r == lane ? 1.f : 0.f;
#pragma unroll
                for (int i = 0; i < r; ++i) s = fmaf(-A[tile::at<kC>(b0 + r, b0 + i)], x[i], s);
                x[r] = s;
            }
#pragma unroll
            for (int r = 0; r < kSub; ++r) X[tile::at<kC>(b0 + r, b0 + lane)] = x[r];
        }
    }
    for (int e = tid; e < kC * kC; e += kThreads) {
        const int r = e / kC, c = e % kC;
        if (c / kSub > r / kSub) X[tile::at<kC>(r, c)] = 0.f;
    }
    __syncthreads();
    // X_IJ = -X_II sum_{J <= K < I} A_IK X_KJ, the blocks of one distance I - J at a time
    for (int dist = 1; dist < kNB; ++dist) {
        const int n = kNB - dist;
        // the inner sums first, into the place of X_IJ: thread (block, row, column)
        for (int e = tid; e < n * kSub * kSub; e += kThreads) {
            const int J = e / (kSub * kSub), r = (e / kSub) % kSub, c = e % kSub, I = J + dist;
            float s = 0.f;
            for (int k = J * kSub; k < I * kSub; ++k)
                s = fmaf(A[tile::at<kC>(I * kSub + r, k)], X[tile::at<kC>(k, J * kSub + c)], s);
            X[tile::at<kC>(I * kSub + r, J * kSub + c)] = s;
        }
        __syncthreads();
        // then -X_II times them, a thread per column and block, from the last row up
        for (int e = tid; e < n * kSub; e += kThreads) {
            const int J = e / kSub, c = e % kSub, I = J + dist;
            float x[kSub];
#pragma unroll
            for (int r = 0; r < kSub; ++r) x[r] = X[tile::at<kC>(I * kSub + r, J * kSub + c)];
#pragma unroll
            for (int r = 0; r < kSub; ++r) {
                float s = 0.f;
#pragma unroll
                for (int i = 0; i <= r; ++i) s = fmaf(-X[tile::at<kC>(I * kSub + r, I * kSub + i)], x[i], s);
                X[tile::at<kC>(I * kSub + r, J * kSub + c)] = s;
            }
        }
        __syncthreads();
    }
}

template <int DK, int DV, typename T>
__global__ void __launch_bounds__(kThreads) k_scan_prep(Args a)
{
    extern __shared__ __align__(128) float sm[];
    using L = PrepSmem<DK, DV>;
    const int h = blockIdx.x % a.nh, ci = blockIdx.x / a.nh, tid = threadIdx.x, warp = tid >> 5;
    Chunk c;
    if (!locate(a, ci, &c)) return;
    const Gates<DK> G{sm + L::KH, sm + L::QS, sm + L::LG, sm + L::TOT, sm + L::BETA, sm + L::INV,
                      reinterpret_cast<int *>(sm + L::WIDE)};
    float *A = sm + L::A, *X = sm + L::X;
    const size_t slot = (size_t)ci * a.nh + h;
    load_gates<DK, T>(a, c, h, G);
    // P (scaled by beta, into A) and M, block by block; each warp's scratch row is in X, which is free
    float *M = a.m + slot * kC * kC;
    constexpr int kPairs = kNB * (kNB + 1) / 2;
    for (int p = warp; p < kPairs; p += kThreads / 32) {
        int I = 0, J = p;
        while (J > I) J -= ++I;
        pair_block<DK>(G, I, J, X + warp * DK, A, M);
    }
    for (int e = tid; e < kC * kC; e += kThreads) {
        const int r = e / kC, col = e % kC;
        if (col / kSub > r / kSub) M[tile::at<kC>(r, col)] = 0.f;
    }
    __syncthreads();
    invert(A, X);
    // g q and W to the workspace, beta g k^ in place of k^
    for (int e = tid; e < kC * DK; e += kThreads) {
        const int r = e / DK, d = e % DK, I = r / kSub, p = tile::at<DK>(r, d);
        const float l = G.lg[p], g = expf(l + between<DK>(G.tot, 0, I, d));
        const float w = expf((G.tot[I * DK + d] - l) + between<DK>(G.tot, I + 1, kNB, d));
        a.qb[slot * kC * DK + p] = G.qs[p] * g;
        a.w[slot * kC * DK + p] = G.kh[p] * w;
        G.kh[p] *= g * G.beta[r];
    }
    for (int d = tid; d < DK; d += kThreads) a.gc[slot * DK + d] = expf(between<DK>(G.tot, 0, kNB, d));
    if (a.x)
        for (int e = tid; e < kC * kC; e += kThreads) a.x[slot * kC * kC + e] = X[e];
    __syncthreads();  // q has been read: V takes its place
    load_tile<DV>(G.qs, static_cast<const T *>(a.v) + (long long)h * DV, a.ldv, c, [](float x) { return x; });
    __syncthreads();
    for (int e = tid; e < kC * DV; e += kThreads) G.qs[e] *= G.beta[e / DV];
    __syncthreads();
    // Kx = X (beta g k^), Uv = X (beta V): a warp takes DK / 8 (DV / 8) columns of all rows
    const tile::Op<kC, false> OX{X};
    {
        constexpr int NT = DK / 64;
        const tile::Op<DK, true> B{G.kh};
        float *out = a.kx + slot * kC * DK;
#pragma unroll
        for (int I = 0; I < kNB; ++I) {
            float acc[1][NT][4];
            tile::zero(acc);
            tile::mma<1, NT>(acc, OX, I * kSub, B, warp * (DK / 8), 0, (I + 1) * kSub);
            tile::each(acc, I * kSub, warp * (DK / 8),
                       [&](int r, int col, float x, float y) { store2(out + tile::at<DK>(r, col), x, y); });
        }
    }
    {
        constexpr int NT = DV / 64;
        const tile::Op<DV, true> B{G.qs};
        float *out = a.u + slot * kC * DV;
#pragma unroll
        for (int I = 0; I < kNB; ++I) {
            float acc[1][NT][4];
            tile::zero(acc);
            tile::mma<1, NT>(acc, OX, I * kSub, B, warp * (DV / 8), 0, (I + 1) * kSub);
            tile::each(acc, I * kSub, warp * (DV / 8),
                       [&](int r, int col, float x, float y) { store2(out + tile::at<DV>(r, col), x, y); });
        }
    }
}

// ---------------------------------------------------------------- the states, chunk by chunk

// Forward:   T = Uv - Kx S,      S <- g_C S + W^T T       (h: S before each chunk; u: T)
// Backward:  T = du + W dS',     dS <- g_C dS' + gh - Kx^T T    (gh: dS' of each chunk; du: T)
// One block per head, sequence and slice of VS value columns.  The state's slice stays in the
// warps' accumulators (warp w: rows w DK / 8 ..) and, for the first product, in shared memory; the
// next chunk's two factors are copied in while a chunk is computed.
constexpr int kSlice = 32;

template <int DK>
struct StateSmem {
    static constexpr int F = 2 * kC * DK;  // one chunk's two factors
    static constexpr int S = 2 * F, T = S + DK * kSlice;
    static constexpr size_t bytes = (size_t)(T + kC * kSlice) * 4;
};

template <int DK, int DV, bool BWD>
__global__ void __launch_bounds__(kThreads) k_scan_state(Args a)
{
    extern __shared__ __align__(128) float sm[];
    using L = StateSmem<DK>;
    const int h = blockIdx.x / (DV / kSlice), col0 = (blockIdx.x % (DV / kSlice)) * kSlice, s = blockIdx.y;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int c0 = seq_chunk0(a, s);
    const int nc = a.cu ? a.pre[s + 1] - c0 : (a.tokens + kC - 1) / kC;
    float *S = sm + L::S, *Tm = sm + L::T;
    const float *src = BWD ? a.gstate : a.state0;
    float *dst = BWD ? a.dstate0 : a.state_out;
    const size_t so = ((size_t)s * a.nh + h) * DK * DV + col0;
    // state tiling: 16 x 8 accumulator tiles; with dk 64 two warps share 16 rows and split the columns
    constexpr int NT = DK == 128 ? kSlice / 8 : kSlice / 16;
    const int m0 = DK == 128 ? warp * 16 : (warp >> 1) * 16, n0 = DK == 128 ? 0 : (warp & 1) * (kSlice / 2);
    float acc[1][NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
            float2 x = make_float2(0.f, 0.f);
            if (src) x = *reinterpret_cast<const float2 *>(src + so + (size_t)(m0 + g + 4 * e) * DV + n0 + 8 * j + 2 * t);
            acc[0][j][e] = x.x;
            acc[0][j][e + 1] = x.y;
        }
    auto put_state = [&](int ci) {  // the state to shared memory and to its place in the workspace
        float *out = (BWD ? a.gh : a.h) + ((size_t)ci * a.nh + h) * DK * DV;
        tile::each(acc, m0, n0, [&](int r, int c, float x, float y) {
            *reinterpret_cast<float2 *>(S + tile::at<kSlice>(r, c)) = make_float2(x, y);
            *reinterpret_cast<float2 *>(out + tile::at<DV>(r, col0 + c)) = make_float2(x, y);
        });
    };
    auto fetch = [&](int i) {  // factors of the i-th chunk in the order of this pass
        if (i < nc) {
            const size_t slot = (size_t)(c0 + (BWD ? nc - 1 - i : i)) * a.nh + h;
            float *F = sm + (i & 1) * L::F;
            tile::copy_async<kThreads>(F, a.kx + slot * kC * DK, kC * DK);
            tile::copy_async<kThreads>(F + kC * DK, a.w + slot * kC * DK, kC * DK);
        }
        tile::cp_commit();
    };
    fetch(0);
    for (int i = 0; i < nc; ++i) {
        const int ci = c0 + (BWD ? nc - 1 - i : i);
        const size_t slot = (size_t)ci * a.nh + h;
        fetch(i + 1);
        const float *F = sm + (i & 1) * L::F;
        const float *A1 = BWD ? F + kC * DK : F, *A2 = BWD ? F : F + kC * DK;
        // T's accumulators start from du, or -Uv
        const int tm = (warp >> 1) * 16, tn = (warp & 1) * (kSlice / 2);
        float *U = (BWD ? a.du : a.u) + slot * kC * DV;
        float ta[1][2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                const float2 x = *reinterpret_cast<const float2 *>(
                    U + tile::at<DV>(tm + g + 4 * e, col0 + tn + 8 * j + 2 * t));
                ta[0][j][e] = BWD ? x.x : -x.x;
                ta[0][j][e + 1] = BWD ? x.y : -x.y;
            }
        float add[NT][4];  // (g q)^T do
        float gr[2];
        gr[0] = a.gc[slot * DK + m0 + g];
        gr[1] = a.gc[slot * DK + m0 + g + 8];
        if (BWD) {
            const float *C2 = a.gh + slot * DK * DV;
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    const float2 x = *reinterpret_cast<const float2 *>(
                        C2 + tile::at<DV>(m0 + g + 4 * e, col0 + n0 + 8 * j + 2 * t));
                    add[j][e] = x.x;
                    add[j][e + 1] = x.y;
                }
        }
        put_state(ci);
        tile::cp_wait<1>();
        __syncthreads();
        tile::mma<1, 2>(ta, tile::Op<DK, false>{A1}, tm, tile::Op<kSlice, true>{S}, tn, 0, DK);
        tile::each(ta, tm, tn, [&](int r, int c, float x, float y) {
            // forward: U = -acc; backward: dU = acc, and -dU is what the second product takes
            *reinterpret_cast<float2 *>(Tm + tile::at<kSlice>(r, c)) = make_float2(-x, -y);
            *reinterpret_cast<float2 *>(U + tile::at<DV>(r, col0 + c)) = BWD ? make_float2(x, y) : make_float2(-x, -y);
        });
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[0][j][e] = fmaf(gr[e >> 1], acc[0][j][e], BWD ? add[j][e] : 0.f);
        __syncthreads();
        tile::mma<1, NT>(acc, tile::Op<DK, true>{A2}, m0, tile::Op<kSlice, true>{Tm}, n0, 0, kC);
        __syncthreads();  // S, T and the factors of this chunk are free
    }
    tile::cp_wait<0>();
    if (dst)
        tile::each(acc, m0, n0, [&](int r, int c, float x, float y) {
            *reinterpret_cast<float2 *>(dst + so + (size_t)r * DV + c) = make_float2(x, y);
        });
}

// ---------------------------------------------------------------- outputs

template <int DK, int DV>
struct OutSmem {
    static constexpr int QB = 0, S = QB + kC * DK, U = S + DK * DV, M = U + kC * DV;
    static constexpr size_t bytes = (size_t)(M + kC * kC) * 4;
};

template <int DK, int DV, typename T>
__global__ void __launch_bounds__(kThreads) k_scan_out(Args a)
{
    extern __shared__ __align__(128) float sm[];
    using L = OutSmem<DK, DV>;
    const int h = blockIdx.x % a.nh, ci = blockIdx.x / a.nh, warp = threadIdx.x >> 5;
    Chunk c;
    if (!locate(a, ci, &c)) return;
    const size_t slot = (size_t)ci * a.nh + h;
    tile::copy_async<kThreads>(sm + L::QB, a.qb + slot * kC * DK, kC * DK);
    tile::copy_async<kThreads>(sm + L::S, a.h + slot * DK * DV, DK * DV);
    tile::copy_async<kThreads>(sm + L::U, a.u + slot * kC * DV, kC * DV);
    tile::copy_async<kThreads>(sm + L::M, a.m + slot * kC * kC, kC * kC);
    tile::cp_commit();
    tile::cp_wait<0>();
    __syncthreads();
    constexpr int NT = DV / 64;
    const int n0 = warp * (DV / 8);
    float acc[kNB][NT][4];
    tile::zero(acc);
    tile::mma<kNB, NT>(acc, tile::Op<DK, false>{sm + L::QB}, 0, tile::Op<DV, true>{sm + L::S}, n0, 0, DK);
    tile::mma<kNB, NT>(acc, tile::Op<kC, false>{sm + L::M}, 0, tile::Op<DV, true>{sm + L::U}, n0, 0, kC);
    T *o = static_cast<T *>(a.o) + ((size_t)c.row0 * a.nh + h) * DV;
    tile::each(acc, 0, n0, [&](int r, int col, float x, float y) {
        if (r < c.n) store2(o + (size_t)r * a.nh * DV + col, x, y);
    });
}

// ---------------------------------------------------------------- token by token

// One block per sequence and head: the whole state in registers, warp w the rows w DK / 8 .., lane l
// the columns l DV / 32 ..  Per token: p = k^^T diag(alpha) S (summed over the warps through shared
// memory), u = beta (v - p), S = diag(alpha) S + k^ u^T, o = q^T S.
template <int DK, int DV, typename T>
__global__ void __launch_bounds__(kThreads) k_scan_tokens(Args a)
{
    constexpr int R = DK / 8, CV = DV / 32;
    __shared__ float kq[3][DK];        // k, then k^; q; alpha
    __shared__ float part[8][DV], norm[8];
    const int h = blockIdx.x, s = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const long long r0 = seq_start(a, s), r1 = seq_end(a, s);
    const size_t so = ((size_t)s * a.nh + h) * DK * DV;
    float S[R][CV];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const float *p = a.state0 + so + (size_t)(warp * R + r) * DV + lane * CV;
#pragma unroll
        for (int j = 0; j < CV; ++j) S[r][j] = 0.f;
        if (a.state0) {
            if (CV == 4) {
                const float4 x = *reinterpret_cast<const float4 *>(p);
                S[r][0] = x.x, S[r][1] = x.y, S[r][CV - 2] = x.z, S[r][CV - 1] = x.w;
            } else {
                const float2 x = *reinterpret_cast<const float2 *>(p);
                S[r][0] = x.x, S[r][1] = x.y;
            }
        }
    }
    for (long long row = r0; row < r1; ++row) {
        float kv = 0.f;
        if (tid < DK) {
            kv = to_f(static_cast<const T *>(a.k)[row * a.ldk + h * DK + tid]);
            kq[0][tid] = kv;
            kq[1][tid] = to_f(static_cast<const T *>(a.q)[row * a.ldq + h * DK + tid]);
            kq[2][tid] = expf(log_alpha(to_f(static_cast<const T *>(a.z)[row * a.ldz + h * DK + tid])));
        }
        const float ss = warp_sum(kv * kv);
        if (lane == 0) norm[warp] = ss;
        const float beta = sigmoid(to_f(static_cast<const T *>(a.b)[row * a.ldb + h]));
        float v[CV];
#pragma unroll
        for (int j = 0; j < CV; ++j) v[j] = to_f(static_cast<const T *>(a.v)[row * a.ldv + h * DV + lane * CV + j]);
        __syncthreads();
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) sum += norm[w];
        const float inv = sum > 0.f ? 1.f / sqrtf(sum) : 0.f;
        float kh[R], p[CV];
#pragma unroll
        for (int j = 0; j < CV; ++j) p[j] = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            kh[r] = kq[0][warp * R + r] * inv;
            const float al = kq[2][warp * R + r];
#pragma unroll
            for (int j = 0; j < CV; ++j) {
                S[r][j] *= al;
                p[j] = fmaf(kh[r], S[r][j], p[j]);
            }
        }
#pragma unroll
        for (int j = 0; j < CV; ++j) part[warp][lane * CV + j] = p[j];
        __syncthreads();
        float u[CV], o[CV];
#pragma unroll
        for (int j = 0; j < CV; ++j) {
            float x = 0.f;
#pragma unroll
            for (int w = 0; w < 8; ++w) x += part[w][lane * CV + j];
            u[j] = beta * (v[j] - x);
            o[j] = 0.f;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float qv = kq[1][warp * R + r];
#pragma unroll
            for (int j = 0; j < CV; ++j) {
                S[r][j] = fmaf(kh[r], u[j], S[r][j]);
                o[j] = fmaf(qv, S[r][j], o[j]);
            }
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < CV; ++j) part[warp][lane * CV + j] = o[j];
        __syncthreads();
        if (tid < DV) {
            float x = 0.f;
#pragma unroll
            for (int w = 0; w < 8; ++w) x += part[w][tid];
            store1(static_cast<T *>(a.o) + ((size_t)row * a.nh + h) * DV + tid, x);
        }
        __syncthreads();
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float *p = a.state_out + so + (size_t)(warp * R + r) * DV + lane * CV;
        if (CV == 4)
            *reinterpret_cast<float4 *>(p) = make_float4(S[r][0], S[r][1], S[r][CV - 2], S[r][CV - 1]);
        else
            *reinterpret_cast<float2 *>(p) = make_float2(S[r][0], S[r][1]);
    }
}

template <class K>
cudaError_t allow_smem(K kernel, size_t bytes)
{
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <int DK, int DV, typename T>
cudaError_t forward_chunks(const Args &a, bool out, cudaStream_t st)
{
    cudaError_t e = allow_smem(k_scan_prep<DK, DV, T>, PrepSmem<DK, DV>::bytes);
    if (e == cudaSuccess) e = allow_smem(k_scan_state<DK, DV, false>, StateSmem<DK>::bytes);
    if (e == cudaSuccess) e = allow_smem(k_scan_out<DK, DV, T>, OutSmem<DK, DV>::bytes);
    if (e != cudaSuccess) return e;
    if (a.cu) k_scan_plan<<<1, 1024, 0, st>>>(a, const_cast<int *>(a.pre));
    const unsigned grid = (unsigned)a.nh * a.max_chunks;
    if (grid) k_scan_prep<DK, DV, T><<<grid, kThreads, PrepSmem<DK, DV>::bytes, st>>>(a);
    k_scan_state<DK, DV, false><<<dim3(a.nh * (DV / kSlice), a.nseq), kThreads, StateSmem<DK>::bytes, st>>>(a);
    if (out && grid) k_scan_out<DK, DV, T><<<grid, kThreads, OutSmem<DK, DV>::bytes, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

template <int DK, int DV, typename T>
cudaError_t forward(const Args &a, bool out, cudaStream_t st)
{
    return forward_chunks<DK, DV, T>(a, out, st);
}

template <int DK, int DV, typename T>
cudaError_t tokens(const Args &a, cudaStream_t st)
{
    k_scan_tokens<DK, DV, T><<<dim3(a.nh, a.nseq), kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

template <int DK, int DV>
cudaError_t reverse(const Args &a, cudaStream_t st)
{
    cudaError_t e = allow_smem(k_scan_state<DK, DV, true>, StateSmem<DK>::bytes);
    if (e != cudaSuccess) return e;
    k_scan_state<DK, DV, true><<<dim3(a.nh * (DV / kSlice), a.nseq), kThreads, StateSmem<DK>::bytes, st>>>(a);
    return cudaGetLastError();
}

#define KDA_SCAN_T(DK, DV, T)                                              \
    template cudaError_t forward<DK, DV, T>(const Args &, bool, cudaStream_t); \
    template cudaError_t tokens<DK, DV, T>(const Args &, cudaStream_t);
#define KDA_SCAN(DK, DV)                                        \
    KDA_SCAN_T(DK, DV, float)                                   \
    KDA_SCAN_T(DK, DV, __nv_bfloat16)                           \
    template cudaError_t reverse<DK, DV>(const Args &, cudaStream_t);
KDA_SCAN(64, 64)
KDA_SCAN(64, 128)
KDA_SCAN(128, 64)
KDA_SCAN(128, 128)

}  // namespace scan
}  // namespace kda
