// scan_grad.cu -- the recurrence over whole sequences: backward (forward and notation: scan.cuh).
//
// The chunks' states and U are computed again, then, with dS' the gradient of the state after a
// chunk and do that of its outputs, from the last chunk to the first
//   dU = M^T do + W dS',     dS = g_C dS' + (g q)^T do - Kx^T dU            (k_scan_state, reversed)
// and for every chunk at once
//   G = X^T dU,  dv = beta G,  db_t = (1 - beta_t) G_t . U_t     (u_t = beta_t (v_t - ..), so the
//                                                 derivative by beta needs no division by beta)
//   dM = do U^T (i <= t),  dP = -beta G U^T (i < t),
//   D1 = do S^T,  D2 = -dv S^T,  D3 = U dS'^T                  (gradients of g q, g k^ and W)
//   dq_t  = g_t D1_t + sum_i dM[t, i] gamma(t, i) k^_i
//   dk^_t = g_t D2_t + sum_i dP[t, i] gamma(t, i) k^_i                               ("row" part)
//         + gamma(C, t) D3_t + sum_{j > t} (dP[j, t] k^_j + dM[j, t] q_j) gamma(j, t)  ("column")
// A decay alpha_t stands in gamma(j, i) for i < t <= j, so its logarithm's gradient is, per channel,
//   dla_t = sum_{j >= t} (q_j dq_j + k^_j dk^row_j - k^_j dk^col_j) + sum_{j < t} W_j D3_j + g_C (S . dS')
// with the column part here without D3 and the pairs j = i (which no decay touches) left out.
// dz = -sigmoid(z) dla, dk = (dk^ - k^ (k^ . dk^)) / |k| (0 for a zero key).
#include "scan_prep.cuh"

namespace kda {
namespace scan {
namespace {

// ---------------------------------------------------------------- fp32: three TF32 products of fp32 tiles

constexpr float kFloor = kFloor2 * 0.693147181f;
constexpr float kRange = 60.f;  // largest decay inside a block that the block's middle can anchor
__device__ __forceinline__ float log_alpha(float z)
{
    const float lz = -(fmaxf(z, 0.f) + log1pf(expf(-fabsf(z))));
    return lz < kFloor ? kFloor : lz;  // keeps a NaN
}

// What the chunk's keys, queries and gates give, in shared memory.
template <int DK>
struct Gates {
    float *kh;    // tile [kC][DK]: k^
    float *qs;    // tile [kC][DK]: q
    float *lg;    // tile [kC][DK]: sums of la inside the blocks
    float *tot;   // [kNB][DK]: the blocks' totals
    float *beta;  // [kC]
    float *inv;   // [kC]: 1 / |k|, or 0
    int *wide;    // [kNB]: a channel decays by more than kRange inside the block
};

template <int DK, typename T>
__device__ __forceinline__ void load_gates(const Args &a, const Chunk &c, int h, const Gates<DK> &G)
{
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    load_tile<DK>(G.kh, static_cast<const T *>(a.k) + (long long)h * DK, a.ldk, c, [](float x) { return x; });
    load_tile<DK>(G.qs, static_cast<const T *>(a.q) + (long long)h * DK, a.ldq, c, [](float x) { return x; });
    load_tile<DK>(G.lg, static_cast<const T *>(a.z) + (long long)h * DK, a.ldz, c, [](float x) { return log_alpha(x); });
    if (tid < kC) G.beta[tid] = tid < c.n ? sigmoid(to_f(static_cast<const T *>(a.b)[(c.row0 + tid) * a.ldb + h])) : 0.f;
    if (tid < kNB) G.wide[tid] = 0;
    __syncthreads();
    for (int r = warp; r < kC; r += kThreads / 32) {
        float x[DK / 32], ss = 0.f;
#pragma unroll
        for (int i = 0; i < DK / 32; ++i) {
            x[i] = G.kh[tile::at<DK>(r, lane + 32 * i)];
            ss = fmaf(x[i], x[i], ss);
        }
        ss = warp_sum(ss);
        const float inv = ss > 0.f ? 1.f / sqrtf(ss) : 0.f;
#pragma unroll
        for (int i = 0; i < DK / 32; ++i) G.kh[tile::at<DK>(r, lane + 32 * i)] = x[i] * inv;
        if (lane == 0) G.inv[r] = inv;
    }
    for (int e = tid; e < kNB * DK; e += kThreads) {
        const int I = e / DK, d = e % DK;
        float s = 0.f, first = 0.f;
#pragma unroll
        for (int t = 0; t < kSub; ++t) {
            float *p = G.lg + tile::at<DK>(I * kSub + t, d);
            s += *p;
            *p = s;
            if (t == 0) first = s;
        }
        G.tot[I * DK + d] = s;
        if (first - s > kRange) G.wide[I] = 1;
    }
    __syncthreads();
}

// Sum of the totals of blocks [I, J) of channel d.
template <int DK>
__device__ __forceinline__ float between(const float *tot, int I, int J, int d)
{
    float s = 0.f;
    for (int K = I; K < J; ++K) s += tot[K * DK + d];
    return s;
}

template <int DK, int DV>
struct GradSmem {
    static constexpr int D = DK > DV ? DK : DV;
    static constexpr int R0 = 0, R1 = R0 + kC * D, R2 = R1 + kC * D;  // do, G, U; then k^, q, LG
    static constexpr int R3 = R2 + kC * D;                            // S, dS'; then the two terms of dla
    static constexpr int R3N = DK * DV > 2 * kC * DK ? DK * DV : 2 * kC * DK;
    static constexpr int XM = R3 + R3N, DP = XM + kC * kC;            // X, then dM; dP
    static constexpr int TOT = DP + kC * kC, BETA = TOT + kNB * DK, INV = BETA + kC, MD = INV + kC;
    static constexpr int GS = MD + kC, RD = GS + DK, WIDE = RD + 2 * kC;
    static constexpr size_t bytes = (size_t)(WIDE + kNB) * 4;
    static_assert(bytes <= 227 * 1024, "");
};

// Rows of dM (m < 16) and of dP (m >= 16) of block I.
struct OpBoth {
    const float *dm, *dp;
    int m0;
    __device__ __forceinline__ void load(int m, int k0, int g, int t, float &x0, float &x1) const
    {
        const tile::Op<kC, false> o{m < kSub ? dm : dp};
        o.load(m0 + (m & (kSub - 1)), k0, g, t, x0, x1);
    }
};

// Element (d, i) = x[i][d] exp(sign LG[i][d] + c(d, block of i)), for i along k.
template <int DK, class F>
struct OpDecayed {
    const float *x, *lg;
    float sign;
    F c;
    __device__ __forceinline__ void load(int n0, int k0, int g, int t, float &x0, float &x1) const
    {
        const tile::Op<DK, true> ox{x}, ol{lg};
        float l0, l1;
        ox.load(n0, k0, g, t, x0, x1);
        ol.load(n0, k0, g, t, l0, l1);
        x0 *= expf(c(n0 + g, k0 / kSub, sign * l0));
        x1 *= expf(c(n0 + g, k0 / kSub, sign * l1));
    }
};
template <int DK, class F>
__device__ __forceinline__ OpDecayed<DK, F> decayed(const float *x, const float *lg, float sign, F c)
{
    return OpDecayed<DK, F>{x, lg, sign, c};
}

// dz / dla.  Everything in dla_t is proportional to alpha_t, which was held at e^kFloor where it is smaller.
__device__ __forceinline__ float dz_factor(float z)
{
    const float x = exp2a(-1.44269504f * fabsf(z));
    const float s = __fdividef(z < 0.f ? -x : -1.f, 1.f + x);
    return z > -kFloor ? -exp2a(1.44269504f * (-z - kFloor)) : s;  // log alpha of a large z is -z
}

template <int DK, int DV>
__global__ void __launch_bounds__(kThreads, 1) k_grad_f32(Args a)
{
    using T = float;
    extern __shared__ __align__(128) float sm[];
    using L = GradSmem<DK, DV>;
    const int h = blockIdx.x % a.nh, ci = blockIdx.x / a.nh, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    Chunk c;
    if (!locate(a, ci, &c)) return;
    const size_t slot = (size_t)ci * a.nh + h;
    float *R0 = sm + L::R0, *R1 = sm + L::R1, *R2 = sm + L::R2, *R3 = sm + L::R3, *XM = sm + L::XM, *DP = sm + L::DP;
    float *beta = sm + L::BETA, *md = sm + L::MD, *gs = sm + L::GS, *rd = sm + L::RD;
    const long long dv0 = (c.row0 * a.nh + h) * DV, dk0 = (c.row0 * a.nh + h) * DK;  // of the dense gradients

    tile::copy_async<kThreads>(XM, static_cast<const float *>(a.x) + slot * kC * kC, kC * kC);
    tile::copy_async<kThreads>(R0, a.du + slot * kC * DV, kC * DV);
    tile::cp_commit();
    tile::copy_async<kThreads>(R2, a.u + slot * kC * DV, kC * DV);
    tile::copy_async<kThreads>(R3, static_cast<const float *>(a.h) + slot * DK * DV, DK * DV);
    tile::cp_commit();
    if (tid < kC) beta[tid] = tid < c.n ? sigmoid(to_f(static_cast<const T *>(a.b)[(c.row0 + tid) * a.ldb + h])) : 0.f;
    tile::cp_wait<1>();
    __syncthreads();
    {  // G = X^T dU
        constexpr int NT = DV / 64;
        const int n0 = warp * (DV / 8);
#pragma unroll
        for (int I = 0; I < kNB; ++I) {
            float acc[1][NT][4];
            tile::zero(acc);
            tile::mma<1, NT>(acc, tile::Op<kC, true>{XM}, I * kSub, tile::Op<kC, false>{R0}, n0, I * kSub, kC);
            tile::each(acc, I * kSub, n0, [&](int r, int col, float x, float y) { store2(R1 + tile::at<DV>(r, col), x, y); });
        }
    }
    tile::cp_wait<0>();
    __syncthreads();
    // do takes dU's place
    load_tile<DV>(R0, static_cast<const T *>(a.go) + (long long)h * DV, (long long)a.nh * DV, c, [](float x) { return x; });
    for (int r = warp; r < kC; r += kThreads / 32) {
        float s = 0.f;
        for (int e = lane; e < DV; e += 32) s = fmaf(R1[tile::at<DV>(r, e)], R2[tile::at<kC>(e, r)], s);
        s = warp_sum(s);
        if (lane == 0 && r < c.n)
            store1(static_cast<T *>(a.db) + (c.row0 + r) * a.nh + h, (1.f - beta[r]) * s);
    }
    const int I = warp >> 1, half = warp & 1, m0 = I * kSub;  // the warp's rows, and half of the columns
    {  // dP = -beta G U^T below the diagonal
        float acc[1][4][4];
        tile::zero(acc);
        const int n0 = half * (kC / 2);
        if (n0 < m0 + kSub) tile::mma<1, 4>(acc, tile::Op<DV, false>{R1}, m0, tile::Op<kC, true>{R2}, n0, 0, DV);
        tile::each(acc, m0, n0, [&](int r, int col, float x, float y) {
            store2(DP + tile::at<kC>(r, col), col < r ? -beta[r] * x : 0.f, col + 1 < r ? -beta[r] * y : 0.f);
        });
    }
    __syncthreads();  // do is there, X and G have been read
    {  // dM = do U^T below the diagonal; the diagonal apart
        float acc[1][4][4];
        tile::zero(acc);
        const int n0 = half * (kC / 2);
        if (n0 < m0 + kSub) tile::mma<1, 4>(acc, tile::Op<DV, false>{R0}, m0, tile::Op<kC, true>{R2}, n0, 0, DV);
        tile::each(acc, m0, n0, [&](int r, int col, float x, float y) {
            store2(XM + tile::at<kC>(r, col), col < r ? x : 0.f, col + 1 < r ? y : 0.f);
            if (col == r) md[r] = x;
            if (col + 1 == r) md[r] = y;
        });
    }
    // dv = beta G
    for (int e = tid; e < kC * (DV / 2); e += kThreads) {
        const int r = e / (DV / 2), col = 2 * (e % (DV / 2));
        float2 *p = reinterpret_cast<float2 *>(R1 + tile::at<DV>(r, col));
        const float2 x = *p, y = make_float2(x.x * beta[r], x.y * beta[r]);
        *p = y;
        if (r < c.n) store2(static_cast<T *>(a.dv) + dv0 + (long long)r * a.nh * DV + col, y.x, y.y);
    }
    // S . dS' per key channel
    const float *gh = a.gh + slot * DK * DV;
    for (int d = tid; d < DK; d += kThreads) {
        float s = 0.f;
#pragma unroll 8
        for (int e = 0; e < DV; ++e) s = fmaf(R3[tile::at<DK>(e, d)], gh[tile::at<DK>(e, d)], s);
        gs[d] = s;
    }
    __syncthreads();
    constexpr int NT = DK / 16;
    const int n0 = half * (DK / 2);
    float a1[1][NT][4], a2[1][NT][4], a3[1][NT][4];
    tile::zero(a1);
    tile::zero(a2);
    tile::zero(a3);
    tile::mma<1, NT>(a1, tile::Op<DV, false>{R0}, m0, tile::Op<DK, true>{R3}, n0, 0, DV);
    tile::mma<1, NT>(a2, tile::Op<DV, false>{R1}, m0, tile::Op<DK, true>{R3}, n0, 0, DV);
    __syncthreads();
    tile::copy_async<kThreads>(R3, gh, DK * DV);
    tile::cp_commit();
    tile::cp_wait<0>();
    __syncthreads();
    tile::mma<1, NT>(a3, tile::Op<kC, true>{R2}, m0, tile::Op<DK, true>{R3}, n0, 0, DV);
    __syncthreads();
    const Gates<DK> Gt{R0, R1, R2, sm + L::TOT, beta, sm + L::INV, reinterpret_cast<int *>(sm + L::WIDE)};
    load_gates<DK, T>(a, c, h, Gt);
    const float *KH = R0, *QS = R1, *LG = R2, *tot = Gt.tot;
    const bool wide = Gt.wide[I];
    const float *mid = LG + (m0 + kSub / 2 - 1) * DK;  // the block's middle row (swizzled)
    const int msw = tile::swz(m0 + kSub / 2 - 1);
    const int g = lane >> 2, t = lane & 3;
    {  // rows: dq and the row part of dk^
        float acc[2][NT][4];
        tile::zero(acc);
        const OpBoth A{XM, DP, m0};
        tile::mma<2, NT>(acc, A, 0, decayed<DK>(KH, LG, -1.f, [&](int d, int J, float l) {
                             return (tot[J * DK + d] + l) + between<DK>(tot, J + 1, I, d);
                         }), n0, 0, m0);
        if (!wide) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float x = expf(mid[(n0 + 8 * j + 2 * t + (e & 1)) ^ msw]);
                    acc[0][j][e] *= x;
                    acc[1][j][e] *= x;
                }
            tile::mma<2, NT>(acc, A, 0, decayed<DK>(KH, LG, -1.f, [&](int d, int, float l) { return mid[d ^ msw] + l; }),
                             n0, m0, m0 + kSub);
        }
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = m0 + g + 8 * (e >> 1), d = n0 + 8 * j + 2 * t + (e & 1), p = tile::at<DK>(r, d);
                const float l = LG[p], gt = expf(l + between<DK>(tot, 0, I, d));
                float x = acc[0][j][e], y = acc[1][j][e];
                const float f = expf(wide ? l : l - mid[d ^ msw]);
                x *= f;
                y *= f;
                if (wide)
                    for (int i = m0; i < r; ++i) {
                        const float k = KH[tile::at<DK>(i, d)] * expf(l - LG[tile::at<DK>(i, d)]);
                        x = fmaf(XM[tile::at<kC>(r, i)], k, x);
                        y = fmaf(DP[tile::at<kC>(r, i)], k, y);
                    }
                a1[0][j][e] = fmaf(gt, a1[0][j][e], x);
                a2[0][j][e] = fmaf(-gt, a2[0][j][e], y);
            }
    }
    tile::each(a1, m0, n0, [&](int r, int d, float x, float y) {
        const float2 k = *reinterpret_cast<const float2 *>(KH + tile::at<DK>(r, d));
        if (r < c.n)
            store2(static_cast<T *>(a.dq) + dk0 + (long long)r * a.nh * DK + d, fmaf(md[r], k.x, x), fmaf(md[r], k.y, y));
    });
    float dot[2] = {0.f, 0.f};
    {  // columns: the rest of dk^, and the terms of dla
        float acc[1][NT][4];
        tile::zero(acc);
        const tile::Op<kC, true> AP{DP}, AM{XM};
        auto later = [&](int d, int J, float l) { return between<DK>(tot, I + 1, J, d) + l; };
        tile::mma<1, NT>(acc, AP, m0, decayed<DK>(KH, LG, 1.f, later), n0, m0 + kSub, kC);
        tile::mma<1, NT>(acc, AM, m0, decayed<DK>(QS, LG, 1.f, later), n0, m0 + kSub, kC);
        if (!wide) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int d = n0 + 8 * j + 2 * t + (e & 1);
                    acc[0][j][e] *= expf(tot[I * DK + d] - mid[d ^ msw]);
                }
            auto inside = [&](int d, int, float l) { return l - mid[d ^ msw]; };
            tile::mma<1, NT>(acc, AP, m0, decayed<DK>(KH, LG, 1.f, inside), n0, m0, m0 + kSub);
            tile::mma<1, NT>(acc, AM, m0, decayed<DK>(QS, LG, 1.f, inside), n0, m0, m0 + kSub);
        }
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = m0 + g + 8 * (e >> 1), d = n0 + 8 * j + 2 * t + (e & 1), p = tile::at<DK>(r, d);
                const float l = LG[p], k = KH[p], q = QS[p], wt = tot[I * DK + d];
                float x = acc[0][j][e] * expf(wide ? wt - l : mid[d ^ msw] - l);
                if (wide)
                    for (int i = r + 1; i < m0 + kSub; ++i) {
                        const float f = expf(LG[tile::at<DK>(i, d)] - l);
                        x = fmaf(DP[tile::at<kC>(i, r)], KH[tile::at<DK>(i, d)] * f, x);
                        x = fmaf(XM[tile::at<kC>(i, r)], QS[tile::at<DK>(i, d)] * f, x);
                    }
                const float w = expf((wt - l) + between<DK>(tot, I + 1, kNB, d)) * a3[0][j][e];
                R3[p] = q * a1[0][j][e] + k * (a2[0][j][e] - x);
                R3[kC * DK + p] = k * w;
                const float dkh = a2[0][j][e] + x + w + md[r] * q;
                a2[0][j][e] = dkh;
                dot[e >> 1] = fmaf(k, dkh, dot[e >> 1]);
            }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        dot[i] += __shfl_xor_sync(0xffffffffu, dot[i], 1);
        dot[i] += __shfl_xor_sync(0xffffffffu, dot[i], 2);
        if (t == 0) rd[half * kC + m0 + g + 8 * i] = dot[i];
    }
    __syncthreads();
    tile::each(a2, m0, n0, [&](int r, int d, float x, float y) {
        const float2 k = *reinterpret_cast<const float2 *>(KH + tile::at<DK>(r, d));
        const float s = rd[r] + rd[kC + r], inv = Gt.inv[r];
        if (r < c.n)
            store2(static_cast<T *>(a.dk) + dk0 + (long long)r * a.nh * DK + d, inv * (x - k.x * s), inv * (y - k.y * s));
    });
    for (int e = tid; e < 2 * DK; e += kThreads) {
        const int d = e % DK;
        float s = 0.f;
        if (e < DK) {  // sums over j >= t
            for (int r = kC - 1; r >= 0; --r) {
                float *p = R3 + tile::at<DK>(r, d);
                s += *p;
                *p = s;
            }
        } else {  // sums over j < t, from g_C (S . dS')
            s = a.gc[slot * DK + d] * gs[d];
            for (int r = 0; r < kC; ++r) {
                float *p = R3 + kC * DK + tile::at<DK>(r, d);
                const float x = *p;
                *p = s;
                s += x;
            }
        }
    }
    __syncthreads();
    for (int e = tid; e < kC * (DK / 4); e += kThreads) {
        const int r = e / (DK / 4), d = 4 * (e % (DK / 4)), p = tile::at<DK>(r, d);
        if (r >= c.n) break;
        float z[4];
        load4(static_cast<const T *>(a.z) + (c.row0 + r) * a.ldz + (long long)h * DK + d, z);
        const float4 x = *reinterpret_cast<const float4 *>(R3 + p), y = *reinterpret_cast<const float4 *>(R3 + kC * DK + p);
        T *dz = static_cast<T *>(a.dz) + dk0 + (long long)r * a.nh * DK + d;
        store2(dz, dz_factor(z[0]) * (x.x + y.x), dz_factor(z[1]) * (x.y + y.y));
        store2(dz + 2, dz_factor(z[2]) * (x.z + y.z), dz_factor(z[3]) * (x.w + y.w));
    }
}

// ---------------------------------------------------------------- bfloat16: planes
// One block of 4 dk threads per chunk and head; warp w has the tokens of block w / (dk / 32) and a share of
// the columns.  Everything that needs value columns comes first: G, dP, dM, then D1, D2, D3, which stay in
// the accumulators, while 32 value columns of S and dS' at a time pass through shared memory.  The pairs of
// tokens of different blocks are products with k^ GL, q GL and k^ GR (the blocks between them multiplied
// into the accumulators on the way); those of one block are taken in the registers of the thread that has
// the channel's 16 tokens, going up the tokens for the rows and down for the columns, with the sums of dla
// in the same two sweeps.

template <int DK, int DV>
struct GradSmem16 {
    static constexpr int kSlab = 32;  // value columns of S and dS' at a time
    // uint16_t elements
    static constexpr int X = 0, DU = X + 2 * kC * kC;              // X, dU; then dM, dP and the diagonal blocks' (dM, dP) in fp32
    static constexpr int DM = 0, DP = DM + 2 * kC * kC, DD = DP + 2 * kC * kC;
    static constexpr int N0 = DU + 2 * kC * DV, N1 = DD + 4 * kNB * kSub * kSub;
    static constexpr int U = N0 > N1 ? N0 : N1;
    static constexpr int GO = U + 2 * kC * DV, G = GO + kC * DV;   // do, one plane; G
    static constexpr int S = G + 2 * kC * DV;                      // two slabs of S and dS'
    static constexpr int SLAB = 4 * kSlab * DK;
    static constexpr int KL = U, QL = KL + 2 * kC * DK, KR = QL + 2 * kC * DK;  // in the place of U, do, G and S
    static constexpr int RAW = KR + 2 * kC * DK;                   // k, q, z as they are
    static constexpr int R = U;                                    // fp32 tiles [kC][dk], in the planes' place
    static constexpr int R4 = DM;                                  // the fourth, in dM's and dP's
    static constexpr int E0 = S + 2 * SLAB, E1 = RAW + 3 * kC * DK;
    static constexpr int END = E0 > E1 ? E0 : E1;
    // floats
    static constexpr int TOT = END / 2, GSP = TOT + kNB * DK, SUM = GSP + 8 * DK, DOT = SUM + 2 * kNB * DK;
    static constexpr int BETA = DOT + (DK / 8) * kSub, INV = BETA + kC;
    static constexpr size_t bytes = (size_t)(INV + kC) * 4;
    static_assert(bytes <= 227 * 1024, "");
};

template <int DK, int DV>
__global__ void __launch_bounds__(4 * DK, 1) k_grad_bf16(Args a)
{
    using T = __nv_bfloat16;
    using planes::B;
    using L = GradSmem16<DK, DV>;
    extern __shared__ __align__(1024) float sm[];
    constexpr int kT = 4 * DK, WQ = DK / 32;  // threads; warps to a block of tokens
    uint16_t *p16 = reinterpret_cast<uint16_t *>(sm);
    uint16_t *GO = p16 + L::GO, *G = p16 + L::G, *U = p16 + L::U, *DM = p16 + L::DM, *DP = p16 + L::DP;
    float2 *dd = reinterpret_cast<float2 *>(p16 + L::DD);
    float *tot = sm + L::TOT, *beta = sm + L::BETA, *inv = sm + L::INV;
    const int h = blockIdx.x % a.nh, ci = blockIdx.x / a.nh, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t4 = lane & 3;
    Chunk c;
    if (!locate(a, ci, &c)) return;
    const size_t slot = (size_t)ci * a.nh + h;
    auto copy = [&](int to, const uint16_t *from, int elements) {
        tile::copy_async<kT>(reinterpret_cast<float *>(p16 + to), reinterpret_cast<const float *>(from), elements / 2);
    };
    auto fetch_slab = [&](int i) {  // value columns kSlab i .. of both planes of S and dS', by 64 channels
        if (i < DV / L::kSlab) {
            const uint16_t *s = static_cast<const uint16_t *>(a.h) + slot * 2 * DK * DV + i * L::kSlab * 64;
            const uint16_t *ds = a.ghp + slot * 2 * DK * DV + i * L::kSlab * 64;
            const int to = L::S + (i & 1) * L::SLAB;
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int b = 0; b < DK / 64; ++b) {
                    const int at = (p * (DK / 64) + b) * L::kSlab * 64, from = p * DK * DV + b * DV * 64;
                    copy(to + at, s + from, L::kSlab * 64);
                    copy(to + 2 * L::kSlab * DK + at, ds + from, L::kSlab * 64);
                }
        }
        tile::cp_commit();
    };
    copy(L::X, static_cast<const uint16_t *>(a.x) + slot * 2 * kC * kC, 2 * kC * kC);
    copy(L::DU, a.dup + slot * 2 * kC * DV, 2 * kC * DV);
    tile::cp_commit();
    copy(L::U, a.up + slot * 2 * kC * DV, 2 * kC * DV);
    for (int e = tid; e < kC * DV / 8; e += kT) {
        const int r = e / (DV / 8), c8 = 8 * (e % (DV / 8));
        uint16_t *to = GO + planes::at<kC>(r, c8);
        if (r < c.n) tile::cp_async16(to, static_cast<const T *>(a.go) + ((c.row0 + r) * a.nh + h) * DV + c8);
        else *reinterpret_cast<uint4 *>(to) = make_uint4(0, 0, 0, 0);
    }
    tile::cp_commit();
    fetch_slab(0);
    fetch_slab(1);
    if (tid < kC) {
        beta[tid] = tid < c.n ? sigmoid(to_f(static_cast<const T *>(a.b)[(c.row0 + tid) * a.ldb + h])) : 0.f;
        inv[tid] = a.inv[slot * kC + tid];
    }
    tile::cp_wait<3>();
    __syncthreads();
    const int I = warp / WQ, part = warp % WQ, m0 = I * kSub;  // the warp's tokens, and its share of the columns
    {  // G = X^T dU, dv = beta G
        constexpr int NT = DV / WQ / 8;
        const int n0 = part * (DV / WQ);
        float acc[NT][4];
        zero(acc);
        for (int k = m0; k < kC; k += 16)
            mma_step<B, false, kC, true, DV, false, NT>(acc, p16 + L::X, kC * kC, m0, k, p16 + L::DU, kC * DV, n0, k);
        T *dv = static_cast<T *>(a.dv) + (c.row0 * a.nh + h) * DV;
        each(acc, m0, n0, [&](int r, int col, float x, float y) {
            planes::put2<B, kC>(G, kC * DV, r, col, x, y);
            if (r < c.n) store2(dv + (long long)r * a.nh * DV + col, beta[r] * x, beta[r] * y);
        });
    }
    tile::cp_wait<2>();
    __syncthreads();  // X and dU are free
    {  // dM = do U^T, dP = -beta G U^T, up to the diagonal
        constexpr int NT = kC / WQ / 8;
        float am[NT][4], ap[NT][4];
        zero(am);
        zero(ap);
        const int n0 = part * (kC / WQ);
        if (n0 <= m0)
#pragma unroll 2
            for (int k = 0; k < DV; k += 16) {
                uint32_t d[4], gh[4], gl[4];
                planes::frag_a<kC, false>(d, GO, m0, k);
                planes::frag_a<kC, false>(gh, G, m0, k);
                planes::frag_a<kC, false>(gl, G + kC * DV, m0, k);
#pragma unroll
                for (int j = 0; j < NT; j += 2) {
                    uint32_t uh[4], ul[4];
                    planes::frag_b<DV, true>(uh, U, n0 + 8 * j, k);
                    planes::frag_b<DV, true>(ul, U + kC * DV, n0 + 8 * j, k);
                    B::mma(am[j], d, ul[0], ul[1]);
                    B::mma(am[j + 1], d, ul[2], ul[3]);
                    planes::mma3<B>(ap[j], ap[j + 1], gh, gl, uh, ul);
                    B::mma(am[j], d, uh[0], uh[1]);
                    B::mma(am[j + 1], d, uh[2], uh[3]);
                }
            }
        each(am, m0, n0, [&](int r, int col, float x, float y) {
            if (col < m0) {
                planes::put2<B, kC>(DM, kC * kC, r, col, x, y);
            } else if (col < m0 + kSub) {
                float2 *p = dd + (I * kSub + (r - m0)) * kSub + col - m0;
                p[0].x = col <= r ? x : 0.f;
                p[1].x = col + 1 <= r ? y : 0.f;
            }
        });
        each(ap, m0, n0, [&](int r, int col, float x, float y) {
            const float b = beta[r];
            if (col < m0) {
                planes::put2<B, kC>(DP, kC * kC, r, col, -b * x, -b * y);
            } else if (col < m0 + kSub) {
                float2 *p = dd + (I * kSub + (r - m0)) * kSub + col - m0;
                p[0].y = col < r ? -b * x : 0.f;
                p[1].y = col + 1 < r ? -b * y : 0.f;
                if ((col == r || col + 1 == r) && r < c.n)  // G_t . U_t
                    store1(static_cast<T *>(a.db) + (c.row0 + r) * a.nh + h, (1.f - b) * (col == r ? x : y));
            }
        });
    }
    const int n0 = part * 32;  // the warp's key channels
    float a1[4][4], a2[4][4], a3[4][4];
    zero(a1);
    zero(a2);
    zero(a3);
    {  // D1 = do S^T, G S^T, D3 = U dS'^T; and S . dS' per channel: two channels, an eighth of a slab's rows
        float x = 0.f, y = 0.f;
        const int cp = tid % (DK / 2), rg = tid / (DK / 2);
#pragma unroll 1
        for (int i = 0; i < DV / L::kSlab; ++i) {
            tile::cp_wait<1>();
            __syncthreads();
            const uint16_t *s = p16 + L::S + (i & 1) * L::SLAB, *ds = s + 2 * L::kSlab * DK;
#pragma unroll
            for (int r = 0; r < L::kSlab / 8; ++r) {
                const int e = planes::at<L::kSlab>(rg * (L::kSlab / 8) + r, 2 * cp);
                const float2 s0 = B::unpack(*reinterpret_cast<const uint32_t *>(s + e));
                const float2 s1 = B::unpack(*reinterpret_cast<const uint32_t *>(s + L::kSlab * DK + e));
                const float2 d0 = B::unpack(*reinterpret_cast<const uint32_t *>(ds + e));
                const float2 d1 = B::unpack(*reinterpret_cast<const uint32_t *>(ds + L::kSlab * DK + e));
                x = fmaf(s0.x + s1.x, d0.x + d1.x, x);
                y = fmaf(s0.y + s1.y, d0.y + d1.y, y);
            }
#pragma unroll
            for (int kk = 0; kk < L::kSlab; kk += 16) {
                const int k = i * L::kSlab + kk;
                uint32_t d[4], gh[4], gl[4], uh[4], ul[4];
                planes::frag_a<kC, false>(d, GO, m0, k);
                planes::frag_a<kC, false>(gh, G, m0, k);
                planes::frag_a<kC, false>(gl, G + kC * DV, m0, k);
                planes::frag_a<DV, true>(uh, U, m0, k);
                planes::frag_a<DV, true>(ul, U + kC * DV, m0, k);
#pragma unroll
                for (int j = 0; j < 4; j += 2) {
                    uint32_t bh[4], bl[4];
                    planes::frag_b<L::kSlab, true>(bh, s, n0 + 8 * j, kk);
                    planes::frag_b<L::kSlab, true>(bl, s + L::kSlab * DK, n0 + 8 * j, kk);
                    B::mma(a1[j], d, bl[0], bl[1]);
                    B::mma(a1[j + 1], d, bl[2], bl[3]);
                    planes::mma3<B>(a2[j], a2[j + 1], gh, gl, bh, bl);
                    B::mma(a1[j], d, bh[0], bh[1]);
                    B::mma(a1[j + 1], d, bh[2], bh[3]);
                    planes::frag_b<L::kSlab, true>(bh, ds, n0 + 8 * j, kk);
                    planes::frag_b<L::kSlab, true>(bl, ds + L::kSlab * DK, n0 + 8 * j, kk);
                    planes::mma3<B>(a3[j], a3[j + 1], uh, ul, bh, bl);
                }
            }
            __syncthreads();  // the slab is free
            fetch_slab(i + 2);
        }
        *reinterpret_cast<float2 *>(sm + L::GSP + rg * DK + 2 * cp) = make_float2(x, y);
    }
    const int ch = tid % DK, blk = tid / DK, row0 = blk * kSub;  // the thread's channel and tokens
    const T *raw = reinterpret_cast<const T *>(p16 + L::RAW);
    {
        T *to = reinterpret_cast<T *>(p16 + L::RAW);
        load_rows<DK, kT>(to, static_cast<const T *>(a.k) + (long long)h * DK, a.ldk, c);
        load_rows<DK, kT>(to + kC * DK, static_cast<const T *>(a.q) + (long long)h * DK, a.ldq, c);
        load_rows<DK, kT>(to + 2 * kC * DK, static_cast<const T *>(a.z) + (long long)h * DK, a.ldz, c);
        tile::cp_commit();
        tile::cp_wait<0>();
        __syncthreads();
        float la[kSub], s = 0.f;
        const T *p = raw + row0 * DK + ch;
#pragma unroll
        for (int t = 0; t < kSub; ++t) {
            la[t] = row0 + t < c.n ? log2_alpha(to_f(p[2 * kC * DK + t * DK])) : 0.f;
            s += la[t];
            const float e = exp2a(s);
            put1<B, kC>(p16 + L::KL, kC * DK, row0 + t, ch, to_f(p[t * DK]) * (inv[row0 + t] * e));
            put1<B, kC>(p16 + L::QL, kC * DK, row0 + t, ch, to_f(p[kC * DK + t * DK]) * e);
        }
        tot[blk * DK + ch] = exp2a(s);
        s = 0.f;
#pragma unroll
        for (int t = kSub - 1; t >= 0; --t) {
            put1<B, kC>(p16 + L::KR, kC * DK, row0 + t, ch, to_f(p[t * DK]) * (inv[row0 + t] * exp2a(s)));
            s += la[t];
        }
    }
    __syncthreads();
    {
        float rq[4][4], rk[4][4], cl[4][4];
        zero(rq);
        zero(rk);
        zero(cl);
        for (int J = 0; J < I; ++J) {  // rows
            if (J) {
                scale_columns(rq, tot + J * DK, n0);
                scale_columns(rk, tot + J * DK, n0);
            }
            mma_step<B, false, kC, false, kC, true, 4>(rq, DM, kC * kC, m0, J * kSub, p16 + L::KR, kC * DK, n0, J * kSub);
            mma_step<B, false, kC, false, kC, true, 4>(rk, DP, kC * kC, m0, J * kSub, p16 + L::KR, kC * DK, n0, J * kSub);
        }
        for (int J = kNB - 1; J > I; --J) {  // columns
            if (J < kNB - 1) scale_columns(cl, tot + J * DK, n0);
            mma_step<B, false, kC, true, kC, true, 4>(cl, DP, kC * kC, m0, J * kSub, p16 + L::KL, kC * DK, n0, J * kSub);
            mma_step<B, false, kC, true, kC, true, 4>(cl, DM, kC * kC, m0, J * kSub, p16 + L::QL, kC * DK, n0, J * kSub);
        }
        __syncthreads();  // the planes, dM and dP are free
        float *R = reinterpret_cast<float *>(p16 + L::R), *R4 = reinterpret_cast<float *>(p16 + L::R4);
        const float b0 = beta[m0 + g], b1 = beta[m0 + g + 8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int col = n0 + 8 * j + 2 * t4;
            float2 be = make_float2(1.f, 1.f), af = be;
#pragma unroll
            for (int K = 0; K < kNB; ++K) {
                const float2 f = *reinterpret_cast<const float2 *>(tot + K * DK + col);
                if (K < I) be.x *= f.x, be.y *= f.y;
                if (K > I) af.x *= f.x, af.y *= f.y;
            }
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                const int at = tile::at<DK>(m0 + g + 4 * e, col);
                const float b = e ? b1 : b0;
                store2(R + at, fmaf(be.x, a1[j][e], rq[j][e]), fmaf(be.y, a1[j][e + 1], rq[j][e + 1]));
                store2(R + kC * DK + at, fmaf(-b * be.x, a2[j][e], rk[j][e]), fmaf(-b * be.y, a2[j][e + 1], rk[j][e + 1]));
                store2(R + 2 * kC * DK + at, cl[j][e], cl[j][e + 1]);
                store2(R4 + at, af.x * a3[j][e], af.y * a3[j][e + 1]);
            }
        }
    }
    __syncthreads();
    const float *R = reinterpret_cast<const float *>(p16 + L::R);
    float *R4 = reinterpret_cast<float *>(p16 + L::R4);
    const float2 *db = dd + blk * kSub * kSub;
    const long long out0 = ((c.row0 + row0) * a.nh + h) * DK + ch;
    const int ld = a.nh * DK, live = c.n - row0;  // the thread's tokens that are there
    float kk[kSub], dkh[kSub], r[kSub], rs = 0.f, vs = 0.f;
    {
        float q[kSub], la[kSub], run[kSub], s = 0.f;
        const T *p = raw + row0 * DK + ch;
#pragma unroll
        for (int t = 0; t < kSub; ++t) {
            kk[t] = to_f(p[t * DK]) * inv[row0 + t];
            q[t] = to_f(p[kC * DK + t * DK]);
            la[t] = t < live ? log2_alpha(to_f(p[2 * kC * DK + t * DK])) : 0.f;
        }
        // up the tokens: dq and the row part of dk^; run[i] = k^_i decayed to t
#pragma unroll
        for (int t = 0; t < kSub; ++t) {
            const int at = tile::at<DK>(row0 + t, ch);
            s += la[t];
            const float e = exp2a(s), al = exp2a(la[t]);
            float dq = e * R[at], dkr = e * R[kC * DK + at];
#pragma unroll
            for (int i = 0; i < t; ++i) {
                const float2 m = db[t * kSub + i];
                run[i] *= al;
                dq = fmaf(m.x, run[i], dq);
                dkr = fmaf(m.y, run[i], dkr);
            }
            run[t] = kk[t];
            r[t] = fmaf(q[t], dq, kk[t] * dkr);
            dkh[t] = dkr;
            if (t < live) static_cast<T *>(a.dq)[out0 + (long long)t * ld] = __float2bfloat16_rn(fmaf(db[t * kSub + t].x, kk[t], dq));
        }
        // down the tokens: the column part; run[i] = its sum over the tokens so far, decayed to t
#pragma unroll
        for (int t = 0; t < kSub; ++t) run[t] = 0.f;
        s = 0.f;
#pragma unroll
        for (int t = kSub - 1; t >= 0; --t) {
            const int at = tile::at<DK>(row0 + t, ch);
            const float e = exp2a(s), al = exp2a(la[t]);
            const float dkc = fmaf(e, R[2 * kC * DK + at], run[t]), w = e * R4[at], v = kk[t] * w;
            s += la[t];
            R4[at] = v;
            vs += v;
            rs += fmaf(-kk[t], dkc, r[t]);
            r[t] = rs;
            dkh[t] = fmaf(db[t * kSub + t].x, q[t], (dkh[t] + dkc) + w);
#pragma unroll
            for (int i = 0; i < t; ++i) {
                const float2 m = db[t * kSub + i];
                run[i] = al * fmaf(m.y, kk[t], fmaf(m.x, q[t], run[i]));
            }
        }
    }
    sm[L::SUM + blk * DK + ch] = rs;
    sm[L::SUM + (kNB + blk) * DK + ch] = vs;
    {
        float x[kSub];
#pragma unroll
        for (int t = 0; t < kSub; ++t) x[t] = kk[t] * dkh[t];
        const float s = sums16(x);
        if (lane < kSub) sm[L::DOT + warp * kSub + lane] = s;
    }
    __syncthreads();
    {
        float gc = 1.f;
        rs = vs = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) vs += sm[L::GSP + w * DK + ch];
#pragma unroll
        for (int K = 0; K < kNB; ++K) gc *= tot[K * DK + ch];
        vs *= gc;
#pragma unroll
        for (int K = 0; K < kNB; ++K) {
            if (K > blk) rs += sm[L::SUM + K * DK + ch];
            if (K < blk) vs += sm[L::SUM + (kNB + K) * DK + ch];
        }
    }
    // dz, and dk = (dk^ - k^ (k^ . dk^)) / |k|
    T *dz = static_cast<T *>(a.dz) + out0, *dk = static_cast<T *>(a.dk) + out0;
#pragma unroll
    for (int t = 0; t < kSub; ++t) {
        const float z = to_f(raw[2 * kC * DK + (row0 + t) * DK + ch]);
        float dot = 0.f;
#pragma unroll
        for (int w = 0; w < WQ; ++w) dot += sm[L::DOT + (blk * WQ + w) * kSub + t];
        if (t < live) {
            dz[(long long)t * ld] = __float2bfloat16_rn(dz_factor(z) * (r[t] + rs + vs));
            dk[(long long)t * ld] = __float2bfloat16_rn(inv[row0 + t] * fmaf(-kk[t], dot, dkh[t]));
        }
        vs += R4[tile::at<DK>(row0 + t, ch)];
    }
}

}  // namespace

template <int DK, int DV, typename T>
cudaError_t backward(const Args &a, cudaStream_t st)
{
    cudaError_t e = forward<DK, DV, T>(a, true, st);
    if (e == cudaSuccess) e = reverse<DK, DV, T>(a, st);
    const unsigned grid = (unsigned)a.nh * a.max_chunks;
    if (e != cudaSuccess || !grid) return e;
    auto run = [&](auto k, int threads, size_t bytes) {
        const cudaError_t r = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
        if (r != cudaSuccess) return r;
        k<<<grid, threads, bytes, st>>>(a);
        return cudaGetLastError();
    };
    if constexpr (sizeof(T) == 2) return run(k_grad_bf16<DK, DV>, 4 * DK, GradSmem16<DK, DV>::bytes);
    else return run(k_grad_f32<DK, DV>, kThreads, GradSmem<DK, DV>::bytes);
}

#define KDA_GRAD(DK, DV)                                                              \
    template cudaError_t backward<DK, DV, float>(const Args &, cudaStream_t);         \
    template cudaError_t backward<DK, DV, __nv_bfloat16>(const Args &, cudaStream_t);
KDA_GRAD(64, 64)
KDA_GRAD(64, 128)
KDA_GRAD(128, 64)
KDA_GRAD(128, 128)

}  // namespace scan
}  // namespace kda
