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
#include "scan_ops.cuh"

namespace kda {
namespace scan {
namespace {

// du = M^T do, gh = (g q)^T do for every chunk and head.
template <int DK, int DV>
struct GradPrepSmem {
    static constexpr int M = 0, GO = M + kC * kC, QB = GO + kC * DV;
    static constexpr size_t bytes = (size_t)(QB + kC * DK) * 4;
};

template <int DK, int DV, typename T>
__global__ void __launch_bounds__(kThreads) k_grad_prep(Args a)
{
    extern __shared__ __align__(128) float sm[];
    using L = GradPrepSmem<DK, DV>;
    const int h = blockIdx.x % a.nh, ci = blockIdx.x / a.nh, warp = threadIdx.x >> 5;
    Chunk c;
    if (!locate(a, ci, &c)) return;
    const size_t slot = (size_t)ci * a.nh + h;
    tile::copy_async<kThreads>(sm + L::M, a.m + slot * kC * kC, kC * kC);
    tile::copy_async<kThreads>(sm + L::QB, a.qb + slot * kC * DK, kC * DK);
    tile::cp_commit();
    load_tile<DV>(sm + L::GO, static_cast<const T *>(a.go) + (long long)h * DV, (long long)a.nh * DV, c,
                  [](float x) { return x; });
    tile::cp_wait<0>();
    __syncthreads();
    // both transposed: rows are value columns
    const tile::Op<DV, true> A{sm + L::GO};
    float *du = a.du + slot * kC * DV, *gh = a.gh + slot * DK * DV;
    constexpr int MT = DV / 64;
    const int m0 = (warp & 3) * (DV / 4), half = warp >> 2;
#pragma unroll
    for (int I = 0; I < 2; ++I) {
        const int n0 = half * 32 + 16 * I;
        float acc[MT][2][4];
        tile::zero(acc);
        tile::mma<MT, 2>(acc, A, m0, tile::Op<kC, true>{sm + L::M}, n0, n0, kC);
        tile::each(acc, m0, n0, [&](int r, int col, float x, float y) { store2(du + tile::at<kC>(r, col), x, y); });
    }
    {
        constexpr int NT = DK / 16;
        const int n0 = half * (DK / 2);
        float acc[MT][NT][4];
        tile::zero(acc);
        tile::mma<MT, NT>(acc, A, m0, tile::Op<DK, true>{sm + L::QB}, n0, 0, kC);
        tile::each(acc, m0, n0, [&](int r, int col, float x, float y) { store2(gh + tile::at<DK>(r, col), x, y); });
    }
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
    const float over = -z - kFloor;  // log alpha of a large z is -z
    return over < 0.f ? -expf(over) : -sigmoid(z);
}

template <int DK, int DV, typename T>
__global__ void __launch_bounds__(kThreads, 1) k_grad(Args a)
{
    extern __shared__ __align__(128) float sm[];
    using L = GradSmem<DK, DV>;
    const int h = blockIdx.x % a.nh, ci = blockIdx.x / a.nh, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    Chunk c;
    if (!locate(a, ci, &c)) return;
    const size_t slot = (size_t)ci * a.nh + h;
    float *R0 = sm + L::R0, *R1 = sm + L::R1, *R2 = sm + L::R2, *R3 = sm + L::R3, *XM = sm + L::XM, *DP = sm + L::DP;
    float *beta = sm + L::BETA, *md = sm + L::MD, *gs = sm + L::GS, *rd = sm + L::RD;
    const long long dv0 = (c.row0 * a.nh + h) * DV, dk0 = (c.row0 * a.nh + h) * DK;  // of the dense gradients

    tile::copy_async<kThreads>(XM, a.x + slot * kC * kC, kC * kC);
    tile::copy_async<kThreads>(R0, a.du + slot * kC * DV, kC * DV);
    tile::cp_commit();
    tile::copy_async<kThreads>(R2, a.u + slot * kC * DV, kC * DV);
    tile::copy_async<kThreads>(R3, a.h + slot * DK * DV, DK * DV);
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

}  // namespace

template <int DK, int DV, typename T>
cudaError_t backward(const Args &a, cudaStream_t st)
{
    cudaError_t e = forward<DK, DV, T>(a, false, st);
    const unsigned grid = (unsigned)a.nh * a.max_chunks;
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(k_grad_prep<DK, DV, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)GradPrepSmem<DK, DV>::bytes);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(k_grad<DK, DV, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)GradSmem<DK, DV>::bytes);
    if (e != cudaSuccess) return e;
    if (grid) k_grad_prep<DK, DV, T><<<grid, kThreads, GradPrepSmem<DK, DV>::bytes, st>>>(a);
    e = reverse<DK, DV>(a, st);
    if (e != cudaSuccess) return e;
    if (grid) k_grad<DK, DV, T><<<grid, kThreads, GradSmem<DK, DV>::bytes, st>>>(a);
    return cudaGetLastError();
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
