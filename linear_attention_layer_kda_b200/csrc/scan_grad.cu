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
#include "scan_kit.cuh"

namespace kda {
namespace scan {
namespace {

template <typename T> __device__ __forceinline__ T from_f(float x);
template <> __device__ __forceinline__ float from_f<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

constexpr float kFloor = kFloor2 * 0.693147181f;

// dz / dla.  Everything in dla_t is proportional to alpha_t, which was held at e^kFloor where it is smaller.
__device__ __forceinline__ float dz_factor(float z)
{
    const float x = exp2a(-1.44269504f * fabsf(z));
    const float s = __fdividef(z < 0.f ? -x : -1.f, 1.f + x);
    return z > -kFloor ? -exp2a(1.44269504f * (-z - kFloor)) : s;  // log alpha of a large z is -z
}

// One block of 4 dk threads per chunk and head; warp w has the tokens of block w / (dk / 32) and a share of
// the columns.  Everything that needs value columns comes first: G, dP, dM, then D1, D2, D3, which stay in
// the accumulators, while 32 value columns of S and dS' at a time pass through shared memory.  The pairs of
// tokens of different blocks are products with k^ GL, q GL and k^ GR (the blocks between them multiplied
// into the accumulators on the way); those of one block are taken in the registers of the thread that has
// the channel's 16 tokens, going up the tokens for the rows and down for the columns, with the sums of dla
// in the same two sweeps.  Bound by issuing instructions (45 % of the slots at 16 warps, the tensor pipe
// 23 %): 4096 chunks and heads of 128 x 128 in bfloat16 take 856 us; with 8 warps and half of the channels
// at a time they took 1227.

template <int DK, int DV, typename T>
struct GradSmem {
    static constexpr int kSlab = 32;  // value columns of S and dS' at a time
    // in 4-byte numbers
    static constexpr int X = 0, DU = X + kC * kC;                  // X, dU; then dM, dP and the diagonal blocks' (dM, dP)
    static constexpr int DM = 0, DP = DM + kC * kC, DD = DP + kC * kC;
    static constexpr int N0 = DU + kC * DV, N1 = DD + 2 * kNB * kSub * kSub;
    static constexpr int U = N0 > N1 ? N0 : N1;
    static constexpr int GO = U + kC * DV, G = GO + kC * DV * (int)sizeof(T) / 4;  // do; G
    static constexpr int S = G + kC * DV;                          // two slabs of S and dS'
    static constexpr int SLAB = 2 * kSlab * DK;
    static constexpr int KL = U, QL = KL + kC * DK, KR = QL + kC * DK;  // in the place of U, do, G and S
    static constexpr int RAW = KR + kC * DK;                       // k, q and, where there is room, z as they are
    static constexpr bool kRawZ = sizeof(T) == 2 || DK == 64;
    static constexpr int R = U;                                    // fp32 tiles [kC][dk], in the same place
    static constexpr int R4 = DM;                                  // the fourth, in dM's and dP's
    static constexpr int E0 = S + 2 * SLAB, E1 = RAW + (kRawZ ? 3 : 2) * kC * DK * (int)sizeof(T) / 4;
    static constexpr int TOT = E0 > E1 ? E0 : E1, GSP = TOT + kNB * DK, SUM = GSP + 8 * DK, DOT = SUM + 2 * kNB * DK;
    static constexpr int BETA = DOT + (DK / 8) * kSub, INV = BETA + kC;
    static constexpr int NOT = INV + kC;                           // 1 - beta
    static constexpr int MB = NOT + kC;                            // barriers: X and dU; U; the slabs
    static constexpr size_t bytes = (size_t)MB * 4 + 4 * 8;
    static_assert(bytes <= 227 * 1024, "");
};

template <int DK, int DV, typename T>
__global__ void __launch_bounds__(4 * DK, 1) k_grad(Args a)
{
    using L = GradSmem<DK, DV, T>;
    using K = Kit<T>;
    using E = typename K::E;
    extern __shared__ __align__(1024) float sm[];
    constexpr bool BF = sizeof(T) == 2;
    constexpr int kT = 4 * DK, WQ = DK / 32;  // threads; warps to a block of tokens
    auto part_of = [&](int at) { return reinterpret_cast<E *>(sm + at); };
    E *GO = part_of(L::GO), *G = part_of(L::G), *U = part_of(L::U), *DM = part_of(L::DM), *DP = part_of(L::DP);
    E *KL = part_of(L::KL), *QL = part_of(L::QL), *KR = part_of(L::KR);
    float2 *dd = reinterpret_cast<float2 *>(sm + L::DD);
    float *tot = sm + L::TOT, *beta = sm + L::BETA, *inv = sm + L::INV;
    const int h = blockIdx.x % a.nh, ci = blockIdx.x / a.nh, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t4 = lane & 3;
    Chunk c;
    if (!locate(a, ci, &c)) return;
    const size_t slot = (size_t)ci * a.nh + h;
    // small loads first: behind the copies they would wait for all of those
    float b0 = 0.f, v0 = 0.f;
    if (tid < kC) {
        if (tid < c.n) b0 = to_f(static_cast<const T *>(a.b)[(c.row0 + tid) * a.ldb + h]);
        v0 = a.inv[slot * kC + tid];
    }
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + L::MB);
    auto copy = [&](int to, const float *from, int numbers, uint64_t *b) {
        if (!a.skip_copies) sm100::bulk_load(sm + to, from, numbers * 4, b);
    };
    const float *du = BF ? reinterpret_cast<const float *>(a.dup) : a.du, *gh = BF ? reinterpret_cast<const float *>(a.ghp) : a.gh;
    auto fetch_slab = [&](int i) {  // value columns kSlab i .. of S and dS', by one thread
        if (i >= DV / L::kSlab) return;
        const float *s = static_cast<const float *>(a.h) + slot * DK * DV, *ds = gh + slot * DK * DV;
        const int to = L::S + (i & 1) * L::SLAB;
        uint64_t *b = bar + 2 + (i & 1);
        if (!a.skip_copies) sm100::mbar_expect_tx(b, L::SLAB * 4);
        if (BF) {  // planes: [2][dk / 64][dv][64], the low plane and the channels from 64 on apart
#pragma unroll
            for (int p = 0; p < 2 * (DK / 64); ++p) {
                const int n = L::kSlab * 64 / 2, from = p * DV * 64 / 2 + i * n;
                copy(to + p * n, s + from, n, b);
                copy(to + L::kSlab * DK + p * n, ds + from, n, b);
            }
        } else {
            copy(to, s + i * L::kSlab * DK, L::kSlab * DK, b);
            copy(to + L::kSlab * DK, ds + i * L::kSlab * DK, L::kSlab * DK, b);
        }
    };
    if (tid == 0) {
        for (int i = 0; i < 4; ++i) sm100::mbar_init(bar + i, 1);
        sm100::mbar_fence_init();
        if (!a.skip_copies) sm100::mbar_expect_tx(bar, (kC * kC + kC * DV) * 4);
        copy(L::X, static_cast<const float *>(a.x) + slot * kC * kC, kC * kC, bar);
        copy(L::DU, du + slot * kC * DV, kC * DV, bar);
        if (!a.skip_copies) sm100::mbar_expect_tx(bar + 1, kC * DV * 4);
        copy(L::U, (BF ? reinterpret_cast<const float *>(a.up) : a.u) + slot * kC * DV, kC * DV, bar + 1);
    }
    constexpr int V = 16 / sizeof(T);
    for (int e = tid; e < kC * DV / V; e += kT) {
        const int r = e / (DV / V), col = V * (e % (DV / V));
        E *to = GO + (BF ? planes::at<kC>(r, col) : tile::at<DV>(r, col));
        if (r < c.n) tile::cp_async16(to, static_cast<const T *>(a.go) + ((c.row0 + r) * a.nh + h) * DV + col);
        else *reinterpret_cast<uint4 *>(to) = make_uint4(0, 0, 0, 0);
    }
    tile::cp_commit();
    if (tid < kC) {
        beta[tid] = tid < c.n ? sigmoid(b0) : 0.f;
        sm[L::NOT + tid] = sigmoid(-b0);  // no difference: a beta near 1 has lost it
        inv[tid] = v0;
    }
    __syncthreads();  // the barriers are there
    bool ok = arrived(a, bar, 0);
    if (tid == 0 && ok) {  // not before: the first product waits for X and dU
        fetch_slab(0);
        fetch_slab(1);
    }
    const int I = warp / WQ, part = warp % WQ, m0 = I * kSub;  // the warp's tokens, and its share of the columns
    {  // G = X^T dU, dv = beta G
        constexpr int NT = DV / WQ / 8;
        const int n0 = part * (DV / WQ);
        float acc[NT][4];
        zero(acc);
        for (int k = m0; k < kC; k += 16)
            K::template step<false, kC, kC, true, DV, kC, false, NT>(acc, part_of(L::X), m0, k, part_of(L::DU), n0, k);
        if (!ok) make_nan(acc);
        T *dv = static_cast<T *>(a.dv) + (c.row0 * a.nh + h) * DV;
        each(acc, m0, n0, [&](int r, int col, float x, float y) {
            K::template put2<kC, DV>(G, r, col, x, y);
            if (r < c.n) store2(dv + (long long)r * a.nh * DV + col, beta[r] * x, beta[r] * y);
        });
    }
    ok = ok && arrived(a, bar + 1, 0);
    tile::cp_wait<0>();
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
                K::template step<BF, kC, DV, false, DV, kC, true, NT>(am, GO, m0, k, U, n0, k);
                K::template step<false, kC, DV, false, DV, kC, true, NT>(ap, G, m0, k, U, n0, k);
            }
        if (!ok) {
            make_nan(am);
            make_nan(ap);
        }
        each(am, m0, n0, [&](int r, int col, float x, float y) {
            if (col < m0) {
                K::template put2<kC, kC>(DM, r, col, x, y);
            } else if (col < m0 + kSub) {
                float2 *p = dd + (I * kSub + (r - m0)) * kSub + col - m0;
                p[0].x = col <= r ? x : 0.f;
                p[1].x = col + 1 <= r ? y : 0.f;
            }
        });
        each(ap, m0, n0, [&](int r, int col, float x, float y) {
            const float b = beta[r];
            if (col < m0) {
                K::template put2<kC, kC>(DP, r, col, -b * x, -b * y);
            } else if (col < m0 + kSub) {
                float2 *p = dd + (I * kSub + (r - m0)) * kSub + col - m0;
                p[0].y = col < r ? -b * x : 0.f;
                p[1].y = col + 1 < r ? -b * y : 0.f;
                if ((col == r || col + 1 == r) && r < c.n)  // G_t . U_t
                    store1(static_cast<T *>(a.db) + (c.row0 + r) * a.nh + h, sm[L::NOT + r] * (col == r ? x : y));
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
            ok = ok && arrived(a, bar + 2 + (i & 1), i >> 1);
            const E *s = part_of(L::S + (i & 1) * L::SLAB), *ds = part_of(L::S + (i & 1) * L::SLAB + L::kSlab * DK);
#pragma unroll
            for (int r = 0; r < L::kSlab / 8; ++r) {
                const float2 u = K::template get2<L::kSlab, DK>(s, rg * (L::kSlab / 8) + r, 2 * cp);
                const float2 v = K::template get2<L::kSlab, DK>(ds, rg * (L::kSlab / 8) + r, 2 * cp);
                x = fmaf(u.x, v.x, x);
                y = fmaf(u.y, v.y, y);
            }
#pragma unroll
            for (int kk = 0; kk < L::kSlab; kk += 16) {
                const int k = i * L::kSlab + kk;
                K::template step<BF, kC, DV, false, L::kSlab, DK, true, 4>(a1, GO, m0, k, s, n0, kk);
                K::template step<false, kC, DV, false, L::kSlab, DK, true, 4>(a2, G, m0, k, s, n0, kk);
                K::template step<false, DV, kC, true, L::kSlab, DK, true, 4>(a3, U, m0, k, ds, n0, kk);
            }
            __syncthreads();  // the slab is free
            if (tid == 0 && ok) fetch_slab(i + 2);
        }
        if (!ok) {
            make_nan(a1);
            make_nan(a2);
            make_nan(a3);
            x = y = nan_f();
            if (tid == 0) drain(a, bar, 4);
        }
        *reinterpret_cast<float2 *>(sm + L::GSP + rg * DK + 2 * cp) = make_float2(x, y);
    }
    const int ch = tid % DK, blk = tid / DK, row0 = blk * kSub;  // the thread's channel and tokens
    const T *raw = reinterpret_cast<const T *>(sm + L::RAW);
    const T *zp = static_cast<const T *>(a.z) + c.row0 * a.ldz + (long long)h * DK + ch;
    auto gate = [&](int t) {  // z of the thread's t-th token; past the chunk's end any value
        return L::kRawZ ? to_f(raw[2 * kC * DK + (row0 + t) * DK + ch]) : to_f(zp[min(row0 + t, c.n - 1) * a.ldz]);
    };
    {
        T *to = reinterpret_cast<T *>(sm + L::RAW);
        load_rows<DK, kT>(to, static_cast<const T *>(a.k) + (long long)h * DK, a.ldk, c);
        load_rows<DK, kT>(to + kC * DK, static_cast<const T *>(a.q) + (long long)h * DK, a.ldq, c);
        if (L::kRawZ) load_rows<DK, kT>(to + 2 * kC * DK, static_cast<const T *>(a.z) + (long long)h * DK, a.ldz, c);
        tile::cp_commit();
        tile::cp_wait<0>();
        __syncthreads();
        float la[kSub], s = 0.f;
        const T *p = raw + row0 * DK + ch;
#pragma unroll
        for (int t = 0; t < kSub; ++t) {
            la[t] = row0 + t < c.n ? log2_alpha(gate(t)) : 0.f;
            s += la[t];
            const float e = exp2a(s);
            K::template put1<kC, DK>(KL, row0 + t, ch, to_f(p[t * DK]) * (inv[row0 + t] * e));
            K::template put1<kC, DK>(QL, row0 + t, ch, to_f(p[kC * DK + t * DK]) * e);
        }
        tot[blk * DK + ch] = exp2a(s);
        s = 0.f;
#pragma unroll
        for (int t = kSub - 1; t >= 0; --t) {
            K::template put1<kC, DK>(KR, row0 + t, ch, to_f(p[t * DK]) * (inv[row0 + t] * exp2a(s)));
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
            K::template step<false, kC, kC, false, kC, DK, true, 4>(rq, DM, m0, J * kSub, KR, n0, J * kSub);
            K::template step<false, kC, kC, false, kC, DK, true, 4>(rk, DP, m0, J * kSub, KR, n0, J * kSub);
        }
        for (int J = kNB - 1; J > I; --J) {  // columns
            if (J < kNB - 1) scale_columns(cl, tot + J * DK, n0);
            K::template step<false, kC, kC, true, kC, DK, true, 4>(cl, DP, m0, J * kSub, KL, n0, J * kSub);
            K::template step<false, kC, kC, true, kC, DK, true, 4>(cl, DM, m0, J * kSub, QL, n0, J * kSub);
        }
        __syncthreads();  // the planes, dM and dP are free
        float *R = sm + L::R, *R4 = sm + L::R4;
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
    const float *R = sm + L::R;
    float *R4 = sm + L::R4;
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
            la[t] = t < live ? log2_alpha(gate(t)) : 0.f;
        }
        // up the tokens: dq and the row part of dk^; run[i] = k^_i decayed to t
#pragma unroll
        for (int t = 0; t < kSub; ++t) {
            const int at = tile::at<DK>(row0 + t, ch);
            s += la[t];
            const float e = exp2a(s), al = exp2a(la[t]);
            float dq = e * R[at], dkr = e * R[kC * DK + at];
#pragma unroll
            for (int i = 0; i < t; i += 2) {
                const float4 m = *reinterpret_cast<const float4 *>(db + t * kSub + i);
                run[i] *= al;
                dq = fmaf(m.x, run[i], dq);
                dkr = fmaf(m.y, run[i], dkr);
                if (i + 1 < t) {
                    run[i + 1] *= al;
                    dq = fmaf(m.z, run[i + 1], dq);
                    dkr = fmaf(m.w, run[i + 1], dkr);
                }
            }
            run[t] = kk[t];
            r[t] = fmaf(q[t], dq, kk[t] * dkr);
            dkh[t] = dkr;
            if (t < live) static_cast<T *>(a.dq)[out0 + (long long)t * ld] = from_f<T>(fmaf(db[t * kSub + t].x, kk[t], dq));
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
            for (int i = 0; i < t; i += 2) {
                const float4 m = *reinterpret_cast<const float4 *>(db + t * kSub + i);
                run[i] = al * fmaf(m.y, kk[t], fmaf(m.x, q[t], run[i]));
                if (i + 1 < t) run[i + 1] = al * fmaf(m.w, kk[t], fmaf(m.z, q[t], run[i + 1]));
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
        const float z = gate(t);
        float dot = 0.f;
#pragma unroll
        for (int w = 0; w < WQ; ++w) dot += sm[L::DOT + (blk * WQ + w) * kSub + t];
        if (t < live) {
            dz[(long long)t * ld] = from_f<T>(dz_factor(z) * (r[t] + rs + vs));
            dk[(long long)t * ld] = from_f<T>(inv[row0 + t] * fmaf(-kk[t], dot, dkh[t]));
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
    return run(k_grad<DK, DV, T>, 4 * DK, GradSmem<DK, DV, T>::bytes);
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
