// scan_prep.cuh -- what a chunk's keys, queries, gates (and, backward, gradients of o) give without
// the states (notation: scan.cuh): Kx, W, Uv and the chunk's decay for the pass over the states; g q
// and M for the outputs; X, M^T do and (g q)^T do for the backward pass.
//
// One block of 4 dk threads per chunk and head: a thread has one channel of one block of 16 tokens in
// registers, where the sums of log alpha, the decays and the pairs of tokens inside the block
// (multiplied up, 32 sums over channels at a time through shuffles) are.  16 warps, not 8 with two
// channels to a thread: with its 200 KB of shared memory a block has the SM for itself, and the phases
// between its barriers wait for latencies more than for instructions.  All else is products of half
// planes in shared memory; the totals of blocks between two tokens are multiplied into the accumulators,
// or into copies of the right factor.
// Bound by issuing instructions (of 100,000 a chunk and head the pairs take a fifth, the splitting as
// much; 53 % of the issue slots at 16 warps): 4096 chunks and heads of 128 x 128 with the backward
// pass's terms take 711 us, 2112 without them 319 us; about 280 KB of each are read or written.
// Half planes have the range of fp16, so each of their scales goes with what cannot be told apart: v and
// do by value column, q and M by token (do takes the inverse, since tokens are what is summed), X diag(beta)
// by token, k^ GL by block of tokens.
#pragma once

#include "scan_ops.cuh"

namespace kda {
namespace scan {

constexpr int kLdA = kC + 4;  // row length of A and X: rows on different banks

template <int DK, int DV, bool BWD>
struct PrepSmem {
    // half planes, in uint16_t elements
    static constexpr int KL = 0, QL = KL + 2 * kC * DK;  // k^ GL, q GL
    static constexpr int KR = QL + 2 * kC * DK;          // six [16][dk]: k^ GR of block J, times the totals up to block I
    static constexpr int V = KR + 2 * 32 * 32;           // v, once KR (and the inverse's scratch before V) is free
    static constexpr int KRN = 6 * 2 * kSub * DK, VN = 2 * 32 * 32 + 2 * kC * DV;
    static constexpr int MP = KR + (KRN > VN ? KRN : VN);  // M, do
    static constexpr int GO = MP + (BWD ? 2 * kC * kC : 0);
    static constexpr int END = GO + (BWD ? 2 * kC * DV : 0);
    // floats
    static constexpr int A = END / 2;                    // beta P; then the planes of X diag(beta)
    static constexpr int X = A + kC * kLdA;              // the pairs' sums; then X
    static constexpr int TOT = X + kC * kLdA, BETA = TOT + kNB * DK, INV = BETA + kC, RED = INV + kC;
    static constexpr int IB = RED + 16 * kSub + 16;      // the inverses of the tokens' scales of beta
    static constexpr int SB = IB + kC;                   // the scales
    static constexpr int QS = SB + kC, QI = QS + kC;     // the tokens' scales of q, and their inverses
    static constexpr int CM = QI + kC;                   // largest |v| of every value column; |do / QS|
    static constexpr size_t bytes = (size_t)(CM + (BWD ? 2 : 1) * DV) * 4;
    static_assert(bytes <= 227 * 1024, "");
};

// X = (I + A)^-1 for the unit lower triangular I + A, first part: the four diagonal blocks by
// substitution, a lane to a column, in four warps; zeros above them.
template <int THREADS>
__device__ __forceinline__ void invert_blocks(const float *A, float *X)
{
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (warp < kNB && lane < kSub) {
        const int b0 = warp * kSub;
        float x[kSub];
#pragma unroll
        for (int r = 0; r < kSub; ++r) {
            float s = r == lane ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
            for (int i = 0; i + 1 < r; i += 2) {
                s = fmaf(-A[(b0 + r) * kLdA + b0 + i], x[i], s);
                s1 = fmaf(-A[(b0 + r) * kLdA + b0 + i + 1], x[i + 1], s1);
            }
            if (r & 1) s = fmaf(-A[(b0 + r) * kLdA + b0 + r - 1], x[r - 1], s);
            x[r] = s + s1;
        }
#pragma unroll
        for (int r = 0; r < kSub; ++r) X[(b0 + r) * kLdA + b0 + lane] = x[r];
    }
    for (int e = tid; e < kC * kC / 4; e += THREADS) {
        const int r = e / (kC / 4), c = 4 * (e % (kC / 4));
        if (c / kSub > r / kSub) *reinterpret_cast<float4 *>(X + r * kLdA + c) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
}
// Second part, after a barrier: two blocks of 16 to one of 32 and two of 32 to one of 64, the lower left
// being -X22 (A21 X11).  S: scratch [32][32].  Ends with a barrier.
template <int N, int THREADS>
__device__ __forceinline__ void invert_join(const float *A, float *X, float *S)
{
    constexpr int W = kC / (2 * N) * N * N / THREADS;  // neighbouring columns of a thread
    static_assert(W == 1 || W == 2 || W == 4, "");
    const int e = threadIdx.x, q = e / (N * N / W), r = (e / (N / W)) % N, c = W * (e % (N / W)), b = q * 2 * N;
    float s[W];
#pragma unroll
    for (int j = 0; j < W; ++j) s[j] = 0.f;
#pragma unroll 16
    for (int k = 0; k < N; ++k) {
        const float l = A[(b + N + r) * kLdA + b + k];
#pragma unroll
        for (int j = 0; j < W; ++j) s[j] = fmaf(l, X[(b + k) * kLdA + b + c + j], s[j]);
    }
#pragma unroll
    for (int j = 0; j < W; ++j) S[q * N * N + r * N + c + j] = s[j];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < W; ++j) s[j] = 0.f;
#pragma unroll 16
    for (int k = 0; k < N; ++k) {
        const float l = -X[(b + N + r) * kLdA + b + N + k];
#pragma unroll
        for (int j = 0; j < W; ++j) s[j] = fmaf(l, S[q * N * N + k * N + c + j], s[j]);
    }
#pragma unroll
    for (int j = 0; j < W; ++j) X[(b + N + r) * kLdA + b + c + j] = s[j];
    __syncthreads();
}

// One element into the planes at p (the low plane n elements further).
template <class P, int R>
__device__ __forceinline__ void put1(uint16_t *p, int n, int r, int c, float x)
{
    const uint32_t hi = P::pack(x, 0.f), lo = P::pack(x - P::unpack(hi).x, 0.f);
    uint16_t *q = p + planes::at<R>(r, c);
    q[0] = (uint16_t)hi;
    q[n] = (uint16_t)lo;
}

// D channels of the chunk's rows as they are, [kC][D], copied asynchronously; rows past the chunk's end are zero.
template <int D, int THREADS, typename T>
__device__ __forceinline__ void load_rows(T *dst, const T *src, long long ld, const Chunk &c)
{
    constexpr int V = 16 / sizeof(T);
    for (int e = threadIdx.x; e < kC * D / V; e += THREADS) {
        const int r = e / (D / V), col = e % (D / V) * V;
        if (r < c.n) tile::cp_async16(dst + r * D + col, src + (c.row0 + r) * ld + col);
        else *reinterpret_cast<uint4 *>(dst + r * D + col) = make_uint4(0, 0, 0, 0);
    }
}

// Four elements as they are in memory
struct Raw4f { float4 v; __device__ __forceinline__ void get(float (&x)[4]) const { x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w; } };
struct Raw4b
{
    uint2 v;
    __device__ __forceinline__ void get(float (&x)[4]) const
    {
        x[0] = __uint_as_float(v.x << 16), x[1] = __uint_as_float(v.x & 0xffff0000u);
        x[2] = __uint_as_float(v.y << 16), x[3] = __uint_as_float(v.y & 0xffff0000u);
    }
};
template <typename T> struct Pick { using R = Raw4f; };
template <> struct Pick<__nv_bfloat16> { using R = Raw4b; };
__device__ __forceinline__ void load_raw(const float *p, Raw4f &r) { r.v = __ldg(reinterpret_cast<const float4 *>(p)); }
__device__ __forceinline__ void load_raw(const __nv_bfloat16 *p, Raw4b &r) { r.v = __ldg(reinterpret_cast<const uint2 *>(p)); }

// Rows of v or do into half planes, from registers that hold them: four neighbouring columns, the same in all of a
// thread's rows.
template <int D, int THREADS, typename T>
struct RowTile {
    static constexpr int N = kC * D / 4 / THREADS;
    static_assert(THREADS % (D / 4) == 0, "");
    typename Pick<T>::R x[N];
    __device__ __forceinline__ void load(const T *src, long long ld, const Chunk &c)
    {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int e = threadIdx.x + i * THREADS, r = e / (D / 4), c4 = 4 * (e % (D / 4));
            x[i].v = {};
            if (r < c.n) load_raw(src + (c.row0 + r) * ld + c4, x[i]);
        }
    }
    // Place of a column in lists of the columns' largest sizes: a warp's columns on different banks.
    static __device__ __forceinline__ int place(int c) { return (c & 3) * (D / 4) + (c >> 2); }
    // Largest size in each column, of the elements times f(row), into m (as bits); m starts at 0.
    template <class F>
    __device__ __forceinline__ void largest(uint32_t *m, F f) const
    {
        float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float s = f((threadIdx.x + i * THREADS) / (D / 4));
            float v[4];
            x[i].get(v);
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = fmaxf(y[j], fabsf(v[j] * s));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) atomicMax(m + place(4 * (threadIdx.x % (D / 4)) + j), __float_as_uint(y[j]));
    }
    // The elements times f(row) and a scale for each column, from its largest size.
    template <class F>
    __device__ __forceinline__ void put(uint16_t *p, const uint32_t *m, F f) const
    {
        const int c4 = 4 * (threadIdx.x % (D / 4));
        float s[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float inv;
            planes::scale_of(__uint_as_float(m[place(c4 + j)]), s[j], inv);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int r = (threadIdx.x + i * THREADS) / (D / 4);
            const float y = f(r);
            float v[4];
            x[i].get(v);
            planes::put2<planes::H, kC>(p, kC * D, r, c4, v[0] * y * s[0], v[1] * y * s[1]);
            planes::put2<planes::H, kC>(p, kC * D, r, c4 + 2, v[2] * y * s[2], v[3] * y * s[3]);
        }
    }
};

// One k step of 16: acc += A B; EXACT: A's first plane is all of it (a bfloat16 number).
template <class P, bool EXACT, int RA, bool KA, int RB, bool KB, int NT>
__device__ __forceinline__ void mma_step(float (&acc)[NT][4], const uint16_t *A, int na, int m0, int ka, const uint16_t *Bp,
                                         int nb, int n0, int kb)
{
    uint32_t ah[4], al[4];
    planes::frag_a<RA, KA>(ah, A, m0, ka);
    if (!EXACT) planes::frag_a<RA, KA>(al, A + na, m0, ka);
#pragma unroll
    for (int j = 0; j < NT; j += 2) {
        uint32_t bh[4], bl[4];
        planes::frag_b<RB, KB>(bh, Bp, n0 + 8 * j, kb);
        planes::frag_b<RB, KB>(bl, Bp + nb, n0 + 8 * j, kb);
        if (!EXACT) {
            planes::mma3<P>(acc[j], acc[j + 1], ah, al, bh, bl);
        } else {
            P::mma(acc[j], ah, bl[0], bl[1]);
            P::mma(acc[j + 1], ah, bl[2], bl[3]);
            P::mma(acc[j], ah, bh[0], bh[1]);
            P::mma(acc[j + 1], ah, bh[2], bh[3]);
        }
    }
}

template <int NT>
__device__ __forceinline__ void zero(float (&acc)[NT][4])
{
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
}
// acc's columns n0 + 8 j + .. times f[column]
template <int NT>
__device__ __forceinline__ void scale_columns(float (&acc)[NT][4], const float *f, int n0)
{
    const int t = threadIdx.x & 3;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const float2 x = *reinterpret_cast<const float2 *>(f + n0 + 8 * j + 2 * t);
        acc[j][0] *= x.x, acc[j][1] *= x.y, acc[j][2] *= x.x, acc[j][3] *= x.y;
    }
}
// f(row, col, x, y) of a 16 x 8 NT accumulator
template <int NT, class F>
__device__ __forceinline__ void each(const float (&acc)[NT][4], int m0, int n0, F f)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        f(m0 + g, n0 + 8 * j + 2 * t, acc[j][0], acc[j][1]);
        f(m0 + g + 8, n0 + 8 * j + 2 * t, acc[j][2], acc[j][3]);
    }
}

template <int DK, int DV, bool BWD, typename T>
__global__ void __launch_bounds__(4 * DK, DK == 64 ? 2 : 1) k_scan_prep(Args a)
{
    extern __shared__ __align__(1024) float sm[];
    using L = PrepSmem<DK, DV, BWD>;
    using planes::kDown;
    using planes::kUp;
    constexpr bool BF = sizeof(T) == 2;
    constexpr int kT = 4 * DK, kW = kT / 32, kWB = DK / 32;  // threads, warps, warps of a block of tokens
    uint16_t *pl16 = reinterpret_cast<uint16_t *>(sm);
    uint16_t *KL = pl16 + L::KL, *QL = pl16 + L::QL, *KR = pl16 + L::KR, *MP = pl16 + L::MP;
    uint16_t *VP = pl16 + L::V, *GO = pl16 + L::GO;
    float *A = sm + L::A, *X = sm + L::X, *tot = sm + L::TOT, *beta = sm + L::BETA, *inv = sm + L::INV, *red = sm + L::RED;
    float *sb = sm + L::SB, *ib = sm + L::IB, *qs = sm + L::QS, *qi = sm + L::QI;
    uint32_t *vmax = reinterpret_cast<uint32_t *>(sm + L::CM), *gmax = vmax + DV;
    uint16_t *XB = reinterpret_cast<uint16_t *>(A);
    float *mx = red + 16 * kSub;  // of the warps: log2 of the largest first decay of their block
    const int h = blockIdx.x % a.nh, ci = blockIdx.x / a.nh, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int blk = tid / DK, d = tid % DK;  // the thread's block of tokens and channel
    Chunk c;
    if (!locate(a, ci, &c)) return;
    const size_t slot = (size_t)ci * a.nh + h;

    // k, q, z as they are, through the place of the planes to come, into registers by channel
    float k[kSub], q[kSub], la[kSub];
    {
        T *raw = reinterpret_cast<T *>(sm);
        load_rows<DK, kT>(raw, static_cast<const T *>(a.k) + (long long)h * DK, a.ldk, c);
        load_rows<DK, kT>(raw + kC * DK, static_cast<const T *>(a.q) + (long long)h * DK, a.ldq, c);
        load_rows<DK, kT>(raw + 2 * kC * DK, static_cast<const T *>(a.z) + (long long)h * DK, a.ldz, c);
        tile::cp_commit();
        if (tid < kC) beta[tid] = tid < c.n ? sigmoid(to_f(static_cast<const T *>(a.b)[(c.row0 + tid) * a.ldb + h])) : 0.f;
        tile::cp_wait<0>();
        __syncthreads();
        const T *p = raw + blk * kSub * DK + d;
#pragma unroll
        for (int t = 0; t < kSub; ++t) {
            k[t] = to_f(p[t * DK]);
            q[t] = to_f(p[kC * DK + t * DK]);
            la[t] = blk * kSub + t < c.n ? log2_alpha(to_f(p[2 * kC * DK + t * DK])) : 0.f;
        }
    }
    float tl = 0.f;  // the block's total, in log2
    {
        float ss[kSub];
        uint32_t m = 0;  // the largest |q| of token `lane`
#pragma unroll
        for (int t = 0; t < kSub; ++t) {
            ss[t] = k[t] * k[t];
            const uint32_t x = __reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(q[t])));
            if (lane == t) m = x;
            tl += la[t];
        }
        tot[blk * DK + d] = tl;
        const float x = sums16(ss);
        if (lane < kSub) red[warp * kSub + lane] = x, X[warp * kSub + lane] = __uint_as_float(m);
        const float f = warp_max(la[0]);
        if (lane == 0) mx[warp] = f;
        if (tid < (BWD ? 2 : 1) * DV) vmax[tid] = 0;
    }
    __syncthreads();
    if (tid < kC) {
        float s = 0.f;
        uint32_t m = 0;
#pragma unroll
        for (int w = 0; w < kWB; ++w) {
            const int i = ((tid >> 4) * kWB + w) * kSub + (tid & 15);
            s += red[i];
            m = max(m, __float_as_uint(X[i]));
        }
        planes::scale_of(__uint_as_float(m), qs[tid], qi[tid]);
        planes::scale_of(beta[tid], sb[tid], ib[tid]);
        const float x = s > 0.f ? 1.f / sqrtf(s) : s == s ? 0.f : s;
        inv[tid] = x;
        if (BWD) a.inv[slot * kC + tid] = x;
    }
    __syncthreads();
    auto largest = [&](int first, int n) {
        float m = mx[first];
        for (int w = 1; w < n; ++w) m = fmaxf(m, mx[first + w]);
        return m;
    };
    // scale of block b's k^ GL: all of it has the decay of the block's first token as a factor
    auto block_scale = [&](int b, float &u, float &iu) { planes::scale_of(exp2a(largest(kWB * b, kWB)), u, iu); };
#pragma unroll
    for (int t = 0; t < kSub; ++t) k[t] *= inv[blk * kSub + t];
    // Log2 of W's scale: what the tokens behind the last key that is not zero leave of it at most (rows of zeros that
    // pad a sequence decay the state all the same).  Nothing where the chunk's last token has a key.
    float wl = 0.f;
    if (!(inv[c.n - 1] > 0.f)) {
        uint32_t m = 0;
#pragma unroll
        for (int t = 0; t < kSub; ++t) {  // the channels' slowest decay at token `lane`
            const uint32_t x = __reduce_min_sync(0xffffffffu, __float_as_uint(fabsf(la[t])));
            if (lane == t) m = x;
        }
        if (lane < kSub) X[warp * kSub + lane] = __uint_as_float(m);
        __syncthreads();
        const uint32_t k0 = __ballot_sync(0xffffffffu, inv[lane] != 0.f), k1 = __ballot_sync(0xffffffffu, inv[lane + 32] != 0.f);
        const int last = k1 ? 63 - __clz(k1) : 31 - __clz(k0);  // -1: no key at all
#pragma unroll
        for (int t = lane; t < kC; t += 32) {
            float x = __int_as_float(0x7f800000);
#pragma unroll
            for (int w = 0; w < kWB; ++w) x = fminf(x, X[((t >> 4) * kWB + w) * kSub + (t & 15)]);
            if (t > last) wl -= x;
        }
        wl = last < 0 ? 0.f : fmaxf(floorf(warp_sum(wl)), -100.f);
        __syncthreads();
    }
    // ---- the planes of k^ GL, q GL, k^ GR, and W and g q for the workspace
    {
        float before = 0.f, after = 0.f, ub, iub;
#pragma unroll
        for (int b = 0; b < kNB; ++b) {
            const float v = tot[b * DK + d];
            if (b < blk) before += v;
            if (b > blk) after += v;
        }
        const float next1 = blk < 2 ? exp2a(tot[(blk + 1) * DK + d]) : 0.f;
        const float next2 = blk < 1 ? exp2a(tot[(blk + 1) * DK + d] + tot[(blk + 2) * DK + d]) : 0.f;
        block_scale(blk, ub, iub);
        const float ub15 = ub * (1.f / 32768.f);
        if (blk == kNB - 1) a.gc[slot * (DK + 4) + d] = exp2a(before + tl);
        if (tid == 0) a.gc[slot * (DK + 4) + DK + 1] = exp2a(wl) * kDown;
        uint16_t *W = a.w + slot * 2 * kC * DK;
        float s = 0.f;
#pragma unroll
        for (int t = 0; t < kSub; ++t) {
            const int r = blk * kSub + t;
            s += la[t];
            const float g = exp2a(s);
            put1<planes::H, kC>(KL, kC * DK, r, d, k[t] * (g * ub));
            put1<planes::H, kC>(QL, kC * DK, r, d, (q[t] * qs[r]) * (g * ub15));
            if (!BWD) {
                const float z = q[t] * exp2a(s + before);
                if (BF) put1<planes::B, kC>(static_cast<uint16_t *>(a.qb) + slot * 2 * kC * DK, kC * DK, r, d, z);
                else static_cast<float *>(a.qb)[slot * kC * DK + tile::at<DK>(r, d)] = z;
            }
        }
        s = 0.f;
#pragma unroll
        for (int t = kSub - 1; t >= 0; --t) {
            const float x = k[t] * (exp2a(s) * kUp);
            put1<planes::H, kC>(W, kC * DK, blk * kSub + t, d, k[t] * (exp2a(s + (after - wl)) * kUp));
            s += la[t];
            if (blk < 3) {  // copies 0 .. 2: blocks (1, 0), (2, 1), (3, 2); 3, 4: (2, 0), (3, 1); 5: (3, 0)
                put1<planes::H, kSub>(KR + blk * 2 * kSub * DK, kSub * DK, t, d, x);
                if (blk < 2) put1<planes::H, kSub>(KR + (3 + blk) * 2 * kSub * DK, kSub * DK, t, d, x * next1);
                if (blk < 1) put1<planes::H, kSub>(KR + 5 * 2 * kSub * DK, kSub * DK, t, d, x * next2);
            }
        }
    }
    RowTile<DV, kT, T> vt;  // on its way while the pairs are computed
    vt.load(static_cast<const T *>(a.v) + (long long)h * DV, a.ldv, c);
    // ---- pairs inside a block: the decay multiplied up from k^_i, columns i and 15 - i at a time: 32 sums
    {
#pragma unroll
        for (int t = 0; t < kSub; ++t) la[t] = exp2a(la[t]);  // alpha from here on
        float *pd = X + warp * 256;
#pragma unroll
        for (int i = 0; i < kSub / 2; ++i) {
            float s[32];
            int n = 0;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int i0 = half ? kSub - 1 - i : i;
                float kg = k[i0];
                s[n++] = kg * q[i0];
#pragma unroll
                for (int t = i0 + 1; t < kSub; ++t) {
                    kg *= la[t];
                    s[n++] = kg * k[t];
                    s[n++] = kg * q[t];
                }
            }
            pd[i * 32 + lane] = sums32(s);
        }
    }
    auto one = [](int) { return 1.f; };
    vt.largest(vmax, one);
    __syncthreads();
    RowTile<DV, kT, T> gt;
    if (BWD) gt.load(static_cast<const T *>(a.go) + (long long)h * DV, (long long)a.nh * DV, c);
    // ---- P (times beta, into A) and M; a warp takes one of twelve 16 x 16 products, then the pairs' sums
    auto put_m = [&](int r, int col, float x, float y) {
        const float sM = qs[r] * 0.0625f;  // |M| <= sqrt(dk) max |q|
        if (BWD) planes::put2<planes::H, kC>(MP, kC * kC, r, col, x * sM, y * sM);
        else if (BF) planes::put2<planes::B, kC>(static_cast<uint16_t *>(a.m) + slot * 2 * kC * kC, kC * kC, r, col, x, y);
        else *reinterpret_cast<float2 *>(static_cast<float *>(a.m) + slot * kC * kC + tile::at<kC>(r, col)) = make_float2(x, y);
    };
    for (int p = warp; p < 12; p += kW) {
        const int b = p >> 1, J = b < 3 ? b : b < 5 ? b - 3 : 0, I = b < 3 ? b + 1 : b < 5 ? b - 1 : 3;
        const bool isM = p & 1;
        float acc[2][4];
        zero(acc);
#pragma unroll 4
        for (int kk = 0; kk < DK; kk += 16)
            mma_step<planes::H, false, kC, false, kSub, false, 2>(acc, isM ? QL : KL, kC * DK, I * kSub, kk, KR + b * 2 * kSub * DK, kSub * DK, 0, kk);
        float ub, iub;
        block_scale(I, ub, iub);
        if (isM)
            each(acc, I * kSub, J * kSub, [&](int r, int col, float x, float y) { put_m(r, col, (x * qi[r]) * (2.f * iub), (y * qi[r]) * (2.f * iub)); });
        else
            each(acc, I * kSub, J * kSub, [&](int r, int col, float x, float y) {
                const float f = beta[r] * (kDown * iub);
                *reinterpret_cast<float2 *>(A + r * kLdA + col) = make_float2(f * x, f * y);
            });
    }
    for (int e = tid; e < kNB * 128; e += kT) {  // two neighbouring columns of one row
        const int I = e >> 7, r = (e >> 3) & 15, c0 = 2 * (e & 7);
        const float *p0 = X + kWB * I * 256;
        float P[2], M[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int i0 = c0 + j, i = i0 < 8 ? i0 : 15 - i0;
            P[j] = M[j] = 0.f;
            if (r >= i0) {  // place of (r, i0) in the column's list: M of the diagonal first, then P, M of each row
                const int n = i * 32 + (i0 < 8 ? 0 : 31 - 2 * i) + (r > i0 ? 2 * (r - i0) : 0);
#pragma unroll
                for (int w = 0; w < kWB; ++w) {
                    M[j] += p0[w * 256 + n];
                    if (r > i0) P[j] += p0[w * 256 + n - 1];
                }
            }
        }
        put_m(I * kSub + r, I * kSub + c0, M[0], M[1]);
        const float f = beta[I * kSub + r];
        *reinterpret_cast<float2 *>(A + (I * kSub + r) * kLdA + I * kSub + c0) = make_float2(f * P[0], f * P[1]);
    }
    for (int e = tid; e < kC * kC / 2; e += kT) {
        const int r = e / (kC / 2), c0 = 2 * (e % (kC / 2));
        if (c0 / kSub > r / kSub) put_m(r, c0, 0.f, 0.f);
    }
    // do meets q and M with tokens as the summed index, so it takes the inverse of their scales
    auto per_q = [&](int r) { return qi[r]; };
    if (BWD) gt.largest(gmax, per_q);
    __syncthreads();
    // the first four warps start on the inverse while the others split v and do
    invert_blocks<kT>(A, X);
    vt.put(VP, vmax, one);
    if (BWD) gt.put(GO, gmax, per_q);
    __syncthreads();
    invert_join<16, kT>(A, X, reinterpret_cast<float *>(KR));
    invert_join<32, kT>(A, X, reinterpret_cast<float *>(KR));
    // Row r of X is beta_r at most, but for the 1 on the diagonal: X diag(beta) with a scale for each row, found
    // from its beta, keeps its bits however small the betas are.
    for (int e = tid; e < kC * kC / 2; e += kT) {
        const int r = e / (kC / 2), c0 = 2 * (e % (kC / 2));
        const float2 x = *reinterpret_cast<const float2 *>(X + r * kLdA + c0);
        planes::put2<planes::H, kC>(XB, kC * kC, r, c0, x.x * (beta[c0] * sb[r]), x.y * (beta[c0 + 1] * sb[r]));
        if (BWD) {
            if (BF) planes::put2<planes::B, kC>(static_cast<uint16_t *>(a.x) + slot * 2 * kC * kC, kC * kC, r, c0, x.x, x.y);
            else *reinterpret_cast<float2 *>(static_cast<float *>(a.x) + slot * kC * kC + tile::at<kC>(r, c0)) = x;
        }
    }
    // the blocks' totals, with the change of scale from the block's successor to the block
    for (int e = tid; e < kNB * DK; e += kT) {
        const int b = e / DK;
        float u0, i0, u1 = 1.f, i1 = 1.f;
        block_scale(b, u0, i0);
        if (b + 1 < kNB) block_scale(b + 1, u1, i1);
        tot[e] = (exp2a(tot[e]) * i1) * u0;
    }
    __syncthreads();
    // ---- Kx = X diag(beta) (g k^): rows I, 32 channels; the blocks before each other multiplied in on the way
    float u0, iu0;
    block_scale(0, u0, iu0);
    // Every row of Kx has its beta and the decay of the chunk's first token as factors: scaled by the largest of
    // both, which keeps them below 2^15 (2^-120: so that ks is a normal number).
    float pk;
    {
        float s, is;
        planes::scale_of(warp_max(fmaxf(beta[lane], beta[lane + 32])), s, is);
        pk = fminf(s * (1.f / 32768.f), iu0 * 0x1p120f);
        if (tid == 0) a.gc[slot * (DK + 4) + DK] = iu0 / pk;
    }
    {
        uint16_t *kx = a.kx + slot * 2 * kC * DK;
        for (int p = warp; p < kNB * (DK / 32); p += kW) {
            const int I = p / (DK / 32), n0 = (p % (DK / 32)) * 32;
            float acc[4][4];
            zero(acc);
            for (int J = I; J >= 0; --J) {
                if (J < I) scale_columns(acc, tot + J * DK, n0);
                mma_step<planes::H, false, kC, false, kC, true, 4>(acc, XB, kC * kC, I * kSub, J * kSub, KL, kC * DK, n0, J * kSub);
            }
            each(acc, I * kSub, n0, [&](int r, int col, float x, float y) {
                planes::put2<planes::H, kC>(kx, kC * DK, r, col, (x * ib[r]) * pk, (y * ib[r]) * pk);
            });
        }
    }
    // the inverses of the scales of value columns m0 + g and m0 + g + 8
    auto inverses = [&](const uint32_t *m, int m0) {
        float s, i0, i1;
        planes::scale_of(__uint_as_float(m[vt.place(m0 + (lane >> 2))]), s, i0);
        planes::scale_of(__uint_as_float(m[vt.place(m0 + (lane >> 2) + 8)]), s, i1);
        return make_float2(i0, i1);
    };
    // ---- Uv, transposed: 16 value columns, 32 tokens
    {
        float *u = a.u + slot * kC * DV;
        for (int p = warp; p < DV / 8; p += kW) {
            const int m0 = (p >> 1) * 16, n0 = (p & 1) * 32;
            float acc[4][4];
            zero(acc);
            for (int kk = 0; kk < n0 + 32; kk += 16)
                mma_step<planes::H, BF, kC, true, kC, false, 4>(acc, VP, kC * DV, m0, kk, XB, kC * kC, n0, kk);
            const float2 iv = inverses(vmax, m0);
            each(acc, m0, n0, [&](int r, int col, float x, float y) {
                const float i = r & 8 ? iv.y : iv.x;
                store2(u + tile::at<kC>(r, col), (x * ib[col]) * i, (y * ib[col + 1]) * i);
            });
        }
    }
    if (BWD) {
        float *du = a.du + slot * kC * DV, *gh = a.gh + slot * DK * DV;
        const float outq = iu0 * 32768.f;
        for (int p = warp; p < DV / 8; p += kW) {  // (M^T do)^T
            const int m0 = (p >> 1) * 16, n0 = (p & 1) * 32;
            float acc[4][4];
            zero(acc);
            for (int kk = n0; kk < kC; kk += 16)
                mma_step<planes::H, BF, kC, true, kC, true, 4>(acc, GO, kC * DV, m0, kk, MP, kC * kC, n0, kk);
            const float2 ig = inverses(gmax, m0);
            each(acc, m0, n0, [&](int r, int col, float x, float y) {
                const float i = (r & 8 ? ig.y : ig.x) * 16.f;
                store2(du + tile::at<kC>(r, col), x * i, y * i);
            });
        }
        for (int p = warp; p < (DV / 16) * (DK / 64); p += kW) {  // ((g q)^T do)^T
            const int m0 = (p % (DV / 16)) * 16, n0 = (p / (DV / 16)) * 64;
            float acc[8][4];
            zero(acc);
            for (int J = kNB - 1; J >= 0; --J) {
                if (J < kNB - 1) scale_columns(acc, tot + J * DK, n0);
                mma_step<planes::H, BF, kC, true, kC, true, 8>(acc, GO, kC * DV, m0, J * kSub, QL, kC * DK, n0, J * kSub);
            }
            const float2 ig = inverses(gmax, m0);
            each(acc, m0, n0, [&](int r, int col, float x, float y) {
                const float i = (r & 8 ? ig.y : ig.x) * outq;
                store2(gh + tile::at<DK>(r, col), x * i, y * i);
            });
        }
    }
}

}  // namespace scan
}  // namespace kda
