// scan.cuh -- the recurrence over whole sequences (forward and backward): what its kernels share.
//
// Per head, with k^ = k / |k|, alpha_t = exp(la_t), la = -softplus(z) and beta = sigmoid(b):
//   S_t = (I - beta_t k^_t k^_t^T) diag(alpha_t) S_{t-1} + beta_t k^_t v_t^T,   o_t = S_t^T q_t.
// A sequence is cut into chunks of kC tokens.  Inside a chunk with the state S before it and the
// decays gamma(t, i) = prod_{i < j <= t} alpha_j (per key channel), g_t = gamma(t, start):
//   P[t, i] = sum_d k^_t k^_i gamma(t, i)  (i < t),   M[t, i] = sum_d q_t k^_i gamma(t, i)  (i <= t)
//   X  = (I + diag(beta) P)^-1                         unit lower triangular
//   Kx = X diag(beta) (g k^),   Uv = X diag(beta) V
//   U  = Uv - Kx S,             o  = (g q) S + M U,    S' = diag(g_C) S + W^T U,   W_t = gamma(C, t) k^_t
// Only U, o and S' need the state; all else is computed for every chunk at once.
//
// Decays are kept as sums of la inside blocks of kSub tokens (LG, restarting at each block) and
// the blocks' totals, so that the difference of two neighbouring tokens' sums is not taken between
// two large numbers.  Every factor used is exp of something <= 0, except inside one block where the
// block's middle is the reference: there a channel whose decay inside the block exceeds e^-60 sends
// that block to a loop over pairs.  la is clamped at -60: one
// such token leaves 1e-26 of a channel, and a block's sums stay below 1000, so that differences of
// neighbouring sums keep four digits even there.
#pragma once

#include "common.cuh"
#include "planes.cuh"
#include "tile_mma.cuh"

namespace kda {
namespace scan {

constexpr int kC = 64;        // tokens per chunk
constexpr int kSub = 16;      // tokens per block of a chunk
constexpr int kNB = kC / kSub;
constexpr int kThreads = 256;
constexpr float kFloor = -60.f;   // of log alpha: alpha^2 is still a normal number
constexpr float kRange = 60.f;  // largest decay inside a block that the block's middle can anchor

struct Args {
    int nh, nseq, max_chunks;
    long long rows;
    int tokens;            // tokens per sequence where all have the same (cu null)
    const int *cu;         // [nseq + 1] first rows, or null
    const int *pre;        // [nseq + 1] first chunks (with cu)
    const void *q, *k, *v, *z, *b;
    long long ldq, ldk, ldv, ldz, ldb;  // elements between rows
    const float *state0;   // [nseq, nh, dk, dv] or null (zeros)
    // per chunk and head, in the workspace (tiles as the kernels read them)
    uint16_t *kx, *w;      // half planes [kC][dk]; W times planes::kUp, Kx times 1 / ks
    float *ks;             // [1]: every Kx has the decay of the chunk's first token as a factor, so that the
                           // largest of that (a power of two near it) is what Kx is scaled by
    float *qb, *m;         // tiles [kC][dk], [kC][kC]
    float *u;              // tile [dv][kC]: Uv, then U
    float *gc;             // [dk]
    float *h;              // tile [dv][dk]: S before the chunk
    float *x;              // tile [kC][kC], only for the backward pass
    void *o;
    float *state_out;
    // backward
    const void *go;        // gradient of o, dense
    const float *gstate;   // gradient of state_out or null (zeros)
    float *du, *gh;        // du: tile [dv][kC]: M^T go, then dU; gh: tile [dv][dk]: (g q)^T go, then the gradient of S'
    void *dq, *dk, *dv, *dz, *db;
    float *dstate0;        // or null
};

struct Chunk {
    int seq;
    long long row0;  // first row
    int n;           // tokens
};

// First row of sequence s; whatever cu holds, the result stays in [0, rows].
__device__ __forceinline__ long long seq_start(const Args &a, int s)
{
    if (!a.cu) return (long long)s * a.tokens;
    const long long r = a.cu[s];
    return r < 0 ? 0 : r > a.rows ? a.rows : r;
}
__device__ __forceinline__ long long seq_end(const Args &a, int s)
{
    const long long b = seq_start(a, s), e = seq_start(a, s + 1);
    return e < b ? b : e;
}
__device__ __forceinline__ int seq_chunk0(const Args &a, int s)
{
    return a.cu ? a.pre[s] : s * ((a.tokens + kC - 1) / kC);
}

__device__ __forceinline__ bool locate(const Args &a, int ci, Chunk *c)
{
    int s;
    if (!a.cu) {
        s = ci / ((a.tokens + kC - 1) / kC);
    } else {
        if (ci >= a.pre[a.nseq]) return false;
        int lo = 0, hi = a.nseq;  // last s with pre[s] <= ci: a sequence with chunks
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a.pre[mid] <= ci) lo = mid; else hi = mid;
        }
        s = lo;
    }
    c->seq = s;
    c->row0 = seq_start(a, s) + (long long)(ci - seq_chunk0(a, s)) * kC;
    const long long left = seq_end(a, s) - c->row0;
    c->n = left < kC ? (int)left : kC;
    return true;
}

__device__ __forceinline__ float log_alpha(float z)
{
    const float lz = -(fmaxf(z, 0.f) + log1pf(expf(-fabsf(z))));
    return lz < kFloor ? kFloor : lz;  // keeps a NaN
}
__device__ __forceinline__ float sigmoid(float x) { return 1.f / (1.f + expf(-x)); }

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }

__device__ __forceinline__ void load4(const float *p, float (&x)[4])
{
    const float4 v = __ldg(reinterpret_cast<const float4 *>(p));
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16 *p, float (&x)[4])
{
    const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p));
    x[0] = __uint_as_float(v.x << 16), x[1] = __uint_as_float(v.x & 0xffff0000u);
    x[2] = __uint_as_float(v.y << 16), x[3] = __uint_as_float(v.y & 0xffff0000u);
}
__device__ __forceinline__ void store2(float *p, float x, float y) { *reinterpret_cast<float2 *>(p) = make_float2(x, y); }
__device__ __forceinline__ void store2(__nv_bfloat16 *p, float x, float y)
{
    *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(x, y);
}
__device__ __forceinline__ void store1(float *p, float x) { *p = x; }
__device__ __forceinline__ void store1(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

// f(x) of D channels of the chunk's rows into a tile; rows past the chunk's end become zero.
template <int D, typename T, class F>
__device__ __forceinline__ void load_tile(float *dst, const T *src, long long ld, const Chunk &c, F f)
{
    for (int e = threadIdx.x; e < kC * (D / 4); e += kThreads) {
        const int r = e / (D / 4), c4 = 4 * (e % (D / 4));
        float x[4] = {0.f, 0.f, 0.f, 0.f};
        if (r < c.n) {
            load4(src + (c.row0 + r) * ld + c4, x);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = f(x[i]);
        }
        *reinterpret_cast<float4 *>(dst + tile::at<D>(r, c4)) = make_float4(x[0], x[1], x[2], x[3]);
    }
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

}  // namespace scan
}  // namespace kda
