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
// Blocks.  A chunk has four blocks of kSub tokens.  Decays are kept per block: GL_t = gamma(t, block's
// start), GR_t = gamma(block's end, t) and the blocks' totals, each the exponential of a sum of
// logarithms that starts inside the block (no difference of large numbers is ever taken).  With them
// gamma(t, i) = GL_t (totals between) GR_i for tokens of different blocks, all factors at most 1, which
// makes P, M and their gradients matrix products; tokens of one block are taken pair by pair, the decay
// multiplied up token by token.  So no decay is ever divided by, however strong it is.
//
// The products: what feeds the fp32 states goes through half planes (22 bits, planes.cuh); for
// bfloat16 activations, what is rounded to bfloat16 next (o and the gradients) through bfloat16
// planes (16 bits against a rounding of 8).  fp32 outputs and gradients of them use three TF32
// products of fp32 tiles (tile_mma.cuh).
#pragma once

#include "common.cuh"
#include "planes.cuh"
#include "sm100.cuh"
#include "tile_mma.cuh"

namespace kda {
namespace scan {

constexpr int kC = 64;        // tokens per chunk
constexpr int kSub = 16;      // tokens per block of a chunk
constexpr int kNB = kC / kSub;
constexpr int kThreads = 256;
constexpr float kFloor2 = -87.f;  // of log2 alpha: alpha^1.4 is still a normal number

struct Args {
    int nh, nseq, max_chunks;
    int chunk_seqs;        // sequences that can have chunks
    long long rows;
    int tokens;            // tokens per sequence where all have the same (cu null)
    const int *cu;         // [nseq + 1] first rows, or null
    const int *pre;        // [nseq + 1] first chunks (with cu)
    const int *list;       // [nseq + 1] the sequences that have chunks, and their number; null: all
    int short_tokens;      // sequences of up to this many tokens go token by token and have no chunks
    const void *q, *k, *v, *z, *b;
    long long ldq, ldk, ldv, ldz, ldb;  // elements between rows
    const float *state0;   // [nseq, nh, dk, dv] or null (zeros)
    // per chunk and head, in the workspace (tiles as the kernels read them)
    uint16_t *kx, *w;      // half planes [kC][dk]; W times 1 / ws, Kx times 1 / ks
    float *gc;             // [dk + 4]: the chunk's decay, ks, ws.  Every row of Kx has its beta and the decay of the chunk's
                           // first token as factors; ks is a power of two near the product of the largest of both.
                           // ws is 2^-14 times what the tokens behind the chunk's last key leave of W
    void *qb, *m;          // g q [kC][dk] and M [kC][kC]: bfloat16 planes, or fp32 tiles
    float *u;              // tile [dv][kC]: Uv; then U for fp32 activations
    uint16_t *up;          // bfloat16 planes [dv][kC] of U, for bfloat16 activations
    void *h;               // S before the chunk, transposed [dv][dk]: bfloat16 planes, or an fp32 tile
    void *x;               // X [kC][kC] (only for the backward pass): bfloat16 planes, or an fp32 tile
    float *inv;            // [kC]: 1 / |k| or 0 (only for the backward pass)
    void *o;
    float *state_out;
    // backward
    const void *go;        // gradient of o, dense
    const float *gstate;   // gradient of state_out or null (zeros)
    float *du, *gh;        // tiles [dv][kC]: M^T go; [dv][dk]: (g q)^T go; for fp32 then dU and the gradient of S'
    uint16_t *dup, *ghp;   // bfloat16 planes of dU and of the gradient of S', for bfloat16 activations
    void *dq, *dk, *dv, *dz, *db;
    float *dstate0;        // or null
    uint64_t wait_ns;      // the longest that a wait for a copy may take
    int skip_copies;       // a test of that: the copies are not issued
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

__device__ __forceinline__ float exp2a(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// log2 alpha = -log2(1 + e^z), held at kFloor2.  With x = e^-|z|: log2(1 + x) by its series where 1 + x would
// round x away (relative error 2^-21), else by the hardware's logarithm (absolute error 2^-22).
__device__ __forceinline__ float log2_alpha(float z)
{
    constexpr float kL = 1.44269504f;
    const float x = exp2a(-kL * fabsf(z));
    float l = x * kL * fmaf(x, fmaf(x, fmaf(x, -0.25f, 0.333333333f), -0.5f), 1.f);
    if (!(x < 0.03125f)) asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(l) : "f"(1.f + x));
    l = -(l + kL * fmaxf(z, 0.f));
    return l < kFloor2 ? kFloor2 : l;  // keeps a NaN
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

// The sum over the warp's lanes of each of 32 values: lane l returns the one of x[l].
__device__ __forceinline__ float sums32(float (&x)[32])
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const float keep = up ? x[i + o] : x[i], give = up ? x[i] : x[i + o];
            x[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
    }
    return x[0];
}
// The same for 16 values: lanes l and l + 16 return the one of x[l].
__device__ __forceinline__ float sums16(float (&x)[16])
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] += __shfl_xor_sync(0xffffffffu, x[i], 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const float keep = up ? x[i + o] : x[i], give = up ? x[i] : x[i + o];
            x[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
    }
    return x[0];
}

// Waits for a barrier's phase, a.wait_ns at most; false if it does not come (copies of memory that is there
// always arrive).  A thread that gave up goes on without further waits and turns all that it computes from
// the data into NaN; no copy is issued to a barrier whose last one is missing, and the thread that issued the
// copies waits for them once more, as long, before it leaves.
__device__ __forceinline__ bool arrived(const Args &a, uint64_t *bar, int phase)
{
    if (sm100::mbar_try_wait(bar, phase & 1)) return true;
    const uint64_t t0 = sm100::globaltimer_ns();
    do {
        if (sm100::mbar_try_wait(bar, phase & 1)) return true;
    } while (sm100::globaltimer_ns() - t0 < a.wait_ns);
    return false;
}
// The last wait for what is on its way to n barriers: of the two parities, one has passed and the other is that of
// the copies, if there are any.
__device__ __forceinline__ void drain(const Args &a, uint64_t *bar, int n)
{
#pragma unroll 1
    for (int i = 0; i < 2 * n; ++i) arrived(a, bar + i / 2, i & 1);
}
__device__ __forceinline__ float nan_f() { return __int_as_float(0x7fc00000); }
template <int NT>
__device__ __forceinline__ void make_nan(float (&acc)[NT][4])
{
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][e] = nan_f();
}

}  // namespace scan
}  // namespace kda
