// norm.cu -- the residual's addition, root-mean-square norm and 8-bit output in one pass, and the
// gradient.
//
//   r = round(x + residual),  rstd = (mean_j r_j^2 + eps)^-1/2,  y_j = w_j rstd r_j
//   per group of 128 columns: scale = max |y| / 448, 2^-126 at least (1 for a group of zeros), y8 = E4M3(y / scale)
// A thread block takes one row and keeps it in registers between the sum of squares and the
// outputs, so x and the residual are read once and every output written once: the kernel is bound
// by those bytes (8192 x 6144 in bfloat16 with both outputs: 78 us, 5.8 TB/s).  The norm is taken
// of the rounded residual, which is what a later layer and the backward pass see.  y8 is rounded
// from the fp32 y, not from its bf16 rounding.
//
//   n = rstd r,  dn = w dy,  dr = rstd (dn - n mean_j(dn_j n_j)) + dresidual,  dw = sum_rows dy n
// The blocks of the backward pass walk the rows with a fixed stride and keep their share of dw in
// registers; the shares are summed by a second kernel in a fixed order (no atomics: the same call
// gives the same bits).  8192 x 4096 in bfloat16: 53 us with the second kernel, 5.0 TB/s.
#include "norm.cuh"

namespace kda {
namespace norm {
namespace {

constexpr int kVec = 8;      // columns of a thread at a time: one 16-byte access in bf16
constexpr int kGroup = 128;  // columns that share a scale: 16 threads
constexpr int kSms = 148;

// (plain loads: an output may be the input itself)
__device__ __forceinline__ void unpack8(uint4 v, float (&x)[8])
{
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8])
{
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ void store8(float *p, const float (&x)[8])
{
    reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&x)[8]) { *reinterpret_cast<uint4 *>(p) = pack8(x); }
// x as its type holds it
__device__ __forceinline__ void round8(const float *, float (&)[8]) {}
__device__ __forceinline__ void round8(const __nv_bfloat16 *, float (&x)[8])
{
    unpack8(pack8(x), x);
}

// The block's sum of x, the same bits in every thread (warps in order).
__device__ __forceinline__ float block_sum(float x, float *warps)
{
    x = warp_sum(x);
    const int n = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = x;
    __syncthreads();
    float s = 0.f;
    for (int w = 0; w < n; ++w) s += warps[w];
    return s;
}

// 8 elements as they are in memory
template <typename T>
struct Raw {
    static constexpr int N = sizeof(T) / 2;
    uint4 v[N];
    __device__ __forceinline__ void load(const T *p)
    {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = reinterpret_cast<const uint4 *>(p)[i];
    }
    __device__ __forceinline__ void get(float (&x)[8]) const
    {
        if (N == 1) {
            unpack8(v[0], x);
        } else {
            const uint32_t u[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[N - 1].x, v[N - 1].y, v[N - 1].z, v[N - 1].w};
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(u[j]);
        }
    }
};

// MT: the most threads that the form is started with.
template <typename TX, typename TR, int IT, int MT>
__global__ void __launch_bounds__(MT) k_norm(Args a)
{
    __shared__ float warps[32];
    const long long row = blockIdx.x;
    const int tid = threadIdx.x, nt = blockDim.x;
    const TX *x = static_cast<const TX *>(a.x) + row * a.hidden;
    const TR *res = static_cast<const TR *>(a.residual) + row * a.hidden;
    TR *ro = static_cast<TR *>(a.residual_out) + row * a.hidden;
    float r[IT][kVec];
    Raw<TX> rx[IT];
    Raw<TR> rr[IT];
    uint4 wv[IT];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < IT; ++i) {  // every load of the row before the first use
        const int c = (i * nt + tid) * kVec;
        if (c < a.hidden) {
            rx[i].load(x + c);
            if (a.residual) rr[i].load(res + c);
            wv[i] = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.weight) + c);
        }
    }
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int c = (i * nt + tid) * kVec;
#pragma unroll
        for (int j = 0; j < kVec; ++j) r[i][j] = 0.f;
        if (c < a.hidden) {
            float y[kVec];
            rx[i].get(r[i]);
            if (a.residual) {
                rr[i].get(y);
#pragma unroll
                for (int j = 0; j < kVec; ++j) r[i][j] += y[j];
            }
            round8(ro, r[i]);
#pragma unroll
            for (int j = 0; j < kVec; ++j) ss = fmaf(r[i][j], r[i][j], ss);
        }
    }
    ss = block_sum(ss, warps);
    const float rstd = 1.f / sqrtf(ss / (float)a.hidden + a.eps);
    if (a.rstd && tid == 0) a.rstd[row] = rstd;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int c = (i * nt + tid) * kVec;
        const bool in = c < a.hidden;
        float y[kVec], m = 0.f;
#pragma unroll
        for (int j = 0; j < kVec; ++j) y[j] = 0.f;
        if (in) {
            store8(ro + c, r[i]);
            unpack8(wv[i], y);
#pragma unroll
            for (int j = 0; j < kVec; ++j) y[j] *= r[i][j] * rstd;
            if (a.y) store8(static_cast<__nv_bfloat16 *>(a.y) + row * a.hidden + c, y);
        }
        if (a.y8) {  // the same for the whole block
#pragma unroll
            for (int j = 0; j < kVec; ++j) m = fmaxf(m, fabsf(y[j]));  // a NaN is left out here and kept in its code
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            const float scale = m > 0.f ? fmaxf(m / 448.f, 0x1p-126f) : 1.f;  // a normal number
            if (in) {
                // y / scale by the reciprocal and one correction with the remainder (Markstein, IBM J. Res. Dev. 34,
                // 1990): the rounded quotient, as long as the remainder is no subnormal number; so tiny groups are
                // scaled up first.  A division for each element made the kernel 11 % slower (73 -> 81 us).
                const bool tiny = scale < 0x1p-90f;
                const float s = tiny ? scale * 0x1p64f : scale, inv = 1.f / s;
                if (tiny)
#pragma unroll
                    for (int j = 0; j < kVec; ++j) y[j] *= 0x1p64f;
#pragma unroll
                for (int j = 0; j < kVec; ++j) {
                    const float q = y[j] * inv;
                    y[j] = fmaf(-fmaf(q, s, -y[j]), inv, q);  // (in this order a zero keeps its sign)
                }
                uint32_t u[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * j], y[4 * j + 1]), __NV_SATFINITE, __NV_E4M3);
                    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * j + 2], y[4 * j + 3]), __NV_SATFINITE, __NV_E4M3);
                    u[j] = lo | hi << 16;
                }
                *reinterpret_cast<uint2 *>(a.y8 + row * a.hidden + c) = make_uint2(u[0], u[1]);
                if ((tid & 15) == 0) a.scale[row * (a.hidden / kGroup) + c / kGroup] = scale;
            }
        }
    }
}

// A block's next row is loaded while the current one is summed and written.
template <typename TR, int IT, int MT>
__global__ void __launch_bounds__(MT) k_norm_grad(GradArgs a, int nparts)
{
    __shared__ float warps[2][32];
    const int tid = threadIdx.x, nt = blockDim.x;
    float dw[IT][kVec];
    uint4 wv[IT];
    Raw<TR> nr[IT], ne[IT];
    Raw<__nv_bfloat16> ny[IT];
    float nrstd = 0.f;
    auto fetch = [&](long long row) {
        if (row >= a.rows) return;
        nrstd = a.rstd[row];
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int c = (i * nt + tid) * kVec;
            if (c >= a.hidden) continue;
            nr[i].load(static_cast<const TR *>(a.residual) + row * a.hidden + c);
            ny[i].load(static_cast<const __nv_bfloat16 *>(a.dy) + row * a.hidden + c);
            if (a.dres) ne[i].load(static_cast<const TR *>(a.dres) + row * a.hidden + c);
        }
    };
#pragma unroll
    for (int i = 0; i < IT; ++i) {
#pragma unroll
        for (int j = 0; j < kVec; ++j) dw[i][j] = 0.f;
        const int c = (i * nt + tid) * kVec;
        wv[i] = c < a.hidden ? *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.weight) + c) : make_uint4(0, 0, 0, 0);
    }
    fetch(blockIdx.x);
    int flip = 0;
    for (long long row = blockIdx.x; row < a.rows; row += nparts, flip ^= 1) {
        const float rstd = nrstd;
        float n[IT][kVec], dn[IT][kVec], dot = 0.f;
        Raw<TR> ce[IT];
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int c = (i * nt + tid) * kVec;
#pragma unroll
            for (int j = 0; j < kVec; ++j) n[i][j] = dn[i][j] = 0.f;
            if (c < a.hidden) {
                float w[kVec];
                nr[i].get(n[i]);
                ny[i].get(dn[i]);
                ce[i] = ne[i];
                unpack8(wv[i], w);
#pragma unroll
                for (int j = 0; j < kVec; ++j) {
                    n[i][j] *= rstd;
                    dw[i][j] = fmaf(dn[i][j], n[i][j], dw[i][j]);
                    dn[i][j] *= w[j];
                    dot = fmaf(dn[i][j], n[i][j], dot);
                }
            }
        }
        fetch(row + nparts);
        dot = block_sum(dot, warps[flip]) / (float)a.hidden;  // two buffers: one barrier per row is enough
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int c = (i * nt + tid) * kVec;
            if (c < a.hidden) {
                float d[kVec];
#pragma unroll
                for (int j = 0; j < kVec; ++j) d[j] = 0.f;
                if (a.dres) ce[i].get(d);
#pragma unroll
                for (int j = 0; j < kVec; ++j) d[j] = fmaf(rstd, dn[i][j] - n[i][j] * dot, d[j]);
                store8(static_cast<TR *>(a.dres_out) + row * a.hidden + c, d);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int c = (i * nt + tid) * kVec;
        if (c < a.hidden) store8(a.parts + (size_t)blockIdx.x * a.hidden + c, dw[i]);
    }
}

// dw[c] = sum of the blocks' shares: 32 columns per block, 8 rows of threads over the shares.
__global__ void __launch_bounds__(256) k_norm_dweight(const float *parts, int nparts, int hidden, float *dw)
{
    __shared__ float s[8][32];
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), w = threadIdx.x >> 5;
    float x = 0.f;
    for (int p = w; p < nparts; p += 8) x += parts[(size_t)p * hidden + c];
    s[w][threadIdx.x & 31] = x;
    __syncthreads();
    if (w == 0) {
        x = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) x += s[i][threadIdx.x];
        dw[c] = x;
    }
}

// Threads of a block, and the 16-byte pieces of a row that each has.  Eight pieces do not fit the registers in the
// gradient, nor at 1024 threads forward: rows of more than 8192 columns backward and 16,384 forward keep part of
// theirs in local memory.  Many rows: blocks of at most 256
// threads, so that several are resident and one's barrier is covered by the others' loads.  Few rows
// (less than two for each SM): as wide as the row allows, which is the shorter path.
struct Shape { int threads, pieces; };
Shape shape_for(int hidden, bool few)
{
    const int vec = hidden / kVec;
    int it = few && vec <= 1024 ? 1 : (vec + 255) / 256;
    if (it > 4) it = 8;
    return {((vec + it - 1) / it + 31) / 32 * 32, it};
}

template <typename TX, typename TR>
cudaError_t launch_norm(const Args &a, cudaStream_t st)
{
    const Shape p = shape_for(a.hidden, a.rows < 2 * kSms);
    const unsigned grid = (unsigned)a.rows;
    switch (p.pieces) {
    case 1: k_norm<TX, TR, 1, 1024><<<grid, p.threads, 0, st>>>(a); break;
    case 2: k_norm<TX, TR, 2, 256><<<grid, p.threads, 0, st>>>(a); break;
    case 3: k_norm<TX, TR, 3, 256><<<grid, p.threads, 0, st>>>(a); break;
    case 4: k_norm<TX, TR, 4, 256><<<grid, p.threads, 0, st>>>(a); break;
    default:
        if (p.threads <= 256) k_norm<TX, TR, 8, 256><<<grid, p.threads, 0, st>>>(a);
        else k_norm<TX, TR, 8, 1024><<<grid, p.threads, 0, st>>>(a);
    }
    return cudaGetLastError();
}

template <typename TR>
cudaError_t launch_grad(const GradArgs &a, int parts, cudaStream_t st)
{
    const Shape p = shape_for(a.hidden, a.rows < 2 * kSms);
    switch (p.pieces) {
    case 1: k_norm_grad<TR, 1, 1024><<<parts, p.threads, 0, st>>>(a, parts); break;
    case 2: k_norm_grad<TR, 2, 256><<<parts, p.threads, 0, st>>>(a, parts); break;
    case 3: k_norm_grad<TR, 3, 256><<<parts, p.threads, 0, st>>>(a, parts); break;
    case 4: k_norm_grad<TR, 4, 256><<<parts, p.threads, 0, st>>>(a, parts); break;
    default:
        if (p.threads <= 256) k_norm_grad<TR, 8, 256><<<parts, p.threads, 0, st>>>(a, parts);
        else k_norm_grad<TR, 8, 1024><<<parts, p.threads, 0, st>>>(a, parts);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t forward(const Args &a, bool x_bf16, bool res_bf16, cudaStream_t st)
{
    if (x_bf16 && res_bf16) return launch_norm<__nv_bfloat16, __nv_bfloat16>(a, st);
    if (x_bf16) return launch_norm<__nv_bfloat16, float>(a, st);
    if (res_bf16) return launch_norm<float, __nv_bfloat16>(a, st);
    return launch_norm<float, float>(a, st);
}

int grad_parts(long long rows, int hidden, int sms)
{
    // about as many blocks as are resident at once
    const Shape p = shape_for(hidden, rows < 2 * kSms);
    const long long n = (long long)sms * (p.threads > 512 || p.pieces > 2 ? 1 : p.pieces == 2 || p.threads > 256 ? 2 : 4);
    return (int)(rows < n ? rows : n);
}

cudaError_t backward(const GradArgs &a, bool res_bf16, int parts, cudaStream_t st)
{
    cudaError_t e = cudaSuccess;
    if (parts > 0) e = res_bf16 ? launch_grad<__nv_bfloat16>(a, parts, st) : launch_grad<float>(a, parts, st);
    if (e != cudaSuccess) return e;
    k_norm_dweight<<<a.hidden / 32, 256, 0, st>>>(a.parts, parts, a.hidden, a.dweight);
    return cudaGetLastError();
}

}  // namespace norm
}  // namespace kda
