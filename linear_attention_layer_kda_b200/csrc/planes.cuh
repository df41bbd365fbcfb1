// planes.cuh -- products on the tensor cores to more than 16 bits, from operands that are split once.
//
// A matrix is kept as two planes of 16-bit numbers, x = hi + lo, and a product is
// hi*hi + hi*lo + lo*hi with fp32 accumulation.  Splitting when a tile is written, not when a
// fragment is read, leaves the inner loops with ldmatrix and mma only; the planes take the 4 bytes
// of an fp32 element, and their m16n8k16 products run at twice the rate of TF32 ones.
//   half planes      22 bits: what is left out is 2^-22 of an element, as long as it is not
//                    below 2^-27 of the largest that the scale allows (fp16's range: the
//                    remainder's unit is 2^-24).  Used, with a power of two as scale, for whatever
//                    feeds an fp32 state.
//   bfloat16 planes  16 bits, fp32's range, no scale.  Used for what is rounded to bfloat16 next
//                    (half a step: 2^-8).
// A plane of R rows is made of slabs of 64 columns, each [R][64] with 128-byte rows whose 16-byte
// pieces are permuted by piece ^= row & 7: ldmatrix then reads eight rows without bank conflicts,
// whether k runs along the rows or along the columns.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace kda {
namespace planes {

// Element (r, c) of a plane of R rows.
template <int R>
__device__ __forceinline__ int at(int r, int c)
{
    return (c >> 6) * (R * 64) + r * 64 + ((((c >> 3) ^ r) & 7) << 3) + (c & 7);
}

__device__ __forceinline__ uint32_t saddr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t a)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a));
}
__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t a)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a));
}

// Four 8 x 8 matrices from the registers of an accumulator's layout (lane (g, t): row g, columns 2 t, 2 t + 1).
__device__ __forceinline__ void stsm(uint32_t a, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3)
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(r0), "r"(r1), "r"(r2), "r"(r3)
                 : "memory");
}

// Fragments of the 16 x 16 tile at (mn0, k0) of an operand: A's a0..a3, or B's b0, b1 of two
// neighbouring n tiles.  KROW false: element (mn, k) is row mn, column k of the plane; true: row k,
// column mn.
template <int R, bool KROW>
__device__ __forceinline__ void frag_a(uint32_t (&r)[4], const void *plane, int m0, int k0)
{
    const int l = threadIdx.x & 31;
    if (KROW) ldsm_t(r, saddr(plane) + 2 * at<R>(k0 + (l & 7) + ((l >> 4) << 3), m0 + (l & 8)));
    else ldsm(r, saddr(plane) + 2 * at<R>(m0 + (l & 15), k0 + ((l >> 4) << 3)));
}
template <int R, bool KROW>
__device__ __forceinline__ void frag_b(uint32_t (&r)[4], const void *plane, int n0, int k0)
{
    const int l = threadIdx.x & 31;
    if (KROW) ldsm_t(r, saddr(plane) + 2 * at<R>(k0 + (l & 15), n0 + ((l >> 4) << 3)));
    else ldsm(r, saddr(plane) + 2 * at<R>(n0 + (l & 7) + ((l >> 4) << 3), k0 + (l & 8)));
}

// The two 16-bit types.
struct H {
    static __device__ __forceinline__ uint32_t pack(float x, float y)
    {
        const __half2 h = __floats2half2_rn(x, y);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    static __device__ __forceinline__ float2 unpack(uint32_t u) { return __half22float2(*reinterpret_cast<const __half2 *>(&u)); }
    static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
    {
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};
struct B {
    static __device__ __forceinline__ uint32_t pack(float x, float y)
    {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    static __device__ __forceinline__ float2 unpack(uint32_t u)
    {
        return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    }
    static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
    {
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};

template <class P>
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo)
{
    hi = P::pack(x, y);
    const float2 f = P::unpack(hi);
    lo = P::pack(x - f.x, y - f.y);
}

// Elements (r, c) and (r, c + 1), c even, into the planes at p (the low plane n elements further).
template <class P, int R>
__device__ __forceinline__ void put2(uint16_t *p, int n, int r, int c, float x, float y)
{
    uint32_t hi, lo;
    split2<P>(x, y, hi, lo);
    uint16_t *q = p + at<R>(r, c);
    *reinterpret_cast<uint32_t *>(q) = hi;
    *reinterpret_cast<uint32_t *>(q + n) = lo;
}

// acc of NT n tiles += A (fragments) B (fragments of pairs of n tiles), the three products.
template <class P>
__device__ __forceinline__ void mma3(float (&c0)[4], float (&c1)[4], const uint32_t (&ah)[4], const uint32_t (&al)[4],
                                     const uint32_t (&bh)[4], const uint32_t (&bl)[4])
{
    P::mma(c0, al, bh[0], bh[1]);
    P::mma(c1, al, bh[2], bh[3]);
    P::mma(c0, ah, bl[0], bl[1]);
    P::mma(c1, ah, bl[2], bl[3]);
    P::mma(c0, ah, bh[0], bh[1]);
    P::mma(c1, ah, bh[2], bh[3]);
}

// The same for N pairs of n tiles, one product after the other over all of them: no accumulator waits
// for its last product.
template <class P, int N>
__device__ __forceinline__ void mma3_wide(float (&c)[2 * N][4], const uint32_t (&ah)[4], const uint32_t (&al)[4],
                                          const uint32_t (&bh)[N][4], const uint32_t (&bl)[N][4])
{
#pragma unroll
    for (int n = 0; n < N; ++n) P::mma(c[2 * n], al, bh[n][0], bh[n][1]), P::mma(c[2 * n + 1], al, bh[n][2], bh[n][3]);
#pragma unroll
    for (int n = 0; n < N; ++n) P::mma(c[2 * n], ah, bl[n][0], bl[n][1]), P::mma(c[2 * n + 1], ah, bl[n][2], bl[n][3]);
#pragma unroll
    for (int n = 0; n < N; ++n) P::mma(c[2 * n], ah, bh[n][0], bh[n][1]), P::mma(c[2 * n + 1], ah, bh[n][2], bh[n][3]);
}

// A power of two that brings values of size up to m to [2^14, 2^15), and its inverse.  Values below
// 2^-99 count as 2^-99.  Where m is not finite nothing that shares the scale can be told from zero: the
// inverse is NaN.
__device__ __forceinline__ void scale_of(float m, float &s, float &inv)
{
    const int e = max((int)(__float_as_uint(m) >> 23) & 255, 28);
    s = __uint_as_float((uint32_t)(268 - e) << 23);
    inv = __uint_as_float(e == 255 ? 0x7fc00000u : (uint32_t)(e - 14) << 23);
}
// for values of size up to 1
constexpr float kUp = 16384.f, kDown = 1.f / 16384.f;

}  // namespace planes
}  // namespace kda
