// tile_mma.cuh -- products of fp32 tiles that sit in shared memory, on the tensor cores, to fp32
// accuracy: each fp32 operand x is split on the way from shared memory into its TF32 rounding hi
// and the remainder lo = x - hi, and a product is lo*hi + hi*lo + hi*hi with fp32 accumulation
// (what is left out, lo*lo and the bits of lo past TF32, is about 2^-23 of the product).
//
// Tiles are row-major with a leading dimension that is a multiple of 32 floats, and column c of
// row r sits at column c ^ swz(r).  The swizzle makes a warp's fragment loads free of bank
// conflicts whether a fragment's k index runs along the rows or along the columns of the tile, so
// one copy of a matrix serves as either operand, transposed or not; aligned groups of four columns
// stay together, so 16-byte accesses work.
#pragma once

#include <stdint.h>

namespace kda {
namespace tile {

__device__ __forceinline__ int swz(int r) { return ((r & 3) << 3) | (r & 4); }
template <int LD>
__device__ __forceinline__ int at(int r, int c) { return r * LD + (c ^ swz(r)); }

__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2])
{
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// x -> its TF32 rounding (half away from zero, in the integer bits) and the remainder.  For an
// infinity or NaN the remainder is NaN, so the product is NaN where the exact one may be infinite.
__device__ __forceinline__ void split(float x, uint32_t &hi, uint32_t &lo)
{
    hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
    lo = __float_as_uint(x - __uint_as_float(hi));
}

// An operand in a tile of leading dimension LD whose element (mn, k) is row mn, column k (KROW
// false: k runs along a row) or row k, column mn (KROW true).  mn and k offsets are multiples of 8.
template <int LD, bool KROW>
struct Op {
    const float *p;
    // elements (mn0 + g, k0 + t) and (mn0 + g, k0 + t + 4) for lane (g, t)
    __device__ __forceinline__ void load(int mn0, int k0, int g, int t, float &x0, float &x1) const
    {
        if (KROW) {
            const int c = (mn0 ^ (t << 3)) | g;
            x0 = p[(k0 + t) * LD + c];
            x1 = p[(k0 + t + 4) * LD + (c ^ 4)];
        } else {
            const float *r = p + (mn0 + g) * LD;
            const int c = k0 ^ swz(g);
            x0 = r[c + t];
            x1 = r[(c ^ 4) + t];
        }
    }
};

// acc[i][j] (+)= A[m0 + 16 i .. + 16][k0, k1) * B[k0, k1)[n0 + 8 j .. + 8]; k0, k1 multiples of 8.
// Accumulator element e of lane (g, t): row g + 8 (e / 2), column 2 t + e % 2 of its tile.
template <int MT, int NT, class OA, class OB>
__device__ __forceinline__ void mma(float (&acc)[MT][NT][4], const OA &A, int m0, const OB &B, int n0, int k0, int k1)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll 2
    for (int k = k0; k < k1; k += 8) {
        uint32_t ah[MT][4], al[MT][4];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            float x[4];
            A.load(m0 + 16 * i, k, g, t, x[0], x[2]);
            A.load(m0 + 16 * i + 8, k, g, t, x[1], x[3]);
#pragma unroll
            for (int e = 0; e < 4; ++e) split(x[e], ah[i][e], al[i][e]);
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            float y[2];
            uint32_t bh[2], bl[2];
            B.load(n0 + 8 * j, k, g, t, y[0], y[1]);
            split(y[0], bh[0], bl[0]);
            split(y[1], bh[1], bl[1]);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                mma_tf32(acc[i][j], al[i], bh);
                mma_tf32(acc[i][j], ah[i], bl);
                mma_tf32(acc[i][j], ah[i], bh);
            }
        }
    }
}

__device__ __forceinline__ void cp_async16(void *smem, const void *g)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(smem)), "l"(g)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

}  // namespace tile
}  // namespace kda
