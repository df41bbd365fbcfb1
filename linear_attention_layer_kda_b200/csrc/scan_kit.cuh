// scan_kit.cuh -- operands of the outputs' and the gradients' products, by the activations' type.
#pragma once

#include "scan_prep.cuh"

namespace kda {
namespace scan {

// How an operand of R rows and C columns is kept and multiplied: bfloat16 planes for bfloat16
// activations, fp32 tiles and three TF32 products for fp32 (the same bytes, half the rate and three
// times the instructions).  `step` is 16 deep; EXACT: the operand is a bfloat16 number, one plane.
template <typename T>
struct Kit {  // bfloat16
    using E = uint16_t;
    template <int R, int C>
    static __device__ __forceinline__ void put2(E *p, int r, int c, float x, float y) { planes::put2<planes::B, R>(p, R * C, r, c, x, y); }
    template <int R, int C>
    static __device__ __forceinline__ void put1(E *p, int r, int c, float x) { scan::put1<planes::B, R>(p, R * C, r, c, x); }
    template <int R, int C>
    static __device__ __forceinline__ float2 get2(const E *p, int r, int c)
    {
        const E *q = p + planes::at<R>(r, c);
        const float2 x = planes::B::unpack(*reinterpret_cast<const uint32_t *>(q)), y = planes::B::unpack(*reinterpret_cast<const uint32_t *>(q + R * C));
        return make_float2(x.x + y.x, x.y + y.y);
    }
    template <bool EXACT, int RA, int CA, bool KA, int RB, int CB, bool KB, int NT>
    static __device__ __forceinline__ void step(float (&acc)[NT][4], const E *A, int m0, int ka, const E *Bp, int n0, int kb)
    {
        mma_step<planes::B, EXACT, RA, KA, RB, KB, NT>(acc, A, RA * CA, m0, ka, Bp, RB * CB, n0, kb);
    }
};
template <>
struct Kit<float> {
    using E = float;
    template <int R, int C>
    static __device__ __forceinline__ void put2(E *p, int r, int c, float x, float y) { store2(p + tile::at<C>(r, c), x, y); }
    template <int R, int C>
    static __device__ __forceinline__ void put1(E *p, int r, int c, float x) { p[tile::at<C>(r, c)] = x; }
    template <int R, int C>
    static __device__ __forceinline__ float2 get2(const E *p, int r, int c) { return *reinterpret_cast<const float2 *>(p + tile::at<C>(r, c)); }
    template <bool EXACT, int RA, int CA, bool KA, int RB, int CB, bool KB, int NT>
    static __device__ __forceinline__ void step(float (&acc)[NT][4], const E *A, int m0, int ka, const E *Bp, int n0, int kb)
    {
        float(&c)[1][NT][4] = reinterpret_cast<float(&)[1][NT][4]>(acc);
        // k offsets of the two operands differ by their tiles' first rows
        tile::mma<1, NT>(c, Shift<tile::Op<CA, KA>>{{A}, ka}, m0, Shift<tile::Op<CB, KB>>{{Bp}, kb}, n0, 0, 16);
    }
    template <class O>
    struct Shift {
        O o;
        int k;
        __device__ __forceinline__ void load(int mn0, int k0, int g, int t, float &x0, float &x1) const { o.load(mn0, k + k0, g, t, x0, x1); }
    };
};

}  // namespace scan
}  // namespace kda
