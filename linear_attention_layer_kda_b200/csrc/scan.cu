// scan.cu -- the recurrence over whole sequences: forward (formulas in scan.cuh).
//
//   k_scan_plan    first chunk of every sequence of a ragged batch (one block)
//   k_scan_prep    per chunk and head: Kx, Uv, W, g q, M (scan_prep.cuh)
//   k_scan_state   per sequence, head and slice of value columns: U and the states, chunk by chunk;
//                  the same kernel run backwards carries the gradient of the states
//   k_scan_out     per chunk and head: o
//   k_scan_tokens  short sequences (a decode step, and those of a ragged batch): the recurrence as
//                  written, state in registers
#include "scan_kit.cuh"

namespace kda {
namespace scan {
namespace {

__global__ void __launch_bounds__(1024) k_scan_plan(Args a, int *pre, int *list)
{
    // chunk counts of 1024 sequences at a time, summed by a block scan; the total never exceeds the
    // chunks that the workspace holds, whatever cu says
    __shared__ int warps[2][32];
    __shared__ int base[2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid < 2) base[tid] = 0;
    __syncthreads();
    for (int s0 = 0; s0 < a.nseq; s0 += 1024) {
        const int s = s0 + tid;
        int n = 0;
        if (s < a.nseq) {
            const long long t = seq_end(a, s) - seq_start(a, s), c = t <= a.short_tokens ? 0 : (t + kC - 1) / kC;
            n = c > a.max_chunks ? a.max_chunks : (int)c;
        }
        int x = n, z = n > 0;  // inclusive sums; x saturates, so that repeated ranges cannot overflow
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, z, o);
            if (lane >= o) x = min(x + y, a.max_chunks), z += v;
        }
        if (lane == 31) warps[0][warp] = x, warps[1][warp] = z;
        __syncthreads();
        int before = base[0];
        z += base[1];
        for (int w = 0; w < warp; ++w) before = min(before + warps[0][w], a.max_chunks), z += warps[1][w];
        x = min(x + before, a.max_chunks);
        if (s < a.nseq) pre[s + 1] = x;
        if (list && n > 0) list[z - 1] = s;
        __syncthreads();
        if (tid == 1023) base[0] = x, base[1] = z;
        __syncthreads();
    }
    if (tid == 0) {
        pre[0] = 0;
        if (list) list[a.nseq] = base[1];
    }
}

// ---------------------------------------------------------------- the states, chunk by chunk

// Forward:   T = Uv - Kx S,      S <- g_C S + W^T T       (h: S before each chunk; u: T)
// Backward:  T = du + W dS',     dS <- g_C dS' + gh - Kx^T T    (gh: dS' of each chunk; du: T)
//
// The chain over the chunks is what cannot run in parallel, so a step is kept short.  Everything is
// held transposed: with value columns as the rows of the accumulators, the result of one product
// has the registers' layout of the next one's left operand.  S and T are split into half planes with
// a scale for each value column, found anew at each step.  Two forms:
//   WK = 4  four warps take 16 value columns and a quarter of the key channels each, so that a step is
//           short.  Their shares of T (a sum over all key channels) go through shared memory: a warp
//           adds up a quarter of the tokens, splits it (with a scale for that quarter) and passes on
//           the operand of the second product.  GR such groups share a block's copies of Kx and W.
//   WK = 1  a warp takes 16 value columns and all key channels: no exchange, one barrier for the
//           copies, half the instructions, but long steps.
// A step's factors arrive by bulk copies, issued a step ahead by one thread (as 16-byte copies of a warp,
// their 140 instructions took as long as all else in a step).
template <int DK, int DV, int WK, int GR, bool BWD>
struct StateSmem {
    static constexpr int F = 2 * kC * DK * 2;           // bytes of a factor's two planes
    static constexpr int F1 = 0, F2 = 2 * F;            // two of each
    static constexpr int T0 = F2 + 2 * F;               // [2][GR][16][kC]: Uv (du) of the group's columns
    static constexpr int GC = T0 + 2 * GR * 16 * kC * 4;                // [2][dk + 4]: the chunk's decay, ks, ws
    static constexpr int GH = GC + 2 * (DK + 4) * 4;                    // [2][GR][16][dk]: (g q)^T do of the columns
    static constexpr int RED = GH + (BWD && WK > 1 ? 2 * GR * 16 * DK * 4 : 0);  // [GR][WK][8][32] float4: shares of T
    static constexpr int AT = RED + (WK > 1 ? GR * WK * 4096 : 0);      // [GR][4][2][32] uint4: T's planes by quarters
    static constexpr int SC = AT + (WK > 1 ? GR * 4 * 1024 : 0);        // [GR][4][32] float2: their scales' inverses
    static constexpr int MB = SC + (WK > 1 ? GR * 4 * 256 : 0);         // two barriers
    static constexpr int ST = (MB + 16 + 1023) / 1024 * 1024;           // WK 1: [GR][2][16][64] planes on their way out
    static constexpr size_t bytes = WK > 1 ? MB + 16 : ST + GR * 4096;
    static_assert(bytes <= 227 * 1024, "");
    static constexpr int kThreads = 32 * (WK * GR + (WK > 1));
};

// Scales for the two value columns (rows g and g + 8 of the accumulators) whose values are x0 and x1 at most
// in this lane, and their inverses.
__device__ __forceinline__ void column_scales(float x0, float x1, float &s0, float &i0, float &s1, float &i1)
{
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
        x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, o));
        x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, o));
    }
    planes::scale_of(x0, s0, i0);
    planes::scale_of(x1, s1, i1);
}
// Two n tiles of an accumulator (16 columns of it) as a left operand's 16 x 16 tile.
__device__ __forceinline__ void split_tile(const float (&x)[4], const float (&y)[4], float s0, float s1, uint32_t (&h)[4], uint32_t (&l)[4])
{
    planes::split2<planes::H>(x[0] * s0, x[1] * s0, h[0], l[0]);
    planes::split2<planes::H>(x[2] * s1, x[3] * s1, h[1], l[1]);
    planes::split2<planes::H>(y[0] * s0, y[1] * s0, h[2], l[2]);
    planes::split2<planes::H>(y[2] * s1, y[3] * s1, h[3], l[3]);
}

template <int DK, int DV, int WK, int GR, bool BWD, bool PL>
__global__ void __launch_bounds__(StateSmem<DK, DV, WK, GR, BWD>::kThreads, 1) k_scan_state(Args a)
{
    extern __shared__ __align__(1024) char smb[];
    using L = StateSmem<DK, DV, WK, GR, BWD>;
    constexpr int kGroups = DV / (16 * GR);
    constexpr int NT = DK / WK / 8;               // n tiles of a warp's key channels
    const int h = blockIdx.x / kGroups;
    int s = blockIdx.y;
    if (!BWD && a.list) {
        if (s >= a.list[a.nseq]) return;
        s = a.list[s];
    }
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int grp = warp / WK, wk = warp % WK;
    const int col0 = ((blockIdx.x % kGroups) * GR + grp) * 16;  // the group's first value column
    const int d0 = wk * (DK / WK);                              // the warp's first key channel
    const int c0 = seq_chunk0(a, s);
    const int nc = a.cu ? a.pre[s + 1] - c0 : (a.tokens + kC - 1) / kC;
    auto slot_of = [&](int i) { return (size_t)(c0 + (BWD ? nc - 1 - i : i)) * a.nh + h; };
    // Copies in groups: group n brings the first product's factor of step n, and of step n - 1 what is
    // needed behind its first barrier: the second factor, Uv (du), decays and gh.
    uint64_t *mbar = reinterpret_cast<uint64_t *>(smb + L::MB);
    auto issue = [&](int n) {
        constexpr int kU = GR * 16 * kC * 4, kG = (DK + 4) * 4, kH = BWD && WK > 1 ? GR * 16 * DK * 4 : 0;
        const bool first = n < nc, second = n > 0 && n <= nc;
        if ((!first && !second) || a.skip_copies) return;
        uint64_t *bar = mbar + (n & 1);
        sm100::mbar_expect_tx(bar, (first ? L::F : 0) + (second ? L::F + kU + kG + kH : 0));
        if (first) sm100::bulk_load(smb + L::F1 + (n & 1) * L::F, (BWD ? a.w : a.kx) + slot_of(n) * 2 * kC * DK, L::F, bar);
        if (second) {
            const int p = (n - 1) & 1;
            const size_t slot = slot_of(n - 1), c16 = (size_t)(blockIdx.x % kGroups) * GR * 16;  // the block's first value column
            sm100::bulk_load(smb + L::F2 + p * L::F, (BWD ? a.kx : a.w) + slot * 2 * kC * DK, L::F, bar);
            sm100::bulk_load(smb + L::T0 + p * kU, (BWD ? a.du : a.u) + slot * kC * DV + c16 * kC, kU, bar);
            sm100::bulk_load(smb + L::GC + p * kG, a.gc + slot * (DK + 4), kG, bar);
            if (kH) sm100::bulk_load(smb + L::GH + p * kH, a.gh + slot * DK * DV + c16 * DK, kH, bar);
        }
    };
    const bool copier = WK > 1 ? warp == WK * GR : tid == 0;
    bool late = false;
    auto wait = [&](int n) { late = late || !arrived(a, mbar + (n & 1), n >> 1); };
    if (tid == 0) {
        sm100::mbar_init(mbar, 1);
        sm100::mbar_init(mbar + 1, 1);
        sm100::mbar_fence_init();
    }
    __syncthreads();
    if (copier && (WK == 1 || lane == 0)) issue(0), issue(1);
    if (WK > 1 && copier) {
        for (int i = 0; i < nc; ++i) {
            __syncthreads();  // a step's first barrier: what group i + 2 replaces has been read
            if (lane == 0) {
                wait(i);
                if (!late) issue(i + 2);
            }
            __syncwarp();
        }
        if (lane == 0 && nc > 0) {
            wait(nc);
            if (late) drain(a, mbar, 2);
        }
        return;
    }
    const float *src = BWD ? a.gstate : a.state0;
    float *dst = BWD ? a.dstate0 : a.state_out;
    const size_t so = ((size_t)s * a.nh + h) * DK * DV + col0;
    float acc[NT][4];  // element e: column g + 8 (e / 2), channel d0 + 8 j + 2 t + e % 2
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            acc[j][e] = src ? src[so + (size_t)(d0 + 8 * j + 2 * t + (e & 1)) * DV + g + 8 * (e >> 1)] : 0.f;
    if (nc > 0) wait(0);
    for (int i = 0; i < nc; ++i) {
        const size_t slot = slot_of(i);
        float *hp = (BWD ? a.gh : static_cast<float *>(a.h)) + slot * DK * DV;
        uint16_t *pp = (BWD ? a.ghp : static_cast<uint16_t *>(a.h)) + slot * 2 * DK * DV;
        if (late) acc[0][0] = acc[0][2] = nan_f();  // T of the columns is NaN, and with it all that follows
        const float *gcp = reinterpret_cast<const float *>(smb + L::GC) + (i & 1) * (DK + 4);
        constexpr int HN = NT < 8 ? NT : 8;  // n tiles of the second product at a time
        float2 gc[HN], add[HN][2];
        auto fetch3 = [&](int n0) {  // their decays and (g q)^T do
            const float *ghp = reinterpret_cast<const float *>(smb + L::GH) + ((i & 1) * GR + grp) * 16 * DK;
#pragma unroll
            for (int n = 0; n < HN; ++n) {
                const int d = d0 + 8 * (n0 + n) + 2 * t;
                gc[n] = *reinterpret_cast<const float2 *>(gcp + d);
                if (BWD) {
                    add[n][0] = *reinterpret_cast<const float2 *>(WK > 1 ? ghp + tile::at<DK>(g, d) : hp + tile::at<DK>(col0 + g, d));
                    add[n][1] = *reinterpret_cast<const float2 *>(WK > 1 ? ghp + tile::at<DK>(g + 8, d) : hp + tile::at<DK>(col0 + g + 8, d));
                }
            }
        };
        auto put_state = [&](int n0) {  // n tiles n0 .. of the state before the step (fp32 backwards: in gh's place)
#pragma unroll
            for (int n = n0; n < n0 + HN; ++n) {
                const int d = d0 + 8 * n + 2 * t;
                if (PL) {
                    planes::put2<planes::B, DV>(pp, DK * DV, col0 + g, d, acc[n][0], acc[n][1]);
                    planes::put2<planes::B, DV>(pp, DK * DV, col0 + g + 8, d, acc[n][2], acc[n][3]);
                } else {
                    *reinterpret_cast<float2 *>(hp + tile::at<DK>(col0 + g, d)) = make_float2(acc[n][0], acc[n][1]);
                    *reinterpret_cast<float2 *>(hp + tile::at<DK>(col0 + g + 8, d)) = make_float2(acc[n][2], acc[n][3]);
                }
            }
        };
        if (BWD && WK == 1 && i + 1 < nc) {  // the next step's, to the L2
            const char *p = reinterpret_cast<const char *>(a.gh + slot_of(i + 1) * DK * DV + col0 * DK);
            for (int e = lane * 128; e < 16 * DK * 4; e += 4096) asm volatile("prefetch.global.L2 [%0];" ::"l"(p + e));
        }
        // T's share of this warp's channels
        float tp[8][4];
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) tp[j][e] = 0.f;
        float s0, i0, s1, i1;
        {
            float m0 = 0.f, m1 = 0.f;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                m0 = fmaxf(m0, fmaxf(fabsf(acc[j][0]), fabsf(acc[j][1])));
                m1 = fmaxf(m1, fmaxf(fabsf(acc[j][2]), fabsf(acc[j][3])));
            }
            column_scales(m0, m1, s0, i0, s1, i1);
        }
        const uint16_t *F1 = reinterpret_cast<const uint16_t *>(smb + L::F1 + (i & 1) * L::F);
#pragma unroll
        for (int j = 0; j < NT; j += 2) {
            uint32_t ah[4], al[4];
            split_tile(acc[j], acc[j + 1], s0, s1, ah, al);
            uint32_t bh[4][4], bl[4][4];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                planes::frag_b<kC, false>(bh[n], F1, 16 * n, d0 + 8 * j);
                planes::frag_b<kC, false>(bl[n], F1 + kC * DK, 16 * n, d0 + 8 * j);
            }
            planes::mma3_wide<planes::H, 4>(tp, ah, al, bh, bl);
        }
        // WK 1, planes: 64 columns of S or T (16 rows, which lie together in the workspace) through shared
        // memory and out by bulk copies; as 4-byte stores to eight rows at a time they were half of a step
        auto put_slab = [&](char *stage, uint16_t *to, int plane, const float (*x)[4]) {
            const uint32_t at = planes::saddr(stage);
            const int r = lane & 7, m = lane >> 3;  // the lane's row of matrix m
#pragma unroll
            for (int n = 0; n < 8; n += 4)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) planes::split2<planes::B>(x[n + j][2 * half], x[n + j][2 * half + 1], hi[j], lo[j]);
                    const uint32_t a = at + 2 * planes::at<16>(r + 8 * half, 8 * (n + m));
                    planes::stsm(a, hi[0], hi[1], hi[2], hi[3]);
                    planes::stsm(a + 2048, lo[0], lo[1], lo[2], lo[3]);
                }
            sm100::fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) {
                sm100::bulk_store(to, stage, 2048);
                sm100::bulk_store(to + plane, stage + 2048, 2048);
                sm100::bulk_commit();
            }
        };
        char *stage = smb + L::ST + grp * 4096;
        // While the products finish; where dS' goes into gh's place (fp32), not before that has arrived.
        constexpr bool kInPlace = BWD && !PL;
        if (WK > 1 && !kInPlace) put_state(0);
        const float *T0 = reinterpret_cast<const float *>(smb + L::T0) + ((i & 1) * GR + grp) * 16 * kC;
        const uint16_t *F2 = reinterpret_cast<const uint16_t *>(smb + L::F2 + (i & 1) * L::F);
        float *U = (BWD ? a.du : a.u) + slot * kC * DV;
        uint16_t *UP = (BWD ? a.dup : a.up) + slot * 2 * kC * DV;
        auto put_u = [&](int j, const float (&x)[4]) {
            if (PL) {
                planes::put2<planes::B, DV>(UP, kC * DV, col0 + g, 8 * j + 2 * t, x[0], x[1]);
                planes::put2<planes::B, DV>(UP, kC * DV, col0 + g + 8, 8 * j + 2 * t, x[2], x[3]);
            } else {
                *reinterpret_cast<float2 *>(U + tile::at<kC>(col0 + g, 8 * j + 2 * t)) = make_float2(x[0], x[1]);
                *reinterpret_cast<float2 *>(U + tile::at<kC>(col0 + g + 8, 8 * j + 2 * t)) = make_float2(x[2], x[3]);
            }
        };
        auto add_t0 = [&](int j, float (&x)[4]) {
            const float2 x0 = *reinterpret_cast<const float2 *>(T0 + tile::at<kC>(g, 8 * j + 2 * t));
            const float2 x1 = *reinterpret_cast<const float2 *>(T0 + tile::at<kC>(g + 8, 8 * j + 2 * t));
            x[0] += x0.x, x[1] += x0.y, x[2] += x1.x, x[3] += x1.y;
        };
        if constexpr (WK > 1) {
            float4 *red = reinterpret_cast<float4 *>(smb + L::RED) + grp * WK * 256;
            uint4 *at = reinterpret_cast<uint4 *>(smb + L::AT) + grp * 4 * 64;
            float2 *sc = reinterpret_cast<float2 *>(smb + L::SC) + grp * 4 * 32;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                red[(wk * 8 + j) * 32 + lane] = make_float4(tp[j][0] * i0, tp[j][1] * i0, tp[j][2] * i1, tp[j][3] * i1);
            wait(i + 1);
            __syncthreads();  // the shares
            const float ks = gcp[DK], ws = gcp[DK + 1], sg = late ? nan_f() : BWD ? ws : -ks, out = BWD ? -ks : ws;
            fetch3(0);
            float u[2][4];    // T for the warp's quarter of the tokens
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int e = 0; e < 4; ++e) u[j][e] = 0.f;
#pragma unroll
                for (int w = 0; w < WK; ++w) {
                    const float4 x = red[(w * 8 + 2 * wk + j) * 32 + lane];
                    u[j][0] += x.x, u[j][1] += x.y, u[j][2] += x.z, u[j][3] += x.w;
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) u[j][e] *= sg;
                add_t0(2 * wk + j, u[j]);
            }
            float m0 = 0.f, m1 = 0.f;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                m0 = fmaxf(m0, fmaxf(fabsf(u[j][0]), fabsf(u[j][1])));
                m1 = fmaxf(m1, fmaxf(fabsf(u[j][2]), fabsf(u[j][3])));
            }
            column_scales(m0, m1, s0, i0, s1, i1);
            uint32_t uh[4], ul[4];
            split_tile(u[0], u[1], s0, s1, uh, ul);
            at[(wk * 2) * 32 + lane] = make_uint4(uh[0], uh[1], uh[2], uh[3]);
            at[(wk * 2 + 1) * 32 + lane] = make_uint4(ul[0], ul[1], ul[2], ul[3]);
            sc[wk * 32 + lane] = make_float2(i0, i1);
            asm volatile("bar.sync 1, %0;" ::"n"(32 * WK * GR) : "memory");  // the copier has nothing to do with it
            if (kInPlace) put_state(0);
            put_u(2 * wk, u[0]);
            put_u(2 * wk + 1, u[1]);
            float p[4][NT][4];  // the quarters' shares have scales of their own
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                acc[n][0] = fmaf(gc[n].x, acc[n][0], BWD ? add[n][0].x : 0.f);
                acc[n][1] = fmaf(gc[n].y, acc[n][1], BWD ? add[n][0].y : 0.f);
                acc[n][2] = fmaf(gc[n].x, acc[n][2], BWD ? add[n][1].x : 0.f);
                acc[n][3] = fmaf(gc[n].y, acc[n][3], BWD ? add[n][1].y : 0.f);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint4 xh = at[(j * 2) * 32 + lane], xl = at[(j * 2 + 1) * 32 + lane];
                const uint32_t ah[4] = {xh.x, xh.y, xh.z, xh.w}, al[4] = {xl.x, xl.y, xl.z, xl.w};
#pragma unroll
                for (int n = 0; n < NT; ++n) p[j][n][0] = p[j][n][1] = p[j][n][2] = p[j][n][3] = 0.f;
                uint32_t bh[NT / 2][4], bl[NT / 2][4];
#pragma unroll
                for (int n = 0; n < NT / 2; ++n) {
                    planes::frag_b<kC, true>(bh[n], F2, d0 + 16 * n, 16 * j);
                    planes::frag_b<kC, true>(bl[n], F2 + kC * DK, d0 + 16 * n, 16 * j);
                }
                planes::mma3_wide<planes::H, NT / 2>(p[j], ah, al, bh, bl);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 x = sc[j * 32 + lane];
                const float f0 = x.x * out, f1 = x.y * out;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    acc[n][0] = fmaf(p[j][n][0], f0, acc[n][0]);
                    acc[n][1] = fmaf(p[j][n][1], f0, acc[n][1]);
                    acc[n][2] = fmaf(p[j][n][2], f1, acc[n][2]);
                    acc[n][3] = fmaf(p[j][n][3], f1, acc[n][3]);
                }
            }
        } else {
            wait(i + 1);
            if (PL && lane == 0) sm100::bulk_wait_read();
            __syncthreads();  // what the next copies replace has been read
            if (copier && !late) issue(i + 2);
            const float ks = gcp[DK], ws = gcp[DK + 1], sg = late ? nan_f() : BWD ? ws : -ks, out = BWD ? -ks : ws;
            i0 *= sg, i1 *= sg;
            float m0 = 0.f, m1 = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                tp[j][0] *= i0, tp[j][1] *= i0, tp[j][2] *= i1, tp[j][3] *= i1;
                add_t0(j, tp[j]);
                if (!PL) put_u(j, tp[j]);
                m0 = fmaxf(m0, fmaxf(fabsf(tp[j][0]), fabsf(tp[j][1])));
                m1 = fmaxf(m1, fmaxf(fabsf(tp[j][2]), fabsf(tp[j][3])));
            }
            column_scales(m0, m1, s0, i0, s1, i1);
            if (PL) {  // T0 has been read: T's planes take its place
                __syncwarp();
                put_slab(smb + L::T0 + ((i & 1) * GR + grp) * 4096, UP + col0 * 64, kC * DV, tp);
            }
            i0 *= out, i1 *= out;
            uint32_t ah[4][4], al[4][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) split_tile(tp[2 * j], tp[2 * j + 1], s0, s1, ah[j], al[j]);
#pragma unroll
            for (int n0 = 0; n0 < NT; n0 += HN) {
                float p[HN][4];
                fetch3(n0);
#pragma unroll
                for (int n = 0; n < HN; ++n) p[n][0] = p[n][1] = p[n][2] = p[n][3] = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t bh[HN / 2][4], bl[HN / 2][4];
#pragma unroll
                    for (int n = 0; n < HN / 2; ++n) {
                        planes::frag_b<kC, true>(bh[n], F2, d0 + 8 * n0 + 16 * n, 16 * j);
                        planes::frag_b<kC, true>(bl[n], F2 + kC * DK, d0 + 8 * n0 + 16 * n, 16 * j);
                    }
                    planes::mma3_wide<planes::H, HN / 2>(p, ah[j], al[j], bh, bl);
                }
                if (PL) {
                    if (lane == 0) sm100::bulk_wait_read();
                    __syncwarp();
                    put_slab(stage, pp + (n0 / 8) * DV * 64 + col0 * 64, DK * DV, acc + n0);
                } else {
                    put_state(n0);
                }
#pragma unroll
                for (int n = 0; n < HN; ++n) {
                    float(&s)[4] = acc[n0 + n];
                    s[0] = fmaf(p[n][0], i0, fmaf(gc[n].x, s[0], BWD ? add[n][0].x : 0.f));
                    s[1] = fmaf(p[n][1], i0, fmaf(gc[n].y, s[1], BWD ? add[n][0].y : 0.f));
                    s[2] = fmaf(p[n][2], i1, fmaf(gc[n].x, s[2], BWD ? add[n][1].x : 0.f));
                    s[3] = fmaf(p[n][3], i1, fmaf(gc[n].y, s[3], BWD ? add[n][1].y : 0.f));
                }
            }
        }
    }
    if (WK == 1 && PL && lane == 0) sm100::bulk_wait();
    if (late) {
        make_nan(acc);
        if (copier) drain(a, mbar, 2);
    }
    if (dst)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                dst[so + (size_t)(d0 + 8 * j + 2 * t + (e & 1)) * DV + g + 8 * (e >> 1)] = acc[j][e];
}

template <int DK, int DV, int WK, int GR, bool BWD, bool PL>
cudaError_t launch_state(const Args &a, cudaStream_t st)
{
    using L = StateSmem<DK, DV, WK, GR, BWD>;
    auto k = k_scan_state<DK, DV, WK, GR, BWD, PL>;
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::bytes);
    if (e != cudaSuccess) return e;
    k<<<dim3(a.nh * (DV / (16 * GR)), BWD ? a.nseq : a.chunk_seqs), L::kThreads, L::bytes, st>>>(a);
    return cudaGetLastError();
}

// Four warps per 16 columns, one such group to a block, make a step shortest, which counts as long as
// that leaves two rounds of blocks or fewer.  With more, one warp per 16 columns and all columns in a
// block (no exchange, half the instructions) has the higher rate: 4 x 2048 tokens of 32 heads 186 us
// against 301 with two groups of four warps.  But its steps are longer, and a batch of different
// lengths waits for the longest one (8 prompts, 32 heads: 189 against 152 us) unless there are several
// blocks for each SM: up to there two groups of four warps.
template <int DK, int DV, bool BWD, bool PL>
cudaError_t state_pass(const Args &a, cudaStream_t st)
{
    const long long pairs = (long long)a.nh * (BWD ? a.nseq : a.chunk_seqs);
    if (pairs * (DV / 16) <= 2 * 148) return launch_state<DK, DV, 4, 1, BWD, PL>(a, st);
    if (a.cu && pairs < 4 * 148) return launch_state<DK, DV, 4, 2, BWD, PL>(a, st);
    return launch_state<DK, DV, 1, DV / 16, BWD, PL>(a, st);
}

// ---------------------------------------------------------------- outputs

// o = (g q) S + M U.  A block takes 64 value columns, so that two are resident and one's copies run under
// the other's products; a warp 16 rows and half of the columns.  For bfloat16 bound by reading the
// operands: 2112 chunks and heads of 128 x 128 take 76 us, 4.5 TB/s.
template <int DK>
struct OutSmem {
    static constexpr int QB = 0, S = QB + 4 * kC * DK, U = S + 4 * 64 * DK, M = U + 4 * 64 * kC, MB = M + 4 * kC * kC;
    static constexpr size_t bytes = MB + 16;
};

template <int DK, int DV, typename T>
__global__ void __launch_bounds__(kThreads, 2) k_scan_out(Args a)
{
    using L = OutSmem<DK>;
    using K = Kit<T>;
    using E = typename K::E;
    extern __shared__ __align__(1024) char smb[];
    constexpr int N = DV / 64;
    const int col0 = (blockIdx.x % N) * 64, h = blockIdx.x / N % a.nh, ci = blockIdx.x / N / a.nh, warp = threadIdx.x >> 5;
    Chunk c;
    if (!locate(a, ci, &c)) return;
    const size_t slot = (size_t)ci * a.nh + h;
    uint64_t *bar = reinterpret_cast<uint64_t *>(smb + L::MB);
    if (threadIdx.x == 0) {
        sm100::mbar_init(bar, 1);
        sm100::mbar_init(bar + 1, 1);
        sm100::mbar_fence_init();
    }
    if (threadIdx.x == 0 && !a.skip_copies) {
        sm100::mbar_expect_tx(bar, L::U);
        sm100::bulk_load(smb + L::QB, static_cast<const float *>(a.qb) + slot * kC * DK, 4 * kC * DK, bar);
        sm100::mbar_expect_tx(bar + 1, L::MB - L::U);
        if (sizeof(T) == 2) {  // planes: [2][dk / 64][dv][64] and [2][dv][64]
            const uint16_t *s = static_cast<const uint16_t *>(a.h) + slot * 2 * DK * DV + col0 * 64, *u = a.up + slot * 2 * kC * DV + col0 * kC;
            for (int b = 0; b < 2 * (DK / 64); ++b) sm100::bulk_load(smb + L::S + b * 64 * 128, s + b * DV * 64, 64 * 128, bar);
            for (int b = 0; b < 2; ++b) sm100::bulk_load(smb + L::U + b * 64 * 128, u + b * DV * kC, 64 * 128, bar + 1);
        } else {
            sm100::bulk_load(smb + L::S, static_cast<const float *>(a.h) + slot * DK * DV + col0 * DK, 4 * 64 * DK, bar);
            sm100::bulk_load(smb + L::U, a.u + slot * kC * DV + col0 * kC, 4 * 64 * kC, bar + 1);
        }
        sm100::bulk_load(smb + L::M, static_cast<const float *>(a.m) + slot * kC * kC, 4 * kC * kC, bar + 1);
    }
    __syncthreads();
    const int n0 = (warp & 1) * 32, m0 = (warp >> 1) * kSub;
    auto part = [&](int off) { return reinterpret_cast<const E *>(smb + off); };
    float acc[4][4];
    zero(acc);
    bool ok = arrived(a, bar, 0);
#pragma unroll 2
    for (int k = 0; k < DK; k += 16) K::template step<false, kC, DK, false, 64, DK, false, 4>(acc, part(L::QB), m0, k, part(L::S), n0, k);
    ok = ok && arrived(a, bar + 1, 0);
    for (int k = 0; k < m0 + kSub; k += 16) K::template step<false, kC, kC, false, 64, kC, false, 4>(acc, part(L::M), m0, k, part(L::U), n0, k);
    if (!ok) {
        make_nan(acc);
        if (threadIdx.x == 0) drain(a, bar, 2);
    }
    T *o = static_cast<T *>(a.o) + ((size_t)c.row0 * a.nh + h) * DV + col0;
    each(acc, m0, n0, [&](int r, int col, float x, float y) {
        if (r < c.n) store2(o + (size_t)r * a.nh * DV + col, x, y);
    });
}

// ---------------------------------------------------------------- token by token

// One block of four warps per sequence, head and 32 value columns, the state's slice in registers: a
// thread has four neighbouring columns of every 16th key channel.  Per token: p = k^^T diag(alpha) S
// (summed over the lanes and, through shared memory, the warps), u = beta (v - p),
// S = diag(alpha) S + k^ u^T, o = q^T S.  For a single token it is bound by reading and writing the
// states: slices this small keep several blocks on an SM, one's loads under another's stores (64
// sequences, 48 heads 128 x 128: 66 us, 6.1 TB/s; a block with a whole state 107 us).
constexpr int kTokenCols = 32;

template <int DK, int DV, typename T>
__global__ void __launch_bounds__(128) k_scan_tokens(Args a)
{
    constexpr int R = DK / 16, N = DV / kTokenCols;
    __shared__ float kq[3][DK];  // k; q; alpha
    __shared__ float4 part[2][4][8];
    __shared__ float norm[4];
    const int h = blockIdx.x / N, c0 = (blockIdx.x % N) * kTokenCols, s = blockIdx.y;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int r0 = warp * 4 + (lane >> 3), c4 = c0 + 4 * (lane & 7);  // the thread's first channel, its columns
    const long long row0 = seq_start(a, s), row1 = seq_end(a, s);
    if (row1 - row0 > a.short_tokens) return;  // by chunks
    const size_t so = ((size_t)s * a.nh + h) * DK * DV + c4;
    float4 S[R];
#pragma unroll
    for (int i = 0; i < R; ++i)
        S[i] = a.state0 ? *reinterpret_cast<const float4 *>(a.state0 + so + (size_t)(r0 + 16 * i) * DV) : make_float4(0.f, 0.f, 0.f, 0.f);
    auto sum_rows = [&](float4 x, int buf) {  // over the block's 16 rows of threads
#pragma unroll
        for (int o = 8; o < 32; o <<= 1) {
            x.x += __shfl_xor_sync(0xffffffffu, x.x, o);
            x.y += __shfl_xor_sync(0xffffffffu, x.y, o);
            x.z += __shfl_xor_sync(0xffffffffu, x.z, o);
            x.w += __shfl_xor_sync(0xffffffffu, x.w, o);
        }
        if (lane < 8) part[buf][warp][lane] = x;
        __syncthreads();
        x = part[buf][0][lane & 7];
#pragma unroll
        for (int w = 1; w < 4; ++w) {
            const float4 y = part[buf][w][lane & 7];
            x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
        }
        return x;
    };
    for (long long row = row0; row < row1; ++row) {
        float kv = 0.f;
        if (tid < DK) {
            kv = to_f(static_cast<const T *>(a.k)[row * a.ldk + h * DK + tid]);
            kq[0][tid] = kv;
            kq[1][tid] = to_f(static_cast<const T *>(a.q)[row * a.ldq + h * DK + tid]);
            kq[2][tid] = exp2a(log2_alpha(to_f(static_cast<const T *>(a.z)[row * a.ldz + h * DK + tid])));
        }
        const float ss = warp_sum(kv * kv);
        if (lane == 0) norm[warp] = ss;
        const float beta = sigmoid(to_f(static_cast<const T *>(a.b)[row * a.ldb + h]));
        float v[4];
        load4(static_cast<const T *>(a.v) + row * a.ldv + h * DV + c4, v);
        __syncthreads();
        const float sum = (norm[0] + norm[1]) + (norm[2] + norm[3]);
        const float inv = sum > 0.f ? 1.f / sqrtf(sum) : sum == sum ? 0.f : sum;
        float4 p = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const float k = kq[0][r0 + 16 * i] * inv, al = kq[2][r0 + 16 * i];
            S[i].x *= al, S[i].y *= al, S[i].z *= al, S[i].w *= al;
            p.x = fmaf(k, S[i].x, p.x), p.y = fmaf(k, S[i].y, p.y), p.z = fmaf(k, S[i].z, p.z), p.w = fmaf(k, S[i].w, p.w);
        }
        p = sum_rows(p, 0);
        p = make_float4(beta * (v[0] - p.x), beta * (v[1] - p.y), beta * (v[2] - p.z), beta * (v[3] - p.w));
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const float k = kq[0][r0 + 16 * i] * inv, q = kq[1][r0 + 16 * i];
            S[i].x = fmaf(k, p.x, S[i].x), S[i].y = fmaf(k, p.y, S[i].y), S[i].z = fmaf(k, p.z, S[i].z), S[i].w = fmaf(k, p.w, S[i].w);
            o.x = fmaf(q, S[i].x, o.x), o.y = fmaf(q, S[i].y, o.y), o.z = fmaf(q, S[i].z, o.z), o.w = fmaf(q, S[i].w, o.w);
        }
        o = sum_rows(o, 1);  // its barrier is also the one before the next token's kq and norm
        if (tid < 8) {
            T *to = static_cast<T *>(a.o) + ((size_t)row * a.nh + h) * DV + c4;
            store2(to, o.x, o.y);
            store2(to + 2, o.z, o.w);
        }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) *reinterpret_cast<float4 *>(a.state_out + so + (size_t)(r0 + 16 * i) * DV) = S[i];
}

template <class K>
cudaError_t allow_smem(K kernel, size_t bytes)
{
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <int DK, int DV, typename T, bool BWD>
cudaError_t forward_chunks(const Args &a, cudaStream_t st)
{
    constexpr bool BF = sizeof(T) == 2;
    auto prep = k_scan_prep<DK, DV, BWD, T>;
    cudaError_t e = allow_smem(prep, PrepSmem<DK, DV, BWD>::bytes);
    if (e != cudaSuccess) return e;
    if (a.cu) k_scan_plan<<<1, 1024, 0, st>>>(a, const_cast<int *>(a.pre), const_cast<int *>(a.list));
    if (a.short_tokens > 0) k_scan_tokens<DK, DV, T><<<dim3(a.nh * (DV / kTokenCols), a.nseq), 128, 0, st>>>(a);
    const unsigned grid = (unsigned)a.nh * a.max_chunks;
    if (grid) prep<<<grid, 4 * DK, PrepSmem<DK, DV, BWD>::bytes, st>>>(a);
    e = state_pass<DK, DV, false, BF>(a, st);
    if (e != cudaSuccess || BWD || !grid) return e;
    e = allow_smem(k_scan_out<DK, DV, T>, OutSmem<DK>::bytes);
    if (e == cudaSuccess) k_scan_out<DK, DV, T><<<grid * (DV / 64), kThreads, OutSmem<DK>::bytes, st>>>(a);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace

template <int DK, int DV, typename T>
cudaError_t forward(const Args &a, bool backward, cudaStream_t st)
{
    return backward ? forward_chunks<DK, DV, T, true>(a, st) : forward_chunks<DK, DV, T, false>(a, st);
}

template <int DK, int DV, typename T>
cudaError_t tokens(const Args &a, cudaStream_t st)
{
    k_scan_tokens<DK, DV, T><<<dim3(a.nh * (DV / kTokenCols), a.nseq), 128, 0, st>>>(a);
    return cudaGetLastError();
}

template <int DK, int DV, typename T>
cudaError_t reverse(const Args &a, cudaStream_t st)
{
    return state_pass<DK, DV, true, sizeof(T) == 2>(a, st);
}

#define KDA_SCAN_T(DK, DV, T)                                                  \
    template cudaError_t forward<DK, DV, T>(const Args &, bool, cudaStream_t); \
    template cudaError_t reverse<DK, DV, T>(const Args &, cudaStream_t);       \
    template cudaError_t tokens<DK, DV, T>(const Args &, cudaStream_t);
#define KDA_SCAN(DK, DV)      \
    KDA_SCAN_T(DK, DV, float) \
    KDA_SCAN_T(DK, DV, __nv_bfloat16)
KDA_SCAN(64, 64)
KDA_SCAN(64, 128)
KDA_SCAN(128, 64)
KDA_SCAN(128, 128)

}  // namespace scan
}  // namespace kda
