// rows.cu -- moves of whole rows (a sequence's state) inside a pool, or from one pool to another.
//
// Every thread makes a chain's moves one after another for its own 16-byte pieces of the rows, so
// an order that is right for one piece is right for the rows, with no synchronisation: the plan
// (rows_plan.cu) gives that order.  A row that goes to several places is read once.  Bound by the
// bytes: each source once, each destination once (20 rows of 3.1 MB moved and 20 cleared: 34 us,
// 5.5 TB/s).
#include "rows.cuh"

namespace kda {
namespace rows {
namespace {

constexpr int kPieces = 4;  // 16-byte pieces of a thread, all in flight at once

template <int N>
struct Table {
    int first[N + 1];
    Step step[N + N / 2];  // a cycle has one more step than moves, and at least two moves
};

template <int N>
__global__ void __launch_bounds__(256)
    k_rows(uint4 *dst, const uint4 *src, long long vecs, const __grid_constant__ Table<N> t)
{
    const int s0 = t.first[blockIdx.y], s1 = t.first[blockIdx.y + 1];
    const long long e0 = (long long)blockIdx.x * (256 * kPieces) + threadIdx.x;
    uint4 x[kPieces], saved[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) x[i] = saved[i] = make_uint4(0, 0, 0, 0);
    int held = kZero;  // what x holds
    for (int s = s0; s < s1; ++s) {
        const Step st = t.step[s];
        if (st.src != held || st.src == kZero) {
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const long long e = e0 + i * 256;
                if (st.src == kZero) x[i] = make_uint4(0, 0, 0, 0);
                else if (st.src == kSaved) x[i] = saved[i];
                else if (e < vecs) x[i] = __ldcs(src + st.src * vecs + e);
            }
            held = st.src;
        }
        if (st.dst == kSave) {
#pragma unroll
            for (int i = 0; i < kPieces; ++i) saved[i] = x[i];
        } else {
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const long long e = e0 + i * 256;
                if (e < vecs) __stcs(dst + st.dst * vecs + e, x[i]);
            }
        }
    }
}

template <int N>
cudaError_t launch(void *dst, const void *src, size_t row_bytes, const Plan &p, cudaStream_t st)
{
    Table<N> t;
    for (size_t i = 0; i < p.first.size(); ++i) t.first[i] = p.first[i];
    for (size_t i = 0; i < p.steps.size(); ++i) t.step[i] = p.steps[i];
    const long long vecs = (long long)(row_bytes / 16);
    const dim3 grid((unsigned)((vecs + 256 * kPieces - 1) / (256 * kPieces)), (unsigned)(p.first.size() - 1));
    k_rows<N><<<grid, 256, 0, st>>>(static_cast<uint4 *>(dst), static_cast<const uint4 *>(src), vecs, t);
    return cudaGetLastError();
}

}  // namespace

cudaError_t run(void *dst, const void *src, size_t row_bytes, const Plan &p, int n, cudaStream_t st)
{
    if (p.steps.empty()) return cudaSuccess;
    // the table travels with the launch (up to 16 KB); the usual few moves take a small one
    return n <= 64 ? launch<64>(dst, src, row_bytes, p, st) : launch<kMaxMoves>(dst, src, row_bytes, p, st);
}

}  // namespace rows
}  // namespace kda
