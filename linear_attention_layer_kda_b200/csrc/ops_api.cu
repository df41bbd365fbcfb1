// ops_api.cu -- the C entry points of the operators around the decode step (include/kda_decode.h):
// the recurrence over whole sequences, the residual norm and the moves of state rows.  They take no
// handle: everything they use is an argument, so calls on different streams, devices or captured
// graphs share nothing.
#include <limits.h>
#include <stdlib.h>

#include <new>

#include "common.cuh"
#include "norm.cuh"
#include "rows.cuh"
#include "scan_ops.cuh"

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

struct Range {
    const char *p;
    size_t n;
};
bool overlaps(const Range &a, const Range &b)
{
    return a.p && b.p && a.n && b.n && a.p < b.p + b.n && b.p < a.p + a.n;
}
// True if an output overlaps an input or another output (a caller leaves out the input that an output may replace).
bool clash(const Range *out, int nout, const Range *in, int nin)
{
    for (int i = 0; i < nout; ++i) {
        for (int j = 0; j < nin; ++j)
            if (overlaps(out[i], in[j])) return true;
        for (int j = 0; j < i; ++j)
            if (overlaps(out[i], out[j])) return true;
    }
    return false;
}

// The current device, if the kernels run on it; its SM count.
int check_device(int *sms)
{
    int dev = -1, major = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess || major != 10 ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        (void)cudaGetLastError();
        return KDA_ERR_NO_DEVICE;
    }
    if (sms) *sms = n;
    return KDA_OK;
}

int launched(cudaError_t e)
{
    if (e == cudaSuccess) return KDA_OK;
    (void)cudaGetLastError();
    return KDA_ERR_CUDA;
}

// ---------------------------------------------------------------- scan

// Sequences of up to this many tokens go token by token, in a ragged batch beside those that go by
// chunks.  32 heads 128 x 128 in bfloat16: 8 sequences 2.2 us a token against 76 us for a chunk,
// 64 sequences 16.6 against 515, one sequence 0.8 against 30.  Beside longer ones they run first, on
// their own: 64 of 24 tokens beside one of 512 537 us against 649, but one of 32 beside one of 2048 315
// against 301.
constexpr int kShort = 32;

// The longest wait of a kernel for its copies, as for the step's (KDA_WAIT_LIMIT_MS, 2 s); with
// KDA_DEBUG_SKIP_SCAN_COPIES set the copies are not made and the waits run out (a test).  Read once.
struct Waits {
    uint64_t ns = 2000000000ull;
    int skip = 0;
    Waits()
    {
        if (const char *e = getenv("KDA_WAIT_LIMIT_MS")) {
            const double ms = atof(e);
            if (ms > 0) ns = (uint64_t)(ms * 1e6);
        }
        if (const char *e = getenv("KDA_DEBUG_SKIP_SCAN_COPIES")) skip = atoi(e) != 0;
    }
};
const Waits &waits()
{
    static const Waits w;
    return w;
}

struct ScanDims {
    size_t esize;
    long long ld[5];   // q, k, v, z, b
    bool ragged;
    int tokens;        // per sequence, not ragged
    int max_chunks, chunk_seqs;
};

int scan_dims(const kda_scan_desc *d, bool ragged, bool backward, ScanDims *s)
{
    if (!d) return KDA_ERR_INVALID_ARG;
    for (int r : d->reserved)
        if (r) return KDA_ERR_INVALID_ARG;
    if (d->dtype != KDA_DTYPE_F32 && d->dtype != KDA_DTYPE_BF16) return KDA_ERR_INVALID_ARG;
    if ((d->head_dk != 64 && d->head_dk != 128) || (d->head_dv != 64 && d->head_dv != 128)) return KDA_ERR_UNSUPPORTED_SHAPE;
    if (d->num_heads < 1 || d->num_heads > 512) return KDA_ERR_UNSUPPORTED_SHAPE;
    if (d->nseq < 1 || d->nseq > 65535) return KDA_ERR_UNSUPPORTED_SHAPE;
    if (d->rows < 0 || d->rows > INT_MAX) return KDA_ERR_UNSUPPORTED_SHAPE;
    s->esize = d->dtype == KDA_DTYPE_BF16 ? 2 : 4;
    const long long nh = d->num_heads;
    const long long width[5] = {nh * d->head_dk, nh * d->head_dk, nh * d->head_dv, nh * d->head_dk, nh};
    const long long ld[5] = {d->ld_q, d->ld_k, d->ld_v, d->ld_z, d->ld_b};
    for (int i = 0; i < 5; ++i) {
        s->ld[i] = ld[i] ? ld[i] : width[i];
        if (s->ld[i] < width[i] || s->ld[i] > INT_MAX) return KDA_ERR_INVALID_ARG;
        if (i < 4 && s->ld[i] * (long long)s->esize % 16) return KDA_ERR_INVALID_ARG;
    }
    s->ragged = ragged;
    s->tokens = 0;
    s->chunk_seqs = d->nseq;
    long long chunks;
    if (!ragged) {
        if (d->rows % d->nseq) return KDA_ERR_INVALID_ARG;
        s->tokens = (int)(d->rows / d->nseq);
        chunks = (long long)d->nseq * ((s->tokens + kda::scan::kC - 1) / kda::scan::kC);
    } else {
        // rows / kC full chunks at most, and a part-filled one for every sequence that goes by chunks
        const long long most = backward ? d->rows : d->rows / (kShort + 1);
        chunks = d->rows / kda::scan::kC + (most < d->nseq ? most : d->nseq);
        if (!backward && most < d->nseq) s->chunk_seqs = (int)most;  // the kernel's list names them
    }
    if (chunks * nh > INT_MAX) return KDA_ERR_UNSUPPORTED_SHAPE;
    s->max_chunks = (int)chunks;
    return KDA_OK;
}

// All sequences go token by token, as far as the host can tell.
bool scan_by_token(const kda_scan_desc *d, const ScanDims &s)
{
    return (s.ragged ? d->rows : s.tokens) <= kShort;
}

// Places of the workspace's parts; returns its size.
size_t scan_layout(const kda_scan_desc *d, const ScanDims &s, bool backward, char *base, kda::scan::Args *a)
{
    using kda::scan::kC;
    const size_t slots = (size_t)s.max_chunks * d->num_heads, dk = d->head_dk, dv = d->head_dv;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        char *p = base ? base + off : nullptr;
        off += align_up(bytes, 256);
        return p;
    };
    a->pre = (const int *)take(s.ragged ? ((size_t)d->nseq + 1) * 4 : 0);
    if (!s.ragged) a->pre = nullptr;
    a->list = nullptr;
    if (s.ragged && !backward) a->list = (const int *)take(((size_t)d->nseq + 1) * 4);
    const bool bf = d->dtype == KDA_DTYPE_BF16;
    a->kx = (uint16_t *)take(slots * kC * dk * 4);
    a->w = (uint16_t *)take(slots * kC * dk * 4);
    a->u = (float *)take(slots * kC * dv * 4);
    a->gc = (float *)take(slots * (dk + 4) * 4);
    a->h = take(slots * dk * dv * 4);
    if (bf) a->up = (uint16_t *)take(slots * kC * dv * 4);
    if (!backward) {
        a->qb = take(slots * kC * dk * 4);
        a->m = take(slots * kC * kC * 4);
    } else {
        a->x = take(slots * kC * kC * 4);
        a->inv = (float *)take(slots * kC * 4);
        a->du = (float *)take(slots * kC * dv * 4);
        a->gh = (float *)take(slots * dk * dv * 4);
        if (bf) a->dup = (uint16_t *)take(slots * kC * dv * 4);
        if (bf) a->ghp = (uint16_t *)take(slots * dk * dv * 4);
    }
    return off;
}

int scan_args(const kda_scan_desc *d, const ScanDims &s, const void *q, const void *k, const void *v, const void *z,
              const void *b, const int *cu, const float *state0, kda::scan::Args *a)
{
    const void *in[4] = {q, k, v, z};
    for (const void *p : in)
        if ((!p && d->rows > 0) || !aligned16(p)) return KDA_ERR_INVALID_ARG;
    if ((!b && d->rows > 0) || (uintptr_t)b % s.esize || (uintptr_t)cu % 4 || !aligned16(state0)) return KDA_ERR_INVALID_ARG;
    a->nh = d->num_heads;
    a->nseq = d->nseq;
    a->max_chunks = s.max_chunks;
    a->chunk_seqs = s.chunk_seqs;
    a->rows = d->rows;
    a->tokens = s.tokens;
    a->cu = cu;
    a->q = q, a->k = k, a->v = v, a->z = z, a->b = b;
    a->ldq = s.ld[0], a->ldk = s.ld[1], a->ldv = s.ld[2], a->ldz = s.ld[3], a->ldb = s.ld[4];
    a->state0 = state0;
    a->wait_ns = waits().ns;
    a->skip_copies = waits().skip;
    return KDA_OK;
}

// Bytes that the inputs of a call cover.
void scan_ranges(const kda_scan_desc *d, const ScanDims &s, const kda::scan::Args &a, Range *r)
{
    const void *p[5] = {a.q, a.k, a.v, a.z, a.b};
    const long long w[5] = {(long long)d->num_heads * d->head_dk, (long long)d->num_heads * d->head_dk,
                            (long long)d->num_heads * d->head_dv, (long long)d->num_heads * d->head_dk, d->num_heads};
    for (int i = 0; i < 5; ++i)
        r[i] = {(const char *)p[i], d->rows > 0 ? (size_t)((d->rows - 1) * s.ld[i] + w[i]) * s.esize : 0};
    r[5] = {(const char *)a.cu, a.cu ? ((size_t)d->nseq + 1) * 4 : 0};
}

template <class F>
cudaError_t by_shape(const kda_scan_desc *d, F f)
{
    const bool bf = d->dtype == KDA_DTYPE_BF16;
    const int key = (d->head_dk == 128) * 4 + (d->head_dv == 128) * 2 + bf;
    switch (key) {
    case 0: return f.template operator()<64, 64, float>();
    case 1: return f.template operator()<64, 64, __nv_bfloat16>();
    case 2: return f.template operator()<64, 128, float>();
    case 3: return f.template operator()<64, 128, __nv_bfloat16>();
    case 4: return f.template operator()<128, 64, float>();
    case 5: return f.template operator()<128, 64, __nv_bfloat16>();
    case 6: return f.template operator()<128, 128, float>();
    default: return f.template operator()<128, 128, __nv_bfloat16>();
    }
}

struct Tokens {
    const kda::scan::Args &a;
    cudaStream_t st;
    template <int DK, int DV, typename T>
    cudaError_t operator()() const { return kda::scan::tokens<DK, DV, T>(a, st); }
};
struct Forward {
    const kda::scan::Args &a;
    cudaStream_t st;
    template <int DK, int DV, typename T>
    cudaError_t operator()() const { return kda::scan::forward<DK, DV, T>(a, false, st); }
};
struct Backward {
    const kda::scan::Args &a;
    cudaStream_t st;
    template <int DK, int DV, typename T>
    cudaError_t operator()() const { return kda::scan::backward<DK, DV, T>(a, st); }
};

}  // namespace

extern "C" {

int kda_scan_workspace_bytes(const kda_scan_desc *d, int ragged, int backward, size_t *bytes)
{
    if (!bytes) return KDA_ERR_INVALID_ARG;
    *bytes = 0;
    ScanDims s;
    if (int rc = scan_dims(d, ragged != 0, backward != 0, &s)) return rc;
    if (!backward && scan_by_token(d, s)) return KDA_OK;
    kda::scan::Args a{};
    *bytes = scan_layout(d, s, backward != 0, nullptr, &a);
    return KDA_OK;
}

int kda_scan_forward(const kda_scan_desc *d, const void *q, const void *k, const void *v, const void *z, const void *b,
                     const int *cu_seqlens, const float *state0, void *o, float *state_out, void *workspace,
                     size_t workspace_bytes, void *cuda_stream)
{
    ScanDims s;
    if (int rc = scan_dims(d, cu_seqlens != nullptr, false, &s)) return rc;
    kda::scan::Args a{};
    if (int rc = scan_args(d, s, q, k, v, z, b, cu_seqlens, state0, &a)) return rc;
    if (!state_out || !aligned16(state_out) || (!o && d->rows > 0) || !aligned16(o)) return KDA_ERR_INVALID_ARG;
    const bool by_token = scan_by_token(d, s);
    const size_t need = by_token ? 0 : scan_layout(d, s, false, static_cast<char *>(workspace), &a);
    if (need && (!workspace || workspace_bytes < need || (uintptr_t)workspace % 256)) return KDA_ERR_INVALID_ARG;
    a.o = o;
    a.state_out = state_out;
    a.short_tokens = s.ragged || by_token ? kShort : 0;
    const size_t ns = (size_t)d->nseq * d->num_heads * d->head_dk * d->head_dv * 4;
    Range in[7];
    scan_ranges(d, s, a, in);
    in[6] = {state0 == state_out ? nullptr : (const char *)state0, ns};
    const Range out[3] = {{(const char *)o, (size_t)d->rows * d->num_heads * d->head_dv * s.esize},
                          {(const char *)state_out, ns},
                          {(const char *)workspace, need}};
    if (clash(out, 3, in, 7)) return KDA_ERR_INVALID_ARG;
    if (int rc = check_device(nullptr)) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
    return launched(by_token ? by_shape(d, Tokens{a, st}) : by_shape(d, Forward{a, st}));
}

int kda_scan_backward(const kda_scan_desc *d, const void *q, const void *k, const void *v, const void *z, const void *b,
                      const int *cu_seqlens, const float *state0, const void *go, const float *dstate_out, void *dq,
                      void *dk, void *dv, void *dz, void *db, float *dstate0, void *workspace, size_t workspace_bytes,
                      void *cuda_stream)
{
    ScanDims s;
    if (int rc = scan_dims(d, cu_seqlens != nullptr, true, &s)) return rc;
    kda::scan::Args a{};
    if (int rc = scan_args(d, s, q, k, v, z, b, cu_seqlens, state0, &a)) return rc;
    const void *more[5] = {go, dq, dk, dv, dz};
    for (const void *p : more)
        if ((!p && d->rows > 0) || !aligned16(p)) return KDA_ERR_INVALID_ARG;
    if ((!db && d->rows > 0) || (uintptr_t)db % s.esize || !aligned16(dstate_out) || !aligned16(dstate0))
        return KDA_ERR_INVALID_ARG;
    const size_t need = scan_layout(d, s, true, static_cast<char *>(workspace), &a);
    if (need && (!workspace || workspace_bytes < need || (uintptr_t)workspace % 256)) return KDA_ERR_INVALID_ARG;
    a.go = go;
    a.gstate = dstate_out;
    a.dq = dq, a.dk = dk, a.dv = dv, a.dz = dz, a.db = db;
    a.dstate0 = dstate0;
    const size_t ns = (size_t)d->nseq * d->num_heads * d->head_dk * d->head_dv * 4;
    const size_t nk = (size_t)d->rows * d->num_heads * d->head_dk * s.esize;
    const size_t nv = (size_t)d->rows * d->num_heads * d->head_dv * s.esize;
    Range in[9];
    scan_ranges(d, s, a, in);
    in[6] = {(const char *)state0, ns};
    in[7] = {dstate0 == dstate_out ? nullptr : (const char *)dstate_out, ns};
    in[8] = {(const char *)go, nv};
    const Range out[7] = {{(const char *)dq, nk}, {(const char *)dk, nk}, {(const char *)dv, nv}, {(const char *)dz, nk},
                          {(const char *)db, (size_t)d->rows * d->num_heads * s.esize},
                          {(const char *)dstate0, ns}, {(const char *)workspace, need}};
    if (clash(out, 7, in, 9)) return KDA_ERR_INVALID_ARG;
    if (int rc = check_device(nullptr)) return rc;
    return launched(by_shape(d, Backward{a, static_cast<cudaStream_t>(cuda_stream)}));
}

static int norm_dims(long long rows, int hidden, int t0, int t1)
{
    if ((t0 != KDA_DTYPE_F32 && t0 != KDA_DTYPE_BF16) || (t1 != KDA_DTYPE_F32 && t1 != KDA_DTYPE_BF16)) return KDA_ERR_INVALID_ARG;
    if (hidden < 128 || hidden > 65536 || hidden % 128 || rows < 0 || rows > INT_MAX) return KDA_ERR_UNSUPPORTED_SHAPE;
    return KDA_OK;
}

int kda_residual_norm(long long rows, int hidden, const void *x, int x_dtype, const void *residual, int residual_dtype,
                      const void *weight, float eps, void *residual_out, void *y, uint8_t *y8, float *scale,
                      float *rstd, void *cuda_stream)
{
    if (int rc = norm_dims(rows, hidden, x_dtype, residual_dtype)) return rc;
    if (!(eps >= 0.f) || !weight || !aligned16(weight) || !y8 != !scale) return KDA_ERR_INVALID_ARG;
    if (rows > 0 && (!x || !residual_out)) return KDA_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(residual) || !aligned16(residual_out) || !aligned16(y) || (uintptr_t)y8 % 8 ||
        (uintptr_t)scale % 4 || (uintptr_t)rstd % 4)
        return KDA_ERR_INVALID_ARG;
    const size_t n = (size_t)rows * hidden, xs = x_dtype == KDA_DTYPE_BF16 ? 2 : 4, rs = residual_dtype == KDA_DTYPE_BF16 ? 2 : 4;
    // residual_out may be residual, or x where the types agree: a row is read before it is written
    const bool same_x = residual_out == x && xs == rs;
    const Range in[3] = {{same_x ? nullptr : (const char *)x, n * xs},
                         {residual == residual_out ? nullptr : (const char *)residual, n * rs},
                         {(const char *)weight, (size_t)hidden * 2}};
    const Range out[5] = {{(const char *)residual_out, n * rs}, {(const char *)y, n * 2}, {(const char *)y8, n},
                          {(const char *)scale, n / 128 * 4}, {(const char *)rstd, (size_t)rows * 4}};
    if (clash(out, 5, in, 3)) return KDA_ERR_INVALID_ARG;
    if (int rc = check_device(nullptr)) return rc;
    if (rows == 0) return KDA_OK;
    kda::norm::Args a{x, residual, weight, residual_out, y, y8, scale, rstd, rows, hidden, eps};
    return launched(kda::norm::forward(a, xs == 2, rs == 2, static_cast<cudaStream_t>(cuda_stream)));
}

int kda_residual_norm_workspace_bytes(long long rows, int hidden, size_t *bytes)
{
    if (!bytes) return KDA_ERR_INVALID_ARG;
    *bytes = 0;
    if (int rc = norm_dims(rows, hidden, KDA_DTYPE_F32, KDA_DTYPE_F32)) return rc;
    int sms = 148;  // without a device, for a 148-SM B200
    (void)check_device(&sms);
    *bytes = (size_t)kda::norm::grad_parts(rows, hidden, sms) * hidden * 4;
    return KDA_OK;
}

int kda_residual_norm_backward(long long rows, int hidden, const void *dy, const void *residual, int residual_dtype,
                               const void *weight, const float *rstd, const void *dresidual, void *dresidual_out,
                               float *dweight, void *workspace, size_t workspace_bytes, void *cuda_stream)
{
    if (int rc = norm_dims(rows, hidden, residual_dtype, residual_dtype)) return rc;
    if (!weight || !aligned16(weight) || !dweight || (uintptr_t)dweight % 4) return KDA_ERR_INVALID_ARG;
    if (rows > 0 && (!dy || !residual || !rstd || !dresidual_out)) return KDA_ERR_INVALID_ARG;
    if (!aligned16(dy) || !aligned16(residual) || !aligned16(dresidual) || !aligned16(dresidual_out) || (uintptr_t)rstd % 4)
        return KDA_ERR_INVALID_ARG;
    int sms = 0;
    if (int rc = check_device(&sms)) return rc;
    const int parts = kda::norm::grad_parts(rows, hidden, sms);
    const size_t need = (size_t)parts * hidden * 4;
    if (need && (!workspace || workspace_bytes < need || !aligned16(workspace))) return KDA_ERR_INVALID_ARG;
    const size_t n = (size_t)rows * hidden, rs = residual_dtype == KDA_DTYPE_BF16 ? 2 : 4;
    const bool same_dy = dresidual_out == dy && rs == 2;
    const Range in[5] = {{same_dy ? nullptr : (const char *)dy, n * 2}, {(const char *)residual, n * rs},
                         {(const char *)weight, (size_t)hidden * 2}, {(const char *)rstd, (size_t)rows * 4},
                         {dresidual == dresidual_out ? nullptr : (const char *)dresidual, n * rs}};
    const Range out[3] = {{(const char *)dresidual_out, n * rs}, {(const char *)dweight, (size_t)hidden * 4},
                          {(const char *)workspace, need}};
    if (clash(out, 3, in, 5)) return KDA_ERR_INVALID_ARG;
    kda::norm::GradArgs a{dy, residual, weight, dresidual, rstd, dresidual_out, static_cast<float *>(workspace), dweight, rows, hidden};
    return launched(kda::norm::backward(a, rs == 2, parts, static_cast<cudaStream_t>(cuda_stream)));
}

int kda_state_rows(void *dst_pool, long long dst_rows, const void *src_pool, long long src_rows, size_t row_bytes,
                   const int *dst, const int *src, int n, void *cuda_stream)
{
    if (n < 0 || n > KDA_STATE_MOVES_MAX || (n > 0 && (!dst || !src))) return KDA_ERR_INVALID_ARG;
    if (dst_rows < 0 || src_rows < 0 || dst_rows > INT_MAX || src_rows > INT_MAX) return KDA_ERR_INVALID_ARG;
    if (row_bytes == 0 || row_bytes % 16 || row_bytes > ((size_t)1 << 40)) return KDA_ERR_UNSUPPORTED_SHAPE;
    if (!aligned16(dst_pool) || !aligned16(src_pool)) return KDA_ERR_INVALID_ARG;
    if (n > 0 && (!dst_pool || !src_pool)) return KDA_ERR_INVALID_ARG;
    for (int i = 0; i < n; ++i)
        if (dst[i] < 0 || dst[i] >= dst_rows || src[i] < -1 || src[i] >= src_rows) return KDA_ERR_INVALID_ARG;
    const Range ro = {(const char *)dst_pool, (size_t)dst_rows * row_bytes}, ri = {(const char *)src_pool, (size_t)src_rows * row_bytes};
    const bool in_place = dst_pool == src_pool;
    if (!in_place && overlaps(ro, ri)) return KDA_ERR_INVALID_ARG;
    try {
        kda::rows::Plan p;
        if (!kda::rows::plan(dst, src, n, in_place, &p)) return KDA_ERR_INVALID_ARG;
        if (int rc = check_device(nullptr)) return rc;
        return launched(kda::rows::run(dst_pool, src_pool, row_bytes, p, n, static_cast<cudaStream_t>(cuda_stream)));
    } catch (const std::bad_alloc &) {
        return KDA_ERR_OUT_OF_MEMORY;
    }
}

}  // extern "C"
