// C ABI of the operators beside the KDA recurrence: argument checks, then the launch.  Nothing is
// enqueued unless every check passes.
#include <algorithm>
#include <stdint.h>

#include "kda_serving.cuh"

namespace {

bool aligned(const void* p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
bool aligned16(const void* p) { return aligned(p, 16); }
size_t elem_size(int dtype) { return dtype == KDA_DTYPE_BF16 ? 2 : 4; }
bool dtype_ok(int dtype) { return dtype == KDA_DTYPE_BF16 || dtype == KDA_DTYPE_FP32; }
bool head_dim_ok(int d) { return d == 64 || d == 128; }

constexpr double kMostElements = 9.0e15;     // element counts stay far from overflow
constexpr long long kMostStride = 1ll << 40;
constexpr int kMostTokens = 2000000000;       // token and sequence counts: sums with a strip stay within 32 bits

struct Range {
    uintptr_t lo, hi;   // [lo, hi)
};
Range range_of(const void* p, size_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return Range{a, p ? a + bytes : a};
}
// `rows` rows of `width` elements, `ld` elements apart
Range rows_of(const void* p, size_t rows, size_t width, long long ld, size_t es) {
    return range_of(p, rows ? ((rows - 1) * (size_t)ld + width) * es : 0);
}
bool overlaps(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }

// ------------------------------------------------------------------ short convolution

// tokens: rows of x and y; n_state: states in the state arrays
int check_conv(const kda::ConvArgs& a, size_t tokens, size_t n_state) {
    if (!dtype_ok(a.dtype) || (a.act != KDA_ACT_NONE && a.act != KDA_ACT_SILU)) return KDA_ERR_UNSUPPORTED;
    if (a.C <= 0 || a.n_seq <= 0 || a.T < 0) return KDA_ERR_INVALID_ARG;
    if (a.T > kMostTokens || a.n_seq > kMostTokens) return KDA_ERR_INVALID_ARG;
    if (a.W < 2 || a.W > 4 || a.C % 8 != 0) return KDA_ERR_UNSUPPORTED;
    const size_t es = elem_size(a.dtype);
    const long long vec = (long long)(16 / es);
    if (a.ldx < a.C || a.ldy < a.C || a.ldx > kMostStride || a.ldy > kMostStride) return KDA_ERR_INVALID_ARG;
    if ((double)tokens * (double)std::max(a.ldx, a.ldy) > kMostElements ||
        (double)n_state * a.W * (double)a.C > kMostElements)
        return KDA_ERR_INVALID_ARG;
    if (!a.weight || (tokens > 0 && (!a.x || !a.y))) return KDA_ERR_INVALID_ARG;
    const void* ptrs[] = {a.x, a.weight, a.bias, a.state, a.y, a.state_out};
    for (const void* p : ptrs)
        if (p && !aligned16(p)) return KDA_ERR_MISALIGNED;
    if (a.ldx % vec != 0 || a.ldy % vec != 0) return KDA_ERR_MISALIGNED;
    const size_t sbytes = n_state * (size_t)(a.W - 1) * a.C * es;
    const Range rx = rows_of(a.x, tokens, a.C, a.ldx, es), ry = rows_of(a.y, tokens, a.C, a.ldy, es);
    const Range rs = range_of(a.state, sbytes), ro = range_of(a.state_out, sbytes);
    const Range ins[] = {rx, range_of(a.weight, (size_t)a.C * a.W * es), range_of(a.bias, (size_t)a.C * es),
                         range_of(a.cu_seqlens, ((size_t)a.n_seq + 1) * sizeof(int)),
                         range_of(a.slots, (size_t)a.n_seq * sizeof(int))};
    for (const Range& r : ins)
        if (overlaps(ry, r) || overlaps(ro, r)) return KDA_ERR_INVALID_ARG;
    if (overlaps(ry, rs) || overlaps(ry, ro)) return KDA_ERR_INVALID_ARG;
    if (a.state_out != a.state && overlaps(ro, rs)) return KDA_ERR_INVALID_ARG;   // the state itself may be updated
    return KDA_OK;
}

int run_conv(kda::ConvArgs& a, size_t tokens, size_t n_state, bool step, cudaStream_t stream) {
    const int rc = check_conv(a, tokens, n_state);
    if (rc != KDA_OK) return rc;
    a.status = kda::current_status_word();
    if (!a.status) return KDA_ERR_CUDA;
    const cudaError_t e = step ? kda::launch_short_conv_step(a, stream) : kda::launch_short_conv(a, stream);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

// ------------------------------------------------------------------ selective scan

int check_ssm(const kda::SsmArgs& a, size_t tokens, size_t n_state, bool step) {
    if (a.n_seq <= 0 || a.T < 0 || a.H <= 0 || a.G <= 0 || a.H % a.G != 0) return KDA_ERR_INVALID_ARG;
    if (!dtype_ok(a.dtype) || !head_dim_ok(a.N) || !head_dim_ok(a.P)) return KDA_ERR_UNSUPPORTED;
    const size_t es = elem_size(a.dtype), HP = (size_t)a.H * a.P, GN = (size_t)a.G * a.N;
    const long long lds[] = {a.ldx, a.lddt, a.ldb, a.ldc};
    const size_t widths[] = {HP, (size_t)a.H, GN, GN};
    for (int i = 0; i < 4; ++i) {
        if (lds[i] < (long long)widths[i] || lds[i] > kMostStride) return KDA_ERR_INVALID_ARG;
        if ((double)tokens * (double)lds[i] > kMostElements) return KDA_ERR_INVALID_ARG;
    }
    if ((double)n_state * HP * a.N > kMostElements || (double)a.n_seq * a.H > 1.0e8) return KDA_ERR_INVALID_ARG;
    if (!a.A || (tokens > 0 && (!a.x || !a.dt || !a.Bm || !a.Cm || !a.y))) return KDA_ERR_INVALID_ARG;
    if (step && !a.ST) return KDA_ERR_INVALID_ARG;
    const void* ptrs[] = {a.x, a.Bm, a.Cm, a.S0, a.y, a.ST};
    for (const void* p : ptrs)
        if (p && !aligned16(p)) return KDA_ERR_MISALIGNED;
    const long long vec = (long long)(16 / es);
    if (a.ldx % vec != 0 || a.ldb % vec != 0 || a.ldc % vec != 0) return KDA_ERR_MISALIGNED;
    if (!aligned(a.dt, es) || !aligned(a.A, 4) || !aligned(a.D, 4) || !aligned(a.dt_bias, 4) ||
        !aligned(a.cu_seqlens, 4) || !aligned(a.slots, 4))
        return KDA_ERR_MISALIGNED;
    const size_t sbytes = n_state * HP * a.N * sizeof(float);
    const Range ry = range_of(a.y, tokens * HP * es), rs = range_of(a.S0, sbytes), ro = range_of(a.ST, sbytes);
    const Range ins[] = {rows_of(a.x, tokens, HP, a.ldx, es),
                         rows_of(a.dt, tokens, a.H, a.lddt, es),
                         rows_of(a.Bm, tokens, GN, a.ldb, es),
                         rows_of(a.Cm, tokens, GN, a.ldc, es),
                         range_of(a.A, a.H * sizeof(float)),
                         range_of(a.D, a.H * sizeof(float)),
                         range_of(a.dt_bias, a.H * sizeof(float)),
                         range_of(a.cu_seqlens, ((size_t)a.n_seq + 1) * sizeof(int)),
                         range_of(a.slots, (size_t)a.n_seq * sizeof(int))};
    for (const Range& r : ins)
        if (overlaps(ry, r) || overlaps(ro, r)) return KDA_ERR_INVALID_ARG;
    if (overlaps(ry, rs) || overlaps(ry, ro)) return KDA_ERR_INVALID_ARG;
    if (a.S0 != a.ST && overlaps(rs, ro)) return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

int run_ssm(kda::SsmArgs& a, size_t tokens, int impl, size_t workspace_bytes, cudaStream_t stream) {
    if (impl != KDA_IMPL_AUTO && impl != KDA_IMPL_TCGEN05 && impl != KDA_IMPL_SIMT) return KDA_ERR_INVALID_ARG;
    const int rc = check_ssm(a, tokens, a.n_seq, false);
    if (rc != KDA_OK) return rc;
    const bool tc = impl != KDA_IMPL_SIMT && kda::ssm_tc_supports(a);
    if (impl == KDA_IMPL_TCGEN05 && !tc) return KDA_ERR_UNSUPPORTED;
    const size_t need = tc ? kda::ssm_tc_workspace(a.n_seq, (long long)tokens, a.H, a.N, a.P) : 0;
    if (need > 0) {
        if (!a.workspace || workspace_bytes < need) return KDA_ERR_INVALID_ARG;
        if (!aligned16(a.workspace)) return KDA_ERR_MISALIGNED;
        const size_t es = elem_size(a.dtype), HP = (size_t)a.H * a.P, GN = (size_t)a.G * a.N;
        const size_t sbytes = (size_t)a.n_seq * HP * a.N * sizeof(float);
        const Range rw = range_of(a.workspace, need);
        const Range others[] = {rows_of(a.x, tokens, HP, a.ldx, es), rows_of(a.dt, tokens, a.H, a.lddt, es),
                                rows_of(a.Bm, tokens, GN, a.ldb, es), rows_of(a.Cm, tokens, GN, a.ldc, es),
                                range_of(a.y, tokens * HP * es), range_of(a.S0, sbytes), range_of(a.ST, sbytes),
                                range_of(a.A, a.H * sizeof(float)), range_of(a.D, a.H * sizeof(float)),
                                range_of(a.dt_bias, a.H * sizeof(float)),
                                range_of(a.cu_seqlens, ((size_t)a.n_seq + 1) * sizeof(int))};
        for (const Range& r : others)
            if (overlaps(rw, r)) return KDA_ERR_INVALID_ARG;
    }
    if (tokens == 0 && !a.cu_seqlens) {
        if (!a.ST || a.S0 == a.ST) return KDA_OK;
        const size_t sbytes = (size_t)a.n_seq * a.H * a.N * a.P * sizeof(float);
        const cudaError_t e = a.S0 ? cudaMemcpyAsync(a.ST, a.S0, sbytes, cudaMemcpyDeviceToDevice, stream)
                                   : cudaMemsetAsync(a.ST, 0, sbytes, stream);
        return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
    }
    a.status = kda::current_status_word();
    if (!a.status) return KDA_ERR_CUDA;
    const cudaError_t e = tc ? kda::launch_ssm_tc(a, stream) : kda::launch_ssm_simt(a, stream);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

// ------------------------------------------------------------------ state pools

constexpr int kMostPools = 512;
constexpr int kMostIndices = 1 << 20;
constexpr double kMostSlotBytes = 1.0e13;

size_t pool_bytes(const kda_pool& p, int n_slots) {
    return (size_t)(n_slots - 1) * p.slot_stride + (size_t)(p.pieces - 1) * p.piece_stride + p.piece_bytes;
}

int check_pool(const kda_pool& p, int n_slots) {
    if (!p.base || p.pieces <= 0 || p.piece_bytes <= 0 || p.slot_stride < p.piece_bytes || p.pieces > (1 << 20) ||
        p.piece_bytes > (1ll << 40) || p.slot_stride > kMostStride || p.piece_stride > kMostStride ||
        (p.pieces > 1 && p.piece_stride < p.piece_bytes))
        return KDA_ERR_INVALID_ARG;
    // sizes and distances far from overflow: those of the pool in 64 bits, the parts of a slot in 32
    if ((double)n_slots * (double)p.slot_stride > kMostElements || (double)p.pieces * (double)p.piece_bytes > kMostSlotBytes)
        return KDA_ERR_INVALID_ARG;
    if (!aligned16(p.base) || p.slot_stride % 16 != 0 || p.piece_bytes % 16 != 0 ||
        (p.pieces > 1 && p.piece_stride % 16 != 0))
        return KDA_ERR_MISALIGNED;
    // no two runs of the pool overlap: slots whole one after another, or each run's slots one after another
    const long long slot = p.pieces > 1 ? (p.pieces - 1) * p.piece_stride + p.piece_bytes : p.piece_bytes;
    const long long run = (n_slots - 1) * p.slot_stride + p.piece_bytes;
    if (n_slots > 1 && p.slot_stride < slot && p.piece_stride < run) return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

struct Span {
    Range r;
    bool written;
};

// No written pool overlaps any other pool of the call (dst[k] may be src[k] itself).
bool pools_apart(const kda_pool* dst, const kda_pool* src, int n, int n_dst, int n_src) {
    Span spans[2 * kMostPools];
    int m = 0;
    for (int k = 0; k < n; ++k) {
        spans[m++] = Span{range_of(dst[k].base, pool_bytes(dst[k], n_dst)), true};
        if (src && src[k].base != dst[k].base)
            spans[m++] = Span{range_of(src[k].base, pool_bytes(src[k], n_src)), false};
    }
    std::sort(spans, spans + m, [](const Span& a, const Span& b) { return a.r.lo < b.r.lo; });
    uintptr_t any = 0, written = 0;
    for (int i = 0; i < m; ++i) {
        if (spans[i].r.lo < (spans[i].written ? any : written)) return false;
        any = std::max(any, spans[i].r.hi);
        if (spans[i].written) written = std::max(written, spans[i].r.hi);
    }
    return true;
}

int check_pools(const kda_pool* dst, const kda_pool* src, int n_pools, int n_dst, int n_src) {
    if (!dst || n_pools <= 0 || n_pools > kMostPools || n_dst <= 0 || (src && n_src <= 0)) return KDA_ERR_INVALID_ARG;
    for (int k = 0; k < n_pools; ++k) {
        int rc = check_pool(dst[k], n_dst);
        if (rc == KDA_OK && src) rc = check_pool(src[k], n_src);
        if (rc != KDA_OK) return rc;
        if (src) {
            if (dst[k].pieces != src[k].pieces || dst[k].piece_bytes != src[k].piece_bytes) return KDA_ERR_INVALID_ARG;
            // one base, one pool: the same slots in the same places
            if (dst[k].base == src[k].base &&
                (n_dst != n_src || dst[k].slot_stride != src[k].slot_stride ||
                 (dst[k].pieces > 1 && dst[k].piece_stride != src[k].piece_stride)))
                return KDA_ERR_INVALID_ARG;
        }
    }
    return pools_apart(dst, src, n_pools, n_dst, n_src) ? KDA_OK : KDA_ERR_INVALID_ARG;
}

// An index array that no written pool covers.
int check_indices(const int* idx, int n, const kda_pool* dst, int n_pools, int n_dst) {
    if (!idx) return KDA_ERR_INVALID_ARG;
    if (!aligned(idx, 4)) return KDA_ERR_MISALIGNED;
    const Range r = range_of(idx, (size_t)n * sizeof(int));
    for (int k = 0; k < n_pools; ++k)
        if (overlaps(r, range_of(dst[k].base, pool_bytes(dst[k], n_dst)))) return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

}  // namespace

extern "C" {

int kda_short_conv(const void* x, const void* weight, const void* bias, const void* state, void* y, void* state_out,
                   int B, int T, int C, int W, long long ldx, long long ldy, int activation, int dtype,
                   struct CUstream_st* stream) {
    if (B <= 0 || T < 0) return KDA_ERR_INVALID_ARG;
    kda::ConvArgs a{x, weight, bias, state, y, state_out, nullptr, B, T, C, W, ldx, ldy, activation, dtype,
                    nullptr, 0, nullptr};
    return run_conv(a, (size_t)B * T, B, false, stream);
}

int kda_short_conv_varlen(const void* x, const void* weight, const void* bias, const int* cu_seqlens,
                          const void* state, void* y, void* state_out, int N, int T_total, int C, int W,
                          long long ldx, long long ldy, int activation, int dtype, struct CUstream_st* stream) {
    if (N <= 0 || T_total < 0 || !cu_seqlens) return KDA_ERR_INVALID_ARG;
    if (!aligned(cu_seqlens, 4)) return KDA_ERR_MISALIGNED;
    kda::ConvArgs a{x, weight, bias, state, y, state_out, cu_seqlens, N, T_total, C, W, ldx, ldy, activation, dtype,
                    nullptr, 0, nullptr};
    return run_conv(a, (size_t)T_total, N, false, stream);
}

int kda_short_conv_step(const void* x, const void* weight, const void* bias, void* state, void* y, int B, int C,
                        int W, long long ldx, long long ldy, int activation, int dtype,
                        struct CUstream_st* stream) {
    if (B <= 0 || !state) return KDA_ERR_INVALID_ARG;
    kda::ConvArgs a{x, weight, bias, state, y, state, nullptr, B, 1, C, W, ldx, ldy, activation, dtype,
                    nullptr, 0, nullptr};
    return run_conv(a, B, B, true, stream);
}

int kda_short_conv_step_paged(const void* x, const void* weight, const void* bias, void* state_pool, int n_slots,
                              const int* slots, void* y, int B, int C, int W, long long ldx, long long ldy,
                              int activation, int dtype, struct CUstream_st* stream) {
    if (B <= 0 || !state_pool || !slots || n_slots <= 0) return KDA_ERR_INVALID_ARG;
    if (!aligned(slots, 4)) return KDA_ERR_MISALIGNED;
    kda::ConvArgs a{x, weight, bias, state_pool, y, state_pool, nullptr, B, 1, C, W, ldx, ldy, activation, dtype,
                    slots, n_slots, nullptr};
    return run_conv(a, B, n_slots, true, stream);
}

int kda_ssm_forward(const void* x, const void* dt, const float* A, const void* Bm, const void* Cm, const float* D,
                    const float* dt_bias, const float* S0, void* y, float* S_T, int B, int T, int H, int G, int N,
                    int P, long long ldx, long long lddt, long long ldb, long long ldc, int dtype, int impl,
                    void* workspace, size_t workspace_bytes, struct CUstream_st* stream) {
    if (B <= 0 || T < 0 || (double)B * T > kMostTokens) return KDA_ERR_INVALID_ARG;
    kda::SsmArgs a{x, dt, A, Bm, Cm, D, dt_bias, S0, y, S_T, nullptr, B, T, H, G, N, P, ldx, lddt, ldb, ldc, dtype,
                   nullptr, 0, nullptr, kda::wait_timeout_ns(), workspace, kda::wait_fault_mode()};
    return run_ssm(a, (size_t)B * T, impl, workspace_bytes, stream);
}

int kda_ssm_forward_varlen(const void* x, const void* dt, const float* A, const void* Bm, const void* Cm,
                           const int* cu_seqlens, const float* D, const float* dt_bias, const float* S0, void* y,
                           float* S_T, int n_seq, int T_total, int H, int G, int N, int P, long long ldx,
                           long long lddt, long long ldb, long long ldc, int dtype, int impl, void* workspace,
                           size_t workspace_bytes, struct CUstream_st* stream) {
    if (n_seq <= 0 || T_total < 0 || T_total > kMostTokens || !cu_seqlens) return KDA_ERR_INVALID_ARG;
    kda::SsmArgs a{x, dt, A, Bm, Cm, D, dt_bias, S0, y, S_T, cu_seqlens, n_seq, T_total, H, G, N, P, ldx, lddt, ldb,
                   ldc, dtype, nullptr, 0, nullptr, kda::wait_timeout_ns(), workspace, kda::wait_fault_mode()};
    return run_ssm(a, (size_t)T_total, impl, workspace_bytes, stream);
}

size_t kda_ssm_workspace(int n_seq, int T_total, int H, int N, int P, int dtype, int impl) {
    if (n_seq <= 0 || T_total < 0 || H <= 0 || !head_dim_ok(N) || !head_dim_ok(P) || dtype != KDA_DTYPE_BF16 ||
        (impl != KDA_IMPL_AUTO && impl != KDA_IMPL_TCGEN05))
        return 0;
    return kda::ssm_tc_workspace(n_seq, T_total, H, N, P);
}

int kda_ssm_decode_step(const void* x, const void* dt, const float* A, const void* Bm, const void* Cm, const float* D,
                        const float* dt_bias, float* S, void* y, int B, int H, int G, int N, int P, long long ldx,
                        long long lddt, long long ldb, long long ldc, int dtype, struct CUstream_st* stream) {
    kda::SsmArgs a{x, dt, A, Bm, Cm, D, dt_bias, S, y, S, nullptr, B, 1, H, G, N, P, ldx, lddt, ldb, ldc, dtype,
                   nullptr, 0, nullptr, kda::wait_timeout_ns(), nullptr, 0};
    const int rc = B <= 0 ? KDA_ERR_INVALID_ARG : check_ssm(a, B, B, true);
    if (rc != KDA_OK) return rc;
    a.status = kda::current_status_word();
    if (!a.status) return KDA_ERR_CUDA;
    return kda::launch_ssm_decode(a, stream) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

int kda_ssm_decode_step_paged(const void* x, const void* dt, const float* A, const void* Bm, const void* Cm,
                              const float* D, const float* dt_bias, float* S_pool, int n_slots, const int* slots,
                              void* y, int B, int H, int G, int N, int P, long long ldx, long long lddt,
                              long long ldb, long long ldc, int dtype, struct CUstream_st* stream) {
    if (!slots || n_slots <= 0 || B <= 0) return KDA_ERR_INVALID_ARG;
    kda::SsmArgs a{x, dt, A, Bm, Cm, D, dt_bias, S_pool, y, S_pool, nullptr, B, 1, H, G, N, P, ldx, lddt, ldb, ldc,
                   dtype, slots, n_slots, nullptr, kda::wait_timeout_ns(), nullptr, 0};
    const int rc = check_ssm(a, B, n_slots, true);
    if (rc != KDA_OK) return rc;
    a.status = kda::current_status_word();
    if (!a.status) return KDA_ERR_CUDA;
    return kda::launch_ssm_decode(a, stream) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

int kda_pool_copy(const kda_pool* dst, const kda_pool* src, int n_pools, int n_dst, int n_src, const int* src_idx,
                  const int* dst_idx, int n, struct CUstream_st* stream) {
    if (!src || n < 0 || n > kMostIndices) return KDA_ERR_INVALID_ARG;
    int rc = check_pools(dst, src, n_pools, n_dst, n_src);
    if (rc != KDA_OK || n == 0) return rc;
    rc = check_indices(src_idx, n, dst, n_pools, n_dst);
    if (rc == KDA_OK) rc = check_indices(dst_idx, n, dst, n_pools, n_dst);
    if (rc != KDA_OK) return rc;
    int* status = kda::current_status_word();
    if (!status) return KDA_ERR_CUDA;
    return kda::launch_pool_copy(dst, src, n_pools, n_dst, n_src, src_idx, dst_idx, n, status, stream) == cudaSuccess
               ? KDA_OK : KDA_ERR_CUDA;
}

int kda_pool_clear(const kda_pool* pools, int n_pools, int n_slots, const int* idx, int n,
                   struct CUstream_st* stream) {
    if (n < 0 || n > kMostIndices) return KDA_ERR_INVALID_ARG;
    int rc = check_pools(pools, nullptr, n_pools, n_slots, 0);
    if (rc != KDA_OK || n == 0) return rc;
    rc = check_indices(idx, n, pools, n_pools, n_slots);
    if (rc != KDA_OK) return rc;
    int* status = kda::current_status_word();
    if (!status) return KDA_ERR_CUDA;
    return kda::launch_pool_clear(pools, n_pools, n_slots, idx, n, status, stream) == cudaSuccess ? KDA_OK
                                                                                                  : KDA_ERR_CUDA;
}

int kda_pool_compact(const kda_pool* pools, int n_pools, int n_slots, const int* slots, const unsigned char* done,
                     int* slots_out, int B, int* workspace, struct CUstream_st* stream) {
    if (B <= 0 || B > kMostIndices) return KDA_ERR_INVALID_ARG;
    int rc = check_pools(pools, nullptr, n_pools, n_slots, 0);
    if (rc != KDA_OK) return rc;
    if (n_slots > 65536) return KDA_ERR_UNSUPPORTED;
    rc = check_indices(slots, B, pools, n_pools, n_slots);
    if (rc == KDA_OK) rc = check_indices(slots_out, B, pools, n_pools, n_slots);
    if (rc == KDA_OK) rc = check_indices(workspace, n_slots + 1, pools, n_pools, n_slots);
    if (rc != KDA_OK) return rc;
    const Range ro = range_of(slots_out, (size_t)B * sizeof(int)), rw = range_of(workspace, ((size_t)n_slots + 1) * sizeof(int));
    const Range rs = range_of(slots, (size_t)B * sizeof(int)), rd = range_of(done, (size_t)B);
    if (overlaps(ro, rw) || overlaps(ro, rd) || overlaps(rw, rd) || overlaps(rw, rs)) return KDA_ERR_INVALID_ARG;
    if (slots_out != slots && overlaps(ro, rs)) return KDA_ERR_INVALID_ARG;
    for (int k = 0; k < n_pools; ++k)
        if (overlaps(rd, range_of(pools[k].base, pool_bytes(pools[k], n_slots)))) return KDA_ERR_INVALID_ARG;
    int* status = kda::current_status_word();
    if (!status) return KDA_ERR_CUDA;
    return kda::launch_pool_compact(pools, n_pools, n_slots, slots, done, slots_out, B, workspace, status, stream) ==
                   cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
