// One token of the selective scan for every (b, h): S <- a S + B (s x)^T, y = S^T C + D x, with
// s = softplus(dt + dt_bias) and a = exp(s A); fp32 states updated in place.
//
// Bound by HBM like the KDA step: each state element is read and written once for four flops.  The
// update is independent per value column, so a state is split over CTAs by 64-column slices, each CTA
// of 256 threads holding 16-byte vectors of 32 (N = 128) or 16 (N = 64) state values per thread in
// registers between the read and the write.  There is no residual here, so the new state does not
// wait for any reduction: it is stored as soon as it is formed, and the column sums S^T C follow
// through warp shuffles and one shared-memory step.  One B200, 256 sequences x 96 heads of 128 x 128,
// bf16: 481 us for 3.2 GB, 1.03 of the measured copy rate (an update in place: the same lines go back).
#include "kda_serving.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kCols = 64;                 // state columns per CTA
constexpr int kLpr = kCols / 4;           // threads per row segment (float4 each)
constexpr int kRpp = kThreads / kLpr;     // rows per pass
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ float4 load4(const float* p) { return __ldg(reinterpret_cast<const float4*>(p)); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
    const uint2 r = __ldg(reinterpret_cast<const uint2*>(p));
    return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u), __uint_as_float(r.y << 16),
                       __uint_as_float(r.y & 0xffff0000u));
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

template <typename T, int N, int P>
__global__ void __launch_bounds__(kThreads)
kda_ssm_decode_kernel(const T* __restrict__ x, const T* __restrict__ dt, const float* __restrict__ A,
                      const T* __restrict__ Bm, const T* __restrict__ Cm, const float* __restrict__ D,
                      const float* __restrict__ dt_bias, float* __restrict__ S, T* __restrict__ y, int H, int rep,
                      long long ldx, long long lddt, long long ldb, long long ldc, const int* __restrict__ slots,
                      int n_slots, int* status) {
    constexpr int NSL = P / kCols;
    constexpr int RPT = N / kRpp;
    __shared__ float bs[N], cs[N];
    __shared__ float4 red[kWarps][kLpr];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int c4 = tid % kLpr, rg = tid / kLpr;
    const size_t bh = blockIdx.x / NSL;
    const int col = (int)(blockIdx.x % NSL) * kCols + 4 * c4;
    const size_t b = bh / H;
    const int h = (int)(bh % H);
    size_t at = bh;
    if (slots) {
        const int sl = slots[b];
        if (sl < 0) return;                       // inactive sequence: nothing is read or written
        if (sl >= n_slots) {
            if (tid == 0) report_status(status, KDA_ERR_INVALID_ARG);
            return;
        }
        at = (size_t)sl * H + h;
    }
    // everything else is asked for before the state, whose loads are many: what its update waits for comes first (481 us;
    // in the other order 490)
    const float raw = load_elem(dt, b * lddt + h), bias = dt_bias ? dt_bias[h] : 0.f, rate = A[h], skip = D ? D[h] : 0.f;
    const int g = h / rep;
    if (tid < N) bs[tid] = load_elem(Bm, b * ldb + (size_t)g * N + tid);
    else if (tid - 128 >= 0 && tid - 128 < N) cs[tid - 128] = load_elem(Cm, b * ldc + (size_t)g * N + (tid - 128));
    const float4 xv = load4(x + b * ldx + (size_t)h * P + col);
    float4* Sv = reinterpret_cast<float4*>(S + at * N * P + col);
    float4 s[RPT];
#pragma unroll
    for (int j = 0; j < RPT; ++j) s[j] = __ldcs(Sv + (size_t)(rg + j * kRpp) * (P / 4));
    const float step = softplus(raw + bias);
    const float a = token_decay(step * rate);
    const float4 u = make_float4(step * xv.x, step * xv.y, step * xv.z, step * xv.w);
    __syncthreads();
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int j = 0; j < RPT; ++j) {
        const int r = rg + j * kRpp;
        const float br = bs[r], cr = cs[r];
        s[j].x = fmaf(br, u.x, a * s[j].x); s[j].y = fmaf(br, u.y, a * s[j].y);
        s[j].z = fmaf(br, u.z, a * s[j].z); s[j].w = fmaf(br, u.w, a * s[j].w);
        __stcs(Sv + (size_t)r * (P / 4), s[j]);
        acc.x = fmaf(cr, s[j].x, acc.x); acc.y = fmaf(cr, s[j].y, acc.y);
        acc.z = fmaf(cr, s[j].z, acc.z); acc.w = fmaf(cr, s[j].w, acc.w);
    }
    // lanes c4 and c4 + 16 of a warp hold the same columns
    acc.x += __shfl_xor_sync(0xffffffffu, acc.x, kLpr); acc.y += __shfl_xor_sync(0xffffffffu, acc.y, kLpr);
    acc.z += __shfl_xor_sync(0xffffffffu, acc.z, kLpr); acc.w += __shfl_xor_sync(0xffffffffu, acc.w, kLpr);
    if (lane < kLpr) red[warp][lane] = acc;
    __syncthreads();
    if (tid < kLpr) {
        float4 o = red[0][tid];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) {
            const float4 t = red[w][tid];
            o.x += t.x; o.y += t.y; o.z += t.z; o.w += t.w;
        }
        if (D) {                              // this thread's columns: tid == c4
            o.x = fmaf(skip, xv.x, o.x); o.y = fmaf(skip, xv.y, o.y);
            o.z = fmaf(skip, xv.z, o.z); o.w = fmaf(skip, xv.w, o.w);
        }
        store4(y + bh * P + col, o);
    }
}

template <typename T, int N, int P>
cudaError_t launch_t(const SsmArgs& a, cudaStream_t s) {
    const unsigned grid = (unsigned)((size_t)a.n_seq * a.H * (P / kCols));
    kda_ssm_decode_kernel<T, N, P><<<grid, kThreads, 0, s>>>(
        static_cast<const T*>(a.x), static_cast<const T*>(a.dt), a.A, static_cast<const T*>(a.Bm),
        static_cast<const T*>(a.Cm), a.D, a.dt_bias, a.ST, static_cast<T*>(a.y), a.H, a.H / a.G, a.ldx, a.lddt, a.ldb,
        a.ldc, a.slots, a.n_slots, a.status);
    return cudaGetLastError();
}

template <typename T>
cudaError_t dispatch(const SsmArgs& a, cudaStream_t s) {
    if (a.N == 128) return a.P == 128 ? launch_t<T, 128, 128>(a, s) : launch_t<T, 128, 64>(a, s);
    return a.P == 128 ? launch_t<T, 64, 128>(a, s) : launch_t<T, 64, 64>(a, s);
}

}  // namespace

cudaError_t launch_ssm_decode(const SsmArgs& a, cudaStream_t s) {
    return a.dtype == KDA_DTYPE_BF16 ? dispatch<__nv_bfloat16>(a, s) : dispatch<float>(a, s);
}

}  // namespace kda
