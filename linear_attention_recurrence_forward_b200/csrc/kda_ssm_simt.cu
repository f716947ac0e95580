// The selective scan in fp32 on CUDA cores, token by token (every dtype, N and P in {64, 128}): the
// library's fp32 path, as the tensor-core kernel's operands are bf16.
//
//   S <- a_t S + B_t (s_t x_t)^T,  y_t = S^T C_t + D x_t,   a_t = exp(s_t A), s_t = softplus(dt_t + dt_bias)
//
// The P columns of S never mix, so a CTA takes one (sequence, head) and 16 columns: four warps of four
// columns, the N rows spread over 16 lanes.  A lane holds N/16 rows x 2 columns of the state in
// registers for the whole sequence.  There is no residual, so nothing in the token loop waits for a
// reduction: a lane keeps its partial column sums of 16 tokens, and a reduce-scatter over the 16 lanes
// (30 shuffles for 16 tokens x 2 columns; a sum per token would take 128) leaves lane l with token l.
// Tokens come 16 at a time through double-buffered shared memory, copied asynchronously (fp32) while
// the stage before is computed.  Bound by the chain through the tokens: 256 tokens x 2 heads of
// 64 x 64 in fp32 take 22 us, a serial loop with synchronous loads and sums per token 82 us.
#include "kda_serving.cuh"

namespace kda {
namespace {

constexpr int kThreads = 128;
constexpr int kCols = 16;        // state columns per CTA
constexpr int kTok = 16;         // tokens per stage

// 16 bytes of a row into shared memory as fp32: asynchronously where they are fp32 already
__device__ __forceinline__ void copy16(float* to, const float* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from)
                 : "memory");
}
__device__ __forceinline__ void copy16(float* to, const __nv_bfloat16* from) {
    const uint4 r = __ldg(reinterpret_cast<const uint4*>(from));
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        to[2 * i] = __uint_as_float(w[i] << 16);
        to[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

template <typename T, int N>
__global__ void __launch_bounds__(kThreads)
kda_ssm_simt_kernel(const T* __restrict__ x, const T* __restrict__ dt, const float* __restrict__ A,
                    const T* __restrict__ Bm, const T* __restrict__ Cm, const float* __restrict__ D,
                    const float* __restrict__ dt_bias, const float* S0, T* __restrict__ y, float* ST,
                    const int* __restrict__ cu_seqlens, int n_seq, int T_all, int H, int rep, int P, long long ldx,
                    long long lddt, long long ldb, long long ldc, int* status) {
    constexpr int RPL = N / 16;          // rows per lane
    __shared__ __align__(16) float bs[2][kTok][N], cs[2][kTok][N];
    __shared__ __align__(16) float xs[2][kTok][kCols];
    __shared__ float2 as[2][kTok];       // (a_t, s_t)
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nsl = P / kCols;
    const int col0 = (int)(blockIdx.x % nsl) * kCols;
    const size_t bh = blockIdx.x / nsl;
    const int b = (int)(bh / H), h = (int)(bh % H), g = h / rep;
    size_t base = (size_t)b * T_all;
    int len = T_all;
    if (cu_seqlens) {
        const bool valid = packed_offsets_valid(cu_seqlens, n_seq, T_all);
        if (!valid && tid == 0) report_status(status, KDA_ERR_INVALID_ARG);
        base = valid ? (size_t)cu_seqlens[b] : 0;
        len = valid ? cu_seqlens[b + 1] - cu_seqlens[b] : 0;
    }
    const int rl = lane & 15;                              // rows 4 rl + 64 k + (0..3)
    const int cl = 4 * warp + 2 * (lane >> 4);             // columns cl, cl + 1 of the slice
    float s[RPL][2];
#pragma unroll
    for (int i = 0; i < RPL; ++i) {
        const int r = 4 * rl + 64 * (i / 4) + i % 4;
        const float2 v = S0 ? *reinterpret_cast<const float2*>(S0 + (bh * N + r) * P + col0 + cl) : make_float2(0.f, 0.f);
        s[i][0] = v.x;
        s[i][1] = v.y;
    }
    const float rate = A[h], bias = dt_bias ? dt_bias[h] : 0.f, skip = D ? D[h] : 0.f;

    // dt of the stage's tokens is loaded a stage ahead of its use, by one thread each
    auto load_dt = [&](int t0) { return tid < kTok && t0 + tid < len ? load_elem(dt, (base + t0 + tid) * lddt + h) : 0.f; };
    auto stage = [&](int t0, int buf) {
        const int n = min(kTok, len - t0);
        constexpr int V = 16 / sizeof(T);              // elements of a 16-byte vector
        constexpr int VN = N / V, VX = kCols / V;
        for (int i = tid; i < n * VN; i += kThreads) {
            const int t = i / VN, k = (i % VN) * V;
            const size_t row = base + t0 + t;
            copy16(&bs[buf][t][k], Bm + row * ldb + (size_t)g * N + k);
            copy16(&cs[buf][t][k], Cm + row * ldc + (size_t)g * N + k);
        }
        for (int i = tid; i < n * VX; i += kThreads) {
            const int t = i / VX, k = (i % VX) * V;
            copy16(&xs[buf][t][k], x + (base + t0 + t) * ldx + (size_t)h * P + col0 + k);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto stage_dt = [&](float v, int t0, int buf) {
        if (tid < kTok && t0 + tid < len) {
            const float st = softplus(v + bias);
            as[buf][tid] = make_float2(token_decay(st * rate), st);
        }
    };

    if (len > 0) {
        stage(0, 0);
        stage_dt(load_dt(0), 0, 0);
    }
    float next_dt = load_dt(kTok);
    for (int t0 = 0, buf = 0; t0 < len; t0 += kTok, buf ^= 1) {
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();                               // this stage is in; the other buffer is free
        if (t0 + kTok < len) {
            stage(t0 + kTok, buf ^ 1);
            stage_dt(next_dt, t0 + kTok, buf ^ 1);
            next_dt = load_dt(t0 + 2 * kTok);
        }
        const int n = min(kTok, len - t0);
        float yp[kTok][2];
        auto token = [&](int t) {
            const float2 at = as[buf][t];
            const float2 xv = *reinterpret_cast<const float2*>(&xs[buf][t][cl]);
            const float u0 = at.y * xv.x, u1 = at.y * xv.y;
            float y0 = 0.f, y1 = 0.f;
#pragma unroll
            for (int k = 0; k < RPL / 4; ++k) {
                const float4 bv = *reinterpret_cast<const float4*>(&bs[buf][t][4 * rl + 64 * k]);
                const float4 cv = *reinterpret_cast<const float4*>(&cs[buf][t][4 * rl + 64 * k]);
                const float br[4] = {bv.x, bv.y, bv.z, bv.w}, cr[4] = {cv.x, cv.y, cv.z, cv.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s[4 * k + i][0] = fmaf(br[i], u0, at.x * s[4 * k + i][0]);
                    s[4 * k + i][1] = fmaf(br[i], u1, at.x * s[4 * k + i][1]);
                    y0 = fmaf(cr[i], s[4 * k + i][0], y0);
                    y1 = fmaf(cr[i], s[4 * k + i][1], y1);
                }
            }
            yp[t][0] = y0;
            yp[t][1] = y1;
        };
        if (n == kTok) {
            // no branch between the tokens: the loads of later ones go out ahead
#pragma unroll
            for (int t = 0; t < kTok; ++t) token(t);
        } else {
#pragma unroll
            for (int t = 0; t < kTok; ++t) {
                yp[t][0] = yp[t][1] = 0.f;
                if (t < n) token(t);
            }
        }
        // sum over the 16 lanes; lane rl keeps token rl
#pragma unroll
        for (int half = kTok / 2; half > 0; half >>= 1) {
            const bool upper = rl & half;
#pragma unroll
            for (int t = 0; t < half; ++t)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const float give = upper ? yp[t][q] : yp[t + half][q], keep = upper ? yp[t + half][q] : yp[t][q];
                    yp[t][q] = keep + __shfl_xor_sync(0xffffffffu, give, half);
                }
        }
        if (rl < n) {
            const float2 xv = *reinterpret_cast<const float2*>(&xs[buf][rl][cl]);
            const size_t o = ((base + t0 + rl) * H + h) * P + col0 + cl;
            store_elem(y, o, D ? fmaf(skip, xv.x, yp[0][0]) : yp[0][0]);
            store_elem(y, o + 1, D ? fmaf(skip, xv.y, yp[0][1]) : yp[0][1]);
        }
    }
    if (!ST) return;
#pragma unroll
    for (int i = 0; i < RPL; ++i) {
        const int r = 4 * rl + 64 * (i / 4) + i % 4;
        *reinterpret_cast<float2*>(ST + (bh * N + r) * P + col0 + cl) = make_float2(s[i][0], s[i][1]);
    }
}

template <typename T>
cudaError_t launch_t(const SsmArgs& a, cudaStream_t s) {
    const long long grid = (long long)a.n_seq * a.H * (a.P / kCols);
    if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    auto run = [&](auto kernel) {
        kernel<<<(unsigned)grid, kThreads, 0, s>>>(
            static_cast<const T*>(a.x), static_cast<const T*>(a.dt), a.A, static_cast<const T*>(a.Bm),
            static_cast<const T*>(a.Cm), a.D, a.dt_bias, a.S0, static_cast<T*>(a.y), a.ST, a.cu_seqlens, a.n_seq, a.T,
            a.H, a.H / a.G, a.P, a.ldx, a.lddt, a.ldb, a.ldc, a.status);
    };
    if (a.N == 128) run(kda_ssm_simt_kernel<T, 128>);
    else run(kda_ssm_simt_kernel<T, 64>);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_ssm_simt(const SsmArgs& a, cudaStream_t s) {
    return a.dtype == KDA_DTYPE_BF16 ? launch_t<__nv_bfloat16>(a, s) : launch_t<float>(a, s);
}

}  // namespace kda
