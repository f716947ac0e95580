// The short causal convolution: y[t,c] = act(bias[c] + sum_{w<W} weight[c,w] u[t-(W-1)+w, c]), u the
// sequence after its last W-1 inputs (the state), for prompts and for single tokens.
//
// Bound by HBM: every element of x is read and every element of y written once for W multiply-adds
// and one sigmoid.  Lanes run along the channels with 16-byte vectors.  In the prompt kernel a thread
// carries the last W-1 inputs of its channels in registers down a strip of tokens, so x is read once
// except for the W-1 rows above each strip (mostly L2 hits: the strip above is in flight), and eight
// rows are loaded before the first is used.
//
// The first W-1 tokens of a sequence, which need the state, and the state after its last token belong
// to blocks of their own, one per sequence and channel range: those read everything before they write
// the new state, and no other block touches it, so state_out may be the state itself.
#include "kda_serving.cuh"

namespace kda {
namespace {

constexpr int kThreads = 128;
constexpr int kAhead = 8;       // rows in flight per thread

template <typename T>
struct Vec {
    static constexpr int n = 16 / sizeof(T);
};

__device__ __forceinline__ void unpack(const uint4& r, float (&f)[4]) {
    f[0] = __uint_as_float(r.x); f[1] = __uint_as_float(r.y); f[2] = __uint_as_float(r.z); f[3] = __uint_as_float(r.w);
}
__device__ __forceinline__ void unpack(const uint4& r, float (&f)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
__device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// v sigmoid(v).  bf16 outputs (relative step 2^-8) take the approximate exponential and division
// (relative error about 2^-21), fp32 outputs the accurate ones.
__device__ __forceinline__ float silu(float v, const __nv_bfloat16*) { return __fdividef(v, 1.f + __expf(-v)); }
__device__ __forceinline__ float silu(float v, const float*) { return v / (1.f + expf(-v)); }

// Weights and bias of a thread's channels, and the filter applied to a window of inputs.
template <typename T, int W>
struct Filter {
    static constexpr int V = Vec<T>::n;
    float w[W][V], b[V];
    bool act;

    __device__ __forceinline__ void load(const T* weight, const T* bias, int c, bool silu_on) {
        // weight rows c .. c+V-1 are V*W contiguous elements, 16-byte aligned since c is a multiple of V
        float flat[W * V];
#pragma unroll
        for (int i = 0; i < W; ++i) {
            float t[V];
            unpack(__ldg(reinterpret_cast<const uint4*>(weight + (size_t)c * W) + i), t);
#pragma unroll
            for (int j = 0; j < V; ++j) flat[i * V + j] = t[j];
        }
#pragma unroll
        for (int i = 0; i < W; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) w[i][j] = flat[j * W + i];
        if (bias) {
            unpack(__ldg(reinterpret_cast<const uint4*>(bias + c)), b);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) b[j] = 0.f;
        }
        act = silu_on;
    }
    // win: the W-1 inputs before `u`, oldest first; shifted by one afterwards
    __device__ __forceinline__ uint4 apply(float (&win)[W - 1][V], const uint4& u) const {
        float cur[V], out[V];
        unpack(u, cur);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float a = b[j];
#pragma unroll
            for (int i = 0; i < W - 1; ++i) a = fmaf(w[i][j], win[i][j], a);
            out[j] = fmaf(w[W - 1][j], cur[j], a);
        }
        push(win, cur);
        if (act) {
#pragma unroll
            for (int j = 0; j < V; ++j) out[j] = silu(out[j], static_cast<const T*>(nullptr));
        }
        return pack(out);
    }
    __device__ __forceinline__ static void push(float (&win)[W - 1][V], const float (&cur)[V]) {
#pragma unroll
        for (int i = 0; i + 1 < W - 1; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) win[i][j] = win[i + 1][j];
#pragma unroll
        for (int j = 0; j < V; ++j) win[W - 2][j] = cur[j];
    }
};

template <typename T>
__device__ __forceinline__ uint4 load_row(const T* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }

// Grid: channel ranges fastest, then one block per sequence (start and state), then the strips.
template <typename T, int W>
__global__ void __launch_bounds__(kThreads)
kda_short_conv_kernel(const T* __restrict__ x, const T* __restrict__ weight, const T* __restrict__ bias,
                      const T* state, T* __restrict__ y, T* state_out, const int* __restrict__ cu_seqlens,
                      int n_seq, int T_all, int C, long long ldx, long long ldy, int act, int strip, int n_cb,
                      int strips_per_seq, int* status) {
    constexpr int V = Vec<T>::n;
    const int cb = blockIdx.x % n_cb;
    const int part = blockIdx.x / n_cb;
    bool valid = true;
    if (cu_seqlens) {
        valid = packed_offsets_valid(cu_seqlens, n_seq, T_all);
        if (!valid && threadIdx.x == 0) report_status(status, KDA_ERR_INVALID_ARG);
    }
    const int c = (cb * kThreads + (int)threadIdx.x) * V;
    if (c >= C) return;
    Filter<T, W> f;
    f.load(weight, bias, c, act != 0);
    float win[W - 1][V];
    const uint4 zero = make_uint4(0, 0, 0, 0);

    if (part < n_seq) {
        // the first W-1 tokens of sequence `part`, then the state after its last
        size_t base = (size_t)part * T_all;
        int len = T_all;
        if (cu_seqlens) {
            base = valid ? (size_t)cu_seqlens[part] : 0;
            len = valid ? cu_seqlens[part + 1] - cu_seqlens[part] : 0;
        }
        const T* xs = x + base * ldx + c;
        const T* st = state ? state + (size_t)part * (W - 1) * C + c : nullptr;
        uint4 raw[W - 1], last[W - 1];
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
            raw[i] = st ? *reinterpret_cast<const uint4*>(st + (size_t)i * C) : zero;
            unpack(raw[i], win[i]);
        }
#pragma unroll
        for (int i = 0; i < W - 1; ++i)
            if (i < len) {
                const uint4 r = f.apply(win, load_row(xs + (size_t)i * ldx));
                *reinterpret_cast<uint4*>(y + (base + i) * ldy + c) = r;
            }
        if (!state_out) return;
        // entry i of the new state is input len - (W-1) + i: of x, or (shorter sequences) of the state
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
            const int t = len - (W - 1) + i;
            if (t >= 0) {
                last[i] = load_row(xs + (size_t)t * ldx);
            } else {
                last[i] = zero;
#pragma unroll
                for (int k = 0; k < W - 1; ++k)
                    if (k == len + i) last[i] = raw[k];
            }
        }
#pragma unroll
        for (int i = 0; i < W - 1; ++i)
            *reinterpret_cast<uint4*>(state_out + ((size_t)part * (W - 1) + i) * C + c) = last[i];
        return;
    }

    // a strip of tokens; tokens nearer than W-1 to their sequence's start belong to the blocks above
    const int s = part - n_seq;
    size_t row0 = 0;            // row of token 0 of this strip's token axis
    int t0, t1, n = 0, start = 0, end = T_all;
    if (cu_seqlens) {
        if (!valid) return;
        t0 = s * strip;
        t1 = min(t0 + strip, cu_seqlens[n_seq]);
        if (t0 >= t1) return;
        // the last sequence that starts at or before t0 (empty ones before it are passed over)
        int lo = 0, hi = n_seq;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (__ldg(cu_seqlens + mid + 1) > t0) hi = mid;
            else lo = mid + 1;
        }
        n = lo;
        start = cu_seqlens[n];
        end = cu_seqlens[n + 1];
    } else {
        row0 = (size_t)(s / strips_per_seq) * T_all;
        t0 = (s % strips_per_seq) * strip;
        t1 = min(t0 + strip, T_all);
    }
    const T* xs = x + row0 * ldx + c;
    T* ys = y + row0 * ldy + c;
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
        const int t = t0 - (W - 1) + i;
        unpack(t >= 0 ? load_row(xs + (size_t)t * ldx) : zero, win[i]);
    }
    for (int tb = t0; tb < t1; tb += kAhead) {
        uint4 raw[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) raw[i] = tb + i < t1 ? load_row(xs + (size_t)(tb + i) * ldx) : zero;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int t = tb + i;
            if (t < t1) {
                while (t >= end) {      // packed only: the next sequence (t < cu[n_seq], so there is one)
                    ++n;
                    start = end;
                    end = __ldg(cu_seqlens + n + 1);
                }
                const uint4 r = f.apply(win, raw[i]);
                if (t - start >= W - 1) *reinterpret_cast<uint4*>(ys + (size_t)t * ldy) = r;
            }
        }
    }
}

constexpr int kStepSeqs = 2;    // sequences in flight per thread of the step kernel

template <typename T, int W>
__global__ void __launch_bounds__(kThreads)
kda_short_conv_step_kernel(const T* __restrict__ x, const T* __restrict__ weight, const T* __restrict__ bias, T* state,
                           T* __restrict__ y, int B, int C, long long ldx, long long ldy, int act, int n_cb,
                           int seqs, const int* __restrict__ slots, int n_slots, int* status) {
    constexpr int V = Vec<T>::n;
    const int cb = blockIdx.x % n_cb;
    const int b0 = (blockIdx.x / n_cb) * seqs;
    const int c = (cb * kThreads + (int)threadIdx.x) * V;
    if (c >= C) return;
    Filter<T, W> f;
    f.load(weight, bias, c, act != 0);
    const int b1 = min(b0 + seqs, B);
    for (int bb = b0; bb < b1; bb += kStepSeqs) {
        uint4 u[kStepSeqs], raw[kStepSeqs][W - 1];
        long long at[kStepSeqs];
#pragma unroll
        for (int k = 0; k < kStepSeqs; ++k) {
            const int b = bb + k;
            at[k] = -1;
            if (b < b1) {
                at[k] = slots ? __ldg(slots + b) : b;
                if (slots && at[k] >= n_slots) {
                    report_status(status, KDA_ERR_INVALID_ARG);
                    at[k] = -1;
                }
            }
            if (at[k] >= 0) {
                u[k] = load_row(x + (size_t)b * ldx + c);
#pragma unroll
                for (int i = 0; i < W - 1; ++i)
                    raw[k][i] = *reinterpret_cast<const uint4*>(state + ((size_t)at[k] * (W - 1) + i) * C + c);
            }
        }
#pragma unroll
        for (int k = 0; k < kStepSeqs; ++k) {
            if (at[k] < 0) continue;
            float win[W - 1][V];
#pragma unroll
            for (int i = 0; i < W - 1; ++i) unpack(raw[k][i], win[i]);
            *reinterpret_cast<uint4*>(y + (size_t)(bb + k) * ldy + c) = f.apply(win, u[k]);
            T* st = state + (size_t)at[k] * (W - 1) * C + c;
#pragma unroll
            for (int i = 0; i + 1 < W - 1; ++i) *reinterpret_cast<uint4*>(st + (size_t)i * C) = raw[k][i + 1];
            *reinterpret_cast<uint4*>(st + (size_t)(W - 2) * C) = u[k];
        }
    }
}

template <typename T, int W>
cudaError_t launch_prompt(const ConvArgs& a, cudaStream_t s) {
    constexpr int V = Vec<T>::n;
    const int n_cb = (a.C / V + kThreads - 1) / kThreads;
    // a short strip gives small problems enough blocks, a long one re-reads fewer rows above it
    const long long tokens = a.cu_seqlens ? a.T : (long long)a.n_seq * a.T;
    int strip = 8;
    while (strip < 64 && tokens / (2 * strip) * n_cb >= 148 * 16) strip *= 2;
    const int per_seq = (a.T + strip - 1) / strip;
    const long long strips = a.cu_seqlens ? per_seq : (long long)a.n_seq * per_seq;
    const long long grid = (a.n_seq + strips) * n_cb;
    if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    kda_short_conv_kernel<T, W><<<(unsigned)grid, kThreads, 0, s>>>(
        static_cast<const T*>(a.x), static_cast<const T*>(a.weight), static_cast<const T*>(a.bias),
        static_cast<const T*>(a.state), static_cast<T*>(a.y), static_cast<T*>(a.state_out), a.cu_seqlens, a.n_seq,
        a.T, a.C, a.ldx, a.ldy, a.act, strip, n_cb, per_seq, a.status);
    return cudaGetLastError();
}

template <typename T, int W>
cudaError_t launch_step(const ConvArgs& a, cudaStream_t s) {
    constexpr int V = Vec<T>::n;
    const int n_cb = (a.C / V + kThreads - 1) / kThreads;
    int seqs = kStepSeqs;    // more sequences per block share the weights, once there are blocks enough
    while (seqs < 8 && (long long)a.n_seq / (2 * seqs) * n_cb >= 148 * 8) seqs *= 2;
    const long long grid = (long long)((a.n_seq + seqs - 1) / seqs) * n_cb;
    if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    kda_short_conv_step_kernel<T, W><<<(unsigned)grid, kThreads, 0, s>>>(
        static_cast<const T*>(a.x), static_cast<const T*>(a.weight), static_cast<const T*>(a.bias),
        static_cast<T*>(a.state_out), static_cast<T*>(a.y), a.n_seq, a.C, a.ldx, a.ldy, a.act, n_cb, seqs, a.slots,
        a.n_slots, a.status);
    return cudaGetLastError();
}

template <typename T>
cudaError_t dispatch(const ConvArgs& a, bool step, cudaStream_t s) {
    if (a.W == 2) return step ? launch_step<T, 2>(a, s) : launch_prompt<T, 2>(a, s);
    if (a.W == 3) return step ? launch_step<T, 3>(a, s) : launch_prompt<T, 3>(a, s);
    return step ? launch_step<T, 4>(a, s) : launch_prompt<T, 4>(a, s);
}

}  // namespace

cudaError_t launch_short_conv(const ConvArgs& a, cudaStream_t s) {
    return a.dtype == KDA_DTYPE_BF16 ? dispatch<__nv_bfloat16>(a, false, s) : dispatch<float>(a, false, s);
}

cudaError_t launch_short_conv_step(const ConvArgs& a, cudaStream_t s) {
    return a.dtype == KDA_DTYPE_BF16 ? dispatch<__nv_bfloat16>(a, true, s) : dispatch<float>(a, true, s);
}

}  // namespace kda
