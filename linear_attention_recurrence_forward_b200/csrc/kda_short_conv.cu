// The short causal convolution: y[t,c] = act(bias[c] + sum_{w<W} weight[c,w] u[t-(W-1)+w, c]), u the
// sequence after its last W-1 inputs (the state), for prompts and for single tokens.
//
// Bound by HBM: every element of x is read and every element of y written once for W multiply-adds
// and one sigmoid.  In the prompt kernel a thread carries the last W-1 inputs of its four channels in
// registers down a strip of tokens, so x is read once except for the W-1 rows above each strip (mostly
// L2 hits: the strip above is in flight), and loads 16 (fp32: 8) rows before it uses the first.  In bf16
// the arithmetic is nearly as long as the traffic: the f32x2 instructions take two channels at once,
// and four channels a thread keep registers low enough for five blocks an SM.  One B200, 16384 x 12288
// bf16 with SiLU: 150 to 154 us (0.80 to 0.82 of the measured copy rate; 127 to 129 us without the
// activation); eight channels a thread with 16-byte loads 159 us, scalar arithmetic 222 us; fp32 262 us (0.94;
// 252 us without the activation).
//
// The first W-1 tokens of a sequence, which need the state, and the state after its last token belong
// to blocks of their own, one per sequence and channel range: those read everything before they write
// the new state, and no other block touches it, so state_out may be the state itself.
#include "kda_serving.cuh"

namespace kda {
namespace {

constexpr int kThreads = 128;

constexpr int kVec = 4;          // channels per thread

// a thread's channels of one row, as they lie in memory
template <typename T>
struct Raw;
template <>
struct Raw<float> {
    using type = uint4;
    static constexpr int ahead = 8, blocks = 1;      // rows in flight per thread, blocks per SM asked of the compiler
};
template <>
struct Raw<__nv_bfloat16> {
    using type = uint2;
    static constexpr int ahead = 16, blocks = 5;
};

// Channels go in pairs, two fp32 lanes of one 64-bit register (the f32x2 instructions).
__device__ __forceinline__ uint64_t pair2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 split2(uint64_t p) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(p));
    return f;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ void unpack(const uint4& r, uint64_t (&f)[2]) {
    f[0] = pair2(__uint_as_float(r.x), __uint_as_float(r.y));
    f[1] = pair2(__uint_as_float(r.z), __uint_as_float(r.w));
}
__device__ __forceinline__ void unpack(const uint2& r, uint64_t (&f)[2]) {
    f[0] = pair2(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u));
    f[1] = pair2(__uint_as_float(r.y << 16), __uint_as_float(r.y & 0xffff0000u));
}
__device__ __forceinline__ void pack(const uint64_t (&f)[2], uint4& r) {
    const float2 a = split2(f[0]), b = split2(f[1]);
    r = make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
}
__device__ __forceinline__ void pack(const uint64_t (&f)[2], uint2& r) {
    const float2 a = split2(f[0]), b = split2(f[1]);
    const __nv_bfloat162 p = __floats2bfloat162_rn(a.x, a.y), q = __floats2bfloat162_rn(b.x, b.y);
    r = make_uint2(*reinterpret_cast<const uint32_t*>(&p), *reinterpret_cast<const uint32_t*>(&q));
}

// SiLU of both lanes for bf16 outputs: v / (1 + 2^(-v log2 e)) by the hardware exponential and reciprocal.  Each is off
// by about 2^-22, and the exponent's rounding by |v log2 e| 2^-24 of the result, 2^-17 at most: far below half a bf16
// step of 2^-8.  Below -87.3, where the reciprocal has no normal value, the result is zero (exact: under 1e-36).
__device__ __forceinline__ uint64_t silu2(uint64_t v, __nv_bfloat16) {
    const float2 a = split2(mul2(v, pair2(-1.4426950408889634f, -1.4426950408889634f)));
    float ex, ey, rx, ry;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(ex) : "f"(a.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(ey) : "f"(a.y));
    const float2 d = split2(add2(pair2(ex, ey), pair2(1.f, 1.f)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(rx) : "f"(d.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(ry) : "f"(d.y));
    return mul2(v, pair2(rx, ry));
}
// And for fp32 outputs: with e = exp(-|v|), v / (1 + e) or, below zero, v e / (1 + e); nothing overflows.  e is
// 2^p' (1 + r ln 2): p' the rounded product of -|v| and log2 e, r what the rounding left out, which a fused multiply-add
// gives exactly, and the low part of log2 e.  Off by 10 * 2^-24 of the value at most: 4 from the exponential, 2 from the
// reciprocal, one from each of four roundings.  16384 x 12288: 262 us, with expf and a division 350 us, with the bf16
// form (57 to 80 * 2^-24 off between -20 and -87, zero below) 256 us.
__device__ __forceinline__ uint64_t silu2(uint64_t v, float) {
    constexpr float kLog2e = 1.44269504f, kLog2eLow = (float)(1.4426950408889634 - (double)kLog2e);
    const float2 x = split2(v);
    const uint64_t mag = pair2(fminf(fabsf(x.x), 128.f), fminf(fabsf(x.y), 128.f));     // e is zero from there on
    const uint64_t p = mul2(mag, pair2(kLog2e, kLog2e));
    uint64_t r = fma2(mag, pair2(-kLog2e, -kLog2e), p);
    r = fma2(mag, pair2(-kLog2eLow, -kLog2eLow), r);
    const float2 q = split2(p);
    float ex, ey, rx, ry;
    asm("ex2.approx.f32 %0, %1;" : "=f"(ex) : "f"(-q.x));
    asm("ex2.approx.f32 %0, %1;" : "=f"(ey) : "f"(-q.y));
    uint64_t e = pair2(ex, ey);
    e = fma2(e, mul2(r, pair2(0.69314718f, 0.69314718f)), e);
    const float2 d = split2(add2(e, pair2(1.f, 1.f))), w = split2(e);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(rx) : "f"(d.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(ry) : "f"(d.y));
    return mul2(mul2(v, pair2(x.x < 0.f ? w.x : 1.f, x.y < 0.f ? w.y : 1.f)), pair2(rx, ry));
}

// Weights and bias of a thread's channels, and the filter applied to a window of inputs.
template <typename T, int W>
struct Filter {
    static constexpr int V = kVec, H = V / 2;
    using R = typename Raw<T>::type;
    uint64_t w[W][H], b[H];
    bool act;

    __device__ __forceinline__ void load(const T* weight, const T* bias, int c, bool silu_on) {
        // weight rows c .. c+V-1 are V*W contiguous elements, 16-byte aligned since c is a multiple of V
        float flat[W * V];
#pragma unroll
        for (int i = 0; i < W; ++i) {
            uint64_t t[H];
            unpack(__ldg(reinterpret_cast<const R*>(weight + (size_t)c * W) + i), t);
#pragma unroll
            for (int j = 0; j < H; ++j) {
                const float2 f = split2(t[j]);
                flat[i * V + 2 * j] = f.x;
                flat[i * V + 2 * j + 1] = f.y;
            }
        }
#pragma unroll
        for (int i = 0; i < W; ++i)
#pragma unroll
            for (int j = 0; j < H; ++j) w[i][j] = pair2(flat[2 * j * W + i], flat[(2 * j + 1) * W + i]);
        if (bias) {
            unpack(__ldg(reinterpret_cast<const R*>(bias + c)), b);
        } else {
#pragma unroll
            for (int j = 0; j < H; ++j) b[j] = 0;
        }
        act = silu_on;
    }
    // win: the W-1 inputs before `u`, oldest first; shifted by one afterwards
    __device__ __forceinline__ R apply(uint64_t (&win)[W - 1][H], const R& u) const {
        uint64_t cur[H], out[H];
        unpack(u, cur);
#pragma unroll
        for (int j = 0; j < H; ++j) {
            uint64_t a = b[j];
#pragma unroll
            for (int i = 0; i < W - 1; ++i) a = fma2(w[i][j], win[i][j], a);
            out[j] = fma2(w[W - 1][j], cur[j], a);
        }
#pragma unroll
        for (int j = 0; j < H; ++j) {
#pragma unroll
            for (int i = 0; i + 1 < W - 1; ++i) win[i][j] = win[i + 1][j];
            win[W - 2][j] = cur[j];
        }
        if (act) {
#pragma unroll
            for (int j = 0; j < H; ++j) out[j] = silu2(out[j], T());
        }
        R r;
        pack(out, r);
        return r;
    }
};

template <typename T>
__device__ __forceinline__ typename Raw<T>::type load_row(const T* p) {
    return __ldg(reinterpret_cast<const typename Raw<T>::type*>(p));
}

// Grid: channel ranges fastest, then one block per sequence (start and state), then the strips.
template <typename T, int W>
__global__ void __launch_bounds__(kThreads, Raw<T>::blocks)
kda_short_conv_kernel(const T* __restrict__ x, const T* __restrict__ weight, const T* __restrict__ bias,
                      const T* state, T* __restrict__ y, T* state_out, const int* __restrict__ cu_seqlens,
                      int n_seq, int T_all, int C, long long ldx, long long ldy, int act, int strip, int n_cb,
                      int strips_per_seq, int* status) {
    constexpr int V = kVec;
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
    uint64_t win[W - 1][V / 2];
    using R = typename Raw<T>::type;
    const R zero{};

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
        R raw[W - 1], last[W - 1];
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
            raw[i] = st ? *reinterpret_cast<const R*>(st + (size_t)i * C) : zero;
            unpack(raw[i], win[i]);
        }
#pragma unroll
        for (int i = 0; i < W - 1; ++i)
            if (i < len) {
                const R r = f.apply(win, load_row(xs + (size_t)i * ldx));
                *reinterpret_cast<R*>(y + (base + i) * ldy + c) = r;
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
            *reinterpret_cast<R*>(state_out + ((size_t)part * (W - 1) + i) * C + c) = last[i];
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
    constexpr int kAhead = Raw<T>::ahead, kFew = 4;
    for (int tb = t0; tb < t1;) {
        if (tb - start >= W - 1 && tb + kAhead <= min(t1, end)) {
            R raw[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) raw[i] = load_row(xs + (size_t)(tb + i) * ldx);
#pragma unroll
            for (int i = 0; i < kAhead; ++i) *reinterpret_cast<R*>(ys + (size_t)(tb + i) * ldy) = f.apply(win, raw[i]);
            tb += kAhead;
            continue;
        }
        // a sequence starts or ends in these rows, or the strip does: a few at a time
        R raw[kFew];
#pragma unroll
        for (int i = 0; i < kFew; ++i) raw[i] = tb + i < t1 ? load_row(xs + (size_t)(tb + i) * ldx) : zero;
#pragma unroll 1
        for (int t = tb; t < min(tb + kFew, t1); ++t) {
            while (t >= end) {          // packed only: the next sequence (t < cu[n_seq], so there is one)
                ++n;
                start = end;
                end = __ldg(cu_seqlens + n + 1);
            }
            const R r = f.apply(win, raw[0]);
            if (t - start >= W - 1) *reinterpret_cast<R*>(ys + (size_t)t * ldy) = r;
#pragma unroll
            for (int i = 0; i + 1 < kFew; ++i) raw[i] = raw[i + 1];
        }
        tb += kFew;
    }
}

// The step: each sequence's state is read, shifted and written back whole.  One B200, 256 sequences x 36864
// channels, bf16, states in a pool: 29 us for 151 MB, 0.80 of the measured copy rate (the first and last
// microseconds, when loads or stores alone are under way, are a good part of so short a launch).
constexpr int kStepSeqs = 2;    // sequences in flight per thread of the step kernel

template <typename T, int W>
__global__ void __launch_bounds__(kThreads)
kda_short_conv_step_kernel(const T* __restrict__ x, const T* __restrict__ weight, const T* __restrict__ bias, T* state,
                           T* __restrict__ y, int B, int C, long long ldx, long long ldy, int act, int n_cb,
                           int seqs, const int* __restrict__ slots, int n_slots, int* status) {
    using R = typename Raw<T>::type;
    constexpr int V = kVec;
    const int cb = blockIdx.x % n_cb;
    const int b0 = (blockIdx.x / n_cb) * seqs;
    const int c = (cb * kThreads + (int)threadIdx.x) * V;
    if (c >= C) return;
    Filter<T, W> f;
    f.load(weight, bias, c, act != 0);
    const int b1 = min(b0 + seqs, B);
    for (int bb = b0; bb < b1; bb += kStepSeqs) {
        R u[kStepSeqs], raw[kStepSeqs][W - 1];
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
                    raw[k][i] = *reinterpret_cast<const R*>(state + ((size_t)at[k] * (W - 1) + i) * C + c);
            }
        }
#pragma unroll
        for (int k = 0; k < kStepSeqs; ++k) {
            if (at[k] < 0) continue;
            uint64_t win[W - 1][V / 2];
#pragma unroll
            for (int i = 0; i < W - 1; ++i) unpack(raw[k][i], win[i]);
            *reinterpret_cast<R*>(y + (size_t)(bb + k) * ldy + c) = f.apply(win, u[k]);
            T* st = state + (size_t)at[k] * (W - 1) * C + c;
#pragma unroll
            for (int i = 0; i + 1 < W - 1; ++i) *reinterpret_cast<R*>(st + (size_t)i * C) = raw[k][i + 1];
            *reinterpret_cast<R*>(st + (size_t)(W - 2) * C) = u[k];
        }
    }
}

template <typename T, int W>
cudaError_t launch_prompt(const ConvArgs& a, cudaStream_t s) {
    constexpr int V = kVec;
    const int n_cb = (a.C / V + kThreads - 1) / kThreads;
    // a short strip gives small problems enough blocks, a long one re-reads fewer rows above it
    const long long tokens = a.cu_seqlens ? a.T : (long long)a.n_seq * a.T;
    int strip = Raw<T>::ahead;
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
    constexpr int V = kVec;
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
