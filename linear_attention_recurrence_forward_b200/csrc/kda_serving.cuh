// Internal declarations of the operators beside the KDA recurrence: the short causal convolution, the
// selective scan and the state pools (arguments already validated by kda_serving_api.cu).
#pragma once

#include "kda_internal.cuh"

namespace kda {

struct ConvArgs {
    const void* x;
    const void* weight;
    const void* bias;          // may be null
    const void* state;         // [n_seq, W-1, C], may be null (zeros); the step kernels update it in place
    void* y;
    void* state_out;           // may be null, may be `state`
    const int* cu_seqlens;     // packed sequences (T = all tokens), or null: n_seq sequences of T tokens
    int n_seq, T, C, W;
    long long ldx, ldy;
    int act, dtype;
    const int* slots;          // step: state of sequence b at slots[b] of n_slots, or null
    int n_slots;
    int* status;
};

struct SsmArgs {
    const void* x;
    const void* dt;
    const float* A;
    const void* Bm;
    const void* Cm;
    const float* D;            // may be null
    const float* dt_bias;      // may be null
    const float* S0;           // may be null; the step kernel uses ST alone, in place
    void* y;
    float* ST;                 // may be null (prefill)
    const int* cu_seqlens;     // packed sequences (T = all tokens), or null: n_seq sequences of T tokens
    int n_seq, T, H, G, N, P;
    long long ldx, lddt, ldb, ldc;
    int dtype;
    const int* slots;
    int n_slots;
    int* status;
    unsigned long long timeout_ns;
    void* workspace;
    int skip_handoff;          // test hook: 1 = the tensor-core path's first hand-off is left out
};

cudaError_t launch_short_conv(const ConvArgs& a, cudaStream_t s);
cudaError_t launch_short_conv_step(const ConvArgs& a, cudaStream_t s);
cudaError_t launch_ssm_simt(const SsmArgs& a, cudaStream_t s);
bool ssm_tc_supports(const SsmArgs& a);
size_t ssm_tc_workspace(int n_seq, long long T_total, int H, int N, int P);
cudaError_t launch_ssm_tc(const SsmArgs& a, cudaStream_t s);
cudaError_t launch_ssm_decode(const SsmArgs& a, cudaStream_t s);
cudaError_t launch_pool_copy(const kda_pool* dst, const kda_pool* src, int n_pools, int n_dst, int n_src,
                             const int* src_idx, const int* dst_idx, int n, int* status, cudaStream_t s);
cudaError_t launch_pool_clear(const kda_pool* pools, int n_pools, int n_slots, const int* idx, int n, int* status,
                              cudaStream_t s);
cudaError_t launch_pool_compact(const kda_pool* pools, int n_pools, int n_slots, const int* slots,
                                const unsigned char* done, int* slots_out, int B, int* workspace, int* status,
                                cudaStream_t s);

// The status word of the current device (null on failure) and the limit of device-side waits.
int* current_status_word();
unsigned long long wait_timeout_ns();
int wait_fault_mode();     // kda_debug_set_wait_fault

// softplus(v) = log(1 + e^v) without overflow or cancellation
__device__ __forceinline__ float softplus(float v) { return fmaxf(v, 0.f) + log1pf(expf(-fabsf(v))); }

// A token's decay e^v, v = step * A.  A state that remembers thousands of tokens is multiplied by thousands of decays just
// below 1, so that what expf is off by there, on one side, adds up (1.3e-8 a token: 1.3e-5 of a state that remembers a
// thousand).  Near 0 it is the power series, 1 + v + .. + v^6 / 720 (what is left out is below 2^-26), whose one rounding
// that counts is the last, to nearest: 1.0e-6 of that state.  Further from 0 a state forgets within a few tokens.
__device__ __forceinline__ float token_decay(float v) {
    float near = fmaf(v, 1.f / 720.f, 1.f / 120.f);
    near = fmaf(v, near, 1.f / 24.f);
    near = fmaf(v, near, 1.f / 6.f);
    near = fmaf(v, near, 0.5f);
    near = fmaf(v, near, 1.f);
    near = fmaf(v, near, 1.f);
    return fabsf(v) < 0.25f ? near : expf(v);
}

}  // namespace kda
