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

}  // namespace kda
