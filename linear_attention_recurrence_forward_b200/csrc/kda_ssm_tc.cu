// The selective scan on the tensor core: bf16 prompts, N and P in {64, 128}, fp32 states.
//
// Chunks of 128 tokens.  With L_r the running sum of s_u A over a chunk (in units of log 2), per head
//
//     y_r = 2^{L_r} S^T C_r + sum_{j<=r} (C_r . B_j) 2^{L_r - L_j} s_j x_j + D x_r
//     S  <- 2^{L_end} S + sum_j B_j (s_j 2^{L_end - L_j} x_j)^T
//
// which is five matrix products a chunk: G = C B^T, Y = C S, Y += Q X with Q the decayed lower triangle
// of G (and D on its diagonal), and the state update in two parts.
//
// A CTA carries one tile of 128 value columns through its tokens: one head of P = 128, or two heads of
// P = 64 that share their B and C (a head without a partner is carried twice and stored once).  Every
// exponent is a difference of later and earlier sums, never above zero for A <= 0, so nothing overflows
// however strong the decay; differences are formed within 32-token blocks and from block totals, which
// keeps their relative precision when a chunk's sum is large.  Off the diagonal blocks of Q the decay
// factors into a row and a column part through the block's last token, so only the four 32 x 32
// diagonal blocks take an exponential per element.
//
// Precision.  Outputs are bf16: S is read as a bf16 operand and Q is rounded to bf16, one rounding of
// each term of y.  The state itself is fp32: B and x are exact bf16 operands, and a weight w = w1 + w2
// (two bf16 values, off by at most 2^-16 w) makes the weighted x the sum of two bf16 values,
// hi = x w1 rounded and lo = x w2 + (x w1 - hi) rounded (x w1 - hi is exact), so a term of the state is
// off by at most 3 * 2^-16 of itself.  One bf16 value would leave 2^-8, a third product costs a fifth
// more tensor time.
//
// What bounds it: HBM moves 64 KB of x and y per chunk of a 128-column tile (2.8K cycles at the
// measured copy rate), the tensor core needs 2.5K cycles, and its operands with the tiles' own traffic
// about 3.5K cycles of shared memory, so operands are kept out of shared memory where a product allows:
// Q and the weighted x are tensor-memory operands, and the state is held transposed (lanes = value
// columns) for that.  The weighted x is transposed on its way by ldmatrix and the 16x128b stores, whose
// fragments have one layout.
//
// Warps (20): 0-3 state, 4-7 decays and weighted x, 8-15 Q and outputs, 16 products, 17 loads of B and x,
// 18 loads of C, 19 stores of y.
// Tensor memory (512 columns): S^T, Y, G (then Q in its place), weighted x hi and lo.
// Order of the products: Y = C S | S += hi | Y += Q X | S += lo | next G.  The scaling of Y runs under
// the hi part, Y's store under the lo part, the state's conversion under the next G.
//
// Long prompts with few heads: the tokens are cut into segments.  A first launch forms the state of every
// segment but the last (B and x only; the first one from S0, the others from zero), going through the
// chunks backwards, so that the weights hold the decay to the segment's end and the products just add up;
// the second starts each segment from the segments before it, S <- 2^{total} S + local, folded in as it
// loads its start state.
//
// Every wait is bounded in time; a wait that runs out sets the status word and an abort flag that ends
// the other warps' waits, the products and loads in flight are drained, and the CTA returns.
#include <cudaTypedefs.h>
#include <mutex>

#include "kda_serving.cuh"
#include "sm100_ptx.cuh"

namespace kda {
namespace {

using namespace sm100;

constexpr int kTok = 128;                    // tokens per chunk
constexpr int kCols = 128;                   // value columns per CTA
constexpr int kStages = 2;                   // of B and x; the state-only kernel has three (no C, no S)
constexpr int kThreads = 640;
constexpr int kStateWarps = 4, kDecayWarps = 4, kScoreWarps = 8;
constexpr int kFirstDecay = kStateWarps, kFirstScore = kFirstDecay + kDecayWarps;
constexpr int kIssueWarp = kFirstScore + kScoreWarps, kLoadWarp = kIssueWarp + 1,
              kLoadCWarp = kLoadWarp + 1, kStoreWarp = kLoadCWarp + 1;
constexpr uint32_t ATOM = 16384;             // [128 rows][64 columns] bf16, 128-byte swizzle
constexpr uint32_t kTile = 2 * ATOM;

// shared memory: per stage B, X; one C (free again after a chunk's second product); S as bf16 (rows = value
// columns, K = N)
constexpr uint32_t OFF_B = 0, OFF_X = kTile, kStageBytes = 2 * kTile;
constexpr uint32_t OFF_C = kStages * kStageBytes, OFF_S = OFF_C + kTile;
constexpr uint32_t SMEM_DYN = OFF_S + kTile + 1024;

// tensor memory columns (the state-only kernel's three groups have their weighted x at TM_HI, TM_G and TM_Y)
constexpr uint32_t TM_S = 0, TM_Y = 128, TM_G = 256, TM_HI = 384, TM_LO = 448, TM_COLS = 512;

struct __align__(16) Scalars {               // of one chunk, per head of the tile
    float neg[2][kTok];                      // -(running sum within the token's 32-token block, inclusive)
    float col[2][kTok];                      // s_j 2^{block end - L_j}
    float step[2][kTok];                     // s_j
    uint16_t w1[2][kTok], w2[2][kTok];       // s_j 2^{chunk end - L_j} as a sum of two bf16 values
    float total[2][4];                       // sums of the four blocks
};

struct Params {
    const __nv_bfloat16* dt;
    const float* A;
    const float* D;
    const float* dt_bias;
    const float* S0;
    __nv_bfloat16* y;
    float* ST;
    const int* cu_seqlens;
    float* seg_state;                        // [unit][H][N][P] local states of the segments
    float* seg_decay;                        // [unit][H] their total decays (log 2)
    long long lddt;
    int n_seq, T, H, G;
    int tiles;                               // column tiles per token range
    int seg_chunks;                          // chunks per segment (0: whole sequences)
    int segs;                                // segments per sequence ([B, T] layout)
    int* status;
    unsigned long long timeout_ns;
    int skip_handoff;
};

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {      // round to nearest even
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// D[tmem] (+)= A[tmem] * B[smem], issued by one thread
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// A: 128 tokens of K in 64 packed columns; B: MN-major tile whose K axis is the tokens.  The K steps are unrolled (a
// rolled loop issues a product every 160 cycles, the tensor core takes one every 64).
__device__ __forceinline__ void issue_ts(uint32_t d, uint32_t a, uint32_t b_base, uint32_t idesc, bool accumulate) {
    const uint64_t bd = smem_desc_sw128(b_base, ATOM, 1024u);
#pragma unroll
    for (int kk = 0; kk < kTok / 16; ++kk)
        mma_bf16_ts(d, a + 8 * kk, bd + ((uint32_t)kk * 2048u >> 4), idesc, (kk > 0 || accumulate) ? 1u : 0u);
}
// both operands K-major, K = N
template <int N>
__device__ __forceinline__ void issue_ss(uint32_t d, uint32_t a_base, uint32_t b_base, uint32_t idesc) {
    issue_mma<N / 16, false, ATOM, false, ATOM>(d, a_base, b_base, idesc, false);
}
__device__ __forceinline__ uint64_t pair2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// two products a b as bf16x2
__device__ __forceinline__ uint32_t mul2_bf16x2(uint64_t a, uint64_t b) {
    const uint64_t r = mul2(a, b);
    float lo, hi;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(r));
    return bf16x2(lo, hi);
}
// v[0..n) *= e
template <int NV>
__device__ __forceinline__ void scale_by(float* v, float e) {
    const uint64_t e2 = pair2(e, e);
#pragma unroll
    for (int i = 0; i < NV; i += 2) {
        const uint64_t r = mul2(pair2(v[i], v[i + 1]), e2);
        asm("mov.b64 {%0, %1}, %2;" : "=f"(v[i]), "=f"(v[i + 1]) : "l"(r));
    }
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
// four 8 x 8 bf16 matrices, transposed: thread i gets rows 2(i%4), 2(i%4)+1 of column i/4 of each
__device__ __forceinline__ void ldmatrix4t(uint32_t addr, uint32_t (&m)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(m[0]), "=r"(m[1]), "=r"(m[2]), "=r"(m[3]) : "r"(addr) : "memory");
}
// 16 lanes x 16 columns: register 2k of thread i goes to lane i/4, column 4k + i%4, register 2k+1 to lane 8 + i/4
__device__ __forceinline__ void tmem_st_16x128(uint32_t taddr, const uint32_t* u) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
                 "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* u) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
                 "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
                 : "memory");
}

// TMEM -> registers, 64 columns, complete on return.  Load and wait are one statement: between two, the
// compiler may move or spill registers that the load has not written yet.
__device__ __forceinline__ void tmem_read64(uint32_t taddr, float* r) {
    uint32_t* u = reinterpret_cast<uint32_t*>(r);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=&r"(u[0]), "=&r"(u[1]), "=&r"(u[2]), "=&r"(u[3]), "=&r"(u[4]), "=&r"(u[5]), "=&r"(u[6]), "=&r"(u[7]),
          "=&r"(u[8]), "=&r"(u[9]), "=&r"(u[10]), "=&r"(u[11]), "=&r"(u[12]), "=&r"(u[13]), "=&r"(u[14]), "=&r"(u[15]),
          "=&r"(u[16]), "=&r"(u[17]), "=&r"(u[18]), "=&r"(u[19]), "=&r"(u[20]), "=&r"(u[21]), "=&r"(u[22]), "=&r"(u[23]),
          "=&r"(u[24]), "=&r"(u[25]), "=&r"(u[26]), "=&r"(u[27]), "=&r"(u[28]), "=&r"(u[29]), "=&r"(u[30]), "=&r"(u[31]),
          "=&r"(u[32]), "=&r"(u[33]), "=&r"(u[34]), "=&r"(u[35]), "=&r"(u[36]), "=&r"(u[37]), "=&r"(u[38]), "=&r"(u[39]),
          "=&r"(u[40]), "=&r"(u[41]), "=&r"(u[42]), "=&r"(u[43]), "=&r"(u[44]), "=&r"(u[45]), "=&r"(u[46]), "=&r"(u[47]),
          "=&r"(u[48]), "=&r"(u[49]), "=&r"(u[50]), "=&r"(u[51]), "=&r"(u[52]), "=&r"(u[53]), "=&r"(u[54]), "=&r"(u[55]),
          "=&r"(u[56]), "=&r"(u[57]), "=&r"(u[58]), "=&r"(u[59]), "=&r"(u[60]), "=&r"(u[61]), "=&r"(u[62]), "=&r"(u[63])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_read32(uint32_t taddr, float* r) {
    uint32_t* u = reinterpret_cast<uint32_t*>(r);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=&r"(u[0]), "=&r"(u[1]), "=&r"(u[2]), "=&r"(u[3]), "=&r"(u[4]), "=&r"(u[5]), "=&r"(u[6]), "=&r"(u[7]),
          "=&r"(u[8]), "=&r"(u[9]), "=&r"(u[10]), "=&r"(u[11]), "=&r"(u[12]), "=&r"(u[13]), "=&r"(u[14]), "=&r"(u[15]),
          "=&r"(u[16]), "=&r"(u[17]), "=&r"(u[18]), "=&r"(u[19]), "=&r"(u[20]), "=&r"(u[21]), "=&r"(u[22]), "=&r"(u[23]),
          "=&r"(u[24]), "=&r"(u[25]), "=&r"(u[26]), "=&r"(u[27]), "=&r"(u[28]), "=&r"(u[29]), "=&r"(u[30]), "=&r"(u[31])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_write32(uint32_t taddr, const float* r) {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(r);
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]),
          "r"(u[8]), "r"(u[9]), "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15]),
          "r"(u[16]), "r"(u[17]), "r"(u[18]), "r"(u[19]), "r"(u[20]), "r"(u[21]), "r"(u[22]), "r"(u[23]),
          "r"(u[24]), "r"(u[25]), "r"(u[26]), "r"(u[27]), "r"(u[28]), "r"(u[29]), "r"(u[30]), "r"(u[31])
        : "memory");
}
// Three runs of 16 columns, 32 apart, and a fourth at `other`.
__device__ __forceinline__ void tmem_read3x16(uint32_t taddr, float* r, uint32_t other, float* r2) {
    uint32_t* u = reinterpret_cast<uint32_t*>(r);
    uint32_t* w = reinterpret_cast<uint32_t*>(r2);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%64];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%65];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47}, [%66];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%67];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=&r"(u[0]), "=&r"(u[1]), "=&r"(u[2]), "=&r"(u[3]), "=&r"(u[4]), "=&r"(u[5]), "=&r"(u[6]), "=&r"(u[7]),
          "=&r"(u[8]), "=&r"(u[9]), "=&r"(u[10]), "=&r"(u[11]), "=&r"(u[12]), "=&r"(u[13]), "=&r"(u[14]), "=&r"(u[15]),
          "=&r"(u[16]), "=&r"(u[17]), "=&r"(u[18]), "=&r"(u[19]), "=&r"(u[20]), "=&r"(u[21]), "=&r"(u[22]), "=&r"(u[23]),
          "=&r"(u[24]), "=&r"(u[25]), "=&r"(u[26]), "=&r"(u[27]), "=&r"(u[28]), "=&r"(u[29]), "=&r"(u[30]), "=&r"(u[31]),
          "=&r"(u[32]), "=&r"(u[33]), "=&r"(u[34]), "=&r"(u[35]), "=&r"(u[36]), "=&r"(u[37]), "=&r"(u[38]), "=&r"(u[39]),
          "=&r"(u[40]), "=&r"(u[41]), "=&r"(u[42]), "=&r"(u[43]), "=&r"(u[44]), "=&r"(u[45]), "=&r"(u[46]), "=&r"(u[47]),
          "=&r"(w[0]), "=&r"(w[1]), "=&r"(w[2]), "=&r"(w[3]), "=&r"(w[4]), "=&r"(w[5]), "=&r"(w[6]), "=&r"(w[7]),
          "=&r"(w[8]), "=&r"(w[9]), "=&r"(w[10]), "=&r"(w[11]), "=&r"(w[12]), "=&r"(w[13]), "=&r"(w[14]), "=&r"(w[15])
        : "r"(taddr), "r"(taddr + 32), "r"(taddr + 64), "r"(other)
        : "memory");
}

// Bounded waits that also end when another warp of the CTA has given up.
struct Waiter {
    volatile int* abort_flag;
    int* status;
    unsigned long long timeout_ns;

    __device__ __noinline__ bool slow(uint32_t a, uint32_t parity) const {
        const uint64_t t0 = global_timer_ns();
        for (;;) {
#pragma unroll 1
            for (int i = 0; i < 32; ++i)
                if (mbar_try_wait(a, parity)) return true;
            if (*abort_flag) return false;
            if (global_timer_ns() - t0 > timeout_ns) {
                *abort_flag = 1;
                report_status(status, KDA_ERR_TIMEOUT);
                return false;
            }
        }
    }
    // one thread
    __device__ __forceinline__ bool one(uint64_t* bar, uint32_t parity) const {
        const uint32_t a = smem_u32(bar);
        return mbar_try_wait(a, parity) || slow(a, parity);
    }
    // a whole warp: the same answer in every lane
    __device__ __forceinline__ bool warp(uint64_t* bar, uint32_t parity) const {
        return __all_sync(0xffffffffu, one(bar, parity)) != 0;
    }
};

__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
}

template <int N, int P, bool STATE_ONLY>
__global__ void __launch_bounds__(kThreads, 1)
kda_ssm_tc_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_b,
                  const __grid_constant__ CUtensorMap tm_c, const __grid_constant__ CUtensorMap tm_y, const Params p) {
    constexpr int NH = P == 64 ? 2 : 1;      // heads per tile
    constexpr int ST = STATE_ONLY ? 3 : kStages;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_base = smem_u32(smem_raw);
    uint8_t* sm = smem_raw + (((raw_base + 1023u) & ~1023u) - raw_base);
    const uint32_t sb = smem_u32(sm);
    __shared__ Scalars scal[STATE_ONLY ? 3 : 2];
    __shared__ uint64_t full[ST], empty[ST], full_c, bar_scal[2], bar_g, bar_cs, bar_upd[3], bar_px, bar_state, bar_w, bar_wst[3],
        bar_behind[3], bar_init, bar_q,
        bar_yfree, bar_staged, yread[kStages], bar_drain;
    __shared__ uint32_t tmem_base_s;
    __shared__ volatile int abort_s;
    __shared__ int seq_s, seg_s;
    __shared__ float seg_total_s[2], behind_s[3][2];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int H = p.H;

    // ---- which tokens and which heads
    const int unit = blockIdx.x / p.tiles, tile = blockIdx.x % p.tiles;
    const int rep = H / p.G;
    const int per_group = (rep + NH - 1) / NH;
    const int g = tile / per_group, h0 = g * rep + (tile % per_group) * NH;
    const int h1 = NH == 2 && h0 + 1 < (g + 1) * rep ? h0 + 1 : h0;      // no partner: the same head again
    int seq, seg, len_seq;
    size_t start;                            // first token of the sequence on the token axis of x, dt and y
    if (p.cu_seqlens) {
        const bool valid = packed_offsets_valid(p.cu_seqlens, p.n_seq, p.T);
        if (!valid && tid == 0) report_status(p.status, KDA_ERR_INVALID_ARG);
        if (p.seg_chunks > 0) {
            // units in order: each sequence's segments (one for an empty sequence)
            if (tid == 0) seq_s = -1;
            __syncthreads();
            if (warp == 0) {
                int before = 0;
                for (int base = 0; base < p.n_seq; base += 32) {
                    const int i = base + lane;
                    int n = 0;
                    if (i < p.n_seq) {
                        const int len = valid ? p.cu_seqlens[i + 1] - p.cu_seqlens[i] : 0;
                        n = max(1, (len + p.seg_chunks * kTok - 1) / (p.seg_chunks * kTok));
                    }
                    int incl = n;
#pragma unroll
                    for (int off = 1; off < 32; off <<= 1) {
                        const int t = __shfl_up_sync(0xffffffffu, incl, off);
                        if (lane >= off) incl += t;
                    }
                    if (unit >= before + incl - n && unit < before + incl) {
                        seq_s = i;
                        seg_s = unit - (before + incl - n);
                    }
                    before += __shfl_sync(0xffffffffu, incl, 31);
                    if (unit < before) break;
                }
            }
            __syncthreads();
            seq = seq_s;
            seg = seg_s;
            if (seq < 0) return;             // the grid holds the most units that T tokens can make
        } else {
            seq = unit;
            seg = 0;
        }
        start = valid ? (size_t)p.cu_seqlens[seq] : 0;
        len_seq = valid ? p.cu_seqlens[seq + 1] - p.cu_seqlens[seq] : 0;
    } else {
        seq = unit / p.segs;
        seg = unit % p.segs;
        start = (size_t)seq * p.T;
        len_seq = p.T;
    }
    const int seg_tokens = p.seg_chunks > 0 ? p.seg_chunks * kTok : 0x7fffffff;
    const int tok0 = seg * (p.seg_chunks * kTok);                        // first token within the sequence
    const int len = min(len_seq - tok0, seg_tokens);
    const bool last_seg = tok0 + len >= len_seq;
    const int n_seg = p.seg_chunks > 0 ? max(1, (len_seq + seg_tokens - 1) / seg_tokens) : 1;
    const int unit0 = unit - seg;            // the sequence's first segment
    if (STATE_ONLY && last_seg) return;
    const int chunks = (len + kTok - 1) / kTok;
    const int row_seq = p.cu_seqlens ? 0 : seq;                          // batch coordinate of the tensor maps
    const int row0 = (p.cu_seqlens ? (int)start : 0) + tok0;             // token coordinate of the first chunk

    if (tid == 0) {
        for (int i = 0; i < ST; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], 1); }
        for (int i = 0; i < kStages; ++i) mbar_init(&yread[i], 1);
        for (int i = 0; i < 2; ++i) mbar_init(&bar_scal[i], kDecayWarps);
        mbar_init(&full_c, 1);
        mbar_init(&bar_g, 1);
        mbar_init(&bar_init, N / 8);
        mbar_init(&bar_cs, 1);
        for (int i = 0; i < 3; ++i) mbar_init(&bar_upd[i], 1);
        mbar_init(&bar_px, 1);
        static_assert(kStateWarps == kDecayWarps, "bar_state counts either");
        mbar_init(&bar_state, kStateWarps);
        mbar_init(&bar_yfree, kScoreWarps);
        mbar_init(&bar_staged, kScoreWarps);
        mbar_init(&bar_w, kDecayWarps);
        for (int i = 0; i < 3; ++i) { mbar_init(&bar_wst[i], kDecayWarps); mbar_init(&bar_behind[i], kDecayWarps); }
        mbar_init(&bar_q, kScoreWarps);
        mbar_init(&bar_drain, 1);
        fence_mbar_init();
        abort_s = 0;
        prefetch_tensormap(&tm_x); prefetch_tensormap(&tm_b); prefetch_tensormap(&tm_c);
        prefetch_tensormap(&tm_y);
    }
    if (warp == 0) {
        tmem_alloc(&tmem_base_s, TM_COLS);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tbase = tmem_base_s;
    const Waiter wait{&abort_s, p.status, p.timeout_ns};
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;            // this warp's tensor-memory lanes
    const int quarter = warp & 3;

    // ---- states: a lane of a warp is one value column, in the warp's quarter of the tensor-memory lanes
    const int col = 32 * quarter + lane;                                // value column of this lane
    const int half = NH == 2 ? col >> 6 : 0;
    const int head = half ? h1 : h0, pc = NH == 2 ? col & 63 : col;
    const bool dup = NH == 2 && half == 1 && h1 == h0;               // carried, not stored
    const size_t s_off = (((size_t)seq * H + head) * N) * P + pc;    // S[seq][head][0][pc]
    auto seg_state = [&](int u) { return p.seg_state + ((size_t)u * H + head) * N * P + pc; };
    auto store_state = [&](float* to, int n0, const float* v) {
        if (!dup) {
#pragma unroll
            for (int i = 0; i < 32; ++i) to[(size_t)(n0 + i) * P] = v[i];
        }
    };
    // The start state of 32 rows n.  Sequences of several segments: the first launch starts segment 0 from
    // S0, and leaves a copy of S0 in the last segment's place, which no local state takes; the second launch
    // reads S0 nowhere else, so that S_T may be S0.
    auto load_start = [&](int n0, float* v) {
        const float* from = STATE_ONLY || n_seg == 1 ? (p.S0 && seg == 0 ? p.S0 + s_off : nullptr)
                                                     : seg_state(seg == 0 ? unit0 + n_seg - 1 : unit0);
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = from ? from[(size_t)(n0 + i) * P] : 0.f;
        if constexpr (STATE_ONLY) {
            if (seg == 0) store_state(seg_state(unit0 + n_seg - 1), n0, v);
        } else {
#pragma unroll 2
            for (int k = 1; k < seg; ++k) {
                const float d = ex2(p.seg_decay[(size_t)(unit0 + k) * H + head]);
                const float* l = seg_state(unit0 + k);
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = fmaf(d, v[i], l[(size_t)(n0 + i) * P]);
            }
        }
    };
    // 32 rows to each group of four warps, in parallel (each start state is as many dependent reads as segments)
    if (!STATE_ONLY && warp < kIssueWarp && 8 * (warp & ~3) < N) {
        const int n0 = 8 * (warp & ~3);
        float v[32];
        load_start(n0, v);
        if (chunks > 0) {
            tmem_write32(tbase + TM_S + lanes + n0, v);
            tmem_wait_st();
            tc_fence_before_sync();
            warp_arrive(&bar_init, lane);
        } else if (p.ST) {
            store_state(p.ST + s_off, n0, v);            // an empty sequence
        }
    }
    if (warp == kLoadWarp) {
        // ------------------------------------------------------------ loads of B and x
        if (lane == 0) {
            int issued = 0;
            for (int c = 0; c < chunks; ++c) {
                const int st = c % ST, t = row0 + (STATE_ONLY ? chunks - 1 - c : c) * kTok;
                uint8_t* s = sm + st * kStageBytes;
                // the stage is free after the last product of its last turn and once its y has been read out
                if (c >= ST && (!wait.one(&empty[st], (uint32_t)(c / ST - 1) & 1) ||
                                (!STATE_ONLY && !wait.one(&yread[st % kStages], (uint32_t)(c / ST - 1) & 1))))
                    break;
                mbar_arrive_expect_tx(&full[st], ATOM * (2 + N / 64));
                for (int i = 0; i < N / 64; ++i) tma_load_4d(s + OFF_B + i * ATOM, &tm_b, &full[st], 64 * i, g, t, row_seq);
                for (int i = 0; i < 2; ++i)
                    tma_load_4d(s + OFF_X + i * ATOM, &tm_x, &full[st], NH == 2 ? 0 : 64 * i, NH == 2 && i ? h1 : h0, t, row_seq);
                ++issued;
                // x of the stage's next turn, which no other CTA reads, into L2 (3% at P = 128)
                if (c + ST < chunks)
                    for (int i = 0; i < 2; ++i)
                        tma_prefetch_4d(&tm_x, NH == 2 ? 0 : 64 * i, NH == 2 && i ? h1 : h0,
                                        STATE_ONLY ? t - ST * kTok : t + ST * kTok, row_seq);
            }
            // nothing may be in flight when the CTA exits
            for (int c = max(0, issued - ST); c < issued; ++c)
                if (!mbar_wait(&full[c % ST], (uint32_t)(c / ST) & 1, p.timeout_ns))
                    report_status(p.status, KDA_ERR_TIMEOUT);
        }
    } else if (warp == kLoadCWarp) {
        // ------------------------------------------------------------ loads of C, each as soon as the last is used up
        if (lane == 0 && !STATE_ONLY) {
            int issued = 0;
            for (int c = 0; c < chunks; ++c) {
                if (c > 0 && !wait.one(&bar_cs, (uint32_t)(c - 1) & 1)) break;
                mbar_arrive_expect_tx(&full_c, kTile / 128 * N);
                for (int i = 0; i < N / 64; ++i)
                    tma_load_4d(sm + OFF_C + i * ATOM, &tm_c, &full_c, 64 * i, g, row0 + c * kTok, row_seq);
                ++issued;
            }
            if (issued > 0 && !mbar_wait(&full_c, (uint32_t)(issued - 1) & 1, p.timeout_ns))
                report_status(p.status, KDA_ERR_TIMEOUT);
        }
    } else if (warp == kStoreWarp) {
        // ------------------------------------------------------------ stores of y from the x tiles
        if (lane == 0 && !STATE_ONLY) {
            for (int c = 0; c < chunks; ++c) {
                const int st = c % kStages;
                if (!wait.one(&bar_staged, c & 1)) break;
                if (!p.cu_seqlens || len - c * kTok >= kTok) {           // whole tiles, clipped at the end of the tensor
                    for (int i = 0; i < 2; ++i)
                        if (!(NH == 2 && i == 1 && h1 == h0))
                            tma_store_4d(&tm_y, sm + st * kStageBytes + OFF_X + i * ATOM, NH == 2 ? 0 : 64 * i,
                                         NH == 2 && i ? h1 : h0, row0 + c * kTok, row_seq);
                    bulk_commit_group();
                    bulk_wait_read_all();
                }
                mbar_arrive(&yread[st]);
            }
            bulk_wait_all();
        }
    } else if (warp == kIssueWarp) {
        // ------------------------------------------------------------ products
        if (lane == 0) {
            const uint32_t id_g = idesc_bf16_f32(128, 128, false, false);
            const uint32_t id_cs = idesc_bf16_f32(128, kCols, false, false);
            const uint32_t id_px = idesc_bf16_f32(128, P, false, true);
            const uint32_t id_up = idesc_bf16_f32(128, N, false, true);
            auto issue_g = [&](int c) {
                if (!wait.one(&full[c % kStages], (uint32_t)(c / kStages) & 1) || !wait.one(&full_c, c & 1)) return false;
                tc_fence_after_sync();
                issue_ss<N>(tbase + TM_G, sb + OFF_C, sb + (c % kStages) * kStageBytes + OFF_B, id_g);
                mma_commit(&bar_g);
                return true;
            };
            bool ok = STATE_ONLY || chunks == 0 || issue_g(0);
            if constexpr (STATE_ONLY) {
                for (int c = 0; c < chunks; ++c) {
                    const uint32_t s = sb + (c % ST) * kStageBytes, w = tbase + TM_HI - 128 * (c % ST);
                    if (!wait.one(&bar_wst[c % ST], (uint32_t)(c / ST) & 1)) break;
                    tc_fence_after_sync();
                    issue_ts(tbase + TM_S, w, s + OFF_B, id_up, c > 0);
                    issue_ts(tbase + TM_S, w + 64, s + OFF_B, id_up, true);
                    mma_commit(&bar_upd[c % ST]);
                    mma_commit(&empty[c % ST]);
                }
                ok = false;
            }
            for (int c = 0; c < chunks && ok; ++c) {
                const uint32_t s = sb + (c % kStages) * kStageBytes, par = c & 1;
                ok = wait.one(&bar_state, par);          // S as bf16 and decayed
                if (ok && !STATE_ONLY && c > 0) ok = wait.one(&bar_yfree, par ^ 1);
                if (!ok) break;
                tc_fence_after_sync();
                if (!STATE_ONLY) {
                    issue_ss<N>(tbase + TM_Y, sb + OFF_C, sb + OFF_S, id_cs);
                    mma_commit(&bar_cs);
                }
                ok = wait.one(&bar_w, par);              // weighted x
                if (!ok) break;
                tc_fence_after_sync();
                issue_ts(tbase + TM_S, tbase + TM_HI, s + OFF_B, id_up, true);
                if (!STATE_ONLY) {
                    ok = wait.one(&bar_q, par);          // Q, and Y scaled
                    if (!ok) break;
                    tc_fence_after_sync();
#pragma unroll
                    for (int i = 0; i < NH; ++i)
                        issue_ts(tbase + TM_Y + i * P, tbase + TM_G + 64 * i, s + OFF_X + (NH == 2 ? i * ATOM : 0), id_px, true);
                    mma_commit(&bar_px);
                }
                issue_ts(tbase + TM_S, tbase + TM_LO, s + OFF_B, id_up, true);
                mma_commit(&bar_upd[0]);
                mma_commit(&empty[c % kStages]);
                if (!STATE_ONLY && c + 1 < chunks) ok = issue_g(c + 1);
            }
            mma_commit(&bar_drain);
            if (!mbar_wait(&bar_drain, 0, p.timeout_ns)) report_status(p.status, KDA_ERR_TIMEOUT);
        }
    } else if (warp < kStateWarps) {
        // ------------------------------------------------------------ state
        bool ok = true;
        for (int c = 0; !STATE_ONLY && c < chunks && ok; ++c) {
            const uint32_t par = c & 1;
            const Scalars& sc = scal[c & 1];
            ok = wait.warp(&bar_scal[c & 1], (c >> 1) & 1) &&
                 (c == 0 ? wait.warp(&bar_init, 0) : wait.warp(&bar_upd[0], par ^ 1));
            if (!ok) break;
            tc_fence_after_sync();
            const float decay = ex2((sc.total[half][0] + sc.total[half][1]) + (sc.total[half][2] + sc.total[half][3]));
            // S: its bf16 copy for this chunk's read-out, then decayed to the chunk's end for the update
#pragma unroll 1
            for (int n0 = 0; n0 < N; n0 += 64) {
                float v[64];
                const uint32_t ta = tbase + TM_S + lanes + n0;
                tmem_read64(ta, v);
#pragma unroll
                for (int i = 0; i < 64; i += 8)
                    *reinterpret_cast<uint4*>(sm + OFF_S + sw128_offset(col, n0 + i, ATOM)) =
                        make_uint4(bf16x2(v[i], v[i + 1]), bf16x2(v[i + 2], v[i + 3]), bf16x2(v[i + 4], v[i + 5]),
                                   bf16x2(v[i + 6], v[i + 7]));
                scale_by<64>(v, decay);
                tmem_write32(ta, v);
                tmem_write32(ta + 32, v + 32);
            }
            tmem_wait_st();
            fence_proxy_async_smem();
            tc_fence_before_sync();
            if (!(p.skip_handoff && c == 0)) warp_arrive(&bar_state, lane);
        }
        if constexpr (STATE_ONLY) {
            // the segment's state: the sum of its chunks, and for the first segment what is left of S0
            ok = wait.warp(&bar_state, 0) && wait.warp(&bar_upd[(chunks - 1) % ST], (uint32_t)((chunks - 1) / ST) & 1);
            tc_fence_after_sync();
            const float decay = ex2(seg_total_s[half]);
#pragma unroll 1
            for (int n0 = 0; n0 < N && ok; n0 += 32) {
                float v[32], start[32];
                tmem_read32(tbase + TM_S + lanes + n0, v);
                load_start(n0, start);
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = fmaf(decay, start[i], v[i]);
                store_state(seg_state(unit), n0, v);
            }
        } else if (ok && chunks > 0 && last_seg && p.ST && wait.warp(&bar_upd[0], (chunks - 1) & 1)) {
            // the state after the last token
            tc_fence_after_sync();
#pragma unroll 1
            for (int n0 = 0; n0 < N; n0 += 32) {
                float v[32];
                tmem_read32(tbase + TM_S + lanes + n0, v);
                store_state(p.ST + s_off, n0, v);
            }
        }
    } else if (warp < (STATE_ONLY ? kIssueWarp : kFirstScore)) {
        // ------------------------------------------------------------ decays and weighted x
        // one group of four warps; in the state-only kernel three, each every third chunk
        const int dw = (warp - kFirstDecay) & 3, group = (warp - kFirstDecay) >> 2;
        constexpr int kGroups = STATE_ONLY ? ST : 1;
        const int j = 32 * dw + lane;                                    // a token here
        float rate[NH], bias[NH], raw[NH], total_all[NH];
#pragma unroll
        for (int i = 0; i < NH; ++i) {
            const int head = i ? h1 : h0;
            rate[i] = p.A[head] * 1.4426950408889634f;                   // decays in powers of two
            bias[i] = p.dt_bias ? p.dt_bias[head] : 0.f;
            total_all[i] = 0.f;
        }
        // the state-only kernel goes through its chunks from the last to the first: the decay behind a chunk is then
        // known when its weights are formed, and the products only add up, with no pass over the state in between
        auto chunk_at = [&](int c) { return STATE_ONLY ? chunks - 1 - c : c; };
        auto load_dt = [&](int c) {
            const int t = chunk_at(c) * kTok + j;
#pragma unroll
            for (int i = 0; i < NH; ++i)
                raw[i] = t < len ? load_elem(p.dt, (start + tok0 + t) * p.lddt + (i ? h1 : h0)) : 0.f;
        };
        load_dt(group);
        bool ok = true;
        for (int c = group; c < chunks; c += kGroups) {
            Scalars& sc = scal[STATE_ONLY ? group : c & 1];
            const int n_valid = min(kTok, len - chunk_at(c) * kTok);
            float sfx[NH], stp[NH];
#pragma unroll
            for (int i = 0; i < NH; ++i) stp[i] = raw[i] + bias[i];
#pragma unroll 1
            for (int i = 0; i < NH; ++i) {                               // the heads change places: one copy of the code
                const float st = j < n_valid ? softplus(stp[0]) : 0.f;
                const float t0 = stp[NH - 1];
                stp[NH - 1] = st;
                if (NH == 2) stp[0] = t0;
            }
#pragma unroll
            for (int i = 0; i < NH; ++i) {
                const float la = stp[i] * rate[i];
                float incl = la, rev = la;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const float a = __shfl_up_sync(0xffffffffu, incl, off), b = __shfl_down_sync(0xffffffffu, rev, off);
                    if (lane >= off) incl += a;
                    if (lane + off < 32) rev += b;
                }
                const float after = __shfl_down_sync(0xffffffffu, rev, 1);
                sfx[i] = lane == 31 ? 0.f : after;                       // tokens after this one in its block
                sc.neg[i][j] = -incl;
                sc.step[i][j] = stp[i];
                sc.col[i][j] = stp[i] * ex2(sfx[i]);
                if (lane == 31) sc.total[i][dw] = incl;
            }
            if (c + kGroups < chunks) load_dt(c + kGroups);
            named_bar_sync(1 + 2 * group, 32 * kDecayWarps);
            if constexpr (STATE_ONLY) {
                // the decay behind the chunk, handed on from group to group
                if (c > 0) (void)wait.warp(&bar_behind[group], (uint32_t)((c - 1) / ST) & 1);
#pragma unroll
                for (int i = 0; i < NH; ++i) total_all[i] = c > 0 ? behind_s[group][i] : 0.f;
            }
#pragma unroll
            for (int i = 0; i < NH; ++i) {
                float after = 0.f, all = 0.f;
#pragma unroll
                for (int b = 3; b >= 0; --b) {
                    if (b > dw) after += sc.total[i][b];
                    all += sc.total[i][b];
                }
                const float w = stp[i] * ex2(sfx[i] + after + (STATE_ONLY ? total_all[i] : 0.f));
                const __nv_bfloat16 w1 = __float2bfloat16_rn(w), w2 = __float2bfloat16_rn(w - __bfloat162float(w1));
                sc.w1[i][j] = __bfloat16_as_ushort(w1);
                sc.w2[i][j] = __bfloat16_as_ushort(w2);
                total_all[i] += all;
            }
            if constexpr (STATE_ONLY) {
                const int next = (group + 1) % ST;
                if (j == 0)
                    for (int i = 0; i < NH; ++i) behind_s[next][i] = total_all[i];
                warp_arrive(&bar_behind[next], lane);
            } else {
                warp_arrive(&bar_scal[c & 1], lane);
            }
            ok = wait.warp(&full[c % ST], (uint32_t)(c / ST) & 1);
            uint8_t* s = sm + (c % ST) * kStageBytes;
            if (ok && p.cu_seqlens && j >= n_valid) {
                // rows of other sequences, or of none: zeros, so that nothing of theirs enters a sum
                const uint4 zero = make_uint4(0, 0, 0, 0);
                for (int i = 0; i < 8; ++i) {
                    for (int a = 0; a < 2; ++a) *reinterpret_cast<uint4*>(s + OFF_X + a * ATOM + j * 128 + i * 16) = zero;
                    for (int a = 0; a < N / 64; ++a) *reinterpret_cast<uint4*>(s + OFF_B + a * ATOM + j * 128 + i * 16) = zero;
                }
                fence_proxy_async_smem();
            }
            // the operand's place is free
            if constexpr (STATE_ONLY) ok = ok && (c < ST || wait.warp(&bar_upd[group], (uint32_t)(c / ST - 1) & 1));
            else ok = ok && (c == 0 || wait.warp(&bar_upd[0], (uint32_t)(c - 1) & 1));
            // w and the zeros of all tokens; all four warps leave together
            ok = named_bar_and(2 + 2 * group, 32 * kDecayWarps, ok);
            if (!ok) break;
            tc_fence_after_sync();
            // 32 value columns per warp, 32 tokens a step
            const int half = NH == 2 ? dw >> 1 : 0;
            const uint32_t* w1 = reinterpret_cast<const uint32_t*>(sc.w1[half]) + (lane & 3);
            const uint32_t* w2 = reinterpret_cast<const uint32_t*>(sc.w2[half]) + (lane & 3);
            const uint32_t xa = smem_u32(s) + OFF_X + (dw >> 1) * ATOM + (lane & 7) * 128 +
                                (((uint32_t)((dw & 1) * 4 + (lane >> 3)) ^ (lane & 7)) << 4);
#pragma unroll 1
            for (int q4 = 0; q4 < 4; ++q4) {
                uint32_t hi[2][8], lo[2][8];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int tg = 4 * q4 + k;                           // 8 tokens
                    uint32_t x[4];
                    ldmatrix4t(xa + tg * 1024, x);
                    const uint32_t a = w1[4 * tg], b = w2[4 * tg];
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        const uint32_t h = mul_bf16x2(x[m], a);
                        const uint32_t rest = fma_bf16x2(x[m], a, h ^ 0x80008000u);
                        hi[m >> 1][2 * k + (m & 1)] = h;
                        lo[m >> 1][2 * k + (m & 1)] = fma_bf16x2(x[m], b, rest);
                    }
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const uint32_t at = tbase + lanes + ((uint32_t)(16 * u) << 16) + 16 * q4 + TM_HI - 128 * group;
                    tmem_st_16x128(at, hi[u]);
                    tmem_st_16x128(at + 64, lo[u]);
                }
            }
            tmem_wait_st();
            tc_fence_before_sync();
            warp_arrive(STATE_ONLY ? &bar_wst[group] : &bar_w, lane);
        }
        if constexpr (STATE_ONLY) if (group == (chunks - 1) % ST) {
            if (ok && j == 0) {
                p.seg_decay[(size_t)unit * H + h0] = seg_total_s[0] = total_all[0];
                if (NH == 2 && h1 != h0) p.seg_decay[(size_t)unit * H + h1] = total_all[NH - 1];
                seg_total_s[1] = total_all[NH - 1];
            }
            warp_arrive(&bar_state, lane);
        }
    } else if (!STATE_ONLY) {
        // ------------------------------------------------------------ Q (the decayed lower triangle of G), outputs
        const int which = (warp - kFirstScore) >> 2;     // of Q: 16 columns of each 32; of Y: 64 columns
        const int r = 32 * quarter + lane;
        const float skip0 = p.D ? p.D[h0] : 0.f, skip1 = p.D ? p.D[h1] : 0.f;
        const uint32_t yt = tbase + TM_Y + lanes + 64 * which;
        bool ok = true;
        for (int c = 0; c < chunks; ++c) {
            const uint32_t par = c & 1;
            const Scalars& sc = scal[c & 1];
            ok = wait.warp(&bar_scal[c & 1], (c >> 1) & 1) && wait.warp(&bar_g, par);
            tc_fence_after_sync();
            float row = 0.f;                             // 2^{L_r}, of this warp's columns of Y
            {
                float off[48], diag[16];                 // G: blocks 0 to 2 of 32 columns, and the diagonal's
                tmem_read3x16(tbase + TM_G + lanes + 16 * which, off, tbase + TM_G + lanes + 32 * quarter + 16 * which, diag);
                tc_fence_before_sync();
                // both warps of these lanes have read G (Q takes its place).  They leave only here, together.
                ok = named_bar_and(3 + quarter, 64, ok);
                if (!ok) break;
                tc_fence_after_sync();
#pragma unroll
                for (int i = 0; i < NH; ++i) {
                    const uint32_t qt = tbase + TM_G + 64 * i + lanes + 8 * which;
                    const float* colf = sc.col[i] + 16 * which;
                    const float lr = -sc.neg[i][r];
                    float e = lr;                        // sum over the tokens after block b up to r
#pragma unroll
                    for (int b = 2; b >= 0; --b) {
                        if (b >= quarter) continue;
                        const float ee = ex2(e);
                        const uint64_t e2 = pair2(ee, ee);
                        e += sc.total[i][b];
                        uint32_t q[8];
#pragma unroll
                        for (int k = 0; k < 16; k += 4) {
                            const float4 f = *reinterpret_cast<const float4*>(colf + 32 * b + k);
                            const float* gb = off + 16 * b + k;
                            q[k / 2] = mul2_bf16x2(pair2(gb[0], gb[1]), mul2(e2, pair2(f.x, f.y)));
                            q[k / 2 + 1] = mul2_bf16x2(pair2(gb[2], gb[3]), mul2(e2, pair2(f.z, f.w)));
                        }
                        tmem_st8(qt + 16 * b, q);
                    }
                    if (NH == 1 || i == which) row = ex2(e);
                    uint32_t q[8];
                    const float skip = i ? skip1 : skip0;
                    const float* negd = sc.neg[i] + 32 * quarter + 16 * which;
                    const float* stepd = sc.step[i] + 32 * quarter + 16 * which;
                    const int dr = lane - 16 * which;    // the column of the diagonal element
#pragma unroll
                    for (int k = 0; k < 16; k += 4) {
                        const float4 l = *reinterpret_cast<const float4*>(negd + k);
                        const float4 st = *reinterpret_cast<const float4*>(stepd + k);
                        const float lj[4] = {l.x, l.y, l.z, l.w}, sj[4] = {st.x, st.y, st.z, st.w};
                        float v[4];
#pragma unroll
                        for (int d = 0; d < 4; ++d) {
                            const float m = diag[k + d] * (ex2(lr + lj[d]) * sj[d]);
                            v[d] = k + d < dr ? m : k + d == dr ? m + skip : 0.f;
                        }
                        q[k / 2] = bf16x2(v[0], v[1]);
                        q[k / 2 + 1] = bf16x2(v[2], v[3]);
                    }
                    tmem_st8(qt + 16 * quarter, q);
#pragma unroll
                    for (int k = 0; k < 8; ++k) q[k] = 0u;
#pragma unroll 1
                    for (int b = quarter + 1; b < 4; ++b) tmem_st8(qt + 16 * b, q);
                }
            }
            // Y = C S: row r by 2^{L_r}
            ok = wait.warp(&bar_cs, par);
            tc_fence_after_sync();
            {
                float v[64];
                tmem_read64(yt, v);
                scale_by<64>(v, row);
                tmem_write32(yt, v);
                tmem_write32(yt + 32, v + 32);
            }
            tmem_wait_st();
            tc_fence_before_sync();
            warp_arrive(&bar_q, lane);
            // Y, finished: into the chunk's own x tile (all its readers are done), from where the load warp stores it
            // in whole lines
            ok = ok && wait.warp(&bar_px, par);
            tc_fence_after_sync();
            uint8_t* tile_y = sm + (c % kStages) * kStageBytes + OFF_X + which * ATOM;
            const bool whole = !p.cu_seqlens || len - c * kTok >= kTok;
            const int t = c * kTok + r;
            __nv_bfloat16* yr = p.y + ((start + tok0 + t) * H + h0) * P + 64 * which;    // heads h0, h0 + 1 are neighbours
            const bool mine = !(NH == 2 && which == 1 && h1 == h0);
            {
                float v[64];
                tmem_read64(yt, v);
                tc_fence_before_sync();                  // the next C S overwrites Y
                warp_arrive(&bar_yfree, lane);
#pragma unroll
                for (int i = 0; i < 64; i += 8) {
                    const uint4 o = make_uint4(bf16x2(v[i], v[i + 1]), bf16x2(v[i + 2], v[i + 3]),
                                               bf16x2(v[i + 4], v[i + 5]), bf16x2(v[i + 6], v[i + 7]));
                    if (whole) *reinterpret_cast<uint4*>(tile_y + sw128_offset(r, i, ATOM)) = o;
                    else if (mine && ok && t < len) *reinterpret_cast<uint4*>(yr + i) = o;   // rows past a packed sequence stay
                }
            }
            fence_proxy_async_smem();
            warp_arrive(&bar_staged, lane);
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 0) tmem_dealloc(tbase, TM_COLS);
}

// [B, T, heads, d] bf16 with rows `ld` apart as a 4-D tensor (d, heads, T, B); box: 64 channels of one head, 128
// tokens.  Rows past T read as zeros: they add nothing to a sum.
bool make_map(CUtensorMap* m, const void* ptr, int B, int T, int heads, int d, long long ld) {
    auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder());
    if (!enc) return false;
    cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)T, (cuuint64_t)B};
    cuuint64_t strides[3] = {(cuuint64_t)d * 2, (cuuint64_t)ld * 2, (cuuint64_t)T * ld * 2};
    cuuint32_t box[4] = {64, 1, (cuuint32_t)kTok, 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ptr), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int tiles_of(int H, int G, int P) {
    const int rep = H / G;
    return G * (P == 64 ? (rep + 1) / 2 : rep);
}

// Chunks per segment (0: sequences are not cut).  With k segments a sequence's tiles run (k - 1)/k of their chunks
// through the state-only launch and all of them, k times as many CTAs, through the second.  The least of the modelled
// times is taken, in waves of 148 CTAs and units of a chunk of the full kernel: a state-only chunk costs kStateCost of
// one, the second launch and the start states about kSplitCost chunks.
constexpr double kStateCost = 0.27, kSplitCost = 6.0;
constexpr int kMostSegments = 8;

int segment_chunks(int n_seq, long long T_total, int H, int P) {
    const double ctas = (double)n_seq * (P == 64 ? (H + 1) / 2 : H);
    const long long chunks = (T_total / n_seq + kTok - 1) / kTok;         // of a sequence, on average
    auto waves = [](double n) { return (double)(long long)((n + 147.0) / 148.0); };
    double best = waves(ctas) * (double)chunks;
    int cut = 0;
    for (int k = 2; k <= kMostSegments && k <= chunks; ++k) {
        const long long len = (chunks + k - 1) / k;
        const double t = len * (waves(ctas * (k - 1)) * kStateCost + waves(ctas * k)) + kSplitCost;
        if (t < best) {
            best = t;
            cut = (int)len;
        }
    }
    return cut;
}

// Upper bound of the units (segments of sequences) of a call.
long long units_of(int n_seq, long long T_total, int seg_chunks) {
    return seg_chunks == 0 ? n_seq : n_seq + T_total / ((long long)seg_chunks * kTok);
}

size_t workspace_of(long long units, int H, int N, int P) {
    return (size_t)units * H * ((size_t)N * P + 1) * sizeof(float);
}

template <int N, int P, bool STATE_ONLY>
cudaError_t launch_one(const CUtensorMap& mx, const CUtensorMap& mb, const CUtensorMap& mc, const CUtensorMap& my,
                       const Params& p, long long units, cudaStream_t s) {
    static std::mutex mu;
    static bool attr_set[64] = {false};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (dev >= 64 || !attr_set[dev]) {
            e = cudaFuncSetAttribute(kda_ssm_tc_kernel<N, P, STATE_ONLY>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_DYN);
            if (e != cudaSuccess) return e;
            if (dev < 64) attr_set[dev] = true;
        }
    }
    const long long grid = units * p.tiles;
    if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    kda_ssm_tc_kernel<N, P, STATE_ONLY><<<(unsigned)grid, kThreads, SMEM_DYN, s>>>(mx, mb, mc, my, p);
    return cudaGetLastError();
}

template <int N, int P>
cudaError_t launch_np(const CUtensorMap& mx, const CUtensorMap& mb, const CUtensorMap& mc, const CUtensorMap& my,
                      const Params& p, long long units, cudaStream_t s) {
    if (p.seg_chunks > 0) {
        const cudaError_t e = launch_one<N, P, true>(mx, mb, mc, my, p, units, s);
        if (e != cudaSuccess) return e;
    }
    return launch_one<N, P, false>(mx, mb, mc, my, p, units, s);
}

}  // namespace

bool ssm_tc_supports(const SsmArgs& a) { return a.dtype == KDA_DTYPE_BF16; }

size_t ssm_tc_workspace(int n_seq, long long T_total, int H, int N, int P) {
    if (T_total == 0) return 0;
    const int seg_chunks = segment_chunks(n_seq, T_total, H, P);
    return seg_chunks == 0 ? 0 : workspace_of(units_of(n_seq, T_total, seg_chunks), H, N, P);
}

cudaError_t launch_ssm_tc(const SsmArgs& a, cudaStream_t s) {
    const int B = a.cu_seqlens ? 1 : a.n_seq;
    if (a.T == 0) {
        // packed sequences without tokens: S_T = S0
        if (!a.ST || a.ST == a.S0) return cudaSuccess;
        const size_t bytes = (size_t)a.n_seq * a.H * a.N * a.P * sizeof(float);
        return a.S0 ? cudaMemcpyAsync(a.ST, a.S0, bytes, cudaMemcpyDeviceToDevice, s) : cudaMemsetAsync(a.ST, 0, bytes, s);
    }
    CUtensorMap mx, mb, mc, my;
    if (!make_map(&mx, a.x, B, a.T, a.H, a.P, a.ldx) || !make_map(&mb, a.Bm, B, a.T, a.G, a.N, a.ldb) ||
        !make_map(&mc, a.Cm, B, a.T, a.G, a.N, a.ldc) || !make_map(&my, a.y, B, a.T, a.H, a.P, (long long)a.H * a.P))
        return cudaErrorInvalidValue;
    Params p{};
    p.dt = static_cast<const __nv_bfloat16*>(a.dt);
    p.A = a.A;
    p.D = a.D;
    p.dt_bias = a.dt_bias;
    p.S0 = a.S0;
    p.y = static_cast<__nv_bfloat16*>(a.y);
    p.ST = a.ST;
    p.cu_seqlens = a.cu_seqlens;
    p.lddt = a.lddt;
    p.n_seq = a.n_seq;
    p.T = a.T;
    p.H = a.H;
    p.G = a.G;
    p.tiles = tiles_of(a.H, a.G, a.P);
    const long long T_total = a.cu_seqlens ? a.T : (long long)a.n_seq * a.T;
    p.seg_chunks = segment_chunks(a.n_seq, T_total, a.H, a.P);
    long long units = units_of(a.n_seq, T_total, p.seg_chunks);
    p.seg_state = static_cast<float*>(a.workspace);
    p.seg_decay = p.seg_state + (size_t)units * a.H * a.N * a.P;          // units does not grow below
    p.segs = 1;
    if (p.seg_chunks > 0 && !a.cu_seqlens) {
        p.segs = (a.T + p.seg_chunks * kTok - 1) / (p.seg_chunks * kTok);
        units = (long long)a.n_seq * p.segs;
    }
    p.status = a.status;
    p.timeout_ns = a.timeout_ns;
    p.skip_handoff = a.skip_handoff;
    if (a.N == 128) return a.P == 128 ? launch_np<128, 128>(mx, mb, mc, my, p, units, s) : launch_np<128, 64>(mx, mb, mc, my, p, units, s);
    return a.P == 128 ? launch_np<64, 128>(mx, mb, mc, my, p, units, s) : launch_np<64, 64>(mx, mb, mc, my, p, units, s);
}

}  // namespace kda
