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
// off by at most 3 * 2^-16 of itself.  The sixteen products of a chunk that add to the state round it towards
// zero, up to 2^-23 of it each (8e-7 a chunk measured: 3.9e-5 after 8192 tokens without decay, 6e-6 of a state
// that remembers a thousand tokens).  With the state's leading bits kept out of those sums (the carried state less
// its bf16 copy, which lies in shared memory, added again a chunk later) 3.3e-7 of it were lost at any length, but
// the launches took 7 to 9 % longer (621 -> 679 us); the outputs' own rounding, 2^-8, hides either.
//
// What bounds it.  Per chunk of a 128-column tile HBM moves 64 KB of x and y (2.8K cycles at the measured
// copy rate with all SMs at it), the tensor core needs 2.5K cycles, and shared memory 3.5K (the products'
// operands and the tiles' own way in and out).  4 x 8192 tokens with 96 heads of 128, three waves of 64
// chunks, take 527 to 535 us for the first 50 ms of a run, at 1965 MHz: 5.4K cycles a chunk, 4.2K where nothing
// contends.  Kept up for seconds the GPU reaches its power limit and about 1.5 GHz, and they take 610 to 636 us:
// 4.8K of the longer cycles, of which HBM takes fewer.  (Times of variants below are of short runs.)  Loops of
// about one length bound it: the warps' own steps, each a pass from tensor memory through registers and back; C S, the
// update, the weighted x and the carried state, which wait for one another; and the loads of B and C.
// Operands are kept out of shared memory where a product allows: Q and the weighted x are tensor-memory
// operands, and the state is held transposed (lanes = value columns) for that.  The weighted x is transposed
// on its way by ldmatrix and the 16x128b stores, whose fragments have one layout.
//
// Sixteen warps do every step together, a quarter of the columns or tokens to a group of four, in an order
// that lets the products run behind them: Q while Y = C S runs, the next chunk's weighted x and carried
// state while Q X runs.  Four more warps issue the products, move the tiles, and form the decays two chunks
// ahead.  Warps that keep to one step each, 21 of them, took 10 % longer with two heads to a tile (480 against
// 424 us at 4 x 8192 tokens, 96 heads of 64) and the same with one.  The issuing and the loading warp run
// whole, with one elected thread at the products and copies, and the warp's number is made uniform: the
// compiler then keeps descriptors and addresses in uniform registers (issued by a lane that merely compares
// itself with 0, each product cost 90 cycles of the thread, more than it takes: 599 against 530 us).
// x has three stages: a tile is y's place when it is done, and is read out (1.8K cycles) while the next two
// are at work; B and C have one, free once they are used.  Tensor memory (512 columns): S^T, Y, G (then Q in
// its place), weighted x hi and lo.
//
// Long prompts with few heads: the tokens are cut into segments.  A first launch forms the state of every
// segment but the last (B and x only; the first one from S0, the others from zero), going through the
// chunks backwards, so that the weights hold the decay to the segment's end and the products just add up;
// the second starts each segment from the segments before it, S <- 2^{total} S + local, folded in as it
// loads its start state.
//
// No barrier completes twice before its waiter has looked (the parity would then stand for the phase before):
// each next phase needs something that the waiter does after its wait.  Every wait is bounded in time; a wait
// that runs out sets the status word and an abort flag that ends the other warps' waits, the products and
// loads in flight are drained, and the CTA returns.
#include <cudaTypedefs.h>
#include <mutex>

#include "kda_serving.cuh"
#include "sm100_ptx.cuh"

namespace kda {
namespace {

using namespace sm100;

constexpr int kTok = 128;                    // tokens per chunk
constexpr int kCols = 128;                   // value columns per CTA
// A token's decay (log 2) is not taken below this: every exponential over such a token is zero all the same, and the
// sums before and after it differ by few enough that the differences of later ones keep their digits.
constexpr float kLeastDecay = -160.f;
constexpr int kStages = 3;                   // of x, which is y's place when it is done
constexpr int kStateStages = 3;              // of B and x together, in the state-only kernel
constexpr int kWorkers = 16;                 // warps that do the arithmetic
constexpr int kIssueWarp = kWorkers, kLoadWarp = kWorkers + 1, kDecayWarp = kWorkers + 2;   // two decay warps
constexpr int kThreads = 32 * (kWorkers + 4);
constexpr uint32_t ATOM = 16384;             // [128 rows][64 columns] bf16, 128-byte swizzle
constexpr uint32_t kTile = 2 * ATOM;

// shared memory: x, B, C, S as bf16 (rows = value columns, K = N)
constexpr uint32_t OFF_X = 0, OFF_B = kStages * kTile, OFF_C = OFF_B + kTile, OFF_S = OFF_C + kTile;
constexpr uint32_t SMEM_DYN = OFF_S + kTile + 1024;
constexpr uint32_t kStageBytes = 2 * kTile;  // state-only kernel: B, then x
static_assert(kStateStages * kStageBytes + 1024 <= SMEM_DYN, "the state-only kernel's stages fit");

// tensor memory columns (the state-only kernel's three groups have their weighted x at TM_W, TM_G and TM_Y)
constexpr uint32_t TM_S = 0, TM_Y = 128, TM_G = 256, TM_W = 384, TM_COLS = 512;
constexpr uint32_t kUpper = 16u << 16;       // the second 16 lanes of a warp's quarter of the tensor memory

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
// TMEM -> registers, 32 columns, complete on return.  Load and wait are one statement: between two, the
// compiler may move or spill registers that the load has not written yet.
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
// Four runs of 8 columns, 32 apart.
__device__ __forceinline__ void tmem_read4x8(uint32_t taddr, float* r) {
    uint32_t* u = reinterpret_cast<uint32_t*>(r);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%32];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%8, %9, %10, %11, %12, %13, %14, %15}, [%33];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%16, %17, %18, %19, %20, %21, %22, %23}, [%34];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%24, %25, %26, %27, %28, %29, %30, %31}, [%35];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=&r"(u[0]), "=&r"(u[1]), "=&r"(u[2]), "=&r"(u[3]), "=&r"(u[4]), "=&r"(u[5]), "=&r"(u[6]), "=&r"(u[7]),
          "=&r"(u[8]), "=&r"(u[9]), "=&r"(u[10]), "=&r"(u[11]), "=&r"(u[12]), "=&r"(u[13]), "=&r"(u[14]), "=&r"(u[15]),
          "=&r"(u[16]), "=&r"(u[17]), "=&r"(u[18]), "=&r"(u[19]), "=&r"(u[20]), "=&r"(u[21]), "=&r"(u[22]), "=&r"(u[23]),
          "=&r"(u[24]), "=&r"(u[25]), "=&r"(u[26]), "=&r"(u[27]), "=&r"(u[28]), "=&r"(u[29]), "=&r"(u[30]), "=&r"(u[31])
        : "r"(taddr), "r"(taddr + 32), "r"(taddr + 64), "r"(taddr + 96)
        : "memory");
}
__device__ __forceinline__ void tmem_st4(uint32_t taddr, const uint32_t* u) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(u[0]), "r"(u[1]),
                 "r"(u[2]), "r"(u[3])
                 : "memory");
}

// Bounded waits of a whole warp, that also end when another warp of the CTA has given up.  The branch is the warp's,
// not a lane's, and all lanes have the same answer.
struct Waiter {
    volatile int* abort_flag;
    int* status;
    unsigned long long timeout_ns;

    __device__ __noinline__ bool slow(uint32_t a, uint32_t parity) const {
        const uint64_t t0 = global_timer_ns();
        for (;;) {
            if (__any_sync(0xffffffffu, *abort_flag)) return false;
#pragma unroll 1
            for (int i = 0; i < 32; ++i)
                if (__all_sync(0xffffffffu, mbar_try_wait(a, parity))) return true;
            if (__any_sync(0xffffffffu, global_timer_ns() - t0 > timeout_ns)) {
                *abort_flag = 1;
                report_status(status, KDA_ERR_TIMEOUT);
                return false;
            }
        }
    }
    __device__ __forceinline__ bool warp(uint64_t* bar, uint32_t parity) const {
        const uint32_t a = smem_u32(bar);
        return __all_sync(0xffffffffu, mbar_try_wait(a, parity)) || slow(a, parity);
    }
};

// A value that is the same in all lanes, so that the compiler knows it.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }
// true in one lane of the (converged) warp
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}

__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
}

// The second launch of a call may start while the first one runs: the first lets it once all of its CTAs are on their
// SMs; the second sets itself up, starts its loads, and waits for the first one's end (and its writes).  At 4096
// tokens and 32 heads of 128 that takes 3.5 us off 59.
__device__ __forceinline__ void let_next_launch_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_launch_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The tokens and heads of a CTA.
struct Job {
    int unit, unit0, seq, seg, n_seg;        // unit: the sequence's segment; unit0: its first segment
    int g, h0, h1;                           // group and heads (h1 == h0: no second head)
    int tok0, len, chunks;                   // first token within the sequence, tokens, chunks
    bool last;                               // the sequence's last segment
    size_t start;                            // token 0 of the job on the token axis of x, dt and y
    int row0, row_seq;                       // coordinates of the first chunk in the tensor maps
};

// Block-wide (it has barriers).  False: the CTA has no job.
template <int NH>
__device__ __forceinline__ bool find_job(const Params& p, Job& job) {
    __shared__ int seq_s, seg_s;
    const int tid = threadIdx.x, lane = tid & 31;
    const int tile = blockIdx.x % p.tiles;
    job.unit = blockIdx.x / p.tiles;
    const int rep = p.H / p.G, per_group = (rep + NH - 1) / NH;
    job.g = tile / per_group;
    job.h0 = job.g * rep + (tile % per_group) * NH;
    job.h1 = NH == 2 && job.h0 + 1 < (job.g + 1) * rep ? job.h0 + 1 : job.h0;
    const int seg_tokens = p.seg_chunks > 0 ? p.seg_chunks * kTok : 0x7fffffff;
    int len_seq;
    size_t start;
    if (p.cu_seqlens) {
        const bool valid = packed_offsets_valid(p.cu_seqlens, p.n_seq, p.T);
        if (!valid && tid == 0) report_status(p.status, KDA_ERR_INVALID_ARG);
        job.seq = job.unit;
        job.seg = 0;
        if (p.seg_chunks > 0) {
            // units in order: each sequence's segments (one for an empty sequence)
            if (tid == 0) seq_s = -1;
            __syncthreads();
            if (tid < 32) {
                int before = 0;
                for (int base = 0; base < p.n_seq; base += 32) {
                    const int i = base + lane;
                    int n = 0;
                    if (i < p.n_seq) {
                        const int len = valid ? p.cu_seqlens[i + 1] - p.cu_seqlens[i] : 0;
                        n = max(1, (len + seg_tokens - 1) / seg_tokens);
                    }
                    int incl = n;
#pragma unroll
                    for (int off = 1; off < 32; off <<= 1) {
                        const int t = __shfl_up_sync(0xffffffffu, incl, off);
                        if (lane >= off) incl += t;
                    }
                    if (job.unit >= before + incl - n && job.unit < before + incl) {
                        seq_s = i;
                        seg_s = job.unit - (before + incl - n);
                    }
                    before += __shfl_sync(0xffffffffu, incl, 31);
                    if (job.unit < before) break;
                }
            }
            __syncthreads();
            job.seq = seq_s;
            job.seg = seg_s;
            if (job.seq < 0) return false;   // the grid holds the most units that T tokens can make
        }
        start = valid ? (size_t)p.cu_seqlens[job.seq] : 0;
        len_seq = valid ? p.cu_seqlens[job.seq + 1] - p.cu_seqlens[job.seq] : 0;
        job.row_seq = 0;
        job.row0 = (int)start;
    } else {
        job.seq = job.unit / p.segs;
        job.seg = job.unit % p.segs;
        start = (size_t)job.seq * p.T;
        len_seq = p.T;
        job.row_seq = job.seq;
        job.row0 = 0;
    }
    job.tok0 = job.seg * (p.seg_chunks * kTok);
    job.row0 += job.tok0;
    job.start = start + job.tok0;
    job.len = min(len_seq - job.tok0, seg_tokens);
    job.last = job.tok0 + job.len >= len_seq;
    job.chunks = (job.len + kTok - 1) / kTok;
    job.n_seg = p.seg_chunks > 0 ? max(1, (len_seq + seg_tokens - 1) / seg_tokens) : 1;
    job.unit0 = job.unit - job.seg;
    return true;
}

// The states of one value column (a lane of the warp, in its quarter of the tensor-memory lanes).
template <int N, int P>
struct Column {
    static constexpr int NH = P == 64 ? 2 : 1;
    const Params& p;
    const Job& job;
    int head, pc;
    bool dup;                                // carried, not stored
    size_t s_off;                            // S[seq][head][0][pc]

    __device__ __forceinline__ Column(const Params& p_, const Job& job_, int col) : p(p_), job(job_) {
        const int half = NH == 2 ? col >> 6 : 0;
        head = half ? job.h1 : job.h0;
        pc = NH == 2 ? col & 63 : col;
        dup = NH == 2 && half == 1 && job.h1 == job.h0;
        s_off = (((size_t)job.seq * p.H + head) * N) * P + pc;
    }
    __device__ __forceinline__ float* seg_state(int unit) const {
        return p.seg_state + ((size_t)unit * p.H + head) * N * P + pc;
    }
    __device__ __forceinline__ void store(float* to, int n0, const float* v) const {
        if (!dup) {
#pragma unroll
            for (int i = 0; i < 32; ++i) to[(size_t)(n0 + i) * P] = v[i];
        }
    }
    __device__ __forceinline__ void load(const float* from, int n0, float* v) const {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = from ? from[(size_t)(n0 + i) * P] : 0.f;
    }
    // The start state of 32 rows n.  Sequences of several segments: the first launch starts segment 0 from S0,
    // and leaves a copy of S0 in the last segment's place, which no local state takes; the second launch reads S0
    // nowhere else, so that S_T may be S0.
    __device__ __forceinline__ void load_start(int n0, float* v) const {
        if (job.n_seg == 1) return load(p.S0 ? p.S0 + s_off : nullptr, n0, v);
        load(seg_state(job.seg == 0 ? job.unit0 + job.n_seg - 1 : job.unit0), n0, v);
#pragma unroll 1
        for (int k = 1; k < job.seg; ++k) {
            const float d = ex2(p.seg_decay[(size_t)(job.unit0 + k) * p.H + head]);
            float l[32];
            load(seg_state(job.unit0 + k), n0, l);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = fmaf(d, v[i], l[i]);
        }
    }
};

// Sums over a block of 32 tokens, one to a lane: up to the token (inclusive), and after it.
__device__ __forceinline__ void block_sums(float la, int lane, float& incl, float& after) {
    float rev = la;
    incl = la;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const float a = __shfl_up_sync(0xffffffffu, incl, off), b = __shfl_down_sync(0xffffffffu, rev, off);
        if (lane >= off) incl += a;
        if (lane + off < 32) rev += b;
    }
    const float next = __shfl_down_sync(0xffffffffu, rev, 1);
    after = lane == 31 ? 0.f : next;
}
__device__ __forceinline__ void store_weight(Scalars& sc, int i, int j, float w) {
    const __nv_bfloat16 w1 = __float2bfloat16_rn(w), w2 = __float2bfloat16_rn(w - __bfloat162float(w1));
    sc.w1[i][j] = __bfloat16_as_ushort(w1);
    sc.w2[i][j] = __bfloat16_as_ushort(w2);
}
// The weighted x of 32 tokens (groups of 8 from tg0 on) and a warp's 32 value columns, hi and lo, into the tensor
// memory at `place` (lanes = value columns, columns = pairs of tokens).
__device__ __forceinline__ void weigh_x(uint32_t place, const Scalars& sc, int half, uint32_t x_tile, int quarter,
                                        int lane, int tg0) {
    const uint32_t xa = x_tile + (quarter >> 1) * ATOM + (lane & 7) * 128 +
                        (((uint32_t)((quarter & 1) * 4 + (lane >> 3)) ^ (lane & 7)) << 4);
    const uint32_t* w1 = reinterpret_cast<const uint32_t*>(sc.w1[half]) + (lane & 3);
    const uint32_t* w2 = reinterpret_cast<const uint32_t*>(sc.w2[half]) + (lane & 3);
    uint32_t hi[2][8], lo[2][8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint32_t x[4];
        ldmatrix4t(xa + (tg0 + k) * 1024, x);
        const uint32_t a = w1[4 * (tg0 + k)], b = w2[4 * (tg0 + k)];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const uint32_t h = mul_bf16x2(x[m], a);
            hi[m >> 1][2 * k + (m & 1)] = h;
            lo[m >> 1][2 * k + (m & 1)] = fma_bf16x2(x[m], b, fma_bf16x2(x[m], a, h ^ 0x80008000u));
        }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        tmem_st_16x128(place + 4 * tg0 + u * kUpper, hi[u]);
        tmem_st_16x128(place + 4 * tg0 + u * kUpper + 64, lo[u]);
    }
}

// Loads of a chunk's x and B.
template <int NH>
__device__ __forceinline__ void load_x(uint8_t* to, const CUtensorMap* tm_x, uint64_t* full, const Job& job, int row) {
    for (int i = 0; i < 2; ++i)
        tma_load_4d(to + i * ATOM, tm_x, full, NH == 2 ? 0 : 64 * i, NH == 2 && i ? job.h1 : job.h0, row, job.row_seq);
}
template <int N>
__device__ __forceinline__ void load_bc(uint8_t* to, const CUtensorMap* tm, uint64_t* full, const Job& job, int row) {
    for (int i = 0; i < N / 64; ++i) tma_load_4d(to + i * ATOM, tm, full, 64 * i, job.g, row, job.row_seq);
}
template <int N>
__device__ __forceinline__ void prefetch_bc(const CUtensorMap* tm, const Job& job, int row) {
    for (int i = 0; i < N / 64; ++i) tma_prefetch_4d(tm, 64 * i, job.g, row, job.row_seq);
}
template <int NH>
__device__ __forceinline__ void prefetch_x(const CUtensorMap* tm_x, const Job& job, int row) {
    for (int i = 0; i < 2; ++i)
        tma_prefetch_4d(tm_x, NH == 2 ? 0 : 64 * i, NH == 2 && i ? job.h1 : job.h0, row, job.row_seq);
}

// ------------------------------------------------------------------ states of the segments

constexpr int kStateThreads = 32 * 18;       // 0-3 the end; 4-15 three groups, each every third chunk; 16 products, 17 loads

template <int N, int P>
__global__ void __launch_bounds__(kStateThreads, 1)
kda_ssm_state_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_b, const Params p) {
    constexpr int NH = P == 64 ? 2 : 1, ST = kStateStages;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_base = smem_u32(smem_raw);
    uint8_t* sm = smem_raw + (((raw_base + 1023u) & ~1023u) - raw_base);
    const uint32_t sb = (raw_base + 1023u) & ~1023u;
    __shared__ Scalars scal[ST];
    __shared__ uint64_t full[ST], empty[ST], bar_w[ST], bar_upd[ST], bar_behind[ST], bar_total, bar_drain;
    __shared__ float behind_s[ST][2], total_s[2];
    __shared__ uint32_t tmem_base_s;
    __shared__ volatile int abort_s;
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31, quarter = warp & 3;
    Job job;
    let_next_launch_start();
    if (!find_job<NH>(p, job) || job.last) return;
    const int chunks = job.chunks;           // all whole
    if (tid == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
            mbar_init(&bar_w[i], 4);
            mbar_init(&bar_upd[i], 1);
            mbar_init(&bar_behind[i], 4);
        }
        mbar_init(&bar_total, 4);
        mbar_init(&bar_drain, 1);
        fence_mbar_init();
        abort_s = 0;
        prefetch_tensormap(&tm_x);
        prefetch_tensormap(&tm_b);
    }
    if (warp == 0) {
        tmem_alloc(&tmem_base_s, TM_COLS);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    constexpr uint32_t tbase = 0;            // all columns are this CTA's
    const Waiter wait{&abort_s, p.status, p.timeout_ns};
    const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
    auto row_of = [&](int c) { return job.row0 + (chunks - 1 - c) * kTok; };   // from the last chunk to the first

    if (warp == 17) {
        const bool leader = elect_one();
        int issued = 0;
        for (int c = 0; c < chunks; ++c) {
            if (c >= ST && !wait.warp(&empty[c % ST], (uint32_t)(c / ST - 1) & 1)) break;
            if (leader) {
                uint8_t* stage = sm + (c % ST) * kStageBytes;
                mbar_arrive_expect_tx(&full[c % ST], ATOM * (2 + N / 64));
                load_bc<N>(stage, &tm_b, &full[c % ST], job, row_of(c));
                load_x<NH>(stage + kTile, &tm_x, &full[c % ST], job, row_of(c));
                if (c + ST < chunks) prefetch_x<NH>(&tm_x, job, row_of(c + ST));
            }
            __syncwarp();
            ++issued;
        }
        // nothing may be in flight when the CTA exits
        for (int c = max(0, issued - ST); c < issued; ++c)
            if (leader && !mbar_wait(&full[c % ST], (uint32_t)(c / ST) & 1, p.timeout_ns)) report_status(p.status, KDA_ERR_TIMEOUT);
        __syncwarp();
    } else if (warp == 16) {
        const bool leader = elect_one();
        const uint32_t id_up = idesc_bf16_f32(128, N, false, true);
        for (int c = 0; c < chunks; ++c) {
            const uint32_t b_tile = sb + (c % ST) * kStageBytes, w = tbase + TM_W - 128 * (c % ST);
            if (!wait.warp(&bar_w[c % ST], (uint32_t)(c / ST) & 1)) break;
            tc_fence_after_sync();
            if (leader) {
                issue_ts(tbase + TM_S, w, b_tile, id_up, c > 0);
                issue_ts(tbase + TM_S, w + 64, b_tile, id_up, true);
                mma_commit(&bar_upd[c % ST]);
                mma_commit(&empty[c % ST]);
            }
            __syncwarp();
        }
        if (leader) {
            mma_commit(&bar_drain);
            if (!mbar_wait(&bar_drain, 0, p.timeout_ns)) report_status(p.status, KDA_ERR_TIMEOUT);
        }
        __syncwarp();
    } else if (warp < 4) {
        // the segment's state: the sum of its chunks, and for the first segment what is left of S0
        const Column<N, P> col(p, job, 32 * quarter + lane);
        bool ok = wait.warp(&bar_total, 0) && wait.warp(&bar_upd[(chunks - 1) % ST], (uint32_t)((chunks - 1) / ST) & 1);
        tc_fence_after_sync();
        const float decay = ex2(total_s[NH == 2 ? quarter >> 1 : 0]);
#pragma unroll 1
        for (int n0 = 0; n0 < N && ok; n0 += 32) {
            float v[32], start[32];
            tmem_read32(tbase + TM_S + lanes + n0, v);
            if (job.seg == 0) {
                col.load(p.S0 ? p.S0 + col.s_off : nullptr, n0, start);
                col.store(col.seg_state(job.unit0 + job.n_seg - 1), n0, start);
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = fmaf(decay, start[i], v[i]);
            }
            col.store(col.seg_state(job.unit), n0, v);
        }
    } else {
        const int group = (warp >> 2) - 1, j = 32 * quarter + lane;
        float rate[NH], bias[NH], raw[NH], behind[NH];
#pragma unroll
        for (int i = 0; i < NH; ++i) {
            const int head = i ? job.h1 : job.h0;
            rate[i] = p.A[head] * 1.4426950408889634f;                   // decays in powers of two
            bias[i] = p.dt_bias ? p.dt_bias[head] : 0.f;
            behind[i] = 0.f;
        }
        auto load_dt = [&](int c) {
#pragma unroll
            for (int i = 0; i < NH; ++i)
                raw[i] = load_elem(p.dt, (job.start + (size_t)(chunks - 1 - c) * kTok + j) * p.lddt + (i ? job.h1 : job.h0));
        };
        if (group < chunks) load_dt(group);
        bool ok = true;
        for (int c = group; c < chunks; c += ST) {
            Scalars& sc = scal[group];
            float after[NH], stp[NH];
#pragma unroll
            for (int i = 0; i < NH; ++i) {
                stp[i] = softplus(raw[i] + bias[i]);
                float incl;
                block_sums(stp[i] * rate[i], lane, incl, after[i]);
                if (lane == 31) sc.total[i][quarter] = incl;
            }
            if (c + ST < chunks) load_dt(c + ST);
            named_bar_sync(1 + 2 * group, 128);
            // the decay behind the chunk, handed on from group to group
            if (c > 0) (void)wait.warp(&bar_behind[group], (uint32_t)((c - 1) / ST) & 1);
            const int next = (group + 1) % ST;
#pragma unroll
            for (int i = 0; i < NH; ++i) {
                behind[i] = c > 0 ? behind_s[group][i] : 0.f;
                float rest = after[i] + behind[i], all = behind[i];
#pragma unroll
                for (int b = 3; b >= 0; --b) {
                    if (b > quarter) rest += sc.total[i][b];
                    all += sc.total[i][b];
                }
                store_weight(sc, i, j, stp[i] * ex2(rest));
                behind[i] = all;
                if (j == 0) behind_s[next][i] = all;
            }
            warp_arrive(&bar_behind[next], lane);
            ok = wait.warp(&full[c % ST], (uint32_t)(c / ST) & 1) &&
                 (c < ST || wait.warp(&bar_upd[group], (uint32_t)(c / ST - 1) & 1));   // the operand's place is free
            ok = named_bar_and(2 + 2 * group, 128, ok);                  // w of all tokens; the four warps leave together
            if (!ok) break;
            tc_fence_after_sync();
#pragma unroll 1
            for (int tg = 0; tg < 16; tg += 4)
                weigh_x(tbase + lanes + TM_W - 128 * group, sc, NH == 2 ? quarter >> 1 : 0, sb + group * kStageBytes + kTile,
                        quarter, lane, tg);
            tmem_wait_st();
            tc_fence_before_sync();
            if (!(p.skip_handoff && c == 0)) warp_arrive(&bar_w[group], lane);
        }
        if (group == (chunks - 1) % ST) {
            if (ok && j == 0) {
                p.seg_decay[(size_t)job.unit * p.H + job.h0] = total_s[0] = behind[0];
                if (NH == 2 && job.h1 != job.h0) p.seg_decay[(size_t)job.unit * p.H + job.h1] = behind[NH - 1];
                total_s[1] = behind[NH - 1];
            }
            warp_arrive(&bar_total, lane);
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 0) tmem_dealloc(tmem_base_s, TM_COLS);
}

// ------------------------------------------------------------------ outputs and states

template <int N, int P>
__global__ void __launch_bounds__(kThreads, 1)
kda_ssm_tc_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_b,
                  const __grid_constant__ CUtensorMap tm_c, const __grid_constant__ CUtensorMap tm_y, const Params p) {
    constexpr int NH = P == 64 ? 2 : 1;      // heads per tile
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_base = smem_u32(smem_raw);
    uint8_t* sm = smem_raw + (((raw_base + 1023u) & ~1023u) - raw_base);
    const uint32_t sb = (raw_base + 1023u) & ~1023u;
    __shared__ Scalars scal[2];
    __shared__ uint64_t full_x[kStages], full_b, full_c, bar_scal[2], scal_free[2], bar_g, bar_cs, bar_upd, bar_px,
        bar_state, bar_w, bar_q, bar_yfree, bar_staged[2], bar_drain;
    __shared__ uint32_t tmem_base_s;
    __shared__ volatile int abort_s;
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31, quarter = warp & 3;
    Job job;
    if (!find_job<NH>(p, job)) return;
    const int chunks = job.chunks;

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(&full_x[i], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar_scal[i], NH);
            mbar_init(&scal_free[i], kWorkers);
            mbar_init(&bar_staged[i], kWorkers);
        }
        mbar_init(&full_b, 1);
        mbar_init(&full_c, 1);
        mbar_init(&bar_drain, 1);
        mbar_init(&bar_g, 1);
        mbar_init(&bar_cs, 1);
        mbar_init(&bar_upd, 1);
        mbar_init(&bar_px, 1);
        mbar_init(&bar_state, kWorkers);
        mbar_init(&bar_w, kWorkers);
        mbar_init(&bar_q, kWorkers);
        mbar_init(&bar_yfree, kWorkers);
        fence_mbar_init();
        abort_s = 0;
        prefetch_tensormap(&tm_x); prefetch_tensormap(&tm_b); prefetch_tensormap(&tm_c); prefetch_tensormap(&tm_y);
    }
    if (warp == 0) {
        tmem_alloc(&tmem_base_s, TM_COLS);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    constexpr uint32_t tbase = 0;            // all columns are this CTA's
    const Waiter wait{&abort_s, p.status, p.timeout_ns};

    if (warp == kLoadWarp) {
        // ------------------------------------------------------------ loads, and stores of y from the x tiles
        const bool leader = elect_one();
        int xs = 0, bs = 0, cs = 0;                                      // loads issued
        auto x_in = [&](int c) {
            if (c >= chunks) return;
            if (leader) {
                const int st = c % kStages;
                mbar_arrive_expect_tx(&full_x[st], kTile);
                load_x<NH>(sm + OFF_X + st * kTile, &tm_x, &full_x[st], job, job.row0 + c * kTok);
                // x of the stage's next turn, which no other CTA reads, into L2
                if (c + kStages < chunks) prefetch_x<NH>(&tm_x, job, job.row0 + (c + kStages) * kTok);
            }
            __syncwarp();
            ++xs;
        };
        auto bc_in = [&](int c, uint32_t off, const CUtensorMap* tm, uint64_t* full, int& n) {
            if (c >= chunks) return;
            if (leader) {
                mbar_arrive_expect_tx(full, kTile / 128 * N);
                load_bc<N>(sm + off, tm, full, job, job.row0 + c * kTok);
                if (c + 1 < chunks) prefetch_bc<N>(tm, job, job.row0 + (c + 1) * kTok);
            }
            __syncwarp();
            ++n;
        };
        auto y_out = [&](int c) {
            // two barriers in turn: the last chunk's y may be in place before y of the one before is looked for (what
            // comes after that needs loads of this warp's)
            if (!wait.warp(&bar_staged[c & 1], (uint32_t)(c >> 1) & 1)) return false;
            if (leader && (!p.cu_seqlens || job.len - c * kTok >= kTok)) {       // whole tiles, clipped at the end of the tensor
                for (int i = 0; i < 2; ++i)
                    if (!(NH == 2 && i == 1 && job.h1 == job.h0))
                        tma_store_4d(&tm_y, sm + OFF_X + (c % kStages) * kTile + i * ATOM, NH == 2 ? 0 : 64 * i,
                                     NH == 2 && i ? job.h1 : job.h0, job.row0 + c * kTok, job.row_seq);
                bulk_commit_group();
            }
            __syncwarp();
            return true;
        };
        bc_in(0, OFF_C, &tm_c, &full_c, cs);
        bc_in(0, OFF_B, &tm_b, &full_b, bs);
        for (int c = 0; c < kStages; ++c) x_in(c);
        wait_for_launch_before();
        for (int c = 0; c < chunks; ++c) {
            // in the order in which their places become free
            if (c > 0 && !y_out(c - 1)) break;
            if (!wait.warp(&bar_cs, c & 1)) break;
            bc_in(c + 1, OFF_C, &tm_c, &full_c, cs);
            if (!wait.warp(&bar_upd, c & 1)) break;
            bc_in(c + 1, OFF_B, &tm_b, &full_b, bs);
            if (c > 0) {                                                 // x, once that y has been read out
                if (leader) bulk_wait_read_all();
                __syncwarp();
                x_in(c + kStages - 1);
            }
            if (c == chunks - 1) (void)y_out(c);
        }
        // nothing may be in flight when the CTA exits
        if (leader) {
            bool done = bs == 0 || mbar_wait(&full_b, (uint32_t)(bs - 1) & 1, p.timeout_ns);
            done = (cs == 0 || mbar_wait(&full_c, (uint32_t)(cs - 1) & 1, p.timeout_ns)) && done;
            for (int c = max(0, xs - kStages); c < xs; ++c)
                done = mbar_wait(&full_x[c % kStages], (uint32_t)(c / kStages) & 1, p.timeout_ns) && done;
            if (!done) report_status(p.status, KDA_ERR_TIMEOUT);
            bulk_wait_all();
        }
        __syncwarp();
    } else if (warp == kIssueWarp) {
        // ------------------------------------------------------------ products
        // the whole warp, so that addresses stay in uniform registers; one thread issues
        const bool leader = elect_one();
        const uint32_t id_g = idesc_bf16_f32(128, 128, false, false);
        const uint32_t id_cs = idesc_bf16_f32(128, kCols, false, false);
        const uint32_t id_px = idesc_bf16_f32(128, P, false, true);
        const uint32_t id_up = idesc_bf16_f32(128, N, false, true);
        wait_for_launch_before();
        for (int c = 0; c < chunks; ++c) {
            const uint32_t par = c & 1;
            // products run in order: G takes the place that Q X of the chunk before has read
            if (!wait.warp(&full_c, par) || !wait.warp(&full_b, par)) break;
            tc_fence_after_sync();
            if (leader) {
                issue_ss<N>(tbase + TM_G, sb + OFF_C, sb + OFF_B, id_g);
                mma_commit(&bar_g);
            }
            __syncwarp();
            if (!wait.warp(&bar_state, par) || !wait.warp(&bar_w, par)) break;   // S decayed and as bf16; the weighted x
            tc_fence_after_sync();
            if (leader) {
                issue_ts(tbase + TM_S, tbase + TM_W, sb + OFF_B, id_up, true);
            }
            __syncwarp();
            if (c > 0 && !wait.warp(&bar_yfree, par ^ 1)) break;      // Y is free
            tc_fence_after_sync();
            if (leader) {
                issue_ss<N>(tbase + TM_Y, sb + OFF_C, sb + OFF_S, id_cs);
                mma_commit(&bar_cs);
                issue_ts(tbase + TM_S, tbase + TM_W + 64, sb + OFF_B, id_up, true);
                mma_commit(&bar_upd);
            }
            __syncwarp();
            if (!wait.warp(&bar_q, par)) break;                          // Q, and Y scaled
            tc_fence_after_sync();
            if (leader) {
#pragma unroll
                for (int i = 0; i < NH; ++i)
                    issue_ts(tbase + TM_Y + i * P, tbase + TM_G + 64 * i,
                             sb + OFF_X + (c % kStages) * kTile + (NH == 2 ? i * ATOM : 0), id_px, true);
                mma_commit(&bar_px);
            }
            __syncwarp();
        }
        if (leader) {
            mma_commit(&bar_drain);
            if (!mbar_wait(&bar_drain, 0, p.timeout_ns)) report_status(p.status, KDA_ERR_TIMEOUT);
        }
        __syncwarp();
    } else if (warp >= kDecayWarp) {
        // ------------------------------------------------------------ decays, up to two chunks ahead: a head to each warp, or
        // every other chunk
        const float rate0 = p.A[job.h0] * 1.4426950408889634f, rate1 = p.A[job.h1] * 1.4426950408889634f;   // powers of two
        const float bias0 = p.dt_bias ? p.dt_bias[job.h0] : 0.f, bias1 = p.dt_bias ? p.dt_bias[job.h1] : 0.f;
        const unsigned short* dt = reinterpret_cast<const unsigned short*>(p.dt) + job.start * p.lddt;
        unsigned short raw[4];                                           // token 32 k + lane; converted when used
        auto load_dt = [&](int n) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int t = n / NH * kTok + 32 * k + lane;
                raw[k] = t < job.len ? dt[t * p.lddt + (n % NH ? job.h1 : job.h0)] : (unsigned short)0;
            }
        };
        load_dt(warp - kDecayWarp);
        wait_for_launch_before();
        for (int n = warp - kDecayWarp; n < chunks * NH; n += 2) {
            const int c = n / NH, i = n % NH;
            const float rate = i ? rate1 : rate0, bias = i ? bias1 : bias0;
            float step[4], incl[4], after[4], total[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const bool in = c * kTok + 32 * k + lane < job.len;
                step[k] = in ? softplus(__bfloat162float(__ushort_as_bfloat16(raw[k])) + bias) : 0.f;
                // compared, so that a NaN stays one (fmaxf would drop it); past the last token nothing decays, at a
                // rate of -infinity too
                const float la = step[k] * rate;
                block_sums(in ? (la < kLeastDecay ? kLeastDecay : la) : 0.f, lane, incl[k], after[k]);
                total[k] = __shfl_sync(0xffffffffu, incl[k], 31);
            }
            load_dt(n + 2);
            if (c >= 2 && !wait.warp(&scal_free[c & 1], (uint32_t)(c / 2 - 1) & 1)) break;
            Scalars& sc = scal[c & 1];
            float behind = 0.f;                                          // the blocks after this one
#pragma unroll
            for (int k = 3; k >= 0; --k) {
                const int j = 32 * k + lane;
                sc.neg[i][j] = -incl[k];
                sc.step[i][j] = step[k];
                sc.col[i][j] = step[k] * ex2(after[k]);
                store_weight(sc, i, j, step[k] * ex2(after[k] + behind));
                behind += total[k];
                if (lane == 0) sc.total[i][k] = total[k];
            }
            warp_arrive(&bar_scal[c & 1], lane);
        }
    } else {
        // ------------------------------------------------------------ the arithmetic, by sixteen warps
        // A warp works on the tensor-memory lanes of its quarter; the four parts share the columns.  After a wait that
        // ran out it goes on to its end with whatever is there (the others count on it at the named barriers); nothing
        // is stored then.
        const int part = warp >> 2;
        const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
        const int r = 32 * quarter + lane;                               // value column of S^T, token of Y, G and Q
        const int half = NH == 2 ? quarter >> 1 : 0;                     // head of this warp's value columns of S^T
        const int yhead = NH == 2 ? part >> 1 : 0;                       // head of this warp's columns of Y
        const Column<N, P> col(p, job, r);
        const bool has_rows = 32 * part < N;                             // of S: 32 rows to a part
        wait_for_launch_before();
        if (has_rows) {
            float v[32];
            col.load_start(32 * part, v);
            if (chunks > 0) tmem_write32(tbase + TM_S + lanes + 32 * part, v);
            else if (p.ST) col.store(p.ST + col.s_off, 32 * part, v);    // an empty sequence
        }
        tmem_wait_st();
        const float skip0 = p.D ? p.D[job.h0] : 0.f, skip1 = p.D ? p.D[job.h1] : 0.f;
        // the chunk's weighted x, 32 tokens to a part
        auto weigh = [&](int c) {
            (void)wait.warp(&bar_scal[c & 1], (uint32_t)(c >> 1) & 1);
            (void)wait.warp(&full_x[c % kStages], (uint32_t)(c / kStages) & 1);
            const uint32_t x_off = OFF_X + (c % kStages) * kTile;
            const int n_valid = job.len - c * kTok;
            if (p.cu_seqlens && n_valid < kTok) {
                // rows of other sequences, or of none: zeros, so that nothing of theirs enters a sum
                (void)wait.warp(&full_b, c & 1);
                if (r >= n_valid && (part < 2 || part - 2 < N / 64)) {
                    uint8_t* row = sm + (part < 2 ? x_off + part * ATOM : OFF_B + (part - 2) * ATOM) + r * 128;
                    for (int i = 0; i < 8; ++i) *reinterpret_cast<uint4*>(row + i * 16) = make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                }
                named_bar_sync(3, 32 * kWorkers);
            }
            tc_fence_after_sync();
            weigh_x(tbase + lanes + TM_W, scal[c & 1], half, sb + x_off, quarter, lane, 4 * part);
            tmem_wait_st();
            tc_fence_before_sync();
            warp_arrive(&bar_w, lane);
        };
        // S: its bf16 copy for the chunk's read-out, then decayed to the chunk's end for the update
        auto carry = [&](int c) {
            const Scalars& sc = scal[c & 1];
            if (has_rows) {
                const float decay = ex2((sc.total[half][0] + sc.total[half][1]) + (sc.total[half][2] + sc.total[half][3]));
                float v[32];
                const uint32_t ta = tbase + TM_S + lanes + 32 * part;
                tmem_read32(ta, v);
#pragma unroll
                for (int i = 0; i < 32; i += 8)
                    *reinterpret_cast<uint4*>(sm + OFF_S + sw128_offset(r, 32 * part + i, ATOM)) =
                        make_uint4(bf16x2(v[i], v[i + 1]), bf16x2(v[i + 2], v[i + 3]), bf16x2(v[i + 4], v[i + 5]),
                                   bf16x2(v[i + 6], v[i + 7]));
                scale_by<32>(v, decay);
                tmem_write32(ta, v);
                tmem_wait_st();
                fence_proxy_async_smem();
            }
            tc_fence_before_sync();
            if (!(p.skip_handoff && c == 0)) warp_arrive(&bar_state, lane);
        };
        if (chunks > 0) {
            weigh(0);
            carry(0);
        }
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
            const uint32_t par = c & 1;
            const Scalars& sc = scal[c & 1];
            // Q: the decayed lower triangle of G, columns 8 part .. 8 part + 7 of each block of 32
            (void)wait.warp(&bar_g, par);
            tc_fence_after_sync();
            {
                float gv[32];
                tmem_read4x8(tbase + TM_G + lanes + 8 * part, gv);
                tc_fence_before_sync();
                named_bar_sync(4 + quarter, 128);                        // all of these lanes' G is read: Q takes its place
                tc_fence_after_sync();
#pragma unroll 1
                for (int i = 0; i < NH; ++i) {
                    const uint32_t qt = tbase + TM_G + 64 * i + lanes + 4 * part;
                    const float lr = -sc.neg[i][r];
                    float e = lr;                                        // sum over the tokens after block b up to r
#pragma unroll
                    for (int b = 3; b >= 0; --b) {
                        const float* gb = gv + 8 * b;
                        const int j0 = 32 * b + 8 * part;
                        uint32_t q[4] = {0u, 0u, 0u, 0u};
                        if (b < quarter) {
                            const float ee = ex2(e);
                            const uint64_t e2 = pair2(ee, ee);
                            e += sc.total[i][b];
#pragma unroll
                            for (int k = 0; k < 8; k += 4) {
                                const float4 f = *reinterpret_cast<const float4*>(&sc.col[i][j0 + k]);
                                q[k / 2] = mul2_bf16x2(pair2(gb[k], gb[k + 1]), mul2(e2, pair2(f.x, f.y)));
                                q[k / 2 + 1] = mul2_bf16x2(pair2(gb[k + 2], gb[k + 3]), mul2(e2, pair2(f.z, f.w)));
                            }
                        } else if (b == quarter) {
                            const float skip = i ? skip1 : skip0;
                            const int dr = lane - 8 * part;              // the column of the diagonal element
#pragma unroll
                            for (int k = 0; k < 8; k += 4) {
                                const float4 l = *reinterpret_cast<const float4*>(&sc.neg[i][j0 + k]);
                                const float4 st = *reinterpret_cast<const float4*>(&sc.step[i][j0 + k]);
                                const float lj[4] = {l.x, l.y, l.z, l.w}, sj[4] = {st.x, st.y, st.z, st.w};
                                float v[4];
#pragma unroll
                                for (int d = 0; d < 4; ++d) {
                                    const float m = gb[k + d] * (ex2(lr + lj[d]) * sj[d]);
                                    v[d] = k + d < dr ? m : k + d == dr ? m + skip : 0.f;
                                }
                                q[k / 2] = bf16x2(v[0], v[1]);
                                q[k / 2 + 1] = bf16x2(v[2], v[3]);
                            }
                        }
                        tmem_st4(qt + 16 * b, q);
                    }
                }
            }
            // Y = C S: row r by 2^{L_r}, 32 columns to a part
            const uint32_t yt = tbase + TM_Y + lanes + 32 * part;
            {
                float sum = -sc.neg[yhead][r];
                for (int b = 0; b < quarter; ++b) sum += sc.total[yhead][b];
                const float row = ex2(sum);
                (void)wait.warp(&bar_cs, par);
                tc_fence_after_sync();
                float v[32];
                tmem_read32(yt, v);
                scale_by<32>(v, row);
                tmem_write32(yt, v);
            }
            tmem_wait_st();
            tc_fence_before_sync();
            warp_arrive(&bar_q, lane);
            warp_arrive(&scal_free[c & 1], lane);                        // the chunk's decays are used up

            // while Q X runs: the next chunk's weighted x and carried state
            if (c + 1 < chunks) {
                (void)wait.warp(&bar_upd, par);                          // the operand's place is free
                weigh(c + 1);
                carry(c + 1);
            }
            // Y, finished: into the chunk's own x tile (all its readers are done), from where it is stored in whole lines
            const bool ok = wait.warp(&bar_px, par);
            tc_fence_after_sync();
            {
                float v[32];
                tmem_read32(yt, v);
                tc_fence_before_sync();                                  // the next C S overwrites Y
                warp_arrive(&bar_yfree, lane);
                const bool whole = !p.cu_seqlens || job.len - c * kTok >= kTok;
                uint8_t* tile = sm + OFF_X + (c % kStages) * kTile;
                const int t = c * kTok + r;
                // heads h0 and h0 + 1 are neighbours in y; a head carried twice is stored once
                const bool mine = ok && t < job.len && !(NH == 2 && part >= 2 && job.h1 == job.h0);
                __nv_bfloat16* yr = p.y + ((job.start + t) * p.H + job.h0) * P + 32 * part;
#pragma unroll
                for (int i = 0; i < 32; i += 8) {
                    const uint4 o = make_uint4(bf16x2(v[i], v[i + 1]), bf16x2(v[i + 2], v[i + 3]), bf16x2(v[i + 4], v[i + 5]),
                                               bf16x2(v[i + 6], v[i + 7]));
                    if (whole) *reinterpret_cast<uint4*>(tile + sw128_offset(r, 32 * part + i, ATOM)) = o;
                    else if (mine) *reinterpret_cast<uint4*>(yr + i) = o;        // rows past a packed sequence stay
                }
            }
            fence_proxy_async_smem();
            warp_arrive(&bar_staged[par], lane);
        }
        // the state after the sequence's last token
        if (chunks > 0 && job.last && p.ST && wait.warp(&bar_upd, (uint32_t)(chunks - 1) & 1) && has_rows && !abort_s) {
            tc_fence_after_sync();
            float v[32];
            tmem_read32(tbase + TM_S + lanes + 32 * part, v);
            col.store(p.ST + col.s_off, 32 * part, v);
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 0) tmem_dealloc(tmem_base_s, TM_COLS);
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

// Shared memory above the default limit, asked for once per kernel and device.
template <int N, int P, bool STATE>
struct AllowSmem {
    static cudaError_t once() {
        static std::mutex mu;
        static bool set[64] = {false};
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        std::lock_guard<std::mutex> lock(mu);
        if (dev < 64 && set[dev]) return cudaSuccess;
        constexpr auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
        if constexpr (STATE) e = cudaFuncSetAttribute(kda_ssm_state_kernel<N, P>, attr, SMEM_DYN);
        else e = cudaFuncSetAttribute(kda_ssm_tc_kernel<N, P>, attr, SMEM_DYN);
        if (e == cudaSuccess && dev < 64) set[dev] = true;
        return e;
    }
};

template <int N, int P>
cudaError_t launch_np(const CUtensorMap& mx, const CUtensorMap& mb, const CUtensorMap& mc, const CUtensorMap& my,
                      const Params& p, long long units, cudaStream_t s) {
    const long long grid = units * p.tiles;
    if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    if (p.seg_chunks > 0) {
        const cudaError_t e = AllowSmem<N, P, true>::once();
        if (e != cudaSuccess) return e;
        kda_ssm_state_kernel<N, P><<<(unsigned)grid, kStateThreads, SMEM_DYN, s>>>(mx, mb, p);
        const cudaError_t err = cudaGetLastError();
        if (err != cudaSuccess) return err;
    }
    const cudaError_t e = AllowSmem<N, P, false>::once();
    if (e != cudaSuccess) return e;
    Params last = p;
    if (p.seg_chunks > 0) last.skip_handoff = 0;                          // the first launch has left out one
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = SMEM_DYN;
    cfg.stream = s;
    cfg.attrs = &early;
    cfg.numAttrs = p.seg_chunks > 0 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kda_ssm_tc_kernel<N, P>, mx, mb, mc, my, last);
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
    if (a.T == 0) return launch_ssm_simt(a, s);      // packed sequences without tokens: the offsets' check and S_T = S0
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
