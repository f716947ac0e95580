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
// each term of y.  The state itself is fp32 and stays accurate to 2^-16 of each term: B and x are exact
// bf16 operands and the weighted x enters as the sum of two bf16 values, hi and lo.
//
// What bounds it: HBM moves 64 KB of x and y per chunk of a 128-column tile (2.8K cycles at the
// measured copy rate), the tensor core needs 2.5K cycles, and its operands with the tiles' own traffic
// about 3.7K cycles of shared memory, so operands are kept out of shared memory where a product allows:
// Q and the weighted x are tensor-memory operands, and the state is held transposed (lanes = value
// columns) for that.
//
// Warps (18): 0-3 state and outputs, 4-7 decays and weighted x, 8-15 Q, 16 products, 17 loads.
// Tensor memory (512 columns): S^T, Y, G (then Q in its place), weighted x hi and lo.
// Order of the products: Y = C S | S += hi | Y += Q X | S += lo | next G.  The scaling of Y runs under
// the hi part, Y's store under the lo part, the state's conversion under the next G.
//
// Long prompts with few heads: the tokens are cut into segments.  A first launch runs the state update
// alone (B and x only) on every segment but the last, the first one from S0, the others from zero; the
// second starts each segment from the segments before it, S <- 2^{total} S + local, folded in as it loads
// its start state.
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
constexpr int kStages = 2;
constexpr int kThreads = 576;
constexpr int kStateWarps = 4, kDecayWarps = 4, kScoreWarps = 8;
constexpr int kFirstDecay = kStateWarps, kFirstScore = kFirstDecay + kDecayWarps;
constexpr int kIssueWarp = kFirstScore + kScoreWarps, kLoadWarp = kIssueWarp + 1;
constexpr uint32_t ATOM = 16384;             // [128 rows][64 columns] bf16, 128-byte swizzle
constexpr uint32_t kTile = 2 * ATOM;

// shared memory: per stage B, X; one C (free again after a chunk's second product); S as bf16 (rows = value
// columns, K = N)
constexpr uint32_t OFF_B = 0, OFF_X = kTile, kStageBytes = 2 * kTile;
constexpr uint32_t OFF_C = kStages * kStageBytes, OFF_S = OFF_C + kTile;
constexpr uint32_t SMEM_DYN = OFF_S + kTile + 1024;

// tensor memory columns
constexpr uint32_t TM_S = 0, TM_Y = 128, TM_G = 256, TM_HI = 384, TM_LO = 448, TM_COLS = 512;

struct Scalars {                             // of one chunk, per head of the tile
    float L[2][kTok];                        // running sum within the token's 32-token block, inclusive
    float col[2][kTok];                      // s_j 2^{block end - L_j}
    float step[2][kTok];                     // s_j
    float w[2][kTok];                        // s_j 2^{chunk end - L_j}
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
// A: 128 tokens of K in 64 packed columns; B: MN-major tile whose K axis is the tokens
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
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* u) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
                 "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
                 : "memory");
}

// TMEM -> registers, 32 columns, complete on return.  Load and wait are one statement: between two, the
// compiler may move or spill registers that the load has not written yet.
__device__ __forceinline__ void tmem_read32(uint32_t taddr, float* r) {
    uint32_t* u = reinterpret_cast<uint32_t*>(r);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]),
          "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]),
          "=r"(u[16]), "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]),
          "=r"(u[24]), "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
        : "r"(taddr)
        : "memory");
}
// Four runs of 16 columns, 32 apart.
__device__ __forceinline__ void tmem_read4x16(uint32_t taddr, float* r) {
    uint32_t* u = reinterpret_cast<uint32_t*>(r);
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
          "=&r"(u[48]), "=&r"(u[49]), "=&r"(u[50]), "=&r"(u[51]), "=&r"(u[52]), "=&r"(u[53]), "=&r"(u[54]), "=&r"(u[55]),
          "=&r"(u[56]), "=&r"(u[57]), "=&r"(u[58]), "=&r"(u[59]), "=&r"(u[60]), "=&r"(u[61]), "=&r"(u[62]), "=&r"(u[63])
        : "r"(taddr), "r"(taddr + 32), "r"(taddr + 64), "r"(taddr + 96)
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
                  const __grid_constant__ CUtensorMap tm_c, const Params p) {
    constexpr int NH = P == 64 ? 2 : 1;      // heads per tile
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_base = smem_u32(smem_raw);
    uint8_t* sm = smem_raw + (((raw_base + 1023u) & ~1023u) - raw_base);
    const uint32_t sb = smem_u32(sm);
    __shared__ Scalars scal[2];
    __shared__ uint64_t full[kStages], empty[kStages], full_c, bar_scal[2], bar_g, bar_cs, bar_upd, bar_px, bar_state, bar_scaled,
        bar_w, bar_q, bar_drain;
    __shared__ uint32_t tmem_base_s;
    __shared__ volatile int abort_s;
    __shared__ int seq_s, seg_s;
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
        for (int i = 0; i < kStages; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], 1); }
        for (int i = 0; i < 2; ++i) mbar_init(&bar_scal[i], kDecayWarps);
        mbar_init(&full_c, 1);
        mbar_init(&bar_g, 1);
        mbar_init(&bar_cs, 1);
        mbar_init(&bar_upd, 1);
        mbar_init(&bar_px, 1);
        mbar_init(&bar_state, kStateWarps);
        mbar_init(&bar_scaled, kStateWarps);
        mbar_init(&bar_w, kDecayWarps);
        mbar_init(&bar_q, kScoreWarps);
        mbar_init(&bar_drain, 1);
        fence_mbar_init();
        abort_s = 0;
        prefetch_tensormap(&tm_x); prefetch_tensormap(&tm_b); prefetch_tensormap(&tm_c);
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

    if (warp == kLoadWarp) {
        // ------------------------------------------------------------ loads
        if (lane == 0) {
            int issued = 0, issued_c = 0;
            for (int c = 0; c < chunks; ++c) {
                const int st = c % kStages;
                if (c >= kStages && !wait.one(&empty[st], (uint32_t)(c / kStages - 1) & 1)) break;
                uint8_t* s = sm + st * kStageBytes;
                const int t = row0 + c * kTok, na = N / 64;
                mbar_arrive_expect_tx(&full[st], ATOM * (2 + na));
                for (int i = 0; i < na; ++i) tma_load_4d(s + OFF_B + i * ATOM, &tm_b, &full[st], 64 * i, g, t, row_seq);
                for (int i = 0; i < 2; ++i)
                    tma_load_4d(s + OFF_X + i * ATOM, &tm_x, &full[st], NH == 2 ? 0 : 64 * i, NH == 2 && i ? h1 : h0, t, row_seq);
                ++issued;
                if (STATE_ONLY) continue;
                if (c > 0 && !wait.one(&bar_cs, (uint32_t)(c - 1) & 1)) break;
                mbar_arrive_expect_tx(&full_c, ATOM * na);
                for (int i = 0; i < na; ++i) tma_load_4d(sm + OFF_C + i * ATOM, &tm_c, &full_c, 64 * i, g, t, row_seq);
                ++issued_c;
            }
            // nothing may be in flight when the CTA exits (a load that never lands ends the wait by its limit)
            for (int c = max(0, issued - kStages); c < issued; ++c)
                if (!mbar_wait(&full[c % kStages], (uint32_t)(c / kStages) & 1, p.timeout_ns))
                    report_status(p.status, KDA_ERR_TIMEOUT);
            if (issued_c > 0 && !mbar_wait(&full_c, (uint32_t)(issued_c - 1) & 1, p.timeout_ns))
                report_status(p.status, KDA_ERR_TIMEOUT);
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
            for (int c = 0; c < chunks && ok; ++c) {
                const uint32_t s = sb + (c % kStages) * kStageBytes, par = c & 1;
                ok = wait.one(&bar_state, par);          // S as bf16 and decayed, Y free
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
                    ok = wait.one(&bar_scaled, par) && wait.one(&bar_q, par);
                    if (!ok) break;
                    tc_fence_after_sync();
#pragma unroll
                    for (int i = 0; i < NH; ++i)
                        issue_ts(tbase + TM_Y + i * P, tbase + TM_G + 64 * i, s + OFF_X + (NH == 2 ? i * ATOM : 0), id_px, true);
                    mma_commit(&bar_px);
                }
                issue_ts(tbase + TM_S, tbase + TM_LO, s + OFF_B, id_up, true);
                mma_commit(&bar_upd);
                mma_commit(&empty[c % kStages]);
                if (!STATE_ONLY && c + 1 < chunks) ok = issue_g(c + 1);
            }
            mma_commit(&bar_drain);
            if (!mbar_wait(&bar_drain, 0, p.timeout_ns)) report_status(p.status, KDA_ERR_TIMEOUT);
        }
    } else if (warp < kStateWarps) {
        // ------------------------------------------------------------ state and outputs
        const int col = 32 * warp + lane;                                // value column of this lane
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
                for (int k = 1; k < seg; ++k) {
                    const float d = ex2(p.seg_decay[(size_t)(unit0 + k) * H + head]);
                    const float* l = seg_state(unit0 + k);
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = fmaf(d, v[i], l[(size_t)(n0 + i) * P]);
                }
            }
        };
        bool ok = true;
        for (int c = 0; c < chunks && ok; ++c) {
            const uint32_t par = c & 1;
            const Scalars& sc = scal[c & 1];
            ok = wait.warp(&bar_scal[c & 1], (c >> 1) & 1) && (c == 0 || wait.warp(&bar_upd, par ^ 1));
            if (!ok) break;
            tc_fence_after_sync();
            const float decay = ex2((sc.total[half][0] + sc.total[half][1]) + (sc.total[half][2] + sc.total[half][3]));
            // S: its bf16 copy for this chunk's read-out, then decayed to the chunk's end for the update
            for (int n0 = 0; n0 < N; n0 += 32) {
                float v[32];
                const uint32_t ta = tbase + TM_S + lanes + n0;
                if (c == 0) {
                    load_start(n0, v);
                } else {
                    tmem_read32(ta, v);
                }
                if (!STATE_ONLY) {
#pragma unroll
                    for (int i = 0; i < 32; i += 8)
                        *reinterpret_cast<uint4*>(sm + OFF_S + sw128_offset(col, n0 + i, ATOM)) =
                            make_uint4(bf16x2(v[i], v[i + 1]), bf16x2(v[i + 2], v[i + 3]), bf16x2(v[i + 4], v[i + 5]),
                                       bf16x2(v[i + 6], v[i + 7]));
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] *= decay;
                tmem_st16(ta, v);
                tmem_st16(ta + 16, v + 16);
            }
            tmem_wait_st();
            fence_proxy_async_smem();
            tc_fence_before_sync();
            if (!(p.skip_handoff && c == 0)) warp_arrive(&bar_state, lane);
            if (STATE_ONLY) continue;
            // Y = C S: row r by 2^{L_r}.  Here a lane is a token.
            const int r = 32 * warp + lane;
            float row[NH];
#pragma unroll
            for (int i = 0; i < NH; ++i) {
                float before = 0.f;
                for (int b = 0; b < quarter; ++b) before += sc.total[i][b];
                row[i] = ex2(sc.L[i][r] + before);
            }
            ok = wait.warp(&bar_cs, par);
            if (!ok) break;
            tc_fence_after_sync();
#pragma unroll
            for (int cb = 0; cb < kCols; cb += 32) {
                float v[32];
                const uint32_t ta = tbase + TM_Y + lanes + cb;
                const float e = row[NH == 2 ? cb >> 6 : 0];
                tmem_read32(ta, v);
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] *= e;
                tmem_st16(ta, v);
                tmem_st16(ta + 16, v + 16);
            }
            tmem_wait_st();
            tc_fence_before_sync();
            warp_arrive(&bar_scaled, lane);
            ok = wait.warp(&bar_px, par);
            if (!ok) break;
            tc_fence_after_sync();
            const int t = tok0 + c * kTok + r;
            __nv_bfloat16* yr = p.y + ((start + t) * H + h0) * P;        // heads h0 and h0 + 1 are neighbours
#pragma unroll
            for (int cb = 0; cb < kCols; cb += 32) {
                float v[32];
                const uint32_t ta = tbase + TM_Y + lanes + cb;
                tmem_read32(ta, v);
                if (t < len_seq && t < tok0 + len && !(NH == 2 && cb >= 64 && h1 == h0)) {
#pragma unroll
                    for (int i = 0; i < 32; i += 8)
                        *reinterpret_cast<uint4*>(yr + cb + i) =
                            make_uint4(bf16x2(v[i], v[i + 1]), bf16x2(v[i + 2], v[i + 3]), bf16x2(v[i + 4], v[i + 5]),
                                       bf16x2(v[i + 6], v[i + 7]));
                }
            }
            tc_fence_before_sync();                                      // the next C S overwrites Y
        }
        // the state after the last token (of the sequence; of the segment in the first launch)
        if (ok && (STATE_ONLY || (last_seg && p.ST))) {
            if (chunks > 0) ok = wait.warp(&bar_upd, (chunks - 1) & 1);
            tc_fence_after_sync();
            for (int n0 = 0; n0 < N && ok; n0 += 32) {
                float v[32];
                if (chunks > 0) {
                    tmem_read32(tbase + TM_S + lanes + n0, v);
                } else {
                    load_start(n0, v);
                }
                store_state(STATE_ONLY ? seg_state(unit) : p.ST + s_off, n0, v);
            }
        }
    } else if (warp < kFirstScore) {
        // ------------------------------------------------------------ decays and weighted x
        const int dw = warp - kFirstDecay;
        const int j = 32 * dw + lane;                                    // a token here
        const int m = j;                                                 // a value column below
        float rate[NH], bias[NH], raw[NH], total_all[NH];
#pragma unroll
        for (int i = 0; i < NH; ++i) {
            const int head = i ? h1 : h0;
            rate[i] = p.A[head] * 1.4426950408889634f;                   // decays in powers of two
            bias[i] = p.dt_bias ? p.dt_bias[head] : 0.f;
            total_all[i] = 0.f;
        }
        auto load_dt = [&](int c) {
            const int t = c * kTok + j;
#pragma unroll
            for (int i = 0; i < NH; ++i)
                raw[i] = t < len ? load_elem(p.dt, (start + tok0 + t) * p.lddt + (i ? h1 : h0)) : 0.f;
        };
        load_dt(0);
        bool ok = true;
        for (int c = 0; c < chunks; ++c) {
            Scalars& sc = scal[c & 1];
            const int n_valid = min(kTok, len - c * kTok);
            float sfx[NH], stp[NH];
#pragma unroll
            for (int i = 0; i < NH; ++i) {
                stp[i] = j < n_valid ? softplus(raw[i] + bias[i]) : 0.f;
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
                sc.L[i][j] = incl;
                sc.step[i][j] = stp[i];
                sc.col[i][j] = stp[i] * ex2(sfx[i]);
                if (lane == 31) sc.total[i][dw] = incl;
            }
            if (c + 1 < chunks) load_dt(c + 1);
            named_bar_sync(1, 32 * kDecayWarps);
#pragma unroll
            for (int i = 0; i < NH; ++i) {
                float after = 0.f, all = 0.f;
#pragma unroll
                for (int b = 3; b >= 0; --b) {
                    if (b > dw) after += sc.total[i][b];
                    all += sc.total[i][b];
                }
                sc.w[i][j] = stp[i] * ex2(sfx[i] + after);
                total_all[i] += all;
            }
            warp_arrive(&bar_scal[c & 1], lane);
            ok = wait.warp(&full[c % kStages], (uint32_t)(c / kStages) & 1);
            uint8_t* s = sm + (c % kStages) * kStageBytes;
            if (ok && p.cu_seqlens && j >= n_valid) {
                // rows of other sequences, or of none: zeros, so that nothing of theirs enters a sum
                const uint4 zero = make_uint4(0, 0, 0, 0);
                for (int i = 0; i < 8; ++i) {
                    for (int a = 0; a < 2; ++a) *reinterpret_cast<uint4*>(s + OFF_X + a * ATOM + j * 128 + i * 16) = zero;
                    for (int a = 0; a < N / 64; ++a) *reinterpret_cast<uint4*>(s + OFF_B + a * ATOM + j * 128 + i * 16) = zero;
                }
                fence_proxy_async_smem();
            }
            if (ok && c > 0) ok = wait.warp(&bar_upd, (uint32_t)(c - 1) & 1);   // the operand's space is free
            // w and the zeros of all tokens; all four warps leave together
            ok = named_bar_and(2, 32 * kDecayWarps, ok);
            if (!ok) break;
            tc_fence_after_sync();
            const float* wv = sc.w[NH == 2 ? m >> 6 : 0];
            const uint8_t* xt = s + OFF_X + (m >> 6) * ATOM + (m & 7) * 2;
            const uint32_t chunk16 = (m & 63) >> 3;
#pragma unroll 2
            for (int t0 = 0; t0 < kTok; t0 += 16) {
                uint32_t hi[8], lo[8];
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const float4 w4 = *reinterpret_cast<const float4*>(wv + t0 + i);
                    const float w[4] = {w4.x, w4.y, w4.z, w4.w};
                    float v[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int t = t0 + i + k;
                        const uint32_t u = *reinterpret_cast<const uint16_t*>(xt + t * 128 + ((chunk16 ^ (t & 7)) << 4));
                        v[k] = __uint_as_float(u << 16) * w[k];
                    }
#pragma unroll
                    for (int k = 0; k < 4; k += 2) {
                        const uint32_t h2 = bf16x2(v[k], v[k + 1]);
                        hi[(i + k) / 2] = h2;
                        lo[(i + k) / 2] = bf16x2(v[k] - __uint_as_float(h2 << 16), v[k + 1] - __uint_as_float(h2 & 0xffff0000u));
                    }
                }
                tmem_st8(tbase + TM_HI + lanes + t0 / 2, hi);
                tmem_st8(tbase + TM_LO + lanes + t0 / 2, lo);
            }
            tmem_wait_st();
            tc_fence_before_sync();
            warp_arrive(&bar_w, lane);
        }
        if (STATE_ONLY && ok && j == 0) {
            p.seg_decay[(size_t)unit * H + h0] = total_all[0];
            if (NH == 2 && h1 != h0) p.seg_decay[(size_t)unit * H + h1] = total_all[NH - 1];
        }
    } else if (!STATE_ONLY) {
        // ------------------------------------------------------------ Q: the decayed lower triangle of G
        const int which = (warp - kFirstScore) >> 2;                     // 16 columns of each 32-column block
        const int r = 32 * quarter + lane;
        float skip[NH];
#pragma unroll
        for (int i = 0; i < NH; ++i) skip[i] = p.D ? p.D[i ? h1 : h0] : 0.f;
        bool ok = true;
        for (int c = 0; c < chunks; ++c) {
            const uint32_t par = c & 1;
            const Scalars& sc = scal[c & 1];
            ok = wait.warp(&bar_scal[c & 1], (c >> 1) & 1) && wait.warp(&bar_g, par);
            tc_fence_after_sync();
            float gv[4][16];
            tmem_read4x16(tbase + TM_G + lanes + 16 * which, &gv[0][0]);
            tc_fence_before_sync();
            // both warps of these lanes have read G (Q takes its place)
            ok = named_bar_and(3 + quarter, 64, ok);
            if (!ok) break;
            tc_fence_after_sync();
#pragma unroll
            for (int i = 0; i < NH; ++i) {
                const float lr = sc.L[i][r];
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    uint32_t q[8];
                    const int j0 = 32 * b + 16 * which;
                    if (b > quarter) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) q[k] = 0u;
                    } else if (b < quarter) {
                        float e = lr;
                        for (int k = b + 1; k < quarter; ++k) e += sc.total[i][k];
                        e = ex2(e);
#pragma unroll
                        for (int k = 0; k < 16; k += 4) {
                            const float4 f = *reinterpret_cast<const float4*>(&sc.col[i][j0 + k]);
                            q[k / 2] = bf16x2(gv[b][k] * (e * f.x), gv[b][k + 1] * (e * f.y));
                            q[k / 2 + 1] = bf16x2(gv[b][k + 2] * (e * f.z), gv[b][k + 3] * (e * f.w));
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < 16; k += 4) {
                            const float4 l = *reinterpret_cast<const float4*>(&sc.L[i][j0 + k]);
                            const float4 s = *reinterpret_cast<const float4*>(&sc.step[i][j0 + k]);
                            const float lj[4] = {l.x, l.y, l.z, l.w}, sj[4] = {s.x, s.y, s.z, s.w};
                            float v[4];
#pragma unroll
                            for (int d = 0; d < 4; ++d) {
                                const int j = j0 + k + d;
                                v[d] = j <= r ? gv[b][k + d] * (ex2(lr - lj[d]) * sj[d]) : 0.f;
                                if (j == r) v[d] += skip[i];
                            }
                            q[k / 2] = bf16x2(v[0], v[1]);
                            q[k / 2 + 1] = bf16x2(v[2], v[3]);
                        }
                    }
                    tmem_st8(tbase + TM_G + 64 * i + lanes + j0 / 2, q);
                }
            }
            tmem_wait_st();
            tc_fence_before_sync();
            warp_arrive(&bar_q, lane);
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

// Chunks per segment (0: sequences are not cut).
int segment_chunks(int, long long, int) { return 0; }

long long units_of(int n_seq, long long T_total, bool packed, int T, int seg_chunks) {
    if (seg_chunks == 0) return n_seq;
    const long long tok = (long long)seg_chunks * kTok;
    return packed ? n_seq + T_total / tok : (long long)n_seq * ((T + tok - 1) / tok);
}

template <int N, int P, bool STATE_ONLY>
cudaError_t launch_one(const CUtensorMap& mx, const CUtensorMap& mb, const CUtensorMap& mc, const Params& p,
                       long long units, cudaStream_t s) {
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
    kda_ssm_tc_kernel<N, P, STATE_ONLY><<<(unsigned)grid, kThreads, SMEM_DYN, s>>>(mx, mb, mc, p);
    return cudaGetLastError();
}

template <int N, int P>
cudaError_t launch_np(const CUtensorMap& mx, const CUtensorMap& mb, const CUtensorMap& mc, const Params& p,
                     long long units, cudaStream_t s) {
    if (p.seg_chunks > 0) {
        const cudaError_t e = launch_one<N, P, true>(mx, mb, mc, p, units, s);
        if (e != cudaSuccess) return e;
    }
    return launch_one<N, P, false>(mx, mb, mc, p, units, s);
}

}  // namespace

bool ssm_tc_supports(const SsmArgs& a) { return a.dtype == KDA_DTYPE_BF16; }

cudaError_t launch_ssm_tc(const SsmArgs& a, cudaStream_t s) {
    const int B = a.cu_seqlens ? 1 : a.n_seq;
    if (a.T == 0) {
        // packed sequences without tokens: S_T = S0
        if (!a.ST || a.ST == a.S0) return cudaSuccess;
        const size_t bytes = (size_t)a.n_seq * a.H * a.N * a.P * sizeof(float);
        return a.S0 ? cudaMemcpyAsync(a.ST, a.S0, bytes, cudaMemcpyDeviceToDevice, s) : cudaMemsetAsync(a.ST, 0, bytes, s);
    }
    CUtensorMap mx, mb, mc;
    if (!make_map(&mx, a.x, B, a.T, a.H, a.P, a.ldx) || !make_map(&mb, a.Bm, B, a.T, a.G, a.N, a.ldb) ||
        !make_map(&mc, a.Cm, B, a.T, a.G, a.N, a.ldc))
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
    p.seg_chunks = segment_chunks(a.n_seq, T_total, p.tiles);
    const long long units = units_of(a.n_seq, T_total, a.cu_seqlens != nullptr, a.T, p.seg_chunks);
    p.segs = p.seg_chunks > 0 && !a.cu_seqlens ? (int)(units / a.n_seq) : 1;
    p.seg_state = static_cast<float*>(a.workspace);
    p.seg_decay = p.seg_state ? p.seg_state + (size_t)units * a.H * a.N * a.P : nullptr;
    p.status = a.status;
    p.timeout_ns = a.timeout_ns;
    p.skip_handoff = a.skip_handoff;
    if (a.N == 128) return a.P == 128 ? launch_np<128, 128>(mx, mb, mc, p, units, s) : launch_np<128, 64>(mx, mb, mc, p, units, s);
    return a.P == 128 ? launch_np<64, 128>(mx, mb, mc, p, units, s) : launch_np<64, 64>(mx, mb, mc, p, units, s);
}

}  // namespace kda
