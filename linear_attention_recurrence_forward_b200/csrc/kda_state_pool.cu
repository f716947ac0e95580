// Slots of state pools copied, cleared and compacted, all pools of a call in one launch.
//
// Bound by HBM: each moved byte is read and written once.  A launch carries the descriptions of up to
// kPools pools in its parameters, so a model's layers go together (a 2 MB slot is 64 blocks' worth of
// work: one layer alone would not fill the GPU).  The work is a flat list of (pool, 32 KB part of a
// slot, pair); a fixed grid of blocks walks it, each part as eight 16-byte loads per thread before the
// first store.  One B200: compacting 192 slots of 256 in eight layers' scan and convolution pools takes
// 353 to 392 us for 2.2 GB (0.87 to 0.96 of the measured copy rate, by which slots move); eight forks of
// one slot in four layers 17 us, as long as the host takes for the call (78 MB: 12 us).
//
// A pair whose destination another pair has too, or (same pool) another pair reads, is left out and
// reported, so no two blocks ever write one slot and none reads a slot that is written.  All blocks come to
// the same verdict.  Up to kFew pairs, a block compares a pair with the whole list where it uses it.  Longer
// lists go in pages of kPage pairs: a block hashes a page's destinations into shared memory and marks them in
// one pass over the list; blocks share the pages out among them.  With slots of 256 bytes, pair by pair
// against by pages: 1025 pairs in one pool 8.4 and 12.5 us, in eight 35 and 31 us; 4096 pairs in sixteen 433
// and 192 us; 65536 pairs in one 6.3 and 0.5 ms, in sixteen 102 and 3.2 ms.
#include "kda_serving.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 8;                               // 16-byte vectors per thread and part
constexpr int kPart = kThreads * kVecs * 16;           // bytes of a part
constexpr int kPools = 40;                             // pools per launch (parameters stay under 4 KB)
constexpr int kMaxBlocks = 148 * 8;

struct PoolPair {
    uint8_t* dst;
    const uint8_t* src;
    long long dst_slot, src_slot, dst_piece, src_piece, piece_bytes;
    long long first;           // first work item of this pool
    int parts;                 // parts per piece
    int pieces;
};
struct PoolBatch {
    PoolPair p[kPools];
    int n;
};

// The work items of a batch when `m` pairs are to be copied: item = ((pool) * m + pair) * parts + part.
__device__ __forceinline__ int pool_of(const PoolBatch& pb, long long per_pair_item) {
    int k = 0;
    while (k + 1 < pb.n && per_pair_item >= pb.p[k + 1].first) ++k;
    return k;
}

// One part of one slot: dst[to] = src[from], or zeros when src is null.
__device__ __forceinline__ void move_part(const PoolPair& p, long long from, long long to, int part) {
    const int piece = part / p.parts;
    const long long off = (long long)(part % p.parts) * kPart;
    const int n = (int)(min((long long)kPart, p.piece_bytes - off) >> 4);
    uint4* d = reinterpret_cast<uint4*>(p.dst + to * p.dst_slot + piece * p.dst_piece + off);
    const uint4* s = reinterpret_cast<const uint4*>(p.src + from * p.src_slot + piece * p.src_piece + off);
    uint4 v[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int k = (int)threadIdx.x + i * kThreads;
        v[i] = make_uint4(0, 0, 0, 0);
        if (p.src && k < n) v[i] = s[k];
    }
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int k = (int)threadIdx.x + i * kThreads;
        if (k < n) d[k] = v[i];
    }
}

// Whether pair i may be copied (block-wide; every thread gets the answer).
__device__ __forceinline__ bool pair_valid(const int* src, const int* dst, int n, int i, int n_src, int n_dst,
                                           bool same) {
    const int s = src[i], d = dst[i];
    bool ok = s < n_src && d < n_dst;
    for (int j = threadIdx.x; j < n; j += kThreads) {
        if (j == i) continue;
        const int sj = src[j], dj = dst[j];
        if (sj < 0 || dj < 0) continue;                  // a skipped pair
        ok = ok && dj != d && !(same && sj == d && s != d);
    }
    return __syncthreads_and(ok) != 0;
}

// same: bit k set where pool k's source and destination are one pool
__global__ void __launch_bounds__(kThreads)
kda_pool_copy_kernel(const __grid_constant__ PoolBatch pb, const int* __restrict__ src, const int* __restrict__ dst,
                     int n, int n_src, int n_dst, unsigned long long same, long long parts_all, int* status) {
    int checked = -1, checked_pool = -1;
    bool ok = false;
    for (long long w = blockIdx.x; w < parts_all * n; w += gridDim.x) {
        // parts of one pair are neighbours, so that a block's check of the pair serves several of them
        const int i = (int)(w / parts_all);
        const long long item = w % parts_all;
        const int s = src[i], d = dst[i];
        if (s < 0 || d < 0) continue;
        const int k = pool_of(pb, item);
        if (i != checked || k != checked_pool) {
            ok = pair_valid(src, dst, n, i, n_src, n_dst, (same >> k) & 1);
            if (!ok && threadIdx.x == 0) report_status(status, KDA_ERR_INVALID_ARG);
            checked = i;
            checked_pool = k;
        }
        if (!ok || (s == d && ((same >> k) & 1))) continue;
        move_part(pb.p[k], s, d, (int)(item - pb.p[k].first));
    }
}

constexpr int kFew = 1024;                             // pairs up to which the kernel above is used
constexpr int kPage = 512;                             // pairs to a page
constexpr int kTable = 4 * kPage;                      // hash table entries: at most a quarter are taken
constexpr uint32_t kRead = 1u << 31;                   // mark: another pair's source; the bits below count destinations
constexpr uint8_t kFineApart = 1, kFineSame = 2;       // verdicts: between two pools, within one

struct Verdicts {
    int key[kTable];                                   // a destination of the page, or -1
    uint32_t mark[kTable];
    uint8_t of[kPage];
};

// The verdicts of pairs first .. first + m - 1 (block-wide: it has barriers).  any: which verdicts the launch's pools
// ask for; a pair that lacks one of them is reported.
__device__ __forceinline__ void judge_page(Verdicts& v, const int* __restrict__ src, const int* __restrict__ dst, int n,
                                           int first, int m, int n_src, int n_dst, uint8_t any, int* status) {
    auto home = [](int d) { return (int)((uint32_t)d * 2654435761u / (0xffffffffu / kTable + 1)); };
    auto find = [&](int d) {                           // ends: three entries in four are empty
        int h = home(d), key;
        while ((key = v.key[h]) != d && key >= 0) h = (h + 1) % kTable;
        return key == d ? h : -1;
    };
    __syncthreads();                                   // the page before is done with
    for (int h = threadIdx.x; h < kTable; h += kThreads) {
        v.key[h] = -1;
        v.mark[h] = 0;
    }
    __syncthreads();
    for (int k = threadIdx.x; k < m; k += kThreads) {
        const int d = dst[first + k];
        if (src[first + k] < 0 || d < 0) continue;     // a skipped pair
        for (int h = home(d);; h = (h + 1) % kTable) {
            const int was = atomicCAS(&v.key[h], -1, d);
            if (was == -1 || was == d) break;
        }
    }
    __syncthreads();
    for (int j = threadIdx.x; j < n; j += kThreads) {
        const int s = src[j], d = dst[j];
        if (s < 0 || d < 0) continue;
        int h = find(d);
        if (h >= 0) atomicAdd(&v.mark[h], 1u);
        if (any & kFineSame) {
            h = find(s);
            if (h >= 0) atomicOr(&v.mark[h], kRead);
        }
    }
    __syncthreads();
    for (int k = threadIdx.x; k < m; k += kThreads) {
        const int s = src[first + k], d = dst[first + k];
        uint8_t fine = 0;
        if (s >= 0 && d >= 0) {
            const uint32_t mark = v.mark[find(d)];
            if (s < n_src && d < n_dst && (mark & ~kRead) == 1)
                fine = kFineApart | (s == d || !(mark & kRead) ? kFineSame : 0);
            if (any & ~fine) report_status(status, KDA_ERR_INVALID_ARG);
        }
        v.of[k] = fine;
    }
    __syncthreads();
}

__global__ void __launch_bounds__(kThreads)
kda_pool_copy_many_kernel(const __grid_constant__ PoolBatch pb, const int* __restrict__ src, const int* __restrict__ dst,
                          int n, int n_src, int n_dst, unsigned long long same, long long parts_all, int* status) {
    __shared__ Verdicts v;
    const uint8_t any = (same ? kFineSame : 0) | (same != (1ull << pb.n) - 1 ? kFineApart : 0);
    const int pages = (n + kPage - 1) / kPage, groups = min(pages, (int)gridDim.x);
    const int group = blockIdx.x % groups, member = blockIdx.x / groups;
    const int members = ((int)gridDim.x - group + groups - 1) / groups;
    for (int page = group; page < pages; page += groups) {
        const int first = page * kPage, m = min(kPage, n - first);
        judge_page(v, src, dst, n, first, m, n_src, n_dst, any, status);
        for (long long w = member; w < parts_all * m; w += members) {
            const int i = (int)(w / parts_all);
            const long long item = w % parts_all;
            const uint8_t fine = v.of[i];
            if (!fine) continue;
            const int k = pool_of(pb, item);
            const bool within = (same >> k) & 1;
            const int s = src[first + i], d = dst[first + i];
            if (!(fine & (within ? kFineSame : kFineApart)) || (s == d && within)) continue;
            move_part(pb.p[k], s, d, (int)(item - pb.p[k].first));
        }
    }
}

__global__ void __launch_bounds__(kThreads)
kda_pool_clear_kernel(const __grid_constant__ PoolBatch pb, const int* __restrict__ idx, int n, int n_slots,
                      long long parts_all, int* status) {
    for (long long w = blockIdx.x; w < parts_all * n; w += gridDim.x) {
        const int i = (int)(w / parts_all);
        const long long item = w % parts_all;
        const int d = idx[i];
        if (d < 0) continue;
        if (d >= n_slots) {
            if (threadIdx.x == 0) report_status(status, KDA_ERR_INVALID_ARG);
            continue;
        }
        const int k = pool_of(pb, item);
        move_part(pb.p[k], 0, d, (int)(item - pb.p[k].first));
    }
}

// ------------------------------------------------------------------ compaction

constexpr int kMaxSlots = 65536;
constexpr int kPlanThreads = 1024;
constexpr int kWords = kMaxSlots / 32;

// Which slots move where.  One block: a bitmap of the live slots and its running counts give every
// slot's rank among the movers (live, >= L) or the holes (free, < L); the k-th mover goes to the k-th
// hole.  plan[0] = number of moves m; mover k at plan[1 + 2k], its hole at plan[2 + 2k] (m <= n_slots/2).
__global__ void __launch_bounds__(kPlanThreads)
kda_pool_plan_kernel(const int* slots, const unsigned char* __restrict__ done, int* slots_out, int B, int n_slots,
                     int* plan, int* status) {
    __shared__ uint32_t live[kWords];
    __shared__ int below[kWords];            // live slots in the words before
    __shared__ int warp_sum[kPlanThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int words = (n_slots + 31) / 32;
    for (int w = tid; w < words; w += kPlanThreads) live[w] = 0;
    __syncthreads();
    bool ok = true;
    for (int b = tid; b < B; b += kPlanThreads) {
        const int s = slots[b];
        if (s < 0 || (done && done[b])) continue;
        if (s >= n_slots) { ok = false; continue; }
        const uint32_t bit = 1u << (s & 31);
        if (atomicOr(&live[s >> 5], bit) & bit) ok = false;      // two live sequences on one slot
    }
    if (!__syncthreads_and(ok)) {
        if (tid == 0) {
            plan[0] = 0;
            report_status(status, KDA_ERR_INVALID_ARG);
        }
        for (int b = tid; b < B; b += kPlanThreads) slots_out[b] = slots[b];
        return;
    }
    // exclusive running count of the live slots by word: each thread a run of words
    const int per = (words + kPlanThreads - 1) / kPlanThreads;
    int sum = 0;
    for (int w = tid * per; w < min(words, (tid + 1) * per); ++w) sum += __popc(live[w]);
    int incl = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += t;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int before = incl - sum, total = 0;
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        if (w < warp) before += warp_sum[w];
        total += warp_sum[w];
    }
    for (int w = tid * per; w < min(words, (tid + 1) * per); ++w) {
        below[w] = before;
        before += __popc(live[w]);
    }
    __syncthreads();
    const int L = total;
    auto live_below = [&](int s) { return below[s >> 5] + __popc(live[s >> 5] & ((1u << (s & 31)) - 1u)); };
    const int front = L < n_slots ? live_below(L) : L;           // live slots < L: they stay
    for (int s = tid; s < n_slots; s += kPlanThreads) {
        const bool is_live = (live[s >> 5] >> (s & 31)) & 1u;
        const int lb = live_below(s);
        if (s < L && !is_live) plan[2 + 2 * (s - lb)] = s;       // hole number s - lb
        if (s >= L && is_live) plan[1 + 2 * (lb - front)] = s;   // mover number lb - front
    }
    if (tid == 0) plan[0] = L - front;
    __syncthreads();                                             // plan is read back below
    for (int b = tid; b < B; b += kPlanThreads) {
        const int s = slots[b];
        int to = -1;
        if (s >= 0 && !(done && done[b])) to = s < L ? s : plan[2 + 2 * (live_below(s) - front)];
        slots_out[b] = to;
    }
}

// Sources are slots >= L and destinations slots < L: no block writes what another reads.
__global__ void __launch_bounds__(kThreads)
kda_pool_move_kernel(const __grid_constant__ PoolBatch pb, const int* __restrict__ plan, long long parts_all) {
    const long long n = plan[0];
    for (long long w = blockIdx.x; w < parts_all * n; w += gridDim.x) {
        const long long i = w / parts_all, item = w % parts_all;
        const int k = pool_of(pb, item);
        move_part(pb.p[k], plan[1 + 2 * i], plan[2 + 2 * i], (int)(item - pb.p[k].first));
    }
}

// Pools first .. of a call as one batch; returns how many it took and the parts of one slot in all of them.
int fill_batch(PoolBatch* pb, const kda_pool* dst, const kda_pool* src, int n_pools, int first, long long* parts_all,
               unsigned long long* same) {
    pb->n = n_pools - first < kPools ? n_pools - first : kPools;
    *parts_all = 0;
    *same = 0;
    for (int k = 0; k < pb->n; ++k) {
        const kda_pool& d = dst[first + k];
        PoolPair& p = pb->p[k];
        p.dst = static_cast<uint8_t*>(d.base);
        p.dst_slot = d.slot_stride;
        p.dst_piece = d.piece_stride;
        p.src = nullptr;
        p.src_slot = p.src_piece = 0;
        if (src) {
            const kda_pool& f = src[first + k];
            p.src = static_cast<const uint8_t*>(f.base);
            p.src_slot = f.slot_stride;
            p.src_piece = f.piece_stride;
            if (f.base == d.base) *same |= 1ull << k;
        }
        p.piece_bytes = d.piece_bytes;
        p.pieces = (int)d.pieces;
        p.parts = (int)((d.piece_bytes + kPart - 1) / kPart);
        p.first = *parts_all;
        *parts_all += (long long)p.parts * p.pieces;
    }
    return pb->n;
}

unsigned blocks_for(long long work) { return (unsigned)(work < kMaxBlocks ? (work > 0 ? work : 1) : kMaxBlocks); }

}  // namespace

cudaError_t launch_pool_copy(const kda_pool* dst, const kda_pool* src, int n_pools, int n_dst, int n_src,
                             const int* src_idx, const int* dst_idx, int n, int* status, cudaStream_t s) {
    for (int at = 0; at < n_pools;) {
        PoolBatch pb;
        long long parts;
        unsigned long long same;
        at += fill_batch(&pb, dst, src, n_pools, at, &parts, &same);
        const auto kernel = n <= kFew ? kda_pool_copy_kernel : kda_pool_copy_many_kernel;
        kernel<<<blocks_for(parts * n), kThreads, 0, s>>>(pb, src_idx, dst_idx, n, n_src, n_dst, same, parts, status);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_pool_clear(const kda_pool* pools, int n_pools, int n_slots, const int* idx, int n, int* status,
                              cudaStream_t s) {
    for (int at = 0; at < n_pools;) {
        PoolBatch pb;
        long long parts;
        unsigned long long same;
        at += fill_batch(&pb, pools, nullptr, n_pools, at, &parts, &same);
        kda_pool_clear_kernel<<<blocks_for(parts * n), kThreads, 0, s>>>(pb, idx, n, n_slots, parts, status);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_pool_compact(const kda_pool* pools, int n_pools, int n_slots, const int* slots,
                                const unsigned char* done, int* slots_out, int B, int* workspace, int* status,
                                cudaStream_t s) {
    kda_pool_plan_kernel<<<1, kPlanThreads, 0, s>>>(slots, done, slots_out, B, n_slots, workspace, status);
    cudaError_t e = cudaGetLastError();
    const long long most = B < n_slots / 2 ? B : n_slots / 2;    // moves: at most a slot in two
    for (int at = 0; at < n_pools && e == cudaSuccess && most > 0;) {
        PoolBatch pb;
        long long parts;
        unsigned long long same;
        at += fill_batch(&pb, pools, pools, n_pools, at, &parts, &same);
        kda_pool_move_kernel<<<blocks_for(parts * most), kThreads, 0, s>>>(pb, workspace, parts);
        e = cudaGetLastError();
    }
    return e;
}

}  // namespace kda
