// topk_kv_evict: keep the `budget` best slots of each (sequence, head).
//
// Bound by HBM: a weight and a position are read per slot, and a kept slot
// above the budget is read and written once.  Two launches, or one where few
// slots move.  512 rows of 8192 slots, half of them kept (1.20 GB): 205 us,
// 5.8 TB/s, 25 us of them for the selection; 8 rows of 131072 cut to an eighth
// (128 MB): 40 us, 20 for the selection, whose three digits cost the cluster a
// barrier and two reads of its neighbours each.
//
// The first selects.  A row belongs to a cluster of 1 to 8 blocks, each with
// a contiguous part of its slots, whose 32-bit keys it reads once and keeps
// in shared memory.  Three histograms of 11, 11 and 10 bits, added up over
// the cluster by reading one another's shared memory, give the budget-th key
// ("edge") and how many keys equal to it are kept.  Then, with K(s) the
// number of kept slots below s, which is a prefix sum of counts,
//     slot s < budget that is not kept is hole number s - K(s),
//     slot s >= budget that is kept is kept slot number K(s),
// and hole j takes kept slot number K(budget) + j.  So holes and movers are
// listed in order without sorting anything.
//
// The second moves the movers into the holes.  Sources lie at or above the
// budget and targets below it, so the moves cannot collide and need no order.
#include <cooperative_groups.h>

#include <type_traits>

#include "topk_device.cuh"
#include "topk_kv.cuh"

namespace cg = cooperative_groups;

namespace topk {
namespace {

constexpr int kBins = 2048;
constexpr int kMostBlocks = 8;  // of a cluster
constexpr int kMoveThreads = 64;
constexpr int kMostHeld = 48 * 1024;  // keys that fit beside the histograms
// Rows with at most so many moves are moved by the blocks that selected.  With
// a budget of 1024: 32 rows of 1101 slots 8.7 us instead of 10.5, 256 of them
// 10.3 instead of 12.1; with 256 moves 32 rows 11.5 instead of 10.8, but 256
// rows 14.4 instead of 15.1 and 512 27.6 instead of 28.7; with 512 moves 32
// rows 16.3 instead of 11.2, and 256 27.6 instead of 21.7.
constexpr int kFused = 256;

struct EvictArgs {
    KvCache c;
    KvEvict e;
    int* lens;    // [seqs] lengths before, clamped
    int* moves;   // [seqs * heads] number of moves M of each row
    int* holes;   // [seqs * heads][room]: holes 0 to M - 1
    int* movers;  // [seqs * heads][room]: the movers, in the row's last M places
    int room;     // moves a row's lists have room for
    int chunks;   // blocks of the second launch per row
    int shift;    // log2 of the lanes that a key takes
    int part;     // slots a block of the first has room for in shared memory
    int fused;    // whether the first launch makes the moves too
    unsigned* ticket;  // then: its blocks that are done, zero before and after
    unsigned* clear;   // the other half of the counters
};

// Order-preserving key: protected above NaN above every number, -0 equal to
// +0.  No key is 0.
__device__ __forceinline__ unsigned evict_key(float w, int pos, int sink, int recent_from) {
    const unsigned u = __float_as_uint(w + 0.0f);
    unsigned key = u ^ ((unsigned)((int)u >> 31) | 0x80000000u);
    if (w != w) key = 0xFFFFFFFEu;
    if (pos < sink || pos >= recent_from) key = 0xFFFFFFFFu;
    return key;
}

// A barrier of the cluster that makes the blocks' shared memory visible to one
// another.  One thread's fence does for all of its block, after the block's
// barrier: a release by every thread takes several times as long.
__device__ __forceinline__ void cluster_sync(int tid) {
    __syncthreads();
    if (tid == 0) asm volatile("fence.acq_rel.cluster;" ::: "memory");
    asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// Moves j0 to j0 + count - 1 (at most 32) of a row, by one warp: a lane looks
// up one move's pages, then all lanes copy the moves' vectors, kUnroll of
// them in flight per lane.  `where`: the warp's 32 entries of shared memory.
__device__ __forceinline__ void move_some(const EvictArgs& a, int b, int h, const int* holes, const int* movers, int j0,
                                          int count, int4* where, int lane) {
    constexpr int kUnroll = 2;  // of keys and of values each
    // A key's vectors take a power of two of lanes, and its value's the same
    // ones: no vector costs a division, and strides are the warp's.
    const int x = (lane & ((1 << a.shift) - 1)) * 8;
    const bool on = x < a.c.dim;
    uint16_t *const k = a.c.k + h * a.c.ks[2] + x, *const v = a.c.v + h * a.c.vs[2] + x;
    int4 at = make_int4(-1, 0, -1, 0);  // source page and slot in it, target page and slot
    if (lane < count) {
        const int from = movers[j0 + lane], to = holes[j0 + lane];
        const int fi = from / a.c.page_size, ti = to / a.c.page_size;
        const int* table = a.c.table + b * a.c.table_stride;
        at = make_int4(table[fi], from - fi * a.c.page_size, table[ti], to - ti * a.c.page_size);
        a.e.weight_out.row(b, h)[to] = a.e.weight.row(b, h)[from];
        a.e.pos_out.row(b, h)[to] = a.e.pos.row(b, h)[from];
        // A move from or to a page that the table does not name is dropped.
        if ((unsigned)at.x >= (unsigned)a.c.pages || (unsigned)at.z >= (unsigned)a.c.pages) at.x = -1;
    }
    __syncwarp();
    where[lane] = at;
    __syncwarp();
    const int total = count << a.shift;
    for (int i0 = lane; i0 < total; i0 += 32 * kUnroll) {
        int4 kv[kUnroll], vv[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int i = i0 + 32 * u;
            if (i < total && on) {
                const int4 q = where[i >> a.shift];
                if (q.x < 0) continue;
                kv[u] = *reinterpret_cast<const int4*>(k + q.x * a.c.ks[0] + q.y * a.c.ks[1]);
                vv[u] = *reinterpret_cast<const int4*>(v + q.x * a.c.vs[0] + q.y * a.c.vs[1]);
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int i = i0 + 32 * u;
            if (i < total && on) {
                const int4 q = where[i >> a.shift];
                if (q.x < 0) continue;
                *reinterpret_cast<int4*>(k + q.z * a.c.ks[0] + q.w * a.c.ks[1]) = kv[u];
                *reinterpret_cast<int4*>(v + q.z * a.c.vs[0] + q.w * a.c.vs[1]) = vv[u];
            }
        }
    }
}

// The last block of a launch that makes the moves too writes the lengths: lens
// may be lens_out, and by then every block has read it.  One warp calls it,
// after a barrier of its block.
__device__ __forceinline__ void write_lens(const EvictArgs& a, int lane) {
    unsigned before = 0;
    if (lane == 0)
        asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(before) : "l"(a.ticket) : "memory");
    if (__shfl_sync(kFullMask, before, 0) + 1 != gridDim.x) return;
    for (int b = lane; b < a.c.seqs; b += 32) a.e.lens_out[b] = min(__ldcg(a.lens + b), a.e.budget);
    if (lane == 0) *a.ticket = 0;
}

// kHeld: the block's keys fit its shared memory; otherwise they are made anew
// from global memory (L2) in each pass.
template <int THREADS, bool kHeld>
__global__ void __launch_bounds__(THREADS) kv_select_kernel(const __grid_constant__ EvictArgs a) {
    constexpr int kWarps = THREADS / 32, kPer = kBins / THREADS;
    extern __shared__ __align__(16) unsigned keys[];
    __shared__ __align__(16) int hist[2][kBins];   // of this digit; of the one before, or cleared for the next
    __shared__ int coarse[2][kWarps];              // the same by kPer * 32 bins, the highest first
    __shared__ int far_coarse[kMostBlocks][32], far_bins[kMostBlocks][kPer][32];  // the cluster's
    __shared__ int scan[kWarps];
    __shared__ int found[3];                       // the bin, how many of its keys are kept, and how many it has
    __shared__ int4 tally;                         // this block: above and at the edge; the same below the budget
    __shared__ int warp_above[kWarps], warp_ties[kWarps];
    cg::cluster_group cluster = cg::this_cluster();
    const int blocks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int row = blockIdx.x / blocks, b = row / a.c.heads, h = row % a.c.heads;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    grid_dependency_wait();
    clear_half(a.clear);
    const int n = a.c.len(b), budget = a.e.budget;
    const float* w = a.e.weight.row(b, h);
    const int* pos = a.e.pos.row(b, h);
    float* wo = a.e.weight_out.row(b, h);
    int* po = a.e.pos_out.row(b, h);
    const bool copy_w = wo != w, copy_p = po != pos;
    if (tid == 0 && h == 0 && rank == 0) a.lens[b] = n;
    // This block's slots: multiples of the warps' rounds.
    const int part = ((n + blocks - 1) / blocks + 31) & ~31, lo = min(rank * part, n), hi = min(lo + part, n);
    if (n <= budget) {  // the whole cluster leaves here
        for (int i = lo + tid; i < hi; i += THREADS) {
            if (copy_w) wo[i] = w[i];
            if (copy_p) po[i] = pos[i];
        }
        if (tid == 0 && rank == 0) a.moves[row] = 0;
        if (a.fused) {
            __syncthreads();
            if (warp == 0) write_lens(a, lane);
        }
        return;
    }
    const int sink = a.e.sink;
    const long long recent_from64 = (long long)a.e.next_pos[b] - a.e.recent;
    const int recent_from = recent_from64 < INT_MIN ? INT_MIN : (int)recent_from64;
    // The key of slot i of this block's part; past its end 0, which is no
    // slot's key, below every edge, and never in an edge's bin.
    auto key_at = [&](int i) {
        return kHeld ? keys[i - lo] : i < hi ? evict_key(w[i], pos[i], sink, recent_from) : 0u;
    };
    const int end = lo < hi ? lo + part : lo;  // a multiple of 32 slots
    auto keys_at = [&](int i, int stop, unsigned (&key)[4]) {  // slots i to i + 3
        if (kHeld) {
            const uint4 q = i < stop ? *reinterpret_cast<const uint4*>(keys + (i - lo)) : make_uint4(0, 0, 0, 0);
            key[0] = q.x;
            key[1] = q.y;
            key[2] = q.z;
            key[3] = q.w;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) key[j] = i < stop ? key_at(i + j) : 0;
        }
    };

    // Four slots a thread at a time, the next four in flight meanwhile; the
    // first four while the histograms are cleared.  Adding 1 at an address
    // that many lanes share is one operation of the hardware, so equal keys
    // (protected slots, slots nothing looked at) cost nothing more.
    float wv[4];
    int pv[4];
    auto fetch = [&](int base) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = base + j * THREADS + tid;
            wv[j] = i < hi ? w[i] : 0.f;
            pv[j] = i < hi ? pos[i] : 0;
        }
    };
    fetch(lo);
    for (int i = tid; i < 2 * kBins; i += THREADS) (&hist[0][0])[i] = 0;
    if (tid == 0) tally = make_int4(0, 0, 0, 0);
    __syncthreads();
    for (int base = lo; base < end; base += 4 * THREADS) {
        float wn[4];
        int pn[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            wn[j] = wv[j];
            pn[j] = pv[j];
        }
        if (base + 4 * THREADS < end) fetch(base + 4 * THREADS);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = base + j * THREADS + tid;
            const unsigned key = i < hi ? evict_key(wn[j], pn[j], sink, recent_from) : 0;
            if (kHeld && i < end) keys[i - lo] = key;
            if (i < hi) {
                atomicAdd(&hist[0][key >> 21], 1);
                if (i < budget) {
                    if (copy_w) wo[i] = wn[j];
                    if (copy_p) po[i] = pn[j];
                }
            }
        }
    }
    unsigned prefix = 0;
    int need = budget;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int up = pass == 0 ? 32 : pass == 1 ? 21 : 10, shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const unsigned mask = (1u << (up - shift)) - 1;
        if (pass > 0) {
            for (int base = lo; base < end; base += 4 * THREADS) {
                unsigned key[4];
                keys_at(base + 4 * tid, end, key);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (((key[j] ^ prefix) >> up) == 0)
                        atomicAdd(&hist[pass & 1][(key[j] >> shift) & mask], 1);
            }
        }
        __syncthreads();
        // Thread t has kPer bins, t = 0 the highest.
        using Vec = typename std::conditional<kPer == 2, int2, int4>::type;
        constexpr int kWide = sizeof(Vec) / 4;
        int* mine = hist[pass & 1];
        auto bins_of = [&](const int* from, int t, int (&own)[kPer]) {  // highest first
            int sum = 0;
#pragma unroll
            for (int i = 0; i < kPer; i += kWide) {
                const Vec v = *reinterpret_cast<const Vec*>(from + kBins - kPer * (t + 1) + i);
                const int* x = reinterpret_cast<const int*>(&v);
#pragma unroll
                for (int j = 0; j < kWide; ++j) {
                    own[kPer - 1 - i - j] = x[j];
                    sum += x[j];
                }
            }
            return sum;
        };
        auto scan_warp = [&](int x) {
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int y = __shfl_up_sync(kFullMask, x, d);
                if (lane >= d) x += y;
            }
            return x;
        };
        // The bin of thread t's among which the need-th key lies, `before` of them above.
        auto look = [&](int t, const int (&own)[kPer], int before, int sum) {
            if (before < need && need <= before + sum) {
#pragma unroll
                for (int j = 0; j < kPer; ++j) {
                    if (before < need && need <= before + own[j]) {
                        found[0] = kBins - 1 - (t * kPer + j);
                        found[1] = need - before;
                        found[2] = own[j];
                    }
                    before += own[j];
                }
            }
        };
        int own[kPer];
        const int sum = bins_of(mine, tid, own);
        if (blocks == 1) {
            const int x = scan_warp(sum);
            if (lane == 31) scan[warp] = x;
            __syncthreads();
            look(tid, own, __reduce_add_sync(kFullMask, lane < warp ? scan[lane] : 0) + x - sum, sum);
        } else {
            // Over the cluster in two steps, so that little is read from other
            // blocks: the warp's worth of bins, then the bin in it.  A warp
            // reads one block.
            const int all = __reduce_add_sync(kFullMask, sum);
            if (lane == 0) coarse[pass & 1][warp] = all;
            cluster_sync(tid);
            if (warp < blocks && lane < kWarps)
                far_coarse[warp][lane] = cluster.map_shared_rank(&coarse[pass & 1][0], warp)[lane];
            __syncthreads();
            int v = 0;
            if (lane < kWarps)
                for (int r = 0; r < blocks; ++r) v += far_coarse[r][lane];
            const int x = scan_warp(v), at = __ffs(__ballot_sync(kFullMask, x >= need)) - 1;
            const int before = __shfl_sync(kFullMask, x - v, at), t = at * 32 + lane;
            if (warp < blocks) {
                bins_of(cluster.map_shared_rank(mine, warp), t, own);
#pragma unroll
                for (int j = 0; j < kPer; ++j) far_bins[warp][j][lane] = own[j];
            }
            __syncthreads();
            if (warp == 0) {
                int some = 0;
#pragma unroll
                for (int j = 0; j < kPer; ++j) {
                    own[j] = 0;
                    for (int r = 0; r < blocks; ++r) own[j] += far_bins[r][j][lane];
                    some += own[j];
                }
                look(t, own, before + scan_warp(some) - some, some);
            }
        }
        // The digit before has been read by every block: cleared for the one after this.
        if (pass == 1)
            for (int i = tid; i < kBins; i += THREADS) hist[0][i] = 0;
        __syncthreads();
        prefix |= (unsigned)found[0] << shift;
        need = found[1];
        if (need == found[2]) {  // all of the bin: no need to look into it
            prefix -= 1;  // above any absent key's 0, and keys equal to it are not kept
            need = 0;
            break;
        }
    }
    const unsigned edge = prefix;  // keys above it are kept, and the first `need` that equal it

    // Counts, by warps with a contiguous part each.
    const int mine = ((part + kWarps - 1) / kWarps + 127) & ~127;
    const int from = min(lo + warp * mine, end), to = min(from + mine, end);
    auto count = [&](int from, int to, int* above, int* ties) {
        int up = 0, at = 0;
        for (int base = from; base < to; base += 128) {
            unsigned key[4];
            keys_at(base + 4 * lane, to, key);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                up += key[j] > edge;
                at += key[j] == edge;
            }
        }
        *above = __reduce_add_sync(kFullMask, up);
        *ties = __reduce_add_sync(kFullMask, at);
    };
    int above, ties, above_low = 0, ties_low = 0;
    count(from, to, &above, &ties);
    if (to <= budget) {
        above_low = above;
        ties_low = ties;
    } else if (from < budget) {  // the warp whose part the budget lies in
        int up = 0, at = 0;
        for (int i = from + lane; i < budget; i += 32) {
            const unsigned key = key_at(i);
            up += key > edge;
            at += key == edge;
        }
        above_low = __reduce_add_sync(kFullMask, up);
        ties_low = __reduce_add_sync(kFullMask, at);
    }
    if (lane == 0) {
        warp_above[warp] = above;
        warp_ties[warp] = ties;
        atomicAdd(&tally.x, above);
        atomicAdd(&tally.y, ties);
        atomicAdd(&tally.z, above_low);
        atomicAdd(&tally.w, ties_low);
    }
    if (blocks > 1) cluster_sync(tid); else __syncthreads();
    int4 t = make_int4(0, 0, 0, 0);
    if (lane < blocks) t = blocks == 1 ? tally : *cluster.map_shared_rank(&tally, lane);
    const int up_low = __reduce_add_sync(kFullMask, t.z), all_ties_low = __reduce_add_sync(kFullMask, t.w);
    const bool lower = lane < rank;
    int up_before = __reduce_add_sync(kFullMask, (lower ? t.x : 0) + (lane < warp ? warp_above[lane] : 0));
    int ties_before = __reduce_add_sync(kFullMask, (lower ? t.y : 0) + (lane < warp ? warp_ties[lane] : 0));
    const int moves = budget - up_low - min(all_ties_low, need);
    if (tid == 0 && rank == 0) a.moves[row] = moves;
    int* holes = a.holes + (size_t)row * a.room;
    int* movers = a.movers + (size_t)row * a.room + (a.room - budget);
    // Of the keys at the edge, all of this warp's are kept or none, but in the
    // one warp of the row where the last of them is.
    const bool some = ties_before < need && need < ties_before + ties;
    const unsigned least = ties_before + ties <= need ? edge : edge + 1;  // edge + 1 == 0 has no key at it
    int kept_before = up_before + min(ties_before, need);
    auto list = [&](int i, bool kept, int before) {  // slot i, with `before` kept ones below it
        if (i < budget) {
            if (!kept) holes[i - before] = i;
        } else if (kept) {
            movers[before] = i;
        }
    };
    if (some) {
        for (int i = from + lane; i - lane < to; i += 32) {
            const unsigned key = key_at(i);
            const unsigned at = __ballot_sync(kFullMask, key == edge);
            const bool kept = key > edge || (key == edge && ties_before + __popc(at & lanemask_lt()) < need);
            const unsigned all = __ballot_sync(kFullMask, kept);
            ties_before += __popc(at);
            list(i, kept, kept_before + __popc(all & lanemask_lt()));
            kept_before += __popc(all);
        }
    } else {
        // A lane has four slots in a row; their number of kept ones is added
        // up over the lanes below by the bits of it.
        const unsigned lower_lanes = lanemask_lt();
        for (int base = from; base < to; base += 128) {
            const int i = base + 4 * lane;
            unsigned key[4];
            keys_at(i, to, key);
            bool kept[4];
            int mine = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                kept[j] = key[j] >= least && least != 0;
                mine += kept[j];
            }
            const unsigned b0 = __ballot_sync(kFullMask, mine & 1), b1 = __ballot_sync(kFullMask, mine & 2),
                           b2 = __ballot_sync(kFullMask, mine & 4);
            int before = kept_before + __popc(b0 & lower_lanes) + 2 * __popc(b1 & lower_lanes) +
                         4 * __popc(b2 & lower_lanes);
            kept_before += __popc(b0) + 2 * __popc(b1) + 4 * __popc(b2);
            if (i >= to) continue;
            if (base + 128 <= budget) {  // alike for the warp, nearly always
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (!kept[j]) holes[i + j - before] = i + j;
                    before += kept[j];
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    list(i + j, kept[j], before);
                    before += kept[j];
                }
            }
        }
    }
    launch_dependents();  // the moves, which wait for this launch's end
    if (blocks > 1) cluster_sync(tid);  // no block leaves while another reads its counts
    if (!a.fused) return;
    if (blocks == 1) __syncthreads();
    // The lists are complete.  The histograms' place takes the looked-up pages.
    static_assert(kWarps <= 32 && sizeof(hist) >= kWarps * 32 * sizeof(int4), "look-ups fit");
    int4* where = reinterpret_cast<int4*>(&hist[0][0]) + warp * 32;
    const int warps = blocks * kWarps, batch = min(32, (moves + warps - 1) / warps);
    for (int j0 = (rank * kWarps + warp) * batch; j0 < moves; j0 += warps * batch)
        move_some(a, b, h, holes, movers + (budget - moves), j0, min(batch, moves - j0), where, lane);
    if (warp == 0) write_lens(a, lane);
}

__global__ void __launch_bounds__(kMoveThreads) kv_move_kernel(const __grid_constant__ EvictArgs a) {
    __shared__ int4 where[kMoveThreads / 32][32];
    const int row = blockIdx.x / a.chunks, chunk = blockIdx.x % a.chunks, b = row / a.c.heads, h = row % a.c.heads;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_dependency_wait();
    if (chunk == 0 && h == 0 && threadIdx.x == 0) {
        const int n = a.lens[b];
        a.e.lens_out[b] = n < a.e.budget ? n : a.e.budget;
    }
    const int moves = a.moves[row];
    const int* holes = a.holes + (size_t)row * a.room;
    const int* movers = a.movers + (size_t)row * a.room + (a.room - moves);
    for (int j0 = (chunk * (kMoveThreads / 32) + warp) * 32; j0 < moves; j0 += a.chunks * kMoveThreads)
        move_some(a, b, h, holes, movers, j0, min(32, moves - j0), where[warp], lane);
}

int room_of(const KvCache& c, const KvEvict& e) {
    const int above = c.capacity() - e.budget;
    return above < 1 ? 1 : above < e.budget ? above : e.budget;
}

template <int THREADS, bool kHeld>
cudaError_t select(const EvictArgs& a, int rows, int blocks, int device, cudaStream_t s) {
    auto kernel = kv_select_kernel<THREADS, kHeld>;
    const size_t smem = kHeld ? (size_t)a.part * 4 : 0;
    constexpr int kMostSmem = kMostHeld * 4;
    static std::atomic<unsigned long long> allowed{0};
    const cudaError_t e = kHeld ? allow_smem(kernel, kMostSmem, device, allowed) : cudaSuccess;
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * blocks));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // it waits before it reads anything
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)blocks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = blocks > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

size_t kv_evict_scratch(const KvCache& c, const KvEvict& e) {
    const size_t rows = (size_t)c.seqs * c.heads;
    return 4 * (c.seqs + rows + 2 * rows * room_of(c, e));
}

cudaError_t kv_evict_launch(int device, int sms, cudaStream_t s, const KvCache& c, const KvEvict& e,
                            const KvState& state, int* launches) {
    const int rows = c.seqs * c.heads;
    EvictArgs a = {c, e};
    a.room = room_of(c, e);
    a.lens = static_cast<int*>(state.scratch);
    a.moves = a.lens + c.seqs;
    a.holes = a.moves + rows;
    a.movers = a.holes + (size_t)rows * a.room;
    a.ticket = state.mine + kKvTicket;
    a.clear = state.other;
    a.fused = a.room <= kFused;
    a.shift = 0;
    while ((1 << a.shift) < c.dim / 8) ++a.shift;
    // The lengths are on the device: what follows goes by the table's capacity,
    // and was measured where that is the longest row's length.  In a table with
    // room to spare it is a plan for longer rows, and too many blocks of moves
    // (512 rows of 4500 slots: 116 us, in a table for 16384 120, for 131072 212;
    // 32 rows of 1074 to 1024: 7.8 us, for 16384 15.4).
    //
    // Blocks per row: as many as keep the SMs busy twice over, and leave each
    // block 1024 slots at least.  (Clusters of 16 were slower: 8 rows of
    // 131072 slots 53 us instead of 43, since not all eight run at once.)
    int blocks = 1;
    while (blocks < 8 && rows * blocks * 2 <= 2 * sms && c.capacity() / (blocks * 2) >= 1024) blocks *= 2;
    while (blocks < 8 && (c.capacity() + blocks - 1) / blocks + 32 > kMostHeld) blocks *= 2;
    a.part = (((c.capacity() + blocks - 1) / blocks + 31) & ~31);
    const bool held = a.part <= kMostHeld;
    cudaError_t err;
    // Short rows spend their time at barriers, which cost less in small blocks
    // (32 rows of 1101 slots: 8.0 us with 256 threads, 9.0 with 1024; 160 of
    // 1500 10.9, with 512 11.2), and more than two of which share an SM (512 of
    // 1100: 14.5 and 18.9, of 4500 115 and 118, but of 8192 211 and 205).  Few
    // long ones need all the threads that an SM takes (8 of 131072: 42 us with 1024, 45 with 512).
    if (blocks == 1 && c.capacity() <= (rows <= 2 * sms ? 2048 : 5120))
        err = select<256, true>(a, rows, blocks, device, s);
    else if (rows * blocks <= sms)
        err = held ? select<1024, true>(a, rows, blocks, device, s) : select<1024, false>(a, rows, blocks, device, s);
    else
        err = held ? select<512, true>(a, rows, blocks, device, s) : select<512, false>(a, rows, blocks, device, s);
    if (err != cudaSuccess) return err;
    ++*launches;
    if (a.fused) return cudaSuccess;
    a.chunks = (a.room + kMoveThreads - 1) / kMoveThreads;
    const long long most = (1 << 20) / rows + 1;
    if (a.chunks > most) a.chunks = (int)most;
    err = launch_pdl(kv_move_kernel, dim3(rows * a.chunks), dim3(kMoveThreads), 0, s, a);
    if (err == cudaSuccess) ++*launches;
    return err;
}

}  // namespace topk
