// topk_kv_attend: attention of one new token over a paged cache.
//
// Every key and value is read once, and per 16-bit element there are only
// 2 * group multiply-adds, so the operator is bound by HBM: 6.79 TB/s of
// measured copy rate is 23 bytes per SM and clock.  With a group of eight
// query heads that is still more arithmetic than the scalar pipes do in that
// time, so both products run on the tensor cores, with the cache as the
// 128-row operand that goes from HBM to shared memory (TMA) to the tensor
// core without passing through registers:
//     S^T [128 slots x heads] = K [128 slots x dim] * Q^T,
//     O^T [dim x heads]      += V^T [dim x 128 slots] * P^T.
// Accumulators are in tensor memory, one lane per slot (S) or per element of
// dim (O), so that each of 128 threads owns one slot's scores.
//
// Softmax is one pass.  p = 2^(s * scale * log2(e) - m + kBias), where m is a
// reference that moves only when some score passes it by kSlack (a factor
// 2^kSlack, far from float32's range), so that O is hardly ever rescaled.  P
// enters the second product as two 16-bit numbers, hi + lo, which the
// product adds up in columns of their own: 16 columns are the least that
// this shape of the instruction takes, and a group of 8 fills them with hi
// and lo, so P keeps 16 bits or more at no cost.
//
// Work is split evenly whatever the lengths are: all (sequence, head) rows'
// tiles of 128 slots are numbered in order, and block c takes the range
// [c * T / n, (c + 1) * T / n) of them.  A row that lies in one block is
// finished there; a row that several blocks share is joined by the second
// launch, which also turns the stored p into weights.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "topk_device.cuh"
#include "topk_kv.cuh"
#include "topk_tcgen05.cuh"

namespace topk {
namespace {

constexpr int kTile = 128;       // slots of a tile
constexpr int kThreads = 224;    // 4 softmax warps, the copy warp, a warp for each product
constexpr int kJoinThreads = 512;
constexpr float kSlack = 8.f;    // p <= 2^(kSlack + kBias) = 2^15: within f16's range
constexpr float kBias = 7.f;     // and f16's smallest step, 2^-24, is 2^-31 of the largest p
constexpr int kRingBytes = 192 * 1024;

__device__ __forceinline__ uint16_t from_float(float x, int bf16) {
    return bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(x)) : __half_as_ushort(__float2half_rn(x));
}

struct AttendArgs {
    KvCache c;
    KvAttend a;
    int group;     // query heads of a key-value head
    int parts;     // parts of at most GP query heads that a group is cut into
    int rows;      // heads * parts: rows of a sequence
    int box;       // slots that one copy takes: a power of two that divides page_size
    float* part_o;    // [2 * blocks][GP][dim]: unnormalised output of a row's share
    float2* part_ml;  // [2 * blocks][GP]: its reference and sum
    float2* row_ml;   // [seqs * rows][GP]: the same of rows that one block finished
    float* p;         // [tile][slot][GP], when weights are wanted
    float* tile_m;    // [tile][GP]: the reference of each tile's p
    unsigned* status;
};

// Where a block's share of the tiles begins and ends, and a walk over it.
struct Walk {
    int b, r, t;    // sequence, row of the sequence, tile of the row
    int n, tiles;   // the sequence's slots and tiles
    int s, e;       // the block's range of tile numbers
    int total, blocks;

    __device__ void enter(const AttendArgs& p) {
        while (b < p.c.seqs) {
            n = p.c.len(b);
            if (n > 0) break;
            ++b;
        }
        tiles = (n + kTile - 1) / kTile;
    }
    __device__ void next(const AttendArgs& p) {
        if (++t < tiles) return;
        t = 0;
        if (++r < p.rows) return;
        r = 0;
        ++b;
        enter(p);
    }
    // The block that tile number x belongs to.
    __device__ int block_of(int x) const { return (int)((((long long)x + 1) * blocks - 1) / total); }
};

// Every thread of the block calls it; sh: THREADS / 32 + 8 words of shared memory.
template <int THREADS>
__device__ Walk find_range(const AttendArgs& p, int* sh) {
    constexpr int W = THREADS / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, seqs = p.c.seqs;
    const int chunk = (seqs + THREADS - 1) / THREADS, lo = tid * chunk, hi = min(lo + chunk, seqs);
    int mine = 0;
    for (int b = lo; b < hi; ++b) mine += (p.c.len(b) + kTile - 1) / kTile * p.rows;
    int x = mine;
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(kFullMask, x, d);
        if (lane >= d) x += y;
    }
    if (lane == 31) sh[warp] = x;
    __syncthreads();
    int before = x - mine, total = 0;
    for (int w = 0; w < W; ++w) {
        if (w < warp) before += sh[w];
        total += sh[w];
    }
    Walk k;
    k.total = total;
    k.blocks = min((int)gridDim.x, total);
    k.s = k.e = k.b = k.r = k.t = k.n = k.tiles = 0;
    if ((int)blockIdx.x < k.blocks) {  // uniform over the block
        k.s = (int)((long long)blockIdx.x * total / k.blocks);
        k.e = (int)(((long long)blockIdx.x + 1) * total / k.blocks);
        if (before <= k.s && k.s < before + mine) {
            int at = before, b = lo;
            for (;; ++b) {
                const int tiles = (p.c.len(b) + kTile - 1) / kTile;
                if (k.s < at + tiles * p.rows) {
                    sh[W] = b;
                    sh[W + 1] = (k.s - at) / tiles;
                    sh[W + 2] = (k.s - at) % tiles;
                    break;
                }
                at += tiles * p.rows;
            }
        }
        __syncthreads();
        k.b = sh[W];
        k.r = sh[W + 1];
        k.t = sh[W + 2];
        k.n = p.c.len(k.b);
        k.tiles = (k.n + kTile - 1) / kTile;
    }
    return k;
}

template <int DP, int GP>
struct Shape {
    static constexpr int kSub = DP / 64;                  // 128-byte columns of a row
    static constexpr int kItem = kTile * DP * 2;          // bytes of a tile's keys or values
    static constexpr int kRing = kRingBytes / kItem;
    static constexpr int kQBytes = kSub * 16 * 128;       // 16 rows of a query block
    static constexpr int kPCols = 2 * GP;                 // hi and lo of every head
    static constexpr int kPRow = kPCols * 2;              // bytes of a slot's row of P
    static constexpr int kPBytes = kPRow * kTile;
    static constexpr int kM = DP == 64 ? 64 : 128;        // rows of one second product
    static constexpr int kOBlocks = DP / kM;
    static constexpr int kTmemS = 0, kTmemO = 32;         // columns: two S buffers of 16, then O
    static constexpr int kTmemCols = 32 + kOBlocks * kPCols <= 64 ? 64 : 128;
    static constexpr size_t kSmem = 1024 + kRingBytes + 2 * kQBytes + 2 * kPBytes;
    // Barriers, by their place in bars[].
    static constexpr int kFull = 0, kEmpty = kRing, kSFull = 2 * kRing, kSFree = kSFull + 2, kPReady = kSFull + 4,
                         kPFree = kSFull + 6, kQFull = kSFull + 8, kQFree = kSFull + 10, kDrain = kSFull + 12,
                         kBars = kSFull + 14;
};

// The bounded wait's slow side: gives up after kWaitSpins tries, or once
// another wait of the block has.
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile int* gave_up, unsigned* status) {
    for (int i = 0; i < kWaitSpins; ++i) {
        if (mbar_try(bar, parity)) return true;
        if (*gave_up) return false;
    }
    *gave_up = 1;
    atomicOr(status, kStatusWaitTimeout);
    return false;
}

// A place in the ring, moved on by n <= kRing items.
template <int RING>
struct Place {
    int at;
    uint32_t phase;
    __device__ __forceinline__ void move(int n) {
        at += n;
        if (at >= RING) {
            at -= RING;
            phase ^= 1;
        }
    }
};

// Sums of v[g] over the warp's lanes, for GP heads at once: lanes halve the
// heads they hold as the sums double in width, so this takes GP - 1 + (5 -
// log2 GP) shuffles instead of 5 * GP.  Returns the sum of head warp_head().
template <int GP>
__device__ __forceinline__ float warp_sums(float (&v)[GP], int lane) {
#pragma unroll
    for (int n = GP / 2, d = 16; d >= 1; n /= 2, d /= 2) {
        if (n == 0) {
            v[0] += __shfl_xor_sync(kFullMask, v[0], d);
        } else {
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const bool high = (lane & d) != 0;
                const float give = high ? v[i] : v[i + n], keep = high ? v[i + n] : v[i];
                v[i] = keep + __shfl_xor_sync(kFullMask, give, d);
            }
        }
    }
    return v[0];
}
template <int GP>
__device__ __forceinline__ int warp_head(int lane) { return lane >> (GP == 8 ? 2 : 1); }

// Two numbers as 16-bit elements in one word, and back.
__device__ __forceinline__ uint32_t pack2(float a, float b, int bf16) {
    if (bf16) {
        const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&x);
    }
    const __half2 x = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&x);
}
__device__ __forceinline__ float2 unpack2(uint32_t x, int bf16) {
    if (bf16) return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u));
    return __half22float2(*reinterpret_cast<const __half2*>(&x));
}

template <int DP, int GP>
__global__ void __launch_bounds__(kThreads, 1)
kv_attend_kernel(const AttendArgs p, const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                 const __grid_constant__ CUtensorMap map_q) {
    using S = Shape<DP, GP>;
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(8) uint64_t bars[S::kBars];
    __shared__ uint32_t tmem_at;
    __shared__ int scan[kThreads / 32 + 8];
    __shared__ __align__(16) float red[4][GP];
    __shared__ volatile int gave_up;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t bar0 = smem_addr(bars);
    if (tid == 0) {
        for (int i = 0; i < S::kBars; ++i) {
            const bool by_threads = i == S::kSFree || i == S::kSFree + 1 || i == S::kPReady || i == S::kPReady + 1;
            mbar_init(&bars[i], by_threads ? 128 : 1);
        }
        mbar_init_fence();
        gave_up = 0;
    }
    if (warp == 4 && lane == 0) {
        prefetch_map(&map_k);
        prefetch_map(&map_v);
        prefetch_map(&map_q);
    }
    if (warp == 5) tmem_alloc(&tmem_at, S::kTmemCols);
    launch_dependents();  // the join waits for this launch's end before it reads anything of it
    Walk w = find_range<kThreads>(p, scan);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_at;
    const uint32_t ring = (smem_addr(smem_raw) + 1023) & ~1023u, q_buf = ring + kRingBytes, p_buf = q_buf + 2 * S::kQBytes;
    const int count = w.e - w.s;  // tiles of this block

    auto wait = [&](int bar, uint32_t parity) {
        if (mbar_try(bar0 + bar * 8, parity)) return true;
        return wait_slow(bar0 + bar * 8, parity, &gave_up, p.status);
    };
    // The block's tiles of the row that x stands in, and the slots of the last of them.
    auto share_of = [&](const Walk& x, int done, int* last) {
        const int n = min(x.tiles - x.t, count - done);
        *last = min(kTile, x.n - (x.t + n - 1) * kTile);
        return n;
    };

    if (warp == 4) {
        // Copies, in the order in which the products use them:
        // K(0), K(1), V(0), K(2), V(1), ..., V(count - 1).
        const uint64_t policy = l2_evict_first_policy();
        constexpr int kPer = (16 * S::kSub + 31) / 32;  // copies of a lane, at most
        struct Tile {
            int row, b, copies;
            int page[kPer], at[kPer];  // of each copy's first slot
        };
        // The pages of a tile, fetched a tile ahead of their use: the load
        // takes as long as a third of a tile's copy.  A lane's slots move by
        // a tile at a time, so that only a new row divides.
        int index[kPer], in[kPer];
        const int step = kTile / p.c.page_size, rest = kTile % p.c.page_size;
        auto fetch = [&](const Walk& x, Tile& t, bool enter) {
            t.row = x.r;
            t.b = x.b;
            const int left = x.n - x.t * kTile;
            t.copies = left >= kTile ? kTile / p.box * S::kSub : (left + p.box - 1) / p.box * S::kSub;
            const int* table = p.c.table + x.b * p.c.table_stride;
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const int i = j * 32 + lane;
                if (enter) {
                    const int slot = x.t * kTile + i / S::kSub * p.box;
                    index[j] = slot / p.c.page_size;
                    in[j] = slot - index[j] * p.c.page_size;
                } else {
                    index[j] += step;
                    in[j] += rest;
                    if (in[j] >= p.c.page_size) {
                        in[j] -= p.c.page_size;
                        ++index[j];
                    }
                }
                t.at[j] = in[j];
                t.page[j] = -1;
                if (i < t.copies) t.page[j] = table[index[j]];
            }
        };
        Place<S::kRing> put = {0, 0};
        int items = 0, q_loads = 0;
        auto wait_warp = [&](int bar, uint32_t parity) { return __all_sync(kFullMask, wait(bar, parity)); };
        auto load = [&](const Tile& t, const CUtensorMap* map) {
            if (items >= S::kRing && !wait_warp(S::kEmpty + put.at, put.phase ^ 1)) return false;
            const uint32_t full = bar0 + (S::kFull + put.at) * 8, dst = ring + put.at * S::kItem;
            if (lane == 0) mbar_expect_at(full, t.copies * p.box * 128);
            __syncwarp();
            const int h = p.parts == 1 ? t.row : t.row / p.parts;
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const int i = j * 32 + lane;
                if (i < t.copies) {
                    // A page outside the pool reads as zeros.
                    const int page = (unsigned)t.page[j] < (unsigned)p.c.pages ? t.page[j] : p.c.pages;
                    tma_load_4d(dst + i % S::kSub * (kTile * 128) + i / S::kSub * p.box * 128, map, i % S::kSub * 64,
                                t.at[j], h, page, full, policy);
                }
            }
            ++items;
            put.move(1);
            return true;
        };
        Walk x = w;
        Tile before, now, after;
        bool enters = true, enters_next = false;
        if (count > 0) fetch(x, now, true);
        for (int it = 0; it <= count; ++it) {
            if (it + 1 < count) {
                x.next(p);
                enters_next = x.t == 0;
                fetch(x, after, enters_next);
            }
            if (it < count) {
                if (enters) {
                    const int buf = q_loads & 1;
                    if (q_loads >= 2 && !wait_warp(S::kQFree + buf, ((q_loads - 2) >> 1) & 1)) break;
                    if (lane == 0) {
                        const uint32_t full = bar0 + (S::kQFull + buf) * 8;
                        mbar_expect_at(full, S::kSub * GP * 128);
                        for (int sub = 0; sub < S::kSub; ++sub)
                            tma_load_3d(q_buf + buf * S::kQBytes + sub * 16 * 128, &map_q, sub * 64,
                                        now.row / p.parts * p.group + now.row % p.parts * GP, now.b, full);
                    }
                    ++q_loads;
                    __syncwarp();
                }
                if (!load(now, &map_k)) break;
            }
            if (it > 0 && !load(before, &map_v)) break;
            before = now;
            now = after;
            enters = enters_next;
        }
        __syncwarp();
        if (gave_up) {  // wait for the copies in flight, so that none lands after the block's end
            for (int i = max(0, items - S::kRing); i < items; ++i)
                mbar_wait(&bars[S::kFull + i % S::kRing], (i / S::kRing) & 1);
            for (int i = max(0, q_loads - 2); i < q_loads; ++i) mbar_wait(&bars[S::kQFull + (i & 1)], (i >> 1) & 1);
        }
    } else if (warp == 5) {
        if (lane == 0) {  // S = K Q^T
            const uint32_t id = mma_idesc(p.c.bf16, kTile, 16, false);
            constexpr uint32_t hi = smem_desc_hi(1024, 128);
            const uint32_t k_lo = smem_desc_lo(ring, 16), q_lo = smem_desc_lo(q_buf, 16);
            Place<S::kRing> get = {0, 0};
            Walk x = w;
            bool ok = true;
            for (int it = 0, piece = 0; it < count && ok; ++piece) {
                int last;
                const int n = share_of(x, it, &last), qb = piece & 1;
                if (!wait(S::kQFull + qb, (piece >> 1) & 1)) break;
                for (int k = 0; k < n; ++k, ++it) {
                    const int buf = it & 1;
                    ok = wait(S::kFull + get.at, get.phase) &&
                         (it < 2 || wait(S::kSFree + buf, ((it >> 1) & 1) ^ 1));
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t a = k_lo + get.at * (S::kItem >> 4), b = q_lo + qb * (S::kQBytes >> 4);
#pragma unroll
                    for (int j = 0; j < DP / 16; ++j)
                        mma_f16(tmem + S::kTmemS + buf * 16, a + (((j >> 2) * (kTile * 128) + (j & 3) * 32) >> 4), hi,
                                b + (((j >> 2) * (16 * 128) + (j & 3) * 32) >> 4), hi, id, j > 0);
                    mma_commit(bar0 + (S::kSFull + buf) * 8);
                    mma_commit(bar0 + (S::kEmpty + get.at) * 8);
                    get.move(it == 0 ? 1 : 2);  // K(t) is item 2t - 1, but K(0) is the first
                }
                mma_commit(bar0 + (S::kQFree + qb) * 8);
                x.t += n - 1;
                x.next(p);
            }
            if (gave_up) {  // wait for the products in flight
                mma_commit(bar0 + S::kDrain * 8);
                mbar_wait(&bars[S::kDrain], 0);
            }
        }
        __syncwarp();
    } else if (warp == 6) {
        if (lane == 0) {  // O += V^T P^T
            const uint32_t id = mma_idesc(p.c.bf16, S::kM, S::kPCols, true);
            constexpr uint32_t hi_v = smem_desc_hi(1024, 128), hi_p = smem_desc_hi(S::kPRow * 8, S::kPRow);
            const uint32_t v_lo = smem_desc_lo(ring, kTile * 128), p_lo = smem_desc_lo(p_buf, 16);
            // V(t) is item 2t + 2, but the last one follows V(t - 1).
            Place<S::kRing> get = {0, 0};
            get.move(count == 1 ? 1 : 2);
            Walk x = w;
            bool ok = true;
            for (int it = 0; it < count && ok;) {
                int last;
                const int n = share_of(x, it, &last);
                for (int k = 0; k < n; ++k, ++it) {
                    const int buf = it & 1, steps = k + 1 < n ? 8 : (last + 15) >> 4;
                    ok = wait(S::kFull + get.at, get.phase) && wait(S::kPReady + buf, (it >> 1) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t a = v_lo + get.at * (S::kItem >> 4), b = p_lo + buf * (S::kPBytes >> 4);
#pragma unroll
                    for (int j = 0; j < kTile / 16; ++j) {
                        if (j >= steps) break;
#pragma unroll
                        for (int m = 0; m < S::kOBlocks; ++m)
                            mma_f16(tmem + S::kTmemO + m * S::kPCols, a + ((m * 2 * (kTile * 128) + j * 2048) >> 4),
                                    hi_v, b + j * (S::kPRow * 16 >> 4), hi_p, id, k > 0 || j > 0);
                    }
                    mma_commit(bar0 + (S::kPFree + buf) * 8);
                    mma_commit(bar0 + (S::kEmpty + get.at) * 8);
                    get.move(it + 2 == count ? 1 : 2);
                }
                x.t += n - 1;
                x.next(p);
            }
            if (gave_up) {
                mma_commit(bar0 + (S::kDrain + 1) * 8);
                mbar_wait(&bars[S::kDrain + 1], 0);
            }
        }
        __syncwarp();
    } else {
        // Softmax: thread tid owns slot tid of each tile, and lane tid of O.
        const float c = p.a.scale * 1.4426950408889634f;
        const uint32_t my_tmem = tmem + ((uint32_t)warp << 21);  // 32 * warp in the address's lane field
        // This slot's row of P: 16-byte chunks, swizzled over the row's width.
        constexpr int kChunks = S::kPRow / 16;
        const int turn = kChunks == 2 ? (tid >> 2) & 1 : (tid >> 1) & 3;
        float m[GP], l[GP];
        Walk x = w;
        bool ok = true;    // false once a wait gave up
        bool leave = false;  // all 128 threads leave at the same barrier
        for (int it = 0; it < count && !leave;) {
            int last;
            const int n = share_of(x, it, &last);
            const int part = p.parts == 1 ? 0 : x.r % p.parts, heads = min(GP, p.group - part * GP);
            const int tile0 = w.s + it;
            for (int k = 0; k < n; ++k, ++it) {
                const int buf = it & 1, valid = k + 1 < n ? kTile : last;
                float s[GP];
                ok = ok && wait(S::kSFull + buf, (it >> 1) & 1);
                __syncwarp();
                tc_fence_after();
#pragma unroll
                for (int g = 0; g < GP; g += 8) tmem_ld8(my_tmem + S::kTmemS + buf * 16 + g, s + g);
                tmem_wait_ld();
                tc_fence_before();
                mbar_arrive_at(bar0 + (S::kSFree + buf) * 8);
                const bool mine = tid < valid;
                bool over = !ok;
#pragma unroll
                for (int g = 0; g < GP; ++g) {
                    if (g >= heads) s[g] = 0.f;  // what a group of fewer heads leaves in its columns
                    if (k > 0) over = over || (mine && s[g] * c > m[g] + kSlack);
                }
                // Some score has passed the reference by kSlack (or there is none yet).
                if (k == 0 || bar_any(1, 128, over)) {
                    leave = bar_any(1, 128, !ok);
                    if (leave) break;
#pragma unroll
                    for (int g = 0; g < GP; ++g) {
                        const float top = warp_max(mine ? s[g] * c : -INFINITY);
                        if (lane == 0) red[warp][g] = top;
                    }
                    bar_sync(1, 128);
                    float f[GP];
#pragma unroll
                    for (int g = 0; g < GP; ++g) {
                        const float top = fmaxf(fmaxf(red[0][g], red[1][g]), fmaxf(red[2][g], red[3][g]));
                        if (k == 0) {
                            m[g] = top;
                            l[g] = 0.f;
                        } else {
                            const float to = fmaxf(m[g], top);
                            f[g] = to == m[g] ? 1.f : exp2_approx(m[g] - to);
                            m[g] = to;
                            l[g] *= f[g];
                        }
                    }
                    if (k > 0) {
                        ok = wait(S::kPFree + (buf ^ 1), ((it - 1) >> 1) & 1);  // the tile before is in O
                        __syncwarp();
                        tc_fence_after();
#pragma unroll
                        for (int o = 0; o < S::kOBlocks * 2; ++o) {  // hi columns and lo columns of each block
                            float v[GP];
                            const uint32_t at = my_tmem + S::kTmemO + o * GP;
#pragma unroll
                            for (int g = 0; g < GP; g += 8) tmem_ld8(at + g, v + g);
                            tmem_wait_ld();
#pragma unroll
                            for (int g = 0; g < GP; ++g) v[g] *= f[g];
#pragma unroll
                            for (int g = 0; g < GP; g += 8) tmem_st8(at + g, v + g);
                            tmem_wait_st();
                        }
                        tc_fence_before();
                    }
                }
#pragma unroll
                for (int g = 0; g < GP; ++g) {
                    const float e = exp2_approx(fmaf(s[g], c, kBias - (m[g] == -INFINITY ? 0.f : m[g])));
                    s[g] = mine ? e : 0.f;
                    l[g] += s[g];
                }
                if (p.p) {
                    float4* to = reinterpret_cast<float4*>(p.p + ((size_t)(tile0 + k) * kTile + tid) * GP);
#pragma unroll
                    for (int g = 0; g < GP; g += 4) to[g / 4] = make_float4(s[g], s[g + 1], s[g + 2], s[g + 3]);
                    if (tid == 0) {
                        float4* tm = reinterpret_cast<float4*>(p.tile_m + (size_t)(tile0 + k) * GP);
#pragma unroll
                        for (int g = 0; g < GP; g += 4) tm[g / 4] = make_float4(m[g], m[g + 1], m[g + 2], m[g + 3]);
                    }
                }
                uint32_t word[GP];  // hi of all heads, then lo
#pragma unroll
                for (int g = 0; g < GP; g += 2) {
                    word[g / 2] = pack2(s[g], s[g + 1], p.c.bf16);
                    const float2 hi = unpack2(word[g / 2], p.c.bf16);
                    word[(GP + g) / 2] = pack2(s[g] - hi.x, s[g + 1] - hi.y, p.c.bf16);
                }
                if (it >= 2) ok = ok && wait(S::kPFree + buf, ((it >> 1) & 1) ^ 1);
                const uint32_t row = p_buf + buf * S::kPBytes + tid * S::kPRow;
#pragma unroll
                for (int i = 0; i < kChunks; ++i)
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(row + ((i ^ turn) << 4)),
                                 "r"(word[4 * i]), "r"(word[4 * i + 1]), "r"(word[4 * i + 2]), "r"(word[4 * i + 3])
                                 : "memory");
                if (valid & 15) {
                    // Rows past the sequence's end inside the last step of 16: zero times NaN is NaN.
                    const int item = it + 1 < count ? 2 * it + 2 : 2 * count - 1, st = item % S::kRing;
                    ok = ok && wait(S::kFull + st, (item / S::kRing) & 1);
                    const int pad = (16 - (valid & 15)) * S::kSub * 8;
                    for (int i = tid; ok && i < pad; i += 128)
                        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                         ring + st * S::kItem + i / 8 % S::kSub * (kTile * 128) +
                                         (valid + i / (S::kSub * 8)) * 128 + (i & 7) * 16),
                                     "r"(0)
                                     : "memory");
                }
                fence_proxy_async_smem();
                mbar_arrive_at(bar0 + (S::kPReady + buf) * 8);
            }
            if (leave) break;

            // The end of the row's share: sums over the 128 slots' threads, then O.
            const int final_it = it - 1;
            const float sum = warp_sums<GP>(l, lane);
            ok = ok && wait(S::kPFree + (final_it & 1), (final_it >> 1) & 1);
            leave = bar_any(1, 128, !ok);
            if (leave) break;
            if ((lane & (32 / GP - 1)) == 0) red[warp][warp_head<GP>(lane)] = sum;
            bar_sync(1, 128);
            tc_fence_after();
            const int row_start = tile0 - x.t;  // tile number of the row's first tile
            const bool whole = row_start >= w.s && row_start + x.tiles <= w.e;
            const int share = 2 * blockIdx.x + (row_start >= w.s ? 1 : 0);
            const int q0 = x.b * p.a.q_heads + (p.parts == 1 ? x.r : x.r / p.parts) * p.group + part * GP;
            float v[S::kOBlocks][2 * GP];
#pragma unroll
            for (int o = 0; o < S::kOBlocks; ++o)
#pragma unroll
                for (int g = 0; g < 2 * GP; g += 8) tmem_ld8(my_tmem + S::kTmemO + o * S::kPCols + g, v[o] + g);
#pragma unroll
            for (int g = 0; g < GP; ++g) l[g] = (red[0][g] + red[1][g]) + (red[2][g] + red[3][g]);
            tmem_wait_ld();
            tc_fence_before();
            if (tid < heads) {
                float mm = m[0], ll = l[0];
#pragma unroll
                for (int g = 1; g < GP; ++g)
                    if (g == tid) {
                        mm = m[g];
                        ll = l[g];
                    }
                if (ll != ll) mm = 0.f;  // a NaN sum says it all: keep it apart from an empty share
                if (whole) {
                    p.row_ml[((size_t)x.b * p.rows + x.r) * GP + tid] = make_float2(mm, ll);
                    if (p.a.lse)
                        p.a.lse[q0 + tid] = ll == 0.f ? -INFINITY : (mm - kBias + log2f(ll)) * 0.6931471805599453f;
                } else {
                    p.part_ml[share * GP + tid] = make_float2(mm, ll);
                }
            }
#pragma unroll
            for (int o = 0; o < S::kOBlocks; ++o) {
                // 64 rows of a product lie in the first 16 lanes of each warp's 32.
                const int d = S::kM == 64 ? warp * 16 + lane : o * 128 + tid;
                if ((S::kM == 64 && lane >= 16) || d >= p.c.dim) continue;
#pragma unroll
                for (int g = 0; g < GP; ++g) {
                    if (g >= heads) break;
                    const float y = v[o][g] + v[o][GP + g];
                    if (whole)
                        p.a.out[(size_t)(q0 + g) * p.c.dim + d] =
                            from_float(l[g] == 0.f ? 0.f : y * __frcp_rn(l[g]), p.c.bf16);
                    else
                        p.part_o[((size_t)share * GP + g) * p.c.dim + d] = y;
                }
            }
            x.t += n - 1;
            x.next(p);
        }
    }
    __syncthreads();
    tc_fence_after();
    if (warp == 5) tmem_dealloc(tmem, S::kTmemCols);
}

// Joins the rows that several blocks share, writes what sequences without
// slots give, and adds the shares to the weights.  Block c takes the tiles
// that block c of the first launch had, so its p may still be in L2.
template <int GP>
__global__ void __launch_bounds__(kJoinThreads) kv_join_kernel(const AttendArgs p) {
    constexpr int kWarps = kJoinThreads / 32;
    __shared__ int scan[kWarps + 8];
    __shared__ float2 ml[GP];
    __shared__ float acc[kJoinThreads];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Walk w = find_range<kJoinThreads>(p, scan);
    for (int b = blockIdx.x; b < p.c.seqs; b += gridDim.x) {
        if (p.c.len(b) > 0) continue;
        for (int i = tid; i < p.a.q_heads * p.c.dim; i += kJoinThreads)
            p.a.out[(size_t)b * p.a.q_heads * p.c.dim + i] = 0;
        if (p.a.lse)
            for (int i = tid; i < p.a.q_heads; i += kJoinThreads) p.a.lse[(size_t)b * p.a.q_heads + i] = -INFINITY;
    }
    grid_dependency_wait();
    int tile = w.s;
    while (tile < w.e) {
        const int count = min(w.tiles - w.t, w.e - tile);  // this block's tiles of the row
        const int row_start = tile - w.t, part = w.r % p.parts, h = w.r / p.parts;
        const int c0 = w.block_of(row_start), c1 = w.block_of(row_start + w.tiles - 1);
        // Statistics of part `pt` of the row's group into ml[]: reference and sum (0 for an empty row).
        auto stats = [&](int pt) {
            const int start = row_start + (pt - part) * w.tiles;
            const int a0 = w.block_of(start), a1 = w.block_of(start + w.tiles - 1);
            const int heads = min(GP, p.group - pt * GP);
            __syncthreads();
            for (int g = warp; g < heads; g += kWarps) {
                float top = -INFINITY, sum = 0.f;
                if (a0 == a1) {
                    const float2 v = p.row_ml[((size_t)w.b * p.rows + h * p.parts + pt) * GP + g];
                    top = v.x;
                    sum = v.y;
                } else {
                    for (int c = a0 + lane; c <= a1; c += 32) {
                        const float2 v = p.part_ml[(2 * c + (c == a0)) * GP + g];
                        if (v.x == -INFINITY) continue;
                        const float to = fmaxf(top, v.x);
                        sum = (top == -INFINITY ? 0.f : sum * exp2f(top - to)) + v.y * exp2f(v.x - to);
                        top = to;
                    }
                    const float all = warp_max(top);
                    sum = top == -INFINITY ? 0.f : sum * exp2f(top - all);
                    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(kFullMask, sum, d);
                    top = all;
                }
                if (lane == 0) ml[g] = make_float2(top, sum);
            }
            __syncthreads();
        };
        const bool weights = p.p && part == 0;
        if (c0 != c1 || weights) stats(part);
        if (c0 != c1) {
            const int heads = min(GP, p.group - part * GP);
            const int q0 = w.b * p.a.q_heads + h * p.group + part * GP;
            const int block = blockIdx.x;
            if (block == c0 && tid < heads && p.a.lse)
                p.a.lse[q0 + tid] = ml[tid].y == 0.f ? -INFINITY
                                                     : (ml[tid].x - kBias + log2f(ml[tid].y)) * 0.6931471805599453f;
            // The row's blocks share out the output's elements; a block's
            // threads share its elements, and the row's pieces where threads are left.
            const int elements = heads * p.c.dim, blocks = c1 - c0 + 1;
            const int each = (elements + blocks - 1) / blocks;
            const int width = each > 256 ? 512 : each > 128 ? 256 : each > 64 ? 128 : each > 32 ? 64 : 32;
            const int ways = kJoinThreads / width, from = (block - c0) * each, to = min(from + each, elements);
            for (int e0 = from; e0 < to; e0 += width) {
                const int i = e0 + tid % width, g = min(i / p.c.dim, heads - 1);
                const float top = ml[g].x;
                float o = 0.f;
                if (i < to)
#pragma unroll 4
                    for (int c = c0 + tid / width; c <= c1; c += ways) {
                        const int share = 2 * c + (c == c0);
                        const float x = p.part_ml[share * GP + g].x, v = p.part_o[(size_t)share * GP * p.c.dim + i];
                        o += x == -INFINITY ? 0.f : v * exp2f(x - top);
                    }
                if (ways > 1) {
                    __syncthreads();
                    acc[tid] = o;
                    __syncthreads();
                    if (tid < width)
                        for (int k = 1; k < ways; ++k) o += acc[k * width + tid];
                }
                if (tid < width && i < to)
                    p.a.out[(size_t)q0 * p.c.dim + i] = from_float(ml[g].y == 0.f ? 0.f : o / ml[g].y, p.c.bf16);
            }
        }
        if (weights) {
            const float* wi = p.a.weight.row(w.b, h);
            float* wo = p.a.weight_out.row(w.b, h);
            for (int pt = 0; pt < p.parts; ++pt) {
                if (pt > 0) stats(pt);
                const int heads = min(GP, p.group - pt * GP);
                const float2 mine = lane < heads ? ml[lane] : make_float2(0.f, 0.f);
                for (int k = warp; k < count; k += kWarps) {
                    // A warp takes a tile; all its loads are in flight at once.
                    const size_t x = tile + k + (size_t)pt * w.tiles;
                    const int slot0 = (w.t + k) * kTile + lane;
                    const float4* v = reinterpret_cast<const float4*>(p.p + (x * kTile + lane) * GP);
                    const float tm = lane < heads ? p.tile_m[x * GP + lane] : -INFINITY;
                    float4 y[4][GP / 4];
                    float old[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
#pragma unroll
                        for (int g = 0; g < GP / 4; ++g) y[i][g] = v[i * 32 * (GP / 4) + g];
                        const int slot = slot0 + i * 32;
                        old[i] = slot < w.n ? (pt == 0 ? wi[slot] : wo[slot]) : 0.f;
                    }
                    float f = 0.f;
                    if (tm != -INFINITY && mine.y != 0.f) f = exp2f(tm - mine.x) / mine.y;
#pragma unroll
                    for (int g = 0; g < GP; ++g) {
                        const float fg = __shfl_sync(kFullMask, f, g);
                        if (g >= heads) continue;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float4 q = y[i][g / 4];
                            old[i] = fmaf(g % 4 == 0 ? q.x : g % 4 == 1 ? q.y : g % 4 == 2 ? q.z : q.w, fg, old[i]);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (slot0 + i * 32 < w.n) wo[slot0 + i * 32] = old[i];
                }
            }
        }
        tile += count;
        w.t += count - 1;
        w.next(p);
    }
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_fn() {
    static const EncodeTiled fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) !=
                cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeTiled>(f);
    }();
    return fn;
}

// A map of 16-bit elements with dense rows of `size[0]`, copied in boxes 64 elements wide.
cudaError_t make_map(CUtensorMap* map, const void* base, bool bf16, int rank, const cuuint64_t* size,
                     const long long* stride, const cuuint32_t* box) {
    const EncodeTiled fn = encode_fn();
    if (!fn) return cudaErrorNotSupported;
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    cuuint64_t bytes[3];
    for (int i = 0; i < rank - 1; ++i) bytes[i] = (cuuint64_t)stride[i] * 2;
    const CUresult r = fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank,
                          const_cast<void*>(base), size, bytes, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

int group_part(const KvCache& c, const KvAttend& a) { return a.q_heads / c.heads <= 8 ? 8 : 16; }

int sm_count(int device) {
    static int counts[64];
    if (device < 0 || device >= 64) return 152;
    if (!counts[device]) cudaDeviceGetAttribute(&counts[device], cudaDevAttrMultiProcessorCount, device);
    return counts[device];
}

// The plan of a call, and its scratch when `scratch` is given.
struct Plan {
    AttendArgs args;
    int blocks;
    size_t bytes;
};

Plan make_plan(int device, const KvCache& c, const KvAttend& a, void* scratch) {
    Plan plan;
    AttendArgs& p = plan.args;
    const int gp = group_part(c, a);
    p = {c, a};
    p.group = a.q_heads / c.heads;
    p.parts = (p.group + gp - 1) / gp;
    p.rows = c.heads * p.parts;
    p.box = c.page_size & -c.page_size;
    if (p.box > kTile) p.box = kTile;
    const size_t rows = (size_t)c.seqs * p.rows, tiles = rows * ((c.capacity() + kTile - 1) / kTile);
    plan.blocks = sm_count(device);
    if ((size_t)plan.blocks > tiles) plan.blocks = (int)tiles;
    char* at = static_cast<char*>(scratch);
    size_t bytes = 0;
    auto take = [&](size_t n) {
        char* q = at ? at + bytes : nullptr;
        bytes += (n + 255) & ~size_t(255);
        return static_cast<void*>(q);
    };
    p.part_o = static_cast<float*>(take(2ull * plan.blocks * gp * c.dim * 4));
    p.part_ml = static_cast<float2*>(take(2ull * plan.blocks * gp * 8));
    p.row_ml = static_cast<float2*>(take(rows * gp * 8));
    p.p = nullptr;
    p.tile_m = nullptr;
    if (a.weight.data) {
        p.p = static_cast<float*>(take(tiles * kTile * gp * 4));
        p.tile_m = static_cast<float*>(take(tiles * gp * 4));
    }
    plan.bytes = bytes;
    return plan;
}

template <int DP, int GP>
cudaError_t launch(const Plan& plan, cudaStream_t s, const CUtensorMap* maps, int* launches) {
    using Sh = Shape<DP, GP>;
    auto kernel = kv_attend_kernel<DP, GP>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Sh::kSmem);
    if (e != cudaSuccess) return e;
    kernel<<<plan.blocks, kThreads, Sh::kSmem, s>>>(plan.args, maps[0], maps[1], maps[2]);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    ++*launches;
    e = launch_pdl(kv_join_kernel<GP>, dim3(plan.blocks), dim3(kJoinThreads), 0, s, plan.args);
    if (e == cudaSuccess) ++*launches;
    return e;
}

}  // namespace

size_t kv_attend_scratch(int device, const KvCache& c, const KvAttend& a) {
    return make_plan(device, c, a, nullptr).bytes;
}

cudaError_t kv_attend_launch(int device, cudaStream_t s, const KvCache& c, const KvAttend& a, void* scratch,
                             unsigned* status, int* launches) {
    Plan plan = make_plan(device, c, a, scratch);
    plan.args.status = status;
    const int gp = group_part(c, a);
    CUtensorMap maps[3];
    const cuuint64_t pool[4] = {(cuuint64_t)c.dim, (cuuint64_t)c.page_size, (cuuint64_t)c.heads, (cuuint64_t)c.pages};
    const cuuint32_t pool_box[4] = {64, (cuuint32_t)plan.args.box, 1, 1};
    const cuuint64_t queries[3] = {(cuuint64_t)c.dim, (cuuint64_t)a.q_heads, (cuuint64_t)c.seqs};
    const cuuint32_t query_box[3] = {64, (cuuint32_t)gp, 1};
    const long long ks[3] = {c.ks[1], c.ks[2], c.ks[0]}, vs[3] = {c.vs[1], c.vs[2], c.vs[0]}, qs[2] = {a.qs[1], a.qs[0]};
    cudaError_t e = make_map(&maps[0], c.k, c.bf16, 4, pool, ks, pool_box);
    if (e == cudaSuccess) e = make_map(&maps[1], c.v, c.bf16, 4, pool, vs, pool_box);
    if (e == cudaSuccess) e = make_map(&maps[2], a.q, c.bf16, 3, queries, qs, query_box);
    if (e != cudaSuccess) return e;
    if (c.dim <= 64) return gp == 8 ? launch<64, 8>(plan, s, maps, launches) : launch<64, 16>(plan, s, maps, launches);
    if (c.dim <= 128) return gp == 8 ? launch<128, 8>(plan, s, maps, launches) : launch<128, 16>(plan, s, maps, launches);
    return gp == 8 ? launch<256, 8>(plan, s, maps, launches) : launch<256, 16>(plan, s, maps, launches);
}

}  // namespace topk
