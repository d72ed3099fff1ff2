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
constexpr int kThreads = 192;    // 4 softmax warps, the copy warp, the product warp
constexpr int kJoinThreads = 256;
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
    static constexpr int kPBytes = kPCols * kTile * 2;
    static constexpr int kM = DP == 64 ? 64 : 128;        // rows of one second product
    static constexpr int kOBlocks = DP / kM;
    static constexpr int kTmemS = 0, kTmemO = 32;         // columns: two S buffers of 16, then O
    static constexpr int kTmemCols = 32 + kOBlocks * kPCols <= 64 ? 64 : 128;
    static constexpr size_t kSmem = 1024 + kRingBytes + 2 * kQBytes + 2 * kPBytes;
};

struct Barriers {
    uint64_t full[12], empty[12];
    uint64_t s_full[2], s_free[2], p_ready[2], p_free[2], q_full[2], q_free[2];
    uint64_t drain;
};

template <int DP, int GP>
__global__ void __launch_bounds__(kThreads, 1)
kv_attend_kernel(const AttendArgs p, const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                 const __grid_constant__ CUtensorMap map_q) {
    using S = Shape<DP, GP>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* ring = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    unsigned char* q_buf = ring + kRingBytes;
    unsigned char* p_buf = q_buf + 2 * S::kQBytes;
    __shared__ Barriers bar;
    __shared__ uint32_t tmem_at;
    __shared__ int scan[kThreads / 32 + 8];
    __shared__ __align__(16) float red[2][4][GP];
    __shared__ volatile int gave_up;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i < S::kRing; ++i) {
            mbar_init(&bar.full[i], 1);
            mbar_init(&bar.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.s_full[i], 1);
            mbar_init(&bar.s_free[i], 128);
            mbar_init(&bar.p_ready[i], 128);
            mbar_init(&bar.p_free[i], 1);
            mbar_init(&bar.q_full[i], 1);
            mbar_init(&bar.q_free[i], 1);
        }
        mbar_init(&bar.drain, 1);
        mbar_init_fence();
        gave_up = 0;
    }
    if (warp == 5) tmem_alloc(&tmem_at, S::kTmemCols);
    launch_dependents();  // the join waits for this launch's end before it reads anything of it
    Walk w = find_range<kThreads>(p, scan);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_at;
    const int count = w.e - w.s;  // tiles of this block

    // A bounded wait; after one gave up, every other gives up too.
    auto wait = [&](uint64_t* b, uint32_t parity) {
        for (int i = 0; i < kWaitSpins; ++i) {
            if (mbar_try_wait(b, parity)) return true;
            if (gave_up) return false;
        }
        gave_up = 1;
        atomicOr(p.status, kStatusWaitTimeout);
        return false;
    };

    if (warp == 4) {
        // Copies, in the order in which the products use them:
        // K(0), K(1), V(0), K(2), V(1), ..., V(count - 1).
        const uint64_t policy = l2_evict_first_policy();
        constexpr int kPer = (16 * S::kSub + 31) / 32;  // copies of a lane, at most
        struct Tile {
            int row, b, slot0, copies;
            int page[kPer];
        };
        // The pages of a tile, fetched a tile ahead of their use: the load
        // takes as long as a third of a tile's copy.
        auto fetch = [&](const Walk& x, Tile& t) {
            t.row = x.r;
            t.b = x.b;
            t.slot0 = x.t * kTile;
            t.copies = (min(kTile, x.n - t.slot0) + p.box - 1) / p.box * S::kSub;
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const int i = j * 32 + lane;
                t.page[j] = p.c.pages;  // outside the pool: reads as zeros
                if (i < t.copies) {
                    const int at = p.c.page_of(t.b, t.slot0 + i / S::kSub * p.box);
                    if (at >= 0) t.page[j] = at;
                }
            }
        };
        int item = 0, piece = -1, q_loads = 0;
        auto wait_warp = [&](uint64_t* b, uint32_t parity) { return __all_sync(kFullMask, wait(b, parity)); };
        auto load = [&](const Tile& t, const CUtensorMap* map) {
            const int st = item % S::kRing;
            if (item >= S::kRing && !wait_warp(&bar.empty[st], ((item / S::kRing) - 1) & 1)) return false;
            if (lane == 0) mbar_arrive_expect_tx(&bar.full[st], t.copies * p.box * 128);
            __syncwarp();
            unsigned char* dst = ring + st * S::kItem;
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const int i = j * 32 + lane;
                if (i < t.copies) {
                    const int box = i / S::kSub, sub = i % S::kSub;
                    tma_load_4d(dst + sub * (kTile * 128) + box * p.box * 128, map, sub * 64,
                                (t.slot0 + box * p.box) % p.c.page_size, t.row / p.parts, t.page[j], &bar.full[st],
                                policy);
                }
            }
            ++item;
            return true;
        };
        Walk x = w;
        Tile before, now, after;
        if (count > 0) fetch(x, now);
        for (int it = 0; it <= count; ++it) {
            if (it + 1 < count) {
                x.next(p);
                fetch(x, after);
            }
            if (it < count) {
                if (it == 0 || now.slot0 == 0) {
                    ++piece;
                    if (piece >= 2 && !wait_warp(&bar.q_free[piece & 1], ((piece - 2) >> 1) & 1)) break;
                    if (lane == 0) {
                        uint64_t* b = &bar.q_full[piece & 1];
                        mbar_arrive_expect_tx(b, S::kSub * GP * 128);
                        for (int sub = 0; sub < S::kSub; ++sub)
                            tma_load_3d(q_buf + (piece & 1) * S::kQBytes + sub * 16 * 128, &map_q, sub * 64,
                                        now.row / p.parts * p.group + now.row % p.parts * GP, now.b, b);
                    }
                    ++q_loads;
                    __syncwarp();
                }
                if (!load(now, &map_k)) break;
            }
            if (it > 0 && !load(before, &map_v)) break;
            before = now;
            now = after;
        }
        __syncwarp();
        if (gave_up) {  // wait for the copies in flight, so that none lands after the block's end
            for (int i = max(0, item - S::kRing); i < item; ++i) mbar_wait(&bar.full[i % S::kRing], (i / S::kRing) & 1);
            for (int i = max(0, q_loads - 2); i < q_loads; ++i) mbar_wait(&bar.q_full[i & 1], (i >> 1) & 1);
        }
    } else if (warp == 5) {
        if (lane == 0 && count > 0) {
            // Products: S(0), S(1), O(0), S(2), O(1), ...
            const uint32_t id_s = mma_idesc(p.c.bf16, kTile, 16, false);
            const uint32_t id_o = mma_idesc(p.c.bf16, S::kM, S::kPCols, true);
            int item = 0, piece = -1;
            Walk x = w, y = w;  // the tiles of S and of O
            bool y_first = true;
            for (int it = 0; it <= count; ++it) {
                if (it < count) {
                    const int buf = it & 1, st = item % S::kRing;
                    if (it == 0 || x.t == 0) {
                        ++piece;
                        if (!wait(&bar.q_full[piece & 1], (piece >> 1) & 1)) break;
                    }
                    if (!wait(&bar.full[st], (item / S::kRing) & 1)) break;
                    if (it >= 2 && !wait(&bar.s_free[buf], ((it - 2) >> 1) & 1)) break;
                    tc_fence_after();
                    const uint32_t ka = smem_addr(ring + st * S::kItem);
                    const uint32_t qa = smem_addr(q_buf + (piece & 1) * S::kQBytes);
#pragma unroll
                    for (int j = 0; j < DP / 16; ++j)
                        mma_f16(tmem + S::kTmemS + buf * 16,
                                smem_desc_sw128(ka + (j >> 2) * (kTile * 128) + (j & 3) * 32, 16, 1024),
                                smem_desc_sw128(qa + (j >> 2) * (16 * 128) + (j & 3) * 32, 16, 1024), id_s, j > 0);
                    mma_commit(&bar.s_full[buf]);
                    mma_commit(&bar.empty[st]);
                    const bool last = x.t + 1 == x.tiles;
                    if (last) mma_commit(&bar.q_free[piece & 1]);
                    x.next(p);
                    ++item;
                }
                if (it > 0) {
                    const int t = it - 1, buf = t & 1, st = item % S::kRing;
                    if (!wait(&bar.full[st], (item / S::kRing) & 1)) break;
                    if (!wait(&bar.p_ready[buf], (t >> 1) & 1)) break;
                    tc_fence_after();
                    const int valid = min(kTile, y.n - y.t * kTile), steps = (valid + 15) / 16;
                    const uint32_t va = smem_addr(ring + st * S::kItem), pa = smem_addr(p_buf + buf * S::kPBytes);
                    for (int j = 0; j < steps; ++j) {
                        const uint64_t db =
                            smem_desc_sw128(pa + (j >> 2) * (S::kPCols * 128) + (j & 3) * 32, 16, 1024);
#pragma unroll
                        for (int m = 0; m < S::kOBlocks; ++m)
                            mma_f16(tmem + S::kTmemO + m * S::kPCols,
                                    smem_desc_sw128(va + m * 2 * (kTile * 128) + j * 2048, kTile * 128, 1024), db,
                                    id_o, !y_first || j > 0);
                    }
                    mma_commit(&bar.empty[st]);
                    mma_commit(&bar.p_free[buf]);
                    y_first = y.t + 1 == y.tiles;
                    y.next(p);
                    ++item;
                }
            }
            if (gave_up) {  // wait for the products in flight
                mma_commit(&bar.drain);
                mbar_wait(&bar.drain, 0);
            }
        }
        __syncwarp();
    } else {
        // Softmax: thread tid owns slot tid of each tile, and lane tid of O.
        const float c = p.a.scale * 1.4426950408889634f;
        const uint32_t lane_base = (uint32_t)warp << 21;  // 32 * warp in the address's lane field
        float m[GP], l[GP];
        Walk x = w;
        bool ok = true;  // false once a wait gave up; all 128 threads leave at the next barrier
        for (int it = 0; it < count; ++it, x.next(p)) {
            const int buf = it & 1, slot0 = x.t * kTile, valid = min(kTile, x.n - slot0);
            const bool first = it == 0 || x.t == 0;
            const int part = x.r % p.parts, heads = min(GP, p.group - part * GP);
            float s[GP];
            ok = ok && wait(&bar.s_full[buf], (it >> 1) & 1);
            __syncwarp();
            tc_fence_after();
#pragma unroll
            for (int g = 0; g < GP; g += 8) tmem_ld8(tmem + lane_base + S::kTmemS + buf * 16 + g, s + g);
            tmem_wait_ld();
            tc_fence_before();
            mbar_arrive(&bar.s_free[buf]);
            const bool mine = tid < valid;
#pragma unroll
            for (int g = 0; g < GP; ++g) {
                const float top = warp_max(mine && g < heads ? s[g] * c : -INFINITY);
                if (lane == 0) red[buf][warp][g] = top;
            }
            if (!bar_all(1, 128, ok)) break;
            float top[GP];
            bool up = false;
#pragma unroll
            for (int g = 0; g < GP; ++g) {
                top[g] = fmaxf(fmaxf(red[buf][0][g], red[buf][1][g]), fmaxf(red[buf][2][g], red[buf][3][g]));
                if (first) {
                    m[g] = top[g];
                    l[g] = 0.f;
                }
                up = up || top[g] > m[g] + kSlack;
            }
            if (up) {  // the same for all 128 threads; the tile before has to be in O
                ok = wait(&bar.p_free[buf ^ 1], ((it - 1) >> 1) & 1);
                __syncwarp();
                tc_fence_after();
                float f[GP];
#pragma unroll
                for (int g = 0; g < GP; ++g) {
                    const float to = fmaxf(m[g], top[g]);
                    f[g] = to == m[g] ? 1.f : exp2_approx(m[g] - to);
                    m[g] = to;
                    l[g] *= f[g];
                }
#pragma unroll
                for (int o = 0; o < S::kOBlocks * 2; ++o) {  // the hi columns, then the lo columns, of each block
                    float v[GP];
                    const uint32_t at = tmem + lane_base + S::kTmemO + o * GP;
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
#pragma unroll
            for (int g = 0; g < GP; ++g) {
                const float ref = m[g] == -INFINITY ? 0.f : m[g];
                s[g] = mine && g < heads ? exp2_approx(fmaf(s[g], c, kBias - ref)) : 0.f;
                l[g] += s[g];
            }
            if (p.p) {
                float* to = p.p + ((size_t)(w.s + it) * kTile + tid) * GP;
#pragma unroll
                for (int g = 0; g < GP; g += 4)
                    *reinterpret_cast<float4*>(to + g) = make_float4(s[g], s[g + 1], s[g + 2], s[g + 3]);
                if (tid == 0)
#pragma unroll
                    for (int g = 0; g < GP; ++g) p.tile_m[(size_t)(w.s + it) * GP + g] = m[g];
            }
            if (it >= 2) ok = ok && wait(&bar.p_free[buf], ((it - 2) >> 1) & 1);
            unsigned char* pb = p_buf + buf * S::kPBytes + (tid >> 6) * (S::kPCols * 128) + (tid & 7) * 2;
#pragma unroll
            for (int g = 0; g < GP; ++g) {
                uint16_t hi, lo;
                if (p.c.bf16) {
                    hi = from_float(s[g], 1);
                    lo = from_float(s[g] - __uint_as_float((unsigned)hi << 16), 1);
                } else {
                    hi = from_float(s[g], 0);
                    lo = from_float(s[g] - __half2float(__ushort_as_half(hi)), 0);
                }
                const int at = (((tid & 63) >> 3) ^ (g & 7)) << 4;
                *reinterpret_cast<uint16_t*>(pb + g * 128 + at) = hi;
                *reinterpret_cast<uint16_t*>(pb + (GP + g) * 128 + at) = lo;
            }
            // The tile's copy in the ring: V(t) is item 2t + 2, but the last one is 2 * count - 1.
            if (valid & 15) {
                // Rows past the sequence's end inside the last step of 16: zero times NaN is NaN.
                const int item_v = it + 1 < count ? 2 * it + 2 : 2 * count - 1;
                ok = ok && wait(&bar.full[item_v % S::kRing], (item_v / S::kRing) & 1);
                unsigned char* v = ring + (item_v % S::kRing) * S::kItem;
                const int pad = (16 - (valid & 15)) * S::kSub * 8;
                for (int i = tid; ok && i < pad; i += 128) {
                    const int row = valid + i / (S::kSub * 8), sub = i / 8 % S::kSub;
                    *reinterpret_cast<int4*>(v + sub * (kTile * 128) + row * 128 + (i & 7) * 16) = make_int4(0, 0, 0, 0);
                }
            }
            fence_proxy_async_smem();
            mbar_arrive(&bar.p_ready[buf]);
            if (x.t + 1 < x.tiles && it + 1 < count) continue;

            // The end of the row's share: sums over the 128 slots' threads, then O.
#pragma unroll
            for (int g = 0; g < GP; ++g)
                for (int d = 16; d; d >>= 1) l[g] += __shfl_xor_sync(kFullMask, l[g], d);
            if (!bar_all(1, 128, ok)) break;  // and red is free again
            if (lane == 0)
#pragma unroll
                for (int g = 0; g < GP; ++g) red[buf][warp][g] = l[g];
            ok = wait(&bar.p_free[buf], (it >> 1) & 1);
            if (!bar_all(1, 128, ok)) break;
#pragma unroll
            for (int g = 0; g < GP; ++g)
                l[g] = (red[buf][0][g] + red[buf][1][g]) + (red[buf][2][g] + red[buf][3][g]);
            tc_fence_after();
            const int row_start = w.s + it - x.t;  // tile number of the row's first tile
            const bool whole = row_start >= w.s && row_start + x.tiles <= w.e;
            const int share = 2 * blockIdx.x + (row_start >= w.s ? 1 : 0);
            const int q0 = x.b * p.a.q_heads + x.r / p.parts * p.group + part * GP;
            if (tid < heads) {
                float mm = m[0], ll = l[0];
#pragma unroll
                for (int g = 1; g < GP; ++g)
                    if (g == tid) {
                        mm = m[g];
                        ll = l[g];
                    }
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
                float hi[GP], lo[GP];
                const uint32_t at = tmem + lane_base + S::kTmemO + o * S::kPCols;
#pragma unroll
                for (int g = 0; g < GP; g += 8) {
                    tmem_ld8(at + g, hi + g);
                    tmem_ld8(at + GP + g, lo + g);
                }
                tmem_wait_ld();
                // 64 rows of a product lie in the first 16 lanes of each warp's 32.
                const int d = S::kM == 64 ? warp * 16 + lane : o * 128 + tid;
                if ((S::kM == 64 && lane >= 16) || d >= p.c.dim) continue;
#pragma unroll
                for (int g = 0; g < GP; ++g) {
                    if (g >= heads) continue;
                    const float v = hi[g] + lo[g];
                    if (whole)
                        p.a.out[(size_t)(q0 + g) * p.c.dim + d] = from_float(l[g] == 0.f ? 0.f : v / l[g], p.c.bf16);
                    else
                        p.part_o[((size_t)share * GP + g) * p.c.dim + d] = v;
                }
            }
            tc_fence_before();
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
    __shared__ int scan[kJoinThreads / 32 + 8];
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
        // Statistics of part `pt` of the row's group into ml[]: reference and 1 / sum (0 for an empty row).
        auto stats = [&](int pt) {
            const int start = row_start + (pt - part) * w.tiles;
            const int a0 = w.block_of(start), a1 = w.block_of(start + w.tiles - 1);
            const int heads = min(GP, p.group - pt * GP);
            __syncthreads();
            for (int g = warp; g < heads; g += kJoinThreads / 32) {
                float top = -INFINITY, sum = 0.f;
                if (a0 == a1) {
                    const float2 v = p.row_ml[((size_t)w.b * p.rows + h * p.parts + pt) * GP + g];
                    top = v.x;
                    sum = v.y;
                } else {
                    for (int c = a0 + lane; c <= a1; c += 32) top = fmaxf(top, p.part_ml[(2 * c + (c == a0)) * GP + g].x);
                    for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, d));
                    for (int c = a0 + lane; c <= a1; c += 32) {
                        const float2 v = p.part_ml[(2 * c + (c == a0)) * GP + g];
                        if (v.x != -INFINITY) sum += v.y * exp2f(v.x - top);
                    }
                    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(kFullMask, sum, d);
                }
                if (lane == 0) ml[g] = make_float2(top, sum);
            }
            __syncthreads();
        };
        stats(part);
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
            const int width = each > 128 ? 256 : each > 64 ? 128 : each > 32 ? 64 : 32, ways = kJoinThreads / width;
            const int from = (block - c0) * each, to = min(from + each, elements);
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
                __syncthreads();
                acc[tid] = o;
                __syncthreads();
                if (tid < width && i < to) {
                    for (int k = 1; k < ways; ++k) o += acc[k * width + tid];
                    p.a.out[(size_t)q0 * p.c.dim + i] = from_float(ml[g].y == 0.f ? 0.f : o / ml[g].y, p.c.bf16);
                }
            }
        }
        if (p.p && part == 0) {
            const float* wi = p.a.weight.row(w.b, h);
            float* wo = p.a.weight_out.row(w.b, h);
            for (int pt = 0; pt < p.parts; ++pt) {
                if (pt > 0) stats(pt);
                const int heads = min(GP, p.group - pt * GP);
                for (int k = warp; k < count; k += kJoinThreads / 32) {
                    const size_t x = tile + k + (size_t)pt * w.tiles;
                    float f[GP];
#pragma unroll
                    for (int g = 0; g < GP; ++g) {
                        f[g] = 0.f;
                        if (g < heads) {
                            const float tm = p.tile_m[x * GP + g];
                            if (tm != -INFINITY && ml[g].y != 0.f) f[g] = exp2f(tm - ml[g].x) / ml[g].y;
                        }
                    }
                    for (int i = 0; i < 4; ++i) {
                        const int in = i * 32 + lane, slot = (w.t + k) * kTile + in;
                        if (slot >= w.n) break;
                        const float4* v = reinterpret_cast<const float4*>(p.p + (x * kTile + in) * GP);
                        float sum = 0.f;
#pragma unroll
                        for (int g = 0; g < GP; g += 4) {
                            const float4 y = v[g / 4];
                            sum += y.x * f[g] + y.y * f[g + 1] + y.z * f[g + 2] + y.w * f[g + 3];
                        }
                        wo[slot] = (pt == 0 ? wi[slot] : wo[slot]) + sum;
                    }
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
    static_assert(Sh::kRing <= 12, "ring barriers");
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
