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
// finished there; the shares of a row that several blocks have are joined by
// the last of them to finish (no block waits for another).  With weights, the
// p are stored, and a second launch adds them up once the sums are known.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "topk_device.cuh"
#include "topk_kv.cuh"
#include "topk_tcgen05.cuh"

namespace topk {
namespace {

constexpr int kTile = 128;       // slots of a tile
constexpr int kThreads = 256;    // 4 softmax warps, copies of keys, of values, and the two products
constexpr int kSoftmax = 128;    // threads of the softmax
constexpr int kCopyK = 4, kCopyV = 5, kMmaS = 6, kMmaO = 7;  // warps
constexpr int kWeightThreads = 256;
constexpr int kJoin = 16;        // shares that one block joins at most
constexpr float kSlack = 8.f;    // p <= 2^(kSlack + kBias) = 2^15: within f16's range
constexpr float kBias = 7.f;     // and f16's smallest step, 2^-24, is 2^-31 of the largest p
constexpr int kRingBytes = 192 * 1024;

__device__ __forceinline__ uint16_t from_float(float x, int bf16) {
    return bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(x)) : __half_as_ushort(__float2half_rn(x));
}

static_assert(kKvCounters / 6 <= kJoin * kJoin, "a row's pieces are joined in two steps");

struct AttendArgs {
    KvCache c;
    KvAttend a;
    int group;     // query heads of a key-value head
    int parts;     // parts of at most GP query heads that a group is cut into
    int rows;      // heads * parts: rows of a sequence
    int box;       // slots that one copy takes: a power of two that divides page_size
    float* part_o;    // [2 * blocks][GP][dim]: unnormalised output of a row's share
    float2* part_ml;  // [2 * blocks][GP]: its reference and sum
    float2* row_ml;   // [seqs * rows][GP]: the same of finished rows
    unsigned* done;   // [3 * blocks]: shares that have arrived, zero before and after
    unsigned* clear;  // the next call's, cleared here in case a call before was cut short
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
    static constexpr int kPCols = GP <= 8 ? 16 : 2 * GP;  // hi of every head, then lo; the rest is not looked at
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
__device__ __forceinline__ int warp_head(int lane) { return lane / (32 / GP); }

// N numbers as 16-bit elements hi and lo = p - hi, all hi and then all lo.
template <bool BF16, int N>
__device__ __forceinline__ void split(const float (&p)[N], uint32_t* words) {
    uint16_t e[2 * N];
#pragma unroll
    for (int g = 0; g < N; ++g) {
        if constexpr (BF16) {
            const __nv_bfloat16 hi = __float2bfloat16_rn(p[g]);
            e[g] = __bfloat16_as_ushort(hi);
            e[N + g] = __bfloat16_as_ushort(__float2bfloat16_rn(p[g] - __bfloat162float(hi)));
        } else {
            const __half hi = __float2half_rn(p[g]);
            e[g] = __half_as_ushort(hi);
            e[N + g] = __half_as_ushort(__float2half_rn(p[g] - __half2float(hi)));
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) words[i] = (uint32_t)e[2 * i] | (uint32_t)e[2 * i + 1] << 16;
}

// N consecutive floats, as wide as they come.
template <int N>
__device__ __forceinline__ void store_row(float* to, const float (&v)[N]) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int g = 0; g < N; g += 4)
            *reinterpret_cast<float4*>(to + g) = make_float4(v[g], v[g + 1], v[g + 2], v[g + 3]);
    } else {
#pragma unroll
        for (int g = 0; g < N; ++g) to[g] = v[g];
    }
}

// kBias - m, what is added to a scaled score; a head without a score above
// -inf yet gets a number that makes any such score pass kSlack.
__device__ __forceinline__ float offset_of(float m) { return m > -INFINITY ? kBias - m : 3.4e38f; }

__device__ __forceinline__ float lse_of(float2 ml) {
    return ml.y == 0.f ? -INFINITY : (ml.x - kBias + log2f(ml.y)) * 0.6931471805599453f;
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
    __shared__ float factor[kJoin][GP];
    __shared__ float2 joined[GP];
    __shared__ unsigned arrived;
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
    if (warp == kCopyK && lane == 0) {
        prefetch_map(&map_k);
        prefetch_map(&map_q);
    }
    if (warp == kCopyV && lane == 0) prefetch_map(&map_v);
    if (tid < 3) p.clear[blockIdx.x * 3 + tid] = 0;
    if (warp == kMmaS) tmem_alloc(&tmem_at, S::kTmemCols);
    launch_dependents();  // the weights' launch waits for this one's end before it reads anything of it
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

    if (warp == kCopyK || warp == kCopyV) {
        // Copies into the ring, in the order in which the products use them:
        // K(0), K(1), V(0), K(2), V(1), ..., V(count - 1).  One warp has the
        // keys, one the values: a copy takes its issuer some 50 clocks, and a
        // tile of small pages is many copies.
        const bool keys = warp == kCopyK;
        const CUtensorMap* map = keys ? &map_k : &map_v;
        const uint64_t policy = l2_evict_first_policy();
        // Lane i holds the page of the tile's i-th box, fetched a tile ahead
        // of its use: the load takes as long as a third of a tile's copy.  A
        // lane's slot moves by a tile at a time, so that only a new row divides.
        int index = 0, in = 0, page, page_next = 0;
        const int step = kTile / p.c.page_size, rest = kTile % p.c.page_size;
        auto fetch = [&](const Walk& x, bool enter) {
            const int first = x.t * kTile + lane * p.box;
            if (enter) {
                index = first / p.c.page_size;
                in = first - index * p.c.page_size;
            } else {
                index += step;
                in += rest;
                if (in >= p.c.page_size) {
                    in -= p.c.page_size;
                    ++index;
                }
            }
            int at = -1;
            if (lane * p.box < kTile && first < x.n) at = p.c.table[x.b * p.c.table_stride + index];
            return at;  // not looked at here: that would wait for the load
        };
        auto wait_warp = [&](int bar, uint32_t parity) { return __all_sync(kFullMask, wait(bar, parity)); };
        Place<S::kRing> put = {0, 0};
        if (!keys) put.move(count == 1 ? 1 : 2);
        int items = 0, q_loads = 0;
        Walk x = w, y = w;  // the tile to copy, and the one after it
        bool enters = true;
        page = count > 0 ? fetch(y, true) : 0;
        int in_now = in;
        for (int it = 0; it < count; ++it) {
            if (it + 1 < count) {
                y.next(p);
                page_next = fetch(y, y.t == 0);
            }
            if (keys && enters) {
                const int buf = q_loads & 1;
                if (q_loads >= 2 && !wait_warp(S::kQFree + buf, ((q_loads - 2) >> 1) & 1)) break;
                if (lane == 0) {
                    const uint32_t full = bar0 + (S::kQFull + buf) * 8;
                    mbar_expect_at(full, S::kSub * GP * 128);
                    for (int sub = 0; sub < S::kSub; ++sub)
                        tma_load_3d(q_buf + buf * S::kQBytes + sub * 16 * 128, &map_q, sub * 64,
                                    x.r / p.parts * p.group + x.r % p.parts * GP, x.b, full);
                }
                ++q_loads;
                __syncwarp();
            }
            // The place was used before when its item number is kRing or more.
            const int item = keys ? (it == 0 ? 0 : 2 * it - 1) : (it + 1 < count ? 2 * it + 2 : 2 * it + 1);
            if (item >= S::kRing && !wait_warp(S::kEmpty + put.at, put.phase ^ 1)) break;
            const uint32_t full = bar0 + (S::kFull + put.at) * 8, dst = ring + put.at * S::kItem;
            const int left = x.n - x.t * kTile, boxes = left >= kTile ? kTile / p.box : (left + p.box - 1) / p.box;
            if (lane == 0) mbar_expect_at(full, boxes * S::kSub * p.box * 128);
            const int h = p.parts == 1 ? x.r : x.r / p.parts;
            if ((unsigned)page >= (unsigned)p.c.pages) page = p.c.pages;  // outside the pool: reads as zeros
            for (int i = 0; i < boxes; ++i) {
                const int pg = __shfl_sync(kFullMask, page, i), at = __shfl_sync(kFullMask, in_now, i);
                if (lane == 0)
#pragma unroll
                    for (int sub = 0; sub < S::kSub; ++sub)
                        tma_load_4d(dst + sub * (kTile * 128) + i * p.box * 128, map, sub * 64, at, h, pg, full, policy);
            }
            ++items;
            put.move(keys ? (it == 0 ? 1 : 2) : (it + 2 == count ? 1 : 2));
            x = y;
            enters = y.t == 0;
            page = page_next;
            in_now = in;
        }
        __syncwarp();
        if (gave_up) {  // wait for this warp's copies in flight, so that none lands after the block's end
            for (int it = max(0, items - S::kRing); it < items; ++it) {
                const int item = keys ? (it == 0 ? 0 : 2 * it - 1) : (it + 1 < count ? 2 * it + 2 : 2 * it + 1);
                mbar_wait(&bars[S::kFull + item % S::kRing], (item / S::kRing) & 1);
            }
            for (int i = max(0, q_loads - 2); i < q_loads; ++i) mbar_wait(&bars[S::kQFull + (i & 1)], (i >> 1) & 1);
        }
    } else if (warp == kMmaS) {
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
    } else if (warp == kMmaO) {
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
        float m[GP], l[GP], offset[GP];
        Walk x = w;
        bool ok = true;      // false once a wait gave up
        bool leave = false;  // all 128 threads leave at the same barrier
        for (int it = 0; it < count && !leave;) {
            int last;
            const int n = share_of(x, it, &last);
            const int part = p.parts == 1 ? 0 : x.r % p.parts, heads = min(GP, p.group - part * GP);
            const int tile0 = w.s + it;
            for (int k = 0; k < n; ++k, ++it) {
                // Columns of heads past `heads` hold whatever lies there, and nothing looks at what comes of them.
                const int buf = it & 1, valid = k + 1 < n ? kTile : last;
                float s[GP], e[GP];
                ok = ok && wait(S::kSFull + buf, (it >> 1) & 1);
                __syncwarp();
                tc_fence_after();
#pragma unroll
                for (int g = 0; g < GP; g += 8) tmem_ld<GP < 8 ? GP : 8>(my_tmem + S::kTmemS + buf * 16 + g, s + g);
                tmem_wait_ld();
                tc_fence_before();
                mbar_arrive_at(bar0 + (S::kSFree + buf) * 8);
                bool over = true;
                if (k > 0) {
                    float top = -INFINITY;
#pragma unroll
                    for (int g = 0; g < GP; ++g) {
                        e[g] = fmaf(s[g], c, offset[g]);
                        top = fmaxf(top, e[g]);
                    }
                    over = bar_any(1, kSoftmax, (top > kSlack + kBias && tid < valid) || !ok);
                }
                // Some score has passed the reference by kSlack, or there is no reference yet.
                if (over) {
                    leave = bar_any(1, kSoftmax, !ok);
                    if (leave) break;
#pragma unroll
                    for (int g = 0; g < GP; ++g) {
                        const float top = warp_max(tid < valid ? s[g] * c : -INFINITY);
                        if (lane == 0) red[warp][g] = top;
                    }
                    bar_sync(1, kSoftmax);
                    float f[GP];
#pragma unroll
                    for (int g = 0; g < GP; ++g) {
                        const float top = fmaxf(fmaxf(red[0][g], red[1][g]), fmaxf(red[2][g], red[3][g]));
                        const float to = k == 0 ? top : fmaxf(m[g], top);
                        f[g] = k == 0 ? 0.f : to == m[g] ? 1.f : exp2_approx(m[g] - to);
                        l[g] = k == 0 ? 0.f : l[g] * f[g];
                        m[g] = to;
                        offset[g] = offset_of(to);
                        e[g] = fmaf(s[g], c, offset[g]);
                    }
                    if (k > 0) {
                        ok = wait(S::kPFree + (buf ^ 1), ((it - 1) >> 1) & 1);  // the tile before is in O
                        __syncwarp();
                        tc_fence_after();
                        constexpr int kStep = 2 * GP < 8 ? 2 * GP : 8;
#pragma unroll
                        for (int o = 0; o < S::kOBlocks; ++o) {
#pragma unroll
                            for (int j = 0; j < 2 * GP; j += kStep) {
                                float v[kStep];
                                const uint32_t at = my_tmem + S::kTmemO + o * S::kPCols + j;
                                tmem_ld<kStep>(at, v);
                                tmem_wait_ld();
#pragma unroll
                                for (int i = 0; i < kStep; ++i) v[i] *= f[(j + i) % GP];
                                tmem_st<kStep>(at, v);
                                tmem_wait_st();
                            }
                        }
                        tc_fence_before();
                    }
                }
#pragma unroll
                for (int g = 0; g < GP; ++g) e[g] = exp2_approx(e[g]);
                if (tid >= valid)
#pragma unroll
                    for (int g = 0; g < GP; ++g) e[g] = 0.f;
#pragma unroll
                for (int g = 0; g < GP; ++g) l[g] += e[g];
                if (p.p) {
                    store_row<GP>(p.p + ((size_t)(tile0 + k) * kTile + tid) * GP, e);
                    if (tid == 0) store_row<GP>(p.tile_m + (size_t)(tile0 + k) * GP, m);
                }
                uint32_t word[GP];
                if (p.c.bf16) split<true, GP>(e, word); else split<false, GP>(e, word);
                if (it >= 2) ok = ok && wait(S::kPFree + buf, ((it >> 1) & 1) ^ 1);
                const uint32_t row = p_buf + buf * S::kPBytes + tid * S::kPRow;
                if constexpr (GP == 1) {
                    asm volatile("st.shared.b32 [%0], %1;" ::"r"(row + (turn << 4)), "r"(word[0]) : "memory");
                } else {
#pragma unroll
                    for (int i = 0; i < GP / 4; ++i)
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(row + ((i ^ turn) << 4)),
                                     "r"(word[4 * i]), "r"(word[4 * i + 1]), "r"(word[4 * i + 2]), "r"(word[4 * i + 3])
                                     : "memory");
                }
                if (valid & 15) {
                    // Rows past the sequence's end inside the last step of 16: zero times NaN is NaN.
                    const int item = it + 1 < count ? 2 * it + 2 : 2 * count - 1, st = item % S::kRing;
                    ok = ok && wait(S::kFull + st, (item / S::kRing) & 1);
                    const int pad = (16 - (valid & 15)) * S::kSub * 8;
                    for (int i = tid; ok && i < pad; i += kSoftmax)
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
            leave = bar_any(1, kSoftmax, !ok);
            if (leave) break;
            if ((lane & (32 / GP - 1)) == 0) red[warp][warp_head<GP>(lane)] = sum;
            bar_sync(1, kSoftmax);
            tc_fence_after();
            const int row_start = tile0 - x.t;  // tile number of the row's first tile
            const bool whole = row_start >= w.s && row_start + x.tiles <= w.e;
            const int share = 2 * blockIdx.x + (row_start >= w.s ? 1 : 0);
            const int q0 = x.b * p.a.q_heads + (p.parts == 1 ? x.r : x.r / p.parts) * p.group + part * GP;
            float2* row_ml = p.row_ml + ((size_t)x.b * p.rows + x.r) * GP;
            constexpr int kStep = 2 * GP < 8 ? 2 * GP : 8;
            float v[S::kOBlocks][2 * GP];
#pragma unroll
            for (int o = 0; o < S::kOBlocks; ++o)
#pragma unroll
                for (int j = 0; j < 2 * GP; j += kStep)
                    tmem_ld<kStep>(my_tmem + S::kTmemO + o * S::kPCols + j, v[o] + j);
#pragma unroll
            for (int g = 0; g < GP; ++g) l[g] = (red[0][g] + red[1][g]) + (red[2][g] + red[3][g]);
            tmem_wait_ld();
            tc_fence_before();
            if (tid < heads) {
                float2 ml = make_float2(m[0], l[0]);
#pragma unroll
                for (int g = 1; g < GP; ++g)
                    if (g == tid) ml = make_float2(m[g], l[g]);
                if (ml.y != ml.y) ml.x = 0.f;  // a NaN sum says it all
                (whole ? row_ml : p.part_ml + share * GP)[tid] = ml;
                if (whole && p.a.lse) p.a.lse[q0 + tid] = lse_of(ml);
            }
#pragma unroll
            for (int g = 0; g < GP; ++g) l[g] = !whole ? 1.f : l[g] == 0.f ? 0.f : __frcp_rn(l[g]);
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
                        p.a.out[(size_t)(q0 + g) * p.c.dim + d] = from_float(l[g] == 0.f ? 0.f : y * l[g], p.c.bf16);
                    else
                        p.part_o[((size_t)share * GP + g) * p.c.dim + d] = y;
                }
            }
            if (!whole) {
                const int c0 = w.block_of(row_start), c1 = w.block_of(row_start + x.tiles - 1), pieces = c1 - c0 + 1;
                // Adds up the shares of `n` blocks, `stride` apart from `first` on: into the
                // output, or (not the row's last step) into the first one's share.
                auto join = [&](int first, int stride, int n, bool final) {
                    for (int g = warp; g < heads; g += kSoftmax / 32) {
                        float2 ml = make_float2(0.f, 0.f);
                        const int c = first + lane * stride;
                        if (lane < n) ml = __ldcg(&p.part_ml[(2 * c + (c == c0)) * GP + g]);
                        const float top = warp_max(ml.y == 0.f ? -INFINITY : ml.x);
                        const float f = ml.y == 0.f ? 0.f : exp2f(ml.x - top);
                        float sum = ml.y * f;
                        for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(kFullMask, sum, d);
                        if (lane < n) factor[lane][g] = f;
                        if (lane == 0) joined[g] = make_float2(top, sum);
                    }
                    bar_sync(1, kSoftmax);
                    const int quads = heads * p.c.dim / 4;
                    for (int i = tid; i < quads; i += kSoftmax) {
                        const int g = 4 * i / p.c.dim;
                        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
                        for (int j = 0; j < n; ++j) {
                            const int c = first + j * stride;
                            const float4* from = reinterpret_cast<const float4*>(
                                p.part_o + (size_t)(2 * c + (c == c0)) * GP * p.c.dim);
                            const float4 y = __ldcg(from + i);
                            const float f = factor[j][g];
                            o.x = fmaf(y.x, f, o.x);
                            o.y = fmaf(y.y, f, o.y);
                            o.z = fmaf(y.z, f, o.z);
                            o.w = fmaf(y.w, f, o.w);
                        }
                        if (final) {
                            const float sum = joined[g].y, r = sum == 0.f ? 0.f : __frcp_rn(sum);
                            uint2 word;
                            word.x = from_float(sum == 0.f ? 0.f : o.x * r, p.c.bf16) |
                                     (uint32_t)from_float(sum == 0.f ? 0.f : o.y * r, p.c.bf16) << 16;
                            word.y = from_float(sum == 0.f ? 0.f : o.z * r, p.c.bf16) |
                                     (uint32_t)from_float(sum == 0.f ? 0.f : o.w * r, p.c.bf16) << 16;
                            *reinterpret_cast<uint2*>(p.a.out + (size_t)q0 * p.c.dim + 4 * i) = word;
                        } else {
                            reinterpret_cast<float4*>(p.part_o + (size_t)(2 * first + (first == c0)) * GP * p.c.dim)[i] = o;
                        }
                    }
                    if (tid < heads) {
                        float2 ml = joined[tid];
                        if (ml.y != ml.y || ml.y == 0.f) ml.x = 0.f;
                        (final ? row_ml : p.part_ml + (2 * first + (first == c0)) * GP)[tid] = ml;
                        if (final && p.a.lse) p.a.lse[q0 + tid] = lse_of(ml);
                    }
                };
                // Whether this block is the last of n to arrive at a counter, which is then zero again.
                auto last_of = [&](unsigned* counter, int n) {
                    bar_sync(1, kSoftmax);
                    if (tid == 0) {  // releases what the barrier collected, and acquires the others'
                        unsigned before;
                        asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(before) : "l"(counter) : "memory");
                        if (before + 1 == (unsigned)n) *counter = 0;
                        arrived = before + 1;
                    }
                    bar_sync(1, kSoftmax);
                    return arrived == (unsigned)n;
                };
                if (pieces <= kJoin) {
                    if (last_of(p.done + 2 * c0 + 1, pieces)) join(c0, 1, pieces, true);
                } else {
                    // Two steps: kJoin neighbours each, then what they left (at most kJoin * kJoin pieces).
                    const int first = c0 + ((int)blockIdx.x - c0) / kJoin * kJoin, n = min(kJoin, c1 - first + 1);
                    if (last_of(p.done + 2 * first + (first == c0), n)) {
                        join(first, 1, n, false);
                        const int groups = (pieces + kJoin - 1) / kJoin;
                        if (last_of(p.done + 2 * gridDim.x + c0, groups)) join(c0, kJoin, groups, true);
                    }
                }
            }
            x.t += n - 1;
            x.next(p);
        }
    }
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaS) tmem_dealloc(tmem, S::kTmemCols);
    // What sequences without slots give.
    for (int b = blockIdx.x; b < p.c.seqs; b += gridDim.x) {
        if (p.c.len(b) > 0) continue;
        const size_t first = (size_t)b * p.a.q_heads;
        for (int i = tid; i < p.a.q_heads * (p.c.dim / 8); i += kThreads)
            reinterpret_cast<int4*>(p.a.out + first * p.c.dim)[i] = make_int4(0, 0, 0, 0);
        if (p.a.lse)
            for (int i = tid; i < p.a.q_heads; i += kThreads) p.a.lse[first + i] = -INFINITY;
    }
}

// Adds the heads' shares to the weights: p * 2^(tile's reference - row's) /
// sum.  Block c takes the tiles that block c of the first launch had, so its
// p may still be in L2; a warp takes a tile, all its loads in flight at once.
template <int GP>
__global__ void __launch_bounds__(kWeightThreads) kv_weight_kernel(const AttendArgs p) {
    constexpr int kWarps = kWeightThreads / 32;
    __shared__ int scan[kWarps + 8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Walk w = find_range<kWeightThreads>(p, scan);
    grid_dependency_wait();
    for (int tile = w.s; tile < w.e;) {
        const int count = min(w.tiles - w.t, w.e - tile);  // this block's tiles of the row
        const int part = w.r % p.parts, h = w.r / p.parts;
        // Of a group in several parts, the block that has the first adds up all.
        for (int pt = 0; part == 0 && pt < p.parts; ++pt) {
            const int heads = min(GP, p.group - pt * GP);
            const float* wi = pt == 0 ? p.a.weight.row(w.b, h) : p.a.weight_out.row(w.b, h);
            float* wo = p.a.weight_out.row(w.b, h);
            float2 ml = make_float2(0.f, 0.f);
            if (lane < heads) ml = p.row_ml[((size_t)w.b * p.rows + w.r + pt) * GP + lane];
            for (int k = warp; k < count; k += kWarps) {
                const size_t x = tile + k + (size_t)pt * w.tiles;
                const int slot0 = (w.t + k) * kTile + lane;
                float y[4][GP], sum[4];
                const float tm = lane < heads ? p.tile_m[x * GP + lane] : 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float* v = p.p + (x * kTile + i * 32 + lane) * GP;
                    if constexpr (GP % 4 == 0) {
#pragma unroll
                        for (int g = 0; g < GP; g += 4) {
                            const float4 q = *reinterpret_cast<const float4*>(v + g);
                            y[i][g] = q.x;
                            y[i][g + 1] = q.y;
                            y[i][g + 2] = q.z;
                            y[i][g + 3] = q.w;
                        }
                    } else {
#pragma unroll
                        for (int g = 0; g < GP; ++g) y[i][g] = v[g];
                    }
                    sum[i] = slot0 + i * 32 < w.n ? wi[slot0 + i * 32] : 0.f;
                }
                const float f = ml.y == 0.f || tm == -INFINITY ? 0.f : exp2f(tm - ml.x) / ml.y;
#pragma unroll
                for (int g = 0; g < GP; ++g) {
                    const float fg = __shfl_sync(kFullMask, f, g);
                    if (g >= heads) break;
#pragma unroll
                    for (int i = 0; i < 4; ++i) sum[i] = fmaf(y[i][g], fg, sum[i]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (slot0 + i * 32 < w.n) wo[slot0 + i * 32] = sum[i];
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

// Query heads that a block handles together: a thread's work on a tile goes
// with them.
int group_part(const KvCache& c, const KvAttend& a) {
    const int group = a.q_heads / c.heads;
    return group == 1 ? 1 : group <= 4 ? 4 : group <= 8 ? 8 : 16;
}

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
    if (plan.blocks > kKvCounters / 6) plan.blocks = kKvCounters / 6;
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
    if (!plan.args.p) return cudaSuccess;
    e = launch_pdl(kv_weight_kernel<GP>, dim3(plan.blocks), dim3(kWeightThreads), 0, s, plan.args);
    if (e == cudaSuccess) ++*launches;
    return e;
}

template <int DP>
cudaError_t launch_dim(const Plan& plan, int gp, cudaStream_t s, const CUtensorMap* maps, int* launches) {
    switch (gp) {
        case 1: return launch<DP, 1>(plan, s, maps, launches);
        case 4: return launch<DP, 4>(plan, s, maps, launches);
        case 8: return launch<DP, 8>(plan, s, maps, launches);
        default: return launch<DP, 16>(plan, s, maps, launches);
    }
}

}  // namespace

size_t kv_attend_scratch(int device, const KvCache& c, const KvAttend& a) {
    return make_plan(device, c, a, nullptr).bytes;
}

cudaError_t kv_attend_launch(int device, cudaStream_t s, const KvCache& c, const KvAttend& a, void* scratch,
                             unsigned* counters, unsigned epoch, unsigned* status, int* launches) {
    Plan plan = make_plan(device, c, a, scratch);
    plan.args.status = status;
    plan.args.done = counters + (epoch & 1) * (kKvCounters / 2);
    plan.args.clear = counters + (~epoch & 1) * (kKvCounters / 2);
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
    if (c.dim <= 64) return launch_dim<64>(plan, gp, s, maps, launches);
    if (c.dim <= 128) return launch_dim<128>(plan, gp, s, maps, launches);
    return launch_dim<256>(plan, gp, s, maps, launches);
}

}  // namespace topk
