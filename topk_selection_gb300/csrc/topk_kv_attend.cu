// topk_kv_attend: attention of one new token over a paged cache.
//
// Every key and value is read once (by groups of up to 16 query heads, of 8
// for dim > 128; a larger group is cut into parts that read them once each),
// and per 16-bit element there are only 2 * group multiply-adds, so the
// operator is bound by HBM: 6.79 TB/s of measured copy rate is 23 bytes per
// SM and clock.  With a group of eight
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
// 2^kSlack, far from float32's range), which is hardly ever.  P enters the
// second product as a sum of 16-bit numbers, each what the ones before it
// left, which the product adds up in columns of their own: two numbers of
// float16 (22 bits), three of bfloat16 (24: all of float32's).  The product is
// far from its rate, so further columns cost what it takes to split and store
// P.  Only 9 to 16 bfloat16 heads at once stay at two numbers, 16 bits: their
// 48 columns would take P's buffers from 16 to 32 KB, and the rings fill the
// shared memory.
//
// The tensor core adds to O in float32, but not to nearest: over a long row
// the error grows with its slots (16384 of them in one block: 7e-6 of O, and
// 3% of float16 outputs lie beside the nearest number).  So with every new
// reference, and every kFold tiles at least, the softmax threads add O up to
// nearest in columns beside it and set it to zero (0.6% then; 393 us of 64 long
// sequences as before, 12 heads on one 32.0 -> 32.2).
//
// Work is split evenly whatever the lengths are: all (sequence, head) rows'
// tiles of 128 slots are numbered in order, and block c takes the range
// [c * T / n, (c + 1) * T / n) of them.  A row that lies in one block is
// finished there; the shares of a row that several blocks have are joined by
// the last of them to finish (no block waits for another).  With weights, the
// p are stored (float32, a head's 128 slots side by side, so that a warp writes
// whole sectors: 32 us against 34 for 12 heads with a slot's side by side), and a
// second launch adds them up once the sums are known: storing and reading
// them costs 8 bytes a slot and head in L2, where a group of eight reads 512
// of keys and values (dim 128) from HBM.
//
// A block has an SM to itself: 192 KB of its shared memory are the rings that
// keep HBM busy.  Its warps: one copies keys and one values (a tile of small
// pages is up to 32 copies), one thread issues each product, and two groups
// of four do the softmax of every other tile, so that their latencies (some
// 1500 clocks a tile for 8 heads, against 2800 in which HBM delivers a tile of
// dim 128) overlap.
//
// Measured: 64 sequences of 4096 to 16384 slots, 64 query heads on 8, dim 128
// (2.69 GB): 393 us, 6.84 TB/s, the rate of a copy.  One sequence of 131071
// with weights (545 MB): 97 us, of which the first launch streams for 78 at
// the copy's rate; 2.5 us pass before the first copy, 5 to 7 between the last
// tile and the last join, and 6 in the second launch.  24 sequences of 501 to
// 2001 with a key-value head for each query head, dim 64 (123 MB): 35 us, the
// same ends around 21 us of streaming.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "topk_device.cuh"
#include "topk_kv.cuh"
#include "topk_tcgen05.cuh"

namespace topk {
namespace {

constexpr int kTile = 128;       // slots of a tile
constexpr int kThreads = 384;    // 2 x 4 softmax warps, copies of keys, of values, and the two products
constexpr int kSoftmax = 128;    // threads of a softmax group
constexpr int kCopyK = 8, kCopyV = 9, kMmaS = 10, kMmaO = 11;  // warps
constexpr int kWeightThreads = 512;
constexpr int kJoin = 32;        // shares that one block joins at most
constexpr float kSlack = 8.f;    // p <= 2^(kSlack + kBias) = 2^15: within f16's range
constexpr float kBias = 7.f;     // and f16's smallest step, 2^-24, is 2^-31 of the largest p
constexpr int kRingBytes = 192 * 1024;
constexpr int kFold = 8;         // tiles of a softmax group that O adds up before it is put aside

__device__ __forceinline__ uint16_t from_float(float x, int bf16) {
    return bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(x)) : __half_as_ushort(__float2half_rn(x));
}

static_assert(kKvBlocks <= kJoin * kJoin, "a row's pieces are joined in two steps");

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
    unsigned* clear;  // the other half of the counters
    int* walk;        // [blocks][Walk::kWords]: where each block begins, when weights are wanted
    float* p;         // [tile][GP][slot]: whole sectors from a warp
    float* tile_m;    // [tile][GP]: the reference of each tile's p
    unsigned* status;
    int spins;        // tries of a wait before it gives up, 0 for kWaitSpins (TOPK_OPT_KV_SPINS)
    int withhold;     // what the first block withholds (TOPK_OPT_KV_WITHHOLD)
};
enum Withhold { kKeys = 1, kValues = 2, kProducts = 3 };

// The code of a launch is fetched anew when the cache it streams has pushed
// it out of L2, and most of it runs once a row or once a launch: that part is
// kept in functions of their own and in loops, not unrolled.

// The first sequence from b on that has slots (seqs: none).
__device__ __noinline__ int seq_from(const int* lens, int b, int seqs) {
    while (b < seqs && lens[b] <= 0) ++b;
    return b;
}

// The first tile of block c's share when `blocks` of them share `total`
// tiles: floor(c * total / blocks), in 32 bits.
__device__ __forceinline__ int share_start(int c, int blocks, int total) {
    const int q = total / blocks;
    return c * q + (int)((unsigned)(c * (total - q * blocks)) / (unsigned)blocks);
}

// The block that tile number x belongs to.
__device__ __noinline__ int block_of(int x, int blocks, int total) {
    int c = min((int)((float)x * (float)blocks / (float)total), blocks - 1);
    while (c > 0 && share_start(c, blocks, total) > x) --c;
    while (c + 1 < blocks && share_start(c + 1, blocks, total) <= x) ++c;
    return c;
}

// Where a block's share of the tiles begins and ends, and a walk over it.
struct Walk {
    int b, h, part, t;  // sequence, key-value head, part of its group, tile of that row
    int n, tiles;       // the sequence's slots and tiles
    int s, e;           // the block's range of tile numbers
    int total, blocks;

    __device__ __forceinline__ void next(const AttendArgs& p) {
        if (++t < tiles) return;
        t = 0;
        if (++part < p.parts) return;
        part = 0;
        if (++h < p.c.heads) return;
        h = 0;
        b = seq_from(p.c.lens, b + 1, p.c.seqs);
        if (b < p.c.seqs) {
            n = p.c.len(b);
            tiles = (n + kTile - 1) / kTile;
        }
    }
    // To and from memory.
    static constexpr int kWords = 12;
    __device__ __forceinline__ void store(int* to) const {
        reinterpret_cast<int4*>(to)[0] = make_int4(b, h, part, t);
        reinterpret_cast<int4*>(to)[1] = make_int4(n, tiles, s, e);
        reinterpret_cast<int4*>(to)[2] = make_int4(total, blocks, 0, 0);
    }
    __device__ __forceinline__ void load(const int* from) {
        const int4 x = reinterpret_cast<const int4*>(from)[0], y = reinterpret_cast<const int4*>(from)[1];
        b = x.x, h = x.y, part = x.z, t = x.w, n = y.x, tiles = y.y, s = y.z, e = y.w;
    }
    __device__ __forceinline__ int row(const AttendArgs& p) const { return (b * p.c.heads + h) * p.parts + part; }
};

// Every thread of the block calls it; sh: THREADS / 32 + 8 words of shared memory.
template <int THREADS>
__device__ __forceinline__ Walk find_range(const AttendArgs& p, int* sh) {
    constexpr int W = THREADS / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, seqs = p.c.seqs;
    const int chunk = (seqs + THREADS - 1) / THREADS, lo = tid * chunk, hi = min(lo + chunk, seqs);
    int mine = 0;
#pragma unroll 1
    for (int b = lo; b < hi; ++b) mine += (p.c.len(b) + kTile - 1) / kTile * p.rows;
    int x = mine;
#pragma unroll 1
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(kFullMask, x, d);
        if (lane >= d) x += y;
    }
    if (lane == 31) sh[warp] = x;
    __syncthreads();
    const int v = lane < W ? sh[lane] : 0;
    const int before = __reduce_add_sync(kFullMask, lane < warp ? v : 0) + x - mine;
    Walk k;
    k.total = __reduce_add_sync(kFullMask, v);
    // One block to a row where one short sequence is all there is: a join costs
    // as much as four tiles (300 slots of 2 heads, dim 64: 9.3 us a call instead of 10.6).
    k.blocks = min((int)gridDim.x, seqs == 1 && k.total <= 4 * p.rows ? p.rows : k.total);
    k.s = k.e = k.b = k.h = k.part = k.t = k.n = k.tiles = 0;
    if ((int)blockIdx.x < k.blocks) {  // uniform over the block
        k.s = share_start(blockIdx.x, k.blocks, k.total);
        k.e = share_start(blockIdx.x + 1, k.blocks, k.total);
        if (before <= k.s && k.s < before + mine) {
            int at = before, b = lo, tiles;
#pragma unroll 1
            for (;; ++b) {
                tiles = (p.c.len(b) + kTile - 1) / kTile;
                if (k.s < at + tiles * p.rows) break;
                at += tiles * p.rows;
            }
            const int row = (k.s - at) / tiles;
            sh[W] = b;
            sh[W + 1] = row;
            sh[W + 2] = k.s - at - row * tiles;
            sh[W + 3] = p.c.len(b);
        }
        __syncthreads();
        k.b = sh[W];
        k.h = sh[W + 1] / p.parts;
        k.part = sh[W + 1] - k.h * p.parts;
        k.t = sh[W + 2];
        k.n = sh[W + 3];
        k.tiles = (k.n + kTile - 1) / kTile;
    }
    return k;
}

template <int DP, int GP>
struct Shape {
    // A tile's keys, and its values, are copied in parts of at most 128
    // elements of dim.  Keys and values have rings of their own: each is
    // filled by one warp and emptied by one thread, in order, which is what
    // the parity of a barrier's phase can tell apart.
    static constexpr int kParts = DP > 128 ? DP / 128 : 1;
    static constexpr int kSub = DP / kParts / 64;         // 128-byte columns of a part's row
    static constexpr int kItem = kTile * kSub * 128;      // bytes of a part
    static constexpr int kRing = kRingBytes / 2 / kItem;
    static constexpr int kQBytes = DP / 64 * 16 * 128;    // 16 rows of a query block
    static constexpr int kTerms = GP <= 8 ? 3 : 2;        // numbers that P is split into at most
    // The first number of every head, then the second, ...; the rest is not looked at.
    static constexpr int kPCols = GP <= 4 ? 16 : 32;
    static constexpr int kPRow = kPCols * 2;              // bytes of a slot's row of P
    static constexpr int kPBytes = kPRow * kTile;
    static constexpr int kM = DP == 64 ? 64 : 128;        // rows of one second product
    static constexpr int kOBlocks = kParts;
    // Tensor memory columns: two S buffers of 16, then O of each softmax
    // group for this row, and of both for the row before, then what is put
    // aside of the same four.
    static constexpr int kTmemS = 0, kTmemO = 32, kOCols = kOBlocks * kPCols;
    static constexpr int kTmemF = kTmemO + 4 * kOCols, kFCols = kOBlocks * GP, kTmemEnd = kTmemF + 4 * kFCols;
    static constexpr int kTmemCols = kTmemEnd <= 128 ? 128 : kTmemEnd <= 256 ? 256 : 512;
    static constexpr size_t kSmem = 1024 + kRingBytes + 2 * kQBytes + 2 * kPBytes;
    // Barriers, by their place in bars[].
    static constexpr int kFullK = 0, kFullV = kRing, kEmptyK = 2 * kRing, kEmptyV = 3 * kRing, kSFull = 4 * kRing,
                         kSFree = kSFull + 2, kPReady = kSFull + 4,
                         kPFree = kSFull + 6, kQFull = kSFull + 8, kQFree = kSFull + 10, kDrain = kSFull + 12,
                         kTold = kSFull + 14, kBars = kSFull + 18;
};

// The bounded wait's slow side: gives up after kWaitSpins tries, or once
// another wait of the block has and *gave_up is 1.  Fewer tries, for tests, are
// in *gave_up as a negative number: as an argument they cost 3% of a case whose
// softmax just keeps up (12 heads on one, 32.9 us instead of 31.8).
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile int* gave_up, unsigned* status) {
#pragma unroll 1
    for (int i = 0; i < kWaitSpins; ++i) {
        if (mbar_try(bar, parity)) return true;
        const int g = *gave_up;
        if (g > 0) return false;
        if (g < 0 && i >= -g) break;
    }
    *gave_up = 1;
    atomicOr(status, kStatusWaitTimeout);
    return false;
}

// A place in a ring, moved on by n <= RING items.
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

// N numbers as sums of TERMS 16-bit elements (of two for float16), each the
// rounded rest of the ones before it: the first of all numbers, then the second, ...
template <bool BF16, int TERMS, int N>
__device__ __forceinline__ void split(const float (&p)[N], uint32_t* words) {
    uint16_t e[TERMS * N + 1] = {};
#pragma unroll
    for (int g = 0; g < N; ++g) {
        float rest = p[g];
#pragma unroll
        for (int t = 0; t < (BF16 ? TERMS : 2); ++t) {
            if constexpr (BF16) {
                const __nv_bfloat16 x = __float2bfloat16_rn(rest);
                e[t * N + g] = __bfloat16_as_ushort(x);
                rest -= __bfloat162float(x);
            } else {
                const __half x = __float2half_rn(rest);
                e[t * N + g] = __half_as_ushort(x);
                rest -= __half2float(x);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < (TERMS * N + 1) / 2; ++i) words[i] = (uint32_t)e[2 * i] | (uint32_t)e[2 * i + 1] << 16;
}

// The columns of STEP heads of a product with P, all TERMS of them; one head's
// lie side by side.  Ready after tmem_wait_ld().
template <int TERMS, int GP, int STEP>
struct Terms {
    float v[TERMS * STEP < 4 ? 4 : TERMS * STEP];
    __device__ __forceinline__ void load(uint32_t at) {
        if constexpr (GP == 1) {
            tmem_ld<4>(at, v);
        } else {
#pragma unroll
            for (int t = 0; t < TERMS; ++t) tmem_ld<STEP>(at + t * GP, v + t * STEP);
        }
    }
    static __device__ __forceinline__ void clear(uint32_t at) {
        constexpr int N = GP == 1 ? 4 : STEP;
        const float zeros[N] = {};
#pragma unroll
        for (int t = 0; t < (GP == 1 ? 1 : TERMS); ++t) tmem_st<N>(at + t * GP, zeros);
    }
    // Head i's sum; float16 has two terms.
    __device__ __forceinline__ float sum(int i, int bf16) const {
        const float x = v[i] + v[STEP + i];
        return TERMS == 3 && bf16 ? x + v[(TERMS - 1) * STEP + i] : x;
    }
};

// N consecutive floats, as wide as they come.
template <int N>
__device__ __forceinline__ void load_row(const float* from, float (&v)[N]) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int g = 0; g < N; g += 4) {
            const float4 x = *reinterpret_cast<const float4*>(from + g);
            v[g] = x.x;
            v[g + 1] = x.y;
            v[g + 2] = x.z;
            v[g + 3] = x.w;
        }
    } else {
#pragma unroll
        for (int g = 0; g < N; ++g) v[g] = from[g];
    }
}

// kBias - m, what is added to a scaled score; a head without a score above
// -inf yet gets a number that makes any such score pass kSlack.
__device__ __forceinline__ float offset_of(float m) { return m > -INFINITY ? kBias - m : 3.4e38f; }

__device__ __forceinline__ float lse_of(float2 ml) {
    return ml.y == 0.f ? -INFINITY : (ml.x - kBias + log2f(ml.y)) * 0.6931471805599453f;
}

// Adds up the shares of `n` blocks, `stride` apart from `first` on: into the
// output, or (not the row's last step) into the first one's share.  128
// threads call it together; `bar` is their barrier.
template <int GP>
__device__ __forceinline__ void join_shares(const AttendArgs& p, int c0, int first, int stride, int n, bool final, int q0,
                                         int heads, float2* row_ml, float (*factor)[GP], float2* joined, int bar,
                                         int me) {
    // A warp has every fourth head, a lane one share; all loads are in flight at once.
    constexpr int kMine = GP < 4 ? 1 : GP / 4, kFly = 8;
    const int lane = me & 31, quarter = me >> 5;
    float2 ml[kMine];
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const int c = first + lane * stride, g = quarter + 4 * i;
        ml[i] = make_float2(0.f, 0.f);
        if (lane < n && g < heads) ml[i] = __ldcg(&p.part_ml[(2 * c + (c == c0)) * GP + g]);
    }
    // Two quads of elements of kFly shares at a time, the first of them under
    // way while the factors are worked out.
    const int quads = heads * p.c.dim / 4;
    const int share = GP * p.c.dim / 4 * 2 * stride;      // from one share to the next
    const int own = first == c0 ? GP * p.c.dim / 4 : 0;  // the row's first block has a place of its own
    const float4* shares = reinterpret_cast<const float4*>(p.part_o + (size_t)2 * first * GP * p.c.dim);
    float4 y[2][kFly];
    auto fetch = [&](int i0, int j0) {
#pragma unroll
        for (int j = 0; j < kFly; ++j)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                y[q][j] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (j0 + j < n && i0 + q * kSoftmax < quads)
                    y[q][j] = __ldcg(shares + (j0 + j == 0 ? own : (j0 + j) * share) + i0 + q * kSoftmax);
            }
    };
    fetch(me, 0);
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const int g = quarter + 4 * i;
        const float top = warp_max(ml[i].y == 0.f ? -INFINITY : ml[i].x);
        const float f = ml[i].y == 0.f ? 0.f : exp2_approx(ml[i].x - top);
        float sum = ml[i].y * f;
#pragma unroll
        for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(kFullMask, sum, d);
        if (g < heads) {
            if (lane < n) factor[lane][g] = f;
            if (lane == 0) joined[g] = make_float2(top, sum);
        }
    }
    bar_sync(bar, kSoftmax);
#pragma unroll 1
    for (int i0 = me; i0 < quads; i0 += 2 * kSoftmax) {
        float4 o[2] = {};
        int g[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) g[q] = min(4 * (i0 + q * kSoftmax) / p.c.dim, GP - 1);
#pragma unroll 1
        for (int j0 = 0; j0 < n; j0 += kFly) {
            if (i0 != me || j0 > 0) fetch(i0, j0);
#pragma unroll
            for (int j = 0; j < kFly; ++j)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const float f = j0 + j < n ? factor[j0 + j][g[q]] : 0.f;
                    o[q].x = fmaf(y[q][j].x, f, o[q].x);
                    o[q].y = fmaf(y[q][j].y, f, o[q].y);
                    o[q].z = fmaf(y[q][j].z, f, o[q].z);
                    o[q].w = fmaf(y[q][j].w, f, o[q].w);
                }
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int i = i0 + q * kSoftmax;
            if (i >= quads) break;
            if (final) {
                const float sum = joined[g[q]].y, r = sum == 0.f ? 0.f : __frcp_rn(sum);
                if (sum == 0.f) o[q] = make_float4(0.f, 0.f, 0.f, 0.f);
                uint2 word;
                word.x = from_float(o[q].x * r, p.c.bf16) | (uint32_t)from_float(o[q].y * r, p.c.bf16) << 16;
                word.y = from_float(o[q].z * r, p.c.bf16) | (uint32_t)from_float(o[q].w * r, p.c.bf16) << 16;
                *reinterpret_cast<uint2*>(p.a.out + (size_t)q0 * p.c.dim + 4 * i) = word;
            } else {
                reinterpret_cast<float4*>(p.part_o + (size_t)2 * first * GP * p.c.dim)[own + i] = o[q];
            }
        }
    }
    if (me < heads) {
        float2 ml = joined[me];
        if (ml.y != ml.y || ml.y == 0.f) ml.x = 0.f;
        (final ? row_ml : p.part_ml + (2 * first + (first == c0)) * GP)[me] = ml;
        if (final && p.a.lse) p.a.lse[q0 + me] = lse_of(ml);
    }
}

// Whether this block is the last of n to arrive at a counter, which is then zero again.
__device__ __forceinline__ bool last_of(unsigned* counter, int n, unsigned* arrived, int bar, int me) {
    bar_sync(bar, kSoftmax);
    if (me == 0) {  // releases what the barrier collected, and acquires the others'
        unsigned before;
        asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(before) : "l"(counter) : "memory");
        if (before + 1 == (unsigned)n) *counter = 0;
        *arrived = before + 1;
    }
    bar_sync(bar, kSoftmax);
    return *arrived == (unsigned)n;
}

// After this block's share of a row that several blocks have: the last of
// them to come here joins them.  Up to kJoin shares at once; more (at most
// kJoin * kJoin) in two steps, neighbours first.
template <int GP>
__device__ __forceinline__ void join_row(const AttendArgs& p, int total, int blocks, int row_start, int tiles, int q0,
                                      int heads, float2* row_ml, float (*factor)[GP], float2* joined,
                                      unsigned* arrived, int bar, int me) {
    const int c0 = block_of(row_start, blocks, total), c1 = block_of(row_start + tiles - 1, blocks, total);
    const int pieces = c1 - c0 + 1, groups = (pieces + kJoin - 1) / kJoin;
    int first = c0, stride = 1, n = pieces;
    bool final = true;
    if (groups > 1) {
        first = c0 + ((int)blockIdx.x - c0) / kJoin * kJoin;
        n = min(kJoin, c1 - first + 1);
        final = false;
    }
    unsigned* counter = p.done + 2 * first + (first == c0);
#pragma unroll 1
    while (last_of(counter, n, arrived, bar, me)) {
        join_shares<GP>(p, c0, first, stride, n, final, q0, heads, row_ml, factor, joined, bar, me);
        if (final) break;
        first = c0;
        stride = kJoin;
        n = groups;
        final = true;
        counter = p.done + 2 * gridDim.x + c0;
    }
}

template <int DP, int GP>
__global__ void __launch_bounds__(kThreads, 1)
kv_attend_kernel(const __grid_constant__ AttendArgs p, const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                 const __grid_constant__ CUtensorMap map_q) {
    using S = Shape<DP, GP>;
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(8) uint64_t bars[S::kBars];
    __shared__ uint32_t tmem_at;
    __shared__ int scan[kThreads / 32 + 8];
    constexpr int kRow = GP < 4 ? 4 : GP;
    __shared__ float red[2][4][GP];                        // of each softmax group and its warps
    __shared__ __align__(16) float each[2][2][kRow];       // two numbers of each head for the group's threads
    __shared__ float told_m[4][GP], told_l[4][4][GP];      // what one group tells the other at a row's end
    __shared__ bool told_aside[4];
    __shared__ float2 joined[2][GP];
    __shared__ unsigned arrived[2];
    __shared__ int issued[3];  // parts of keys and of values that were asked for, and queries
    __shared__ volatile int gave_up;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t bar0 = smem_addr(bars);
    if (tid == 0) {
#pragma unroll 1
        for (int i = 0; i < S::kBars; ++i) {
            const bool by_threads = i / 2 == S::kSFree / 2 || i / 2 == S::kPReady / 2 || i >= S::kTold;
            mbar_init(&bars[i], by_threads ? kSoftmax : 1);
        }
        mbar_init_fence();
        gave_up = -p.spins;
    }
    if (warp == kCopyK && lane == 0) {
        prefetch_map(&map_k);
        prefetch_map(&map_q);
    }
    if (warp == kCopyV && lane == 0) prefetch_map(&map_v);
    grid_dependency_wait();
    clear_half(p.clear);
    if (warp == kMmaS) tmem_alloc(&tmem_at, S::kTmemCols);
    launch_dependents();  // the weights' launch waits for this one's end before it reads anything of it
    Walk w = find_range<kThreads>(p, scan);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_at;
    const uint32_t ring = (smem_addr(smem_raw) + 1023) & ~1023u, q_buf = ring + kRingBytes, p_buf = q_buf + 2 * S::kQBytes;
    const int count = w.e - w.s;  // tiles of this block
    if (p.p && tid == kSoftmax) w.store(p.walk + blockIdx.x * Walk::kWords);

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

    auto withholds = [&](int what) { return p.withhold == what && blockIdx.x == 0; };
    if (warp == kCopyK || warp == kCopyV) {
        // Copies into the rings.  One warp has the keys, one the values: a
        // copy takes its issuer some 50 clocks, and a tile of small pages is
        // many copies.
        const bool keys = warp == kCopyK;
        const CUtensorMap* map = keys ? &map_k : &map_v;
        const int full0 = keys ? S::kFullK : S::kFullV, empty0 = keys ? S::kEmptyK : S::kEmptyV;
        const uint32_t my_ring = keys ? ring : ring + kRingBytes / 2;
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
        int items = 0, q_loads = 0;
        Walk x = w, y = w;  // the tile to copy, and the one after it
        bool enters = true;
        page = count > 0 ? fetch(y, true) : 0;
        int in_now = in;
#pragma unroll 1
        for (int it = 0; it < count && !withholds(keys ? kKeys : kValues); ++it) {
            if (it + 1 < count) {
                y.next(p);
                page_next = fetch(y, y.t == 0);
            }
            if (keys && enters) {
                const int buf = q_loads & 1;
                if (q_loads >= 2 && !wait_warp(S::kQFree + buf, ((q_loads - 2) >> 1) & 1)) break;
                if (lane == 0) {
                    const uint32_t full = bar0 + (S::kQFull + buf) * 8;
                    mbar_expect_at(full, DP / 64 * GP * 128);
                    for (int sub = 0; sub < DP / 64; ++sub)
                        tma_load_3d(q_buf + buf * S::kQBytes + sub * 16 * 128, &map_q, sub * 64,
                                    x.h * p.group + x.part * GP, x.b, full);
                }
                ++q_loads;
                __syncwarp();
            }
            const int left = x.n - x.t * kTile, boxes = left >= kTile ? kTile / p.box : (left + p.box - 1) / p.box;
            if ((unsigned)page >= (unsigned)p.c.pages) page = p.c.pages;  // outside the pool: reads as zeros
            bool ok = true;
#pragma unroll
            for (int part = 0; part < S::kParts; ++part) {
                ok = ok && (items < S::kRing || wait_warp(empty0 + put.at, put.phase ^ 1));
                if (!ok) break;
                const uint32_t full = bar0 + (full0 + put.at) * 8, dst = my_ring + put.at * S::kItem;
                if (lane == 0) mbar_expect_at(full, boxes * S::kSub * p.box * 128);
#pragma unroll 1
                for (int i0 = 0; i0 < boxes; i0 += 4) {
                    int pg[4], at[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        pg[i] = __shfl_sync(kFullMask, page, i0 + i);
                        at[i] = __shfl_sync(kFullMask, in_now, i0 + i);
                    }
                    if (lane == 0)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (i0 + i >= boxes) break;
#pragma unroll
                            for (int sub = 0; sub < S::kSub; ++sub)
                                tma_load_4d(dst + sub * (kTile * 128) + (i0 + i) * p.box * 128, map,
                                            (part * S::kSub + sub) * 64, at[i], x.h, pg[i], full, policy);
                        }
                    __syncwarp();
                }
                ++items;
                put.move(1);
            }
            if (!ok) break;
            x = y;
            enters = y.t == 0;
            page = page_next;
            in_now = in;
        }
        if (lane == 0) {
            issued[keys ? 0 : 1] = items;
            if (keys) issued[2] = q_loads;
        }
    } else if (warp == kMmaS) {
        if (lane == 0) {  // S = K Q^T
            const uint32_t id = mma_idesc(p.c.bf16, kTile, 16, false);
            constexpr uint32_t hi = smem_desc_hi(1024, 128);
            const uint32_t k_lo = smem_desc_lo(ring, 16), q_lo = smem_desc_lo(q_buf, 16);
            Place<S::kRing> get = {0, 0};
            Walk x = w;
            bool ok = true;
#pragma unroll 1
            for (int it = 0, piece = 0; it < count && ok; ++piece) {
                int last;
                const int n = share_of(x, it, &last), qb = piece & 1;
                if (!wait(S::kQFull + qb, (piece >> 1) & 1)) break;
#pragma unroll 1
                for (int k = 0; k < n; ++k, ++it) {
                    const int buf = it & 1;
                    ok = it < 2 || wait(S::kSFree + buf, ((it >> 1) & 1) ^ 1);
#pragma unroll
                    for (int part = 0; part < S::kParts; ++part) {
                        ok = ok && wait(S::kFullK + get.at, get.phase);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t a = k_lo + get.at * (S::kItem >> 4);
                        const uint32_t b = q_lo + ((qb * S::kQBytes + part * S::kSub * 16 * 128) >> 4);
#pragma unroll
                        for (int j = 0; j < S::kSub * 4; ++j)
                            mma_f16(tmem + S::kTmemS + buf * 16,
                                    a + (((j >> 2) * (kTile * 128) + (j & 3) * 32) >> 4), hi,
                                    b + (((j >> 2) * (16 * 128) + (j & 3) * 32) >> 4), hi, id, part > 0 || j > 0);
                        mma_commit(bar0 + (S::kEmptyK + get.at) * 8);
                        get.move(1);
                    }
                    if (!ok) break;
                    mma_commit(bar0 + (S::kSFull + buf) * 8);
                }
                mma_commit(bar0 + (S::kQFree + qb) * 8);
                x.t += n - 1;
                x.next(p);
            }
        }
    } else if (warp == kMmaO) {
        if (lane == 0) {  // O += V^T P^T
            const uint32_t id = mma_idesc(p.c.bf16, S::kM, S::kPCols, true);
            constexpr uint32_t hi_v = smem_desc_hi(1024, 128), hi_p = smem_desc_hi(S::kPRow * 8, S::kPRow);
            const uint32_t v_lo = smem_desc_lo(ring + kRingBytes / 2, kTile * 128), p_lo = smem_desc_lo(p_buf, 16);
            Place<S::kRing> get = {0, 0};
            Walk x = w;
            bool ok = true;
#pragma unroll 1
            for (int it = 0, piece = 0; it < count && ok; ++piece) {
                int last;
                const int n = share_of(x, it, &last);
#pragma unroll 1
                for (int k = 0; k < n; ++k, ++it) {
                    const int buf = it & 1, steps = k + 1 < n ? 8 : (last + 15) >> 4;
                    const uint32_t o = tmem + S::kTmemO + ((piece & 1) * 2 + buf) * S::kOCols;
                    ok = wait(S::kPReady + buf, (it >> 1) & 1);
#pragma unroll
                    for (int part = 0; part < S::kParts; ++part) {
                        ok = ok && wait(S::kFullV + get.at, get.phase);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t a = v_lo + get.at * (S::kItem >> 4), b = p_lo + buf * (S::kPBytes >> 4);
#pragma unroll
                        for (int j = 0; j < kTile / 16; ++j) {
                            if (j >= steps) break;
                            mma_f16(o + part * S::kPCols, a + (j * 2048 >> 4), hi_v, b + j * (S::kPRow * 16 >> 4), hi_p,
                                    id, k > 1 || j > 0);
                        }
                        mma_commit(bar0 + (S::kEmptyV + get.at) * 8);
                        get.move(1);
                    }
                    if (!ok) break;
                    if (it >= 2 || !withholds(kProducts)) mma_commit(bar0 + (S::kPFree + buf) * 8);
                }
                x.t += n - 1;
                x.next(p);
            }
        }
    } else {
        // Softmax.  The two groups of 128 threads take the tiles in turn, each
        // with its own buffers of S and P, reference, sum and O, so that one
        // group's waits are the other's work; the group that has a row's
        // last tile puts the two together.  Thread `me` owns slot `me` of
        // each of its group's tiles, and lane `me` of O.
        const int group = warp >> 2, me = tid & (kSoftmax - 1), quarter = warp & 3;
        const float c = p.a.scale * 1.4426950408889634f;
        const uint32_t my_tmem = tmem + ((uint32_t)quarter << 21);  // 32 * quarter in the address's lane field
        const uint32_t my_s = my_tmem + S::kTmemS + group * 16;
        // This slot's row of P: 16-byte chunks, swizzled over the row's width.
        constexpr int kChunks = S::kPRow / 16;
        const int turn = kChunks == 2 ? (me >> 2) & 1 : (me >> 1) & 3;
        const uint32_t my_p = p_buf + group * S::kPBytes + me * S::kPRow;
        // What goes with a head alone is worked out by thread g of the group
        // for head g, and handed to the others in `each`.
        float l[GP], offset[GP], my_m = 0.f;
        float* const first_of = each[group][0];
        float* const second_of = each[group][1];
        Walk x = w;
        bool ok = true;      // false once a wait gave up
        bool leave = false;  // all threads of the group leave at the same barrier
#pragma unroll 1
        for (int it0 = 0, piece = 0; it0 < count && !leave; ++piece) {
            int last;
            const int n = share_of(x, it0, &last);
            const int heads = min(GP, p.group - x.part * GP);
            const int tile0 = w.s + it0;
            const uint32_t my_o = my_tmem + S::kTmemO + ((piece & 1) * 2 + group) * S::kOCols;
            const uint32_t my_f = my_tmem + S::kTmemF + ((piece & 1) * 2 + group) * S::kFCols;
            bool aside = false;  // whether the columns beside O hold something
            const int k0 = (it0 ^ group) & 1;
#pragma unroll 1
            for (int k = k0; k < n; k += 2) {
                // Columns of heads past `heads` hold whatever lies there, and nothing looks at what comes of them.
                const int it = it0 + k, valid = k + 1 < n ? kTile : last;
                float s[GP], e[GP];
                ok = ok && wait(S::kSFull + group, (it >> 1) & 1);
                __syncwarp();
                tc_fence_after();
#pragma unroll
                for (int g = 0; g < GP; g += 8) tmem_ld<GP < 8 ? GP : 8>(my_s + g, s + g);
                tmem_wait_ld();
                tc_fence_before();
                mbar_arrive_at(bar0 + (S::kSFree + group) * 8);
                bool over = true;
                if (k > k0) {
                    float top = -INFINITY;
#pragma unroll
                    for (int g = 0; g < GP; ++g) {
                        e[g] = fmaf(s[g], c, offset[g]);
                        top = fmaxf(top, e[g]);
                    }
                    const bool due = (k >> 1) % kFold == 0;
                    over = bar_any(1 + group, kSoftmax, (top > kSlack + kBias && me < valid) || due || !ok);
                }
                // Some score has passed the reference by kSlack, there is no reference yet, or O has added up enough.
                if (over) {
                    leave = bar_any(1 + group, kSoftmax, !ok);
                    if (leave) break;
#pragma unroll
                    for (int g = 0; g < GP; ++g) {
                        const float top = warp_max(me < valid ? s[g] * c : -INFINITY);
                        if (lane == 0) red[group][quarter][g] = top;
                    }
                    bar_sync(1 + group, kSoftmax);
                    if (me < GP) {
                        const float top = fmaxf(fmaxf(red[group][0][me], red[group][1][me]),
                                                fmaxf(red[group][2][me], red[group][3][me]));
                        const float to = k == k0 ? top : fmaxf(my_m, top);
                        first_of[me] = k == k0 ? 0.f : to == my_m ? 1.f : exp2_approx(my_m - to);
                        second_of[me] = offset_of(to);
                        my_m = to;
                    }
                    bar_sync(1 + group, kSoftmax);
                    float f[GP];
                    load_row<GP>(first_of, f);
                    load_row<GP>(second_of, offset);
#pragma unroll
                    for (int g = 0; g < GP; ++g) {
                        l[g] = k == k0 ? 0.f : l[g] * f[g];
                        e[g] = fmaf(s[g], c, offset[g]);
                    }
                    if (k > k0) {
                        ok = wait(S::kPFree + group, ((it >> 1) & 1) ^ 1);  // the group's tile before is in O
                        __syncwarp();
                        tc_fence_after();
                        constexpr int kStep = GP < 8 ? GP : 8;
#pragma unroll
                        for (int j = 0; j < S::kFCols; j += kStep) {
                            Terms<S::kTerms, GP, kStep> v;
                            float sum[kStep] = {};
                            const uint32_t at = my_o + j / GP * S::kPCols + j % GP;
                            v.load(at);
                            if (aside) tmem_ld<kStep>(my_f + j, sum);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < kStep; ++i)
                                sum[i] = (sum[i] + v.sum(i, p.c.bf16)) * f[(j + i) % GP];
                            tmem_st<kStep>(my_f + j, sum);
                            v.clear(at);
                        }
                        tmem_wait_st();
                        aside = true;
                        tc_fence_before();
                    }
                }
#pragma unroll
                for (int g = 0; g < GP; ++g) e[g] = exp2_approx(e[g]);
                if (me >= valid)
#pragma unroll
                    for (int g = 0; g < GP; ++g) e[g] = 0.f;
#pragma unroll
                for (int g = 0; g < GP; ++g) l[g] += e[g];
                if (p.p) {
                    float* const to = p.p + (size_t)(tile0 + k) * GP * kTile + me;
#pragma unroll
                    for (int g = 0; g < GP; ++g)
                        if (g < heads) to[g * kTile] = e[g];
                    if (me < GP) p.tile_m[(size_t)(tile0 + k) * GP + me] = my_m;
                }
                uint32_t word[(S::kTerms * GP + 1) / 2];
                if (p.c.bf16) split<true, S::kTerms, GP>(e, word); else split<false, S::kTerms, GP>(e, word);
                if (it >= 2) ok = ok && wait(S::kPFree + group, ((it >> 1) & 1) ^ 1);
                if constexpr (GP <= 4) {
                    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(my_p + ((GP == 4 ? 1 ^ turn : turn) << 4)),
                                 "r"(word[GP == 4 ? 4 : 0]), "r"(word[GP == 4 ? 5 : 1])
                                 : "memory");
                }
                if constexpr (GP > 1) {
#pragma unroll
                    for (int i = 0; i < S::kTerms * GP / 8; ++i)
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(my_p + ((i ^ turn) << 4)),
                                     "r"(word[4 * i]), "r"(word[4 * i + 1]), "r"(word[4 * i + 2]), "r"(word[4 * i + 3])
                                     : "memory");
                }
                if (valid & 15) {
                    // Rows past the sequence's end inside the last step of 16: zero times NaN is NaN.
                    const int pad = (16 - (valid & 15)) * S::kSub * 8;
                    // The use of the place before this one has to be over, or its phase could be taken for
                    // this one's.  It was three places back: the tile it - 3, whose product came before
                    // the one waited for above, or with two places to a tile perhaps the last one's.
                    if (S::kParts > 1 && it > 0) ok = ok && wait(S::kPFree + (group ^ 1), ((it - 1) >> 1) & 1);
#pragma unroll
                    for (int part = 0; part < S::kParts; ++part) {
                        const int item = it * S::kParts + part, st = item % S::kRing;
                        ok = ok && wait(S::kFullV + st, (item / S::kRing) & 1);
#pragma unroll 1
                        for (int i = me; ok && i < pad; i += kSoftmax)
                            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                             ring + kRingBytes / 2 + st * S::kItem + i / 8 % S::kSub * (kTile * 128) +
                                             (valid + i / (S::kSub * 8)) * 128 + (i & 7) * 16),
                                         "r"(0)
                                         : "memory");
                    }
                }
                fence_proxy_async_smem();
                mbar_arrive_at(bar0 + (S::kPReady + group) * 8);
            }
            if (leave) break;

            // The end of the row's share: sums over the slots' threads, of this
            // group and of the other.  A group without a tile of the row has
            // nothing to tell, but says so; it is never more than three rows
            // ahead of the other, since products are made in order.
            const int final_it = it0 + n - 1, slot4 = piece & 3;
            it0 += n;
            if (k0 < n) {
                const float sum = warp_sums<GP>(l, lane);
                if ((final_it & 1) != group) {
                    if ((lane & (32 / GP - 1)) == 0) told_l[slot4][quarter][warp_head<GP>(lane)] = sum;
                    if (me < GP) told_m[slot4][me] = my_m;
                    if (me == 0) told_aside[slot4] = aside;
                } else {
                    ok = ok && wait(S::kTold + slot4, (piece >> 2) & 1);
                    ok = ok && wait(S::kPFree + group, (final_it >> 1) & 1);  // and all products before it
                    leave = bar_any(1 + group, kSoftmax, !ok);
                    if (leave) break;
                    if ((lane & (32 / GP - 1)) == 0) red[group][quarter][warp_head<GP>(lane)] = sum;
                    bar_sync(1 + group, kSoftmax);
                }
            }
            if ((final_it & 1) != group) {
                mbar_arrive_at(bar0 + (S::kTold + slot4) * 8);
                x.t += n - 1;
                x.next(p);
                continue;
            }
            const int row_start = tile0 - x.t;  // tile number of the row's first tile
            const bool whole = row_start >= w.s && row_start + x.tiles <= w.e;
            const int share = 2 * blockIdx.x + (row_start >= w.s ? 1 : 0);
            const int q0 = x.b * p.a.q_heads + x.h * p.group + x.part * GP;
            float2* row_ml = p.row_ml + (size_t)x.row(p) * GP;
            if (me < GP) {
                // The two groups' sums on a common reference, and the factor of each one's O.
                float2 ml = make_float2(my_m, (red[group][0][me] + red[group][1][me]) +
                                                  (red[group][2][me] + red[group][3][me]));
                float fa = 1.f, fb = 0.f;
                if (n > 1) {
                    const float mb = told_m[slot4][me], lb = (told_l[slot4][0][me] + told_l[slot4][1][me]) +
                                                             (told_l[slot4][2][me] + told_l[slot4][3][me]);
                    const float to = fmaxf(ml.y == 0.f ? -INFINITY : ml.x, lb == 0.f ? -INFINITY : mb);
                    fa = ml.y == 0.f ? 0.f : exp2_approx(ml.x - to);
                    fb = lb == 0.f ? 0.f : exp2_approx(mb - to);
                    ml = make_float2(to, ml.y * fa + lb * fb);
                }
                if (ml.y != ml.y || ml.y == 0.f) ml.x = 0.f;  // a NaN sum, or none, says it all
                if (me < heads) {
                    (whole ? row_ml : p.part_ml + share * GP)[me] = ml;
                    if (whole && p.a.lse) p.a.lse[q0 + me] = lse_of(ml);
                }
                if (whole) {
                    const float r = ml.y == 0.f ? 0.f : __frcp_rn(ml.y);
                    fa = ml.y == 0.f ? -1.f : fa * r;  // below 0: the head has no sum, and gives 0
                    fb *= r;
                }
                first_of[me] = fa;
                second_of[me] = fb;
            }
            bar_sync(1 + group, kSoftmax);
            tc_fence_after();
#pragma unroll 1
            for (int o = 0; o < S::kOBlocks; ++o) {
                // 64 rows of a product lie in the first 16 lanes of each warp's 32.
                const int d = S::kM == 64 ? quarter * 16 + lane : o * 128 + me;
                const bool in = (S::kM == 128 || lane < 16) && d < p.c.dim;
                constexpr int kStep = GP < 8 ? GP : 8;
#pragma unroll
                for (int j = 0; j < GP; j += kStep) {
                    // This group's O, what it put aside, and the same of the other.
                    Terms<S::kTerms, GP, kStep> own, other;
                    float own_f[kStep] = {}, other_f[kStep] = {}, v[kStep], fa[kStep], fb[kStep];
                    const uint32_t at = my_o + o * S::kPCols + j, at_f = my_f + o * GP + j;
                    const int away = group == 0 ? 1 : -1;
                    own.load(at);
                    if (aside) tmem_ld<kStep>(at_f, own_f);
                    if (n > 1) {
                        other.load(at + away * S::kOCols);
                        if (told_aside[slot4]) tmem_ld<kStep>(at_f + away * S::kFCols, other_f);
                    }
                    load_row<kStep>(first_of + j, fa);
                    load_row<kStep>(second_of + j, fb);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < kStep; ++i) {
                        // A factor that has come down to 0 still lets a value that is not finite through.
                        v[i] = (own_f[i] + own.sum(i, p.c.bf16)) * fa[i];
                        if (n > 1) v[i] += (other_f[i] + other.sum(i, p.c.bf16)) * fb[i];
                        if (fa[i] < 0.f) v[i] = 0.f;
                    }
                    if (whole) {
                        uint16_t* to = p.a.out + (size_t)(q0 + j) * p.c.dim + d;
#pragma unroll
                        for (int i = 0; i < kStep; ++i)
                            if (in && j + i < heads) to[i * p.c.dim] = from_float(v[i], p.c.bf16);
                    } else {
                        float* to = p.part_o + ((size_t)share * GP + j) * p.c.dim + d;
#pragma unroll
                        for (int i = 0; i < kStep; ++i)
                            if (in && j + i < heads) to[i * p.c.dim] = v[i];
                    }
                }
            }
            tc_fence_before();
            if (!whole) {
                // The group's P is free: its products are over, and it writes the next one behind a barrier.
                static_assert(S::kPBytes >= kJoin * GP * sizeof(float), "a join's factors fit where P was");
                const uint32_t at = p_buf + group * S::kPBytes - smem_addr(smem_raw);
                auto* factor = reinterpret_cast<float(*)[GP]>(smem_raw + at);
                join_row<GP>(p, x.total, x.blocks, row_start, x.tiles, q0, heads, row_ml, factor, joined[group],
                             &arrived[group], 1 + group, me);
            }
            x.t += n - 1;
            x.next(p);
        }
    }
    __syncwarp();
    __syncthreads();
    if (gave_up > 0) {
        // Every wait is over, so all warps see the same.  Copies and products
        // in flight end before the block does and tensor memory is freed.
        if (warp == kCopyK || warp == kCopyV) {
            const bool keys = warp == kCopyK;
            const int full0 = keys ? S::kFullK : S::kFullV;
            const int items = issued[keys ? 0 : 1], q_loads = keys ? issued[2] : 0;
#pragma unroll 1
            for (int i = max(0, items - S::kRing); i < items; ++i)
                mbar_wait(&bars[full0 + i % S::kRing], (i / S::kRing) & 1);
#pragma unroll 1
            for (int i = max(0, q_loads - 2); i < q_loads; ++i) mbar_wait(&bars[S::kQFull + (i & 1)], (i >> 1) & 1);
        } else if ((warp == kMmaS || warp == kMmaO) && lane == 0) {
            const int drain = S::kDrain + (warp == kMmaO);
            mma_commit(bar0 + drain * 8);
            mbar_wait(&bars[drain], 0);
        }
        __syncwarp();
        __syncthreads();
    }
    tc_fence_after();
    if (warp == kMmaS) tmem_dealloc(tmem, S::kTmemCols);
    // What sequences without slots give.
#pragma unroll 1
    for (int b = blockIdx.x; b < p.c.seqs; b += gridDim.x) {
        if (p.c.lens[b] > 0) continue;
        const size_t first = (size_t)b * p.a.q_heads;
#pragma unroll 1
        for (int i = tid; i < p.a.q_heads * (p.c.dim / 8); i += kThreads)
            reinterpret_cast<int4*>(p.a.out + first * p.c.dim)[i] = make_int4(0, 0, 0, 0);
        if (p.a.lse)
#pragma unroll 1
            for (int i = tid; i < p.a.q_heads; i += kThreads) p.a.lse[first + i] = -INFINITY;
    }
}

// Adds the heads' shares to the weights: p * 2^(tile's reference - row's) /
// sum.  Block c takes the tiles that block c of the first launch had, so its
// p may still be in L2; a warp takes every kWarps-th of them, and all of a
// tile's loads are in flight at once.
template <int GP>
__global__ void __launch_bounds__(kWeightThreads, 1) kv_weight_kernel(const __grid_constant__ AttendArgs p) {
    constexpr int kWarps = kWeightThreads / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    launch_dependents();
    grid_dependency_wait();
    Walk w;
    w.load(p.walk + blockIdx.x * Walk::kWords);
    int ahead = warp;  // tiles still to go to this warp's next
    bool enters = true;
    float2 ml = make_float2(0.f, 0.f);
#pragma unroll 1
    for (int tile = w.s; tile + ahead < w.e;) {
        const int left = w.tiles - w.t;
        if (ahead >= left) {  // on to the next row
            ahead -= left;
            tile += left;
            w.t = w.tiles - 1;
            w.next(p);
            enters = true;
            continue;
        }
        w.t += ahead;
        tile += ahead;
        ahead = kWarps;
        // Of a group in several parts, the block that has the first adds up all.
#pragma unroll 1
        for (int pt = 0; w.part == 0 && pt < p.parts; ++pt) {
            const int heads = min(GP, p.group - pt * GP);
            const float* wi = pt == 0 ? p.a.weight.row(w.b, w.h) : p.a.weight_out.row(w.b, w.h);
            float* wo = p.a.weight_out.row(w.b, w.h);
            const size_t x = tile + (size_t)pt * w.tiles;
            const int slot0 = w.t * kTile + lane * 4;
            const float4* const from = reinterpret_cast<const float4*>(p.p + x * GP * kTile) + lane;
            float4 y[GP];
            float tm = 0.f, sum[4];
            if (lane < heads) {
                tm = p.tile_m[x * GP + lane];
                if (enters || p.parts > 1) ml = p.row_ml[((size_t)w.row(p) + pt) * GP + lane];
            }
#pragma unroll
            for (int g = 0; g < GP; ++g)
                if (g < heads) y[g] = from[g * (kTile / 4)];
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[i] = slot0 + i < w.n ? wi[slot0 + i] : 0.f;
            const float f = ml.y == 0.f ? 0.f : exp2f(tm - ml.x) / ml.y;  // a NaN sum reaches every tile
#pragma unroll
            for (int g = 0; g < GP; ++g) {
                const float fg = __shfl_sync(kFullMask, f, g);
                if (g >= heads) break;
                sum[0] = fmaf(y[g].x, fg, sum[0]);
                sum[1] = fmaf(y[g].y, fg, sum[1]);
                sum[2] = fmaf(y[g].z, fg, sum[2]);
                sum[3] = fmaf(y[g].w, fg, sum[3]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (slot0 + i < w.n) wo[slot0 + i] = sum[i];
        }
        enters = false;
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
    return group == 1 ? 1 : group <= 4 ? 4 : group <= 8 || c.dim > 128 ? 8 : 16;
}

// The plan of a call, and its scratch when `scratch` is given.
struct Plan {
    AttendArgs args;
    int blocks;
    size_t bytes;
};

Plan make_plan(int sms, const KvCache& c, const KvAttend& a, void* scratch) {
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
    plan.blocks = sms;
    if ((size_t)plan.blocks > tiles) plan.blocks = (int)tiles;
    if (plan.blocks > kKvBlocks) plan.blocks = kKvBlocks;
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
    p.walk = nullptr;
    if (a.weight.data) {
        p.walk = static_cast<int*>(take(plan.blocks * Walk::kWords * 4));
        p.p = static_cast<float*>(take(tiles * kTile * gp * 4));
        p.tile_m = static_cast<float*>(take(tiles * gp * 4));
    }
    plan.bytes = bytes;
    return plan;
}

template <int DP, int GP>
cudaError_t launch(const Plan& plan, int device, cudaStream_t s, const CUtensorMap* maps, int* launches) {
    using Sh = Shape<DP, GP>;
    auto kernel = kv_attend_kernel<DP, GP>;
    static std::atomic<unsigned long long> allowed{0}, allowed_weights{0};
    cudaError_t e = allow_smem(kernel, (int)Sh::kSmem, device, allowed);
    if (e != cudaSuccess) return e;
    // Started early, it sets up its barriers and waits for the launch before it.
    e = launch_pdl(kernel, dim3(plan.blocks), dim3(kThreads), Sh::kSmem, s, plan.args, maps[0], maps[1], maps[2]);
    if (e != cudaSuccess) return e;
    ++*launches;
    if (!plan.args.p) return cudaSuccess;
    // Started early, its blocks take the SMs that the first launch leaves one
    // by one: the shared memory, which it does not use, keeps two of them from
    // sharing the SM that is free first (131072 slots: 10.2 us of it without, 5.6 with).
    constexpr int kAlone = 120 * 1024;
    e = allow_smem(kv_weight_kernel<GP>, kAlone, device, allowed_weights);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kv_weight_kernel<GP>, dim3(plan.blocks), dim3(kWeightThreads), kAlone, s, plan.args);
    if (e == cudaSuccess) ++*launches;
    return e;
}

template <int DP>
cudaError_t launch_dim(const Plan& plan, int gp, int device, cudaStream_t s, const CUtensorMap* maps, int* launches) {
    switch (gp) {
        case 1: return launch<DP, 1>(plan, device, s, maps, launches);
        case 4: return launch<DP, 4>(plan, device, s, maps, launches);
        case 8: return launch<DP, 8>(plan, device, s, maps, launches);
        default: break;
    }
    if constexpr (DP <= 128) return launch<DP, 16>(plan, device, s, maps, launches);
    return cudaErrorInvalidValue;
}

}  // namespace

size_t kv_attend_scratch(int sms, const KvCache& c, const KvAttend& a) {
    return make_plan(sms, c, a, nullptr).bytes;
}

cudaError_t kv_attend_launch(int device, int sms, cudaStream_t s, const KvCache& c, const KvAttend& a,
                             const KvState& state, int* launches) {
    Plan plan = make_plan(sms, c, a, state.scratch);
    plan.args.status = state.status;
    plan.args.spins = kv_spins_option();
    plan.args.withhold = kv_withhold_option();
    plan.args.done = state.mine;
    plan.args.clear = state.other;
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
    if (c.dim <= 64) return launch_dim<64>(plan, gp, device, s, maps, launches);
    if (c.dim <= 128) return launch_dim<128>(plan, gp, device, s, maps, launches);
    return launch_dim<256>(plan, gp, device, s, maps, launches);
}

}  // namespace topk
