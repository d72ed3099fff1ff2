// topk_sample_rows: a token from each row of logits, with temperature, top-k,
// top-p and min-p, by one given uniform number.
//
// With the row in TopK order (value descending, the lower column first among
// equals), weights w_i = 2^(c x_i), c = log2(e) / temperature, and C(i) the
// weights up to and with i, every rule keeps a prefix of the order, and the
// token is where C passes u times the kept weight.  So all that is ever asked
// is where C (or the rank) passes a number, and how large C is there.
//
// One cluster of blocks has a row.  Bound by HBM for large batches in float32
// and by instructions in 16 bits: an exponential and a bin for each element.
//   1. The row's largest value.
//   2. The weights of each octave (factor of two below the largest), 64 of
//      them.  A weight is a 24-bit number times 2^octave, so octaves are sums of
//      integers: exact, in any order.  Each thread adds in cells of its own.
//   3. The octave that is asked for is cut into 64 parts, and the part again,
//      until what is left fits a list (or is one value, whose elements are
//      equal).  Usually everything down to that octave fits at once.
//   4. The list is sorted and summed up, and gives the answer.
//
// A weight is off by 2^-21.5 of itself, so a number that lies within 2^-20 of
// an element's border (relative, of the smaller side) cannot be told from its
// neighbour's.  Such a row goes through 2 to 4 once more with weights of 42
// bits, right to 2^-36.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <cfloat>
#include <cmath>
#include <initializer_list>

#include "../../include/topk.h"
#include "topk_device.cuh"
#include "topk_kv.cuh"

namespace cg = cooperative_groups;

namespace topk {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kBins = 64;
constexpr int kList = 1024;         // elements that a list has room for
constexpr int kMostBlocks = 8;      // of a cluster
constexpr int kBits = 41;           // a weight of 1 in its octave is 2^kBits
constexpr int kPart = 21;           // bits of a 42-bit weight that a cell adds up at a time
constexpr int kCellAdds = 240;      // elements that a cell has room for: 240 * 2^24 < 2^32
constexpr int kListShift = 11;      // and in a list 2^(kBits + kListShift): 1024 of them stay below 2^63
constexpr int kMaxCols = 1 << 21;   // 2^21 weights of an octave stay below 2^63

struct SampleArgs {
    const char* logits;
    long long stride;  // bytes between rows
    int rows, cols;
    topk_sampling p;
    double log_min_p;  // of p.min_p
    int pieces;        // of a warp's share, as many of its elements as cells have room for in each
    const float* u;
    int32_t* token;
    float* logp;
    int fine;  // 1: 42 bits from the start
};

enum Type { kF16, kBf16, kF32 };

template <Type kType>
struct Logit {
    static constexpr int kBytes = kType == kF32 ? 4 : 2, kMany = 16 / kBytes;  // of a vector
    using Word = typename std::conditional<kType == kF32, unsigned, uint16_t>::type;
    static constexpr Word kNone = kType == kF32 ? 0xFF800000u : kType == kBf16 ? 0xFF80u : 0xFC00u;  // -inf

    static __device__ __forceinline__ float widen(Word w) {
        if constexpr (kType == kF32) return __uint_as_float(w);
        else if constexpr (kType == kBf16) return __uint_as_float((unsigned)w << 16);
        else return __half2float(__ushort_as_half(w));
    }
    static __device__ __forceinline__ float at(const int4& v, int i) {
        const unsigned w[4] = {(unsigned)v.x, (unsigned)v.y, (unsigned)v.z, (unsigned)v.w};
        if constexpr (kType == kF32) return __uint_as_float(w[i]);
        else if constexpr (kType == kBf16) return __uint_as_float(i & 1 ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
        else return __half2float(__ushort_as_half((unsigned short)(i & 1 ? w[i >> 1] >> 16 : w[i >> 1] & 0xFFFFu)));
    }
    // The type's values in order, numbered; -0 and +0 have a number each.
    static __device__ __forceinline__ unsigned number(float x) {
        if constexpr (kType == kF16) {
            const unsigned b = __half_as_ushort(__float2half_rn(x));
            return b & 0x8000u ? 0xFFFFu - b : b | 0x8000u;
        } else {
            const unsigned b = __float_as_uint(x), k = b ^ ((unsigned)((int)b >> 31) | 0x80000000u);
            return kType == kBf16 ? k >> 16 : k;
        }
    }
    static __device__ __forceinline__ float value(unsigned k) {
        if constexpr (kType == kF16)
            return __half2float(__ushort_as_half((unsigned short)(k & 0x8000u ? k & 0x7FFFu : 0xFFFFu - k)));
        if constexpr (kType == kBf16) k <<= 16;
        return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : kType == kBf16 ? ~k & 0xFFFF0000u : ~k);
    }
};

// What the blocks of a cluster tell each other; two of them, used in turn, so
// that one barrier an exchange is enough.
struct alignas(16) Exchange {
    unsigned long long bins[kBins];
    unsigned long long list[kList];
    int count;
    float top;
};

struct Shared {
    Exchange exchange[2];
    unsigned long long list[kList];     // the cluster's, sorted
    unsigned long long through[kList];  // weights up to and with each
    unsigned long long bins[kBins];     // of the cluster
    unsigned long long above[kBins + 1];   // sums of the bins before each; the last one: of all
    unsigned long long octave[kBins];      // weights of each octave, in its own unit
    unsigned long long before[kBins + 1];  // weights above each octave; the last one: of all
    int upper[kBins], lower[kBins];     // bounds on the number of elements down to and with each octave
    unsigned long long table[64];       // 2^(i / 64), times 2^kBits
    unsigned long long scan[kWarps];
    float warp_top[kWarps];
    float min_from;
};

// Sums of weights are whole numbers of 2^-kBits times a weight of 1 in the
// largest value's octave; within an octave o, of 2^-(kBits + o).
using Sum = unsigned long long;

// a * f, 0 <= f <= 1, rounded down or up.
__device__ __forceinline__ Sum times(Sum a, float f, bool up) {
    const unsigned bits = __float_as_uint(f);
    const int exponent = bits >> 23;
    const Sum mantissa = exponent ? (bits & 0x7FFFFFu) | 0x800000u : 0u;  // what is below 2^-126 is 0
    const Sum low = a * mantissa, high = __umul64hi(a, mantissa);
    const int down = 150 - exponent;  // 23 and more
    if (down >= 128) return up && mantissa && a;
    const Sum whole = down >= 64 ? high >> (down - 64) : high << (64 - down) | low >> down;
    const Sum rest = down >= 64 ? low | (high & ((1ull << (down - 64)) - 1)) : low << (64 - down);
    return whole + (up && rest);
}

enum What { kCount, kFast, kFineHigh, kFineLow };
enum By { kOctaves, kLinear, kNumbers };

constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: what is added to it is rounded to a whole number

// The weight of x in its octave with 42 bits: 2^f from a table of 2^(i / 64)
// and the series of e^a for the rest, with what is lost in a sum or product
// kept as a second number.
__device__ __noinline__ unsigned long long fine_weight(float x, float top, float c_hi, float c_lo,
                                                       const unsigned long long* table) {
    const float d = x - top, v = d - x, d_lo = (x - (d - v)) - (top + v);
    const float n = __fmaf_rd(d, c_hi, kMagic) - kMagic;
    const float p = d * c_hi;
    const float f = p - n;
    const float f_lo = fmaf(d, c_hi, -p) + fmaf(d, c_lo, d_lo * c_hi) + (p - (f + n));
    const int i = min(63, (int)(f * 64.f));
    const float r = f - i * 0.015625f;
    constexpr float kLn2 = 0.693147182464599609375f, kLn2Low = -1.9046543e-9f;
    const float a = r * kLn2, a_lo = fmaf(r, kLn2, -a) + fmaf(r, kLn2Low, f_lo * kLn2);
    const float all = a + a_lo, q = all * all * fmaf(all, fmaf(all, 1.f / 24, 1.f / 6), 0.5f);
    constexpr float kScale = 17592186044416.f;  // 2^44
    const long long g = (__float2ll_rn(a * kScale) + __float2ll_rn((a_lo + q) * kScale)) << 20;
    return table[i] + (unsigned long long)(__mul64hi((long long)(table[i] << 20), g) >> 20);
}

template <Type kType>
struct Row {
    using L = Logit<kType>;
    const char* base;   // 16-byte aligned, at or before the row's first element
    int skip, end;      // elements of the first vector before the row; skip + cols
    int v0, v1;         // this warp's vectors
    float top;          // the largest value
    // Fast weights are 2^(c (x - ref)); ref is 0 where c * top is small enough
    // for that, else the largest value (then what differs from it too much to
    // be subtracted exactly has no weight).  Fine ones have ref = top.
    float ref, c_hi, c_lo, low;  // low: what lies below it has no weight
    int octave0;                 // bits of kMagic plus the largest value's exponent
    bool fine;

    __device__ __forceinline__ int4 load(int v) const {
        const int at = v * L::kMany;
        if (at >= skip && at + L::kMany <= end) return __ldg(reinterpret_cast<const int4*>(base) + v);
        union { int4 v; typename L::Word w[L::kMany]; } r;
        for (int i = 0; i < L::kMany; ++i)
            r.w[i] = at + i >= skip && at + i < end ? __ldg(reinterpret_cast<const typename L::Word*>(base) + at + i) : L::kNone;
        return r.v;
    }

    // f(vector, its number) for each of the warp's vectors, by all lanes at once; what is past the end is -inf.
    template <typename F>
    __device__ __forceinline__ void each_vector(int from, int to, F f) const {
        constexpr int kUnroll = 4;
        const int lane = threadIdx.x & 31;
        union { int4 v; typename L::Word w[L::kMany]; } none;
        for (int i = 0; i < L::kMany; ++i) none.w[i] = L::kNone;
        for (int v = from + lane; v - lane < to; v += 32 * kUnroll) {
            int4 raw[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) raw[u] = v + 32 * u < to ? load(v + 32 * u) : none.v;
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) f(raw[u], v + 32 * u);
        }
    }

    // Bits of kMagic plus the exponent of x's weight.
    __device__ __forceinline__ float magic(float x) const { return __fmaf_rd(x - ref, c_hi, kMagic); }
    __device__ __forceinline__ int octave(float x) const { return octave0 - __float_as_int(magic(x)); }

    // The weight of x in its octave, 2^23 to 2^24.
    __device__ __forceinline__ unsigned fast(float x, float t) const {
        const float d = x - ref, n = t - kMagic, f = __saturatef(fmaf(d, c_lo, fmaf(d, c_hi, -n)));
        float w;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w) : "f"(f));
        return __float_as_uint(w) - 0x3F000000u;
    }
    // The same with 42 bits, 2^41 to 2^42.
    __device__ __forceinline__ unsigned long long slow(float x, const unsigned long long* table) const {
        return fine_weight(x, top, c_hi, c_lo, table);
    }
    __device__ __forceinline__ unsigned long long weight(float x, const unsigned long long* table) const {
        return fine ? slow(x, table) : (unsigned long long)fast(x, magic(x)) << (kBits - 23);
    }
};

// A barrier of the cluster that makes the blocks' shared memory visible to one
// another (topk_kv_evict.cu has the reason for its form).
__device__ __forceinline__ void cluster_sync(int blocks) {
    __syncthreads();
    if (blocks == 1) return;
    if (threadIdx.x == 0) asm volatile("fence.acq_rel.cluster;" ::: "memory");
    asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// A region: the elements from `lo` to `hi`, with the weights above it, and how
// those in it are cut into 64 bins, the largest values first.
struct Region {
    float lo, hi;
    By by;
    float scale;   // kLinear
    unsigned number;  // kNumbers: hi's
    int shift;
};

template <Type kType>
struct Sampler {
    using L = Logit<kType>;
    Row<kType> row;
    Shared& s;
    unsigned* cells;  // [kBins][kThreads]
    int blocks, rank, turn, pieces;
    int listed = 0;       // elements in the list
    int list_octave = 0;  // the octave in which it begins
    Sum list_from = 0;    // weights in that octave above it

    __device__ Sampler(Shared& s, unsigned* cells) : s(s), cells(cells) {}

    __device__ __forceinline__ Exchange& mine() { return s.exchange[turn]; }
    __device__ __forceinline__ const Exchange* theirs(int r) {
        return blocks == 1 ? &s.exchange[turn] : cg::this_cluster().map_shared_rank(&s.exchange[turn], r);
    }

    __device__ __forceinline__ int bin(const Region& g, float x) const {
        if (g.by == kOctaves) return row.octave(x);
        if (g.by == kLinear) return kBins - 1 - min(kBins - 1, (int)((x - g.lo) * g.scale));
        return (int)((g.number - L::number(x + 0.f)) >> g.shift);
    }

    // Adds up `what` of the region's elements by bins over the cluster, into s.bins.
    template <bool kHot>
    __device__ void add_up(const Region& g, What what, int shift) {
        const int tid = threadIdx.x;
        Sum sum = 0;  // of bin tid / 4, by a quarter of the threads
        constexpr int step = 32 * (kCellAdds / L::kMany);  // vectors of a warp that its cells have room for
        int from = row.v0;
        for (int piece = 0; piece < pieces; ++piece, from += step) {
            for (int b = 0; b < kBins; ++b) cells[b * kThreads + tid] = 0;
            const int to = min(from + step, row.v1);
            if constexpr (kHot) {
                row.each_vector(from, to, [&](const int4& v, int) {
#pragma unroll
                    for (int i = 0; i < L::kMany; ++i) {
                        const float x = L::at(v, i);
                        if (x >= g.lo) {
                            const float t = row.magic(x);
                            cells[min((unsigned)(row.octave0 - __float_as_int(t)), kBins - 1u) * kThreads + tid] += row.fast(x, t);
                        }
                    }
                });
            } else {
                row.each_vector(from, to, [&](const int4& v, int) {
                    for (int i = 0; i < L::kMany; ++i) {
                        const float x = L::at(v, i);
                        if (x >= g.lo && x <= g.hi) {
                            unsigned w = 1;
                            if (what == kFast) w = row.fast(x, row.magic(x));
                            if (what == kFineHigh) w = (unsigned)(row.slow(x, s.table) >> kPart);
                            if (what == kFineLow) w = (unsigned)row.slow(x, s.table) & ((1u << kPart) - 1);
                            cells[min((unsigned)bin(g, x), kBins - 1u) * kThreads + tid] += w;
                        }
                    }
                });
            }
            __syncthreads();
            const uint4* from4 = reinterpret_cast<const uint4*>(cells + (tid >> 2) * kThreads + (tid & 3) * (kThreads / 4));
#pragma unroll 4
            for (int i = 0; i < kThreads / 16; ++i) {
                const uint4 q = from4[(i + tid) & (kThreads / 16 - 1)];
                sum += (Sum)q.x + q.y + ((Sum)q.z + q.w);
            }
            __syncthreads();
        }
        sum += __shfl_xor_sync(kFullMask, sum, 1);
        sum += __shfl_xor_sync(kFullMask, sum, 2);
        if ((tid & 3) == 0) mine().bins[tid >> 2] = sum;
        cluster_sync(blocks);
        if (tid < 32) {  // two bins each
            Sum v[kMostBlocks][2] = {};
#pragma unroll
            for (int r = 0; r < kMostBlocks; ++r) {
                if (r >= blocks) break;
                const ulonglong2 q = reinterpret_cast<const ulonglong2*>(theirs(r)->bins)[tid];
                v[r][0] = q.x;
                v[r][1] = q.y;
            }
            Sum b0 = 0, b1 = 0;
#pragma unroll
            for (int r = 0; r < kMostBlocks; ++r) {
                b0 += v[r][0];
                b1 += v[r][1];
            }
            b0 = (what == kFineLow ? s.bins[2 * tid] : 0) + (b0 << shift);
            b1 = (what == kFineLow ? s.bins[2 * tid + 1] : 0) + (b1 << shift);
            s.bins[2 * tid] = b0;
            s.bins[2 * tid + 1] = b1;
            write_scan(s.above, b0, b1);
        }
        turn ^= 1;
        __syncthreads();
    }
    // Sums of the bins before each: two of a lane's, by one warp.
    static __device__ void write_scan(Sum* to, Sum b0, Sum b1) {
        const int lane = threadIdx.x & 31;
        Sum x = b0 + b1;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const Sum y = __shfl_up_sync(kFullMask, x, d);
            if (lane >= d) x += y;
        }
        to[2 * lane] = x - b0 - b1;
        to[2 * lane + 1] = x - b1;
        if (lane == 31) to[kBins] = x;
    }
    // The first bin up to and with which the sums are more than t (strict) or
    // not less; the last one that has anything if t is past them all.
    static __device__ int bin_of(const Sum* sums, Sum t, bool strict) {
        const int i = threadIdx.x;
        const Sum next = i < kBins ? sums[i + 1] : 0, all = sums[kBins];
        const int at = __syncthreads_count(i < kBins && (strict ? next <= t : next < t));
        return min(at, __syncthreads_count(i < kBins && next < all));
    }
    __device__ void add_up_weights(const Region& g) {
        if (row.fine) {
            add_up<false>(g, kFineHigh, kPart);
            add_up<false>(g, kFineLow, 0);
        } else if (g.by == kOctaves) {
            add_up<true>(g, kFast, kBits - 23);
        } else {
            add_up<false>(g, kFast, kBits - 23);
        }
    }

    // The smallest number k in [lo, hi] for which f(value of k), which is true
    // from some value on and for hi, is true.  All lanes of each warp.
    template <typename F>
    __device__ unsigned first(unsigned lo, unsigned hi, F f) {
        const int lane = threadIdx.x & 31;
        while (lo < hi) {
            const unsigned step = (hi - lo) / 32 + 1;
            const unsigned long long at = lo + (unsigned long long)lane * step;
            const unsigned yes = __ballot_sync(kFullMask, at >= hi || f(L::value((unsigned)at)));
            const int k = yes ? __ffs(yes) - 1 : 32;  // the first lane that says so
            const unsigned long long up = lo + (unsigned long long)k * step;
            if (k > 0) lo = lo + (unsigned)(k - 1) * step + 1;
            hi = up < hi ? (unsigned)up : hi;
        }
        return hi;
    }
    // Bins b0 to b1 of a region.
    __device__ Region part(const Region& g, int b0, int b1) {
        const unsigned klo = L::number(g.lo), khi = L::number(g.hi);
        auto upto = [&](int b) {
            return first(klo, khi, [&](float x) { return x >= g.lo && bin(g, x) <= b; });
        };
        Region r = g;
        r.lo = L::value(upto(b1));
        if (b0 > 0) r.hi = L::value(upto(b0 - 1) - 1);
        return r;
    }
    // How a region is cut; `level` counts the cuts before.
    __device__ void cut(Region& g, int level) {
        const float scale = kBins / (g.hi - g.lo);
        if (level == 0 && scale > 0 && scale < FLT_MAX) {
            g.by = kLinear;
            g.scale = scale;
            return;
        }
        g.by = kNumbers;
        g.number = L::number(g.hi + 0.f);
        const unsigned range = g.number - L::number(g.lo);
        g.shift = 0;
        while (range >> g.shift >= kBins) ++g.shift;
    }

    // Collects the region's elements, at most kList, and sorts and sums them up.
    __device__ void gather(const Region& g, int octave, Sum in_octave) {
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
        if (tid == 0) mine().count = 0;
        __syncthreads();
        row.each_vector(row.v0, row.v1, [&](const int4& v, int at) {
#pragma unroll
            for (int i = 0; i < L::kMany; ++i) {
                const float x = L::at(v, i);
                if (x >= g.lo && x <= g.hi) {
                    const int n = atomicAdd(&mine().count, 1);
                    const unsigned b = __float_as_uint(x + 0.f), key = b ^ ((unsigned)((int)b >> 31) | 0x80000000u);
                    if (n < kList)
                        mine().list[n] = (unsigned long long)key << 32 | ~(unsigned)(at * L::kMany + i - row.skip);
                }
            }
        });
        cluster_sync(blocks);
        int n = 0;
        for (int r = 0; r < blocks; ++r) {
            const Exchange* e = theirs(r);
            const int some = min(e->count, kList);
            for (int i = tid; i < some; i += kThreads)
                if (n + i < kList) s.list[n + i] = e->list[i];
            n += some;
        }
        n = min(n, kList);
        turn ^= 1;
        const int size = next_pow2(max(n, 2));
        for (int i = n + tid; i < size; i += kThreads) s.list[i] = 0;
        block_sort_smem_desc(s.list, size);
        constexpr int kPer = kList / kThreads;
        Sum own[kPer], sum = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int at = tid * kPer + i;
            if (at < n) {
                const float x = listed_value(at);
                sum += row.weight(x, s.table) << kListShift >> (row.octave(x) - octave);
            }
            own[i] = sum;
        }
        Sum x = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const Sum y = __shfl_up_sync(kFullMask, x, d);
            if (lane >= d) x += y;
        }
        if (lane == 31) s.scan[warp] = x;
        __syncthreads();
        Sum before = x - sum;
        for (int w = 0; w < warp; ++w) before += s.scan[w];
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (tid * kPer + i < n) s.through[tid * kPer + i] = before + own[i];
        __syncthreads();
        listed = n;
        list_octave = octave;
        list_from = in_octave;
    }
    __device__ __forceinline__ float listed_value(int i) const {
        const unsigned k = (unsigned)(s.list[i] >> 32);
        return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
    }
    // Weights up to and with element i - 1 of the list.
    __device__ __forceinline__ Sum list_sum(int i) const {
        return s.before[list_octave] + ((list_from + (i > 0 ? s.through[i - 1] >> kListShift : 0)) >> list_octave);
    }

    // An element of the order: the weights before it and up to and with it,
    // and where it is: at `index` in the list, or the `index`-th that equals
    // `value`.
    struct Place {
        Sum before, through;
        int index;
        bool in_list;
        float value;
    };

    __device__ Place in_list(Sum t, bool strict) {
        const Sum from = s.before[list_octave], rel = t > from ? (t - from) << list_octave : 0;
        const Sum edge = rel > list_from ? (rel - list_from) << kListShift : 0;
        int count = 0;
        for (int i = threadIdx.x; i - (int)threadIdx.x < listed; i += kThreads)
            count += __syncthreads_count(i < listed && (strict ? s.through[i] <= edge : s.through[i] < edge));
        const int i = max(min(count, listed - 1), 0);
        return {list_sum(i), list_sum(i + 1), i, true, listed_value(i)};
    }

    // The first element up to and with which the weights are more than t
    // (strict) or not less.
    __device__ Place find(Sum t, bool strict) {
        if (listed && t >= list_sum(0) && t <= list_sum(listed)) return in_list(t, strict);
        const int o = bin_of(s.before, t, strict);
        Region g = {row.low, row.top, kOctaves, 0.f, 0u, 0};
        if (s.upper[o] <= kList) {  // all down to there
            gather(part(g, 0, o), 0, 0);
            return in_list(t, strict);
        }
        g = part(g, o, o);
        const Sum rel = t > s.before[o] ? (t - s.before[o]) << o : 0;
        Sum above = 0, room = most(s.octave[o]);  // both of the octave
        for (int level = 0; room > kList && g.lo != g.hi; ++level) {
            cut(g, level);
            add_up_weights(g);
            const int b = bin_of(s.above, rel > above ? rel - above : 0, strict);
            above += s.above[b];
            room = most(s.bins[b]);
            g = part(g, b, b);
        }
        if (room <= kList) {
            gather(g, o, above);
            return in_list(t, strict);
        }
        return equals(g.hi, o, above, strict ? (rel > above ? rel - above : 0) / row.weight(g.hi, s.table)
                                             : ((rel > above ? rel - above : 1) - 1) / row.weight(g.hi, s.table));
    }
    // The i-th, from 0, of the elements that equal x, with `above` in octave o above them.
    __device__ Place equals(float x, int o, Sum above, Sum i) {
        const Sum w = row.weight(x, s.table), from = s.before[o];
        i = min(i, (Sum)kMaxCols);
        return {from + ((above + i * w) >> o), from + ((above + (i + 1) * w) >> o), (int)i, false, x};
    }
    // Weights of 2^kBits at least: how many there are at most.
    __device__ __forceinline__ static Sum most(Sum sum) { return sum / ((1ull << kBits) - (1ull << (kBits - 15))); }

    // Weights of the first k elements of the order.
    __device__ Sum first_k(int k) {
        const int reach = __syncthreads_count(threadIdx.x < kBins - 1 && s.lower[threadIdx.x] < k);  // no further than here
        const Region all = {row.low, row.top, kOctaves, 0.f, 0u, 0};
        if (s.upper[reach] <= kList) {
            gather(part(all, 0, reach), 0, 0);
            return list_sum(min(k, listed));
        }
        add_up<false>(all, kCount, 0);
        if (s.above[kBins] <= (Sum)k) return s.before[kBins];
        const int o = bin_of(s.above, k, false);
        Sum need = k - s.above[o], room = s.bins[o], above = 0;
        Region g = part(all, o, o);
        for (int level = 0; room > kList && g.lo != g.hi; ++level) {
            cut(g, level);
            add_up<false>(g, kCount, 0);
            const int b = bin_of(s.above, need, false);
            need -= s.above[b];
            room = s.bins[b];
            add_up_weights(g);
            above += s.above[b];
            g = part(g, b, b);
        }
        if (room <= kList) {
            gather(g, o, above);
            return list_sum((int)min(need, (Sum)listed));
        }
        return equals(g.hi, o, above, need - 1).through;
    }

    // Weights of the values from `from` on.
    __device__ Sum down_to(float from) {
        if (listed && list_octave == 0 && list_from == 0 && listed_value(listed - 1) < from) {
            int count = 0;
            for (int i = threadIdx.x; i - (int)threadIdx.x < listed; i += kThreads)
                count += __syncthreads_count(i < listed && listed_value(i) >= from);
            return list_sum(count);
        }
        const Region g = {fmaxf(from, row.low), row.top, kOctaves, 0.f, 0u, 0};
        add_up_weights(g);
        Sum all = 0;
        for (int i = 0; i < kBins; ++i) all += s.bins[i] >> i;
        return all;
    }

    // The sums of all octaves -> what is above each, and bounds on numbers.
    __device__ void octaves() {
        const int lane = threadIdx.x;
        if (lane < 32) {
            const Sum b0 = s.bins[2 * lane], b1 = s.bins[2 * lane + 1];
            s.octave[2 * lane] = b0;
            s.octave[2 * lane + 1] = b1;
            write_scan(s.before, b0 >> 2 * lane, b1 >> (2 * lane + 1));
            int upper = (int)(most(b0) + most(b1)), lower = (int)(least(b0) + least(b1));  // 2^21 and a little at most
            const int upper1 = (int)most(b1), lower1 = (int)least(b1);
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int yu = __shfl_up_sync(kFullMask, upper, d), yl = __shfl_up_sync(kFullMask, lower, d);
                if (lane >= d) {
                    upper += yu;
                    lower += yl;
                }
            }
            s.upper[2 * lane] = upper - upper1;
            s.upper[2 * lane + 1] = upper;
            s.lower[2 * lane] = lower - lower1;
            s.lower[2 * lane + 1] = lower;
        }
        __syncthreads();
    }
    // Weights of 2^(kBits + 1) at most: how many there are at least.
    __device__ __forceinline__ static Sum least(Sum sum) { return (sum + (2ull << kBits) - 1) >> (kBits + 1); }

    // The column of the i-th element that equals x, counting from 0; by the
    // warp that has it, -1 from all others.
    __device__ int column_of(float x, int i) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        auto matches = [&](const int4& v) {
            unsigned m = 0;
#pragma unroll
            for (int e = 0; e < L::kMany; ++e) m |= (L::at(v, e) == x ? 1u : 0u) << e;
            return m;
        };
        int count = 0;
        row.each_vector(row.v0, row.v1, [&](const int4& v, int) { count += __popc(matches(v)); });
        count = __reduce_add_sync(kFullMask, count);
        if (lane == 0) mine().bins[warp] = (unsigned long long)count;
        cluster_sync(blocks);
        int before = 0;
        for (int r = 0; r <= rank; ++r)
            for (int w = 0; w < (r == rank ? warp : kWarps); ++w) before += (int)theirs(r)->bins[w];
        // Whether the last one of all is meant: rounding may have put i past it.
        int all = 0;
        for (int r = 0; r < blocks; ++r)
            for (int w = 0; w < kWarps; ++w) all += (int)theirs(r)->bins[w];
        turn ^= 1;
        i = min(i, all - 1);
        int column = -1;
        if (i < before || i >= before + count) return column;
        for (int v = row.v0; v < row.v1 && column < 0; v += 32) {
            unsigned m = v + lane < row.v1 ? matches(row.load(v + lane)) : 0u;
            const int some = __popc(m);
            int sum = some;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int y = __shfl_up_sync(kFullMask, sum, d);
                if (lane >= d) sum += y;
            }
            const int first = before + sum - some;
            int found = -1;
            if (i >= first && i < first + some) {
                for (int k = first; k < i; ++k) m &= m - 1;
                found = (v + lane) * L::kMany + __ffs(m) - 1 - row.skip;
            }
            column = __reduce_max_sync(kFullMask, found);
            before += __shfl_sync(kFullMask, sum, 31);
        }
        return column;
    }
};

// Whether t is so near one of an element's borders that weights of 24 bits do not tell on which side it lies.
__device__ __forceinline__ bool near_border(Sum t, Sum before, Sum through, Sum all) {
    const Sum room = min(t, all > t ? all - t : 0) >> 20;
    return (before > 0 && (t > before ? t - before : 0) < room) || (through < all && (through > t ? through - t : 0) < room);
}

template <Type kType>
__global__ void __launch_bounds__(kThreads, 2) sample_rows_kernel(const __grid_constant__ SampleArgs a) {
    using L = Logit<kType>;
    extern __shared__ __align__(16) unsigned cells[];
    __shared__ Shared s;
    cg::cluster_group cluster = cg::this_cluster();
    const int blocks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int r = blockIdx.x / blocks, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    grid_dependency_wait();  // launched early (launch_pdl): the previous kernel's writes first

    Sampler<kType> sampler(s, cells);
    Row<kType>& row = sampler.row;
    sampler.blocks = blocks;
    sampler.rank = rank;
    sampler.turn = 0;
    sampler.pieces = a.pieces;
    const char* start = a.logits + r * a.stride;
    row.skip = (int)((reinterpret_cast<uintptr_t>(start) & 15) / L::kBytes);
    row.base = start - row.skip * L::kBytes;
    row.end = row.skip + a.cols;
    const int vectors = (row.end + L::kMany - 1) / L::kMany;
    // Contiguous shares: of a block, and of each of its warps.
    const int parts = blocks * kWarps, share = (vectors + parts - 1) / parts;
    row.v0 = min((rank * kWarps + warp) * share, vectors);
    row.v1 = min(row.v0 + share, vectors);

    // The largest value; NaN if there is one.
    float top = -INFINITY;
    row.each_vector(row.v0, row.v1, [&](const int4& v, int) {
#pragma unroll
        for (int i = 0; i < L::kMany; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(top) : "f"(L::at(v, i)));
    });
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const float y = __shfl_xor_sync(kFullMask, top, d);
        asm("max.NaN.f32 %0, %0, %1;" : "+f"(top) : "f"(y));
    }
    if (lane == 0) s.warp_top[warp] = top;
    __syncthreads();
    if (tid == 0) {
        for (int w = 0; w < kWarps; ++w) asm("max.NaN.f32 %0, %0, %1;" : "+f"(top) : "f"(s.warp_top[w]));
        s.exchange[0].top = top;
    }
    cluster_sync(blocks);
    for (int b = 0; b < blocks; ++b) {
        const float y = sampler.theirs(b)->top;
        if (b == 0) top = y;
        asm("max.NaN.f32 %0, %0, %1;" : "+f"(top) : "f"(y));
    }
    sampler.turn ^= 1;
    top += 0.f;  // -0 is 0
    row.top = top;

    float temperature = a.p.temperatures ? a.p.temperatures[r] : a.p.temperature;
    const float top_p = a.p.top_ps ? a.p.top_ps[r] : a.p.top_p, min_p = a.p.min_ps ? a.p.min_ps[r] : a.p.min_p;
    const int top_k = a.p.top_ks ? a.p.top_ks[r] : a.p.top_k;
    float u = a.u[r];
    const bool sane = top >= -FLT_MAX && top <= FLT_MAX && temperature >= 0 && top_p == top_p && min_p == min_p && u == u;
    if (!sane) {  // the whole cluster leaves here
        if (rank == 0 && tid == 0) {
            a.token[r] = -1;
            a.logp[r] = NAN;
        }
        cluster_sync(blocks);
        return;
    }
    const bool greedy = temperature == 0;
    u = greedy ? 0.f : fminf(fmaxf(u, 0.f), 0x1.fffffep-1f);
    const bool cut_p = top_p < 1 && !greedy, cut_m = min_p > 0 && !greedy, cut_k = top_k > 0 && top_k < a.cols && !greedy;
    temperature = fminf(fmaxf(temperature, 0x1p-60f), 0x1p60f);
    // log2(e) / temperature as a sum of two.
    constexpr float kLog2e = 1.44269502162933349609375f, kLog2eLow = 1.92596299e-8f;
    row.c_hi = kLog2e / temperature;
    row.c_lo = (fmaf(-row.c_hi, temperature, kLog2e) + kLog2eLow) / temperature;
    // 61.9 octaves below the largest value: no element from there on is in
    // octave 64, whatever the rounding.
    row.low = fmaxf(__fmaf_ru(temperature, -42.9f, top), -FLT_MAX);
    float min_from = -INFINITY;
    if (cut_m) {
        if (tid == 0) {  // 64-bit arithmetic is slow: once a block
            const double log_min = a.p.min_ps ? log(fmin((double)min_p, 1.0)) : a.log_min_p;
            s.min_from = __double2float_ru((double)top + (double)temperature * log_min);
        }
        __syncthreads();
        min_from = s.min_from;
        if (!cut_p) row.low = fmaxf(row.low, min_from);
    }

    for (int pass = a.fine; pass < 2; ++pass) {
        row.fine = pass == 1;
        row.ref = row.fine || fabsf(top) * row.c_hi >= 128.f ? top : 0.f;
        row.octave0 = __float_as_int(row.magic(top));
        if (row.fine && tid < 64) s.table[tid] = (unsigned long long)__double2ll_rn(exp2(tid / 64.0) * 0x1p41);
        __syncthreads();
        sampler.listed = 0;
        const Region all = {row.low, top, kOctaves, 0.f, 0u, 0};
        sampler.add_up_weights(all);
        sampler.octaves();
        Sum kept = s.before[kBins];
        if (cut_k) kept = sampler.first_k(top_k);
        if (cut_p) {
            const Sum t = times(kept, fmaxf(top_p, 0.f), true);
            const auto at = sampler.find(t, false);
            if (!row.fine && near_border(t, at.before, at.through, kept)) continue;
            kept = min(kept, at.through);
            if (cut_m) kept = min(kept, sampler.down_to(min_from));
        }
        const Sum t = times(kept, u, false);
        const auto at = sampler.find(t, true);
        if (!row.fine && near_border(t, at.before, at.through, kept)) continue;
        int column;
        bool writes;
        if (at.in_list) {
            column = (int)~(unsigned)s.list[at.index];
            writes = rank == 0 && tid == 0;
        } else {
            column = sampler.column_of(at.value, at.index);
            writes = column >= 0 && lane == 0;
        }
        if (writes) {
            const Sum w = at.through - at.before, rest = kept > w ? kept - w : 0;
            // log(w / kept): near 1 by what the others have, else from the
            // value itself, which is exact.
            float logp;
            if (greedy || rest == 0) {
                logp = 0.f;
            } else if (w > rest) {
                logp = log1pf(-((float)rest / (float)kept));
            } else {
                const double c = (double)row.c_hi + row.c_lo;
                const int octave0 = row.octave0 - __float_as_int(kMagic);
                logp = (float)((((double)at.value - row.ref) * c - octave0 + kBits - log2f((float)kept)) *
                               0.69314718055994530942);
            }
            a.token[r] = column;
            a.logp[r] = logp;
        }
        break;
    }
    cluster_sync(blocks);  // no block leaves while another reads its shared memory
}

template <Type kType>
cudaError_t launch(SampleArgs& a, int device, int sms, cudaStream_t s) {
    auto kernel = sample_rows_kernel<kType>;
    constexpr int kSmem = kBins * kThreads * 4;
    static std::atomic<unsigned long long> allowed{0};
    const cudaError_t e = allow_smem(kernel, kSmem, device, allowed);
    if (e != cudaSuccess) return e;
    int blocks = 1;
    while (blocks < kMostBlocks && a.cols / (2 * blocks) >= 2048 && (long long)a.rows * blocks * 2 <= 4 * sms) blocks *= 2;
    while (blocks < kMostBlocks && a.cols / (2 * blocks) >= 16384) blocks *= 2;
    // A row has a vector more at most than its elements fill.
    const int vectors = (a.cols + Logit<kType>::kMany - 1) / Logit<kType>::kMany + 1, parts = blocks * kWarps;
    constexpr int kPiece = 32 * (kCellAdds / Logit<kType>::kMany);
    a.pieces = ((vectors + parts - 1) / parts + kPiece - 1) / kPiece;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.rows * blocks));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
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

bool misaligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

std::atomic<int> g_sums{0};

}  // namespace

bool set_sample_sums(int value) {
    if (value < 0 || value > 1) return false;
    g_sums.store(value, std::memory_order_relaxed);
    return true;
}

}  // namespace topk

extern "C" int topk_sample_rows(const void* logits, int dtype, int64_t stride, int rows, int cols,
                                const struct topk_sampling* sampling, const float* u, int32_t* token, float* logp,
                                struct CUstream_st* stream) {
    using namespace topk;
    if (!logits || !sampling || !u || !token || !logp || rows < 1 || cols < 1 || stride < cols)
        return TOPK_ERR_INVALID_ARG;
    if (dtype != TOPK_KV_F16 && dtype != TOPK_KV_BF16 && dtype != TOPK_SAMPLE_F32) return TOPK_ERR_INVALID_ARG;
    const int bytes = dtype == TOPK_SAMPLE_F32 ? 4 : 2;
    const topk_sampling& p = *sampling;
    if (misaligned(logits, bytes) || misaligned(u, 4) || misaligned(token, 4) || misaligned(logp, 4) ||
        misaligned(p.temperatures, 4) || misaligned(p.top_ks, 4) || misaligned(p.top_ps, 4) || misaligned(p.min_ps, 4))
        return TOPK_ERR_INVALID_ARG;
    if ((!p.temperatures && !(p.temperature >= 0)) || (!p.top_ps && p.top_p != p.top_p) ||
        (!p.min_ps && p.min_p != p.min_p))
        return TOPK_ERR_INVALID_ARG;
    if (cols > kMaxCols || rows > (1 << 24) || stride > (int64_t(1) << 38)) return TOPK_ERR_UNSUPPORTED;
    for (const void* q : {logits, (const void*)u, (const void*)token, (const void*)logp, (const void*)p.temperatures,
                          (const void*)p.top_ks, (const void*)p.top_ps, (const void*)p.min_ps}) {
        if (!q) continue;
        const int rc = device_pointer(q);
        if (rc != TOPK_OK) return rc;
    }
    int device = 0, sms = 0;
    cudaError_t e = current_device(&device, &sms);
    if (e == cudaSuccess) {
        SampleArgs a = {static_cast<const char*>(logits), (long long)stride * bytes, rows, cols, p,
                        p.min_p > 0 ? std::log(std::fmin((double)p.min_p, 1.0)) : 0.0, 0, u, token, logp,
                        g_sums.load(std::memory_order_relaxed)};
        cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
        e = dtype == TOPK_SAMPLE_F32 ? launch<kF32>(a, device, sms, s)
            : dtype == TOPK_KV_BF16  ? launch<kBf16>(a, device, sms, s)
                                     : launch<kF16>(a, device, sms, s);
        note_unreleased_launch(device, s);
    }
    if (e != cudaSuccess) {
        note_cuda_error((int)e);
        return TOPK_ERR_CUDA;
    }
    note_launch();
    return TOPK_OK;
}
