// topk_sample_rows: a token from each row of logits, with temperature, top-k,
// top-p and min-p, by one given uniform number.
//
// With the row in TopK order (value descending, the lower column first among
// equals), weights w_i = 2^(c x_i), c = log2(e) / temperature, and C(i) the
// weights up to and with i, every rule keeps a prefix of the order, and the
// token is where C passes u times the kept weight.  So all that is ever asked
// is where C (or the rank) passes a number, and how large C is there.
//
// One cluster of blocks has a row; its parts stay in L2 between the passes.
//   1. The row's largest value, and that of each thread's groups of vectors:
//      later passes read only the groups that can have what they look for.
//   2. Where few elements can be meant (top_k up to 512, min_p, temperature 0),
//      they are collected at once: for top_k, those that are not below a number
//      that at least k groups' largest values reach.
//   3. Else, or where those were too many: the weights of each octave (factor of
//      two), 64 of them.  A weight is a 24-bit number times 2^octave, so octaves
//      are sums of integers: exact, in any order.  A block adds up in cells of
//      shared memory, two atomic additions an element (4.4 cycles of an SM for
//      32 elements; cells of each thread's own cost 3.5, but their 64 KB left
//      two blocks to an SM).
//   4. The octave that is asked for is cut into 64 parts, and the part again,
//      until what is left fits a list (or is one value, whose elements are
//      equal).
//   5. The list, of at most 512 elements, is sorted and summed up with weights
//      of 42 bits, right to 2^-36, and gives the answer.
//
// A sum of fast weights is off by 2^-23.4 of itself at most.  A number that lies
// nearer to an element's border than that could put it is looked up once more
// with exact sums of 42-bit weights: one pass for what is above the list, and,
// should the number lie outside the list after all, 3 to 5 with 42 bits.
//
// What bounds it: the passes' latencies (a barrier of the cluster costs 1 to 2
// us, and there are 3 of them for top_k, 6 for top_p) and instructions, 20 an
// element for 3 and 4; HBM only where nothing but 1 is done.  Measured: one row
// of 131072 (bfloat16, top_k 50, top_p 0.95) 13 us; 256 of 160000 the same 36 us
// (2.2 TB/s), with an array of top_k 76 us, with temperature 0 50 us, with top_k
// 500 or 1000 alone 252 and 323 us; 64 of 131001 float32 with top_p 0.95 91 to
// 105 us (some rows need the exact pass); 128 of 32768, nothing cut off, 33 to
// 38 us; 512 of 262144 float32 with min_p 285 to 293 us (1.9 TB/s).
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
constexpr int kBlocksPerSm = 4;  // 64 registers a thread, and spills (64 rows with top_p: 96 us, 102 with three blocks)
constexpr int kBins = 64;
constexpr int kList = 512;          // elements that a list has room for (with 1024, 114 us instead of 93 for 64 rows with top_p)
constexpr int kMostBlocks = 8;      // of a cluster
constexpr int kBits = 41;           // a weight of 1 in its octave is 2^kBits
constexpr int kFastBits = 24;       // and a fast one 2^kFastBits
constexpr int kListShift = 11;      // in a list 2^(kBits + kListShift): kList of them stay below 2^63
constexpr int kMaxCols = 1 << 21;   // 2^21 weights of an octave, each below 2^(kBits + 0.5), stay below 2^63
constexpr int kGroup = 4;           // vectors of a thread's group, whose largest value is kept
constexpr int kMostFew = 512;       // top_k up to which a threshold is looked for first

struct SampleArgs {
    const char* logits;
    long long stride;  // bytes between rows
    int rows, cols;
    topk_sampling p;
    double log_min_p;  // of p.min_p
    int rounds;        // groups of a thread
    const float* u;
    int32_t* token;
    float* logp;
};

enum Type { kF16, kBf16, kF32 };

// NaN if one is.
__device__ __forceinline__ float larger_of(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

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
    // The same where i is not known to the compiler.
    static __device__ __forceinline__ float pick(const int4& v, int i) {
        const int k = kType == kF32 ? i : i >> 1;
        const unsigned w = (unsigned)(k < 2 ? k == 0 ? v.x : v.y : k == 2 ? v.z : v.w);
        if constexpr (kType == kF32) return __uint_as_float(w);
        else return widen((Word)(i & 1 ? w >> 16 : w));
    }
    // The largest of a vector's values and m's, as 32 bits of the type; NaN if there is one.
    static __device__ __forceinline__ unsigned largest(unsigned m, const int4& v) {
        const unsigned w[4] = {(unsigned)v.x, (unsigned)v.y, (unsigned)v.z, (unsigned)v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) m = larger(m, w[i]);
        return m;
    }
    static __device__ __forceinline__ unsigned larger(unsigned a, unsigned b) {
        if constexpr (kType == kF32) a = __float_as_uint(larger_of(__uint_as_float(a), __uint_as_float(b)));
        else if constexpr (kType == kBf16) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(a), "r"(b));
        else asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(a) : "r"(a), "r"(b));
        return a;
    }
    static constexpr unsigned kNothing = kType == kF32 ? kNone : kNone * 0x10001u;
    static __device__ __forceinline__ float single(unsigned m) {
        if constexpr (kType == kF32) return __uint_as_float(m);
        else return larger_of(widen((Word)m), widen((Word)(m >> 16)));
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
    float top, low;  // the largest value; the least of the threads' largest ones
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
    unsigned long long table[65];       // kPowers
    unsigned long long scan[kWarps];
    float warp_top[kWarps], warp_low[kWarps];
    float min_from, part_lo, part_hi;
};

// Where a block adds up weights: [2][kBins][32] cells, a column for each lane
// so that no two meet, a weight's upper bits in the first half and its lower
// ones in the second; and the largest values of the threads' groups behind
// them, [rounds][kThreads].
constexpr int kCells = kBins * 32;
__device__ __forceinline__ unsigned* cell_memory() {
    extern __shared__ __align__(16) unsigned memory[];
    return memory;
}

// 2^(i / 64 - 1/2), i from 0 to 64, times 2^kBits.
struct Powers {
    unsigned long long at[65];
    constexpr Powers() : at() {
        for (int i = 0; i < 65; ++i) {
            double term = 1, sum = 0;
            for (int n = 1; n < 30; ++n) {  // the series of e^((i / 64 - 1/2) ln 2)
                sum += term;
                term *= (i - 32) * (0.69314718055994530942 / 64) / n;
            }
            at[i] = (unsigned long long)(sum * (double)(1ull << kBits) + 0.5);
        }
    }
};
__constant__ const Powers kPowers;

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

enum What { kCount, kFast, kFineHigh, kFineLow };  // the last two: 28 upper and 14 lower bits of 42-bit weights
enum By { kOctaves, kLinear, kNumbers };

constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: what is added to it is rounded to a whole number

// 2^(c (x - ref)) in its octave with 42 bits: 2^f, -1/2 <= f <= 1/2, from a
// table and the series of e^a for the rest, with what is lost in a sum or
// product kept as a second number.
__device__ __forceinline__ unsigned long long fine_weight(float x, float ref, float c_hi, float c_lo,
                                                       const unsigned long long* table) {
    const float d = x - ref, n = fmaf(d, c_hi, kMagic) - kMagic;
    const float p = d * c_hi;
    const float f = p - n;
    const float f_lo = fmaf(d, c_hi, -p) + d * c_lo + (p - (f + n));
    const int i = min(max((int)fmaf(f, 64.f, 32.f), 0), 64);
    const float r = f - (i - 32) * 0.015625f;
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
    // Weights are 2^(c (x - ref)).  ref is 0 where c * top is small enough for
    // that, else the largest value: what differs from it by so much that the
    // difference is not exact has no weight.
    float ref, c_hi, c_lo, low;  // low: what lies below it has no weight
    int octave0;                 // bits of kMagic plus the octave of the largest value
    bool fine;
    int rounds;             // groups of a thread
    float* groups;          // their largest values, [rounds][kThreads]

    int whole0, whole1;  // the warp's vectors that lie in the row whole; one before them and one behind may not

    __device__ __forceinline__ static int4 nothing() {
        return make_int4((int)L::kNothing, (int)L::kNothing, (int)L::kNothing, (int)L::kNothing);
    }
    // One of the warp's vectors; what is not the row's is -inf.
    __device__ __forceinline__ int4 load(int v) const {
        if (v >= whole0 && v < whole1) return __ldg(reinterpret_cast<const int4*>(base) + v);
        union { int4 v; typename L::Word w[L::kMany]; } r;
        const int at = v * L::kMany;
        for (int i = 0; i < L::kMany; ++i)
            r.w[i] = at + i >= skip && at + i < end ? __ldg(reinterpret_cast<const typename L::Word*>(base) + at + i) : L::kNone;
        return r.v;
    }
    // A group's vectors, v and each 32nd after it; all loads are under way before any is waited for.
    __device__ __forceinline__ void load_group(int v, bool on, int4 (&raw)[kGroup]) const {
#pragma unroll
        for (int u = 0; u < kGroup; ++u) {
            raw[u] = nothing();
            if (on && v + 32 * u >= whole0 && v + 32 * u < whole1) raw[u] = __ldg(reinterpret_cast<const int4*>(base) + v + 32 * u);
        }
        if (v0 == whole0 && v1 == whole1) return;
        if (on && v == v0 && v < whole0) raw[0] = load(v);
        const int last = v1 - 1;
        if (on && last >= whole1 && last >= v && last < v + 32 * kGroup && ((last - v) & 31) == 0) {
            const int4 x = load(last);
#pragma unroll
            for (int u = 0; u < kGroup; ++u)
                if (v + 32 * u == last) raw[u] = x;
        }
    }
    // f(vector, its number) for the thread's vectors in rounds [from, to) whose
    // group has a value from `least` on; what is past the row's end is -inf.
    template <typename F>
    __device__ __forceinline__ void each_vector(int from, int to, float least, F f) const {
        const int lane = threadIdx.x & 31;
        for (int i = from; i < to; ++i) {
            const bool on = groups[i * kThreads + threadIdx.x] >= least;
            if (!__any_sync(kFullMask, on)) continue;
            const int v = v0 + i * (32 * kGroup) + lane;
            int4 raw[kGroup];
            load_group(v, on, raw);
            if (!on) continue;
#pragma unroll
            for (int u = 0; u < kGroup; ++u) f(raw[u], v + 32 * u);
        }
    }
    // The groups' largest values, and the thread's.
    __device__ __forceinline__ float look_through() const {
        const int lane = threadIdx.x & 31;
        float all = -INFINITY;
        int4 next[kGroup];
        load_group(v0 + lane, true, next);
        for (int i = 0; i < rounds; ++i) {
            int4 raw[kGroup];
#pragma unroll
            for (int u = 0; u < kGroup; ++u) raw[u] = next[u];
            if (i + 1 < rounds) load_group(v0 + (i + 1) * (32 * kGroup) + lane, true, next);
            unsigned m = L::kNothing;
#pragma unroll
            for (int u = 0; u < kGroup; ++u) m = L::largest(m, raw[u]);
            const float x = L::single(m);
            groups[i * kThreads + threadIdx.x] = x;
            all = larger_of(all, x);
        }
        return all;
    }

    // kMagic plus the whole number nearest to x's exponent.
    __device__ __forceinline__ float magic(float x) const { return fmaf(x - ref, c_hi, kMagic); }
    __device__ __forceinline__ int octave(float x) const { return octave0 - __float_as_int(magic(x)); }

    // The weight of x in its octave, 2^(kFastBits - 1/2) to 2^(kFastBits + 1/2):
    // 1 + f q(f) with q interpolating (2^f - 1) / f at Chebyshev's points, off
    // by 2^-27.5 of it; roundings make that 2^-23.6.  (The special function unit
    // gives 2^-22.)
    __device__ __forceinline__ unsigned fast(float x, float t) const {
        const float d = x - ref, f = fmaf(d, c_lo, fmaf(d, c_hi, kMagic - t));
        constexpr float kOne = 1 << kFastBits;
        float q = 0.00015453163f * kOne;
        q = fmaf(q, f, 0.0013390863f * kOne);
        q = fmaf(q, f, 0.0096180826f * kOne);
        q = fmaf(q, f, 0.0555035711f * kOne);
        q = fmaf(q, f, 0.2402265076f * kOne);
        q = fmaf(q, f, 0.6931471880f * kOne);
        return __float2uint_rn(fmaf(q, f, kOne));
    }
    // The same with 42 bits, 2^(kBits - 1/2) to 2^(kBits + 1/2).
    __device__ __forceinline__ Sum slow(float x, const unsigned long long* table) const {
        return fine_weight(x, ref, c_hi, c_lo, table);
    }
    __device__ __forceinline__ Sum weight(float x, const unsigned long long* table) const {
        return fine ? slow(x, table) : (Sum)fast(x, magic(x)) << (kBits - kFastBits);
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

// A region: the elements from `lo` to `hi`, and how they are cut into 64 bins,
// the largest values first.
struct Region {
    float lo, hi;
    By by;
    float scale;      // kLinear
    unsigned number;  // kNumbers: hi's
    int shift;
};

// A prefix of the order: what is above `value`, and the first `ties` that equal it.
struct Prefix {
    float value;
    int ties;
    Sum sum;     // of its weights
    bool exact;  // whether of 42-bit ones
};

// An element of the order: the weights before it and up to and with it, and
// where it is: at `index` in the list, or the `index`-th that equals `value`.
struct Place {
    Sum before, through;
    int index;
    bool in_list;
    float value;
};

template <Type kType>
struct Sampler {
    using L = Logit<kType>;
    Row<kType> row;
    Shared& s;
    int blocks, rank, turn = 0;
    // The list, or, where there are too many equal elements, those: what is above them.
    int listed = 0;       // elements in the list
    Sum base = 0;         // weights above the octave in which it begins, or above itself
    int list_octave = 0;  // that octave
    Sum list_from = 0;    // weights in that octave above it
    float list_top = 0;   // no element in between is above this one
    bool exact = false;   // whether what is above it is known to 42 bits
    int equal = 0;        // the number of equal elements

    __device__ Sampler(Shared& s) : s(s) {}

    __device__ __forceinline__ Exchange& mine() { return s.exchange[turn]; }
    __device__ __forceinline__ const Exchange* theirs(int r) {
        return blocks == 1 ? &s.exchange[turn] : cg::this_cluster().map_shared_rank(&s.exchange[turn], r);
    }
    __device__ __forceinline__ Region everything() const { return {row.low, row.top, kOctaves, 0.f, 0u, 0}; }

    __device__ __forceinline__ int bin(const Region& g, float x) const {
        if (g.by == kOctaves) return row.octave(x);
        if (g.by == kLinear) return kBins - 1 - min(kBins - 1, (int)((x - g.lo) * g.scale));
        return (int)((g.number - L::number(x + 0.f)) >> g.shift);
    }

    // Adds up `what` of the region's elements by bins over the cluster, into
    // s.bins.  kWay: fast weights by octaves, where every element up to the
    // top counts; fast weights in kLinear bins; or as `what` and the region
    // say, which is rare.
    enum Way { kByOctaves, kByLinear, kAnyhow };
    template <Way kWay>
    __device__ void add_up(const Region& g, What what) {
        const int tid = threadIdx.x, lane = tid & 31;
        unsigned *high = cell_memory() + lane, *low = high + kCells;
        // A cell has 2^21 / 8 / 32 numbers at most, below 2^14.
        const int split = what == kFast ? kFastBits / 2 : 14;
        row.each_vector(0, row.rounds, g.lo, [&](const int4& v, int) {
            if constexpr (kWay != kAnyhow) {
#pragma unroll
                for (int i = 0; i < L::kMany; ++i) {
                    const float x = L::at(v, i);
                    if (x >= g.lo && (kWay == kByOctaves || x <= g.hi)) {
                        const float t = row.magic(x);
                        const unsigned w = row.fast(x, t);
                        const int b = kWay == kByOctaves
                                          ? row.octave0 - __float_as_int(t)
                                          : kBins - 1 - min(kBins - 1, (int)((x - g.lo) * g.scale));
                        const unsigned at = min((unsigned)b, kBins - 1u) * 32;
                        atomicAdd(high + at, w >> (kFastBits / 2));
                        atomicAdd(low + at, w & ((1u << (kFastBits / 2)) - 1));
                    }
                }
            } else if (L::single(L::largest(L::kNothing, v)) >= g.lo) {
#pragma unroll 1
                for (int i = 0; i < L::kMany; ++i) {
                    const float x = L::pick(v, i);
                    if (!(x >= g.lo && x <= g.hi)) continue;
                    unsigned w = 1;
                    if (what == kFast) w = row.fast(x, row.magic(x));
                    if (what == kFineHigh || what == kFineLow) {
                        const Sum m = row.slow(x, s.table);
                        w = what == kFineHigh ? (unsigned)(m >> 14) : (unsigned)m & 0x3FFFu;
                    }
                    const unsigned at = min((unsigned)bin(g, x), kBins - 1u) * 32;
                    atomicAdd(high + at, w >> split);
                    atomicAdd(low + at, w & ((1u << split) - 1));
                }
            }
        });
        __syncthreads();
        // A bin's 32 columns by kEach threads, which leave zeros behind.
        constexpr int kEach = kThreads / kBins, kVectors = 32 / kEach / 4;
        Sum sum = 0;
        uint4* mine4 = reinterpret_cast<uint4*>(cell_memory()) + tid * kVectors;
#pragma unroll
        for (int i = 0; i < kVectors; ++i) {
            const uint4 h = mine4[i], l = mine4[i + kCells / 4], zero = {0, 0, 0, 0};
            sum += (((Sum)h.x + h.y + h.z + h.w) << split) + ((Sum)l.x + l.y + l.z + l.w);
            mine4[i] = mine4[i + kCells / 4] = zero;
        }
#pragma unroll
        for (int d = 1; d < kEach; d <<= 1) sum += __shfl_xor_sync(kFullMask, sum, d);
        if (tid % kEach == 0) mine().bins[tid / kEach] = sum;
        join_bins(what == kFineLow, what == kFast ? kBits - kFastBits : what == kFineHigh ? 14 : 0);
    }
    // The blocks' bins -> s.bins, and what is above each.  add: to what is there.
    __device__ void join_bins(bool add, int shift) {
        const int tid = threadIdx.x;
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
            b0 = (add ? s.bins[2 * tid] : 0) + (b0 << shift);
            b1 = (add ? s.bins[2 * tid + 1] : 0) + (b1 << shift);
            s.bins[2 * tid] = b0;
            s.bins[2 * tid + 1] = b1;
            write_scan(s.above, b0, b1);
        }
        turn ^= 1;
        __syncthreads();
    }
    __device__ void add_up_weights(const Region& g) {
        if (row.fine) {
            add_up<kAnyhow>(g, kFineHigh);
            add_up<kAnyhow>(g, kFineLow);
        } else if (g.by == kOctaves) {
            add_up<kByOctaves>(g, kFast);
        } else if (g.by == kLinear) {
            add_up<kByLinear>(g, kFast);
        } else {
            add_up<kAnyhow>(g, kFast);
        }
    }
    // The sum of the numbers of this lane and those before it.
    static __device__ __forceinline__ Sum through(Sum x) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const Sum y = __shfl_up_sync(kFullMask, x, d);
            if (lane >= d) x += y;
        }
        return x;
    }
    // Sums of the bins before each: two of a lane's, by one warp.
    static __device__ void write_scan(Sum* to, Sum b0, Sum b1) {
        const int lane = threadIdx.x & 31;
        const Sum x = through(b0 + b1);
        to[2 * lane] = x - b0 - b1;
        to[2 * lane + 1] = x - b1;
        if (lane == 31) to[kBins] = x;
    }
    // What an octave's sum, in its own unit, has below a whole unit of octave 0,
    // in 2^-56 units: 64 of them leave room for the carries.  Without them all
    // octaves together could be off by 2^-35 of the row.
    static __device__ __forceinline__ Sum below(Sum b, int o) { return (b << (63 - o) << 1) >> 8; }
    // The first bin up to and with which the sums are more than t (strict) or
    // not less; the last one that has anything if t is past them all.
    static __device__ int bin_of(const Sum* sums, Sum t, bool strict) {
        const int i = threadIdx.x;
        const Sum next = i < kBins ? sums[i + 1] : 0, all = sums[kBins];
        const int at = __syncthreads_count(i < kBins && (strict ? next <= t : next < t));
        return min(at, __syncthreads_count(i < kBins && next < all));
    }

    // The smallest number k in [lo, hi] for which f(value of k), which is true
    // from some value on and for hi, is true.  By one warp.
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
    // Bins b0 to b1 of a region.  One warp looks for the borders: the others'
    // instructions are better spent on other rows.
    __device__ Region part(const Region& g, int b0, int b1) {
        if (threadIdx.x < 32) {
            const unsigned klo = L::number(g.lo), khi = L::number(g.hi);
            auto upto = [&](int b) {
                return first(klo, khi, [&](float x) { return x >= g.lo && bin(g, x) <= b; });
            };
            const float lo = L::value(upto(b1)), hi = b0 > 0 ? L::value(upto(b0 - 1) - 1) : g.hi;
            if (threadIdx.x == 0) {
                s.part_lo = lo;
                s.part_hi = hi;
            }
        }
        __syncthreads();
        Region r = g;
        r.lo = s.part_lo;
        r.hi = s.part_hi;
        __syncthreads();
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

    // Collects the elements from lo to hi, which begin in `octave` below
    // in_octave weights of it, and sorts and sums them up.  False, and no
    // list, if they are more than fit.
    __device__ bool gather(float lo, float hi, int octave, Sum in_octave) {
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
        if (tid == 0) mine().count = 0;
        __syncthreads();
        row.each_vector(0, row.rounds, lo, [&](const int4& v, int at) {
            unsigned in = 0;
#pragma unroll
            for (int i = 0; i < L::kMany; ++i) in |= L::at(v, i) >= lo && L::at(v, i) <= hi ? 1u << i : 0u;
            for (; in; in &= in - 1) {
                const int i = __ffs(in) - 1;
                const float x = L::pick(v, i);
                const int n = atomicAdd(&mine().count, 1);
                const unsigned b = __float_as_uint(x + 0.f), key = b ^ ((unsigned)((int)b >> 31) | 0x80000000u);
                if (n < kList)
                    mine().list[n] = (unsigned long long)key << 32 | ~(unsigned)(at * L::kMany + i - row.skip);
            }
        });
        cluster_sync(blocks);
        int counts[kMostBlocks], n = 0;
#pragma unroll
        for (int r = 0; r < kMostBlocks; ++r) counts[r] = r < blocks ? theirs(r)->count : 0;
#pragma unroll
        for (int r = 0; r < kMostBlocks; ++r) n += counts[r];
        const bool fits = n <= kList;
        if (fits) {
            n = 0;
#pragma unroll
            for (int r = 0; r < kMostBlocks; ++r) {
                if (counts[r] == 0) continue;
                const Exchange* e = theirs(r);
                for (int i = tid; i < counts[r]; i += kThreads) s.list[n + i] = e->list[i];
                n += counts[r];
            }
        }
        turn ^= 1;
        listed = equal = 0;
        if (!fits || n == 0) {
            __syncthreads();
            return false;
        }
        sort_list(n);
        constexpr int kPer = kList / kThreads;
        Sum own[kPer], sum = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int at = tid * kPer + i;
            if (at < n) {
                const float x = listed_value(at);
                sum += row.slow(x, s.table) << kListShift >> (row.octave(x) - octave);
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
        list_top = hi;
        exact = hi == row.top;
        base = exact ? 0 : s.before[octave];
        return true;
    }
    // Sorts s.list[0..n), descending; no two are equal.  A warp sorts 32 of
    // them by shuffles, and a number's place is the sum of its places in all
    // sorted pieces: three barriers instead of one for each step of a network.
    __device__ void sort_list(int n) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, pieces = (n + 31) / 32;
        constexpr int kPer = kList / kThreads;
        unsigned long long key[kPer];
        int rank[kPer];
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int piece = warp + j * kWarps, at = piece * 32 + lane;
            unsigned long long v[1] = {at < n ? s.list[at] : 0ull};  // no number is 0
            if (piece < pieces) {
                warp_sort_desc(v, lane);
                s.list[at] = v[0];
            }
            key[j] = v[0];
            rank[j] = lane;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int piece = warp + j * kWarps;
            if (piece >= pieces) continue;
            for (int p = 0; p < pieces; ++p) {
                if (p == piece) continue;
                const unsigned long long* other = s.list + p * 32;
                int above = 0;
#pragma unroll
                for (int d = 16; d > 0; d >>= 1)
                    if (other[above + d - 1] > key[j]) above += d;
                rank[j] += above + (other[above] > key[j]);
            }
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (key[j] != 0) s.list[rank[j]] = key[j];
        __syncthreads();
    }
    __device__ __forceinline__ float listed_value(int i) const {
        const unsigned k = (unsigned)(s.list[i] >> 32);
        return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
    }
    // Weights up to and with element i - 1 of the list.
    __device__ __forceinline__ Sum list_sum(int i) const {
        return base + ((list_from + (i > 0 ? s.through[i - 1] >> kListShift : 0)) >> list_octave);
    }
    // Whether the first element up to and with which the weights are more than
    // t (strict) or not less is in the list, or one of the equal elements.
    __device__ __forceinline__ bool holds(Sum t, bool strict) const {
        if (listed) {
            const Sum to = list_sum(listed);
            return t >= list_sum(0) && (strict ? t < to : t <= to) && (strict || t > list_sum(0) || exact);
        }
        return equal > 0;
    }
    __device__ Place place(Sum t, bool strict) {
        const Sum rel = t > base ? (t - base) << list_octave : 0, in = rel > list_from ? rel - list_from : 0;
        if (listed) {
            const Sum edge = in << kListShift;
            int count = 0;
            for (int i = threadIdx.x; i - (int)threadIdx.x < listed; i += kThreads)
                count += __syncthreads_count(i < listed && (strict ? s.through[i] <= edge : s.through[i] < edge));
            const int i = min(count, listed - 1);
            return {list_sum(i), list_sum(i + 1), i, true, listed_value(i)};
        }
        const Sum w = exact ? row.slow(list_top, s.table) : row.weight(list_top, s.table);
        const Sum i = min(strict ? in / w : (in > 0 ? in - 1 : 0) / w, (Sum)max(equal - 1, 0));
        return {base + ((list_from + i * w) >> list_octave), base + ((list_from + (i + 1) * w) >> list_octave), (int)i, false,
                list_top};
    }
    // The prefix up to and with a place.
    __device__ Prefix prefix_to(const Place& p) {
        int ties = p.index + 1;
        if (p.in_list) {
            ties = 0;
            for (int i = threadIdx.x; i - (int)threadIdx.x <= p.index; i += kThreads)
                ties += __syncthreads_count(i <= p.index && listed_value(i) == p.value);
        }
        return {p.value, ties, p.through, exact};
    }

    // Weights lie between 2^(kBits - 1/2) and 2^(kBits + 1/2): how many of them
    // there are at most, and at least, with room for roundings.
    __device__ __forceinline__ static int most(Sum sum) {
        return (int)((float)sum * (1.0002f / 1554944255988.f)) + (sum > 0);
    }
    __device__ __forceinline__ static int least(Sum sum) {
        return max((int)((float)sum * (0.9998f / 3109888511976.f)), sum > 0 ? 1 : 0);
    }

    // Makes the list, or the run of equal elements, in which the first element
    // lies up to and with which the weights are more than t (strict) or not less.
    __device__ void look_for(Sum t, bool strict) {
        const int o = bin_of(s.before, t, strict);
        Region g = everything();
        if (s.upper[o] <= kList) {  // all down to there
            gather(part(g, 0, o).lo, row.top, 0, 0);
            return;
        }
        g = part(g, o, o);
        const Sum rel = t > s.before[o] ? (t - s.before[o]) << o : 0;
        narrow(g, o, s.octave[o], most(s.octave[o]), false, [&](Sum above) {
            return bin_of(s.above, rel > above ? rel - above : 0, strict);
        });
    }
    // Cuts a region of octave o, with `sum` of weights and at most `room`
    // elements, until it fits a list or is one value.  pick(weights above):
    // the bin to go on with; counted: the room is known by counting, and pick
    // finds the counts in s.bins.
    template <typename F>
    __device__ void narrow(Region g, int o, Sum sum, Sum room, bool counted, F pick) {
        Sum above = 0;
        for (int level = 0; room > kList && g.lo != g.hi; ++level) {
            cut(g, level);
            int b = 0;
            if (counted) {
                add_up<kAnyhow>(g, kCount);
                b = pick(above);
                room = s.bins[b];
            }
            add_up_weights(g);
            if (!counted) {
                b = pick(above);
                room = most(s.bins[b]);
            }
            above += s.above[b];
            sum = s.bins[b];
            g = part(g, b, b);
        }
        if (room <= kList) {
            gather(g.lo, g.hi, o, above);
            return;
        }
        const Sum w = row.weight(g.hi, s.table);
        listed = 0;
        equal = (int)min(sum / w, (Sum)kMaxCols);
        list_octave = o;
        list_from = above;
        list_top = g.hi;
        exact = row.fine;
        base = s.before[o];
    }

    // The first k elements of the order.
    __device__ Prefix first_k(int k) {
        const int reach = __syncthreads_count(threadIdx.x < kBins - 1 && s.lower[threadIdx.x] < k);  // no further than here
        if (s.upper[reach] <= kList) {
            gather(part(everything(), 0, reach).lo, row.top, 0, 0);
            return prefix_of(min(k, listed));
        }
        add_up<kAnyhow>(everything(), kCount);
        if (s.above[kBins] <= (Sum)k) return all();
        const int o = bin_of(s.above, k, false);
        Sum need = k - s.above[o], room = s.bins[o];
        narrow(part(everything(), o, o), o, s.octave[o], room, true, [&](Sum) {
            const int b = bin_of(s.above, need, false);
            need -= s.above[b];
            return b;
        });
        if (listed) return prefix_of((int)min(need, (Sum)listed));
        const Sum w = row.weight(list_top, s.table);
        return {list_top, (int)need, base + ((list_from + need * w) >> list_octave), row.fine};
    }
    __device__ Prefix prefix_of(int n) {  // of the list's first n
        return prefix_to({list_sum(n - 1), list_sum(n), n - 1, true, listed_value(n - 1)});
    }
    __device__ Prefix all() const { return {-INFINITY, 0, s.before[kBins], row.fine}; }

    // Weights of 42 bits of what is above x, and of a prefix.  What an entry has
    // below a whole unit of octave 0 is added up by itself, in 2^-32 units, and
    // carried once: rounded away entry by entry, equal ones would all be off by
    // the same amount (2^20 of them in octave 21 by 2^-22 of the whole row).
    __device__ void add_up_exactly(float x, Sum* above, Prefix* p) {
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
        auto below = [](Sum m, int o) { return (m << (63 - o) << 1) >> 32; };  // of m >> o
        Sum a = 0, a_below = 0, b = 0, b_below = 0;
        const float from = fmaxf(row.low, fminf(x, p->value));
        row.each_vector(0, row.rounds, from, [&](const int4& v, int) {
            if (!(L::single(L::largest(L::kNothing, v)) >= from)) return;
#pragma unroll 1
            for (int i = 0; i < L::kMany; ++i) {
                const float y = L::pick(v, i);
                if (!(y >= row.low && (y > x || y > p->value))) continue;
                const int o = row.octave(y);
                const Sum m = row.slow(y, s.table), w = m >> o, w_below = below(m, o);
                if (y > x) {
                    a += w;
                    a_below += w_below;
                }
                if (y > p->value) {
                    b += w;
                    b_below += w_below;
                }
            }
        });
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            a += __shfl_xor_sync(kFullMask, a, d);
            a_below += __shfl_xor_sync(kFullMask, a_below, d);
            b += __shfl_xor_sync(kFullMask, b, d);
            b_below += __shfl_xor_sync(kFullMask, b_below, d);
        }
        static_assert(4 * kWarps <= kBins);
        if (lane == 0) {
            Sum* q = mine().bins + 4 * warp;
            q[0] = a;
            q[1] = a_below;
            q[2] = b;
            q[3] = b_below;
        }
        cluster_sync(blocks);
        a = a_below = b = b_below = 0;
        for (int r = 0; r < blocks; ++r) {
            const Sum* q = theirs(r)->bins;
            for (int w = 0; w < kWarps; ++w) {
                a += q[4 * w];
                a_below += q[4 * w + 1];
                b += q[4 * w + 2];
                b_below += q[4 * w + 3];
            }
        }
        turn ^= 1;
        *above = a + (a_below >> 32);
        if (!p->exact && p->ties > 0) {
            const int o = row.octave(p->value);
            const Sum m = row.slow(p->value, s.table) * p->ties;
            b += m >> o;
            b_below += below(m, o);
        }
        if (!p->exact) p->sum = b + (b_below >> 32);
        p->exact = true;
    }

    // Where the weights pass `share` of a prefix: more than that (strict) or
    // not less.  False where weights of 24 bits do not tell, nor those of 42 of
    // what is above the elements that they led to.
    __device__ bool find(Prefix* p, float share, bool strict, Place* at) {
        Sum t = times(p->sum, share, !strict);
        if (!holds(t, strict) || !listed) look_for(t, strict);
        *at = place(t, strict);
        if (row.fine || (p->exact && exact) || !near_border(t, *at, *p)) return true;
        Sum above = 0;
        add_up_exactly(list_top, &above, p);
        if (!exact) {
            base = above;
            list_from = 0;
            exact = true;
        }
        t = times(p->sum, share, !strict);
        if (!inside(t, strict)) return false;
        *at = place(t, strict);
        return true;
    }
    // Whether t lies between what is above the list, or the equal elements, and what is above those behind it.
    __device__ __forceinline__ bool inside(Sum t, bool strict) const {
        Sum to;
        if (listed) to = list_sum(listed);
        else to = base + ((list_from + row.slow(list_top, s.table) * equal) >> list_octave);
        const Sum from = base + (list_from >> list_octave);
        return strict ? t >= from && t < to : (t > from || base == 0) && t <= to;
    }
    // Whether t is so near one of an element's borders that weights of 24 bits
    // do not tell on which side it lies.  With the sums b above the list, l in
    // it (which is exact) and z of the prefix, of weights off by a share e at
    // most, t / z lies off by e ((1 - t / z) b + t / z (z - b)) / z at most.
    // Where only one of b and z is made of such weights, by e b or e t.
    __device__ __forceinline__ bool near_border(Sum t, const Place& p, const Prefix& of) {
        const Sum all = of.sum, left = all > t ? all - t : 0, in = listed ? list_sum(listed) - list_sum(0) : 0;
        // e is 2^-23.4; with (1 - u) b and u (z - b - l) both below min(t, z - t):
        const Sum room = (of.exact == exact ? min(t, left) + in : t) >> 22;
        return (p.before > 0 && (t > p.before ? t - p.before : 0) < room) ||
               (p.through < all && (p.through > t ? p.through - t : 0) < room);
    }

    // The part of a prefix from `from` on.
    __device__ Prefix down_to(const Prefix& p, float from) {
        if (p.value >= from) return p;  // all of it
        // A number below `from`, and above every value below that.
        const Prefix q = {nextafterf(from, -INFINITY), 0, 0, row.fine};
        if (listed && base == 0 && exact && listed_value(listed - 1) < from) {
            int count = 0;
            for (int i = threadIdx.x; i - (int)threadIdx.x < listed; i += kThreads)
                count += __syncthreads_count(i < listed && listed_value(i) >= from);
            return {q.value, 0, list_sum(count), true};
        }
        Region g = everything();
        g.lo = fmaxf(from, row.low);
        add_up_weights(g);
        Sum all = 0, rest = 0;
        for (int i = 0; i < kBins; ++i) {
            all += s.bins[i] >> i;
            rest += below(s.bins[i], i);
        }
        __syncthreads();
        return {q.value, 0, all + (rest >> 56), row.fine};
    }

    // The sums of all octaves -> what is above each, and bounds on numbers.
    __device__ void octaves() {
        const int lane = threadIdx.x;
        if (lane < 32) {
            const Sum b0 = s.bins[2 * lane], b1 = s.bins[2 * lane + 1];
            s.octave[2 * lane] = b0;
            s.octave[2 * lane + 1] = b1;
            write_scan(s.before, b0 >> 2 * lane, b1 >> (2 * lane + 1));
            const Sum r0 = below(b0, 2 * lane), r1 = below(b1, 2 * lane + 1), r = through(r0 + r1);
            s.before[2 * lane] += (r - r0 - r1) >> 56;
            s.before[2 * lane + 1] += (r - r1) >> 56;
            if (lane == 31) s.before[kBins] += r >> 56;
            int upper = most(b0) + most(b1), lower = least(b0) + least(b1);  // 2^21 and a little at most
            const int upper1 = most(b1), lower1 = least(b1);
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

    // A number that at least k elements are not below, and not many more: by
    // the groups' largest values, in 64 bins between the least of the threads'
    // largest ones and the largest.  -inf if they do not tell.
    __device__ float threshold(int k, float least) {
        const int tid = threadIdx.x;
        const float scale = kBins / (row.top - least);
        if (!(scale > 0 && scale < FLT_MAX)) return -INFINITY;  // the same for the cluster
        if (tid < kBins) mine().bins[tid] = 0;
        __syncthreads();
        for (int i = 0; i < row.rounds; ++i) {
            const float x = row.groups[i * kThreads + tid];
            if (x >= least) {
                const int b = kBins - 1 - min(kBins - 1, (int)((x - least) * scale));
                atomicAdd(reinterpret_cast<unsigned*>(&mine().bins[b]), 1u);  // its lower half
            }
        }
        __syncthreads();
        join_bins(false, 0);
        if (s.above[kBins] < (Sum)k) return -INFINITY;
        const int b = bin_of(s.above, k, false);
        // A little below the bin's edge, for the roundings of both ways.
        return fmaf((float)(kBins - 1 - b), (row.top - least) * (1.f / kBins), least) -
               (fabsf(row.top) + fabsf(least)) * 0x1p-20f;
    }

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
        row.each_vector(0, row.rounds, x, [&](const int4& v, int) { count += __popc(matches(v)); });
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

template <Type kType>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) sample_rows_kernel(const __grid_constant__ SampleArgs a) {
    using L = Logit<kType>;
    __shared__ Shared s;
    cg::cluster_group cluster = cg::this_cluster();
    const int blocks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int r = blockIdx.x / blocks, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    grid_dependency_wait();  // launched early (launch_pdl): the previous kernel's writes first

    Sampler<kType> sampler(s);
    Row<kType>& row = sampler.row;
    sampler.blocks = blocks;
    sampler.rank = rank;
    const char* start = a.logits + r * a.stride;
    row.skip = (int)((reinterpret_cast<uintptr_t>(start) & 15) / L::kBytes);
    row.base = start - row.skip * L::kBytes;
    row.end = row.skip + a.cols;
    row.rounds = a.rounds;
    row.groups = reinterpret_cast<float*>(cell_memory() + 2 * kCells);
    for (int i = tid; i < kCells / 2; i += kThreads) reinterpret_cast<uint4*>(cell_memory())[i] = {0, 0, 0, 0};
    const int vectors = (row.end + L::kMany - 1) / L::kMany;
    // Contiguous shares: of a block, and of each of its warps.
    const int parts = blocks * kWarps, share = (vectors + parts - 1) / parts;
    row.v0 = min((rank * kWarps + warp) * share, vectors);
    row.v1 = min(row.v0 + share, vectors);
    row.whole0 = max(row.v0, row.skip > 0 ? 1 : 0);
    row.whole1 = max(min(row.v1, row.end / L::kMany), row.whole0);
    if (tid < 65) s.table[tid] = kPowers.at[tid];

    // The largest value, NaN if there is one; and the least of the threads' largest.
    float top = row.look_through(), low = top > -INFINITY ? top : INFINITY;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        top = larger_of(top, __shfl_xor_sync(kFullMask, top, d));
        low = fminf(low, __shfl_xor_sync(kFullMask, low, d));
    }
    if (lane == 0) {
        s.warp_top[warp] = top;
        s.warp_low[warp] = low;
    }
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < kWarps; ++w) {
            top = larger_of(top, s.warp_top[w]);
            low = fminf(low, s.warp_low[w]);
        }
        s.exchange[0].top = top;
        s.exchange[0].low = low;
    }
    cluster_sync(blocks);
    for (int b = 0; b < blocks; ++b) {
        const float y = sampler.theirs(b)->top, z = sampler.theirs(b)->low;
        top = b == 0 ? y : larger_of(top, y);
        low = b == 0 ? z : fminf(low, z);
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
    row.ref = fabsf(top) * row.c_hi >= 128.f ? top : 0.f;
    row.octave0 = __float_as_int(row.magic(top));
    row.fine = false;
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

    Place at = {};
    Prefix kept = {};
    // Where few elements can be meant, they are collected at once.
    float from = greedy ? top : cut_m && !cut_p ? min_from : -INFINITY;
    if (cut_k && top_k <= kMostFew) from = fmaxf(from, sampler.threshold(top_k, low));
    bool found = from > -INFINITY && sampler.gather(fmaxf(from, row.low), top, 0, 0);
    if (found) {
        kept = sampler.prefix_of(cut_k ? min(top_k, sampler.listed) : sampler.listed);
        if (cut_p) {
            found = sampler.find(&kept, fmaxf(top_p, 0.f), false, &at);
            kept = sampler.prefix_to(at);
            if (cut_m) kept = sampler.down_to(kept, min_from);
        }
        found = sampler.find(&kept, u, true, &at);
    }
    for (int pass = 0; pass < 2 && !found; ++pass) {
        row.fine = pass == 1;
        sampler.listed = sampler.equal = 0;
        sampler.add_up_weights(sampler.everything());
        sampler.octaves();
        kept = cut_k ? sampler.first_k(top_k) : sampler.all();
        if (cut_p) {
            if (!sampler.find(&kept, fmaxf(top_p, 0.f), false, &at)) continue;
            kept = sampler.prefix_to(at);
            if (cut_m) kept = sampler.down_to(kept, min_from);
        }
        found = sampler.find(&kept, u, true, &at);
    }
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
        const Sum w = at.through - at.before, rest = kept.sum > w ? kept.sum - w : 0;
        // log(w / kept): near 1 by what the others have, else from the value
        // itself, which is exact.
        float logp;
        if (greedy || rest == 0) {
            logp = 0.f;
        } else if (w > rest) {
            logp = log1pf(-((float)rest / (float)kept.sum));
        } else {
            const double c = (double)row.c_hi + row.c_lo;
            const int octave0 = row.octave0 - __float_as_int(kMagic);
            const int up = __clzll((long long)kept.sum);  // the logarithm of a number from 1 to 2, and the rest exactly
            const float part = log2f((float)(kept.sum << up) * 0x1p-63f);
            logp = (float)((((double)at.value - row.ref) * c - octave0 + kBits - (63 - up) - (double)part) *
                           0.69314718055994530942);
        }
        a.token[r] = column;
        a.logp[r] = logp;
    }
    cluster_sync(blocks);  // no block leaves while another reads its shared memory
}

template <Type kType>
cudaError_t launch(SampleArgs& a, int device, int sms, cudaStream_t s) {
    auto kernel = sample_rows_kernel<kType>;
    // Blocks of a row: 8192 elements each at least, and as many as fill the
    // SMs four times over, or once where few elements are looked at again, and
    // blocks do little but read (256 rows of 160000 with top_k 50: 36 us, 76
    // with more; 512 of 262144 with min_p: 291 us, 470 with fewer).  Of an array
    // of top_k nothing is known here.  Four blocks fit an SM as long as a row's
    // blocks have 19 rounds at most (20.2 + 16 KB, and one for each round); 33
    // rounds, as of 131072 float32 in one block, leave room for three.
    const bool light = !a.p.top_ks && a.p.top_k > 0 && a.p.top_k <= kMostFew;
    int blocks = 1;
    while (blocks < kMostBlocks && a.cols / (2 * blocks) >= 8192 &&
           (long long)a.rows * blocks * 2 <= (long long)(light ? 1 : 4) * kBlocksPerSm * sms)
        blocks *= 2;
    while (blocks < kMostBlocks && (long long)kMostBlocks * a.cols > (long long)blocks * kMaxCols) blocks *= 2;
    // A row has a vector more at most than its elements fill.
    const int vectors = (a.cols + Logit<kType>::kMany - 1) / Logit<kType>::kMany + 1, parts = blocks * kWarps;
    a.rounds = ((vectors + parts - 1) / parts + 32 * kGroup - 1) / (32 * kGroup);
    // The most that kMaxCols take: 65 rounds of float32, 33 of 16 bits.
    constexpr int kMostRounds = ((kMaxCols / Logit<kType>::kMany + 1) / (kMostBlocks * kWarps) + 32 * kGroup) / (32 * kGroup);
    const int smem = (2 * kCells + a.rounds * kThreads) * 4;
    static std::atomic<unsigned long long> allowed{0};
    const cudaError_t e = allow_smem(kernel, (2 * kCells + kMostRounds * kThreads) * 4, device, allowed);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.rows * blocks));
    cfg.blockDim = dim3(kThreads);
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

bool misaligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

}  // namespace
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
                        p.min_p > 0 ? std::log(std::fmin((double)p.min_p, 1.0)) : 0.0, 0, u, token, logp};
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
