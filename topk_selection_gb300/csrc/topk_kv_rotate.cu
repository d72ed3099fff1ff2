// topk_kv_rotate, topk_kv_append_rotated: the norm of each head of queries and
// keys and the rotation by their positions, in one pass over them; the second
// writes keys and values into their pages.
//
//     y = x * rsqrt(mean(x^2) + eps) * w      (where there is a norm)
//     (y_a, y_b) -> (y_a cos t - y_b sin t, y_b cos t + y_a sin t)
//
// for each pair p of elements (a, b), t = position * freq[p]; elements that no
// pair has stay as they are.  float32 throughout, rounded once at the end.
//
// Bound by HBM for prompts: every element is read and written once.  One wave
// of blocks, whose warps take a token's heads at a time, or some of them.  A
// lane has the same eight pairs of each head, both vectors of them, so that
// nothing is exchanged for the rotation; a norm costs the shuffles of one sum.
// A token's angles are worked out once, shared out over the warp.  Vectors come
// by asynchronous copies through a ring in shared memory, two steps ahead: what
// is on its way needs no registers (in registers it took 117 of them, two
// blocks an SM, and 138 us where it is 122 now).  Half of the time is issued
// instructions, so two numbers are multiplied by one where that can be.
//
// Measured: 20011 tokens of 64 + 8 heads, dim 128 (738 MB) 122 us, 6.0 TB/s,
// 89% of a copy's rate; appended prompts, 40942 tokens of 32 + 8 + 8 heads
// (1.0 GB), 162 us, 6.2 TB/s, 92%; one token each of 64 sequences 3.9 and 5.0
// us a call, which is the host's.
//
// Heads whose pairs do not fill vectors (halves of which half the turned
// elements are no multiple of 8, or a dim that is none of 16) go through single
// elements, two bytes a lane and nothing ahead, values too: 4093 tokens of 16 +
// 16 heads of 80 of which 40 elements are turned take 39 us as halves, 11 as
// neighbours; 10240 tokens' keys and values of the same heads, appended, 205
// and 27 us.
//
// Angles.  A product of 32 bits knows a position of 10^6 times a frequency
// near 1 to 0.06 radians only.  Here a frequency becomes a whole number of
// 2^-64 turns per position, so that the product with the position, whole turns
// dropped, is the low half of one multiplication of integers: good to 2^-32
// turns, and (1 + freq / 2) 2^-64 of a turn for each position, and no reduction
// follows but to the nearest quarter.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>

#include "../../include/topk.h"
#include "topk_device.cuh"
#include "topk_kv.cuh"

namespace topk {
namespace {

constexpr int kRotateThreads = 256, kWarps = kRotateThreads / 32;
constexpr int kUnroll = 2;  // heads of a step that a lane has
constexpr int kDepth = 3;   // steps of a warp in its ring, all but one of them on the way
// Blocks of an SM.  Without a cache the instructions want more warps (20011
// tokens of 64 + 8 heads: 122 us with three, 127 with two); with one the pages'
// writes are better off with fewer (16 prompts, 40942 tokens of 32 + 8 + 8
// heads: 162 us with two, 185 with three).
constexpr int kBlocks = 3, kBlocksCache = 2;
// Steps of a unit at most without a cache, so that the warps finish together
// (122 us with 3 or 4, 129 with all nine of a token).
constexpr int kSteps = 3;

enum Kind { kQueries, kKeys, kValues };

struct RotateArgs {
    KvCache c;  // of an append
    KvRotate r;
    // By kind, where their tensors lie: strides of tokens and heads in vectors
    // of 8 elements, so that 32 bits do.
    const uint16_t* in[3];
    unsigned in_token[3], in_head[3];
    uint16_t* out[2];  // of keys only where there is no cache
    unsigned out_token[2], out_head[2];
    const uint16_t* norm[2];
    unsigned norm_head[2];
    int heads[3];
    int lanes;     // that a head takes
    int steps[3];  // of queries, keys and, in an append, values, added up: a step is the heads that a warp has in flight
    int chunk;     // steps of a unit: a token and some of its heads
    int chunks;    // units of a token
    int units;     // of all tokens
    int tokens_on, parts_on;  // from a warp's unit to its next: so many tokens, and units of a token, on
};

// A frequency as a whole number of 2^-64 turns per position.
__device__ __forceinline__ unsigned long long turns_of(float freq) {
    const unsigned bits = __float_as_uint(freq);
    const int exponent = (bits >> 23) & 255, down = 150 - exponent;
    // freq = mantissa * 2^-down; 2^64 / (2 pi), whole.
    const unsigned long long mantissa = exponent ? (bits & 0x7FFFFFu) | 0x800000u : 0u;
    constexpr unsigned long long kPerRadian = 0x28BE60DB9391054Aull;
    const unsigned long long low = mantissa * kPerRadian, high = __umul64hi(mantissa, kPerRadian);
    unsigned long long per;
    if (down >= 64) per = down < 96 ? high >> (down - 64) : 0;
    else if (down > 0) per = (high << (64 - down)) | (low >> down);
    else per = low << (-down & 63);
    return bits >> 31 ? 0 - per : per;
}

// cos and sin at a position.
__device__ __forceinline__ void turn(unsigned long long per, int pos, float* c, float* s) {
    const int at = (int)((per * (unsigned long long)(long long)pos) >> 32);  // 2^-32 turns
    const int quarter = (int)((unsigned)at + 0x20000000u) >> 30;
    const float z = (float)(int)((unsigned)at - ((unsigned)quarter << 30)) * 1.46291808e-9f;  // 2 pi / 2^32
    // Taylor's series up to z = pi / 4: the next terms are 2^-28 and 2^-32 of the sum.
    const float z2 = z * z;
    const float sin0 =
        fmaf(z * z2, fmaf(z2, fmaf(z2, fmaf(z2, 1.f / 362880, -1.f / 5040), 1.f / 120), -1.f / 6), z);
    const float cos0 = fmaf(
        z2, fmaf(z2, fmaf(z2, fmaf(z2, fmaf(z2, -1.f / 3628800, 1.f / 40320), -1.f / 720), 1.f / 24), -0.5f), 1.f);
    const float cs = quarter & 1 ? sin0 : cos0, sn = quarter & 1 ? cos0 : sin0;
    *c = (quarter + 1) & 2 ? -cs : cs;
    *s = quarter & 2 ? -sn : sn;
}

template <bool kBf16>
__device__ __forceinline__ float widen(uint16_t x) {
    if (kBf16) return __uint_as_float((unsigned)x << 16);
    return __half2float(__ushort_as_half(x));
}
template <bool kBf16>
__device__ __forceinline__ uint16_t narrow(float x) {
    if (kBf16) return __bfloat16_as_ushort(__float2bfloat16_rn(x));
    return __half_as_ushort(__float2half_rn(x));
}

// Two numbers that one instruction takes: what is not arithmetic takes most of
// the instructions here, so that every second one of it counts.
struct Two {
    float a, b;
};
__device__ __forceinline__ unsigned long long bits(Two x) {
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x.a), "f"(x.b));
    return r;
}
__device__ __forceinline__ Two two(unsigned long long r) {
    Two x;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x.a), "=f"(x.b) : "l"(r));
    return x;
}
__device__ __forceinline__ Two mul(Two x, Two y) {
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits(x)), "l"(bits(y)));
    return two(r);
}
__device__ __forceinline__ Two fma(Two x, Two y, Two z) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits(x)), "l"(bits(y)), "l"(bits(z)));
    return two(r);
}

// The eight elements of a vector, two by two.
template <bool kBf16>
__device__ __forceinline__ void unpack(const int4& v, Two* x) {
    const unsigned w[4] = {(unsigned)v.x, (unsigned)v.y, (unsigned)v.z, (unsigned)v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (kBf16) {
            x[i] = {__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u)};
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            x[i] = {f.x, f.y};
        }
    }
}
template <bool kBf16>
__device__ __forceinline__ int4 pack(const Two* x) {
    unsigned w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (kBf16) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(x[i].a, x[i].b);
            w[i] = *reinterpret_cast<const unsigned*>(&b);
        } else {
            const __half2 b = __floats2half2_rn(x[i].a, x[i].b);
            w[i] = *reinterpret_cast<const unsigned*>(&b);
        }
    }
    return make_int4((int)w[0], (int)w[1], (int)w[2], (int)w[3]);
}

// The last sequence whose tokens start at or before t: by a warp, 32
// candidates a round, or by each lane for itself.
__device__ __forceinline__ int find_seq(const int* starts, int seqs, int t, int lane) {
    int base = 0, range = seqs;
    while (range > 1) {
        const int step = (range + 31) / 32, at = base + lane * step;
        const bool on = lane * step < range && starts[at] <= t;
        const int k = 31 - __clz(__ballot_sync(kFullMask, on) | 1u);
        base += k * step;
        range = min(step, range - k * step);
    }
    return base;
}
__device__ __forceinline__ int find_seq(const int* starts, int seqs, int t) {
    int base = 0, range = seqs;
    while (range > 1) {
        const int half = range / 2;
        if (starts[base + half] <= t) {
            base += half;
            range -= half;
        } else {
            range = half;
        }
    }
    return base;
}

// A 16-byte copy to shared memory that goes on by itself; each lane waits for its own.
__device__ __forceinline__ void copy_async(int4* to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kMore>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kMore) : "memory");
}

// How a lane's share of a head lies: kHalves and kNeighbours, two vectors of
// eight elements, x[0..3] and x[4..7]; kSingle, four pairs of single elements,
// x[0..3], for heads whose pairs do not fill vectors.
enum Layout { kHalves, kNeighbours, kSingle };

template <bool kBf16, Layout kLayout>
struct Share {
    static constexpr bool kWide = kLayout != kSingle;
    static constexpr int kMany = kWide ? 8 : 4;  // of two elements each
    static constexpr int kTurns = kWide ? 8 : 4;  // pairs that are turned together, or not, by an angle each
    int unit, half, dim;  // unit: the lane's number in its head
    bool neighbours;

    // The number in the head of the pair that has angle i.  In kHalves a lane's
    // pairs are all turned or none.
    __device__ __forceinline__ int pair(int i) const {
        return kLayout == kHalves ? 8 * unit + i : kLayout == kSingle ? unit + 32 * i : (i < 4 ? 0 : dim / 4 - 4) + 4 * unit + i;
    }
    __device__ __forceinline__ bool turned(int i) const { return pair(kLayout == kHalves ? 0 : i) < half; }
    // Wide: the vectors' places in the head.  Each of the two lies beside the
    // neighbouring lanes', so that they read and write whole sectors together:
    // in the two halves of what is turned, or of what is not, or of the head.
    __device__ __forceinline__ int first() const { return 8 * unit + (kLayout == kHalves && 8 * unit >= half ? half : 0); }
    __device__ __forceinline__ int second() const {
        return 8 * unit + (kLayout == kHalves && 8 * unit < half ? half : dim / 2);
    }
    // Single: the places in the head of pair i's elements.
    __device__ __forceinline__ bool has(int i) const { return 2 * pair(i) < dim; }
    __device__ __forceinline__ int a(int i) const {
        const int p = pair(i);
        return neighbours || p >= half ? 2 * p : p;
    }
    __device__ __forceinline__ int b(int i) const {
        const int p = pair(i);
        return neighbours || p >= half ? 2 * p + 1 : p + half;
    }

    __device__ __forceinline__ void take(const uint16_t* from, Two (&x)[kMany]) const {
        if constexpr (kWide) {
            unpack<kBf16>(__ldg(reinterpret_cast<const int4*>(from + first())), x);
            unpack<kBf16>(__ldg(reinterpret_cast<const int4*>(from + second())), x + 4);
        } else {
#pragma unroll
            for (int i = 0; i < kMany; ++i)
                x[i] = has(i) ? Two{widen<kBf16>(from[a(i)]), widen<kBf16>(from[b(i)])} : Two{0.f, 0.f};
        }
    }
    __device__ __forceinline__ void put(uint16_t* to, const Two (&x)[kMany]) const {
        if constexpr (kWide) {
            *reinterpret_cast<int4*>(to + first()) = pack<kBf16>(x);
            *reinterpret_cast<int4*>(to + second()) = pack<kBf16>(x + 4);
        } else {
#pragma unroll
            for (int i = 0; i < kMany; ++i) {
                if (!has(i)) continue;
                to[a(i)] = narrow<kBf16>(x[i].a);
                to[b(i)] = narrow<kBf16>(x[i].b);
            }
        }
    }
    // Cosines and sines of the lane's angles, as turn() takes them.  What is
    // not turned stays as it is, were it infinite.
    struct Angles {
        Two c[kLayout == kHalves ? 4 : kTurns], s[kLayout == kHalves ? 4 : kTurns], minus[kLayout == kHalves ? 4 : 1];
        __device__ __forceinline__ void set(int i, float cs, float sn) {
            if constexpr (kLayout == kHalves) {
                (i & 1 ? c[i / 2].b : c[i / 2].a) = cs;
                (i & 1 ? s[i / 2].b : s[i / 2].a) = sn;
                (i & 1 ? minus[i / 2].b : minus[i / 2].a) = -sn;
            } else {
                c[i] = {cs, cs};
                s[i] = {-sn, sn};
            }
        }
    };
    __device__ __forceinline__ void turn(Two (&x)[kMany], const Angles& t) const {
        if constexpr (kLayout == kHalves) {
            if (!turned(0)) return;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const Two a = x[i], b = x[i + 4];
                x[i] = fma(a, t.c[i], mul(b, t.minus[i]));
                x[i + 4] = fma(b, t.c[i], mul(a, t.s[i]));
            }
        } else {
#pragma unroll
            for (int i = 0; i < kMany; ++i) {
                if (!turned(i)) continue;
                x[i] = fma(x[i], t.c[i], mul({x[i].b, x[i].a}, t.s[i]));
            }
        }
    }
};

// kShift: log2 of the lanes that a head is given.
template <bool kBf16, Layout kLayout, int kShift, bool kCache>
__global__ void __launch_bounds__(kRotateThreads, kCache ? kBlocksCache : kBlocks) kv_rotate_kernel(const __grid_constant__ RotateArgs a) {
    using Share = Share<kBf16, kLayout>;
    constexpr bool kWide = Share::kWide;
    constexpr int kMany = Share::kMany, kTurns = Share::kTurns;
    constexpr int kAtOnce = 32 >> kShift;  // heads that a warp has at a time
    __shared__ __align__(16) unsigned long long turns[TOPK_KV_MAX_DIM / 2];
    __shared__ bool odd[TOPK_KV_MAX_DIM / 2];  // a frequency that is no number
    __shared__ __align__(16) float trig[kWide ? kRotateThreads / 32 : 1][2][TOPK_KV_MAX_DIM / 2];  // of a warp's token
    extern __shared__ __align__(16) int4 rings[];  // [kWarps][kDepth][kUnroll][2][32]
    const int lane = threadIdx.x & 31, warp = __shfl_sync(kFullMask, (int)threadIdx.x >> 5, 0);
    grid_dependency_wait();  // launched early (launch_pdl): the previous kernel's writes first
    // Units w0, w0 + all, ... are this warp's: all warps together go through
    // memory in order (2% to 4% faster than a stretch of units for each).
    const int all = gridDim.x * kWarps, w0 = blockIdx.x * kWarps + warp;
    const int count = w0 < a.units ? (a.units - w0 + all - 1) / all : 0;
    const int sub = lane >> kShift;
    const Share share = {lane & ((1 << kShift) - 1), a.r.half, a.r.dim, a.r.neighbours};
    const bool on = share.unit < a.lanes;

    // A walk over the units' steps.
    struct Walk {
        int left, token, part;  // units left, this one counted; the token, and which of its units
        int at, to;             // the next step, and the one behind the last
    };
    auto begin = [&](Walk& p) {
        p.at = p.part * a.chunk;
        p.to = min(p.at + a.chunk, a.steps[2]);
    };
    auto go_on = [&](Walk& p) {
        if (++p.at < p.to) return;
        --p.left;
        p.token += a.tokens_on;
        p.part += a.parts_on;
        if (p.part >= a.chunks) {
            p.part -= a.chunks;
            ++p.token;
        }
        begin(p);
    };
    // A step's heads: of one kind, kUnroll * kAtOnce from `base` on.
    struct Step {
        int kind, base;
    };
    auto step_of = [&](int i) -> Step {
        const int kind = i < a.steps[0] ? 0 : i < a.steps[1] ? 1 : 2, first = kind == 0 ? 0 : a.steps[kind - 1];
        return {kind, (i - first) * (kUnroll * kAtOnce) + sub};  // this lane's first
    };
    // Of a kind: by an index, or by choice where that is faster (162 against 183 us
    // for the prompts above; without a cache 125 against 122).
    auto of = [](const auto& x, int kind) { return !kCache ? x[kind] : kind == 0 ? x[0] : kind == 1 ? x[1] : x[2]; };
    auto of2 = [](const auto& x, int kind) { return !kCache ? x[kind] : kind == 0 ? x[0] : x[1]; };
    auto vectors = [](unsigned n, unsigned each) { return (unsigned long long)n * each * 8; };
    auto source = [&](const Step& s, int t) {
        return of(a.in, s.kind) + vectors(t, of(a.in_token, s.kind)) + vectors(s.base, of(a.in_head, s.kind));
    };
    int4* ring = rings + warp * (kDepth * kUnroll * 2 * 32) + lane;
    auto fetch = [&](Walk& p, int place) {
        if (!kWide) return;
        if (p.left > 0) {
            const Step s = step_of(p.at);
            const uint16_t* x = source(s, p.token);
            const unsigned long long apart = vectors(kAtOnce, of(a.in_head, s.kind));
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                if (on && s.base + u * kAtOnce < of(a.heads, s.kind)) {
                    copy_async(ring + ((place * kUnroll + u) * 2) * 32, x + u * apart + share.first());
                    copy_async(ring + ((place * kUnroll + u) * 2 + 1) * 32, x + u * apart + share.second());
                }
            }
            go_on(p);
        }
        copies_end();
    };
    Walk now_at = {count, w0 / a.chunks, w0 % a.chunks};
    begin(now_at);
    Walk ahead = now_at;
#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i) fetch(ahead, i);  // does not depend on what follows

    if (threadIdx.x < a.r.half) {
        const float f = a.r.freq[threadIdx.x];
        turns[threadIdx.x] = turns_of(f);
        odd[threadIdx.x] = !(fabsf(f) <= 3.402823466e38f);
    }
    __syncthreads();

    typename Share::Angles angles;
    // The places of 32 units' tokens, a lane each.
    int position = 0, seq = -1, slot_held = -1, page = -1, in_page = 0;
    int now_position = 0, now_seq = 0, now_slot = 0, now_page = 0, now_in_page = 0;
    int left_before = 0, place = 0;
    while (now_at.left > 0) {
        const int t = now_at.token;
        if (now_at.left != left_before) {  // a new token, or other heads of it
            left_before = now_at.left;
            const int unit = count - now_at.left;
            if ((unit & 31) == 0) {
                position = 0, seq = -1, slot_held = -1, page = -1, in_page = 0;
                const bool valid = lane < now_at.left;
                const int mine = valid ? (w0 + (unit + lane) * all) / a.chunks : 0;
                if (kCache) {
                    int b = mine;
                    if (a.r.starts) {
                        if (count == 1) b = find_seq(a.r.starts, a.c.seqs, t, lane);
                        else if (valid) b = find_seq(a.r.starts, a.c.seqs, mine);
                    }
                    if (valid) {
                        long long i = 0;  // starts are the caller's: neither this nor the slot may wrap
                        bool in = true;
                        if (a.r.starts) {
                            int end = a.r.starts[b + 1];
                            while (end <= mine && b + 1 < a.c.seqs) end = a.r.starts[++b + 1];
                            i = (long long)mine - a.r.starts[b];
                            in = mine < end && i >= 0;  // else past the last sequence's tokens
                        }
                        if (in) {
                            seq = b;
                            const int n = a.c.len(b);
                            position = (int)((unsigned)(a.r.next_pos ? a.r.next_pos[b] : n) + (unsigned)i);
                            if (n + i < a.c.capacity()) {
                                slot_held = (int)(n + i);
                                page = a.c.page_of(b, slot_held);
                                in_page = slot_held % a.c.page_size;
                            }
                        }
                    }
                } else if (valid) {
                    seq = 0;
                    position = a.r.pos[mine];
                }
            }
            const int from = unit & 31;
            now_position = __shfl_sync(kFullMask, position, from);
            now_seq = __shfl_sync(kFullMask, seq, from);
            if (kCache) {
                now_slot = __shfl_sync(kFullMask, slot_held, from);
                now_page = __shfl_sync(kFullMask, page, from);
                now_in_page = __shfl_sync(kFullMask, in_page, from);
            }
            // The warp works out each angle once, and its lanes take theirs.
            auto work_out = [&](int pair, float* c, float* s) {
                turn(turns[pair], now_position, c, s);
                if (odd[pair]) *c = *s = __int_as_float(0x7FFFFFFF);
            };
            if constexpr (kWide) {
                float(&mine)[2][TOPK_KV_MAX_DIM / 2] = trig[threadIdx.x >> 5];
                __syncwarp();  // the token before is done with
                for (int p = lane; p < a.r.half; p += 32) work_out(p, &mine[0][p], &mine[1][p]);
                __syncwarp();
                if (on) {
#pragma unroll
                    for (int i = 0; i < kTurns; i += 4) {
                        const float4 c = *reinterpret_cast<const float4*>(&mine[0][share.pair(i)]);
                        const float4 s = *reinterpret_cast<const float4*>(&mine[1][share.pair(i)]);
                        angles.set(i, c.x, s.x);
                        angles.set(i + 1, c.y, s.y);
                        angles.set(i + 2, c.z, s.z);
                        angles.set(i + 3, c.w, s.w);
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < kTurns; ++i) {
                    if (!share.turned(i)) continue;
                    float c, s;
                    work_out(share.pair(i), &c, &s);
                    angles.set(i, c, s);
                }
            }
        }
        const Step now = step_of(now_at.at);
        go_on(now_at);
        copies_wait<kDepth - 2>();
        const int4* raw = ring + place * (kUnroll * 2 * 32);
        // Into the place of the step before, which is done with.
        fetch(ahead, place == 0 ? kDepth - 1 : place - 1);
        place = place == kDepth - 1 ? 0 : place + 1;
        if (now_seq < 0) continue;
        uint16_t* target = nullptr;
        unsigned long long apart;  // between the heads of a step
        if (!kCache || now.kind == kQueries) {
            const int kind = now.kind & 1;
            target = of2(a.out, kind) + vectors(t, of2(a.out_token, kind)) + vectors(now.base, of2(a.out_head, kind));
            apart = vectors(kAtOnce, of2(a.out_head, kind));
        } else {
            uint16_t* pool = now.kind == kKeys ? a.c.k : a.c.v;
            const long long* strides = now.kind == kKeys ? a.c.ks : a.c.vs;
            if (now_page >= 0) target = pool + now_page * strides[0] + now_in_page * strides[1] + now.base * strides[2];
            apart = kAtOnce * strides[2];
        }
        const bool value = kCache && now.kind == kValues;
        const uint16_t* w = value ? nullptr : of2(a.norm, now.kind & 1);
        const unsigned w_head = of2(a.norm_head, now.kind & 1);
        Two weight[kMany];
        if (w && w_head == 0 && on) share.take(w, weight);  // one for all heads
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int h = now.base + u * kAtOnce;
            const bool mine = on && h < of(a.heads, now.kind);
            uint16_t* to_here = target + u * apart;
            if (kCache && now.kind == kKeys && mine && share.unit == 0 && now_slot >= 0) {
                if (a.r.weight.data) a.r.weight.row(now_seq, h)[now_slot] = 0.f;
                if (a.r.pos_rows.data) a.r.pos_rows.row(now_seq, h)[now_slot] = now_position;
            }
            if (value) {  // copied
                if (mine && target) {
                    if (kWide) {
                        *reinterpret_cast<int4*>(to_here + share.first()) = raw[(2 * u) * 32];
                        *reinterpret_cast<int4*>(to_here + share.second()) = raw[(2 * u + 1) * 32];
                    } else {
                        const uint16_t* x = source(now, t) + u * vectors(kAtOnce, a.in_head[kValues]);
                        for (int i = lane; i < a.r.dim; i += 32) to_here[i] = x[i];
                    }
                }
                continue;
            }
            Two x[kMany];
            if constexpr (kWide) {
                unpack<kBf16>(raw[(2 * u) * 32], x);
                unpack<kBf16>(raw[(2 * u + 1) * 32], x + 4);
            } else if (mine) {
                share.take(source(now, t) + u * vectors(kAtOnce, a.in_head[now.kind]), x);
            }
            if (w) {  // by all lanes, which add up
                Two sums = {0.f, 0.f};
                if (mine) {
#pragma unroll
                    for (int i = 0; i < kMany; ++i) sums = fma(x[i], x[i], sums);
                }
                float sum = sums.a + sums.b;
#pragma unroll
                for (int d = 1; d < (1 << kShift); d <<= 1) sum += __shfl_xor_sync(kFullMask, sum, d);
                if (w_head != 0 && mine) share.take(w + vectors(h, w_head), weight);
                if (mine) {
                    float r;  // to 2^-22.4
                    asm("rsqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(fmaf(sum, a.r.per_dim, a.r.eps)));
#pragma unroll
                    for (int i = 0; i < kMany; ++i) x[i] = mul(mul(x[i], {r, r}), weight[i]);
                }
            }
            if (!mine || !target) continue;
            share.turn(x, angles);
            share.put(to_here, x);
        }
    }
}

template <bool kBf16, Layout kLayout, int kShift, bool kCache>
cudaError_t launch(const RotateArgs& a, int device, int blocks, cudaStream_t s) {
    auto kernel = kv_rotate_kernel<kBf16, kLayout, kShift, kCache>;
    constexpr int kSmem = kLayout == kSingle ? 0 : kWarps * kDepth * kUnroll * 2 * 32 * (int)sizeof(int4);
    static std::atomic<unsigned long long> allowed{0};
    const cudaError_t e = kSmem ? allow_smem(kernel, kSmem, device, allowed) : cudaSuccess;
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, dim3((unsigned)blocks), dim3(kRotateThreads), kSmem, s, a);
}
using Launch = cudaError_t (*)(const RotateArgs&, int, int, cudaStream_t);
template <bool kBf16, bool kCache>
Launch launch_of(Layout layout, int shift) {
    if (layout == kSingle) return launch<kBf16, kSingle, 5, kCache>;
    if (layout == kHalves)
        return shift == 2   ? launch<kBf16, kHalves, 2, kCache>
               : shift == 3 ? launch<kBf16, kHalves, 3, kCache>
                            : launch<kBf16, kHalves, 4, kCache>;
    return shift == 2   ? launch<kBf16, kNeighbours, 2, kCache>
           : shift == 3 ? launch<kBf16, kNeighbours, 3, kCache>
                        : launch<kBf16, kNeighbours, 4, kCache>;
}

}  // namespace

cudaError_t kv_rotate_launch(int device, int sms, cudaStream_t s, const KvCache* c, const KvRotate& r, bool bf16) {
    RotateArgs a = {};
    if (c) a.c = *c;
    a.r = r;
    // Two vectors to a lane where pairs fill them: always for neighbours, else
    // where half of the turned elements is a whole number of vectors.
    const bool wide = r.dim % 16 == 0 && (r.neighbours || r.half % 8 == 0);
    const Layout layout = !wide ? kSingle : r.neighbours ? kNeighbours : kHalves;
    a.lanes = wide ? r.dim / 16 : 32;
    int shift = 2;
    while ((1 << shift) < a.lanes) ++shift;
    const int heads = kUnroll * (32 >> shift);
    a.steps[0] = (r.q_heads + heads - 1) / heads;
    a.steps[1] = a.steps[0] + (r.heads + heads - 1) / heads;
    a.steps[2] = a.steps[1] + (c ? (r.heads + heads - 1) / heads : 0);
    const int all = a.steps[2];
    a.chunk = 1;
    while (a.chunk < all && (c || a.chunk < kSteps) && (long long)r.tokens * ((all + 2 * a.chunk - 1) / (2 * a.chunk)) >= sms * 16) a.chunk *= 2;
    a.chunks = (all + a.chunk - 1) / a.chunk;
    a.chunk = (all + a.chunks - 1) / a.chunks;
    if ((long long)r.tokens * a.chunks > (1 << 30)) {  // units are numbered in 32 bits
        a.chunk = all;
        a.chunks = 1;
    }
    if (r.tokens > (1 << 30)) return cudaErrorInvalidValue;
    a.units = r.tokens * a.chunks;
    const int blocks = std::min((a.units + kWarps - 1) / kWarps, sms * (c ? kBlocksCache : kBlocks));
    a.tokens_on = blocks * kWarps / a.chunks;
    a.parts_on = blocks * kWarps % a.chunks;
    auto set = [&](int kind, const uint16_t* x, const long long* strides, int n) {
        a.in[kind] = x;
        a.in_token[kind] = (unsigned)(strides[0] / 8);
        a.in_head[kind] = (unsigned)(strides[1] / 8);
        a.heads[kind] = n;
    };
    set(kQueries, r.q, r.qs, r.q_heads);
    set(kKeys, r.k, r.ks, r.heads);
    set(kValues, r.v, r.vs, r.heads);
    auto set_out = [&](int kind, uint16_t* x, const long long* strides, const uint16_t* norm, long long norm_stride) {
        a.out[kind] = x;
        a.out_token[kind] = (unsigned)(strides[0] / 8);
        a.out_head[kind] = (unsigned)(strides[1] / 8);
        a.norm[kind] = norm;
        a.norm_head[kind] = (unsigned)(norm_stride / 8);
    };
    set_out(kQueries, r.q_out, r.qos, r.q_norm, r.q_norm_stride);
    set_out(kKeys, r.k_out, r.kos, r.k_norm, r.k_norm_stride);
    const Launch go = bf16 ? (c ? launch_of<true, true>(layout, shift) : launch_of<true, false>(layout, shift))
                           : (c ? launch_of<false, true>(layout, shift) : launch_of<false, false>(layout, shift));
    return go(a, device, blocks, s);
}

}  // namespace topk
