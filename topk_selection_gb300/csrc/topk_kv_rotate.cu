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
// Bound by HBM for prompts: every element is read and written once.  A warp
// has one token and some of its heads.  A lane has the same eight pairs of
// each head, both vectors of them, so that nothing is exchanged for the
// rotation, the angles' cosines and sines are worked out once for all heads,
// and a norm costs the shuffles of one sum.
//
// Angles.  A product of 32 bits knows a position of 10^6 times a frequency
// near 1 to 0.06 radians only.  Here a frequency becomes a whole number of
// 2^-64 turns per position, so that the product with the position, whole turns
// dropped, is the low half of one multiplication of integers: good to 2^-32
// turns at any position, and no reduction follows but to the nearest quarter.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "topk_device.cuh"
#include "topk_kv.cuh"

namespace topk {
namespace {

constexpr int kRotateThreads = 256;

struct RotateArgs {
    KvCache c;  // of an append
    KvRotate r;
    int units;   // lanes that a head takes
    int shift;   // log2 of the lanes that it is given
    int slots;   // heads of queries, keys and, in an append, values
    int rounds;  // of a warp: heads that its lanes take at a time, one after another
    int chunks;  // warps of a token
};

// cos and sin of pos * freq.
__device__ __forceinline__ void turn(float freq, int pos, float* c, float* s) {
    const unsigned bits = __float_as_uint(freq);
    const int exponent = (bits >> 23) & 255;
    const unsigned long long mantissa = exponent ? (bits & 0x7FFFFFu) | 0x800000u : 0u;
    // freq = mantissa * 2^(exponent - 150); 2^64 / (2 pi), whole.
    constexpr unsigned long long kPerRadian = 0x28BE60DB9391054Aull;
    const unsigned long long low = mantissa * kPerRadian, high = __umul64hi(mantissa, kPerRadian);
    const int down = 150 - exponent;
    unsigned long long per;  // 2^-64 turns per position
    if (down >= 64) per = down < 96 ? high >> (down - 64) : 0;
    else if (down > 0) per = (high << (64 - down)) | (low >> down);
    else per = low << (-down & 63);
    if (bits >> 31) per = 0 - per;
    const int at = (int)((per * (unsigned long long)(long long)pos) >> 32);  // 2^-32 turns
    const int quarter = (int)((unsigned)at + 0x20000000u) >> 30;
    const float z = (float)(int)((unsigned)at - ((unsigned)quarter << 30)) * 1.46291807926715968e-9f;  // 2 pi / 2^32
    // Taylor's series up to z = pi / 4: the next terms are 2^-28 and 2^-32 of the sum.
    const float z2 = z * z;
    const float sin0 =
        fmaf(z * z2, fmaf(z2, fmaf(z2, fmaf(z2, 1.f / 362880, -1.f / 5040), 1.f / 120), -1.f / 6), z);
    const float cos0 = fmaf(
        z2, fmaf(z2, fmaf(z2, fmaf(z2, fmaf(z2, -1.f / 3628800, 1.f / 40320), -1.f / 720), 1.f / 24), -0.5f), 1.f);
    const float cs = quarter & 1 ? sin0 : cos0, sn = quarter & 1 ? cos0 : sin0;
    *c = (quarter + 1) & 2 ? -cs : cs;
    *s = quarter & 2 ? -sn : sn;
    if (exponent == 255) *c = *s = __int_as_float(0x7FFFFFFF);  // no number times a position
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

// The eight elements of a vector.
template <bool kBf16>
__device__ __forceinline__ void unpack(const int4& v, float* x) {
    const unsigned w[4] = {(unsigned)v.x, (unsigned)v.y, (unsigned)v.z, (unsigned)v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (kBf16) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
}
template <bool kBf16>
__device__ __forceinline__ int4 pack(const float* x) {
    unsigned w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (kBf16) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const unsigned*>(&b);
        } else {
            const __half2 b = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const unsigned*>(&b);
        }
    }
    return make_int4((int)w[0], (int)w[1], (int)w[2], (int)w[3]);
}

// The last sequence whose tokens start at or before t: 32 candidates a round.
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

// How a lane's share of a head lies: kHalves and kNeighbours, two vectors of
// eight elements; kSingle, four pairs of single elements, for heads whose
// pairs do not fill vectors.
enum Layout { kHalves, kNeighbours, kSingle };

template <Layout kLayout>
struct Share {
    static constexpr bool kWide = kLayout != kSingle;
    static constexpr int kPairs = kWide ? 8 : 4, kMany = 2 * kPairs;
    int unit, half, dim;
    bool neighbours;
    // Pair i of the lane: the places of its two elements in the share, its
    // number in the head, and whether it is turned.  A vector without turned
    // pairs has none that matter.
    static __device__ __forceinline__ constexpr int a(int i) { return kLayout == kNeighbours ? 2 * i : i; }
    static __device__ __forceinline__ constexpr int b(int i) { return kLayout == kNeighbours ? 2 * i + 1 : kPairs + i; }
    __device__ __forceinline__ int pair(int i) const { return kWide ? 8 * unit + i : unit + 32 * i; }
    __device__ __forceinline__ bool turned(int i) const { return pair(i) < half; }
    // Wide: the vectors' places in the head.
    __device__ __forceinline__ bool behind() const { return kLayout == kNeighbours || 8 * unit >= half; }
    __device__ __forceinline__ int first() const { return behind() ? 16 * unit : 8 * unit; }
    __device__ __forceinline__ int second() const { return behind() ? 16 * unit + 8 : half + 8 * unit; }
    // Single: the place in the head of element i of the share, or -1.
    __device__ __forceinline__ int place(int i) const {
        const int p = pair(i % kPairs), second = i >= kPairs;
        if (2 * p >= dim) return -1;
        return neighbours || p >= half ? 2 * p + second : p + second * half;
    }

    template <bool kBf16>
    __device__ __forceinline__ void load(const uint16_t* from, float (&x)[kMany]) const {
        if constexpr (kWide) {
            split<kBf16>(__ldg(reinterpret_cast<const int4*>(from + first())),
                         __ldg(reinterpret_cast<const int4*>(from + second())), x);
        } else {
#pragma unroll
            for (int i = 0; i < kMany; ++i) x[i] = place(i) >= 0 ? widen<kBf16>(from[place(i)]) : 0.f;
        }
    }
    template <bool kBf16>
    static __device__ __forceinline__ void split(const int4& v0, const int4& v1, float (&x)[kMany]) {
        if constexpr (kWide) {
            unpack<kBf16>(v0, x);
            unpack<kBf16>(v1, x + 8);
        }
    }
    template <bool kBf16>
    __device__ __forceinline__ void store(uint16_t* to, const float (&x)[kMany]) const {
        if constexpr (kWide) {
            *reinterpret_cast<int4*>(to + first()) = pack<kBf16>(x);
            *reinterpret_cast<int4*>(to + second()) = pack<kBf16>(x + 8);
        } else {
#pragma unroll
            for (int i = 0; i < kMany; ++i)
                if (place(i) >= 0) to[place(i)] = narrow<kBf16>(x[i]);
        }
    }
};

template <bool kBf16, Layout kLayout, bool kCache>
__global__ void __launch_bounds__(kRotateThreads) kv_rotate_kernel(const __grid_constant__ RotateArgs a) {
    using Share = Share<kLayout>;
    constexpr bool kWide = Share::kWide;
    constexpr int kMany = Share::kMany, kPairs = Share::kPairs;
    constexpr int kUnroll = kWide ? 2 : 1;  // heads in flight of a lane
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long job = (long long)blockIdx.x * (kRotateThreads / 32) + warp;
    const int t = (int)(job / a.chunks), chunk = (int)(job - (long long)t * a.chunks);
    if (t >= a.r.tokens) return;
    grid_dependency_wait();  // launched early (launch_pdl): the previous kernel's writes first
    const int at_once = 32 >> a.shift, sub = lane >> a.shift;
    const Share share = {lane & ((1 << a.shift) - 1), a.r.half, a.r.dim, a.r.neighbours};
    const bool on = share.unit < a.units;
    const int from = chunk * a.rounds * at_once, to = min(from + a.rounds * at_once, a.slots);
    const int keys = a.r.q_heads, values = a.r.q_heads + a.r.heads;  // where they begin among the slots

    auto source = [&](int slot) -> const uint16_t* {
        if (slot < keys) return a.r.q + t * a.r.qs[0] + slot * a.r.qs[1];
        if (slot < values) return a.r.k + t * a.r.ks[0] + (slot - keys) * a.r.ks[1];
        return a.r.v + t * a.r.vs[0] + (slot - values) * a.r.vs[1];
    };
    int4 next[kUnroll][2];  // of the slots after these, under way
    auto fetch = [&](int base) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int slot = base + u * at_once + sub;
            if (kWide && on && slot < to) {
                const uint16_t* x = source(slot);
                next[u][0] = __ldcs(reinterpret_cast<const int4*>(x + share.first()));
                next[u][1] = __ldcs(reinterpret_cast<const int4*>(x + share.second()));
            }
        }
    };
    fetch(from);  // does not depend on what follows

    int position, seq = 0, slot_held = -1, page = -1, in_page = 0;
    if (kCache) {
        int b = a.r.starts ? find_seq(a.r.starts, a.c.seqs, t, lane) : t;
        long long i = 0;  // starts are the caller's: neither this nor the slot may wrap
        if (a.r.starts) {
            int end = a.r.starts[b + 1];
            while (end <= t && b + 1 < a.c.seqs) end = a.r.starts[++b + 1];
            i = (long long)t - a.r.starts[b];
            if (t >= end || i < 0) return;  // past the last sequence's tokens
        }
        seq = b;
        const int n = a.c.len(b);
        position = (int)((unsigned)(a.r.next_pos ? a.r.next_pos[b] : n) + (unsigned)i);
        if (n + i < a.c.capacity()) {
            slot_held = (int)(n + i);
            page = a.c.page_of(b, slot_held);
            in_page = slot_held % a.c.page_size;
        }
    } else {
        position = a.r.pos[t];
    }
    float cs[kPairs], sn[kPairs];
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
        cs[i] = 1.f;
        sn[i] = 0.f;
        if (on && share.turned(i)) turn(a.r.freq[share.pair(i)], position, &cs[i], &sn[i]);
    }

    for (int base = from; base < to; base += kUnroll * at_once) {
        int4 raw[kUnroll][2];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            raw[u][0] = next[u][0];
            raw[u][1] = next[u][1];
        }
        if (base + kUnroll * at_once < to) fetch(base + kUnroll * at_once);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int slot = base + u * at_once + sub;
            const bool mine = on && slot < to, query = slot < keys, value = slot >= values;
            uint16_t* target = nullptr;
            if (mine) {
                if (query) {
                    target = a.r.q_out + t * a.r.qos[0] + slot * a.r.qos[1];
                } else if (!kCache) {
                    target = a.r.k_out + t * a.r.kos[0] + (slot - keys) * a.r.kos[1];
                } else {
                    const int h = slot - (value ? values : keys);
                    if (page >= 0)
                        target = value ? a.c.v + page * a.c.vs[0] + in_page * a.c.vs[1] + h * a.c.vs[2]
                                       : a.c.k + page * a.c.ks[0] + in_page * a.c.ks[1] + h * a.c.ks[2];
                    if (!value && share.unit == 0 && slot_held >= 0) {
                        if (a.r.weight.data) a.r.weight.row(seq, h)[slot_held] = 0.f;
                        if (a.r.pos_rows.data) a.r.pos_rows.row(seq, h)[slot_held] = position;
                    }
                }
            }
            if (kCache && value && target) {  // copied
                if (kWide) {
                    *reinterpret_cast<int4*>(target + share.first()) = raw[u][0];
                    *reinterpret_cast<int4*>(target + share.second()) = raw[u][1];
                } else {
                    const uint16_t* x = source(slot);
                    for (int i = lane; i < a.r.dim; i += 32) target[i] = x[i];
                }
            }
            const bool turned = mine && !value;
            float x[kMany];
            if (kWide) Share::template split<kBf16>(raw[u][0], raw[u][1], x);
            else if (turned) share.template load<kBf16>(source(slot), x);
            if (a.r.q_norm || a.r.k_norm) {  // the whole warp: its lanes add up
                float sum = 0.f;
                if (turned) {
#pragma unroll
                    for (int i = 0; i < kMany; ++i) sum = fmaf(x[i], x[i], sum);
                }
                for (int d = 1; d < (1 << a.shift); d <<= 1) sum += __shfl_xor_sync(kFullMask, sum, d);
                const uint16_t* w = query ? a.r.q_norm : a.r.k_norm;
                if (turned && w) {
                    const float r = rsqrtf(sum * a.r.per_dim + a.r.eps);
                    float weight[kMany];
                    share.template load<kBf16>(w + (query ? slot * a.r.q_norm_stride : (slot - keys) * a.r.k_norm_stride),
                                               weight);
#pragma unroll
                    for (int i = 0; i < kMany; ++i) x[i] = x[i] * r * weight[i];
                }
            }
            if (!turned || !target) continue;
#pragma unroll
            for (int i = 0; i < kPairs; ++i) {
                if (!share.turned(i)) continue;  // as it is, were it infinite
                float &first = x[Share::a(i)], &second = x[Share::b(i)];
                const float y = first * cs[i] - second * sn[i];
                second = second * cs[i] + first * sn[i];
                first = y;
            }
            share.template store<kBf16>(target, x);
        }
    }
}

template <bool kBf16, bool kCache>
auto kernel_of(Layout layout) {
    return layout == kHalves       ? kv_rotate_kernel<kBf16, kHalves, kCache>
           : layout == kNeighbours ? kv_rotate_kernel<kBf16, kNeighbours, kCache>
                                   : kv_rotate_kernel<kBf16, kSingle, kCache>;
}

}  // namespace

cudaError_t kv_rotate_launch(int sms, cudaStream_t s, const KvCache* c, const KvRotate& r, bool bf16) {
    RotateArgs a = {};
    if (c) a.c = *c;
    a.r = r;
    a.slots = r.q_heads + (c ? 2 : 1) * r.heads;
    // Two vectors to a lane where pairs fill them: always for neighbours, else
    // where half of the turned elements is a whole number of vectors.
    const bool wide = r.dim % 16 == 0 && (r.neighbours || r.half % 8 == 0);
    const Layout layout = !wide ? kSingle : r.neighbours ? kNeighbours : kHalves;
    a.units = wide ? r.dim / 16 : 32;
    while ((1 << a.shift) < a.units) ++a.shift;
    const int at_once = 32 >> a.shift, all = (a.slots + at_once - 1) / at_once;
    // 16 warps an SM at least, then longer ones, up to a token's heads.
    a.rounds = 1;
    while (a.rounds < all && (long long)r.tokens * ((all + 2 * a.rounds - 1) / (2 * a.rounds)) >= sms * 16) a.rounds *= 2;
    a.chunks = (all + a.rounds - 1) / a.rounds;
    const long long blocks = ((long long)r.tokens * a.chunks + kRotateThreads / 32 - 1) / (kRotateThreads / 32);
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
    auto kernel = bf16 ? (c ? kernel_of<true, true>(layout) : kernel_of<true, false>(layout))
                       : (c ? kernel_of<false, true>(layout) : kernel_of<false, false>(layout));
    return launch_pdl(kernel, dim3((unsigned)blocks), dim3(kRotateThreads), 0, s, a);
}

}  // namespace topk
