// topk_kv_append: copy new tokens' keys and values into their pages.
//
// Nothing is computed: bound by HBM for prompts (every element is read and
// written once) and by the launch for a decoding step.  An item is one
// token's head, its key and value copied as 16-byte vectors.  A warp takes up
// to 32 items: a lane looks up one item's place, and all lanes copy, eight
// vectors in flight each.  With few items a warp takes one, so that a step of
// decoding is spread over the GPU.  The copies' reads do not depend on the
// look-up, so the first are under way while it runs.
//
// Measured: 40942 tokens of 8 heads, dim 128 (338 MB): 54 us, 6.2 TB/s, 92%
// of a copy's rate; one token each of 64 sequences: 3.7 us a call, which is
// the host's.
#include "topk_device.cuh"
#include "topk_kv.cuh"

namespace topk {
namespace {

constexpr int kAppendThreads = 256;

struct AppendArgs {
    KvCache c;
    const uint16_t *k_new, *v_new;
    long long kns[2], vns[2];
    int tokens;
    const int* starts;
    KvRows<float> weight;
    KvRows<int> pos;
    const int* next_pos;
    int per;    // items of a warp
    int shift;  // log2 of the lanes that a key takes
};

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

__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const __grid_constant__ AppendArgs a) {
    constexpr int kUnroll = 4;  // of keys and of values each
    __shared__ int4 where[kAppendThreads / 32][32];  // token, head, page (-1: nowhere) and slot in it
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long items = (long long)a.tokens * a.c.heads;
    const long long first = ((long long)blockIdx.x * (kAppendThreads / 32) + warp) * a.per;
    if (first >= items) return;
    grid_dependency_wait();  // launched early (launch_pdl): the previous kernel's writes first
    const int count = (int)min((long long)a.per, items - first);
    const int t = (int)((first + lane) / a.c.heads), h = (int)(first + lane - (long long)t * a.c.heads);
    where[warp][lane] = make_int4(t, h, -1, 0);
    __syncwarp();
    // A key's vectors take a power of two of lanes, and its value's the same
    // ones: no vector costs a division, and strides are the warp's.
    const int total = count << a.shift, x = (lane & ((1 << a.shift) - 1)) * 8;
    const bool on = x < a.c.dim;
    bool looked_up = false;
    for (int i0 = lane; i0 - lane < total; i0 += 32 * kUnroll) {
        int4 k[kUnroll], v[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int i = i0 + 32 * u;
            if (i < total && on) {
                const int4 at = where[warp][i >> a.shift];
                k[u] = __ldcs(reinterpret_cast<const int4*>(a.k_new + at.x * a.kns[0] + at.y * a.kns[1] + x));
                v[u] = __ldcs(reinterpret_cast<const int4*>(a.v_new + at.x * a.vns[0] + at.y * a.vns[1] + x));
            }
        }
        if (!looked_up) {
            looked_up = true;
            int b = a.starts ? find_seq(a.starts, a.c.seqs, __shfl_sync(kFullMask, t, 0), lane) : t;
            if (lane < count) {
                long long i = 0;  // starts are the caller's: neither this nor the slot may wrap
                bool in = true;
                if (a.starts) {
                    int next = a.starts[b + 1];
                    while (next <= t && b + 1 < a.c.seqs) next = a.starts[++b + 1];
                    in = t < next;  // else past the last sequence's tokens
                    i = (long long)t - a.starts[b];
                }
                const long long at = a.c.len(b) + i;
                if (in && i >= 0 && at < a.c.capacity()) {
                    const int slot = (int)at;
                    where[warp][lane].z = a.c.page_of(b, slot);
                    where[warp][lane].w = slot % a.c.page_size;
                    if (a.weight.data) a.weight.row(b, h)[slot] = 0.f;
                    if (a.pos.data) a.pos.row(b, h)[slot] = a.next_pos[b] + (int)i;
                }
            }
            __syncwarp();
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int i = i0 + 32 * u;
            if (i < total && on) {
                const int4 at = where[warp][i >> a.shift];
                if (at.z < 0) continue;
                *reinterpret_cast<int4*>(a.c.k + at.z * a.c.ks[0] + at.w * a.c.ks[1] + at.y * a.c.ks[2] + x) = k[u];
                *reinterpret_cast<int4*>(a.c.v + at.z * a.c.vs[0] + at.w * a.c.vs[1] + at.y * a.c.vs[2] + x) = v[u];
            }
        }
    }
}

}  // namespace

cudaError_t kv_append_launch(int sms, cudaStream_t s, const KvCache& c, const uint16_t* k_new,
                             const long long* k_stride, const uint16_t* v_new, const long long* v_stride, int tokens,
                             const int* starts, KvRows<float> weight, KvRows<int> pos, const int* next_pos) {
    AppendArgs a = {c, k_new, v_new, {k_stride[0], k_stride[1]}, {v_stride[0], v_stride[1]},
                    tokens, starts, weight, pos, next_pos, 1, 0};
    while ((1 << a.shift) < c.dim / 8) ++a.shift;  // dim is at most 256: 32 lanes
    const long long items = (long long)tokens * c.heads;
    // 16 warps an SM at least, then longer ones (40942 tokens of 8 heads: 164 us
    // with one item a warp, 59 with 8 or 16, 62 with 32).
    while (a.per < 16 && items / (2 * a.per) >= sms * 16) a.per *= 2;
    const long long warps = (items + a.per - 1) / a.per, blocks = (warps + kAppendThreads / 32 - 1) / (kAppendThreads / 32);
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
    return launch_pdl(kv_append_kernel, dim3((unsigned)blocks), dim3(kAppendThreads), 0, s, a);
}

}  // namespace topk
