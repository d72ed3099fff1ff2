// topk_kv_append: copy new tokens' keys and values into their pages.
//
// Nothing is computed: bound by HBM for prompts and by the launch for a
// decoding step.  A warp takes one token's head and moves its key and value
// as 16-byte vectors, half of the warp each.
#include "topk_device.cuh"
#include "topk_kv.cuh"

namespace topk {
namespace {

struct AppendArgs {
    KvCache c;
    const uint16_t *k_new, *v_new;
    long long kns[2], vns[2];
    int tokens;
    const int* starts;
    KvRows<float> weight;
    KvRows<int> pos;
    const int* next_pos;
};

__global__ void __launch_bounds__(256) kv_append_kernel(const AppendArgs a) {
    const int lane = threadIdx.x & 31;
    const long long item = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int t = (int)(item / a.c.heads), h = (int)(item % a.c.heads);
    if (t >= a.tokens) return;
    int b = t, i = 0;
    if (a.starts) {
        if (t >= a.starts[a.c.seqs]) return;
        int lo = 0, hi = a.c.seqs - 1;  // the last sequence whose tokens start at or before t
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (a.starts[mid] <= t) lo = mid; else hi = mid - 1;
        }
        b = lo;
        i = t - a.starts[b];
    }
    const int slot = a.c.len(b) + i;
    if (i < 0 || slot >= a.c.capacity()) return;
    const int page = a.c.page_of(b, slot);
    const int at = slot % a.c.page_size;
    if (page >= 0) {
        const bool v = lane >= 16;
        const uint16_t* src = v ? a.v_new + t * a.vns[0] + h * a.vns[1] : a.k_new + t * a.kns[0] + h * a.kns[1];
        uint16_t* dst = v ? a.c.v + page * a.c.vs[0] + at * a.c.vs[1] + h * a.c.vs[2]
                          : a.c.k + page * a.c.ks[0] + at * a.c.ks[1] + h * a.c.ks[2];
        for (int x = (lane & 15) * 8; x < a.c.dim; x += 128)
            *reinterpret_cast<int4*>(dst + x) = *reinterpret_cast<const int4*>(src + x);
    }
    if (lane == 0) {
        if (a.weight.data) a.weight.row(b, h)[slot] = 0.f;
        if (a.pos.data) a.pos.row(b, h)[slot] = a.next_pos[b] + i;
    }
}

}  // namespace

cudaError_t kv_append_launch(cudaStream_t s, const KvCache& c, const uint16_t* k_new, const long long* k_stride,
                             const uint16_t* v_new, const long long* v_stride, int tokens, const int* starts,
                             KvRows<float> weight, KvRows<int> pos, const int* next_pos) {
    AppendArgs a = {c, k_new, v_new, {k_stride[0], k_stride[1]}, {v_stride[0], v_stride[1]},
                    tokens, starts, weight, pos, next_pos};
    const long long warps = (long long)tokens * c.heads;
    const long long blocks = (warps + 7) / 8;
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
    kv_append_kernel<<<(unsigned)blocks, 256, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace topk
