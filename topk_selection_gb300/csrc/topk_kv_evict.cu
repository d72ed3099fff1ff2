// topk_kv_evict: keep the `budget` best slots of each (sequence, head).
//
// Two launches.  The first selects: a radix select over 32-bit keys (8-bit
// digits) finds the budget-th key, and a pass in slot order lists the holes
// below the budget and the kept slots above it.  The second moves the kept
// slots into the holes.  Sources lie at or above the budget and targets below
// it, so the moves cannot collide and need no order.
#include "topk_device.cuh"
#include "topk_kv.cuh"

namespace topk {
namespace {

constexpr int kSelThreads = 512;

struct EvictArgs {
    KvCache c;
    KvEvict e;
    int* lens;    // [seqs] lengths before, clamped
    int* moves;   // [seqs * heads] number of moves
    int* holes;   // [seqs * heads][room]
    int* movers;  // [seqs * heads][room]
    int room;     // moves a row's lists have room for
    int chunks;   // blocks of the second launch per row
};

// Order-preserving key: protected above NaN above every number, -0 equal to +0.
__device__ __forceinline__ unsigned evict_key(const EvictArgs& a, float w, int pos, int next_pos) {
    if (pos < a.e.sink || (long long)pos >= (long long)next_pos - a.e.recent) return 0xFFFFFFFFu;
    if (w != w) return 0xFFFFFFFEu;
    const unsigned u = __float_as_uint(w + 0.0f);
    return (u >> 31) ? ~u : u | 0x80000000u;
}

// Exclusive prefix of v over the block's threads, and the total in *total.
__device__ int block_scan(int v, int* warp_sums, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(kFullMask, x, d);
        if (lane >= d) x += y;
    }
    __syncthreads();
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < kSelThreads / 32; ++w) {
        if (w < warp) before += warp_sums[w];
        all += warp_sums[w];
    }
    *total = all;
    return before + x - v;
}

__global__ void __launch_bounds__(kSelThreads) kv_select_kernel(const EvictArgs a) {
    __shared__ int hist[256];
    __shared__ int warp_sums[kSelThreads / 32];
    __shared__ unsigned s_prefix;
    __shared__ int s_need;
    const int row = blockIdx.x, b = row / a.c.heads, h = row % a.c.heads;
    const int n = a.c.len(b), next_pos = a.e.next_pos[b], budget = a.e.budget;
    const float* w = a.e.weight.row(b, h);
    const int* pos = a.e.pos.row(b, h);
    float* wo = a.e.weight_out.row(b, h);
    int* po = a.e.pos_out.row(b, h);
    const int tid = threadIdx.x;
    if (tid == 0 && h == 0) a.lens[b] = n;
    if (n <= budget) {
        for (int i = tid; i < n; i += kSelThreads) {
            wo[i] = w[i];
            po[i] = pos[i];
        }
        if (tid == 0) a.moves[row] = 0;
        return;
    }
    if (tid == 0) {
        s_prefix = 0;
        s_need = budget;
    }
    __syncthreads();
    for (int shift = 24; shift >= 0; shift -= 8) {
        const unsigned prefix = s_prefix;
        const int need = s_need;
        for (int i = tid; i < 256; i += kSelThreads) hist[i] = 0;
        __syncthreads();
        for (int i = tid; i < n; i += kSelThreads) {
            const unsigned key = evict_key(a, w[i], pos[i], next_pos);
            if (shift == 24 || (key >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(key >> shift) & 255], 1);
        }
        __syncthreads();
        if (tid == 0) {
            int left = need, d = 255;
            while (d > 0 && hist[d] < left) left -= hist[d--];
            s_prefix = prefix | ((unsigned)d << shift);
            s_need = left;
        }
        __syncthreads();
    }
    const unsigned edge = s_prefix;
    const int ties = s_need;  // keys equal to `edge` to keep, lowest slots first
    int tie_base = 0, hole_base = 0, mover_base = 0;
    int* holes = a.holes + (size_t)row * a.room;
    int* movers = a.movers + (size_t)row * a.room;
    for (int base = 0; base < n; base += kSelThreads) {
        const int i = base + tid;
        const unsigned key = i < n ? evict_key(a, w[i], pos[i], next_pos) : 0;
        const bool tie = i < n && key == edge;
        int total;
        const int rank = tie_base + block_scan(tie, warp_sums, &total);
        tie_base += total;
        const bool kept = i < n && (key > edge || (tie && rank < ties));
        const bool hole = i < n && i < budget && !kept, mover = kept && i >= budget;
        if (kept && i < budget) {
            wo[i] = w[i];
            po[i] = pos[i];
        }
        const int hr = hole_base + block_scan(hole, warp_sums, &total);
        hole_base += total;
        if (hole) holes[hr] = i;
        const int mr = mover_base + block_scan(mover, warp_sums, &total);
        mover_base += total;
        if (mover) movers[mr] = i;
    }
    if (tid == 0) a.moves[row] = mover_base;
}

__global__ void __launch_bounds__(256) kv_move_kernel(const EvictArgs a) {
    const int row = blockIdx.x / a.chunks, chunk = blockIdx.x % a.chunks, b = row / a.c.heads, h = row % a.c.heads;
    const int lane = threadIdx.x & 31;
    if (chunk == 0 && h == 0 && threadIdx.x == 0) {
        const int n = a.lens[b];
        a.e.lens_out[b] = n < a.e.budget ? n : a.e.budget;
    }
    const int moves = a.moves[row];
    for (int j = chunk * 8 + (threadIdx.x >> 5); j < moves; j += a.chunks * 8) {
        const int to = a.holes[(size_t)row * a.room + j], from = a.movers[(size_t)row * a.room + j];
        if (lane == 0) {
            a.e.weight_out.row(b, h)[to] = a.e.weight.row(b, h)[from];
            a.e.pos_out.row(b, h)[to] = a.e.pos.row(b, h)[from];
        }
        const int dp = a.c.page_of(b, to), sp = a.c.page_of(b, from);
        if (dp < 0 || sp < 0) continue;
        const int ds = to % a.c.page_size, ss = from % a.c.page_size;
        const bool v = lane >= 16;
        uint16_t* pool = v ? a.c.v : a.c.k;
        const long long* st = v ? a.c.vs : a.c.ks;
        uint16_t* dst = pool + dp * st[0] + ds * st[1] + h * st[2];
        const uint16_t* src = pool + sp * st[0] + ss * st[1] + h * st[2];
        for (int x = (lane & 15) * 8; x < a.c.dim; x += 128)
            *reinterpret_cast<int4*>(dst + x) = *reinterpret_cast<const int4*>(src + x);
    }
}

int room_of(const KvCache& c, const KvEvict& e) {
    const int above = c.capacity() - e.budget;
    return above < 1 ? 1 : above < e.budget ? above : e.budget;
}

}  // namespace

size_t kv_evict_scratch(const KvCache& c, const KvEvict& e) {
    const size_t rows = (size_t)c.seqs * c.heads;
    return 4 * (c.seqs + rows + 2 * rows * room_of(c, e));
}

cudaError_t kv_evict_launch(int, cudaStream_t s, const KvCache& c, const KvEvict& e, void* scratch, unsigned*,
                            int* launches) {
    const int rows = c.seqs * c.heads;
    EvictArgs a = {c, e};
    a.room = room_of(c, e);
    a.lens = static_cast<int*>(scratch);
    a.moves = a.lens + c.seqs;
    a.holes = a.moves + rows;
    a.movers = a.holes + (size_t)rows * a.room;
    kv_select_kernel<<<rows, kSelThreads, 0, s>>>(a);
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    ++*launches;
    a.chunks = (a.room + 63) / 64;
    const long long most = (1 << 20) / rows + 1;
    if (a.chunks > most) a.chunks = (int)most;
    kv_move_kernel<<<rows * a.chunks, 256, 0, s>>>(a);
    err = cudaGetLastError();
    if (err == cudaSuccess) ++*launches;
    return err;
}

}  // namespace topk
