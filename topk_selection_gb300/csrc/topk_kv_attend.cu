// topk_kv_attend: attention of one new token over a paged cache.
//
// The plainest form: one block per (sequence, query head) writes its scores
// to scratch, reduces them and adds up its output; a second launch adds the
// heads' shares to the slots' weights.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "topk_device.cuh"
#include "topk_kv.cuh"

namespace topk {
namespace {

__device__ __forceinline__ float to_float(uint16_t x, int bf16) {
    return bf16 ? __uint_as_float((unsigned)x << 16) : __half2float(__ushort_as_half(x));
}
__device__ __forceinline__ uint16_t from_float(float x, int bf16) {
    return bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(x)) : __half_as_ushort(__float2half_rn(x));
}

struct AttendArgs {
    KvCache c;
    KvAttend a;
    float* score;  // [seqs * q_heads][capacity]
    float* stats;  // [seqs * q_heads][2]: largest score, sum
};

__device__ float block_reduce(float x, bool max, float* sh) {
    for (int d = 16; d; d >>= 1) {
        const float y = __shfl_xor_sync(kFullMask, x, d);
        x = max ? fmaxf(x, y) : x + y;
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = x;
    __syncthreads();
    x = sh[0];
    for (int w = 1; w < 8; ++w) x = max ? fmaxf(x, sh[w]) : x + sh[w];
    return x;
}

__global__ void __launch_bounds__(256) kv_attend_kernel(const AttendArgs p) {
    __shared__ float qs[256], red[8];
    const int row = blockIdx.x, b = row / p.a.q_heads, j = row % p.a.q_heads;
    const int h = j / (p.a.q_heads / p.c.heads);
    const int n = p.c.len(b), dim = p.c.dim, tid = threadIdx.x, lane = tid & 31;
    float* sc = p.score + (size_t)row * p.c.capacity();
    if (tid < dim) qs[tid] = to_float(p.a.q[b * p.a.qs[0] + j * p.a.qs[1] + tid], p.c.bf16);
    __syncthreads();
    float top = -INFINITY;
    for (int t = tid >> 5; t < n; t += 8) {
        const int page = p.c.page_of(b, t);
        float s = 0.f;
        if (page >= 0) {
            const uint16_t* k = p.c.k + page * p.c.ks[0] + (t % p.c.page_size) * p.c.ks[1] + h * p.c.ks[2];
            for (int x = lane; x < dim; x += 32) s += qs[x] * to_float(k[x], p.c.bf16);
        }
        for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(kFullMask, s, d);
        s *= p.a.scale;
        if (lane == 0) sc[t] = s;
        top = fmaxf(top, s);
    }
    top = block_reduce(top, true, red);
    const float ref = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
    for (int t = tid; t < n; t += 256) {
        const float e = expf(sc[t] - ref);
        sc[t] = e;
        sum += e;
    }
    sum = block_reduce(sum, false, red);
    __syncthreads();
    if (tid < dim) {
        float o = 0.f;
        for (int t = 0; t < n; ++t) {
            const int page = p.c.page_of(b, t);
            if (page < 0) continue;
            o += sc[t] * to_float(p.c.v[page * p.c.vs[0] + (t % p.c.page_size) * p.c.vs[1] + h * p.c.vs[2] + tid],
                                  p.c.bf16);
        }
        p.a.out[(size_t)row * dim + tid] = from_float(sum == 0.f ? 0.f : o / sum, p.c.bf16);
    }
    if (tid == 0) {
        p.stats[row] = sum;
        if (p.a.lse) p.a.lse[row] = sum == 0.f ? -INFINITY : ref + logf(sum);
    }
}

__global__ void __launch_bounds__(256) kv_weight_kernel(const AttendArgs p) {
    const int row = blockIdx.x, b = row / p.c.heads, h = row % p.c.heads, group = p.a.q_heads / p.c.heads;
    const int n = p.c.len(b);
    const float* w = p.a.weight.row(b, h);
    float* wo = p.a.weight_out.row(b, h);
    for (int t = threadIdx.x; t < n; t += 256) {
        float share = 0.f;
        for (int g = 0; g < group; ++g) {
            const int r = b * p.a.q_heads + h * group + g;
            const float sum = p.stats[r];
            if (sum != 0.f) share += p.score[(size_t)r * p.c.capacity() + t] / sum;
        }
        wo[t] = w[t] + share;
    }
}

}  // namespace

size_t kv_attend_scratch(int, const KvCache& c, const KvAttend& a) {
    return 4 * (size_t)c.seqs * a.q_heads * (c.capacity() + 1);
}

cudaError_t kv_attend_launch(int, cudaStream_t s, const KvCache& c, const KvAttend& a, void* scratch, unsigned*,
                             int* launches) {
    AttendArgs p = {c, a};
    p.stats = static_cast<float*>(scratch);
    p.score = p.stats + (size_t)c.seqs * a.q_heads;
    kv_attend_kernel<<<c.seqs * a.q_heads, 256, 0, s>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    ++*launches;
    if (!a.weight.data) return e;
    kv_weight_kernel<<<c.seqs * c.heads, 256, 0, s>>>(p);
    e = cudaGetLastError();
    if (e == cudaSuccess) ++*launches;
    return e;
}

}  // namespace topk
