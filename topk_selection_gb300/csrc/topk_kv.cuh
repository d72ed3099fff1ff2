// Shared by the key-value cache operators' files: the cache as the kernels
// see it, and the launch functions behind the C ABI (include/topk.h holds the
// contract).
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <mutex>

#include "topk_internal.h"

namespace topk {

struct KvCache {
    uint16_t* k;  // 16-bit elements, f16 or bf16 alike where they are only moved
    uint16_t* v;
    long long ks[3], vs[3];  // elements between pages, slots, heads
    const int* table;
    long long table_stride;
    const int* lens;
    int pages, page_size, heads, dim;
    int seqs, width;  // width: table entries of a sequence
    int bf16;

    __host__ __device__ int capacity() const { return width * page_size; }
    // Slots that sequence b holds.
    __device__ int len(int b) const {
        const int n = lens[b];
        return n < 0 ? 0 : n > capacity() ? capacity() : n;
    }
    // Page of sequence b's slot, or -1 when the table names none.
    __device__ int page_of(int b, int slot) const {
        const int p = table[b * table_stride + slot / page_size];
        return (unsigned)p < (unsigned)pages ? p : -1;
    }
};

// Allows a kernel `bytes` of dynamic shared memory on a device; asked once
// per device, of which `done` keeps a bit.
template <typename Kernel>
cudaError_t allow_smem(Kernel kernel, int bytes, int device, std::atomic<unsigned long long>& done) {
    const unsigned long long bit = 1ull << (device & 63);
    if (device < 64 && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

// A per-slot side array, [seqs, heads, slots].
template <typename T>
struct KvRows {
    T* data;
    long long seq, head;
    __device__ T* row(int b, int h) const { return data + b * seq + h * head; }
};

// Counters, in two halves that calls use in turn by their epoch.  A call finds
// its half zero and leaves it zero, and clears the other one, which a call
// before it may have left otherwise if its waits gave up.  A graph's calls
// always have the same half: topk_check_stream clears both when it reports.
constexpr int kKvBlocks = 256;               // of an attend at most
constexpr int kKvTicket = 3 * kKvBlocks;     // an evict's word, behind three of each block of an attend
constexpr int kKvHalf = 3 * kKvBlocks + 32;
constexpr int kKvStatusWords = 32;
constexpr int kKvStateWords = kKvStatusWords + 2 * kKvHalf;
// The whole grid calls it.
__device__ __forceinline__ void clear_half(unsigned* half) {
    for (unsigned i = blockIdx.x * blockDim.x + threadIdx.x; i < kKvHalf; i += gridDim.x * blockDim.x) half[i] = 0;
}

// What a call has of its stream (topk_api.cu).
struct KvState {
    void* scratch;       // no contents to rely on
    unsigned* status;    // sticky; topk_check_stream reads it
    unsigned* mine;      // the call's half of the counters
    unsigned* other;
    // Other host threads' calls on the stream wait until this one has made its
    // launches: they share the scratch, which another's launch between two of
    // one call's would overwrite.
    std::unique_lock<std::mutex> turn;
};
// At least scratch_bytes of it, 256-byte aligned.  Returns a topk_status.
int kv_state(int device, cudaStream_t s, size_t scratch_bytes, KvState* state);
// Test options TOPK_OPT_KV_SPINS and TOPK_OPT_KV_WITHHOLD (topk_api.cu).
int kv_spins_option();
int kv_withhold_option();
// TOPK_OK for device or managed memory, TOPK_ERR_INVALID_ARG for host memory.
int device_pointer(const void* p);
// The current device, and its number of SMs, which is asked for once.
cudaError_t current_device(int* device, int* sms);
// Counts n kernel launches.
void note_launches(int n);

// sms: the device's number of SMs.
cudaError_t kv_append_launch(int sms, cudaStream_t s, const KvCache& c, const uint16_t* k_new,
                             const long long* k_stride, const uint16_t* v_new, const long long* v_stride, int tokens,
                             const int* starts, KvRows<float> weight, KvRows<int> pos, const int* next_pos);

struct KvRotate {
    const uint16_t *q, *k, *v;
    long long qs[2], ks[2], vs[2];  // elements between tokens, heads
    uint16_t *q_out, *k_out;
    long long qos[2], kos[2];
    int tokens, q_heads, heads, dim;
    int half;         // turned pairs of a head
    bool neighbours;  // pairs of elements side by side, not half of the turned ones apart
    const float* freq;
    const uint16_t *q_norm, *k_norm;  // null: no norm
    long long q_norm_stride, k_norm_stride;  // elements between heads, 0 where they share one
    float eps, per_dim;
    const int* pos;  // of each token; null in an append, which has what follows
    const int *starts, *next_pos;
    KvRows<float> weight;
    KvRows<int> pos_rows;
};
// c: the cache of an append, or null.
cudaError_t kv_rotate_launch(int device, int sms, cudaStream_t s, const KvCache* c, const KvRotate& r, bool bf16);

struct KvAttend {
    const uint16_t* q;
    long long qs[2];  // elements between sequences, query heads
    int q_heads;
    float scale;
    uint16_t* out;
    float* lse;
    KvRows<const float> weight;
    KvRows<float> weight_out;
};
size_t kv_attend_scratch(int sms, const KvCache& c, const KvAttend& a);
cudaError_t kv_attend_launch(int device, int sms, cudaStream_t s, const KvCache& c, const KvAttend& a,
                             const KvState& state, int* launches);

struct KvEvict {
    KvRows<const float> weight;
    KvRows<const int> pos;
    const int* next_pos;
    int budget, sink, recent;
    KvRows<float> weight_out;
    KvRows<int> pos_out;
    int* lens_out;
};
size_t kv_evict_scratch(const KvCache& c, const KvEvict& e);
cudaError_t kv_evict_launch(int device, int sms, cudaStream_t s, const KvCache& c, const KvEvict& e,
                            const KvState& state, int* launches);

}  // namespace topk
