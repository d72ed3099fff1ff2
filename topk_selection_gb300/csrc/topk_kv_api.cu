// C ABI of the key-value cache operators: argument checks, scratch and
// dispatch.  The contract is in include/topk.h.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "../../include/topk.h"
#include "topk_internal.h"
#include "topk_kv.cuh"

namespace {

bool misaligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

int cuda_fail(cudaError_t e) {
    topk::note_cuda_error((int)e);
    return TOPK_ERR_CUDA;
}

// Strides of 16-byte granularity, as the kernels' wide loads and tensor maps need.
bool strides_ok(const int64_t* s, int n) {
    for (int i = 0; i < n; ++i)
        if (s[i] <= 0 || (s[i] & 7) || s[i] >= (int64_t(1) << 38)) return false;
    return true;
}

int check_cache(const topk_kv_cache* c, topk::KvCache* out) {
    if (!c || !c->k || !c->v || !c->table || !c->lens) return TOPK_ERR_INVALID_ARG;
    if (c->dtype != TOPK_KV_F16 && c->dtype != TOPK_KV_BF16) return TOPK_ERR_INVALID_ARG;
    if (c->pages < 1 || c->page_size < 1 || c->heads < 1 || c->dim < 1 || c->table_width < 1 || c->seqs < 1 ||
        c->table_stride < c->table_width)
        return TOPK_ERR_INVALID_ARG;
    if (misaligned(c->k, 16) || misaligned(c->v, 16) || misaligned(c->table, 4) || misaligned(c->lens, 4))
        return TOPK_ERR_INVALID_ARG;
    if (!strides_ok(c->k_stride, 3) || !strides_ok(c->v_stride, 3)) return TOPK_ERR_INVALID_ARG;
    if ((c->page_size & 7) || c->page_size > 65536 || (c->dim & 7) || c->dim > TOPK_KV_MAX_DIM ||
        c->seqs > 65535 || c->heads > 4096 || (int64_t)c->table_width * c->page_size >= (int64_t(1) << 30) ||
        (int64_t)c->seqs * c->heads > (1 << 24))
        return TOPK_ERR_UNSUPPORTED;
    topk::KvCache& o = *out;
    o.k = static_cast<uint16_t*>(c->k);
    o.v = static_cast<uint16_t*>(c->v);
    for (int i = 0; i < 3; ++i) {
        o.ks[i] = c->k_stride[i];
        o.vs[i] = c->v_stride[i];
    }
    o.table = c->table;
    o.table_stride = c->table_stride;
    o.lens = c->lens;
    o.pages = c->pages;
    o.page_size = c->page_size;
    o.heads = c->heads;
    o.dim = c->dim;
    o.seqs = c->seqs;
    o.width = c->table_width;
    o.bf16 = c->dtype == TOPK_KV_BF16;
    return TOPK_OK;
}

// Strides of a side array; that of a dimension with one element is no matter.
struct Steps {
    int64_t seq, head;
    Steps(const topk_kv_rows* r, const topk::KvCache& c)
        : seq(c.seqs > 1 ? r->seq_stride : 0), head(c.heads > 1 ? r->head_stride : 0) {}
    bool operator==(const Steps& o) const { return seq == o.seq && head == o.head; }
};

// Whether some row of an array of `slots` slots meets a row of another one,
// `apart` elements behind it, of `others` slots and the same strides; with
// apart == 0, a row of its own other than itself.  Two rows that are ds
// sequences and dh heads apart are apart + ds * seq + dh * head elements apart:
// for each dh, the least ds that takes this above -others decides.
bool rows_meet(const Steps& at, const topk::KvCache& c, int64_t slots, int64_t others, int64_t apart) {
    const int64_t most = at.seq > 0 ? c.seqs - 1 : 0;
    auto meet = [&](int64_t from, int64_t first, int64_t last) {  // some ds in [first, last]
        if (first > last) return false;
        int64_t ds = first;
        if (at.seq > 0 && from + first * at.seq <= -others) ds = first + (-others - from - first * at.seq) / at.seq + 1;
        return ds <= last && from + ds * at.seq > -others && from + ds * at.seq < slots;
    };
    const int heads = at.head > 0 ? c.heads - 1 : 0;
    for (int dh = -heads; dh <= heads; ++dh) {
        const int64_t from = apart + dh * at.head;
        if (apart == 0 && dh == 0) {  // all but itself
            if (meet(from, -most, -1) || meet(from, 1, most)) return true;
        } else if (meet(from, -most, most)) {
            return true;
        }
    }
    return false;
}

// A side array with at least `slots` slots whose rows do not lie in one another.
int check_rows(const topk_kv_rows* r, const topk::KvCache& c, int slots) {
    constexpr int64_t kMost = int64_t(1) << 44;  // elements that addresses have room for
    if (misaligned(r->data, 4) || r->slots < slots) return TOPK_ERR_INVALID_ARG;
    const Steps at(r, c);
    if ((c.heads > 1 && at.head < r->slots) || (c.seqs > 1 && at.seq < r->slots)) return TOPK_ERR_INVALID_ARG;
    if (r->head_stride < 0 || r->seq_stride < 0 || at.seq > kMost || at.head > kMost) return TOPK_ERR_INVALID_ARG;
    const bool nested = c.seqs == 1 || c.heads == 1 || at.seq >= (c.heads - 1) * at.head + r->slots ||
                        at.head >= (c.seqs - 1) * at.seq + r->slots;
    return nested || !rows_meet(at, c, r->slots, r->slots, 0) ? TOPK_OK : TOPK_ERR_INVALID_ARG;
}

template <typename T>
topk::KvRows<T> rows_of(const topk_kv_rows* r) {
    if (!r) return {nullptr, 0, 0};
    return {static_cast<T*>(r->data), r->seq_stride, r->head_stride};
}

bool present(const topk_kv_rows* r) { return r && r->data; }

// The elements that a side array spans.
int64_t span(const topk_kv_rows* r, const topk::KvCache& c) {
    const Steps at(r, c);
    return (c.seqs - 1) * at.seq + (c.heads - 1) * at.head + r->slots;
}

// Whether `out` is the same array as `in`, or overlaps none of it.  Arrays
// with the same strides may have their rows between one another's.
bool same_or_apart(const topk_kv_rows* in, const topk_kv_rows* out, const topk::KvCache& c) {
    const Steps at(in, c);
    const bool alike = at == Steps(out, c);
    if (in->data == out->data) return alike;
    const int64_t apart =
        (int64_t)(reinterpret_cast<uintptr_t>(out->data) - reinterpret_cast<uintptr_t>(in->data)) / 4;
    if (apart >= span(in, c) || -apart >= span(out, c)) return true;
    return alike && !rows_meet(at, c, in->slots, out->slots, apart);
}

int on_device(std::initializer_list<const void*> ps) {
    for (const void* p : ps) {
        if (!p) continue;
        const int rc = topk::device_pointer(p);
        if (rc != TOPK_OK) return rc;
    }
    return TOPK_OK;
}

// The current device, and its number of SMs, which is asked for once.
cudaError_t current_device(int* device, int* sms) {
    static std::atomic<int> counts[64];
    cudaError_t e = cudaGetDevice(device);
    if (e != cudaSuccess) return e;
    std::atomic<int>* known = *device < 64 ? &counts[*device] : nullptr;
    *sms = known ? known->load(std::memory_order_relaxed) : 0;
    if (*sms > 0) return cudaSuccess;
    e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *device);
    if (e == cudaSuccess && known) known->store(*sms, std::memory_order_relaxed);
    return e;
}

}  // namespace

extern "C" {

int topk_kv_append(const struct topk_kv_cache* cache, const void* k_new, const int64_t* k_new_stride,
                   const void* v_new, const int64_t* v_new_stride, int tokens, const int32_t* starts,
                   const struct topk_kv_rows* weight, const struct topk_kv_rows* pos, const int32_t* next_pos,
                   struct CUstream_st* stream) {
    topk::KvCache c;
    int rc = check_cache(cache, &c);
    if (rc != TOPK_OK) return rc;
    if (tokens < 0 || !k_new_stride || !v_new_stride || (!starts && tokens != c.seqs)) return TOPK_ERR_INVALID_ARG;
    if (present(pos) != (next_pos != nullptr)) return TOPK_ERR_INVALID_ARG;
    if (present(weight) && (rc = check_rows(weight, c, c.capacity())) != TOPK_OK) return rc;
    if (present(pos) && (rc = check_rows(pos, c, c.capacity())) != TOPK_OK) return rc;
    if (tokens == 0) return TOPK_OK;
    if (!k_new || !v_new || misaligned(k_new, 16) || misaligned(v_new, 16) || misaligned(starts, 4) ||
        misaligned(next_pos, 4) || !strides_ok(k_new_stride, 2) || !strides_ok(v_new_stride, 2))
        return TOPK_ERR_INVALID_ARG;
    rc = on_device({c.k, c.v, c.table, c.lens, k_new, v_new, starts, present(weight) ? weight->data : nullptr,
                    present(pos) ? pos->data : nullptr, next_pos});
    if (rc != TOPK_OK) return rc;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    int device = 0, sms = 0;
    cudaError_t e = current_device(&device, &sms);
    if (e != cudaSuccess) return cuda_fail(e);
    const long long ks[2] = {k_new_stride[0], k_new_stride[1]}, vs[2] = {v_new_stride[0], v_new_stride[1]};
    e = topk::kv_append_launch(sms, s, c, static_cast<const uint16_t*>(k_new), ks,
                               static_cast<const uint16_t*>(v_new), vs, tokens, starts, rows_of<float>(weight),
                               rows_of<int>(pos), next_pos);
    topk::note_unreleased_launch(device, s);  // behind the launch: another thread's may have come between
    if (e != cudaSuccess) return cuda_fail(e);
    topk::note_launch();
    return TOPK_OK;
}

int topk_kv_attend(const struct topk_kv_cache* cache, const void* q, const int64_t* q_stride, int q_heads, float scale,
                   void* out, float* lse, const struct topk_kv_rows* weight, const struct topk_kv_rows* weight_out,
                   struct CUstream_st* stream) {
    topk::KvCache c;
    int rc = check_cache(cache, &c);
    if (rc != TOPK_OK) return rc;
    if (!q || !q_stride || !out || q_heads < 1 || q_heads % c.heads || !std::isfinite(scale) || misaligned(q, 16) ||
        misaligned(out, 16) || misaligned(lse, 4) || !strides_ok(q_stride, 2))
        return TOPK_ERR_INVALID_ARG;
    if (present(weight) != present(weight_out)) return TOPK_ERR_INVALID_ARG;
    if (present(weight)) {
        if ((rc = check_rows(weight, c, c.capacity())) != TOPK_OK) return rc;
        if ((rc = check_rows(weight_out, c, c.capacity())) != TOPK_OK) return rc;
        if (!same_or_apart(weight, weight_out, c)) return TOPK_ERR_INVALID_ARG;
    }
    // Tiles of 128 slots are numbered in 32 bits.
    if ((int64_t)c.seqs * q_heads * ((c.capacity() + 127) / 128) > INT32_MAX) return TOPK_ERR_UNSUPPORTED;
    if ((int64_t)c.seqs * q_heads > (1 << 24)) return TOPK_ERR_UNSUPPORTED;
    rc = on_device({c.k, c.v, c.table, c.lens, q, out, lse, present(weight) ? weight->data : nullptr,
                    present(weight_out) ? weight_out->data : nullptr});
    if (rc != TOPK_OK) return rc;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    int device = 0, sms = 0;
    cudaError_t e = current_device(&device, &sms);
    if (e != cudaSuccess) return cuda_fail(e);
    topk::KvAttend a = {};
    a.q = static_cast<const uint16_t*>(q);
    a.qs[0] = q_stride[0];
    a.qs[1] = q_stride[1];
    a.q_heads = q_heads;
    a.scale = scale;
    a.out = static_cast<uint16_t*>(out);
    a.lse = lse;
    a.weight = rows_of<const float>(weight);
    a.weight_out = rows_of<float>(weight_out);
    topk::KvState state;
    rc = topk::kv_state(device, s, topk::kv_attend_scratch(sms, c, a), &state);
    if (rc != TOPK_OK) return rc;
    int launches = 0;
    e = topk::kv_attend_launch(device, sms, s, c, a, state, &launches);
    topk::note_unreleased_launch(device, s);
    topk::note_launches(launches);
    return e == cudaSuccess ? TOPK_OK : cuda_fail(e);
}

int topk_kv_evict(const struct topk_kv_cache* cache, const struct topk_kv_rows* weight,
                  const struct topk_kv_rows* pos, const int32_t* next_pos, int budget, int sink, int recent,
                  const struct topk_kv_rows* weight_out, const struct topk_kv_rows* pos_out, int32_t* lens_out,
                  struct CUstream_st* stream) {
    topk::KvCache c;
    int rc = check_cache(cache, &c);
    if (rc != TOPK_OK) return rc;
    if (!present(weight) || !present(pos) || !next_pos || !present(weight_out) || !present(pos_out) || !lens_out)
        return TOPK_ERR_INVALID_ARG;
    if (budget < 1 || sink < 0 || recent < 0 || (int64_t)sink + recent > budget || misaligned(next_pos, 4) ||
        misaligned(lens_out, 4))
        return TOPK_ERR_INVALID_ARG;
    const int keep = budget < c.capacity() ? budget : c.capacity();
    if ((rc = check_rows(weight, c, c.capacity())) != TOPK_OK || (rc = check_rows(pos, c, c.capacity())) != TOPK_OK ||
        (rc = check_rows(weight_out, c, keep)) != TOPK_OK || (rc = check_rows(pos_out, c, keep)) != TOPK_OK)
        return rc;
    if (!same_or_apart(weight, weight_out, c) || !same_or_apart(pos, pos_out, c)) return TOPK_ERR_INVALID_ARG;
    if (lens_out != c.lens && lens_out < c.lens + c.seqs && c.lens < lens_out + c.seqs) return TOPK_ERR_INVALID_ARG;
    rc = on_device({c.k, c.v, c.table, c.lens, weight->data, pos->data, next_pos, weight_out->data, pos_out->data,
                    lens_out});
    if (rc != TOPK_OK) return rc;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    int device = 0, sms = 0;
    cudaError_t err = current_device(&device, &sms);
    if (err != cudaSuccess) return cuda_fail(err);
    topk::KvEvict e = {};
    e.weight = rows_of<const float>(weight);
    e.pos = rows_of<const int>(pos);
    e.next_pos = next_pos;
    e.budget = budget;
    e.sink = sink;
    e.recent = recent;
    e.weight_out = rows_of<float>(weight_out);
    e.pos_out = rows_of<int>(pos_out);
    e.lens_out = lens_out;
    topk::KvState state;
    rc = topk::kv_state(device, s, topk::kv_evict_scratch(c, e), &state);
    if (rc != TOPK_OK) return rc;
    int launches = 0;
    err = topk::kv_evict_launch(device, sms, s, c, e, state, &launches);
    topk::note_unreleased_launch(device, s);
    topk::note_launches(launches);
    return err == cudaSuccess ? TOPK_OK : cuda_fail(err);
}

}  // extern "C"
