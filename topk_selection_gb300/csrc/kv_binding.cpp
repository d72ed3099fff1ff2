// Python binding of a decoding step's operators (the key-value cache's and
// the sampling of rows): checks of tensors and marshalling into the C ABI's
// structures (include/topk.h), nothing else.
//
// A decoder calls these operators several times per token and layer, and a
// small call takes the GPU a few microseconds.  Reading the shapes, strides
// and addresses of ten tensors takes longer than that in Python (measured: 9
// to 15 us a call), so it is done here.  The library itself stays free of
// torch: it is loaded by ctypes, which hands over its functions' addresses.
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/AutogradState.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/function.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/autograd/functions/utils.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <exception>
#include <initializer_list>
#include <optional>
#include <sstream>

#include "../../include/topk.h"

namespace {

decltype(&topk_kv_append) g_append = nullptr;
decltype(&topk_kv_attend) g_attend = nullptr;
decltype(&topk_kv_evict) g_evict = nullptr;
decltype(&topk_kv_rotate) g_rotate = nullptr;
decltype(&topk_kv_append_rotated) g_append_rotated = nullptr;
decltype(&topk_sample_rows) g_sample = nullptr;

// A Python exception that is already set, on its way out.
struct Raised {};

[[noreturn]] void raise(PyObject* type, const std::string& what) {
    PyErr_SetString(type, what.c_str());
    throw Raised();
}

std::string text(c10::IntArrayRef sizes) {
    std::ostringstream s;
    s << "(";
    for (size_t i = 0; i < sizes.size(); ++i) {
        if (sizes[i] < 0) s << "*"; else s << sizes[i];
        if (i + 1 < sizes.size()) s << ", ";
    }
    s << (sizes.size() == 1 ? ",)" : ")");
    return s.str();
}

// The tensor behind `o`, of this type, device and shape (-1: any size).
const at::Tensor& tensor(PyObject* o, const char* name, at::ScalarType type, c10::Device device,
                         std::initializer_list<int64_t> want) {
    if (!THPVariable_Check(o)) raise(PyExc_TypeError, std::string(name) + " must be a torch.Tensor");
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.scalar_type() != type)
        raise(PyExc_TypeError, std::string(name) + " must be " + c10::toString(type) + ", got " +
                                   c10::toString(t.scalar_type()));
    if (t.device() != device)
        raise(PyExc_ValueError, std::string(name) + " must be on " + device.str() + ", got " + t.device().str());
    const c10::IntArrayRef have = t.sizes();
    bool fits = have.size() == want.size();
    for (size_t i = 0; fits && i < have.size(); ++i) fits = want.begin()[i] < 0 || want.begin()[i] == have[i];
    if (!fits)
        raise(PyExc_ValueError, std::string(name) + " must have shape " +
                                    text(c10::IntArrayRef(want.begin(), want.size())) + ", got " + text(have));
    return t;
}

// All strides but the last, which has to be 1.  A dimension of one element
// may have any stride in torch: the library gets one that it accepts, which
// nothing is multiplied by.
void strides(const at::Tensor& t, const char* name, int64_t* to) {
    const int last = (int)t.dim() - 1;
    if (t.size(last) > 1 && t.stride(last) != 1)
        raise(PyExc_ValueError, std::string(name) + " must be contiguous in its last dimension");
    for (int i = 0; i < last; ++i) to[i] = t.size(i) == 1 ? 8 : t.stride(i);
}

struct Cache {
    topk_kv_cache c;
    at::ScalarType type;
    c10::Device device{c10::kCPU};
};

const int32_t* ints(PyObject* o, const char* name, const Cache& c, int64_t n) {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o, name, at::kInt, c.device, {n});
    if (!t.is_contiguous()) raise(PyExc_ValueError, std::string(name) + " must be contiguous");
    return static_cast<const int32_t*>(t.const_data_ptr());
}

Cache cache(PyObject* k_pages, PyObject* v_pages, PyObject* table, PyObject* lens) {
    Cache r;
    if (!THPVariable_Check(k_pages)) raise(PyExc_TypeError, "k_pages must be a torch.Tensor");
    const at::Tensor& k0 = THPVariable_Unpack(k_pages);
    r.type = k0.scalar_type();
    r.device = k0.device();
    if (r.type != at::kHalf && r.type != at::kBFloat16)
        raise(PyExc_TypeError, "k_pages must be a float16 or bfloat16 tensor");
    if (!r.device.is_cuda()) raise(PyExc_ValueError, "k_pages must be a CUDA tensor");
    const at::Tensor& k = tensor(k_pages, "k_pages", r.type, r.device, {-1, -1, -1, -1});
    const at::Tensor& v = tensor(v_pages, "v_pages", r.type, r.device, {k.size(0), k.size(1), k.size(2), k.size(3)});
    const at::Tensor& t = tensor(table, "table", at::kInt, r.device, {-1, -1});
    if (t.size(1) > 1 && t.stride(1) != 1) raise(PyExc_ValueError, "the rows of table must be contiguous");
    for (const int64_t n : {k.size(0), k.size(1), k.size(2), k.size(3), t.size(0), t.size(1)})
        if (n > INT32_MAX) raise(PyExc_ValueError, "the cache is too large");
    topk_kv_cache& c = r.c;
    c.k = k.data_ptr();
    c.v = v.data_ptr();
    c.dtype = r.type == at::kBFloat16 ? TOPK_KV_BF16 : TOPK_KV_F16;
    c.pages = (int)k.size(0);
    c.page_size = (int)k.size(1);
    c.heads = (int)k.size(2);
    c.dim = (int)k.size(3);
    strides(k, "k_pages", c.k_stride);
    strides(v, "v_pages", c.v_stride);
    c.table = static_cast<const int32_t*>(t.const_data_ptr());
    c.seqs = (int)t.size(0);
    c.table_width = (int)t.size(1);
    c.table_stride = c.seqs > 1 ? t.stride(0) : c.table_width;
    c.lens = ints(lens, "lens", r, c.seqs);
    if (lens == Py_None) raise(PyExc_TypeError, "lens must be a torch.Tensor");
    return r;
}

// A side array [seqs, heads, slots]; None is absent.
topk_kv_rows rows(PyObject* o, const char* name, at::ScalarType type, const Cache& c) {
    if (o == Py_None) return {nullptr, 0, 0, 0};
    const at::Tensor& t = tensor(o, name, type, c.device, {c.c.seqs, c.c.heads, -1});
    if (t.size(2) > 1 && t.stride(2) != 1)
        raise(PyExc_ValueError, std::string(name) + " must be contiguous in its last dimension");
    return {t.data_ptr(), t.stride(0), t.stride(1), (int)std::min<int64_t>(t.size(2), INT32_MAX)};
}

int integer(PyObject* o) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised();
    return v > INT32_MAX ? INT32_MAX : v < INT32_MIN ? INT32_MIN : (int)v;
}

// The stream of a call: a handle, or None for the current one.  It is the
// current one while this lives, so that memory is allocated for the stream
// that uses it.
struct Stream {
    CUstream_st* handle;
    std::optional<c10::cuda::CUDAStreamGuard> on;

    Stream(PyObject* o, const Cache& c) : Stream(o, c.device.index()) {}
    Stream(PyObject* o, c10::DeviceIndex device) {
        if (o == Py_None) {
            handle = c10::cuda::getCurrentCUDAStream(device).stream();
            return;
        }
        handle = static_cast<CUstream_st*>(PyLong_AsVoidPtr(o));
        if (!handle && PyErr_Occurred()) throw Raised();
        // torch counts the legacy stream, by either of its handles, as its default one.
        const bool legacy = !handle || handle == cudaStreamLegacy;
        on.emplace(legacy ? c10::cuda::getDefaultCUDAStream(device)
                          : c10::cuda::getStreamFromExternal(handle, device));
    }
};

// Whether autograd follows one of these (tensors or None, looked at before).
// The operators have no backward pass.
bool followed(std::initializer_list<PyObject*> tensors) {
    if (!c10::GradMode::is_enabled()) return false;
    for (PyObject* o : tensors)
        if (o != Py_None && THPVariable_Unpack(o).requires_grad()) return true;
    return false;
}

// Refuses to write what autograd follows, as torch's own operators do.
void check_written(const char* name, std::initializer_list<PyObject*> tensors) {
    if (followed(tensors))
        raise(PyExc_RuntimeError, std::string(name) +
                                      " has no gradient, and a tensor that it writes requires grad: call it under "
                                      "torch.no_grad(), or detach() the tensor");
}

// Counts a change of tensors that a call has written, by which autograd knows
// that what it saved of them is stale.
void written(std::initializer_list<PyObject*> tensors) {
    for (PyObject* o : tensors) {
        if (o == Py_None) continue;
        const at::Tensor& t = THPVariable_Unpack(o);
        if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
    }
}

// Runs f with every exception turned into a Python one, after a check of the
// number of arguments.
template <typename F>
PyObject* guarded(Py_ssize_t have, Py_ssize_t want, F f) {
    try {
        if (have != want) raise(PyExc_TypeError, "wrong number of arguments");
        return f();
    } catch (const Raised&) {
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

template <typename F>
int call(c10::Device device, F f) {
    const c10::cuda::CUDAGuard on(device);
    int rc = 0;
    Py_BEGIN_ALLOW_THREADS
    rc = f();
    Py_END_ALLOW_THREADS
    return rc;
}

template <typename F>
int call(const Cache& c, F f) {
    return call(c.device, f);
}

// (k_pages, v_pages, table, lens, k_new, v_new, starts, weight, pos, next_pos, stream) -> status
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 11, [&]() -> PyObject* {
        const Cache c = cache(a[0], a[1], a[2], a[3]);
        const at::Tensor& k = tensor(a[4], "k_new", c.type, c.device, {-1, c.c.heads, c.c.dim});
        const at::Tensor& v = tensor(a[5], "v_new", c.type, c.device, {k.size(0), c.c.heads, c.c.dim});
        if ((a[8] == Py_None) != (a[9] == Py_None)) raise(PyExc_ValueError, "pos and next_pos come together");
        if (k.size(0) > INT32_MAX) raise(PyExc_ValueError, "too many tokens");
        int64_t ks[2], vs[2];
        strides(k, "k_new", ks);
        strides(v, "v_new", vs);
        const int32_t* starts = ints(a[6], "starts", c, (int64_t)c.c.seqs + 1);
        const topk_kv_rows weight = rows(a[7], "weight", at::kFloat, c), pos = rows(a[8], "pos", at::kInt, c);
        const int32_t* next_pos = ints(a[9], "next_pos", c, c.c.seqs);
        const Stream s(a[10], c);
        check_written("kv_append", {a[0], a[1], a[7]});
        if (followed({a[4], a[5]}) &&
            PyErr_WarnEx(PyExc_UserWarning, "kv_append has no gradient: none will reach k_new and v_new", 2) != 0)
            throw Raised();
        if (k.size(0) == 0) return PyLong_FromLong(TOPK_OK);
        const int rc = call(c, [&] {
            return g_append(&c.c, k.const_data_ptr(), ks, v.const_data_ptr(), vs, (int)k.size(0), starts, &weight,
                            &pos, next_pos, s.handle);
        });
        if (rc == TOPK_OK) written({a[0], a[1], a[7], a[8]});
        return PyLong_FromLong(rc);
    });
}

// (q, k_pages, v_pages, table, lens, scale, weight, weight_out, out, lse, stream) -> (out, lse), or a status
PyObject* attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 11, [&]() -> PyObject* {
        const Cache c = cache(a[1], a[2], a[3], a[4]);
        const at::Tensor& q = tensor(a[0], "q", c.type, c.device, {c.c.seqs, -1, c.c.dim});
        const int64_t q_heads = q.size(1);
        if (q_heads > INT32_MAX) raise(PyExc_ValueError, "too many query heads");
        int64_t qs[2];
        strides(q, "q", qs);
        double scale = 1.0 / std::sqrt((double)c.c.dim);
        if (a[5] != Py_None) {
            scale = PyFloat_AsDouble(a[5]);
            if (scale == -1.0 && PyErr_Occurred()) throw Raised();
        }
        if (a[6] == Py_None && a[7] != Py_None) raise(PyExc_ValueError, "weight_out needs weight");
        const topk_kv_rows weight = rows(a[6], "weight", at::kFloat, c);
        const topk_kv_rows weight_out = a[7] == Py_None ? weight : rows(a[7], "weight_out", at::kFloat, c);
        const Stream s(a[10], c);
        const at::Tensor out = a[8] != Py_None
                                   ? tensor(a[8], "out", c.type, c.device, {c.c.seqs, q_heads, c.c.dim})
                                   : at::Tensor(at::detail::empty_cuda({c.c.seqs, q_heads, c.c.dim}, c.type, c.device,
                                                                       std::nullopt));
        const at::Tensor lse = a[9] != Py_None ? tensor(a[9], "lse", at::kFloat, c.device, {c.c.seqs, q_heads})
                                               : at::Tensor(at::detail::empty_cuda({c.c.seqs, q_heads}, at::kFloat,
                                                                                   c.device, std::nullopt));
        if (!out.is_contiguous() || !lse.is_contiguous())
            raise(PyExc_ValueError, "out and lse must be contiguous");
        check_written("kv_attend", {a[6], a[7], a[8], a[9]});
        const bool follow = followed({a[0], a[1], a[2]});
        if (follow && (a[8] != Py_None || a[9] != Py_None))
            raise(PyExc_RuntimeError, "kv_attend has no gradient, and q or the pools require grad: out and lse cannot be "
                                      "given then");
        const int rc = c.c.seqs == 0 ? (int)TOPK_OK : call(c, [&] {  // an empty batch: nothing to do
            return g_attend(&c.c, q.const_data_ptr(), qs, (int)q_heads, (float)scale, out.data_ptr(),
                            static_cast<float*>(lse.data_ptr()), &weight, &weight_out, s.handle);
        });
        if (rc != TOPK_OK) return PyLong_FromLong(rc);
        written({a[7] == Py_None ? a[6] : a[7], a[8], a[9]});
        if (follow) {  // a backward pass that comes here says that there is none
            std::shared_ptr<torch::autograd::Node> node(new torch::autograd::NotImplemented("kv_attend"),
                                                        torch::autograd::deleteNode);
            node->set_next_edges(torch::autograd::collect_next_edges(q, THPVariable_Unpack(a[1]),
                                                                     THPVariable_Unpack(a[2])));
            torch::autograd::set_history(out, node);
            torch::autograd::set_history(lse, node);
        }
        PyObject* pair = PyTuple_New(2);
        if (!pair) throw Raised();
        PyTuple_SET_ITEM(pair, 0, THPVariable_Wrap(out));
        PyTuple_SET_ITEM(pair, 1, THPVariable_Wrap(lse));
        return pair;
    });
}

// (k_pages, v_pages, table, lens, weight, pos, next_pos, budget, sink, recent, weight_out, pos_out, lens_out,
// stream) -> status
PyObject* evict(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 14, [&]() -> PyObject* {
        const Cache c = cache(a[0], a[1], a[2], a[3]);
        const topk_kv_rows weight = rows(a[4], "weight", at::kFloat, c), pos = rows(a[5], "pos", at::kInt, c);
        const int32_t* next_pos = ints(a[6], "next_pos", c, c.c.seqs);
        const int budget = integer(a[7]), sink = integer(a[8]), recent = integer(a[9]);
        const topk_kv_rows weight_out = rows(a[10], "weight_out", at::kFloat, c),
                           pos_out = rows(a[11], "pos_out", at::kInt, c);
        int32_t* lens_out = const_cast<int32_t*>(ints(a[12], "lens_out", c, c.c.seqs));
        const Stream s(a[13], c);
        check_written("kv_evict", {a[0], a[1], a[10]});
        const int rc = c.c.seqs == 0 ? (int)TOPK_OK : call(c, [&] {
            return g_evict(&c.c, &weight, &pos, next_pos, budget, sink, recent, &weight_out, &pos_out, lens_out,
                           s.handle);
        });
        if (rc == TOPK_OK) written({a[0], a[1], a[10], a[11], a[12]});
        return PyLong_FromLong(rc);
    });
}

double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised();
    return v;
}

// What the two operators that rotate have in common, of `dim` elements a head.
struct Rotation {
    topk_kv_rotation r = {};

    // A norm's weights, one row for all heads or one for each.
    const void* norm(PyObject* o, const char* name, at::ScalarType type, c10::Device device, int64_t heads, int64_t dim,
                     int64_t* stride) {
        *stride = 0;
        if (o == Py_None) return nullptr;
        if (!THPVariable_Check(o)) raise(PyExc_TypeError, std::string(name) + " must be a torch.Tensor");
        const bool shared = THPVariable_Unpack(o).dim() == 1;
        const at::Tensor& t = shared ? tensor(o, name, type, device, {dim}) : tensor(o, name, type, device, {heads, dim});
        int64_t apart[2] = {0, 0};
        strides(t, name, apart);
        if (!shared) *stride = t.size(0) == 1 ? 0 : apart[0];
        return t.const_data_ptr();
    }

    Rotation(PyObject* freq, PyObject* q_norm, PyObject* k_norm, PyObject* eps, PyObject* pairing, at::ScalarType type,
             c10::Device device, int64_t q_heads, int64_t heads, int64_t dim) {
        const at::Tensor& f = tensor(freq, "freq", at::kFloat, device, {-1});
        if (!f.is_contiguous()) raise(PyExc_ValueError, "freq must be contiguous");
        if (f.size(0) < 1 || 2 * f.size(0) > dim)
            raise(PyExc_ValueError, "freq must have 1 to dim / 2 elements, got " + std::to_string(f.size(0)));
        r.freq = static_cast<const float*>(f.const_data_ptr());
        r.pairs = (int)f.size(0);
        const char* name = PyUnicode_Check(pairing) ? PyUnicode_AsUTF8(pairing) : nullptr;
        if (name && !std::strcmp(name, "halves")) r.pairing = TOPK_KV_HALVES;
        else if (name && !std::strcmp(name, "neighbours")) r.pairing = TOPK_KV_NEIGHBOURS;
        else raise(PyExc_ValueError, "pairing must be \"halves\" or \"neighbours\"");
        r.eps = (float)number(eps);
        r.q_norm = norm(q_norm, "q_norm", type, device, q_heads, dim, &r.q_norm_stride);
        r.k_norm = norm(k_norm, "k_norm", type, device, heads, dim, &r.k_norm_stride);
    }
};

// A tensor [tokens, heads, dim], both of them any if below 0.
topk_kv_heads heads_of(const at::Tensor& t, const char* name) {
    if (t.size(1) > INT32_MAX) raise(PyExc_ValueError, std::string(name) + " has too many heads");
    topk_kv_heads h = {const_cast<void*>(t.const_data_ptr()), {0, 0}, (int)t.size(1)};
    strides(t, name, h.stride);
    return h;
}

// The output of a rotation: the one given, or a new one.
at::Tensor rotated(PyObject* o, const char* name, const at::Tensor& in) {
    const int64_t tokens = in.size(0), heads = in.size(1), dim = in.size(2);
    if (o == Py_None)
        return at::Tensor(at::detail::empty_cuda({tokens, heads, dim}, in.scalar_type(), in.device(), std::nullopt));
    return tensor(o, name, in.scalar_type(), in.device(), {tokens, heads, dim});
}

// Refuses a gradient that would get lost without a word: what a call returns
// anew gets a backward pass that says that there is none.
void check_followed(const char* name, const char* of, std::initializer_list<PyObject*> read,
                    std::initializer_list<PyObject*> given) {
    for (PyObject* o : given)
        if (o != Py_None && followed(read))
            raise(PyExc_RuntimeError, std::string(name) + " has no gradient, and " + of +
                                          " require grad: outputs cannot be given then");
}

// Refuses a tangent, which would get lost as well: the operators have no
// derivatives in forward mode either.
void check_tangents(const char* name, std::initializer_list<PyObject*> tensors) {
    if (!c10::AutogradState::get_tls_state().get_fw_grad_mode()) return;
    for (PyObject* o : tensors)
        if (o != Py_None && THPVariable_Unpack(o)._fw_grad(0).defined())
            raise(PyExc_NotImplementedError, std::string(name) + " has no derivative in forward mode, and a tensor has a "
                                                                 "tangent: unpack it first");
}

void no_backward(const char* name, std::initializer_list<PyObject*> read, std::initializer_list<const at::Tensor*> made) {
    torch::autograd::variable_list from;
    for (PyObject* o : read)
        if (o != Py_None) from.push_back(THPVariable_Unpack(o));
    std::shared_ptr<torch::autograd::Node> node(new torch::autograd::NotImplemented(name), torch::autograd::deleteNode);
    node->set_next_edges(torch::autograd::collect_next_edges(from));
    for (const at::Tensor* t : made)
        if (t->defined()) torch::autograd::set_history(*t, node);
}

PyObject* wrapped(const at::Tensor& t) {
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}

PyObject* two(const at::Tensor& a, const at::Tensor& b) {
    PyObject* pair = PyTuple_New(2);
    if (!pair) throw Raised();
    PyTuple_SET_ITEM(pair, 0, wrapped(a));
    PyTuple_SET_ITEM(pair, 1, wrapped(b));
    return pair;
}

// (q, k, pos, freq, q_norm, k_norm, eps, pairing, q_out, k_out, stream) -> (q_out, k_out), or a status
PyObject* rotate(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 11, [&]() -> PyObject* {
        PyObject* const some = a[0] != Py_None ? a[0] : a[1];
        if (some == Py_None) raise(PyExc_ValueError, "q and k cannot both be absent");
        if (!THPVariable_Check(some)) raise(PyExc_TypeError, "q and k must be a torch.Tensor");
        const at::Tensor& lead = THPVariable_Unpack(some);
        const at::ScalarType type = lead.scalar_type();
        const c10::Device device = lead.device();
        if (type != at::kHalf && type != at::kBFloat16)
            raise(PyExc_TypeError, "q and k must be float16 or bfloat16 tensors");
        if (!device.is_cuda()) raise(PyExc_ValueError, "q and k must be CUDA tensors");
        const char* const lead_name = a[0] != Py_None ? "q" : "k";
        tensor(some, lead_name, type, device, {-1, -1, -1});
        const int64_t tokens = lead.size(0), dim = lead.size(2);
        if (tokens > INT32_MAX || dim > INT32_MAX) raise(PyExc_ValueError, "too many tokens");
        const at::Tensor q = a[0] == Py_None ? at::Tensor() : tensor(a[0], "q", type, device, {tokens, -1, dim});
        const at::Tensor k = a[1] == Py_None ? at::Tensor() : tensor(a[1], "k", type, device, {tokens, -1, dim});
        if ((!q.defined() && (a[4] != Py_None || a[8] != Py_None)) || (!k.defined() && (a[5] != Py_None || a[9] != Py_None)))
            raise(PyExc_ValueError, "a norm or an output was given for what is absent");
        const at::Tensor& pos = tensor(a[2], "pos", at::kInt, device, {tokens});
        if (!pos.is_contiguous()) raise(PyExc_ValueError, "pos must be contiguous");
        const Rotation rotation(a[3], a[4], a[5], a[6], a[7], type, device, q.defined() ? q.size(1) : 0,
                                k.defined() ? k.size(1) : 0, dim);
        const Stream s(a[10], device.index());
        // Outputs are known to be tensors before anything is asked of them.
        const at::Tensor q_out = q.defined() ? rotated(a[8], "q_out", q) : at::Tensor();
        const at::Tensor k_out = k.defined() ? rotated(a[9], "k_out", k) : at::Tensor();
        check_tangents("kv_rotate", {a[0], a[1], a[3], a[4], a[5], a[8], a[9]});
        check_written("kv_rotate", {a[8], a[9]});
        check_followed("kv_rotate", "q, k, freq or the norms", {a[0], a[1], a[3], a[4], a[5]}, {a[8], a[9]});
        topk_kv_heads h[4] = {};
        if (q.defined()) {
            h[0] = heads_of(q, "q");
            h[2] = heads_of(q_out, "q_out");
        }
        if (k.defined()) {
            h[1] = heads_of(k, "k");
            h[3] = heads_of(k_out, "k_out");
        }
        const int rc = tokens == 0 ? (int)TOPK_OK : call(device, [&] {
            return g_rotate(type == at::kBFloat16 ? TOPK_KV_BF16 : TOPK_KV_F16, (int)tokens, (int)dim, &rotation.r,
                            static_cast<const int32_t*>(pos.const_data_ptr()), &h[0], &h[1], &h[2], &h[3], s.handle);
        });
        if (rc != TOPK_OK) return PyLong_FromLong(rc);
        written({a[8], a[9]});
        if (followed({a[0], a[1], a[3], a[4], a[5]}))
            no_backward("kv_rotate", {a[0], a[1], a[3], a[4], a[5]}, {&q_out, &k_out});
        return two(q_out, k_out);
    });
}

// (k_pages, v_pages, table, lens, k_new, v_new, freq, starts, weight, pos, next_pos, k_norm, eps, pairing, q, q_norm,
// q_out, stream) -> q_out or None, or a status
PyObject* append_rotated(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 18, [&]() -> PyObject* {
        const Cache c = cache(a[0], a[1], a[2], a[3]);
        const at::Tensor& k = tensor(a[4], "k_new", c.type, c.device, {-1, c.c.heads, c.c.dim});
        const at::Tensor& v = tensor(a[5], "v_new", c.type, c.device, {k.size(0), c.c.heads, c.c.dim});
        const int64_t tokens = k.size(0);
        if (tokens > INT32_MAX) raise(PyExc_ValueError, "too many tokens");
        const int32_t* starts = ints(a[7], "starts", c, (int64_t)c.c.seqs + 1);
        if (!starts && tokens != c.c.seqs)
            raise(PyExc_ValueError, "without starts there must be one token for each sequence");
        if (a[9] != Py_None && a[10] == Py_None) raise(PyExc_ValueError, "pos needs next_pos");
        const topk_kv_rows weight = rows(a[8], "weight", at::kFloat, c), pos = rows(a[9], "pos", at::kInt, c);
        const int32_t* next_pos = ints(a[10], "next_pos", c, c.c.seqs);
        const at::Tensor q = a[14] == Py_None ? at::Tensor() : tensor(a[14], "q", c.type, c.device, {tokens, -1, c.c.dim});
        if (!q.defined() && (a[15] != Py_None || a[16] != Py_None))
            raise(PyExc_ValueError, "q_norm or q_out was given without q");
        const Rotation rotation(a[6], a[15], a[11], a[12], a[13], c.type, c.device, q.defined() ? q.size(1) : 0,
                                c.c.heads, c.c.dim);
        const Stream s(a[17], c);
        const at::Tensor q_out = q.defined() ? rotated(a[16], "q_out", q) : at::Tensor();
        check_tangents("kv_append_rotated",
                       {a[0], a[1], a[4], a[5], a[6], a[8], a[11], a[14], a[15], a[16]});
        check_written("kv_append_rotated", {a[0], a[1], a[8], a[16]});
        check_followed("kv_append_rotated", "q, freq or q_norm", {a[6], a[14], a[15]}, {a[16]});
        if (followed({a[4], a[5], a[6], a[11]}) &&
            PyErr_WarnEx(PyExc_UserWarning,
                         "kv_append_rotated has no gradient: none will reach k_new, v_new, freq and k_norm", 2) != 0)
            throw Raised();
        topk_kv_heads h[4] = {heads_of(k, "k_new"), heads_of(v, "v_new"), {}, {}};
        if (q.defined()) {
            h[2] = heads_of(q, "q");
            h[3] = heads_of(q_out, "q_out");
        }
        const int rc = tokens == 0 ? (int)TOPK_OK : call(c, [&] {
            return g_append_rotated(&c.c, &rotation.r, (int)tokens, starts, &h[0], &h[1], &weight, &pos, next_pos, &h[2],
                                    &h[3], s.handle);
        });
        if (rc != TOPK_OK) return PyLong_FromLong(rc);
        written({a[16]});
        if (tokens) written({a[0], a[1], a[8], a[9]});
        if (followed({a[6], a[14], a[15]})) no_backward("kv_append_rotated", {a[6], a[14], a[15]}, {&q_out});
        return wrapped(q_out);
    });
}

// (logits, u, temperature, top_k, top_p, min_p, token, logp, stream) -> (token, logp), or a status
PyObject* sample(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 9, [&]() -> PyObject* {
        if (!THPVariable_Check(a[0])) raise(PyExc_TypeError, "logits must be a torch.Tensor");
        const at::ScalarType type = THPVariable_Unpack(a[0]).scalar_type();
        const c10::Device device = THPVariable_Unpack(a[0]).device();
        if (type != at::kHalf && type != at::kBFloat16 && type != at::kFloat)
            raise(PyExc_TypeError, "logits must be a float16, bfloat16 or float32 tensor");
        if (!device.is_cuda()) raise(PyExc_ValueError, "logits must be a CUDA tensor");
        const at::Tensor& x = tensor(a[0], "logits", type, device, {-1, -1});
        const int64_t rows = x.size(0), cols = x.size(1);
        if (rows > INT32_MAX || cols > INT32_MAX) raise(PyExc_ValueError, "logits has too many rows or columns");
        if (cols < 1) raise(PyExc_ValueError, "logits must have a column");
        if (cols > 1 && x.stride(1) != 1) raise(PyExc_ValueError, "the rows of logits must be contiguous");
        auto vector = [&](PyObject* o, const char* name, at::ScalarType t) {
            const at::Tensor& v = tensor(o, name, t, device, {rows});
            if (!v.is_contiguous()) raise(PyExc_ValueError, std::string(name) + " must be contiguous");
            return const_cast<void*>(v.const_data_ptr());
        };
        const float* u = static_cast<const float*>(vector(a[1], "u", at::kFloat));
        topk_sampling p = {};
        // What it returns is the parameter's tensor, or None.
        auto parameter = [&](PyObject* o, const char* name, float* one, const float** each) -> PyObject* {
            if (!THPVariable_Check(o)) {
                *one = (float)number(o);
                return Py_None;
            }
            *each = static_cast<const float*>(vector(o, name, at::kFloat));
            return o;
        };
        PyObject* const temperature = parameter(a[2], "temperature", &p.temperature, &p.temperatures);
        if (THPVariable_Check(a[3])) p.top_ks = static_cast<const int32_t*>(vector(a[3], "top_k", at::kInt));
        else p.top_k = integer(a[3]);
        PyObject* const top_p = parameter(a[4], "top_p", &p.top_p, &p.top_ps);
        PyObject* const min_p = parameter(a[5], "min_p", &p.min_p, &p.min_ps);
        if (!p.temperatures) {
            const double given = number(a[2]);
            if (!(given >= 0)) raise(PyExc_ValueError, "temperature must not be negative");
            // One above 0 stays above 0 in 32 bits: 0 has another meaning, and less than 2^-60 counts as that.
            if (given > 0) p.temperature = std::max(p.temperature, 0x1p-60f);
        }
        const Stream s(a[8], device.index());
        if (a[6] != Py_None) vector(a[6], "token", at::kInt);
        if (a[7] != Py_None) vector(a[7], "logp", at::kFloat);
        const std::initializer_list<PyObject*> read = {a[0], a[1], temperature, top_p, min_p};
        check_tangents("sample_rows", read);
        check_tangents("sample_rows", {a[7]});
        check_written("sample_rows", {a[7]});
        check_followed("sample_rows", "the logits, u or parameters", read, {a[7]});
        const at::Tensor token = a[6] != Py_None ? THPVariable_Unpack(a[6])
                                                 : at::Tensor(at::detail::empty_cuda({rows}, at::kInt, device, std::nullopt));
        const at::Tensor logp = a[7] != Py_None ? THPVariable_Unpack(a[7])
                                                : at::Tensor(at::detail::empty_cuda({rows}, at::kFloat, device, std::nullopt));
        const int rc = rows == 0 ? (int)TOPK_OK : call(device, [&] {
            return g_sample(x.const_data_ptr(),
                            type == at::kFloat ? TOPK_SAMPLE_F32 : type == at::kBFloat16 ? TOPK_KV_BF16 : TOPK_KV_F16,
                            rows == 1 ? std::max(cols, x.stride(0)) : x.stride(0), (int)rows, (int)cols, &p, u,
                            static_cast<int32_t*>(token.data_ptr()), static_cast<float*>(logp.data_ptr()), s.handle);
        });
        if (rc != TOPK_OK) return PyLong_FromLong(rc);
        written({a[6], a[7]});
        if (followed(read)) no_backward("sample_rows", read, {&logp});
        return two(token, logp);
    });
}

// (address of topk_kv_append, of topk_kv_attend, of topk_kv_evict, of topk_kv_rotate, of topk_kv_append_rotated, of
// topk_sample_rows)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 6, [&]() -> PyObject* {
        void* f[6];
        for (int i = 0; i < 6; ++i) {
            f[i] = PyLong_AsVoidPtr(a[i]);
            if (!f[i]) raise(PyExc_ValueError, "a function's address is missing");
        }
        g_append = reinterpret_cast<decltype(g_append)>(f[0]);
        g_attend = reinterpret_cast<decltype(g_attend)>(f[1]);
        g_evict = reinterpret_cast<decltype(g_evict)>(f[2]);
        g_rotate = reinterpret_cast<decltype(g_rotate)>(f[3]);
        g_append_rotated = reinterpret_cast<decltype(g_append_rotated)>(f[4]);
        g_sample = reinterpret_cast<decltype(g_sample)>(f[5]);
        Py_RETURN_NONE;
    });
}

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {{"append", fast(append), METH_FASTCALL, nullptr},
                         {"attend", fast(attend), METH_FASTCALL, nullptr},
                         {"evict", fast(evict), METH_FASTCALL, nullptr},
                         {"rotate", fast(rotate), METH_FASTCALL, nullptr},
                         {"append_rotated", fast(append_rotated), METH_FASTCALL, nullptr},
                         {"sample", fast(sample), METH_FASTCALL, nullptr},
                         {"bind", fast(bind), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "kv_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_kv_binding() { return PyModule_Create(&module); }
