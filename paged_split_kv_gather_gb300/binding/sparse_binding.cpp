// sparse_binding.cpp -- argument marshalling of the block-sparse entry points, compiled.
//
// These calls sit between the layers of a decoding step, where a kernel takes 2-10 us;
// reading a dozen tensors' pointers, shapes and strides from interpreted code takes
// 15-25 us a call, from here about 1 us.  Only checks and marshalling: every step of the
// computation is behind the C ABI, whose functions are given by address (set_entry), so
// this module and ctypes use one copy of the library.  A check of a tensor's type, shape
// or device raises ValueError; the library's own refusals come back as its status.
#include <cstdint>
#include <stdexcept>
#include <string>

#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include "../../include/fdec.h"

namespace {

using Tensor = at::Tensor;

struct Bad : std::runtime_error {  // -> ValueError
    using std::runtime_error::runtime_error;
};

void need(bool ok, const char* message) {
    if (!ok) throw Bad(message);
}

const Tensor& tensor(PyObject* o, const char* what) {
    if (!THPVariable_Check(o)) throw Bad(std::string(what) + " must be a tensor");
    return THPVariable_Unpack(o);
}

// A tensor or None (an undefined tensor).
Tensor maybe(PyObject* o, const char* what) { return o == Py_None ? Tensor() : tensor(o, what); }

void* ptr(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Bad("");
    return v;
}

int small(PyObject* o, const char* what) {
    const int64_t v = integer(o);
    if (v < INT32_MIN || v > INT32_MAX) throw Bad(std::string(what) + " does not fit 32 bits");
    return static_cast<int>(v);
}

float real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Bad("");
    return static_cast<float>(v);
}

// The stream given, or the current one of the tensors' device.
cudaStream_t stream_of(PyObject* o, c10::Device device) {
    if (o == Py_None) return device.is_cuda() ? c10::cuda::getCurrentCUDAStream(device.index()).stream() : nullptr;
    if (PyLong_Check(o)) return reinterpret_cast<cudaStream_t>(PyLong_AsVoidPtr(o));
    PyObject* handle = PyObject_GetAttrString(o, "cuda_stream");
    if (handle == nullptr) throw Bad("");
    void* s = PyLong_AsVoidPtr(handle);
    Py_DECREF(handle);
    return static_cast<cudaStream_t>(s);
}

fdec_dtype dtype_of(const Tensor& t) {
    if (t.scalar_type() == at::kBFloat16) return FDEC_BF16;
    if (t.scalar_type() == at::kHalf) return FDEC_F16;
    throw Bad(std::string("expected bfloat16 or float16, got ") + c10::toString(t.scalar_type()));
}

// FDEC_KV_SAME for a cache of the 16-bit type, FDEC_KV_E4M3 for one of 1-byte codes.
int kv_of(const Tensor& t, at::ScalarType type) {
    if (t.scalar_type() == type) return FDEC_KV_SAME;
    if (t.scalar_type() == at::kFloat8_e4m3fn || t.scalar_type() == at::kByte) return FDEC_KV_E4M3;
    throw Bad(std::string("expected a cache of the 16-bit type or of E4M3 codes, got ") + c10::toString(t.scalar_type()));
}

int as_int(int64_t v) {
    need(v <= INT32_MAX, "a size does not fit 32 bits");
    return static_cast<int>(v);
}

// The stride of a dimension; 0 for one of a single index, whose stride may be anything.
int64_t step(const Tensor& t, int dim) { return t.size(dim) > 1 ? t.stride(dim) : 0; }

// Entries between two rows of a page table.
int64_t table_stride(const Tensor& t) { return t.size(0) > 1 ? t.stride(0) : t.size(1); }

fdec_kv_desc pool(const Tensor& t) {
    need(t.dim() == 4 && t.stride(3) == 1, "caches must be 4-D [page, kv_head, slot, dim] with a unit dim stride");
    return {t.data_ptr(), t.size(0), step(t, 0), step(t, 1), step(t, 2)};
}

fdec_rows rows(const Tensor& t) {
    need(t.dim() == 3 && t.stride(2) == 1, "rows must be [n, heads, head_dim] with a unit dim stride");
    return {t.data_ptr(), step(t, 0), step(t, 1)};
}

const int32_t* index(const Tensor& t, int64_t dim, const char* what) {
    if (t.scalar_type() != at::kInt || t.dim() != dim || (t.numel() > 0 && t.stride(dim - 1) != 1))
        throw Bad(std::string(what) + " must be an int32 tensor with contiguous rows, of " + std::to_string(dim) +
                  " dimension(s)");
    return static_cast<const int32_t*>(t.data_ptr());
}

void on(const Tensor& first, std::initializer_list<const Tensor*> others) {
    for (const Tensor* t : others)
        if (t->defined() && t->device() != first.device())
            throw Bad("tensors on " + first.device().str() + " and " + t->device().str());
}

uint32_t* error_word(const Tensor& t) {
    if (!t.defined()) return nullptr;
    need(t.element_size() == 4 && t.numel() >= 1, "device_errors must hold one 32-bit value");
    return static_cast<uint32_t*>(t.data_ptr());
}

// Token and head strides of q [B, Q, Hq, D], tokens flattened.
void q_strides(const Tensor& q, int64_t* tok, int64_t* head) {
    need(q.dim() == 4 && q.stride(3) == 1, "q must be [B, Q, Hq, D] with a unit head_dim stride");
    if (q.size(1) == 1) {
        *tok = step(q, 0);
    } else {
        need(q.size(0) <= 1 || q.stride(0) == q.size(1) * q.stride(1), "q tokens must flatten to one stride (b*q_len + i)");
        *tok = q.stride(1);
    }
    *head = step(q, 2);
}

decltype(&fdec_norm_rope_append) g_norm_rope_append = nullptr;
decltype(&fdec_page_bounds) g_page_bounds = nullptr;
decltype(&fdec_select_pages) g_select_pages = nullptr;
decltype(&fdec_run_selected) g_run_selected = nullptr;
void (*g_checks_only)(int) = nullptr;
constexpr int kChecksOnly = -1;  // the status of a call that has passed its checks and launched nothing

// The library call f(stream) on the device of its tensors.  Tensors that are not on a GPU
// go through its checks, which touch no element, and are refused where it would launch.
template <typename F>
fdec_status on_device(const Tensor& t, PyObject* stream, F&& f) {
    const cudaStream_t s = stream_of(stream, t.device());
    if (t.is_cuda()) {
        const c10::cuda::CUDAGuard guard(t.device());
        return f(s);
    }
    struct ChecksOnly {
        ChecksOnly() { g_checks_only(1); }
        ~ChecksOnly() { g_checks_only(0); }
    };
    const fdec_status st = [&] {
        const ChecksOnly scope;
        return f(s);
    }();
    need(static_cast<int>(st) != kChecksOnly, "tensors must be on a CUDA device");
    return st;
}

// Run f() -> status; C++ exceptions become Python ones.
template <typename F>
PyObject* guarded(F&& f) {
    try {
        return PyLong_FromLong(static_cast<long>(f()));
    } catch (const Bad& e) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::exception& e) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

bool has(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    return false;
}

// q, k_new, v_new, q_weight, k_weight, cos_sin, batch_indices, positions, q_out, k, v, page_table, page_size, eps,
// interleaved, rope_positions, k_scale, v_scale, device_errors, stream
PyObject* norm_rope_append(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    if (!has(n_args, 20)) return nullptr;
    return guarded([&] {
        const Tensor &q = tensor(a[0], "q"), &k_new = tensor(a[1], "k_new"), &v_new = tensor(a[2], "v_new");
        const Tensor q_weight = maybe(a[3], "q_weight"), k_weight = maybe(a[4], "k_weight"), cs = maybe(a[5], "cos_sin");
        const Tensor &bi = tensor(a[6], "batch_indices"), &pos = tensor(a[7], "positions"), &q_out = tensor(a[8], "q_out");
        const Tensor &k = tensor(a[9], "k"), &v = tensor(a[10], "v"), &table = tensor(a[11], "page_table");
        const Tensor rope = maybe(a[15], "rope_positions"), errors = maybe(a[18], "device_errors");
        const int page_size = small(a[12], "page_size");
        const fdec_dtype dtype = dtype_of(q);
        const at::ScalarType type = q.scalar_type();
        need(q.dim() == 3 && k_new.dim() == 3 && k_new.sizes() == v_new.sizes() && k_new.size(0) == q.size(0) &&
                 k_new.size(2) == q.size(2) && q_out.sizes() == q.sizes(),
             "q, q_out must be [n, Hq, D] and k_new, v_new [n, Hk, D]");
        need(k_new.scalar_type() == type && v_new.scalar_type() == type && q_out.scalar_type() == type,
             "q, k_new, v_new and q_out must have one type");
        const int64_t n = q.size(0), hq = q.size(1), hk = k_new.size(1), d = q.size(2);
        for (const Tensor* w : {&q_weight, &k_weight})
            need(!w->defined() || (w->scalar_type() == type && w->dim() == 1 && w->size(0) == d && w->is_contiguous()),
                 "weights must be contiguous [head_dim] tensors of the rows' type");
        need(!cs.defined() || (cs.scalar_type() == at::kFloat && cs.dim() == 2 && cs.is_contiguous()),
             "cos_sin must be a contiguous float32 [positions, rot_dim] tensor");
        const int32_t* bi_p = index(bi, 1, "batch_indices");
        const int32_t* pos_p = index(pos, 1, "positions");
        const int32_t* rope_p = rope.defined() ? index(rope, 1, "rope_positions") : nullptr;
        need(bi.size(0) == n && pos.size(0) == n && (!rope.defined() || rope.size(0) == n),
             "batch_indices, positions and rope_positions must have one entry per token");
        const int32_t* table_p = index(table, 2, "page_table");
        const int kv = kv_of(k, type);
        need(v.scalar_type() == k.scalar_type() && k.dim() == 4 && v.dim() == 4 && k.size(1) == hk &&
                 k.size(2) == page_size && k.size(3) == d && v.sizes().slice(1) == k.sizes().slice(1),
             "k and v must be caches [page, Hk, page_size, D] of one type");
        on(q, {&k_new, &v_new, &q_weight, &k_weight, &cs, &bi, &pos, &rope, &q_out, &k, &v, &table, &errors});
        return on_device(q, a[19], [&](cudaStream_t stream) {
            return g_norm_rope_append(rows(q), rows(k_new), rows(v_new), ptr(q_weight), ptr(k_weight), real(a[13]),
                                      static_cast<const float*>(ptr(cs)), cs.defined() ? cs.size(0) : 0,
                                      cs.defined() ? as_int(cs.size(1)) : 0, PyObject_IsTrue(a[14]), bi_p, pos_p, rope_p,
                                      as_int(n), as_int(hq), as_int(hk), as_int(d), page_size, dtype, kv, real(a[16]),
                                      real(a[17]), rows(q_out), pool(k), pool(v), table_p, as_int(table.size(0)),
                                      table_stride(table), error_word(errors), stream);
        });
    });
}

// k, bounds, page_table, begins, seq_lens, page_size, expected_tokens, device_errors, stream
PyObject* page_bounds(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    if (!has(n_args, 9)) return nullptr;
    return guarded([&] {
        const Tensor &k = tensor(a[0], "k"), &bounds = tensor(a[1], "bounds"), &table = tensor(a[2], "page_table");
        const Tensor begins = maybe(a[3], "begins"), errors = maybe(a[7], "device_errors");
        const Tensor& lens = tensor(a[4], "seq_lens");
        const int page_size = small(a[5], "page_size");
        const fdec_dtype dtype = dtype_of(bounds);
        const int kv = kv_of(k, bounds.scalar_type());
        need(k.dim() == 4 && k.size(2) == page_size && bounds.dim() == 4 && bounds.size(1) == k.size(1) &&
                 bounds.size(2) == 2 && bounds.size(3) == k.size(3),
             "need k [page, Hk, page_size, D] and bounds [page, Hk, 2, D]");
        const int32_t* table_p = index(table, 2, "page_table");
        const int32_t* begins_p = begins.defined() ? index(begins, 1, "begins") : nullptr;
        const int32_t* lens_p = index(lens, 1, "seq_lens");
        need(lens.size(0) == table.size(0) && (!begins.defined() || begins.size(0) == table.size(0)),
             "begins and seq_lens must have one entry per sequence");
        on(k, {&bounds, &table, &begins, &lens, &errors});
        int64_t expected = integer(a[6]);
        if (expected <= 0) expected = table.size(1) * page_size;
        if (expected > INT32_MAX) expected = INT32_MAX;
        return on_device(k, a[8], [&](cudaStream_t stream) {
            return g_page_bounds(pool(k), pool(bounds), table_p, as_int(table.size(0)), table_stride(table), begins_p,
                                 lens_p, as_int(k.size(1)), as_int(k.size(3)), page_size, dtype, kv,
                                 static_cast<int>(expected), error_word(errors), stream);
        });
    });
}

// q, bounds, page_table, seq_lens, page_size, max_pages, budget, page_ids, counts, page_indices, workspace, first_pages,
// last_pages, causal, device_errors, stream
PyObject* select_pages(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    if (!has(n_args, 16)) return nullptr;
    return guarded([&] {
        const Tensor &q = tensor(a[0], "q"), &bounds = tensor(a[1], "bounds"), &table = tensor(a[2], "page_table");
        const Tensor &lens = tensor(a[3], "seq_lens"), &ids = tensor(a[7], "page_ids"), &counts = tensor(a[8], "counts");
        const Tensor indices = maybe(a[9], "page_indices"), errors = maybe(a[14], "device_errors");
        const Tensor& ws = tensor(a[10], "workspace");
        const int page_size = small(a[4], "page_size"), budget = small(a[6], "budget");
        const int64_t max_pages = integer(a[5]);
        const fdec_dtype dtype = dtype_of(q);
        int64_t tok, head;
        q_strides(q, &tok, &head);
        const int64_t b = q.size(0), q_len = q.size(1), hq = q.size(2), d = q.size(3);
        need(bounds.scalar_type() == q.scalar_type() && bounds.dim() == 4 && bounds.size(2) == 2 && bounds.size(3) == d,
             "bounds must be [page, Hk, 2, D] of q's type");
        const int64_t hk = bounds.size(1);
        const int32_t* table_p = index(table, 2, "page_table");
        const int32_t* lens_p = index(lens, 1, "seq_lens");
        need(table.size(0) == b && lens.size(0) == b && table.size(1) >= max_pages,
             "page_table must be [B, >= max_pages] and seq_lens [B]");
        for (const Tensor* t : {&ids, &indices})
            if (t->defined()) {
                index(*t, 3, "page_ids and page_indices");
                need(t->size(0) == b * q_len && t->size(1) == hk && t->size(2) == budget && t->is_contiguous(),
                     "page_ids and page_indices must be contiguous [B * Q, Hk, budget]");
            }
        index(counts, 2, "counts");
        need(counts.size(0) == b * q_len && counts.size(1) == hk && counts.is_contiguous(),
             "counts must be contiguous [B * Q, Hk]");
        need(ws.is_contiguous(), "workspace must be contiguous");
        on(q, {&bounds, &table, &lens, &ids, &counts, &indices, &ws, &errors});
        return on_device(q, a[15], [&](cudaStream_t stream) {
            return g_select_pages(q.data_ptr(), tok, head, pool(bounds), table_p, table_stride(table), lens_p, as_int(b),
                                  as_int(q_len), page_size, as_int(hq), as_int(hk), as_int(d), dtype,
                                  PyObject_IsTrue(a[13]), max_pages, budget, small(a[11], "first_pages"),
                                  small(a[12], "last_pages"), static_cast<int32_t*>(ids.data_ptr()),
                                  static_cast<int32_t*>(counts.data_ptr()), static_cast<int32_t*>(ptr(indices)),
                                  ws.data_ptr(), static_cast<size_t>(ws.numel()) * ws.element_size(),
                                  error_word(errors), stream);
        });
    });
}

// plan handle, its (batch, num_qo_heads, num_kv_heads, head_dim, page_size, is bf16, element bytes of the cache) tuple,
// q, k, v, page_ids, counts, out, lse, workspace, scale, k_scale, v_scale, stream
PyObject* run_selected(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    if (!has(n_args, 14)) return nullptr;
    return guarded([&] {
        fdec_plan_t plan = static_cast<fdec_plan_t>(PyLong_AsVoidPtr(a[0]));
        if (PyErr_Occurred()) throw Bad("");
        need(PyTuple_Check(a[1]) && PyTuple_GET_SIZE(a[1]) == 7, "bad plan description");
        int64_t m[7];
        for (int i = 0; i < 7; ++i) m[i] = integer(PyTuple_GET_ITEM(a[1], i));
        const int64_t n = m[0], hq = m[1], hk = m[2], d = m[3], page_size = m[4];
        const Tensor &q = tensor(a[2], "q"), &k = tensor(a[3], "k"), &v = tensor(a[4], "v");
        const Tensor &ids = tensor(a[5], "page_ids"), &counts = tensor(a[6], "counts"), &out = tensor(a[7], "out");
        const Tensor lse = maybe(a[8], "lse");
        const Tensor& ws = tensor(a[9], "workspace");
        int64_t tok, head;
        q_strides(q, &tok, &head);
        need(q.scalar_type() == (m[5] ? at::kBFloat16 : at::kHalf) && q.size(0) * q.size(1) == n && q.size(2) == hq &&
                 q.size(3) == d,
             "q must be [N, 1, Hq, D] as planned");
        for (const Tensor* t : {&k, &v}) {
            need(t->dim() == 4 && t->size(1) == hk && t->size(2) == page_size && t->size(3) == d,
                 "k and v must be caches [page, Hk, page_size, D] as planned");
            need(t->element_size() == m[6] && (m[6] == 1 || t->scalar_type() == q.scalar_type()),
                 "k and v must hold the element type that was planned");
        }
        const bool f32 = out.scalar_type() == at::kFloat;
        need((f32 || out.scalar_type() == q.scalar_type()) && out.numel() == n * hq * d && out.is_contiguous(),
             "out must be contiguous [N, 1, Hq, D], float32 or of q's type");
        need(!lse.defined() || (lse.scalar_type() == at::kFloat && lse.numel() == n * hq && lse.is_contiguous()),
             "lse must be contiguous float32 [N, 1, Hq]");
        const int32_t* ids_p = index(ids, 3, "page_ids");
        const int32_t* counts_p = index(counts, 2, "counts");
        need(ids.size(0) == n && ids.size(1) == hk && ids.is_contiguous(), "page_ids must be contiguous [N, Hk, W]");
        need(counts.size(0) == n && counts.size(1) == hk && counts.is_contiguous(), "counts must be contiguous [N, Hk]");
        on(q, {&k, &v, &ids, &counts, &out, &lse, &ws});
        return on_device(q, a[13], [&](cudaStream_t stream) {
            return g_run_selected(plan, q.data_ptr(), tok, head, pool(k), pool(v), ids_p, ids.size(2), counts_p,
                                  real(a[10]), real(a[11]), real(a[12]), out.data_ptr(),
                                  f32 ? FDEC_OUT_F32 : FDEC_OUT_SAME, static_cast<float*>(ptr(lse)), ws.data_ptr(),
                                  stream);
        });
    });
}

// The addresses of fdec_norm_rope_append, fdec_page_bounds, fdec_select_pages, fdec_run_selected and
// fdec_internal_checks_only.
PyObject* set_entries(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    if (!has(n_args, 5)) return nullptr;
    void* p[5];
    for (int i = 0; i < 5; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (PyErr_Occurred()) return nullptr;
    }
    g_norm_rope_append = reinterpret_cast<decltype(&fdec_norm_rope_append)>(p[0]);
    g_page_bounds = reinterpret_cast<decltype(&fdec_page_bounds)>(p[1]);
    g_select_pages = reinterpret_cast<decltype(&fdec_select_pages)>(p[2]);
    g_run_selected = reinterpret_cast<decltype(&fdec_run_selected)>(p[3]);
    g_checks_only = reinterpret_cast<decltype(g_checks_only)>(p[4]);
    Py_RETURN_NONE;
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(norm_rope_append), FAST(page_bounds), FAST(select_pages), FAST(run_selected),
                         FAST(set_entries), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_sparse_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__sparse_binding(void) { return PyModule_Create(&module); }
