// sparse_binding.cpp -- argument marshalling of the block-sparse entry points, compiled.
//
// These calls sit between the layers of a decoding step, where a kernel takes 2-10 us;
// reading a dozen tensors' pointers, shapes and strides from interpreted code takes
// 15-25 us a call, from here about 1 us.  Only checks and marshalling: every step of the
// computation is behind the C ABI, whose functions are given by address (set_entry), so
// this module and ctypes use one copy of the library.  A check of a tensor's type, shape
// or device raises ValueError; the library's own refusals come back as its status.
#include "marshal.h"

namespace {

decltype(&fdec_norm_rope_append) g_norm_rope_append = nullptr;
decltype(&fdec_page_bounds) g_page_bounds = nullptr;
decltype(&fdec_select_pages) g_select_pages = nullptr;
decltype(&fdec_run_selected) g_run_selected = nullptr;

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

PyMethodDef methods[] = {FAST(norm_rope_append), FAST(page_bounds), FAST(select_pages), FAST(run_selected),
                         FAST(set_entries), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_sparse_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__sparse_binding(void) { return PyModule_Create(&module); }
