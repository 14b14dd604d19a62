// draft_binding.cpp -- argument marshalling of the entry points of speculative decoding,
// compiled, as that of the block-sparse ones is and for the same reason.
#include "marshal.h"

#include <cmath>
#include <vector>

namespace {

decltype(&fdec_tree_attention) g_tree_attention = nullptr;
decltype(&fdec_verify_drafts) g_verify_drafts = nullptr;
decltype(&fdec_keep_path) g_keep_path = nullptr;
decltype(&fdec_reserve_pages) g_reserve_pages = nullptr;
void (*g_table_columns)(int64_t) = nullptr;

// The calls of its scope look at the columns of a page table's view only: between its rows, and behind the last one,
// lies what is not the view's.
struct Columns {
    explicit Columns(const Tensor& table) : some(table.size(0) > 1 && table.stride(0) > table.size(1)) {
        if (some) g_table_columns(table.size(1));
    }
    ~Columns() {
        if (some) g_table_columns(-1);
    }
    Columns(const Columns&) = delete;
    const bool some;
};

// An int32 tensor [batch][nodes], contiguous.
int32_t* grid(const Tensor& t, int64_t batch, int64_t nodes, const char* what) {
    index(t, 2, what);
    if (t.size(0) != batch || t.size(1) != nodes || !t.is_contiguous())
        throw Bad(std::string(what) + " must be a contiguous [batch, num_nodes] tensor");
    return static_cast<int32_t*>(t.data_ptr());
}

// An int32 tensor [batch].
int32_t* line(const Tensor& t, int64_t batch, const char* what) {
    index(t, 1, what);
    if (t.size(0) != batch) throw Bad(std::string(what) + " must have one entry per sequence");
    return static_cast<int32_t*>(t.data_ptr());
}

// The caches of a call: a sequence of tensors [page, kv_head, slot, dim] or [layer, page, kv_head, slot, dim].
std::vector<fdec_cache> caches_of(PyObject* o, int page_size, std::vector<Tensor>* kept) {
    struct Ref {
        PyObject* o;
        ~Ref() { Py_XDECREF(o); }
    } seq{PySequence_Fast(o, "caches must be a sequence of tensors")};
    if (seq.o == nullptr) throw Bad("");
    std::vector<fdec_cache> out;
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq.o);
    for (Py_ssize_t i = 0; i < n; ++i) {
        const Tensor& t = tensor(PySequence_Fast_GET_ITEM(seq.o, i), "a cache");
        const int64_t d = t.dim();
        need((d == 4 || d == 5) && t.stride(d - 1) == 1 && t.size(d - 2) == page_size,
             "caches must be [page, kv_head, page_size, dim] or [layer, page, kv_head, page_size, dim] with a unit dim stride");
        const int64_t eb = t.element_size();
        fdec_cache c = {};
        c.base = t.data_ptr();
        c.num_layers = d == 5 ? as_int(t.size(0)) : 1;
        c.num_heads = as_int(t.size(d - 3));
        c.row_bytes = as_int(t.size(d - 1) * eb);
        c.num_pages = t.size(d - 4);
        c.stride_layer = d == 5 ? step(t, 0) * eb : 0;
        c.stride_page = step(t, static_cast<int>(d) - 4) * eb;
        c.stride_head = step(t, static_cast<int>(d) - 3) * eb;
        c.stride_token = step(t, static_cast<int>(d) - 2) * eb;
        out.push_back(c);
        kept->push_back(t);
    }
    return out;
}

void on_all(const Tensor& first, const std::vector<Tensor>& others) {
    for (const Tensor& t : others) on(first, {&t});
}

// q, k, v, page_table, prefix_lens, parents, o_prefix, lse_prefix, out, lse, page_size, node_counts, scale, k_scale,
// v_scale, device_errors, stream
PyObject* tree_attention(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    if (!has(n_args, 17)) return nullptr;
    return guarded([&] {
        const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
        const Tensor &table = tensor(a[3], "page_table"), &prefix = tensor(a[4], "prefix_lens");
        const Tensor parents = maybe(a[5], "parents"), o_prefix = maybe(a[6], "o_prefix");
        const Tensor lse_prefix = maybe(a[7], "lse_prefix"), lse = maybe(a[9], "lse");
        const Tensor& out = tensor(a[8], "out");
        const int page_size = small(a[10], "page_size");
        const Tensor counts = maybe(a[11], "node_counts"), errors = maybe(a[15], "device_errors");
        const fdec_dtype dtype = dtype_of(q);
        int64_t tok, head;
        q_strides(q, &tok, &head);
        const int64_t b = q.size(0), n = q.size(1), hq = q.size(2), d = q.size(3);
        const int kv = kv_of(k, q.scalar_type());
        need(v.scalar_type() == k.scalar_type() && k.dim() == 4 && v.dim() == 4 && k.size(2) == page_size &&
                 k.size(3) == d && v.sizes().slice(1) == k.sizes().slice(1),
             "k and v must be caches [page, Hk, page_size, D] of one type");
        const int32_t* table_p = index(table, 2, "page_table");
        need(table.size(0) == b, "page_table must have one row per sequence");
        const int32_t* prefix_p = line(prefix, b, "prefix_lens");
        const int32_t* counts_p = counts.defined() ? line(counts, b, "node_counts") : nullptr;
        const int32_t* parents_p = parents.defined() ? grid(parents, b, n, "parents") : nullptr;
        const bool f32 = out.scalar_type() == at::kFloat;
        need((f32 || out.scalar_type() == q.scalar_type()) && out.numel() == q.numel() && out.is_contiguous(),
             "out must be contiguous [B, N, Hq, D], float32 or of q's type");
        need(!o_prefix.defined() || (o_prefix.scalar_type() == at::kFloat && o_prefix.numel() == q.numel() &&
                                     o_prefix.is_contiguous()),
             "o_prefix must be contiguous float32 [B, N, Hq, D]");
        for (const Tensor* t : {&lse, &lse_prefix})
            need(!t->defined() || (t->scalar_type() == at::kFloat && t->numel() == b * n * hq && t->is_contiguous()),
                 "lse and lse_prefix must be contiguous float32 [B, N, Hq]");
        on(q, {&k, &v, &table, &prefix, &counts, &parents, &o_prefix, &lse_prefix, &out, &lse, &errors});
        const double scale = a[12] == Py_None ? 1.0 / std::sqrt(static_cast<double>(d)) : real(a[12]);
        const Columns columns(table);
        return on_device(q, a[16], [&](cudaStream_t stream) {
            return g_tree_attention(q.data_ptr(), tok, head, pool(k), pool(v), table_p, table_stride(table), prefix_p,
                                    counts_p, parents_p, as_int(b), as_int(n), page_size, as_int(hq), as_int(k.size(1)),
                                    as_int(d), dtype, kv, static_cast<float>(scale), real(a[13]), real(a[14]),
                                    static_cast<const float*>(ptr(o_prefix)), static_cast<const float*>(ptr(lse_prefix)),
                                    out.data_ptr(), f32 ? FDEC_OUT_F32 : FDEC_OUT_SAME, static_cast<float*>(ptr(lse)),
                                    error_word(errors), stream);
        });
    });
}

// target_probs, draft_probs, tokens, parents, uniforms, path, path_lens, out_tokens, node_counts, device_errors, stream
PyObject* verify_drafts(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    if (!has(n_args, 11)) return nullptr;
    return guarded([&] {
        const Tensor &target = tensor(a[0], "target_probs"), &tokens = tensor(a[2], "tokens");
        const Tensor draft = maybe(a[1], "draft_probs"), parents = maybe(a[3], "parents");
        const Tensor &uniforms = tensor(a[4], "uniforms"), &path = tensor(a[5], "path");
        const Tensor &lens = tensor(a[6], "path_lens"), &words = tensor(a[7], "out_tokens");
        const Tensor counts = maybe(a[8], "node_counts"), errors = maybe(a[9], "device_errors");
        need(target.dim() == 3 && (target.size(2) <= 1 || target.stride(2) == 1),
             "target_probs must be [batch, num_nodes, vocab] with a unit vocab stride");
        const int64_t b = target.size(0), n = target.size(1), v = target.size(2);
        int type;
        switch (target.scalar_type()) {
            case at::kFloat: type = FDEC_PROB_F32; break;
            case at::kBFloat16: type = FDEC_PROB_BF16; break;
            case at::kHalf: type = FDEC_PROB_F16; break;
            default: throw Bad("probabilities must be float32, bfloat16 or float16");
        }
        need(!draft.defined() || (draft.scalar_type() == target.scalar_type() && draft.dim() == 3 && draft.size(0) == b &&
                                  draft.size(1) >= n - 1 && draft.size(2) == v && (v <= 1 || draft.stride(2) == 1)),
             "draft_probs must be [batch, >= num_nodes - 1, vocab] of target_probs' type with a unit vocab stride");
        const int32_t* tokens_p = grid(tokens, b, n, "tokens");
        const int32_t* parents_p = parents.defined() ? grid(parents, b, n, "parents") : nullptr;
        const int32_t* counts_p = counts.defined() ? line(counts, b, "node_counts") : nullptr;
        need(uniforms.scalar_type() == at::kFloat && uniforms.dim() == 2 && uniforms.size(0) == b && uniforms.size(1) == n &&
                 uniforms.is_contiguous(),
             "uniforms must be contiguous float32 [batch, num_nodes]");
        int32_t* path_p = grid(path, b, n, "path");
        int32_t* lens_p = line(lens, b, "path_lens");
        int32_t* words_p = grid(words, b, n, "out_tokens");
        on(target, {&draft, &tokens, &parents, &uniforms, &path, &lens, &words, &counts, &errors});
        // (draft rows of a chain of one node: none, and none is read)
        const void* draft_p = draft.defined() && draft.numel() > 0 ? draft.data_ptr() : nullptr;
        return on_device(target, a[10], [&](cudaStream_t stream) {
            return g_verify_drafts(target.data_ptr(), step(target, 0), step(target, 1), draft_p,
                                   draft_p != nullptr ? step(draft, 0) : 0, draft_p != nullptr ? step(draft, 1) : 0, type,
                                   tokens_p, parents_p, counts_p, static_cast<const float*>(uniforms.data_ptr()), as_int(b),
                                   as_int(n), as_int(v), path_p, lens_p, words_p, error_word(errors), stream);
        });
    });
}

// caches, page_table, prefix_lens, path, path_lens, seq_lens, page_size, device_errors, stream
PyObject* keep_path(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    if (!has(n_args, 9)) return nullptr;
    return guarded([&] {
        const Tensor &table = tensor(a[1], "page_table"), &prefix = tensor(a[2], "prefix_lens");
        const Tensor &path = tensor(a[3], "path"), &path_lens = tensor(a[4], "path_lens"), &lens = tensor(a[5], "seq_lens");
        const int page_size = small(a[6], "page_size");
        const Tensor errors = maybe(a[7], "device_errors");
        std::vector<Tensor> kept;
        const std::vector<fdec_cache> caches = caches_of(a[0], page_size, &kept);
        const int32_t* table_p = index(table, 2, "page_table");
        const int64_t b = table.size(0);
        const int32_t* path_p = index(path, 2, "path");
        need(path.size(0) == b, "path must have one row per sequence");
        const int32_t* prefix_p = line(prefix, b, "prefix_lens");
        const int32_t* path_lens_p = line(path_lens, b, "path_lens");
        int32_t* lens_p = line(lens, b, "seq_lens");
        on(table, {&prefix, &path, &path_lens, &lens, &errors});
        on_all(table, kept);
        const Columns columns(table);
        return on_device(table, a[8], [&](cudaStream_t stream) {
            return g_keep_path(caches.data(), as_int(static_cast<int64_t>(caches.size())), table_p, as_int(b),
                               table_stride(table), page_size, prefix_p, path_p, table_stride(path), path_lens_p,
                               as_int(path.size(1)), lens_p, error_word(errors), stream);
        });
    });
}

// page_table, seq_lens, new_lens, granted, num_pages, page_size, workspace, sources, caches, device_errors, stream
PyObject* reserve_pages(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    if (!has(n_args, 11)) return nullptr;
    return guarded([&] {
        const Tensor &table = tensor(a[0], "page_table"), &lens = tensor(a[1], "seq_lens"), &want = tensor(a[2], "new_lens");
        const Tensor &granted = tensor(a[3], "granted"), &ws = tensor(a[6], "workspace");
        const int64_t num_pages = integer(a[4]);
        const int page_size = small(a[5], "page_size");
        const Tensor sources = maybe(a[7], "sources"), errors = maybe(a[9], "device_errors");
        std::vector<Tensor> kept;
        const std::vector<fdec_cache> caches = caches_of(a[8], page_size, &kept);
        index(table, 2, "page_table");
        const int64_t b = table.size(0);
        const int32_t* lens_p = line(lens, b, "seq_lens");
        const int32_t* want_p = line(want, b, "new_lens");
        int32_t* granted_p = line(granted, b, "granted");
        const int32_t* sources_p = sources.defined() ? line(sources, b, "sources") : nullptr;
        need(ws.is_contiguous(), "workspace must be contiguous");
        on(table, {&lens, &want, &granted, &ws, &sources, &errors});
        on_all(table, kept);
        const Columns columns(table);
        return on_device(table, a[10], [&](cudaStream_t stream) {
            return g_reserve_pages(static_cast<int32_t*>(table.data_ptr()), as_int(b), table_stride(table), page_size,
                                   lens_p, want_p, sources_p, granted_p, num_pages, caches.data(),
                                   as_int(static_cast<int64_t>(caches.size())), ws.data_ptr(),
                                   static_cast<size_t>(ws.numel()) * ws.element_size(), error_word(errors), stream);
        });
    });
}

// The addresses of fdec_tree_attention, fdec_verify_drafts, fdec_keep_path, fdec_reserve_pages,
// fdec_internal_table_columns and fdec_internal_checks_only.
PyObject* set_entries(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    if (!has(n_args, 6)) return nullptr;
    void* p[6];
    for (int i = 0; i < 6; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (PyErr_Occurred()) return nullptr;
    }
    g_tree_attention = reinterpret_cast<decltype(&fdec_tree_attention)>(p[0]);
    g_verify_drafts = reinterpret_cast<decltype(&fdec_verify_drafts)>(p[1]);
    g_keep_path = reinterpret_cast<decltype(&fdec_keep_path)>(p[2]);
    g_reserve_pages = reinterpret_cast<decltype(&fdec_reserve_pages)>(p[3]);
    g_table_columns = reinterpret_cast<decltype(g_table_columns)>(p[4]);
    g_checks_only = reinterpret_cast<decltype(g_checks_only)>(p[5]);
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {FAST(tree_attention), FAST(verify_drafts), FAST(keep_path), FAST(reserve_pages),
                         FAST(set_entries), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_draft_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__draft_binding(void) { return PyModule_Create(&module); }
