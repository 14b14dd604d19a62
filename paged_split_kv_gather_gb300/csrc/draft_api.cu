// draft_api.cu -- entry points of speculative decoding: argument checks of
// fdec_tree_attention, fdec_verify_drafts, fdec_keep_path and fdec_reserve_pages.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/fdec.h"
#include "fdec_internal.h"

using namespace fdec;

namespace {

fdec_status fail(fdec_status st, const char* msg) { return static_cast<fdec_status>(record_failure(st, msg)); }

fdec_status fail_cuda(cudaError_t e, const char* what) { return static_cast<fdec_status>(record_cuda_failure(e, what)); }

// log2 of a page size, -1 if it is none that the library takes.
int page_shift_of(int page_size) {
    for (int s = 0; s <= 8; ++s)
        if (page_size == 1 << s) return s;
    return -1;
}

bool aligned(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

bool overlap(const void* a, size_t a_bytes, const void* b, size_t b_bytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + b_bytes && y < x + a_bytes;
}

struct Span {
    const void* base;  // or null
    size_t bytes;
};

bool clash(Span a, Span b) {
    return a.base != nullptr && b.base != nullptr && overlap(a.base, a.bytes, b.base, b.bytes);
}

template <size_t N>
bool clash(Span a, const Span (&others)[N]) {
    return std::any_of(others, others + N, [&](Span b) { return clash(a, b); });
}

// Bytes of `rows` rows of int32, `cols` of `stride` entries each.
size_t table_bytes(int64_t rows, int64_t stride, int64_t cols) {
    return (static_cast<size_t>(rows - 1) * stride + cols) * 4;
}

// A pool of rows of 16-byte multiples (eb bytes an element).
fdec_status check_pool(const fdec_kv_desc& d, int eb) {
    if (d.base == nullptr) return fail(FDEC_ERR_INVALID_ARG, "null pool");
    if (d.num_pages < 1 || d.num_pages > INT32_MAX) return fail(FDEC_ERR_INVALID_ARG, "pools need 1 .. 2^31-1 pages");
    const int64_t unit = 16 / eb;
    if (!aligned(d.base, 16)) return fail(FDEC_ERR_LAYOUT, "pools must be 16-byte aligned");
    if (d.stride_page < 0 || d.stride_head < 0 || d.stride_token < 0 || d.stride_page % unit != 0 ||
        d.stride_head % unit != 0 || d.stride_token % unit != 0)
        return fail(FDEC_ERR_LAYOUT, "pool strides must be non-negative multiples of 16 bytes");
    return FDEC_OK;
}

fdec_status check_tree(int batch, int num_nodes) {
    if (batch < 1) return fail(FDEC_ERR_INVALID_ARG, "batch must be >= 1");
    if (num_nodes < 1) return fail(FDEC_ERR_INVALID_ARG, "num_nodes must be >= 1");
    if (num_nodes > kMaxNodes) return fail(FDEC_ERR_UNSUPPORTED, "num_nodes must be at most 64");
    return FDEC_OK;
}

// The caches of a call that moves rows; *fewest: the fewest pages of any.  Rows are written, so no two may be one.
fdec_status take_caches(const fdec_cache* caches, int num_caches, int page_size, CacheList<kMaxCaches>* out,
                        int64_t* fewest) {
    if (num_caches < 0 || num_caches > kMaxCaches) return fail(FDEC_ERR_INVALID_ARG, "between 0 and 128 caches a call");
    if (num_caches > 0 && caches == nullptr) return fail(FDEC_ERR_INVALID_ARG, "null caches");
    *out = {};
    out->n = num_caches;
    *fewest = INT32_MAX;
    int64_t blocks = 0;
    for (int i = 0; i < num_caches; ++i) {
        const fdec_cache& c = caches[i];
        if (c.base == nullptr) return fail(FDEC_ERR_INVALID_ARG, "null cache");
        if (c.num_layers < 1 || c.num_heads < 1 || c.row_bytes < 1 || c.num_pages < 1 || c.num_pages > INT32_MAX)
            return fail(FDEC_ERR_INVALID_ARG, "a cache needs layers, heads, bytes in a row and 1 .. 2^31-1 pages");
        if (c.reserved != 0) return fail(FDEC_ERR_INVALID_ARG, "reserved fields must be 0");
        const int64_t strides[4] = {c.stride_layer, c.stride_page, c.stride_head, c.stride_token};
        bool wide = aligned(c.base, 16) && c.row_bytes % 16 == 0;
        if (!aligned(c.base, 8) || c.row_bytes % 8 != 0)
            return fail(FDEC_ERR_LAYOUT, "caches must hold rows of multiples of 8 bytes, 8-byte aligned");
        for (const int64_t s : strides) {
            if (s < 0 || s % 8 != 0) return fail(FDEC_ERR_LAYOUT, "cache strides must be non-negative multiples of 8 bytes");
            wide = wide && s % 16 == 0;
        }
        if ((c.num_layers > 1 && c.stride_layer == 0) || (c.num_pages > 1 && c.stride_page == 0) ||
            (c.num_heads > 1 && c.stride_head == 0) || (page_size > 1 && c.stride_token == 0))
            return fail(FDEC_ERR_LAYOUT, "a cache's rows must not lie on one another (a stride of 0)");
        for (int j = 0; j < i; ++j)
            if (caches[j].base == c.base) return fail(FDEC_ERR_INVALID_ARG, "a cache is given twice");
        CacheRows& r = out->c[i];
        r.base = static_cast<uint8_t*>(c.base);
        r.s_layer = c.stride_layer;
        r.s_page = c.stride_page;
        r.s_head = c.stride_head;
        r.s_token = c.stride_token;
        r.layers = c.num_layers;
        r.heads = c.num_heads;
        r.row_vecs = c.row_bytes / (wide ? 16 : 8);
        r.wide = wide;
        r.first_block = static_cast<int>(blocks);
        const int64_t columns = static_cast<int64_t>(c.num_layers) * c.num_heads;
        if (columns > INT32_MAX / r.row_vecs) return fail(FDEC_ERR_UNSUPPORTED, "too many rows at a position");
        blocks += (columns * r.row_vecs + kColumnThreads - 1) / kColumnThreads;
        if (blocks > 1 << 24) return fail(FDEC_ERR_UNSUPPORTED, "too many rows at a position");
        *fewest = std::min(*fewest, c.num_pages);
    }
    return FDEC_OK;
}

}  // namespace

extern "C" {

fdec_status fdec_tree_attention(const void* q, int64_t q_stride_tok, int64_t q_stride_head, fdec_kv_desc k,
                                fdec_kv_desc v, const int32_t* page_table, int64_t page_table_stride,
                                const int32_t* prefix_lens, const int32_t* node_counts, const int32_t* parents,
                                int batch, int num_nodes, int page_size, int num_qo_heads, int num_kv_heads,
                                int head_dim, fdec_dtype dtype, int kv_dtype, float scale, float k_scale, float v_scale,
                                const float* o_prefix, const float* lse_prefix, void* out, int out_type, float* lse,
                                uint32_t* device_errors, cudaStream_t stream) {
    clear_failure();
    fdec_status st = check_tree(batch, num_nodes);
    if (st != FDEC_OK) return st;
    if (num_kv_heads < 1 || num_qo_heads < 1 || num_qo_heads % num_kv_heads != 0)
        return fail(FDEC_ERR_INVALID_ARG, "num_qo_heads must be a positive multiple of num_kv_heads >= 1");
    if (num_qo_heads > 65536) return fail(FDEC_ERR_UNSUPPORTED, "too many heads");
    if (dtype != FDEC_F16 && dtype != FDEC_BF16)
        return fail(FDEC_ERR_INVALID_ARG, "dtype must be FDEC_F16 or FDEC_BF16");
    if (kv_dtype != FDEC_KV_SAME && kv_dtype != FDEC_KV_E4M3)
        return fail(kv_dtype == FDEC_KV_Q8_0 ? FDEC_ERR_UNSUPPORTED : FDEC_ERR_INVALID_ARG,
                    "kv_dtype must be FDEC_KV_SAME or FDEC_KV_E4M3");
    if (head_dim != 64 && head_dim != 128 && head_dim != 192 && head_dim != 256 && head_dim != 512)
        return fail(FDEC_ERR_UNSUPPORTED, "head_dim must be one of 64, 128, 192, 256, 512");
    const bool kv8 = kv_dtype == FDEC_KV_E4M3;
    if (kv8 && head_dim != 128 && head_dim != 256)
        return fail(FDEC_ERR_UNSUPPORTED, "E4M3 caches support head_dim 128 and 256");
    if (page_shift_of(page_size) < 0)
        return fail(FDEC_ERR_UNSUPPORTED, "page_size must be a power of two in [1, 256]");
    if (page_table_stride < 1) return fail(FDEC_ERR_INVALID_ARG, "page_table_stride must be >= 1");
    if (out_type != FDEC_OUT_F32 && out_type != FDEC_OUT_SAME)
        return fail(FDEC_ERR_INVALID_ARG, "out_type must be FDEC_OUT_F32 or FDEC_OUT_SAME");
    const float scale_log2 = scale * k_scale * 1.4426950408889634074f;
    if (!std::isfinite(scale) || !std::isfinite(k_scale) || !std::isfinite(v_scale) || !std::isfinite(scale_log2))
        return fail(FDEC_ERR_INVALID_ARG, "scale, k_scale and v_scale must be finite");
    if (q == nullptr || page_table == nullptr || prefix_lens == nullptr || out == nullptr)
        return fail(FDEC_ERR_INVALID_ARG, "null q, page_table, prefix_lens or out");
    if ((o_prefix == nullptr) != (lse_prefix == nullptr))
        return fail(FDEC_ERR_INVALID_ARG, "o_prefix and lse_prefix come together");
    if (!aligned(q, 16) || q_stride_tok < 0 || q_stride_head < 0 || q_stride_tok % 8 != 0 || q_stride_head % 8 != 0)
        return fail(FDEC_ERR_LAYOUT, "q rows must start on 16-byte boundaries");
    if (!aligned(out, 16) || !aligned(o_prefix, 16)) return fail(FDEC_ERR_LAYOUT, "out and o_prefix must be 16-byte aligned");
    if (!aligned(lse, 4) || !aligned(lse_prefix, 4) || !aligned(page_table, 4) || !aligned(prefix_lens, 4) ||
        !aligned(node_counts, 4) || !aligned(parents, 4) || !aligned(device_errors, 4))
        return fail(FDEC_ERR_LAYOUT, "misaligned lse or index array");
    st = check_pool(k, kv8 ? 1 : 2);
    if (st == FDEC_OK) st = check_pool(v, kv8 ? 1 : 2);
    if (st != FDEC_OK) return st;
    const size_t rows = static_cast<size_t>(batch) * num_nodes * num_qo_heads;
    const size_t out_bytes = rows * head_dim * (out_type == FDEC_OUT_F32 ? 4 : 2);
    if (o_prefix != nullptr && !(out == o_prefix && out_type == FDEC_OUT_F32) &&
        overlap(out, out_bytes, o_prefix, rows * head_dim * 4))
        return fail(FDEC_ERR_INVALID_ARG, "out overlaps o_prefix and is not o_prefix in fp32");
    const size_t q_bytes = (static_cast<size_t>(batch) * num_nodes - 1) * q_stride_tok * 2 +
                           static_cast<size_t>(num_qo_heads - 1) * q_stride_head * 2 + head_dim * 2;
    if (overlap(out, out_bytes, q, q_bytes)) return fail(FDEC_ERR_INVALID_ARG, "out overlaps q");
    if (lse != nullptr && (overlap(lse, rows * 4, out, out_bytes) || overlap(lse, rows * 4, q, q_bytes) ||
                           (o_prefix != nullptr && overlap(lse, rows * 4, o_prefix, rows * head_dim * 4))))
        return fail(FDEC_ERR_INVALID_ARG, "lse overlaps out, q or o_prefix");
    if (lse_prefix != nullptr && overlap(out, out_bytes, lse_prefix, rows * 4))
        return fail(FDEC_ERR_INVALID_ARG, "out overlaps lse_prefix");
    if (lse != nullptr && lse_prefix != nullptr && lse != lse_prefix && overlap(lse, rows * 4, lse_prefix, rows * 4))
        return fail(FDEC_ERR_INVALID_ARG, "lse overlaps lse_prefix and is not lse_prefix");
    const int eb = kv8 ? 1 : 2;
    TreeParams p = {};
    p.q = static_cast<const uint16_t*>(q);
    p.q_st = q_stride_tok;
    p.q_sh = q_stride_head;
    p.k_base = static_cast<const uint8_t*>(k.base);
    p.k_pages = k.num_pages;
    p.k_sp = k.stride_page * eb;
    p.k_sh = k.stride_head * eb;
    p.k_st = k.stride_token * eb;
    p.v_base = static_cast<const uint8_t*>(v.base);
    p.v_pages = v.num_pages;
    p.v_sp = v.stride_page * eb;
    p.v_sh = v.stride_head * eb;
    p.v_st = v.stride_token * eb;
    p.page_table = page_table;
    p.pt_stride = page_table_stride;
    p.pt_cols = table_columns(page_table_stride);
    p.prefix_lens = prefix_lens;
    p.node_counts = node_counts;
    p.parents = parents;
    p.o_prefix = o_prefix;
    p.lse_prefix = lse_prefix;
    p.out = static_cast<float*>(out);
    p.lse = lse;
    p.err = device_errors;
    p.batch = batch;
    p.nodes = num_nodes;
    p.hq = num_qo_heads;
    p.hk = num_kv_heads;
    p.group = num_qo_heads / num_kv_heads;
    p.page_shift = page_shift_of(page_size);
    p.out_type = out_type == FDEC_OUT_F32 ? kOutF32 : dtype == FDEC_BF16 ? kOutBF16 : kOutF16;
    // (never 0: a masked logit, -inf, times it stays -inf)
    p.scale_log2 = scale_log2 == 0.f ? 1e-38f : scale_log2;
    p.v_scale = v_scale;
    if (static_cast<int64_t>(batch) * num_nodes * num_qo_heads > INT32_MAX)
        return fail(FDEC_ERR_UNSUPPORTED, "batch x num_nodes x num_qo_heads must be below 2^31");
    if (checks_only()) return static_cast<fdec_status>(kChecksOnly);
    int num_sms = 0;
    cudaError_t e = current_num_sms(&num_sms);
    if (e == cudaSuccess) e = launch_tree_attention(p, head_dim, dtype == FDEC_BF16, kv8, num_sms, stream);
    if (e != cudaSuccess) return fail_cuda(e, "launching the tree attention");
    return FDEC_OK;
}

fdec_status fdec_verify_drafts(const void* target_probs, int64_t target_stride_seq, int64_t target_stride_node,
                               const void* draft_probs, int64_t draft_stride_seq, int64_t draft_stride_node,
                               int prob_dtype, const int32_t* tokens, const int32_t* parents,
                               const int32_t* node_counts, const float* uniforms, int batch, int num_nodes, int vocab,
                               int32_t* path, int32_t* path_lens, int32_t* out_tokens, uint32_t* device_errors,
                               cudaStream_t stream) {
    clear_failure();
    fdec_status st = check_tree(batch, num_nodes);
    if (st != FDEC_OK) return st;
    if (batch > 1 << 20) return fail(FDEC_ERR_UNSUPPORTED, "batch must be at most 2^20");
    if (prob_dtype != FDEC_PROB_F16 && prob_dtype != FDEC_PROB_BF16 && prob_dtype != FDEC_PROB_F32)
        return fail(FDEC_ERR_INVALID_ARG, "prob_dtype must be FDEC_PROB_F16, FDEC_PROB_BF16 or FDEC_PROB_F32");
    if (vocab < 1) return fail(FDEC_ERR_INVALID_ARG, "vocab must be >= 1");
    if (vocab > 1 << 24) return fail(FDEC_ERR_UNSUPPORTED, "vocab must be at most 2^24");
    if (target_probs == nullptr || tokens == nullptr || uniforms == nullptr || path == nullptr || path_lens == nullptr ||
        out_tokens == nullptr)
        return fail(FDEC_ERR_INVALID_ARG, "null target_probs, tokens, uniforms, path, path_lens or out_tokens");
    const int eb = prob_dtype == FDEC_PROB_F32 ? 4 : 2;
    if (!aligned(target_probs, eb) || !aligned(draft_probs, eb) || target_stride_seq < 0 || target_stride_node < 0 ||
        draft_stride_seq < 0 || draft_stride_node < 0)
        return fail(FDEC_ERR_LAYOUT, "misaligned probabilities or a negative stride");
    if (!aligned(tokens, 4) || !aligned(parents, 4) || !aligned(node_counts, 4) || !aligned(uniforms, 4) ||
        !aligned(path, 4) || !aligned(path_lens, 4) || !aligned(out_tokens, 4) || !aligned(device_errors, 4))
        return fail(FDEC_ERR_LAYOUT, "misaligned array");
    // Every sequence's nodes are read before its results are written: arrays of one shape may be the same one.
    const size_t line = static_cast<size_t>(batch) * 4, grid = line * num_nodes;
    const Span nodes[3] = {{tokens, grid}, {parents, grid}, {uniforms, grid}};
    const auto probs = [&](const void* base, int64_t seq, int64_t node, int rows) {
        return Span{base, (static_cast<size_t>(batch - 1) * seq + static_cast<size_t>(rows - 1) * node + vocab) * eb};
    };
    const Span rows[2] = {probs(target_probs, target_stride_seq, target_stride_node, num_nodes),
                          num_nodes == 1 ? Span{}
                                         : probs(draft_probs, draft_stride_seq, draft_stride_node, num_nodes - 1)};
    for (const void* result : {static_cast<const void*>(path), static_cast<const void*>(out_tokens)}) {
        const Span r = {result, grid};
        for (const Span& in : nodes)
            if (in.base != result && clash(r, in))
                return fail(FDEC_ERR_INVALID_ARG, "path or out_tokens overlaps tokens, parents or uniforms and is not "
                                                  "that array");
        if (clash(r, Span{node_counts, line}) || clash(r, rows))
            return fail(FDEC_ERR_INVALID_ARG, "path or out_tokens overlaps node_counts or probabilities");
    }
    const Span lens = {path_lens, line};
    if (clash(lens, nodes) || clash(lens, rows) || (node_counts != path_lens && clash(lens, Span{node_counts, line})))
        return fail(FDEC_ERR_INVALID_ARG, "path_lens overlaps an input and is not node_counts");
    if (clash(Span{path, grid}, Span{out_tokens, grid}) || clash(lens, {Span{path, grid}, Span{out_tokens, grid}}))
        return fail(FDEC_ERR_INVALID_ARG, "path, path_lens and out_tokens must not overlap");
    VerifyParams p = {};
    p.target = target_probs;
    p.t_seq = target_stride_seq;
    p.t_node = target_stride_node;
    p.draft = draft_probs;
    p.d_seq = draft_probs != nullptr ? draft_stride_seq : 0;
    p.d_node = draft_probs != nullptr ? draft_stride_node : 0;
    p.tokens = tokens;
    p.parents = parents;
    p.node_counts = node_counts;
    p.uniforms = uniforms;
    p.path = path;
    p.path_lens = path_lens;
    p.out_tokens = out_tokens;
    p.err = device_errors;
    p.batch = batch;
    p.nodes = num_nodes;
    p.vocab = vocab;
    if (checks_only()) return static_cast<fdec_status>(kChecksOnly);
    const cudaError_t e = launch_verify_drafts(p, prob_dtype, stream);
    if (e != cudaSuccess) return fail_cuda(e, "launching the verification");
    return FDEC_OK;
}

fdec_status fdec_keep_path(const fdec_cache* caches, int num_caches, const int32_t* page_table, int batch,
                           int64_t page_table_stride, int page_size, const int32_t* prefix_lens, const int32_t* path,
                           int64_t path_stride, const int32_t* path_lens, int num_nodes, int32_t* seq_lens,
                           uint32_t* device_errors, cudaStream_t stream) {
    clear_failure();
    fdec_status st = check_tree(batch, num_nodes);
    if (st != FDEC_OK) return st;
    if (num_caches < 1) return fail(FDEC_ERR_INVALID_ARG, "need a cache");
    if (page_shift_of(page_size) < 0)
        return fail(FDEC_ERR_UNSUPPORTED, "page_size must be a power of two in [1, 256]");
    if (page_table_stride < 1 || path_stride < num_nodes)
        return fail(FDEC_ERR_INVALID_ARG, "need page_table_stride >= 1 and path_stride >= num_nodes");
    if (page_table == nullptr || prefix_lens == nullptr || path == nullptr || path_lens == nullptr || seq_lens == nullptr)
        return fail(FDEC_ERR_INVALID_ARG, "null page_table, prefix_lens, path, path_lens or seq_lens");
    if (!aligned(page_table, 4) || !aligned(prefix_lens, 4) || !aligned(path, 4) || !aligned(path_lens, 4) ||
        !aligned(seq_lens, 4) || !aligned(device_errors, 4))
        return fail(FDEC_ERR_LAYOUT, "misaligned index array");
    const size_t bytes = static_cast<size_t>(batch) * 4;
    const int64_t cols = table_columns(page_table_stride);
    if (clash(Span{seq_lens, bytes}, {Span{prefix_lens, bytes}, Span{path_lens, bytes},
                                      Span{path, table_bytes(batch, path_stride, num_nodes)},
                                      Span{page_table, table_bytes(batch, page_table_stride, cols)}}))
        return fail(FDEC_ERR_INVALID_ARG, "seq_lens overlaps prefix_lens, path, path_lens or page_table");
    CacheList<kMaxCaches> list;
    KeepParams p = {};
    st = take_caches(caches, num_caches, page_size, &list, &p.num_pages);
    if (st != FDEC_OK) return st;
    p.page_table = page_table;
    p.pt_stride = page_table_stride;
    p.pt_cols = cols;
    p.prefix_lens = prefix_lens;
    p.path = path;
    p.path_stride = path_stride;
    p.path_lens = path_lens;
    p.seq_lens = seq_lens;
    p.err = device_errors;
    p.batch = batch;
    p.nodes = num_nodes;
    p.page_shift = page_shift_of(page_size);
    if (checks_only()) return static_cast<fdec_status>(kChecksOnly);
    const cudaError_t e = launch_keep_path(p, list, stream);
    if (e != cudaSuccess) return fail_cuda(e, "launching the path's moves");
    return FDEC_OK;
}

namespace {

// Workspace of fdec_reserve_pages: two bit sets, pages in use by blocks, the sequences' last pages and copies.
struct ReserveLayout {
    size_t off_shared, off_taken, off_last, off_copies, bytes;
    int words, blocks;
};

bool reserve_layout(int batch, int64_t num_pages, ReserveLayout* out) {
    if (batch < 1 || num_pages < 1 || num_pages > 1 << 26) return false;
    out->words = static_cast<int>((num_pages + 31) / 32);
    out->off_shared = static_cast<size_t>(out->words) * 4;
    out->blocks = static_cast<int>((num_pages + kCountedPages - 1) / kCountedPages);
    out->off_taken = 2 * out->off_shared;
    out->off_last = out->off_taken + static_cast<size_t>(out->blocks) * 4;
    out->off_copies = (out->off_last + static_cast<size_t>(batch) * 4 + 15) / 16 * 16;
    out->bytes = (out->off_copies + static_cast<size_t>(batch) * 16 + 255) / 256 * 256;
    return true;
}

}  // namespace

fdec_status fdec_reserve_pages_workspace(int batch, int64_t num_pages, size_t* workspace_bytes) {
    clear_failure();
    if (workspace_bytes == nullptr) return fail(FDEC_ERR_INVALID_ARG, "null output pointer");
    *workspace_bytes = 0;
    ReserveLayout l;
    if (!reserve_layout(batch, num_pages, &l))
        return fail(FDEC_ERR_INVALID_ARG, "batch must be >= 1 and num_pages in [1, 2^26]");
    *workspace_bytes = l.bytes;
    return FDEC_OK;
}

fdec_status fdec_reserve_pages(int32_t* page_table, int batch, int64_t page_table_stride, int page_size,
                               const int32_t* seq_lens, const int32_t* new_lens, const int32_t* sources,
                               int32_t* granted, int64_t num_pages, const fdec_cache* caches, int num_caches,
                               void* workspace, size_t workspace_bytes, uint32_t* device_errors, cudaStream_t stream) {
    clear_failure();
    if (batch < 1 || page_table_stride < 1) return fail(FDEC_ERR_INVALID_ARG, "need batch >= 1, page_table_stride >= 1");
    if (batch > 1 << 16) return fail(FDEC_ERR_UNSUPPORTED, "batch must be at most 65536");
    const int shift = page_shift_of(page_size);
    if (shift < 0) return fail(FDEC_ERR_UNSUPPORTED, "page_size must be a power of two in [1, 256]");
    if (page_table_stride > INT32_MAX) return fail(FDEC_ERR_UNSUPPORTED, "page_table_stride must be below 2^31");
    ReserveLayout l;
    if (!reserve_layout(batch, num_pages, &l)) return fail(FDEC_ERR_INVALID_ARG, "num_pages must be in [1, 2^26]");
    if (page_table == nullptr || seq_lens == nullptr || new_lens == nullptr || granted == nullptr)
        return fail(FDEC_ERR_INVALID_ARG, "null page_table, seq_lens, new_lens or granted");
    if (!aligned(page_table, 4) || !aligned(seq_lens, 4) || !aligned(new_lens, 4) || !aligned(sources, 4) ||
        !aligned(granted, 4) || !aligned(device_errors, 4))
        return fail(FDEC_ERR_LAYOUT, "misaligned index array");
    const size_t bytes = static_cast<size_t>(batch) * 4;
    const int64_t cols = table_columns(page_table_stride);
    const Span inputs[3] = {{seq_lens, bytes}, {new_lens, bytes}, {sources, bytes}};
    const Span table = {page_table, table_bytes(batch, page_table_stride, cols)};
    if (clash(Span{granted, bytes}, inputs) || clash(Span{granted, bytes}, table))
        return fail(FDEC_ERR_INVALID_ARG, "granted overlaps seq_lens, new_lens, sources or page_table");
    if (clash(table, inputs))
        return fail(FDEC_ERR_INVALID_ARG, "page_table overlaps seq_lens, new_lens or sources");
    if (workspace == nullptr || !aligned(workspace, 256) || workspace_bytes < l.bytes)
        return fail(FDEC_ERR_WORKSPACE, "workspace missing, not 256-byte aligned or smaller than "
                                        "fdec_reserve_pages_workspace says");
    if (clash(Span{workspace, l.bytes}, inputs) || clash(Span{workspace, l.bytes}, {table, Span{granted, bytes}}))
        return fail(FDEC_ERR_INVALID_ARG, "workspace overlaps another array");
    CacheList<kMaxCaches> list;
    int64_t fewest = 0;
    const fdec_status st = take_caches(caches, num_caches, page_size, &list, &fewest);
    if (st != FDEC_OK) return st;
    if (num_pages > fewest) return fail(FDEC_ERR_INVALID_ARG, "num_pages is more than a cache has");
    ReserveParams p = {};
    p.page_table = page_table;
    p.pt_stride = page_table_stride;
    p.pt_cols = cols;
    p.seq_lens = seq_lens;
    p.new_lens = new_lens;
    p.sources = sources;
    p.granted = granted;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.used = reinterpret_cast<unsigned*>(ws);
    p.shared = reinterpret_cast<unsigned*>(ws + l.off_shared);
    p.taken = reinterpret_cast<int32_t*>(ws + l.off_taken);
    p.blocks = l.blocks;
    p.last_page = reinterpret_cast<int32_t*>(ws + l.off_last);
    p.copies = reinterpret_cast<int4*>(ws + l.off_copies);
    p.err = device_errors;
    p.num_pages = num_pages;
    p.words = l.words;
    p.batch = batch;
    p.page_shift = shift;
    if (checks_only()) return static_cast<fdec_status>(kChecksOnly);
    int num_sms = 0;
    cudaError_t e = current_num_sms(&num_sms);
    if (e == cudaSuccess) e = launch_reserve_pages(p, list, num_sms, stream);
    if (e != cudaSuccess) return fail_cuda(e, "launching the page reservation");
    return FDEC_OK;
}

}  // extern "C"
