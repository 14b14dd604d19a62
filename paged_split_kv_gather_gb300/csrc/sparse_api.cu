// sparse_api.cu -- entry points of block-sparse decoding: argument checks of
// fdec_norm_rope_append, fdec_page_bounds and fdec_select_pages.  (The attention over
// the selected pages, fdec_run_selected, runs a plan and lives with the plans.)
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/fdec.h"
#include "fdec_internal.h"

using namespace fdec;

namespace {

fdec_status fail(fdec_status st, const char* msg) { return static_cast<fdec_status>(record_failure(st, msg)); }

fdec_status fail_cuda(cudaError_t e, const char* what) { return static_cast<fdec_status>(record_cuda_failure(e, what)); }

bool head_dim_ok(int d) { return d == 64 || d == 128 || d == 192 || d == 256 || d == 512; }

// log2 of a page size, -1 if it is none that the library takes.
int page_shift_of(int page_size) {
    for (int s = 0; s <= 8; ++s)
        if (page_size == 1 << s) return s;
    return -1;
}

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
bool aligned4(const void* p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }

fdec_status check_common(int batch, int num_kv_heads, int head_dim, int page_size, fdec_dtype dtype, int kv_dtype) {
    if (batch < 1 || num_kv_heads < 1) return fail(FDEC_ERR_INVALID_ARG, "batch and num_kv_heads must be >= 1");
    if (dtype != FDEC_F16 && dtype != FDEC_BF16)
        return fail(FDEC_ERR_INVALID_ARG, "dtype must be FDEC_F16 or FDEC_BF16");
    if (kv_dtype != FDEC_KV_SAME && kv_dtype != FDEC_KV_E4M3)
        return fail(kv_dtype == FDEC_KV_Q8_0 ? FDEC_ERR_UNSUPPORTED : FDEC_ERR_INVALID_ARG,
                    "kv_dtype must be FDEC_KV_SAME or FDEC_KV_E4M3");
    if (!head_dim_ok(head_dim)) return fail(FDEC_ERR_UNSUPPORTED, "head_dim must be one of 64, 128, 192, 256, 512");
    if (kv_dtype == FDEC_KV_E4M3 && head_dim != 128 && head_dim != 256)
        return fail(FDEC_ERR_UNSUPPORTED, "E4M3 caches support head_dim 128 and 256");
    if (page_shift_of(page_size) < 0)
        return fail(FDEC_ERR_UNSUPPORTED, "page_size must be a power of two in [1, 256]");
    return FDEC_OK;
}

// A pool of rows of 16-byte multiples (eb bytes an element).
fdec_status check_pool(const fdec_kv_desc& d, int eb) {
    if (d.base == nullptr) return fail(FDEC_ERR_INVALID_ARG, "null pool");
    if (d.num_pages < 1 || d.num_pages > INT32_MAX) return fail(FDEC_ERR_INVALID_ARG, "pools need 1 .. 2^31-1 pages");
    const int64_t unit = 16 / eb;
    if (!aligned16(d.base)) return fail(FDEC_ERR_LAYOUT, "pools must be 16-byte aligned");
    if (d.stride_page < 0 || d.stride_head < 0 || d.stride_token < 0 || d.stride_page % unit != 0 ||
        d.stride_head % unit != 0 || d.stride_token % unit != 0)
        return fail(FDEC_ERR_LAYOUT, "pool strides must be non-negative multiples of 16 bytes");
    return FDEC_OK;
}

fdec_status check_rows(const fdec_rows& r) {
    if (r.base == nullptr) return fail(FDEC_ERR_INVALID_ARG, "null rows");
    if (!aligned16(r.base) || r.stride_tok < 0 || r.stride_head < 0 || r.stride_tok % 8 != 0 || r.stride_head % 8 != 0)
        return fail(FDEC_ERR_LAYOUT, "rows must start on 16-byte boundaries");
    return FDEC_OK;
}

}  // namespace

extern "C" {

fdec_status fdec_norm_rope_append(fdec_rows q, fdec_rows k_new, fdec_rows v_new, const void* q_weight,
                                  const void* k_weight, float eps, const float* cos_sin, int64_t cos_sin_rows,
                                  int rot_dim, int interleaved, const int32_t* batch_indices, const int32_t* positions,
                                  const int32_t* rope_positions, int n_tokens, int num_qo_heads, int num_kv_heads,
                                  int head_dim, int page_size, fdec_dtype dtype, int kv_dtype, float k_scale,
                                  float v_scale, fdec_rows q_out, fdec_kv_desc k, fdec_kv_desc v,
                                  const int32_t* page_table, int batch, int64_t page_table_stride,
                                  uint32_t* device_errors, cudaStream_t stream) {
    clear_failure();
    fdec_status st = check_common(batch, num_kv_heads, head_dim, page_size, dtype, kv_dtype);
    if (st != FDEC_OK) return st;
    if (n_tokens < 0 || num_qo_heads < 1 || page_table_stride < 1)
        return fail(FDEC_ERR_INVALID_ARG, "need n_tokens >= 0, num_qo_heads >= 1, page_table_stride >= 1");
    if (num_qo_heads > 65536 || num_kv_heads > 65536) return fail(FDEC_ERR_UNSUPPORTED, "too many heads");
    if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(FDEC_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (rot_dim < 0 || rot_dim > head_dim || rot_dim % 16 != 0)
        return fail(FDEC_ERR_INVALID_ARG, "rot_dim must be a multiple of 16 in [0, head_dim]");
    if (rot_dim > 0 && (cos_sin == nullptr || cos_sin_rows < 1))
        return fail(FDEC_ERR_INVALID_ARG, "rot_dim > 0 needs a cos_sin table");
    const bool kv8 = kv_dtype == FDEC_KV_E4M3;
    const auto scale_ok = [](float x) { return x > 0.f && std::isfinite(x) && std::isfinite(1.f / x); };
    if (kv8 ? !scale_ok(k_scale) || !scale_ok(v_scale) : (k_scale != 1.f || v_scale != 1.f))
        return fail(FDEC_ERR_INVALID_ARG,
                    "k_scale and v_scale must be > 0 with a finite reciprocal (and 1 for a 16-bit cache)");
    if (n_tokens == 0) return FDEC_OK;
    if (batch_indices == nullptr || positions == nullptr || page_table == nullptr)
        return fail(FDEC_ERR_INVALID_ARG, "null batch_indices, positions or page_table");
    const fdec_rows* rows[4] = {&q, &k_new, &v_new, &q_out};
    for (const fdec_rows* r : rows) {
        st = check_rows(*r);
        if (st != FDEC_OK) return st;
    }
    const int eb = kv8 ? 1 : 2;
    st = check_pool(k, eb);
    if (st == FDEC_OK) st = check_pool(v, eb);
    if (st != FDEC_OK) return st;
    if (!aligned16(q_weight) || !aligned16(k_weight) || !aligned16(cos_sin))
        return fail(FDEC_ERR_LAYOUT, "weights and cos_sin must be 16-byte aligned");
    if (!aligned4(batch_indices) || !aligned4(positions) || !aligned4(rope_positions) || !aligned4(page_table) ||
        !aligned4(device_errors))
        return fail(FDEC_ERR_LAYOUT, "misaligned index array");
    NormRopeParams p;
    p.q = static_cast<const uint8_t*>(q.base);
    p.q_st = q.stride_tok * 2;
    p.q_sh = q.stride_head * 2;
    p.k_new = static_cast<const uint8_t*>(k_new.base);
    p.k_new_st = k_new.stride_tok * 2;
    p.k_new_sh = k_new.stride_head * 2;
    p.v_new = static_cast<const uint8_t*>(v_new.base);
    p.v_new_st = v_new.stride_tok * 2;
    p.v_new_sh = v_new.stride_head * 2;
    p.q_weight = static_cast<const uint16_t*>(q_weight);
    p.k_weight = static_cast<const uint16_t*>(k_weight);
    p.cos_sin = cos_sin;
    p.cos_rows = cos_sin_rows;
    p.batch_indices = batch_indices;
    p.positions = positions;
    p.rope_positions = rope_positions;
    p.q_out = static_cast<uint8_t*>(const_cast<void*>(q_out.base));
    p.q_out_st = q_out.stride_tok * 2;
    p.q_out_sh = q_out.stride_head * 2;
    p.page_table = page_table;
    p.pt_stride = page_table_stride;
    p.k_base = static_cast<uint8_t*>(const_cast<void*>(k.base));
    p.k_pages = k.num_pages;
    p.k_sp = k.stride_page * eb;
    p.k_sh = k.stride_head * eb;
    p.k_st = k.stride_token * eb;
    p.v_base = static_cast<uint8_t*>(const_cast<void*>(v.base));
    p.v_pages = v.num_pages;
    p.v_sp = v.stride_page * eb;
    p.v_sh = v.stride_head * eb;
    p.v_st = v.stride_token * eb;
    p.err = device_errors;
    p.n_tokens = n_tokens;
    p.batch = batch;
    p.hq = num_qo_heads;
    p.hk = num_kv_heads;
    p.page_shift = page_shift_of(page_size);
    p.rot = rot_dim;
    p.eps = eps;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.k_inv = 1.f / k_scale;
    p.v_inv = 1.f / v_scale;
    if (checks_only()) return static_cast<fdec_status>(kChecksOnly);
    int num_sms = 0;
    cudaError_t e = current_num_sms(&num_sms);
    if (e == cudaSuccess) e = launch_norm_rope(p, head_dim, dtype == FDEC_BF16, kv8, interleaved != 0, num_sms, stream);
    if (e != cudaSuccess) return fail_cuda(e, "launching the norm, rotation and append");
    return FDEC_OK;
}

fdec_status fdec_page_bounds(fdec_kv_desc k, fdec_kv_desc bounds, const int32_t* page_table, int batch,
                             int64_t page_table_stride, const int32_t* begins, const int32_t* seq_lens_dev,
                             int num_kv_heads, int head_dim, int page_size, fdec_dtype dtype, int kv_dtype,
                             int expected_tokens, uint32_t* device_errors, cudaStream_t stream) {
    clear_failure();
    fdec_status st = check_common(batch, num_kv_heads, head_dim, page_size, dtype, kv_dtype);
    if (st != FDEC_OK) return st;
    if (page_table_stride < 1 || expected_tokens < 0)
        return fail(FDEC_ERR_INVALID_ARG, "need page_table_stride >= 1, expected_tokens >= 0");
    if (page_table == nullptr || seq_lens_dev == nullptr)
        return fail(FDEC_ERR_INVALID_ARG, "null page_table or seq_lens");
    const int eb = kv_dtype == FDEC_KV_E4M3 ? 1 : 2;
    st = check_pool(k, eb);
    if (st == FDEC_OK) st = check_pool(bounds, 2);
    if (st != FDEC_OK) return st;
    if (!aligned4(page_table) || !aligned4(begins) || !aligned4(seq_lens_dev) || !aligned4(device_errors))
        return fail(FDEC_ERR_LAYOUT, "misaligned index array");
    BoundsParams p;
    p.k_base = static_cast<const uint8_t*>(k.base);
    p.k_pages = k.num_pages;
    p.k_sp = k.stride_page * eb;
    p.k_sh = k.stride_head * eb;
    p.k_st = k.stride_token * eb;
    p.b_base = static_cast<uint8_t*>(const_cast<void*>(bounds.base));
    p.b_pages = bounds.num_pages;
    p.b_sp = bounds.stride_page * 2;
    p.b_sh = bounds.stride_head * 2;
    p.b_st = bounds.stride_token * 2;
    p.page_table = page_table;
    p.pt_stride = page_table_stride;
    p.begins = begins;
    p.seq_lens = seq_lens_dev;
    p.err = device_errors;
    p.batch = batch;
    p.hk = num_kv_heads;
    p.page_shift = page_shift_of(page_size);
    // Pages of a sequence that the launch has CTAs for: those of expected_tokens tokens
    // that begin inside a page, as many as a grid holds; the kernel walks the rest.
    const int64_t pages = (static_cast<int64_t>(expected_tokens) + page_size - 1) / page_size + (expected_tokens > 1);
    const int64_t most = std::max<int64_t>(1, (int64_t{1} << 30) / (static_cast<int64_t>(batch) * num_kv_heads));
    p.span = static_cast<int>(std::max<int64_t>(1, std::min({pages, page_table_stride, most})));
    if (static_cast<int64_t>(batch) * num_kv_heads > (int64_t{1} << 30))
        return fail(FDEC_ERR_UNSUPPORTED, "batch x num_kv_heads too large");
    if (checks_only()) return static_cast<fdec_status>(kChecksOnly);
    int num_sms = 0;
    cudaError_t e = current_num_sms(&num_sms);
    if (e == cudaSuccess)
        e = launch_page_bounds(p, head_dim, dtype == FDEC_BF16, kv_dtype == FDEC_KV_E4M3, num_sms, stream);
    if (e != cudaSuccess) return fail_cuda(e, "launching the page bounds");
    return FDEC_OK;
}

namespace {

// Workspace of fdec_select_pages: 64-bit keys, scores, magnitudes.
struct SelectLayout {
    size_t off_abs, off_scores, bytes;
    int64_t score_stride;  // floats a row: whole 16-byte vectors
};

bool select_layout(int64_t rows, int64_t max_pages, SelectLayout* out) {
    const auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    if (rows < 1 || max_pages < 1 || rows > INT32_MAX || max_pages > INT32_MAX) return false;
    const size_t n = static_cast<size_t>(rows), m = static_cast<size_t>(max_pages);
    out->score_stride = (max_pages + 3) / 4 * 4;
    out->off_scores = up(n * m * 8);
    out->off_abs = up(out->off_scores + n * static_cast<size_t>(out->score_stride) * 4);
    out->bytes = up(out->off_abs + n * static_cast<size_t>(select_abs_stride(max_pages)) * 4);
    return true;
}

}  // namespace

fdec_status fdec_select_pages_workspace(int batch, int q_len, int num_kv_heads, int64_t max_pages,
                                        size_t* workspace_bytes) {
    clear_failure();
    if (workspace_bytes == nullptr) return fail(FDEC_ERR_INVALID_ARG, "null output pointer");
    *workspace_bytes = 0;
    SelectLayout l;
    if (batch < 1 || q_len < 1 || num_kv_heads < 1 || static_cast<int64_t>(batch) * q_len > INT32_MAX ||
        !select_layout(static_cast<int64_t>(batch) * q_len * num_kv_heads, max_pages, &l))
        return fail(FDEC_ERR_INVALID_ARG, "batch, q_len, num_kv_heads and max_pages must be >= 1 (and rows below 2^31)");
    *workspace_bytes = l.bytes;
    return FDEC_OK;
}

fdec_status fdec_select_pages(const void* q, int64_t q_stride_tok, int64_t q_stride_head, fdec_kv_desc bounds,
                              const int32_t* page_table, int64_t page_table_stride, const int32_t* seq_lens_dev,
                              int batch, int q_len, int page_size, int num_qo_heads, int num_kv_heads, int head_dim,
                              fdec_dtype dtype, int causal, int64_t max_pages, int budget, int first_pages,
                              int last_pages, int32_t* page_ids, int32_t* counts, int32_t* page_indices,
                              void* workspace, size_t workspace_bytes, uint32_t* device_errors, cudaStream_t stream) {
    clear_failure();
    fdec_status st = check_common(batch, num_kv_heads, head_dim, page_size, dtype, FDEC_KV_SAME);
    if (st != FDEC_OK) return st;
    if (q_len < 1) return fail(FDEC_ERR_INVALID_ARG, "q_len must be >= 1");
    if (num_qo_heads < 1 || num_qo_heads % num_kv_heads != 0)
        return fail(FDEC_ERR_INVALID_ARG, "num_qo_heads must be a positive multiple of num_kv_heads");
    if (max_pages < 1 || max_pages > page_table_stride)
        return fail(FDEC_ERR_CAPACITY, "max_pages must be in [1, page_table_stride]");
    if (max_pages * page_size > INT32_MAX) return fail(FDEC_ERR_UNSUPPORTED, "max_pages x page_size must be below 2^31");
    if (first_pages < 0 || last_pages < 1 || budget < 1 || budget - first_pages < last_pages)
        return fail(FDEC_ERR_INVALID_ARG, "need first_pages >= 0, last_pages >= 1 and budget >= first_pages + last_pages");
    if (q == nullptr || page_table == nullptr || seq_lens_dev == nullptr || page_ids == nullptr || counts == nullptr)
        return fail(FDEC_ERR_INVALID_ARG, "null q, page_table, seq_lens, page_ids or counts");
    if (reinterpret_cast<uintptr_t>(q) % 2 != 0) return fail(FDEC_ERR_LAYOUT, "misaligned q");
    if (!aligned4(page_table) || !aligned4(seq_lens_dev) || !aligned4(page_ids) || !aligned4(counts) ||
        !aligned4(page_indices) || !aligned4(device_errors))
        return fail(FDEC_ERR_LAYOUT, "misaligned index array");
    st = check_pool(bounds, 2);
    if (st != FDEC_OK) return st;
    const int64_t rows = static_cast<int64_t>(batch) * q_len * num_kv_heads;
    SelectLayout l;
    if (static_cast<int64_t>(batch) * q_len > INT32_MAX || !select_layout(rows, max_pages, &l))
        return fail(FDEC_ERR_UNSUPPORTED, "batch x q_len x num_kv_heads must be below 2^31");
    if (workspace == nullptr || reinterpret_cast<uintptr_t>(workspace) % 256 != 0 || workspace_bytes < l.bytes)
        return fail(FDEC_ERR_WORKSPACE, "workspace missing, not 256-byte aligned or smaller than "
                                        "fdec_select_pages_workspace says");
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    SelectParams p;
    p.q = static_cast<const uint16_t*>(q);
    p.q_st = q_stride_tok;
    p.q_sh = q_stride_head;
    p.b_base = static_cast<const uint8_t*>(bounds.base);
    p.b_pages = bounds.num_pages;
    p.b_sp = bounds.stride_page * 2;
    p.b_sh = bounds.stride_head * 2;
    p.b_st = bounds.stride_token * 2;
    p.page_table = page_table;
    p.pt_stride = page_table_stride;
    p.seq_lens = seq_lens_dev;
    p.page_ids = page_ids;
    p.counts = counts;
    p.page_indices = page_indices;
    p.chunk_abs = reinterpret_cast<float*>(ws + l.off_abs);
    p.abs_stride = select_abs_stride(max_pages);
    p.scores = reinterpret_cast<float*>(ws + l.off_scores);
    p.score_stride = l.score_stride;
    p.near_keys = reinterpret_cast<unsigned long long*>(ws);
    p.err = device_errors;
    p.batch = batch;
    p.q_len = q_len;
    p.hk = num_kv_heads;
    p.group = num_qo_heads / num_kv_heads;
    p.page_shift = page_shift_of(page_size);
    p.causal = causal != 0 && q_len > 1;
    p.max_pages = static_cast<int>(max_pages);
    p.budget = budget;
    p.first = first_pages;
    p.last = last_pages;
    p.head_dim = p.chunk = p.n_chunks = p.chain = 0;
    if (checks_only()) return static_cast<fdec_status>(kChecksOnly);
    int num_sms = 0;
    cudaError_t e = current_num_sms(&num_sms);
    if (e == cudaSuccess) e = launch_select_pages(p, head_dim, dtype == FDEC_BF16, num_sms, stream);
    if (e != cudaSuccess) return fail_cuda(e, "launching the page selection");
    return FDEC_OK;
}

}  // extern "C"
