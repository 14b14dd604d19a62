// fdec_internal.h -- kernel parameter blocks and launcher declarations shared by
// the C-ABI layer (fdec_api.cu) and the kernel translation units.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

namespace fdec {

// The split granularity: every split is a run of whole 64-token blocks (the HRX
// decode_split producer runs one workgroup per 64-token KV block).
constexpr int kBlockTokens = 64;
// One pipeline stage carries 32 consecutive tokens of K and V (one per lane).
constexpr int kStageTokens = 32;

// Type of the output rows: fp32 (fdec_run and its kin), or the query's 16-bit type.
enum OutType : int { kOutF32 = 0, kOutBF16 = 1, kOutF16 = 2 };

// Work item of the split kernel: sequence, [block_begin, block_end) in 64-token
// blocks, and the partial slot (-1: the item covers its whole sequence and
// writes out/lse directly).
struct WorkItem {
    int32_t seq;
    int32_t block_begin;
    int32_t block_end;
    int32_t slot;
};

// Reduction task: merge partial slots [src, src + count) of one sequence into
// slot dst of the next level, or into out/lse when dst < 0.
struct ReduceTask {
    int32_t seq;
    int32_t src;
    int32_t count;
    int32_t dst;
};

struct SplitParams {
    const uint16_t* q;
    int64_t q_stride_tok;
    int64_t q_stride_head;
    const uint8_t* k_base;   // byte strides below
    int64_t k_pages, k_sp, k_sh, k_st;
    const uint8_t* v_base;
    int64_t v_pages, v_sp, v_sh, v_st;
    // q8_0 caches: the binary16 block-scale rows (head_dim / 32 per token), byte strides
    const uint8_t* ks_base;
    int64_t ks_sp, ks_sh, ks_st;
    const uint8_t* vs_base;
    int64_t vs_sp, vs_sh, vs_st;
    const int32_t* page_table;
    int64_t pt_stride;
    const int32_t* seq_lens;
    const int32_t* capacity;   // planned capacity per sequence (workspace copy)
    const WorkItem* items;
    float* part_o;             // [slot][Hk][rows][D]
    float2* part_ml;           // [slot][Hk][rows]  (m in log2 units, l)
    float* out;                // [B*Q*Hq][D]
    float* lse;                // [B*Q*Hq] or null
    unsigned* err;
    int q_len, hq, hk, group, rows, page_shift, causal;
    float scale_log2;          // scale * k_scale * log2(e): logits are kept in log2 units
    float v_scale;             // value scale (quantised caches; 1 otherwise), applied to O
    // Persistent split kernel: work units = items x KV heads x row groups, in item
    // order; CTA c starts with unit c and takes the units past the grid from the
    // ticket counter (advanced by exactly n_units per launch).
    int n_units;
    unsigned long long* ticket;
    // One sequence (batch 1): its work items are runs of seq1_bps blocks in order, so
    // a unit's item follows from its index with no table read (0: read the table).
    int seq1_bps, seq1_blocks, seq1_capacity;
};

// fdec_run_selected: page-table row and length seq * hk + kvh are those of the pages that
// KV head kvh of query token seq has selected.  The split kernels are compiled apart for
// these parameters: as run-time branches of one build the differences cost the other
// calls up to 6 us (cold instruction fetches) of a flushed 2048-token decode.
struct SelectedParams : SplitParams {
    int per_head;              // 1: run as selected; 0: as the SplitParams that they contain
    int out_type;              // OutType of `out`
    // Shares: instead of planned items, CTA c takes the c-th of grid equal runs of the
    // 64-token blocks that the lists hold at run time (see split_persist_kernel.cuh).
    // 0: planned items.
    int shares;
    int n_lists;               // batch x hk
    int share_cap;             // the capacity of every sequence if they are equal, else -1
    int2* share_rec;           // [n_lists x row groups] first and last CTA of each unit
    float* share_o;            // [2 grid][16][D] partials: 2 c: a unit begun before CTA c, 2 c + 1: one that goes on
    float2* share_ml;          // [2 grid][16]
};

struct ReduceParams {
    const ReduceTask* tasks;
    const float* src_o;        // [slot][Hk][rows][D]
    const float2* src_ml;      // (m in log2 units, l) per source row
    const float* src_lse;      // natural-log lse per source row when normalized_input
    float* dst_o;
    float2* dst_ml;
    float* out;                // final: [B*Q*Hq][D]
    float* lse;                // final: [B*Q*Hq] or null
    int out_type;              // OutType of `out`
    int hk, rows, group, q_len, hq, head_dim;
    int normalized_input;      // 1: sources are normalised (o, lse) states (merge_states)
    int src_rows_stride;       // rows per (slot, kv head) in the source arrays
    int warps_per_unit;        // 1, 2 or 4 (reduce_warps_per_unit of the largest task)
};

// Launch the split kernel for head_dim D (defined in split_d<D>.cu); rc is the
// compile-time query-row group.  With launch == false only the kernel's
// shared-memory attribute is set (done at upload, outside any capture).
cudaError_t launch_split_d64(const SelectedParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int rc,
                               bool bf16, dim3 grid, cudaStream_t s, bool launch);
cudaError_t launch_split_d128(const SelectedParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int rc,
                               bool bf16, dim3 grid, cudaStream_t s, bool launch);
cudaError_t launch_split_d192(const SelectedParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int rc,
                               bool bf16, dim3 grid, cudaStream_t s, bool launch);
cudaError_t launch_split_d256(const SelectedParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int rc,
                               bool bf16, dim3 grid, cudaStream_t s, bool launch);
cudaError_t launch_split_d512(const SelectedParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int rc,
                               bool bf16, dim3 grid, cudaStream_t s, bool launch);

// The tensor-core split kernel (head_dim 64, 128, 192, 256, 512; query rows in
// groups of 16).  kv8: K/V stored as E4M3 codes (head_dim 128 and 256).
cudaError_t launch_split_mma(const SelectedParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int head_dim,
                             bool bf16, bool kv8, dim3 grid, cudaStream_t s, bool launch);
cudaError_t launch_split_mma_selected(const SelectedParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int head_dim,
                                      bool bf16, bool kv8, dim3 grid, cudaStream_t s, bool launch);
size_t split_mma_smem_bytes(int head_dim, bool kv8);
// The persistent form of the tensor-core split kernel (16-bit caches, every head_dim;
// q rows 16-byte aligned): CTAs stay resident and take work units until none is left,
// so a unit's pipeline fill is paid once per CTA and not once per work item.
cudaError_t launch_split_mma_persist(const SelectedParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int head_dim,
                                     bool bf16, dim3 grid, cudaStream_t s, bool launch);
cudaError_t launch_split_mma_persist_selected(const SelectedParams& p, const CUtensorMap& tk, const CUtensorMap& tv,
                                              int head_dim, bool bf16, dim3 grid, cudaStream_t s, bool launch);
inline bool split_mma_persist_supported(int head_dim) {
    return head_dim == 64 || head_dim == 128 || head_dim == 192 || head_dim == 256 || head_dim == 512;
}
constexpr int split_mma_persist_ctas_per_sm(int head_dim) { return head_dim > 256 ? 1 : 2; }
// Page lists of head_dim 64 with four CTAs an SM: 800 lists of 2048 tokens 75 us against 79
// with three, 99 with two, 77 with five.  (Three at head_dim 128: 148 against 134 with two.)
constexpr int split_mma_persist_ctas_per_sm_selected(int head_dim) {
    return head_dim == 64 ? 4 : split_mma_persist_ctas_per_sm(head_dim);
}
int split_mma_threads(int head_dim, bool kv8);
inline bool split_mma_kv8_supported(int head_dim) { return head_dim == 128 || head_dim == 256; }
// Whether the tensor-core split kernels stage pages smaller than a stage one box per
// page ([box][region][rows][128 B]) rather than region-major: all but 16-bit head_dim
// 512 (MmaLayout / PersistLayout BOXMAJ); their tensor maps then take every region.
inline bool split_mma_box_major(int head_dim, bool kv8) { return kv8 || head_dim <= 256; }
// q8_0 caches (int8 codes in blocks of 32 with one binary16 scale each) on the
// one-CTA-per-item tensor-core kernel, head_dim 128 and 256.
cudaError_t launch_split_mma_q8(const SplitParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int head_dim,
                                bool bf16, dim3 grid, cudaStream_t s, bool launch);
size_t split_mma_q8_smem_bytes(int head_dim);
int split_mma_q8_threads(int head_dim);
constexpr int kMmaRows = 16;

// The tcgen05 dense-query split kernel (head_dim 64, 128, 192, 256; `tiles` 128-row
// query tiles per CTA: 1 or 2 for head_dim 64 and 128, 1 above; 64-token stages: its
// tensor maps use boxes of min(page_size, 64) token rows).
cudaError_t launch_split_tc(const SelectedParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int tiles, int head_dim,
                            bool bf16, dim3 grid, cudaStream_t s, bool launch);
size_t split_tc_smem_bytes(int tiles, int head_dim);
int split_tc_threads(int tiles, bool bf16);
inline bool split_tc_supported(int head_dim) {
    return head_dim == 64 || head_dim == 128 || head_dim == 192 || head_dim == 256;
}
inline int split_tc_max_tiles(int head_dim) { return head_dim <= 128 ? 2 : 1; }
constexpr int kTcRows = 128;
constexpr int kTcStageTokens = 64;

// Shared-memory bytes and threads of the split kernel for (D, RC); 0 if not built.
size_t split_smem_bytes(int head_dim, int rc);
int split_threads(int head_dim);
int split_max_rc(int head_dim);

// Merge of the units that shares have cut (SelectedParams::shares): after the split launch.
struct ShareMergeParams {
    const int2* rec;
    const float* o;            // [2 grid][16][D]
    const float2* ml;          // [2 grid][16]
    float* out;
    float* lse;                // or null
    int out_type, hk, rows, group, hq, head_dim, units, row_groups, grid;
};
cudaError_t launch_share_merge(const ShareMergeParams& p, cudaStream_t s);

int reduce_warps_per_unit(int max_count);
cudaError_t launch_reduce(const ReduceParams& p, int num_tasks, cudaStream_t s);

// Paged KV append (fdec_append, fdec_append_e4m3).  Strides in bytes; every row
// is row_bytes long (a multiple of 16) and starts on a 16-byte boundary.
struct AppendParams {
    const uint8_t* k_new;
    const uint8_t* v_new;
    int64_t new_st, new_sh;
    const int32_t* batch_indices;
    const int32_t* positions;
    const int32_t* page_table;
    int64_t pt_stride;
    uint8_t* k_base;
    int64_t k_pages, k_sp, k_sh, k_st;
    uint8_t* v_base;
    int64_t v_pages, v_sp, v_sh, v_st;
    unsigned* err;
    int n_tokens, batch, hk, row_bytes, page_shift;
};
cudaError_t launch_append(const AppendParams& p, cudaStream_t s);

// Norm, rotation and paged write of new tokens' rows (fdec_norm_rope_append).  Strides
// in bytes; rows start on 16-byte boundaries.
struct NormRopeParams {
    const uint8_t* q;
    int64_t q_st, q_sh;
    const uint8_t* k_new;
    int64_t k_new_st, k_new_sh;
    const uint8_t* v_new;
    int64_t v_new_st, v_new_sh;
    const uint16_t* q_weight;  // [head_dim] or null (ones)
    const uint16_t* k_weight;
    const float* cos_sin;      // [cos_rows][rot]: rot / 2 cosines, then rot / 2 sines
    int64_t cos_rows;
    const int32_t* batch_indices;
    const int32_t* positions;
    const int32_t* rope_positions;  // null: positions
    uint8_t* q_out;
    int64_t q_out_st, q_out_sh;
    const int32_t* page_table;
    int64_t pt_stride;
    uint8_t* k_base;
    int64_t k_pages, k_sp, k_sh, k_st;
    uint8_t* v_base;
    int64_t v_pages, v_sp, v_sh, v_st;
    unsigned* err;
    int n_tokens, batch, hq, hk, page_shift, rot;
    float eps, k_scale, v_scale, k_inv, v_inv;  // inv: 1 / scale
};
cudaError_t launch_norm_rope(const NormRopeParams& p, int head_dim, bool bf16, bool kv8, bool pairs, int num_sms,
                             cudaStream_t s);

// Minimum and maximum of each page's keys (fdec_page_bounds).  Strides in bytes.
struct BoundsParams {
    const uint8_t* k_base;
    int64_t k_pages, k_sp, k_sh, k_st;
    uint8_t* b_base;           // b_st: bytes from a page's minimum row to its maximum row
    int64_t b_pages, b_sp, b_sh, b_st;
    const int32_t* page_table;
    int64_t pt_stride;
    const int32_t* begins;     // null: 0
    const int32_t* seq_lens;
    unsigned* err;
    int batch, hk, page_shift, span;
};
cudaError_t launch_page_bounds(const BoundsParams& p, int head_dim, bool bf16, bool kv8, int num_sms, cudaStream_t s);

// Page selection (fdec_select_pages).  q strides in elements, bounds strides in bytes.
struct SelectParams {
    const uint16_t* q;
    int64_t q_st, q_sh;
    const uint8_t* b_base;
    int64_t b_pages, b_sp, b_sh, b_st;
    const int32_t* page_table;
    int64_t pt_stride;
    const int32_t* seq_lens;
    int32_t* page_ids;         // [rows][budget], rows = batch x q_len x hk
    int32_t* counts;           // [rows]
    int32_t* page_indices;     // [rows][budget] or null
    float* chunk_abs;          // [rows][abs_stride] each scoring CTA's largest sum of magnitudes
    int64_t abs_stride;
    float* scores;             // [rows][score_stride], 16-byte aligned
    int64_t score_stride;      // max_pages rounded up to a multiple of 4
    unsigned long long* near_keys;  // [rows][max_pages]
    unsigned* err;
    int batch, q_len, hk, group, page_shift, causal;
    int max_pages, budget, first, last;
    int head_dim, chunk, n_chunks, chain;  // set by the launcher
};
int64_t select_abs_stride(int64_t max_pages);
cudaError_t launch_select_pages(SelectParams p, int head_dim, bool bf16, int num_sms, cudaStream_t s);

// Attention of drafted trees joined with the prefix's state (fdec_tree_attention).  q
// strides in elements, cache strides in bytes.
struct TreeParams {
    const uint16_t* q;
    int64_t q_st, q_sh;
    const uint8_t* k_base;
    int64_t k_pages, k_sp, k_sh, k_st;
    const uint8_t* v_base;
    int64_t v_pages, v_sp, v_sh, v_st;
    const int32_t* page_table;
    int64_t pt_stride, pt_cols;
    const int32_t* prefix_lens;
    const int32_t* node_counts;  // null: nodes each
    const int32_t* parents;      // null: a chain
    const float* o_prefix;       // [batch][nodes][hq][D] or null
    const float* lse_prefix;
    float* out;                  // of out_type (OutType)
    float* lse;                  // or null
    unsigned* err;
    int batch, nodes, hq, hk, group, page_shift, out_type;
    float scale_log2;            // scale x k_scale x log2(e)
    float v_scale;
    // Set by the launcher: CTAs of a sequence's KV head, or 0: shares of so many tiles, one more in the first.
    int parts, share, share_more;
    uint64_t group_inv;  // set by the launcher: ceil(2^40 / group)
};
cudaError_t launch_tree_attention(const TreeParams& p, int head_dim, bool bf16, bool kv8, int num_sms, cudaStream_t s);

// Most nodes of a drafted tree: a node's ancestors are the bits of one 64-bit word.
constexpr int kMaxNodes = 64;

// Verification of drafted tokens (fdec_verify_drafts).  Strides in elements.
struct VerifyParams {
    const void* target;
    int64_t t_seq, t_node;
    const void* draft;           // or null
    int64_t d_seq, d_node;
    const int32_t* tokens;
    const int32_t* parents;      // null: a chain
    const int32_t* node_counts;  // null: nodes each
    const float* uniforms;
    int32_t* path;
    int32_t* path_lens;
    int32_t* out_tokens;
    unsigned* err;
    int batch, nodes, vocab;
    int chunk;                   // tokens of a warp, set by the launcher
};
cudaError_t launch_verify_drafts(const VerifyParams& p, int prob_dtype, cudaStream_t s);

// Caches of a call that moves rows, as kernel arguments.  first_block: blocks of columns
// of the caches before this one.
struct CacheRows {
    uint8_t* base;
    int64_t s_layer, s_page, s_head, s_token;
    int layers, heads, row_vecs;  // row_vecs: vectors of a row (16 bytes, or 8 where wide is 0)
    int wide;
    int first_block;
};
constexpr int kMaxCaches = 128;
constexpr int kColumnThreads = 256;  // of a block, a column each
constexpr int kRowsAhead = 4;        // rows of a column in flight
template <int N>
struct CacheList {
    CacheRows c[N];
    int n;
};

struct KeepParams {
    const int32_t* page_table;
    int64_t pt_stride, pt_cols;
    const int32_t* prefix_lens;
    const int32_t* path;
    int64_t path_stride;
    const int32_t* path_lens;
    int32_t* seq_lens;
    unsigned* err;
    int64_t num_pages;           // the fewest of any cache
    int batch, nodes, page_shift;
};
cudaError_t launch_keep_path(const KeepParams& p, const CacheList<kMaxCaches>& caches, cudaStream_t s);

struct ReserveParams {
    int32_t* page_table;
    int64_t pt_stride, pt_cols;
    const int32_t* seq_lens;
    const int32_t* new_lens;
    const int32_t* sources;      // or null
    int32_t* granted;
    unsigned* used;              // [words] a bit a page: some entry in use names it
    unsigned* shared;            // [words] two do
    int32_t* taken;              // [blocks] pages in use of every kCountedPages, if there are many
    int32_t* last_page;          // [batch] the page of a sequence's (its source's) last, partly filled part
    int4* copies;                // [batch] (from page, to page, rows, 0)
    unsigned* err;
    int64_t num_pages;
    int words, blocks, batch, page_shift;
};
constexpr int kCountedPages = 1024;
cudaError_t launch_reserve_pages(const ReserveParams& p, const CacheList<kMaxCaches>& caches, int num_sms,
                                 cudaStream_t s);

// Shared by the entry points' translation units (defined in fdec_api.cu): record the
// message of a failed call (never throws) and return its status.
int record_failure(int status, const char* message) noexcept;
int record_cuda_failure(cudaError_t e, const char* what) noexcept;
void clear_failure() noexcept;
// Whether this thread's calls stop where they would launch, with kChecksOnly as their
// status: how the binding has tensors refused that are not on a GPU, after every other
// check of theirs (see sparse_binding.cpp).
constexpr int kChecksOnly = -1;
bool checks_only() noexcept;
// Columns of this thread's page tables: a row's stride, or fewer where the binding was given a
// view of some columns (what lies between its rows is another's).
int64_t table_columns(int64_t stride) noexcept;
// SM count of the current device, queried once per device.
cudaError_t current_num_sms(int* num_sms);
// One task given by value (p.tasks must be null): used by fdec_merge_states.
cudaError_t launch_reduce_single(const ReduceParams& p, ReduceTask task, cudaStream_t s);

}  // namespace fdec
