// tree_attention.cu -- attention of drafted trees, joined with the prefix's state.
//
//   z_j = scale q.K_j over a node and its ancestors, M = max(lse_p, max z),
//   w = exp(lse_p - M), l = w + sum exp(z_j - M),  out = (w o_p + sum exp(z_j - M) V_j) / l
//
// A CTA takes a run of a sequence's and KV head's query rows (row = node x group + head).  The
// tree's keys and values, at most 64 rows, are staged once in shared memory; a warp then takes
// 16 query rows at a time with mma.sync.m16n8k16: S of 16 x 64 in registers, the ancestors a
// 64-bit word a node, one maximum and sum (every key is there, so nothing is rescaled), P V in
// blocks of 64 columns.  The prefix's state enters as one more key, whose value is o_p.
//
// Bytes: 2 D of q, 4 D of o_p, 4 D or 2 D of the result for a query row, against 4 D x 64
// operations or less: bound by HBM, if anything hides the latencies.  Queries and o_p are
// therefore copied into shared memory a tile and a block ahead (requested where they are
// used, or held in registers, 64 trees of 64 nodes took 73 and 52 us; now 40.5, 4.6 TB/s, with
// the L1 pipe 56 % busy).  Few small trees are latencies: lengths, page ids, keys and values
// are three dependent reads (of 3.7 us for one tree; 1 us for the first two), which is why the
// rest is asked for behind them and the ancestors are another warp's.  mma.sync keeps S and P in registers; a tcgen05 tile of 128 rows
// would be mostly empty for trees of a few nodes, and the tensor pipe is not what bounds.
//
// P V multiplies f16 values: V as f16, and each probability as two f16 values (22 bits,
// and no more than 2^-33 off; scaled by 2^8), which makes the result as good as fp32
// sums; one value would leave 2^-12.  f16 and E4M3 values are f16 values; a bf16 cache's are
// rewritten as they are staged, times the power of two that brings the largest of the tree's
// below 2^15: exact but for values 2^-29 of that and less, which are off by 2^-40 of it.
// That holds while the tree's values are of one size (kSpread); where they are not, a large
// row that a node does not see, or hardly, would cost it the bits of the others.  V then stays
// bf16, which is exact, and a probability, normalised first, is three bf16 values (24 bits of
// its own size, however small): 1.5 times the products, 43.3 us instead of 40.5 for 64 trees of 64.
#include <algorithm>
#include <cstdint>

#include <cuda_fp8.h>

#include "../../include/fdec.h"
#include "fdec_internal.h"
#include "split_mma_kernel.cuh"

namespace fdec {

namespace {

constexpr int kTreeWarps = 4;
constexpr int kTreeThreads = kTreeWarps * 32;

// Rows of K and V are staged 16 bytes apart modulo 128, so that the eight rows of an ldmatrix lie on different banks.
// Behind them each warp has room for the queries of a tile (their first 128 dims) and for 16 x 64 floats of the
// prefix's rows.
constexpr int kSlotBytes = 16 * 64 * 4;
template <int D>
struct TreeShape {
    static constexpr int PITCH = 2 * D + 16;
    static constexpr int QD = D < 128 ? D : 128;
    static constexpr int Q_BYTES = 16 * QD * 2;
    static size_t smem(int rows) {  // rows of K and V that are staged
        return static_cast<size_t>(rows) * 2 * PITCH + kTreeWarps * (Q_BYTES + kSlotBytes);
    }
};

// Four E4M3 codes -> two words of 16-bit values (exact).
template <bool BF16>
__device__ __forceinline__ uint2 widen4(uint32_t codes) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const __half2_raw h =
            __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes >> (16 * i)), __NV_E4M3);
        if constexpr (BF16) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
            w[i] = pack2<true>(f.x, f.y);
        } else {
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
    return make_uint2(w[0], w[1]);
}

// x, y as sums of three bf16 values each.
__device__ __forceinline__ void split_three(float x, float y, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
    hi = pack2<true>(x, y);
    const float2 h = unpack2<true>(hi);
    x -= h.x, y -= h.y;
    mid = pack2<true>(x, y);
    const float2 m = unpack2<true>(mid);
    lo = pack2<true>(x - m.x, y - m.y);
}

// The bits of the larger magnitude in each half (infinities and NaN are the largest).
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t w) { return __vmaxu2(a, w & 0x7fff7fffu); }

// x, y as sums of two f16 values each.
__device__ __forceinline__ void split_two(float x, float y, uint32_t& hi, uint32_t& lo) {
    hi = pack2<false>(x, y);
    const float2 r = unpack2<false>(hi);
    lo = pack2<false>(x - r.x, y - r.y);
}

// mma_16816 into zeros.
template <bool BF16>
__device__ __forceinline__ void mma_16816_new(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (BF16) {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%10, %10, %10, %10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
    } else {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%10, %10, %10, %10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
    }
}

// S += Q K^T over 32 dims (FIRST: into zeros): a warp's 16 rows and 2 KS tiles of 8 keys.
template <bool BF16, int KS, bool FIRST>
__device__ __forceinline__ void add_scores(float (&s)[2 * KS][4], const uint32_t (&a0)[4],
                                           const uint32_t (&a1)[4], uint32_t k_addr, int pitch) {
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
#pragma unroll
        for (int j = 2 * ks; j < 2 * ks + 2; ++j) {
            uint32_t r0, r1, r2, r3;
            ldmatrix_x4(k_addr + j * 8 * pitch, r0, r1, r2, r3);
            if constexpr (FIRST)
                mma_16816_new<BF16>(s[j], a0, r0, r1);
            else
                mma_16816<BF16>(s[j], a0, r0, r1);
            mma_16816<BF16>(s[j], a1, r2, r3);
        }
    }
}

// Eight columns of V's row j (chunk c of 16 bytes) into shared memory.  Of 16 columns, those of pairs 0, 2, 4, 6 come
// first, then those of pairs 1, 3, 5, 7: the product's lane t then has columns 4t .. 4t + 3 in its two tiles of 8.
__device__ __forceinline__ void put_values(uint8_t* row, int c, uint4 v) {
    uint8_t* at = row + (c >> 1) * 32 + (c & 1) * 8;
    *reinterpret_cast<uint2*>(at) = make_uint2(v.x, v.z);
    *reinterpret_cast<uint2*>(at + 16) = make_uint2(v.y, v.w);
}

// A bf16 cache's values count as of one size while the largest is less than 2^(kSpread + 1) times the largest of any
// eight neighbours (that are not all zeros).  Up to there the 2^-33 that a probability's split may be off cost a node
// 2^-24, half a step of fp32, of what the rows that it does see hold in those columns.
constexpr unsigned kSpread = 8;

// CTAs on an SM that the registers of S, P and O are to allow.  (A fourth, with 128 registers a thread: 512 heads of 4
// tiles of 16 nodes 8.4 us instead of 10.6; but at head_dim 256 16 trees of 13 nodes 6.5 us instead of 6.0.)
constexpr int tree_ctas(int head_dim, int ks) { return ks == 1 && head_dim <= 128 ? 4 : 3; }

template <int D, bool BF16, bool KV8, int KS>
__global__ void __launch_bounds__(kTreeThreads, tree_ctas(D, KS)) tree_attention_kernel(const TreeParams p) {
    using S = TreeShape<D>;
    constexpr int kPShift = 8;                 // p x 2^8 is split
    constexpr bool kRewrite = BF16 && !KV8;    // V is not f16 as it is stored
    constexpr uint32_t kInf = kRewrite ? 0x7f80 : 0x7c00;
    extern __shared__ __align__(128) uint8_t smem[];
    // What is known of the trees of the CTA's next kTreeWarps runs of tiles.
    __shared__ uint64_t s_anc[kTreeWarps][kMaxNodes];                           // a node and its ancestors
    __shared__ int64_t s_k[kTreeWarps][kMaxNodes], s_v[kTreeWarps][kMaxNodes];  // byte offsets of the nodes' rows
    __shared__ uint64_t s_valid[kTreeWarps];                                    // nodes whose rows can be read
    __shared__ int s_count[kTreeWarps];
    __shared__ unsigned s_max, s_min, s_odd[2];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int N = p.nodes, g = p.group;
    const int tiles_max = (N * g + 15) / 16;  // of a sequence's KV head

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // The CTA's tiles: a part of a sequence's KV head, or an equal share of all tiles, a run of them for each sequence
    // and KV head in it.
    int bh, first, left;  // sequence and KV head, its first tile of a run, tiles from there on
    const int c = blockIdx.x;
    if (p.parts > 0) {
        bh = c / p.parts;
        const int part = c - bh * p.parts;
        first = tiles_max * part / p.parts;
        left = tiles_max * (part + 1) / p.parts - first;
    } else {
        const int at_tile = c * p.share + min(c, p.share_more);
        bh = at_tile / tiles_max;
        first = at_tile - bh * tiles_max;
        left = p.share + (c < p.share_more);
    }
    int b = bh / p.hk, kvh = bh - b * p.hk;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const auto next_run = [&] {
        left -= tiles_max - first;
        first = 0;
        ++bh;
        if (++kvh == p.hk) kvh = 0, ++b;
    };
    for (int run = 0; left > 0; ++run, next_run()) {
        const int count = min(left, tiles_max - first);
        __syncthreads();  // what was staged before has been read
        if (tid == 0) {
            s_max = s_odd[0] = s_odd[1] = 0;
            s_min = 0xffffffffu;
        }

        if (run % kTreeWarps == 0) {
            // Warp w takes the rows of the run w from here and, meanwhile, the ancestors of the run w + 1: of a single run
            // two warps share the work.
            constexpr int H = KS > 2 ? 2 : 1;  // halves of the 64 nodes that there can be
            const int w_anc = (warp + 1) % kTreeWarps;
            const auto has = [&](int ahead) { return ahead == 0 || ahead * tiles_max < first + left; };
            const auto seq_of = [&](int ahead) { return ahead == 0 ? b : (bh + ahead) / p.hk; };
            const bool has_rows = has(warp), has_anc = has(w_anc);
            const auto reports = [&](int ahead, int b_of) {  // one CTA a sequence
                return p.err != nullptr && bh + ahead == b_of * p.hk && (ahead > 0 || first == 0);
            };
            int up[H], n_anc = N;
            if (has_anc) {
                const int b_of = seq_of(w_anc);
                if (p.node_counts != nullptr) n_anc = p.node_counts[b_of];
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    const int i = lane + 32 * h;
                    up[h] = p.parents == nullptr ? i - 1 : i < N ? p.parents[static_cast<int64_t>(b_of) * N + i] : -1;
                }
            }
            if (has_rows) {
                const int b_of = seq_of(warp), kvh_of = bh + warp - b_of * p.hk;
                unsigned flags = 0;
                int n = p.node_counts != nullptr ? p.node_counts[b_of] : N;
                int64_t prefix = p.prefix_lens[b_of];
                int64_t page[H], slot_of[H];
                bool behind[H];  // past the page table
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    const int i = lane + 32 * h;
                    const int64_t pos = max(prefix, static_cast<int64_t>(0)) + i, pi = pos >> p.page_shift;
                    slot_of[h] = pos & ((1 << p.page_shift) - 1);
                    behind[h] = pi >= p.pt_cols;
                    page[h] = i < N && !behind[h] ? p.page_table[static_cast<int64_t>(b_of) * p.pt_stride + pi] : -1;
                }
                if (n < 0 || n > N) {
                    flags |= FDEC_DEVERR_SEQ_LEN;
                    n = min(max(n, 0), N);
                }
                if (prefix < 0 && n > 0) flags |= FDEC_DEVERR_SEQ_LEN;
                uint64_t valid = 0;
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    const int i = lane + 32 * h;
                    const bool ok = i < n && page[h] >= 0 && page[h] < p.k_pages && page[h] < p.v_pages;
                    if (i < n && !ok) flags |= behind[h] ? FDEC_DEVERR_SEQ_LEN : FDEC_DEVERR_PAGE_ID;
                    valid |= static_cast<uint64_t>(__ballot_sync(0xffffffffu, ok)) << (32 * h);
                    s_k[warp][i] = page[h] * p.k_sp + slot_of[h] * p.k_st + kvh_of * p.k_sh;
                    s_v[warp][i] = page[h] * p.v_sp + slot_of[h] * p.v_st + kvh_of * p.v_sh;
                }
                if (lane == 0) {
                    s_valid[warp] = valid;
                    s_count[warp] = n;
                }
                if (flags != 0 && reports(warp, b_of)) atomicOr(p.err, flags);
            }
            if (has_anc) {
                uint64_t anc[H];
                bool bad = false;
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    const int i = lane + 32 * h;
                    if (up[h] < -1 || up[h] >= i) {
                        bad |= i < min(n_anc, N);
                        up[h] = -1;
                    }
                    anc[h] = uint64_t{1} << i;
                }
                // ancestors: bits of a node's path, by pointer doubling (a path has at most 16 KS - 1 steps)
#pragma unroll 1
                for (int step = 0; step < 6; ++step) {
                    bool rest = false;
#pragma unroll
                    for (int h = 0; h < H; ++h) rest |= up[h] >= 0;
                    if (!__any_sync(0xffffffffu, rest)) break;
                    uint64_t a[H];
                    int u[H];
#pragma unroll
                    for (int h = 0; h < H; ++h) {
                        const int from = up[h] & 31;
                        uint64_t a0 = __shfl_sync(0xffffffffu, anc[0], from);
                        int u0 = __shfl_sync(0xffffffffu, up[0], from);
                        if constexpr (H > 1) {
                            const uint64_t a1 = __shfl_sync(0xffffffffu, anc[H - 1], from);
                            const int u1 = __shfl_sync(0xffffffffu, up[H - 1], from);
                            a0 = up[h] < 32 ? a0 : a1;
                            u0 = up[h] < 32 ? u0 : u1;
                        }
                        a[h] = up[h] < 0 ? 0 : a0;
                        u[h] = up[h] < 0 ? -1 : u0;
                    }
#pragma unroll
                    for (int h = 0; h < H; ++h) {
                        anc[h] |= a[h];
                        up[h] = u[h];
                    }
                }
#pragma unroll
                for (int h = 0; h < H; ++h) s_anc[w_anc][lane + 32 * h] = anc[h];
                if (bad && reports(w_anc, seq_of(w_anc))) atomicOr(p.err, FDEC_DEVERR_TREE);
            }
        }
        __syncthreads();
        const int known = run % kTreeWarps;
        const int n = s_count[known], R = n * g;
        const uint64_t valid = s_valid[known];
        const int tiles = min((R + 15) / 16, first + count);
        if (first >= tiles) continue;

        // A warp's tiles of 16 query rows.  What they read is copied ahead of its use into the warp's part of shared
        // memory: the queries of the next tile once this one's have been multiplied, the prefix's rows in blocks of 64
        // columns, each once the one before it has been joined.
        constexpr int CB = D / 64, QD = S::QD;
        const int gq = lane >> 2, t = lane & 3;
        // With fewer tiles than warps, warps share one: each computes S and takes a part of the columns of O.
        const int split = tiles - first > 2 ? 1 : min(tiles - first == 2 ? 2 : kTreeWarps, CB);
        const int T0 = first + warp / split, part = warp % split;
        const int cb0 = part * CB / split, cb1 = (part + 1) * CB / split;
        // Heads of more than QD dims: S, too, in parts, blocks of 32 dims [d0, d1), added up through shared memory (16
        // trees of 13 nodes, head_dim 256, 6.0 us instead of 6.9; at 128 dims the sums would cost what they save).
        constexpr bool kAddParts = D > QD;
        const int d0 = kAddParts ? part * (D / 32) / split : 0, d1 = kAddParts ? (part + 1) * (D / 32) / split : D / 32;
        const int my_tiles = T0 < tiles ? (split > 1 ? 1 : (tiles - T0 + kTreeWarps - 1) / kTreeWarps) : 0;
        const uint32_t q_slot = smem_addr(smem) + 2 * 16 * KS * S::PITCH + warp * (S::Q_BYTES + kSlotBytes);
        const uint32_t slot = q_slot + S::Q_BYTES;
        // Lane l: the (token, head) index in out and lse of row l % 16 of a tile (-1 past the last), its node.
        int rows = -1, nodes = 0;
        int row[2], node[2];       // of the lane's two rows of S
        float lse_in[2];
        const auto query = [&](int row, int node) {
            const int64_t tok = static_cast<int64_t>(b) * N + node;
            return p.q + tok * p.q_st + (row - tok * p.hq) * p.q_sh;
        };
        const auto next_tile = [&](int it) {
            const int r = (T0 + it * kTreeWarps) * 16 + (lane & 15);
            // (r / g: r is below 2^22 and g at most 2^16, so what group_inv has too much stays below 2^38 / 2^40 / g)
            nodes = it < my_tiles && r < R ? static_cast<int>(static_cast<uint64_t>(r) * p.group_inv >> 40) : 0;
            rows = it < my_tiles && r < R ? (b * N + nodes) * p.hq + kvh * g + (r - nodes * g) : -1;
            if (it < my_tiles) {
                const uint16_t* mine = rows >= 0 ? query(rows, nodes) : p.q;
                constexpr int CH = QD / 8, RPI = 32 / CH;  // 16-byte pieces of a row, rows at a time
#pragma unroll
                for (int k = 0; k < 16 / RPI; ++k) {
                    const int r = k * RPI + lane / CH, c = lane % CH;
                    const uint16_t* from = reinterpret_cast<const uint16_t*>(
                        __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine), r));
                    // (zeros past the last row, and past the part's dims)
                    const bool there = __shfl_sync(0xffffffffu, rows, r) >= 0 && (!kAddParts || d0 * 4 + c < d1 * 4);
                    const uint32_t to = q_slot + r * QD * 2 + (c ^ (r & 7)) * 16;
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to),
                                 "l"(there ? from + d0 * 32 + c * 8 : p.q), "r"(there ? 16 : 0)
                                 : "memory");
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                row[h] = __shfl_sync(0xffffffffu, rows, gq + 8 * h);
                node[h] = __shfl_sync(0xffffffffu, nodes, gq + 8 * h);
                lse_in[h] = row[h] >= 0 && p.lse_prefix != nullptr ? p.lse_prefix[row[h]] : -INFINITY;
            }
        };
        const auto request_prefix = [&](int cb, int rows) {
            if (p.o_prefix != nullptr) {
                const float* from = p.o_prefix + cb * 64 + (lane & 15) * 4;
                const uint32_t to = slot + (lane >> 4) * 256;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int r = 2 * k + (lane >> 4), row = __shfl_sync(0xffffffffu, rows, r);
                    // pieces of 64 bytes change places in odd rows, so that two rows' lie on different banks
                    const uint32_t piece = ((lane & 15) ^ ((r & 1) << 2)) * 16;
                    if (row >= 0) cp_async_16(to + k * 512 + piece, from + static_cast<int64_t>(row) * D);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        // K and V rows, widened to 16 bits; rows past the tree and unreadable ones are zeros
        constexpr int staged = 16 * KS;
        uint8_t* sm_k = smem;
        uint8_t* sm_v = smem + staged * S::PITCH;
        // Rows of V with an infinite or NaN value are not multiplied as the others (0 times it would reach every row):
        // they are zeros in shared memory, and are added for the rows that see them.
        // Of eight values each, if not of those rows: the largest magnitude, and the least of those that are
        // not 0, less 1.
        uint32_t most = 0, least = 0xffffffffu;
        const auto note = [&](int j, uint32_t two) {
            const uint32_t x = max(two & 0xffffu, two >> 16);
            if (x >= kInf) {
                atomicOr(&s_odd[j >> 5], 1u << (j & 31));
            } else {
                most = max(most, x);
                least = min(least, x - 1);
            }
        };
        constexpr int CH = KV8 ? D / 16 : D / 8;  // 16-byte chunks of a stored row
        constexpr int PER = (staged * CH + kTreeThreads - 1) / kTreeThreads;  // of a thread
        // V's chunks stay in registers until the largest value is known (but for the widest rows)
        constexpr bool kHeld = kRewrite && PER <= 16;
        constexpr int U = PER < 8 ? PER : 8;
        uint4 held[kHeld ? (PER + U - 1) / U * U : 1];
#pragma unroll
        for (int i0 = 0; i0 < PER; i0 += U) {
            uint4 kk[U], vv[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = tid + (i0 + u) * kTreeThreads, j = c / CH;
                kk[u] = vv[u] = make_uint4(0, 0, 0, 0);
                if (c < staged * CH && (valid >> j & 1)) {
                    kk[u] = *reinterpret_cast<const uint4*>(p.k_base + s_k[known][j] + (c - j * CH) * 16);
                    vv[u] = *reinterpret_cast<const uint4*>(p.v_base + s_v[known][j] + (c - j * CH) * 16);
                }
            }
            if (i0 == 0) {
                next_tile(0);
                request_prefix(cb0, rows);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = tid + (i0 + u) * kTreeThreads, j = c / CH;
                if (c >= staged * CH) break;
                if constexpr (KV8) {
                    const uint32_t kw[4] = {kk[u].x, kk[u].y, kk[u].z, kk[u].w};
                    const uint32_t vw[4] = {vv[u].x, vv[u].y, vv[u].z, vv[u].w};
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint2 ka = widen4<BF16>(kw[2 * h]), kb = widen4<BF16>(kw[2 * h + 1]);
                        const uint2 va = widen4<false>(vw[2 * h]), vb = widen4<false>(vw[2 * h + 1]);
                        *reinterpret_cast<uint4*>(sm_k + j * S::PITCH + (c - j * CH) * 32 + h * 16) =
                            make_uint4(ka.x, ka.y, kb.x, kb.y);
                        put_values(sm_v + j * S::PITCH, (c - j * CH) * 2 + h, make_uint4(va.x, va.y, vb.x, vb.y));
                        note(j, larger(larger(larger(larger(0, va.x), va.y), vb.x), vb.y));
                    }
                } else {
                    *reinterpret_cast<uint4*>(sm_k + j * S::PITCH + (c - j * CH) * 16) = kk[u];
                    if constexpr (kHeld)
                        held[i0 + u] = vv[u];
                    else
                        put_values(sm_v + j * S::PITCH, c - j * CH, vv[u]);
                    note(j, larger(larger(larger(larger(0, vv[u].x), vv[u].y), vv[u].z), vv[u].w));
                }
            }
        }
        if constexpr (kRewrite) {
            most = __reduce_max_sync(0xffffffffu, most);
            least = __reduce_min_sync(0xffffffffu, least);
            if (lane == 0) {
                atomicMax(&s_max, most);
                atomicMin(&s_min, least);
            }
        }
        __syncthreads();
        const uint64_t odd = s_odd[0] | static_cast<uint64_t>(s_odd[1]) << 32;
        // (110: the factor that undoes it stays a normal number; only values below 2^-112 lose by that)
        const int up = kRewrite ? min(14 - (static_cast<int>(s_max >> 7) - 127), 110) : 0;
        const float factor = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
        // V stays bf16; a row that is not finite is added with its fp32 probabilities
        const bool wide = kRewrite && (odd != 0 || (s_max >> 7) > ((s_min + 1) >> 7) + kSpread);
        const float scale = fabsf(p.scale_log2);
        if (kRewrite || odd != 0 || p.scale_log2 < 0.f) {
            if constexpr (kRewrite) {
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const int c = tid + i * kTreeThreads, j = c / CH;
                    if (c >= staged * CH) break;
                    const auto f16 = [&](uint32_t x) {
                        const float2 y = unpack2<true>(x);
                        return pack2<false>(y.x * factor, y.y * factor);
                    };
                    if constexpr (kHeld) {
                        const uint4 v = held[i];
                        put_values(sm_v + j * S::PITCH, c - j * CH,
                                   wide ? v : make_uint4(f16(v.x), f16(v.y), f16(v.z), f16(v.w)));
                    } else if (!wide) {
                        uint4* at = reinterpret_cast<uint4*>(sm_v + j * S::PITCH + (c - j * CH) * 16);
                        const uint4 v = *at;
                        *at = make_uint4(f16(v.x), f16(v.y), f16(v.z), f16(v.w));
                    }
                }
            }
            if (odd != 0 || p.scale_log2 < 0.f) {
                __syncthreads();
                for (int c = tid; c < staged * (D / 8); c += kTreeThreads) {
                    const int j = c / (D / 8), at = (c - j * (D / 8)) * 16;
                    if (odd >> j & 1) *reinterpret_cast<uint4*>(sm_v + j * S::PITCH + at) = make_uint4(0, 0, 0, 0);
                    if (p.scale_log2 < 0.f) {  // the scale's sign goes to K: the largest product is the largest logit
                        uint4* k = reinterpret_cast<uint4*>(sm_k + j * S::PITCH + at);
                        const uint4 x = *k;
                        *k = make_uint4(x.x ^ 0x80008000u, x.y ^ 0x80008000u, x.z ^ 0x80008000u, x.w ^ 0x80008000u);
                    }
                }
            }
            __syncthreads();
        }
        const float v_factor = p.v_scale * exp2f(static_cast<float>(-kPShift - up));  // (the products' scales undone)

        const uint32_t k_addr = smem_addr(sm_k) + (lane & 7) * S::PITCH + (lane >> 3) * 16;
        const int q_row = (lane & 7) + ((lane >> 3) & 1) * 8;
        const uint32_t q_addr = q_slot + q_row * QD * 2;
        const uint32_t v_addr = smem_addr(sm_v) + ((lane & 7) + ((lane >> 3) & 1) * 8) * S::PITCH + (lane >> 4) * 16;
        const bool f32 = p.out_type == kOutF32;
        // The warp's tiles.  RAW: probabilities are kept in fp32, for V in bf16 and for rows that are not finite
        // (a body of its own: with branches in one body, 64 trees of 64 nodes took 1 % longer, at head_dim 192
        // 96 of them 8 %).
        const auto walk = [&](auto raw) {
            constexpr bool RAW = decltype(raw)::value;
            for (int it = 0; it < my_tiles; ++it) {
                constexpr int NT = 2 * KS;
                float s[NT][4];
                asm volatile("cp.async.wait_group 1;" ::: "memory");
                __syncwarp();  // the tile's queries are there (the prefix's first block may not be)
#pragma unroll
                for (int c = 0; c < QD / 32; ++c) {  // S = Q K^T, 32 dims at a time
                    uint32_t a0[4], a1[4];
                    ldmatrix_x4(q_addr + ((4 * c + (lane >> 4)) ^ (lane & 7)) * 16, a0[0], a0[1], a0[2], a0[3]);
                    ldmatrix_x4(q_addr + ((4 * c + 2 + (lane >> 4)) ^ (lane & 7)) * 16, a1[0], a1[1], a1[2], a1[3]);
                    if (c == 0)
                        add_scores<BF16, KS, true>(s, a0, a1, k_addr + d0 * 64, S::PITCH);
                    else if (!kAddParts || d0 + c < d1)
                        add_scores<BF16, KS, false>(s, a0, a1, k_addr + (d0 + c) * 64, S::PITCH);
                }
                if constexpr (kAddParts) {  // the other dims from where they are
                    const uint16_t* from[2] = {(row[0] >= 0 ? query(row[0], node[0]) : p.q) + 2 * t,
                                               (row[1] >= 0 ? query(row[1], node[1]) : p.q) + 2 * t};
                    const auto word = [&](int h, int d) {
                        return row[h] >= 0 ? *reinterpret_cast<const uint32_t*>(from[h] + d) : 0u;
                    };
#pragma unroll 6
                    for (int d = d0 * 32 + QD; d < d1 * 32; d += 32) {
                        const uint32_t a0[4] = {word(0, d), word(1, d), word(0, d + 8), word(1, d + 8)};
                        const uint32_t a1[4] = {word(0, d + 16), word(1, d + 16), word(0, d + 24), word(1, d + 24)};
                        add_scores<BF16, KS, false>(s, a0, a1, k_addr + d * 2, S::PITCH);
                    }
                    if (split > 1) {  // (where the queries lay)
                        const uint32_t at = lane * 16;
                        __syncwarp();
#pragma unroll
                        for (int j = 0; j < NT; ++j)
                            asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(q_slot + at + j * 512),
                                         "f"(s[j][0]), "f"(s[j][1]), "f"(s[j][2]), "f"(s[j][3])
                                         : "memory");
                        asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / split), "r"(32 * split) : "memory");
#pragma unroll
                        for (int j = 0; j < NT; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
                        for (int k = 0; k < split; ++k) {  // (every warp in the same order)
                            const uint32_t from = q_slot + (k - part) * (S::Q_BYTES + kSlotBytes) + at;
#pragma unroll
                            for (int j = 0; j < NT; ++j) {
                                const float4 x = lds128f<0>(from + j * 512);
                                s[j][0] += x.x, s[j][1] += x.y, s[j][2] += x.z, s[j][3] += x.w;
                            }
                        }
                    }
                }

                float w[2], vs[2], norm[2], lse_out[2];
                const int out_row[2] = {row[0], row[1]}, out_node[2] = {node[0], node[1]};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint64_t vis = row[h] < 0 ? 0 : s_anc[known][node[h]] & valid;
                    const float before = lse_in[h] * 1.4426950408889634f;
                    // the lane's columns of a tile of 8 keys are 2t and 2t + 1
                    const uint64_t mine = vis >> (2 * t);
                    const uint32_t bits[2] = {static_cast<uint32_t>(mine), static_cast<uint32_t>(mine >> 32)};
                    float top = -INFINITY;
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float& z = s[j][2 * h + e];
                            if (!(bits[j >> 2] & (1u << ((j & 3) * 8 + e)))) z = -INFINITY;
                            top = fmaxf(top, z);
                        }
                    }
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    top = fmaxf(top * scale, before);
                    const float m = top == -INFINITY ? 0.f : top;
                    float sum = 0.f;
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float& z = s[j][2 * h + e];
                            z = exp2_approx(fmaf(z, scale, kPShift - m));
                            sum += z;
                        }
                    }
                    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                    w[h] = exp2_approx(before - m);
                    sum = sum * (1.f / (1 << kPShift)) + w[h];
                    const float inv = sum == 0.f ? 0.f : 1.f / sum;
                    lse_out[h] = sum == 0.f ? -INFINITY : m * 0.6931471805599453f + logf(sum);
                    w[h] *= inv;
                    vs[h] = RAW && kRewrite ? p.v_scale : v_factor * inv;
                    norm[h] = inv * (1.f / (1 << kPShift));
                }
                if (p.lse != nullptr && t == 0 && part == 0) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if (out_row[h] >= 0) p.lse[out_row[h]] = lse_out[h];
                }
                // an empty state counts for nothing, whatever its values
                const bool empty[2] = {row[0] >= 0 && lse_in[0] == -INFINITY, row[1] >= 0 && lse_in[1] == -INFINITY};
                const bool states = !__any_sync(0xffffffffu, empty[0] || empty[1]);
                const int rows_now = rows;
                __syncwarp();  // the queries have been read
                if (it + 1 < my_tiles) {
                    next_tile(it + 1);
                } else {
                    rows = -1;
                    asm volatile("cp.async.commit_group;" ::: "memory");
                }

                // Two probabilities as their f16 high and low parts, or (raw) as they are in fp32.
                uint32_t pf[KS][2][4];
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float x = s[2 * ks + (e >> 1)][2 * (e & 1)], y = s[2 * ks + (e >> 1)][2 * (e & 1) + 1];
                        if constexpr (RAW) {
                            if constexpr (kRewrite) x *= norm[e & 1], y *= norm[e & 1];
                            pf[ks][0][e] = __float_as_uint(x);
                            pf[ks][1][e] = __float_as_uint(y);
                        } else {
                            split_two(x, y, pf[ks][0][e], pf[ks][1][e]);
                        }
                    }
                }

                // O in blocks of 64 columns
                const auto finish = [&](int cb, const float (&acc)[8][4]) {
                    if (cb == cb0)
                        asm volatile("cp.async.wait_group 1;" ::: "memory");  // (the next queries may be on their way)
                    else
                        asm volatile("cp.async.wait_group 0;" ::: "memory");
                    __syncwarp();  // the warp's copies of the block are there
                    // the lane's columns 16 j + 4 t .. + 3 of the block: its products' tiles 2 j and 2 j + 1
                    const uint32_t from = slot + gq * 256 + t * 16;
                    const auto place = [&](int h, int j) { return from + h * 2048 + (j ^ (gq & 1)) * 64; };
                    if (!states) {
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            if (empty[h]) {
#pragma unroll
                                for (int j = 0; j < 4; ++j)
                                    asm volatile("st.shared.v4.f32 [%0], {%1, %1, %1, %1};" ::"r"(place(h, j)), "f"(0.f)
                                                 : "memory");
                            }
                    }
                    // Rows of V that are not finite: their share is added to the state's, which is weighed here.
                    if (RAW && odd != 0) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float4 o[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const float4 x = lds128f<0>(place(h, j));
                                o[j] = make_float4(w[h] * x.x, w[h] * x.y, w[h] * x.z, w[h] * x.w);
                            }
                            for (uint64_t rest = odd; rest != 0; rest &= rest - 1) {
                                const int key = __ffsll(static_cast<long long>(rest)) - 1;
                                uint32_t even = 0, uneven = 0;
#pragma unroll
                                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                                    for (int e = 0; e < 2; ++e)
                                        // (selected in registers: not an index into memory)
                                        asm volatile("{\n\t.reg .pred p;\n\tsetp.eq.s32 p, %4, %5;\n\t"
                                                     "selp.b32 %0, %2, %0, p;\n\tselp.b32 %1, %3, %1, p;\n\t}"
                                                     : "+r"(even), "+r"(uneven)
                                                     : "r"(pf[ks][0][2 * e + h]), "r"(pf[ks][1][2 * e + h]),
                                                       "r"(key >> 3), "r"(2 * ks + e));
                                const float pr = __shfl_sync(0xffffffffu, __uint_as_float(key & 1 ? uneven : even),
                                                             (lane & ~3) | ((key & 7) >> 1)) * vs[h];
                                const uint64_t seen = out_row[h] < 0 ? 0 : s_anc[known][out_node[h]] & valid;
                                if (!(seen >> key & 1)) continue;
                                const uint8_t* v_row = p.v_base + s_v[known][key] + (cb * 64 + 4 * t) * (KV8 ? 1 : 2);
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    uint2 v;
                                    if constexpr (KV8)
                                        v = widen4<false>(*reinterpret_cast<const uint32_t*>(v_row + j * 16));
                                    else
                                        v = *reinterpret_cast<const uint2*>(v_row + j * 32);
                                    const float2 x = unpack2<BF16 && !KV8>(v.x), y = unpack2<BF16 && !KV8>(v.y);
                                    o[j].x += pr * x.x;
                                    o[j].y += pr * x.y;
                                    o[j].z += pr * y.x;
                                    o[j].w += pr * y.y;
                                }
                            }
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(place(h, j)), "f"(o[j].x),
                                             "f"(o[j].y), "f"(o[j].z), "f"(o[j].w)
                                             : "memory");
                        }
                    }
                    const float weight[2] = {RAW && odd != 0 ? 1.f : w[0], RAW && odd != 0 ? 1.f : w[1]};
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (out_row[h] < 0) continue;
                        const int64_t at = static_cast<int64_t>(out_row[h]) * D + cb * 64 + 4 * t;
                        const auto joined = [&](int j) {
                            const float4 o = lds128f<0>(place(h, j));
                            return make_float4(vs[h] * acc[2 * j][2 * h] + weight[h] * o.x,
                                               vs[h] * acc[2 * j][2 * h + 1] + weight[h] * o.y,
                                               vs[h] * acc[2 * j + 1][2 * h] + weight[h] * o.z,
                                               vs[h] * acc[2 * j + 1][2 * h + 1] + weight[h] * o.w);
                        };
                        if (f32) {
#pragma unroll
                            for (int j = 0; j < 4; ++j) *reinterpret_cast<float4*>(p.out + at + j * 16) = joined(j);
                        } else {
                            uint16_t* out = reinterpret_cast<uint16_t*>(p.out) + at;
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const float4 x = joined(j);
                                *reinterpret_cast<uint2*>(out + j * 16) =
                                    make_uint2(pack2<BF16>(x.x, x.y), pack2<BF16>(x.z, x.w));
                            }
                        }
                    }
                    __syncwarp();  // and have been read
                    request_prefix(cb + 1 < cb1 ? cb + 1 : cb0, cb + 1 < cb1 ? rows_now : rows);
                };
#pragma unroll 1
                for (int cb = cb0; cb < cb1; ++cb) {
                    float acc[8][4];
                    // acc (+)= P V of 16 keys: P in N parts, the smallest first.
                    const auto products = [&](auto bf16, int ks, const auto& part) {
                        constexpr bool kBF16 = decltype(bf16)::value;
                        constexpr int N = sizeof(part) / sizeof(part[0]);
#pragma unroll
                        for (int dp = 0; dp < 4; ++dp) {
                            uint32_t r0, r1, r2, r3;
                            ldmatrix_x4_trans(v_addr + ks * 16 * S::PITCH + cb * 128 + dp * 32, r0, r1, r2, r3);
                            if (ks == 0) {
                                mma_16816_new<kBF16>(acc[2 * dp], part[N - 1], r0, r1);
                                mma_16816_new<kBF16>(acc[2 * dp + 1], part[N - 1], r2, r3);
                            } else {
                                mma_16816<kBF16>(acc[2 * dp], part[N - 1], r0, r1);
                                mma_16816<kBF16>(acc[2 * dp + 1], part[N - 1], r2, r3);
                            }
#pragma unroll
                            for (int i = N - 2; i >= 0; --i) {
                                mma_16816<kBF16>(acc[2 * dp], part[i], r0, r1);
                                mma_16816<kBF16>(acc[2 * dp + 1], part[i], r2, r3);
                            }
                        }
                    };
                    if constexpr (RAW) {
#pragma unroll
                        for (int ks = 0; ks < KS; ++ks) {
                            uint32_t part[kRewrite ? 3 : 2][4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float x = __uint_as_float(pf[ks][0][e]), y = __uint_as_float(pf[ks][1][e]);
                                if constexpr (kRewrite)
                                    split_three(x, y, part[0][e], part[1][e], part[2][e]);
                                else
                                    split_two(x, y, part[0][e], part[1][e]);
                            }
                            products(std::bool_constant<kRewrite>{}, ks, part);
                        }
                    } else {
#pragma unroll
                        for (int ks = 0; ks < KS; ++ks) products(std::false_type{}, ks, pf[ks]);
                    }
                    finish(cb, acc);
                }
            }
        };
        if (kRewrite ? wide : odd != 0)
            walk(std::true_type{});
        else
            walk(std::false_type{});
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
}

template <int D, bool BF16, bool KV8, int KS>
cudaError_t launch_tree_one(TreeParams p, int num_sms, cudaStream_t s) {
    constexpr int kDevices = 64;
    static int resident_on[kDevices] = {};  // CTAs on an SM, 0: not asked yet
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    int resident = dev < kDevices ? __atomic_load_n(&resident_on[dev], __ATOMIC_ACQUIRE) : 0;
    if (resident == 0) {
        const auto kernel = tree_attention_kernel<D, BF16, KV8, KS>;
        const size_t smem = TreeShape<D>::smem(16 * KS);
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&resident, kernel, kTreeThreads, smem);
        if (e != cudaSuccess) return e;
        resident = std::max(resident, 1);
        if (dev < kDevices) __atomic_store_n(&resident_on[dev], resident, __ATOMIC_RELEASE);
    }
    // Up to as many sequences' KV heads as CTAs are resident, or with fewer tiles in each than a CTA has warps: parts
    // of one head each, as an equal share that spans two stages two trees (256 heads of 6 tiles: 7.0 us, 9.0 shared).
    // Else equal shares: whole heads in a second round would leave most of the machine idle (512 heads of 16 tiles:
    // 40 us, 49 a head a CTA).  What is resident is asked for, as shared memory holds fewer CTAs than registers where
    // heads of more than 128 dims meet more than 32 nodes (768 heads of 16 tiles, head_dim 192: 109 us; 140 with three
    // CTAs an SM taken for granted, of which two fit).
    const int64_t heads = static_cast<int64_t>(p.batch) * p.hk;
    const int64_t slots = static_cast<int64_t>(num_sms) * resident;
    const int per_head = (p.nodes * p.group + 15) / 16;
    const bool whole = heads <= slots || per_head < kTreeWarps;
    const int64_t wide = std::min<int64_t>((per_head + kTreeWarps - 1) / kTreeWarps, 2 * slots / heads);
    // (a part for every tile where the machine has room twice over: warps then share the tiles)
    p.parts = !whole ? 0 : heads * per_head <= slots / 2 ? per_head : static_cast<int>(std::max<int64_t>(1, wide));
    const int64_t grid = p.parts > 0 ? heads * p.parts : slots;
    p.share = static_cast<int>(heads * per_head / slots);
    p.share_more = static_cast<int>(heads * per_head % slots);
    p.group_inv = ((uint64_t{1} << 40) + p.group - 1) / p.group;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(kTreeThreads, 1, 1);
    cfg.dynamicSmemBytes = TreeShape<D>::smem(16 * KS);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tree_attention_kernel<D, BF16, KV8, KS>, p);
}

template <int D, bool BF16, bool KV8>
cudaError_t launch_tree(const TreeParams& p, int num_sms, cudaStream_t s) {
    if (p.nodes <= 16) return launch_tree_one<D, BF16, KV8, 1>(p, num_sms, s);
    if (p.nodes <= 32) return launch_tree_one<D, BF16, KV8, 2>(p, num_sms, s);
    return launch_tree_one<D, BF16, KV8, 4>(p, num_sms, s);
}

template <int D>
cudaError_t launch_tree_d(const TreeParams& p, bool bf16, bool kv8, int num_sms, cudaStream_t s) {
    if (kv8) {
        if constexpr (D == 128 || D == 256)
            return bf16 ? launch_tree<D, true, true>(p, num_sms, s) : launch_tree<D, false, true>(p, num_sms, s);
        return cudaErrorInvalidValue;
    }
    return bf16 ? launch_tree<D, true, false>(p, num_sms, s) : launch_tree<D, false, false>(p, num_sms, s);
}

}  // namespace

cudaError_t launch_tree_attention(const TreeParams& p, int head_dim, bool bf16, bool kv8, int num_sms, cudaStream_t s) {
    switch (head_dim) {
        case 64: return launch_tree_d<64>(p, bf16, kv8, num_sms, s);
        case 128: return launch_tree_d<128>(p, bf16, kv8, num_sms, s);
        case 192: return launch_tree_d<192>(p, bf16, kv8, num_sms, s);
        case 256: return launch_tree_d<256>(p, bf16, kv8, num_sms, s);
        case 512: return launch_tree_d<512>(p, bf16, kv8, num_sms, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace fdec
