// select_pages.cu -- which pages of a long cache a query token attends to.
//
// From the bounds of a page's keys (page_bounds.cu) the largest logit that any key of
// the page can have for query head q_h is sum_d max(q_hd min_d, q_hd max_d): a positive
// q takes the maximum and a negative one the minimum.  The heads of a KV group share
// their pages; summed over the group's heads the score is linear in the two rows,
//
//   score = sum_d [ max_d * sum_h max(q_hd, 0) + min_d * sum_h min(q_hd, 0) ],
//
// so it costs two products an element whatever the group's size, and the kernel is
// bound by reading 4 D bytes a page and KV head once.  The page table's first `first`
// and newest `last` pages are always taken, then the largest scores up to `budget`,
// ties to the lower index; a NaN score counts as infinite.
//
// The order of the pages is that of the exact scores, not of how fp32 sums round: the
// fp32 scores come with a bound E on their error (below), the K-th largest score T of
// the row puts every page above T + 2E in and every page below T - 2E out, and where
// more pages lie between than are still wanted, those few are summed again in 64 bits.
// (64 bits throughout would be bound by the fp64 units: 1/60 of the fp32 rate.)
//
// One launch: a row (query token, KV head) is cut into chunks of pages, one CTA each;
// the last CTA of a row to finish (a counter per row) selects.  Selection is a radix
// select of 11 + 11 + 10 bits over the row's scores.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/fdec.h"
#include "device_utils.cuh"
#include "fdec_internal.h"

namespace fdec {

namespace {

constexpr int kSelThreads = 256;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kNear = 256;  // pages near the border that are ranked in shared memory

template <int D>
struct SelShape {
    static constexpr int CHUNKS = D / 4;  // 16-byte chunks of a page's two rows
    static constexpr int LPP = D == 64 || D == 192 ? 16 : 32;  // lanes per page
    static constexpr int CPL = CHUNKS / LPP;
    static constexpr int PPW = 32 / LPP;                       // pages per load instruction
    static constexpr int U = CPL >= 3 ? 2 : 8 / CPL;           // load groups in flight
};

// Loads that stay where they are written: scores of other CTAs, after their counter.
__device__ __forceinline__ float ld_cg(const float* p) {
    float v;
    asm volatile("ld.global.cg.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float v;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(v) : "f"(a), "f"(b));
    return v;
}

__device__ __forceinline__ float not_nan(float s) { return s != s ? INFINITY : s; }
__device__ __forceinline__ double not_nan(double s) { return s != s ? static_cast<double>(INFINITY) : s; }

// Unsigned integers in the order of the (non-NaN) floats.
__device__ __forceinline__ uint32_t ordered(float s) {
    const uint32_t b = __float_as_uint(s);
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float from_ordered(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ unsigned long long ordered(double s) {
    const unsigned long long b = __double_as_longlong(s + 0.0);  // -0 as 0
    return (b >> 63) ? ~b : b | (1ull << 63);
}

// Sum of a value over the CTA, to every thread.
__device__ __forceinline__ int block_sum(int v, int* s_sum) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = v;
    __syncthreads();
    int t = 0;
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w) t += s_sum[w];
    return t;
}

struct SelShared {
    union {
        int hist[kBins];
        double weight64[kBins / 2];
    };
    unsigned long long near_key[kNear];
    int near_idx[kNear];
    float err[kSelWarps];
    int sum[kSelWarps];
    int bin, above, near_n, last, cut_idx;
    unsigned long long cut_key;
};

// 64-bit score of one page, by one warp.
template <int D, bool BF16>
__device__ __forceinline__ double score64(const SelectParams& p, const double* w64, int64_t page, int h, int lane) {
    double s = 0.0;
    const uint16_t* rows = reinterpret_cast<const uint16_t*>(p.b_base + page * p.b_sp + h * p.b_sh);
    for (int e = lane; e < 2 * D; e += 32) {
        const int side = e / D, d = e - side * D;
        s += w64[e] * static_cast<double>(load_16bit<BF16>(rows + side * (p.b_st / 2) + d));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kSelThreads) select_pages_kernel(const __grid_constant__ SelectParams p) {
    using S = SelShape<D>;
    constexpr int LPP = S::LPP, CPL = S::CPL, PPW = S::PPW, U = S::U;
    __shared__ SelShared sm;
    __shared__ __align__(16) float s_w[2 * D];  // weights of the minimum row, then of the maximum row
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = blockIdx.x / p.n_chunks;  // (sequence, query, KV head)
    const int chunk = static_cast<int>(blockIdx.x - row * p.n_chunks);
    const int h = static_cast<int>(row % p.hk);
    const int64_t tok = row / p.hk;
    const int b = static_cast<int>(tok / p.q_len);
    const int qi = static_cast<int>(tok - static_cast<int64_t>(b) * p.q_len);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    int64_t L = p.seq_lens[b];
    const int64_t room = static_cast<int64_t>(p.max_pages) << p.page_shift;
    if (L < 0 || L > room) {
        if (tid == 0 && p.err != nullptr) atomicOr(p.err, FDEC_DEVERR_SEQ_LEN);
        L = L < 0 ? 0 : room;
    }
    const int64_t seen = max(static_cast<int64_t>(0), p.causal ? L - p.q_len + qi + 1 : L);
    const int M = static_cast<int>((seen + (1 << p.page_shift) - 1) >> p.page_shift);  // <= max_pages
    const int32_t* table = p.page_table + static_cast<int64_t>(b) * p.pt_stride;
    int32_t* ids = p.page_ids + row * p.budget;
    int32_t* index = p.page_indices != nullptr ? p.page_indices + row * p.budget : nullptr;
    const bool all = M <= p.budget;
    const int n_cand = all ? 0 : M - p.first - p.last;  // >= 1: budget >= first + last
    const int need = all ? 0 : p.budget - p.first - p.last;
    if (need == 0) {  // nothing to choose
        if (chunk != 0) return;
        for (int x = tid; x < p.budget; x += kSelThreads) {
            const int j = all ? (x < M ? x : -1) : (x < p.first ? x : M - p.budget + x);
            ids[x] = j >= 0 ? table[j] : -1;
            if (index != nullptr) index[x] = j;
        }
        if (tid == 0)
            p.counts[row] = static_cast<int32_t>(
                all ? seen : seen - (static_cast<int64_t>(M - p.budget) << p.page_shift));
        return;
    }
    const int n_active = (n_cand + p.chunk - 1) / p.chunk;
    if (chunk >= n_active) return;

    // ---- the weights of this row's two bound rows
    const uint16_t* q = p.q + tok * p.q_st + static_cast<int64_t>(h) * p.group * p.q_sh;
    for (int d = tid; d < D; d += kSelThreads) {
        float neg = 0.f, pos = 0.f;
        for (int g = 0; g < p.group; ++g) {
            const float v = load_16bit<BF16>(q + g * p.q_sh + d);
            // a NaN goes into both sums
            neg += v > 0.f ? 0.f : v;
            pos += v < 0.f ? 0.f : v;
        }
        s_w[d] = neg;
        s_w[D + d] = pos;
    }
    __syncthreads();
    const int sub = lane / LPP, l = lane - sub * LPP;
    float w[CPL][8];
    int64_t off[CPL];  // byte offset of this lane's chunks in a page's rows
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
        const int x = l + LPP * c;  // chunk: min row first, then max row
        const int side = x / (D / 8), k = x - side * (D / 8);
        off[c] = h * p.b_sh + side * p.b_st + k * 16;
#pragma unroll
        for (int e = 0; e < 8; ++e) w[c][e] = s_w[side * D + 8 * k + e];
    }

    // ---- scores of this CTA's pages
    float* scores = p.scores + row * p.max_pages;
    const int begin = chunk * p.chunk, end = min(begin + p.chunk, n_cand);
    float abs_max = 0.f;  // the largest sum of magnitudes that this lane has seen
    for (int i0 = begin + warp * PPW; i0 < end; i0 += kSelWarps * PPW * U) {
        int page[U];
        uint4 raw[U][CPL];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * kSelWarps * PPW + sub;
            page[u] = -1;
            if (i < end) {
                page[u] = table[p.first + i];
                if (page[u] < 0 || page[u] >= p.b_pages) {
                    if (l == 0 && p.err != nullptr) atomicOr(p.err, FDEC_DEVERR_PAGE_ID);
                    page[u] = -1;
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int c = 0; c < CPL; ++c)
                raw[u][c] = page[u] >= 0 ? *reinterpret_cast<const uint4*>(p.b_base + page[u] * p.b_sp + off[c])
                                         : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float s = 0.f, a = 0.f;
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
                const uint32_t v[4] = {raw[u][c].x, raw[u][c].y, raw[u][c].z, raw[u][c].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 f = unpack2<BF16>(v[k]);
                    s = fmaf(f.x, w[c][2 * k], s);
                    s = fmaf(f.y, w[c][2 * k + 1], s);
                    a = fmaf(fabsf(f.x), fabsf(w[c][2 * k]), a);
                    a = fmaf(fabsf(f.y), fabsf(w[c][2 * k + 1]), a);
                }
            }
            abs_max = max_nan(abs_max, a);
#pragma unroll
            for (int o = LPP / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            const int i = i0 + u * kSelWarps * PPW + sub;
            if (l == 0 && i < end) scores[i] = page[u] >= 0 ? s : -INFINITY;
        }
    }
    // The row's largest sum of magnitudes is at most the sum over a page's lanes of each
    // lane's largest (NaN and infinity carry through).
#pragma unroll
    for (int o = LPP / 2; o > 0; o >>= 1) abs_max += __shfl_xor_sync(0xffffffffu, abs_max, o);
#pragma unroll
    for (int o = LPP; o < 32; o <<= 1) abs_max = max_nan(abs_max, __shfl_xor_sync(0xffffffffu, abs_max, o));
    if (lane == 0) sm.err[warp] = abs_max;
    __threadfence();
    __syncthreads();
    if (tid == 0) {
        float a = sm.err[0];
#pragma unroll
        for (int x = 1; x < kSelWarps; ++x) a = max_nan(a, sm.err[x]);
        atomicMax(p.row_abs + row, __float_as_uint(a) & 0x7fffffffu);  // magnitudes order as integers
        __threadfence();
        sm.last = atomicAdd(p.row_count + row, 1u) == static_cast<unsigned>(n_active) - 1u;
    }
    __syncthreads();
    if (!sm.last) return;

    // ---- this CTA is the row's last: select
    __threadfence();
    // Error of an fp32 score: the weights (group - 1 additions of one sign), a chain of
    // 8 CPL products, log2(LPP) additions; in units of 2^-24 of the sum of magnitudes,
    // rounded up, with room for the rounding of that sum itself.
    const float sum_abs = __uint_as_float(atomicAdd(p.row_abs + row, 0u));
    const float E = sum_abs * ((p.group + 8 * CPL + 8) * 6.0e-8f) + 1e-37f;
    auto score_of = [&](int i) { return not_nan(ld_cg(scores + i)); };
    uint32_t prefix = 0;
    int want = need;  // the want-th largest among those with the prefix
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
        const int bits = pass == 2 ? 10 : 11;
        const uint32_t mask = pass == 0 ? 0u : ~0u << (shift + bits);
        for (int x = tid; x < kBins; x += kSelThreads) sm.hist[x] = 0;
        __syncthreads();
        for (int i = tid; i < n_cand; i += kSelThreads) {
            const uint32_t k = ordered(score_of(i));
            if ((k & mask) == prefix) atomicAdd(&sm.hist[(k >> shift) & ((1u << bits) - 1u)], 1);
        }
        __syncthreads();
        // bins from the top: thread t has bins kBins - 8 t - 1 .. kBins - 8 t - 8
        constexpr int PER = kBins / kSelThreads;
        int mine = 0;
#pragma unroll
        for (int x = 0; x < PER; ++x) mine += sm.hist[kBins - 1 - (tid * PER + x)];
        int upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        if (lane == 31) sm.sum[warp] = upto;
        __syncthreads();
        for (int x = 0; x < warp; ++x) upto += sm.sum[x];
        int before = upto - mine;
        if (before < want && want <= upto) {
            for (int x = 0; x < PER; ++x) {
                const int bin = kBins - 1 - (tid * PER + x);
                const int n = sm.hist[bin];
                if (want <= before + n) {
                    sm.bin = bin;
                    sm.above = before;
                    break;
                }
                before += n;
            }
        }
        __syncthreads();
        prefix |= static_cast<uint32_t>(sm.bin) << shift;
        want -= sm.above;
        __syncthreads();
    }
    const float T = from_ordered(prefix);
    const bool sure_E = E < INFINITY;
    // 2 E from T, and a rounding more
    const float lo = sure_E ? T - 2.5f * E : -INFINITY;
    const float hi = sure_E ? T + 2.5f * E : INFINITY;
    int n_hi = 0, n_near = 0;
    for (int i = tid; i < n_cand; i += kSelThreads) {
        const float s = score_of(i);
        n_hi += s > hi;
        n_near += s >= lo && s <= hi;
    }
    n_hi = block_sum(n_hi, sm.sum);
    n_near = block_sum(n_near, sm.sum);
    const int take_near = need - n_hi;  // of the pages near the border: 1 .. n_near
    const bool refine = take_near < n_near;
    unsigned long long* key64 = p.near_keys + row * p.max_pages;
    if (refine) {
        for (int e = tid; e < 2 * D; e += kSelThreads) {
            const int side = e / D, d = e - side * D;
            double v = 0.0;
            for (int g = 0; g < p.group; ++g) {
                const float x = load_16bit<BF16>(q + g * p.q_sh + d);
                v += side == 0 ? (x > 0.f ? 0.f : x) : (x < 0.f ? 0.f : x);
            }
            sm.weight64[e] = v;
        }
        if (tid == 0) sm.near_n = 0;
        __syncthreads();
        for (int i0 = warp * 32; i0 < n_cand; i0 += kSelThreads) {
            const int i = i0 + lane;
            const float s = i < n_cand ? score_of(i) : 0.f;
            unsigned todo = __ballot_sync(0xffffffffu, i < n_cand && s >= lo && s <= hi);
            while (todo != 0u) {
                const int x = __ffs(todo) - 1;
                todo &= todo - 1;
                const int id = table[p.first + i0 + x];
                const bool ok = id >= 0 && id < p.b_pages;
                const double v = ok ? not_nan(score64<D, BF16>(p, sm.weight64, id, h, lane))
                                    : -static_cast<double>(INFINITY);
                if (lane == 0) {
                    key64[i0 + x] = ordered(v);
                    const int at = atomicAdd(&sm.near_n, 1);
                    if (at < kNear) {
                        sm.near_key[at] = ordered(v);
                        sm.near_idx[at] = i0 + x;
                    }
                }
            }
        }
        __threadfence_block();
        __syncthreads();
        if (n_near <= kNear) {  // the rank of each among them
            for (int x = tid; x < n_near; x += kSelThreads) {
                const unsigned long long k = sm.near_key[x];
                const int i = sm.near_idx[x];
                int rank = 0;
                for (int y = 0; y < n_near; ++y)
                    rank += sm.near_key[y] > k || (sm.near_key[y] == k && sm.near_idx[y] < i);
                if (rank == take_near - 1) {
                    sm.cut_key = k;
                    sm.cut_idx = i;
                }
            }
        } else {  // many (equal pages, infinities): the key bit by bit, then the index
            auto near = [&](int i) {
                const float s = score_of(i);
                return s >= lo && s <= hi;
            };
            unsigned long long cut = 0;
            for (int bit = 63; bit >= 0; --bit) {
                const unsigned long long t = cut | (1ull << bit);
                int n = 0;
                for (int i = tid; i < n_cand; i += kSelThreads) n += near(i) && key64[i] >= t;
                if (block_sum(n, sm.sum) >= take_near) cut = t;
            }
            int n = 0;
            for (int i = tid; i < n_cand; i += kSelThreads) n += near(i) && key64[i] > cut;
            const int ties = take_near - block_sum(n, sm.sum);  // of those equal to the cut: the first ones
            int low = 0, high = n_cand - 1;  // smallest index with `ties` of them at or below it
            while (low < high) {
                const int mid = (low + high) / 2;
                n = 0;
                for (int i = tid; i <= mid; i += kSelThreads) n += near(i) && key64[i] == cut;
                if (block_sum(n, sm.sum) >= ties)
                    high = mid;
                else
                    low = mid + 1;
            }
            if (tid == 0) {
                sm.cut_key = cut;
                sm.cut_idx = low;
            }
        }
        __syncthreads();
    }
    auto take = [&](int i) {
        const float s = score_of(i);
        if (s > hi) return true;
        if (!(s >= lo)) return false;
        if (!refine) return true;
        const unsigned long long k = key64[i];
        return k > sm.cut_key || (k == sm.cut_key && i <= sm.cut_idx);
    };

    // ---- write the taken pages in order: each warp a run of the candidates
    const int seg = (n_cand + kSelWarps * 32 - 1) / (kSelWarps * 32) * 32;
    const int s0 = min(warp * seg, n_cand), s1 = min(s0 + seg, n_cand);
    int n_taken = 0;
    for (int i0 = s0; i0 < s1; i0 += 32) n_taken += __popc(__ballot_sync(0xffffffffu, i0 + lane < s1 && take(i0 + lane)));
    __syncthreads();
    if (lane == 0) sm.sum[warp] = n_taken;
    __syncthreads();
    int at = p.first;
    for (int x = 0; x < warp; ++x) at += sm.sum[x];
    for (int i0 = s0; i0 < s1; i0 += 32) {
        const int i = i0 + lane;
        const bool t = i < s1 && take(i);
        const unsigned m = __ballot_sync(0xffffffffu, t);
        if (t) {
            const int x = at + __popc(m & ((1u << lane) - 1u));
            ids[x] = table[p.first + i];
            if (index != nullptr) index[x] = p.first + i;
        }
        at += __popc(m);
    }
    for (int x = tid; x < p.first + p.last; x += kSelThreads) {
        const int at2 = x < p.first ? x : p.budget - p.last + (x - p.first);
        const int j = x < p.first ? x : M - p.last + (x - p.first);
        ids[at2] = table[j];
        if (index != nullptr) index[at2] = j;
    }
    if (tid == 0) {
        p.counts[row] = static_cast<int32_t>(seen - (static_cast<int64_t>(M - p.budget) << p.page_shift));
        p.row_count[row] = 0u;  // as the next call expects them
        p.row_abs[row] = 0u;
    }
}

template <int D>
cudaError_t launch_select_d(const SelectParams& p, int64_t blocks, bool bf16, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
    cfg.blockDim = dim3(kSelThreads, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return bf16 ? cudaLaunchKernelEx(&cfg, select_pages_kernel<D, true>, p)
                : cudaLaunchKernelEx(&cfg, select_pages_kernel<D, false>, p);
}

}  // namespace

cudaError_t launch_select_pages(SelectParams p, int head_dim, bool bf16, int num_sms, cudaStream_t s) {
    const int64_t rows = static_cast<int64_t>(p.batch) * p.q_len * p.hk;
    const int64_t cand = std::max(1, p.max_pages - p.first - p.last);
    // Pages per CTA: enough CTAs to fill the machine several times over (rows differ in
    // length, and the CTAs that select leave others to stream), none below 32 pages.
    int64_t chunk = (rows * cand + num_sms * 12 - 1) / (num_sms * 12);
    chunk = std::min<int64_t>(std::max<int64_t>((chunk + 31) / 32 * 32, 32), (cand + 31) / 32 * 32);
    // at most 2^31 - 1 CTAs
    while (rows * ((cand + chunk - 1) / chunk) > INT32_MAX && chunk < cand) chunk *= 2;
    p.chunk = static_cast<int>(chunk);
    p.n_chunks = static_cast<int>((cand + chunk - 1) / chunk);
    const int64_t blocks = rows * p.n_chunks;
    switch (head_dim) {
        case 64: return launch_select_d<64>(p, blocks, bf16, s);
        case 128: return launch_select_d<128>(p, blocks, bf16, s);
        case 192: return launch_select_d<192>(p, blocks, bf16, s);
        case 256: return launch_select_d<256>(p, blocks, bf16, s);
        case 512: return launch_select_d<512>(p, blocks, bf16, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace fdec
