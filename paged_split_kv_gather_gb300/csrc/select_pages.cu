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
// (64 bits throughout would be bound by the fp64 units: 1/60 of the fp32 rate.)  E is of the
// finite terms: infinite and NaN ones decide a score exactly.  Where one hides the bound of
// a chunk, the choosing CTA reads that chunk once more (4096 pages, one of them with a NaN:
// 40 us; of 16384 56); where scores are exact, as with weights of 0 or pages of zeros, ties are
// found by index (13 us, 30 us).  Only many pages of equal or nearly equal nonzero scores
// around the border are all scored in 64 bits, by their row's CTA: 0.2 us a page.
//
// Two launches.  score_pages_kernel streams the bounds: a row (query token, KV head) is
// cut into chunks of pages, one CTA each.  choose_pages_kernel, its programmatic
// dependent, has one CTA a row: the row's scores go to shared memory, the bin of the
// K-th largest among 256 over their range is found, and the few scores in and near that
// bin are compared with each other.  (Choosing in the row's last CTA to finish scoring,
// counted by an atomic, was measured first: the count's fences cost every CTA 1.4-2.1 us,
// and the choosing CTAs' registers and shared memory took from what streams beside them.)
//
// GB300, us a call in a stream of calls: 4 rows of 4096 pages (head_dim 128) 10.0, of
// which scoring 3 and choosing 5; 64 x 8 ragged rows of up to 2048 pages (head_dim 192,
// 308 MB) 68, scoring 57 of them at 5.4 TB/s; 16 query tokens x 8 heads of 512 pages 13.3.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "../../include/fdec.h"
#include "device_utils.cuh"
#include "fdec_internal.h"

namespace fdec {

namespace {

constexpr int kScoreThreads = 256;
constexpr int kScoreWarps = kScoreThreads / 32;
constexpr int kBins = 256;
constexpr int kNear = 256;  // keys that are compared each with each
constexpr int kMinChunk = 32;  // pages a scoring CTA has at least

template <int D>
struct SelShape {
    static constexpr int CHUNKS = D / 4;  // 16-byte chunks of a page's two rows
    static constexpr int LPP = D == 64 || D == 192 ? 16 : 32;  // lanes per page
    static constexpr int CPL = CHUNKS / LPP;
    static constexpr int PPW = 32 / LPP;                       // pages per load instruction
    static constexpr int U = CPL <= 1 ? 8 : CPL <= 3 ? 4 : 2;  // page groups of a round
    // Rounds of a warp that its ring of shared memory holds, all but one of them in flight
    // while it computes: 12 or 16 loads of 16 bytes a thread beside those computed on.  As
    // registers there was room for 8 to 12 and none beside (a batch of 64 ragged rows, the
    // whole call: 71 us; rounds of half the size 68, of a quarter 80; this 66).
    static constexpr int R = 24 / (U * CPL);
    static constexpr int CTAS = 2;  // resident an SM
    static constexpr int SMEM = R * U * CPL * kScoreThreads * 16;
};

// Loads from L2 that stay where they are written, before or after a wait: what the scoring
// launch read too, and its scores.
__device__ __forceinline__ float ld_cg(const float* p) {
    float v;
    asm volatile("ld.global.cg.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ int ld_cg(const int32_t* p) {
    int v;
    asm volatile("ld.global.cg.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ uint16_t ld_cg(const uint16_t* p) {
    uint16_t v;
    asm volatile("ld.global.cg.u16 %0, [%1];" : "=h"(v) : "l"(p) : "memory");
    return v;
}
template <bool BF16>
__device__ __forceinline__ float to_float(uint16_t v) {
    return unpack2<BF16>(v).x;
}
__device__ __forceinline__ float4 ld_cg4(const float* p) {
    float4 v;
    asm volatile("ld.global.cg.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float v;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(v) : "f"(a), "f"(b));
    return v;
}

// Maxima of two pairs of 16-bit magnitudes: they order as integers, NaN above infinity.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The magnitudes of two 16-bit elements, 0 where they are not finite.
template <bool BF16>
__device__ __forceinline__ uint32_t finite_u16x2(uint32_t w) {
    constexpr uint32_t INF = BF16 ? 0x7f80u : 0x7c00u;
    const uint32_t m = w & 0x7fff7fffu;
    return ((m & 0xffffu) < INF ? m & 0xffffu : 0u) | ((m >> 16) < INF ? m & 0xffff0000u : 0u);
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

// What both kernels derive from a row's length.
struct SelRow {
    int64_t seen;  // tokens that the query sees
    int M;         // pages of them, <= max_pages
    int n_cand;    // pages to choose among (0: all are taken, or none is free)
    int need;      // pages to choose
    bool all, bad;
};

__device__ __forceinline__ SelRow sel_row(const SelectParams& p, int64_t L, int qi) {
    SelRow r;
    const int64_t room = static_cast<int64_t>(p.max_pages) << p.page_shift;
    r.bad = L < 0 || L > room;
    if (r.bad) L = L < 0 ? 0 : room;
    r.seen = max(static_cast<int64_t>(0), p.causal ? L - p.q_len + qi + 1 : L);
    r.M = static_cast<int>((r.seen + (1 << p.page_shift) - 1) >> p.page_shift);
    r.all = r.M <= p.budget;
    r.need = r.all ? 0 : p.budget - p.first - p.last;
    r.n_cand = r.need == 0 ? 0 : r.M - p.first - p.last;  // > need
    return r;
}

// Sum over the LPP lanes of a page of N pages' values at once: halves of the values are
// exchanged for halves of the lanes (N - 1 + log2(LPP / N) shuffles instead of
// N log2(LPP)).  s[0] of lane l is then the sum of value (l % LPP) * N / LPP.
template <int N, int O>
__device__ __forceinline__ void fold(float* s, int lane) {
    if constexpr (O > 0) {
        if constexpr (N > 1) {
            const bool up = (lane & O) != 0;
#pragma unroll
            for (int k = 0; k < N / 2; ++k) {
                const float give = up ? s[k] : s[k + N / 2];
                const float keep = up ? s[k + N / 2] : s[k];
                s[k] = keep + __shfl_xor_sync(0xffffffffu, give, O);
            }
            fold<N / 2, O / 2>(s, lane);
        } else {
            s[0] += __shfl_xor_sync(0xffffffffu, s[0], O);
            fold<1, O / 2>(s, lane);
        }
    }
}

// 64-bit score of one page, by one warp: 16-byte chunks of the two rows, all in flight.
template <bool BF16>
__device__ __forceinline__ double score64(const SelectParams& p, const double* w64, int64_t page, int h, int lane) {
    constexpr int MAX = 4;  // chunks a lane at head_dim 512
    const int per_row = p.head_dim / 8, n = 2 * per_row;
    const uint8_t* rows = p.b_base + page * p.b_sp + h * p.b_sh;
    uint4 raw[MAX];
#pragma unroll
    for (int c = 0; c < MAX; ++c) {
        const int x = lane + 32 * c, side = x >= per_row ? 1 : 0;
        raw[c] = x < n ? *reinterpret_cast<const uint4*>(rows + side * p.b_st + (x - side * per_row) * 16)
                       : make_uint4(0u, 0u, 0u, 0u);
    }
    double s = 0.0;
#pragma unroll
    for (int c = 0; c < MAX; ++c) {
        const int x = lane + 32 * c;
        if (x >= n) continue;
        const uint32_t v[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 f = unpack2<BF16>(v[k]);
            s = fma(w64[8 * x + 2 * k], static_cast<double>(f.x), s);
            s = fma(w64[8 * x + 2 * k + 1], static_cast<double>(f.y), s);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// An upper bound, for one of nw warps, of the finite terms' sums of magnitudes: of the chunks
// where infinite or NaN terms hid it (this warp's pages are read once more), and of the others.
// Such terms make their page's score infinite or NaN however it is summed; only the finite
// ones' sums have an error to bound.
// (Finding it while scoring was measured first: a select and an addition more for every word
// cost each call 1-3 %, a second pass in the scoring kernel's registers its spills.)
template <bool BF16>
__device__ __noinline__ float finite_magnitudes(const SelectParams& p, const double* w64, const float* chunk_abs,
                                                const int32_t* table, int h, int n_cand, int nw) {
    constexpr int U = 2;  // pages in flight: few registers, which the kernel pays in every call
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per_row = p.head_dim / 8;
    float sum = 0.f, others = 0.f;
#pragma unroll 1
    for (int x = lane; x < 2 * per_row; x += 32) {  // this lane's 16-byte chunks of the two rows
        const int side = x >= per_row ? 1 : 0;
        const uint8_t* rows = p.b_base + h * p.b_sh + side * p.b_st + (x - side * per_row) * 16;
        uint32_t top[4] = {0u, 0u, 0u, 0u};
#pragma unroll 1
        for (int begin = 0; begin < n_cand; begin += p.chunk) {
            const float known = ld_cg(chunk_abs + begin / p.chunk);
            if (known < INFINITY) {
                others = fmaxf(others, known);
                continue;
            }
            const int end = min(begin + p.chunk, n_cand);
#pragma unroll 1
            for (int i = begin + warp; i < end; i += nw * U) {
                uint4 raw[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int id = i + u * nw < end ? table[p.first + i + u * nw] : -1;
                    raw[u] = make_uint4(0u, 0u, 0u, 0u);
                    if (id >= 0 && id < p.b_pages) raw[u] = *reinterpret_cast<const uint4*>(rows + id * p.b_sp);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    top[0] = max_u16x2(top[0], finite_u16x2<BF16>(raw[u].x));
                    top[1] = max_u16x2(top[1], finite_u16x2<BF16>(raw[u].y));
                    top[2] = max_u16x2(top[2], finite_u16x2<BF16>(raw[u].z));
                    top[3] = max_u16x2(top[3], finite_u16x2<BF16>(raw[u].w));
                }
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 t = unpack2<BF16>(top[k]);
            const float wx = fabsf(__double2float_rn(w64[8 * x + 2 * k]));
            const float wy = fabsf(__double2float_rn(w64[8 * x + 2 * k + 1]));
            if (wx < INFINITY) sum += t.x * wx;
            if (wy < INFINITY) sum += t.y * wy;
        }
    }
    __syncwarp();
    others = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(others)));  // (not negative)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return fmaxf(fmaxf(sum, others), 1.2e-38f);
}

// QB: query tokens of a sequence that one CTA scores against the pages it reads, 1, 2 or 4
// (with more of them in the call, q_len / QB such groups).
template <int D, bool BF16, int QB>
__global__ void __launch_bounds__(kScoreThreads, SelShape<D>::CTAS)
score_pages_kernel(const __grid_constant__ SelectParams p) {
    using S = SelShape<D>;
    constexpr int LPP = S::LPP, CPL = S::CPL, PPW = S::PPW, U = S::U;
    // Weights of the chunks (of the minimum row, then of the maximum row): elements 0 .. 3
    // of every chunk, then 4 .. 7 (a warp's 16-byte loads of them meet no bank twice).
    __shared__ __align__(16) float4 s_w[QB][2][S::CHUNKS];
    __shared__ float s_abs[QB][kScoreWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t unit = blockIdx.x / p.n_chunks;  // (sequence, group of query tokens, KV head)
    const int chunk = static_cast<int>(blockIdx.x - unit * p.n_chunks);
    const int h = static_cast<int>(unit % p.hk);
    const int64_t seq_group = unit / p.hk;
    const int q_groups = (p.q_len + QB - 1) / QB;
    const int b = static_cast<int>(seq_group / q_groups);
    const int qi = static_cast<int>(seq_group - static_cast<int64_t>(b) * q_groups) * QB;  // the first of them
    const int64_t tok = static_cast<int64_t>(b) * p.q_len + qi;
    // The choosing kernel may start only once every CTA here has passed its wait: it then
    // may read this launch's inputs before its own.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // Requested together: the length, this warp's first page ids, the query rows.
    const int64_t L = p.seq_lens[b];
    const int32_t* table = p.page_table + static_cast<int64_t>(b) * p.pt_stride;
    const int sub = lane / LPP, l = lane - sub * LPP;
    const int begin = chunk * p.chunk;
    // Ids of this warp's round k (0 where there is none).
    auto load_ids = [&](int k, int stop, int (&id)[U]) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = begin + (warp + (k * U + u) * kScoreWarps) * PPW + sub;
            id[u] = i < stop ? table[p.first + i] : 0;
        }
    };
    int id[U];
    load_ids(0, min(begin + p.chunk, p.max_pages - p.first), id);
    const uint16_t* q = p.q + tok * p.q_st + static_cast<int64_t>(h) * p.group * p.q_sh;
    float q0[8];  // element tid of the group's first eight heads
#pragma unroll
    for (int g = 0; g < 8; ++g) q0[g] = tid < D && g < p.group ? load_16bit<BF16>(q + g * p.q_sh + tid) : 0.f;
    int end[QB], end_all = 0;  // where this chunk ends for each query token (it may not begin)
#pragma unroll
    for (int y = 0; y < QB; ++y) {
        const int n = qi + y < p.q_len ? sel_row(p, L, qi + y).n_cand : 0;
        end[y] = min(begin + p.chunk, n);
        end_all = max(end_all, end[y]);
    }
    if (begin >= end_all) return;

    // ---- the weights of the two bound rows
#pragma unroll
    for (int y = 0; y < QB; ++y) {
        const uint16_t* qy = q + y * p.q_st;
        const bool there = qi + y < p.q_len;
        for (int d = tid; d < D; d += kScoreThreads) {
            float neg = 0.f, pos = 0.f;
            for (int g0 = 0; g0 < p.group; g0 += 8) {
                if (y != 0 || d != tid || g0 != 0) {
#pragma unroll
                    for (int g = 0; g < 8; ++g)
                        q0[g] = there && g0 + g < p.group ? load_16bit<BF16>(qy + (g0 + g) * p.q_sh + d) : 0.f;
                }
#pragma unroll
                for (int g = 0; g < 8; ++g) {  // a NaN goes into both sums
                    neg += q0[g] > 0.f ? 0.f : q0[g];
                    pos += q0[g] < 0.f ? 0.f : q0[g];
                }
            }
            float* to = reinterpret_cast<float*>(&s_w[y][(d >> 2) & 1][d / 8]) + (d & 3);
            to[0] = neg;
            to[4 * (D / 8)] = pos;
        }
    }
    __syncthreads();
    const uint8_t* base = p.b_base + h * p.b_sh;
    int64_t off[CPL];  // byte offset of this lane's chunks in a page's rows
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
        const int x = l + LPP * c, side = x / (D / 8);
        off[c] = side * p.b_st + (x - side * (D / 8)) * 16;
    }

    // ---- scores of this CTA's pages
    float* scores = p.scores + (tok * p.hk + h) * p.score_stride;
    const int64_t q_step = p.hk * p.score_stride;  // to the next query token's scores
    uint32_t top[CPL][4];  // largest magnitude that each of this lane's elements has had
#pragma unroll
    for (int c = 0; c < CPL; ++c)
#pragma unroll
        for (int k = 0; k < 4; ++k) top[c][k] = 0u;
    // The bounds come through a ring in shared memory of which each thread reads only what
    // it has copied itself: its own copies' completion is all it waits for.
    extern __shared__ __align__(16) uint4 ring[];
    const int n_rounds = max(0, (end_all - (begin + warp * PPW) + kScoreWarps * PPW * U - 1) / (kScoreWarps * PPW * U));
    uint64_t bad = 0u;  // per round in flight, U bits: groups whose page id is outside the pool (page 0 is read)
    auto issue = [&](int k) {
        bad <<= U;
        if (k < n_rounds) {
            const int id0 = __shfl_sync(0xffffffffu, id[0], 0);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                // groups past the end read the round's first page again; nothing is stored for them
                const int i = begin + (warp + (k * U + u) * kScoreWarps) * PPW + sub;
                const int from = i < end_all ? id[u] : id0;
                const bool in = from >= 0 && from < p.b_pages;
                if (!in) bad |= 1u << u;
                const uint8_t* rows = base + static_cast<int64_t>(in ? from : 0) * p.b_sp;
#pragma unroll
                for (int c = 0; c < CPL; ++c)
                    cp_async_16(smem_addr(&ring[(((k % S::R) * U + u) * CPL + c) * kScoreThreads + tid]), rows + off[c]);
            }
            load_ids(k + 1, end_all, id);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll 1
    for (int k = 0; k < S::R - 1; ++k) issue(k);
#pragma unroll 1
    for (int k = 0; k < n_rounds; ++k) {
        issue(k + S::R - 1);
        asm volatile("cp.async.wait_group %0;" ::"n"(S::R - 1) : "memory");
        float2 a[QB][U];  // even and odd elements
#pragma unroll
        for (int y = 0; y < QB; ++y)
#pragma unroll
            for (int u = 0; u < U; ++u) a[y][u] = make_float2(0.f, 0.f);
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
            float2 w[QB][4];
#pragma unroll
            for (int y = 0; y < QB; ++y) {
                const float4 w0 = s_w[y][0][l + LPP * c], w1 = s_w[y][1][l + LPP * c];
                w[y][0] = make_float2(w0.x, w0.y), w[y][1] = make_float2(w0.z, w0.w);
                w[y][2] = make_float2(w1.x, w1.y), w[y][3] = make_float2(w1.z, w1.w);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint4 raw = ring[(((k % S::R) * U + u) * CPL + c) * kScoreThreads + tid];
                const uint32_t v[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = unpack2<BF16>(v[e]);
#pragma unroll
                    for (int y = 0; y < QB; ++y) a[y][u] = __ffma2_rn(f, w[y][e], a[y][u]);
                    top[c][e] = max_u16x2(top[c][e], v[e] & 0x7fff7fffu);
                }
            }
        }
        constexpr int LPU = LPP / U;  // lanes that end up with the same page
        const unsigned out = static_cast<unsigned>(bad >> (U * (S::R - 1))) & ((1u << U) - 1u);
        const int u_mine = l / LPU;
        const int i = begin + (warp + (k * U + u_mine) * kScoreWarps) * PPW + sub;
        const bool out_mine = (out >> u_mine) & 1u;
#pragma unroll
        for (int y = 0; y < QB; ++y) {
            float s[U];
#pragma unroll
            for (int u = 0; u < U; ++u) s[u] = a[y][u].x + a[y][u].y;
            fold<U, LPP / 2>(s, lane);
            if (l % LPU == 0 && i < end[y]) scores[y * q_step + i] = out_mine ? -INFINITY : s[0];
        }
        if (l % LPU == 0 && i < end_all && out_mine && p.err != nullptr) atomicOr(p.err, FDEC_DEVERR_PAGE_ID);
    }
    // A page's sum of magnitudes is at most the sum of each element's largest times its
    // weight (NaN and infinity carry through); 0 only where all elements are.
    uint32_t any = 0u;
#pragma unroll
    for (int c = 0; c < CPL; ++c) any |= top[c][0] | top[c][1] | top[c][2] | top[c][3];
    const float least = any != 0u ? 1.2e-38f : 0.f;
#pragma unroll
    for (int y = 0; y < QB; ++y) {
        float abs_max = 0.f;
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
            const float4 w0 = s_w[y][0][l + LPP * c], w1 = s_w[y][1][l + LPP * c];
            const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 t = unpack2<BF16>(top[c][k]);
                abs_max += t.x * fabsf(w[2 * k]);
                abs_max += t.y * fabsf(w[2 * k + 1]);
            }
        }
        abs_max = max_nan(abs_max, least);
#pragma unroll
        for (int o = LPP / 2; o > 0; o >>= 1) abs_max += __shfl_xor_sync(0xffffffffu, abs_max, o);
#pragma unroll
        for (int o = LPP; o < 32; o <<= 1) abs_max = max_nan(abs_max, __shfl_xor_sync(0xffffffffu, abs_max, o));
        if (lane == 0) s_abs[y][warp] = abs_max;
    }
    __syncthreads();
    if (tid < QB && qi + tid < p.q_len) {
        float a = s_abs[tid][0];
#pragma unroll
        for (int x = 1; x < kScoreWarps; ++x) a = max_nan(a, s_abs[tid][x]);
        p.chunk_abs[((tok + tid) * p.hk + h) * p.abs_stride + chunk] = a;
    }
}

template <int NW>
struct ChooseShared {
    // Scores held at a time, 16 a thread: 4096, 8192 or 16384.  A row that fits is loaded once,
    // a longer one again in each pass (a row of 8192 pages: 11.8 us whole, 15.2 in halves).
    static constexpr int TILE = NW * 32 * 16;
    uint32_t key[TILE];  // a tile's scores as ordered integers; then its taken pages
    double weight64[2 * 512];
    int hist[kBins];
    unsigned long long near_key[kNear];
    uint32_t near_k32[kNear];
    int near_idx[kNear];
    float abs_max[NW];
    int sum[NW], sum_hi[NW], sum_taken[NW];  // one use each: no barrier between uses
    uint32_t kmin[NW], kmax[NW], cut32;
    int bin, above, near_n, cut_idx;
    unsigned long long cut_key;
};

// (The bounds on CTAs an SM: the registers without finite_magnitudes, which is rarely called;
// with 64 instead of 48 at 8 warps a batch of 64 x 8 rows took 43 us instead of 40.)
template <bool BF16, int NW>
__global__ void __launch_bounds__(NW * 32, NW == 8 ? 5 : NW == 16 ? 2 : 1) choose_pages_kernel(const __grid_constant__ SelectParams p) {
    constexpr int NT = NW * 32;
    static_assert(NT >= kBins && NT >= kNear && NW <= 32, "one bin, one near key a thread");
    constexpr int kTile = ChooseShared<NW>::TILE;
    extern __shared__ __align__(16) unsigned char choose_smem[];
    ChooseShared<NW>& sm = *reinterpret_cast<ChooseShared<NW>*>(choose_smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = blockIdx.x;
    const int h = static_cast<int>(row % p.hk);
    const int64_t tok = row / p.hk;
    const int b = static_cast<int>(tok / p.q_len);
    const int qi = static_cast<int>(tok - static_cast<int64_t>(b) * p.q_len);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // The scoring launch's own inputs are complete here (all its CTAs have passed their
    // wait for whatever came before); they are read past L1, its scores after the wait below.
    const SelRow r = sel_row(p, ld_cg(p.seq_lens + b), qi);
    const int n_cand = r.n_cand, need = r.need;
    const int32_t* table = p.page_table + static_cast<int64_t>(b) * p.pt_stride;
    int32_t* ids = p.page_ids + row * p.budget;
    int32_t* index = p.page_indices != nullptr ? p.page_indices + row * p.budget : nullptr;
    if (tid < kBins) sm.hist[tid] = 0;
    if (tid == 0) {
        sm.near_n = 0;
        if (r.bad && p.err != nullptr) atomicOr(p.err, FDEC_DEVERR_SEQ_LEN);
        // all pages but the newest are full
        p.counts[row] = static_cast<int32_t>(
            r.all ? r.seen : r.seen - (static_cast<int64_t>(r.M - p.budget) << p.page_shift));
    }
    if (need == 0) {  // nothing to choose
        for (int x = tid; x < p.budget; x += NT) {
            const int j = r.all ? (x < r.M ? x : -1) : (x < p.first ? x : r.M - p.budget + x);
            ids[x] = j >= 0 ? ld_cg(table + j) : -1;
            if (index != nullptr) index[x] = j;
        }
        // The next kernel waits for this grid alone, and it may overwrite what the scoring
        // CTAs still read: this grid must not complete before them.
        asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
    }
    for (int x = tid; x < p.first + p.last; x += NT) {
        const int to = x < p.first ? x : p.budget - p.last + (x - p.first);
        const int j = x < p.first ? x : r.M - p.last + (x - p.first);
        ids[to] = ld_cg(table + j);
        if (index != nullptr) index[to] = j;
    }
    // The weights in 64 bits, for pages near the border (computed while the scoring launch
    // still runs: 2 us of a call that needs them, if left until it does).
    const uint16_t* q = p.q + tok * p.q_st + static_cast<int64_t>(h) * p.group * p.q_sh;
    for (int d = tid; d < p.head_dim; d += NT) {
        double neg = 0.0, pos = 0.0;
        for (int g0 = 0; g0 < p.group; g0 += 4) {
            float x[4];
#pragma unroll
            for (int g = 0; g < 4; ++g) x[g] = g0 + g < p.group ? to_float<BF16>(ld_cg(q + (g0 + g) * p.q_sh + d)) : 0.f;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                if (!(x[g] > 0.f)) neg += x[g];  // a NaN goes into both sums
                if (!(x[g] < 0.f)) pos += x[g];
            }
        }
        sm.weight64[d] = neg;
        sm.weight64[p.head_dim + d] = pos;
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the scores
    const float* scores = p.scores + row * p.score_stride;
    // The row's largest sum of magnitudes, reduced with the tile's load below.
    float sum_abs = 0.f;
    const int n_active = (n_cand + p.chunk - 1) / p.chunk;
    for (int x = tid; x < n_active; x += NT) sum_abs = max_nan(sum_abs, p.chunk_abs[row * p.abs_stride + x]);
    // The row's scores as ordered integers, in shared memory (in tiles of kTile, loaded
    // again in each pass, for longer rows).  The loops over them are not unrolled: this
    // code runs once a row, and fetching it costs more than its steps.
    const int n_tiles = (n_cand + kTile - 1) / kTile;
    uint32_t r_min = ~0u, r_max = 0u;  // range of what this thread has loaded
    auto load = [&](int t) {
        const int n = min(kTile, n_cand - t * kTile);
        const float* src = scores + t * kTile;
        for (int i = 4 * tid; i < n; i += 4 * NT) {  // whole vectors: the row's stride is a multiple of 4
            const float4 f = ld_cg4(src + i);
            const uint4 k = make_uint4(ordered(not_nan(f.x) + 0.f), ordered(not_nan(f.y) + 0.f),  // -0 as 0
                                       ordered(not_nan(f.z) + 0.f), ordered(not_nan(f.w) + 0.f));
            *reinterpret_cast<uint4*>(sm.key + i) = k;
            r_min = min(r_min, k.x), r_max = max(r_max, k.x);
            if (i + 1 < n) r_min = min(r_min, k.y), r_max = max(r_max, k.y);
            if (i + 2 < n) r_min = min(r_min, k.z), r_max = max(r_max, k.z);
            if (i + 3 < n) r_min = min(r_min, k.w), r_max = max(r_max, k.w);
        }
        __syncthreads();
    };
    // f(key, index) over the row's pages
    auto each = [&](auto&& f) {
        for (int t = 0; t < n_tiles; ++t) {
            if (n_tiles > 1) {
                __syncthreads();
                load(t);
            }
            const int n = min(kTile, n_cand - t * kTile);
#pragma unroll 2
            for (int i = tid; i < n; i += NT) f(sm.key[i], t * kTile + i);
        }
    };
    for (int t = 0; t < n_tiles; ++t) {
        if (t > 0) __syncthreads();
        load(t);
    }
    uint32_t k_min = __reduce_min_sync(0xffffffffu, r_min), k_max = __reduce_max_sync(0xffffffffu, r_max);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum_abs = max_nan(sum_abs, __shfl_xor_sync(0xffffffffu, sum_abs, o));
    if (lane == 0) {
        sm.kmin[warp] = k_min;
        sm.kmax[warp] = k_max;
        sm.abs_max[warp] = sum_abs;
    }
    __syncthreads();
    k_min = __reduce_min_sync(0xffffffffu, lane < NW ? sm.kmin[lane] : ~0u);
    k_max = __reduce_max_sync(0xffffffffu, lane < NW ? sm.kmax[lane] : 0u);
    // Error of an fp32 score: the weights (group - 1 additions of one sign), a chain of
    // 4 CPL products in each of two sums, 1 + log2(LPP) additions (at most 16 and 6); in
    // units of 2^-24 of the sum of magnitudes, with room for the rounding of that sum (and
    // 1e-37 for products below the normal range).  0 where every finite term is.
    sum_abs = lane < NW ? sm.abs_max[lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum_abs = max_nan(sum_abs, __shfl_xor_sync(0xffffffffu, sum_abs, o));
    // Whether f(w) holds for a weight of the row (of all threads, to all threads).
    auto any_weight = [&](auto&& f) {
        bool is = false;
        for (int d = tid; d < 2 * p.head_dim; d += NT) is = is || f(sm.weight64[d]);
        return __syncthreads_or(is) != 0;
    };
    if (!(sum_abs < INFINITY)) {
        if (any_weight([](double w) { return w != w; })) {
            sum_abs = 0.f;  // every score is NaN
        } else if (!any_weight([](double w) { return fabs(w) > 1.7e38 && fabs(w) < static_cast<double>(INFINITY); })) {
            // (else a weight is finite, but perhaps not in 32 bits)
            const float mine = finite_magnitudes<BF16>(p, sm.weight64, p.chunk_abs + row * p.abs_stride, table, h, n_cand, NW);
            if (lane == 0) sm.abs_max[warp] = mine;
            __syncthreads();
            sum_abs = lane < NW ? sm.abs_max[lane] : 0.f;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum_abs = fmaxf(sum_abs, __shfl_xor_sync(0xffffffffu, sum_abs, o));
        }
    }
    const float E = sum_abs == 0.f ? 0.f : sum_abs * ((p.group + p.chain + 9) * 6.0e-8f) + 1e-37f;
    const bool sure_E = E < INFINITY;
    const float margin = 2.5f * E;  // 2 E, and a rounding more
    unsigned long long* key64 = p.near_keys + row * p.max_pages;
    // The want-th largest key T lies in [k_min, k_max]: 256 equal bins over that range and
    // the one that T is in, until few keys lie within the margin of that bin.  Keys above
    // (`hi`) are taken, keys below (`lo`) are not.
    int want = need, n_near, take_near;
    uint32_t lo, hi;
    // The bin of sm.hist that the want-th largest key is in (sm.bin), and how many lie above it.
    auto find_bin = [&]() {
        __syncthreads();
        // bins from the top, one a thread
        const int mine = tid < kBins ? sm.hist[kBins - 1 - tid] : 0;
        int upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        if (lane == 31) sm.sum[warp] = upto;
        __syncthreads();
        upto += __reduce_add_sync(0xffffffffu, lane < warp ? sm.sum[lane] : 0);
        if (tid < kBins && upto - mine < want && want <= upto) {
            sm.bin = kBins - 1 - tid;
            sm.above = upto - mine;
        }
        __syncthreads();
    };
    while (true) {
        const int shift = max(0, 24 - __clz(k_max - k_min));  // (k_max - k_min) >> shift < kBins = 256
        each([&](uint32_t k, int) {
            if (k >= k_min && k <= k_max) atomicAdd(&sm.hist[(k - k_min) >> shift], 1);
        });
        find_bin();
        want -= sm.above;
        k_min += static_cast<uint32_t>(sm.bin) << shift;
        k_max -= k_max - k_min > (1u << shift) - 1u ? k_max - k_min - ((1u << shift) - 1u) : 0u;
        lo = sure_E ? ordered(from_ordered(k_min) - margin + 0.f) : 1u;
        hi = sure_E ? ordered(from_ordered(k_max) + margin + 0.f) : ~0u;
        int n_hi = 0;
        each([&](uint32_t k, int i) {
            n_hi += k > hi;
            if (k >= lo && k <= hi) {
                const int x = atomicAdd(&sm.near_n, 1);
                if (x < kNear) {
                    sm.near_k32[x] = k;
                    sm.near_idx[x] = i;
                }
            }
        });
        n_hi = __reduce_add_sync(0xffffffffu, n_hi);
        if (lane == 0) sm.sum_hi[warp] = n_hi;
        __syncthreads();
        n_hi = __reduce_add_sync(0xffffffffu, lane < NW ? sm.sum_hi[lane] : 0);
        n_near = sm.near_n;
        take_near = need - n_hi;  // of the keys near the border: 1 .. n_near
        if (n_near <= kNear || shift == 0) break;
        __syncthreads();  // everybody has read the counts
        if (tid < kBins) sm.hist[tid] = 0;
        if (tid == 0) sm.near_n = 0;
        __syncthreads();
    }
    auto score_at = [&](int i) {
        const int id = table[p.first + i];
        return id >= 0 && id < p.b_pages ? ordered(not_nan(score64<BF16>(p, sm.weight64, id, h, lane)))
                                         : ordered(-static_cast<double>(INFINITY));
    };
    bool refine = true;  // whether the order near the border is that of 64-bit scores
    if (n_near <= kNear) {
        int rank = 0;  // of this thread's key among them
        if (tid < n_near) {
            const uint32_t k = sm.near_k32[tid];
            const int i = sm.near_idx[tid];
            for (int y = 0; y < n_near; ++y)
                rank += sm.near_k32[y] > k || (sm.near_k32[y] == k && sm.near_idx[y] < i);
            if (rank == take_near - 1) sm.cut32 = k;
        }
        __syncthreads();
        const float T = from_ordered(sm.cut32);
        const uint32_t lo_T = sure_E ? ordered(T - margin + 0.f) : 1u;
        const uint32_t hi_T = sure_E ? ordered(T + margin + 0.f) : ~0u;
        // fp32 decides unless a key that it leaves out lies within the margin of T
        refine = __syncthreads_or(tid < n_near && rank >= take_near && sm.near_k32[tid] >= lo_T);
        if (refine) {
            for (int x = warp; x < n_near; x += NW) {
                const uint32_t k32 = sm.near_k32[x];
                const unsigned long long k = k32 > hi_T ? ~0ull : k32 < lo_T ? 0ull : score_at(sm.near_idx[x]);
                if (lane == 0) sm.near_key[x] = k;
            }
            __syncthreads();
            if (tid < n_near) {
                const unsigned long long k = sm.near_key[tid];
                const int i = sm.near_idx[tid];
                rank = 0;
                for (int y = 0; y < n_near; ++y)
                    rank += sm.near_key[y] > k || (sm.near_key[y] == k && sm.near_idx[y] < i);
                if (rank == take_near - 1) {
                    sm.cut_key = k;
                    sm.cut_idx = i;
                }
            }
            __syncthreads();
        }
    } else {  // many: equal pages, queries of zeros
        auto near = [&](int i) {
            const uint32_t k = ordered(not_nan(ld_cg(scores + i)) + 0.f);
            return k >= lo && k <= hi;
        };
        // Scores without a finite term, or of weights that are all 0, and infinite ones (the
        // margin then reaches no other) are exact, and those near the border equal: their order
        // is that of the indices.
        refine = !(sure_E && (E == 0.f || !(fabsf(from_ordered(k_max)) < INFINITY) ||
                              !any_weight([](double w) { return w != 0.0; })));
        unsigned long long cut = 0;
        int ties = take_near;  // of those equal to the cut: the first ones
        if (refine) {
            for (int i = warp; i < n_cand; i += NW) {
                if (!near(i)) continue;
                const unsigned long long k = score_at(i);
                if (lane == 0) key64[i] = k;
            }
            __threadfence_block();
            want = take_near;
            for (int shift = 56; shift >= 0; shift -= 8) {  // the key's bytes from the top
                __syncthreads();
                if (tid < kBins) sm.hist[tid] = 0;
                __syncthreads();
                for (int i = tid; i < n_cand; i += NT)
                    if (near(i) && (shift == 56 || key64[i] >> (shift + 8) == cut))
                        atomicAdd(&sm.hist[(key64[i] >> shift) & 255], 1);
                find_bin();
                want -= sm.above;
                cut = cut << 8 | static_cast<unsigned long long>(sm.bin);
            }
            ties = want;
        }
        // The index of the last tie taken: each thread counts those of a run of pages.
        auto tie = [&](int i) { return near(i) && (!refine || key64[i] == cut); };
        const int seg = (n_cand + NT - 1) / NT;
        const int from = tid * seg, to = min(from + seg, n_cand);
        int mine = 0;
        for (int i = from; i < to; ++i) mine += tie(i);
        int upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        __syncthreads();
        if (lane == 31) sm.sum[warp] = upto;
        __syncthreads();
        upto += __reduce_add_sync(0xffffffffu, lane < warp ? sm.sum[lane] : 0);
        if (upto - mine < ties && ties <= upto) {
            int n = upto - mine, i = from;
            while (n += tie(i), n < ties) ++i;
            sm.cut_key = cut;
            sm.cut_idx = i;
        }
        __syncthreads();
    }
    auto take = [&](uint32_t k, int i) {
        if (k > hi) return true;
        if (k < lo) return false;
        if (!refine) return n_near <= kNear ? k >= sm.cut32 : i <= sm.cut_idx;
        unsigned long long k64 = 0;
        if (n_near <= kNear) {
            for (int y = 0; y < n_near; ++y)
                if (sm.near_idx[y] == i) k64 = sm.near_key[y];
        } else {
            k64 = key64[i];
        }
        return k64 > sm.cut_key || (k64 == sm.cut_key && i <= sm.cut_idx);
    };

    // ---- write the taken pages in order: each warp a run of a tile
    static_assert(kTile / NT <= 32, "one word of taken flags a lane");
    int at = p.first;
    for (int t = 0; t < n_tiles; ++t) {
        if (n_tiles > 1) {
            __syncthreads();
            load(t);
        }
        const int n = min(kTile, n_cand - t * kTile);
        const int run = (n + NT - 1) / NT * 32;  // pages a warp, in words of 32
        const int i0 = warp * run;
        uint32_t mine = 0u;  // lane x: the flags of word x
        int n_taken = 0;
#pragma unroll 1
        for (int x = 0; x < run / 32; ++x) {
            const int i = i0 + 32 * x + lane;
            const uint32_t m = __ballot_sync(0xffffffffu, i < n && take(sm.key[i], t * kTile + i));
            if (lane == x) mine = m;
            n_taken += __popc(m);
        }
        if (lane == 0) sm.sum_taken[warp] = n_taken;
        __syncthreads();  // also: every key of the tile has been read
        const int before = __reduce_add_sync(0xffffffffu, lane < warp ? sm.sum_taken[lane] : 0);
        const int total = __reduce_add_sync(0xffffffffu, lane < NW ? sm.sum_taken[lane] : 0);
        int upto = __popc(mine);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        int x = before + upto - __popc(mine);
        while (mine != 0u) {
            sm.key[x++] = static_cast<uint32_t>(t * kTile + i0 + 32 * lane + __ffs(mine) - 1);
            mine &= mine - 1u;
        }
        __syncthreads();
        for (int y = tid; y < total; y += NT) {
            const int j = p.first + static_cast<int>(sm.key[y]);
            ids[at + y] = table[j];
            if (index != nullptr) index[at + y] = j;
        }
        at += total;
    }
}

cudaLaunchConfig_t dependent_launch(int64_t blocks, int threads, cudaStream_t s, cudaLaunchAttribute* attr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.stream = s;
    attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr->val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

// Allow the scoring kernel its shared memory, once per kernel and device.
template <int D, bool BF16, int QB>
cudaError_t allow_score_smem() {
    static std::atomic<unsigned long long> done{0};  // one bit per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && (done.load(std::memory_order_acquire) & (1ull << dev))) return cudaSuccess;
    e = cudaFuncSetAttribute(score_pages_kernel<D, BF16, QB>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             SelShape<D>::SMEM);
    if (e == cudaSuccess && dev < 64) done.fetch_or(1ull << dev, std::memory_order_release);
    return e;
}

template <int D, int QB>
cudaError_t launch_score_q(SelectParams& p, bool bf16, int num_sms, cudaStream_t s) {
    const int64_t rows = static_cast<int64_t>(p.batch) * ((p.q_len + QB - 1) / QB) * p.hk;
    const int64_t cand = std::max(1, p.max_pages - p.first - p.last);
    // Pages per CTA: one wave of CTAs while that leaves each at most 384 KB to stream;
    // more CTAs than that for more pages, as rows differ in length.  (A batch of 64:
    // 96 KB 93 us, 192 KB 76, 384 KB 71, 768 KB 74.)
    const int64_t wave = static_cast<int64_t>(num_sms) * SelShape<D>::CTAS;
    const int64_t per_row = std::max<int64_t>(1, wave / rows);  // CTAs a row in one wave
    int64_t chunk = std::min<int64_t>((cand + per_row - 1) / per_row, (384 << 10) / (4 * D));
    chunk = std::min((chunk + kMinChunk - 1) / kMinChunk * kMinChunk, (cand + kMinChunk - 1) / kMinChunk * kMinChunk);
    // at most 2^31 - 1 CTAs
    while (rows * ((cand + chunk - 1) / chunk) > INT32_MAX && chunk < cand) chunk *= 2;
    p.chunk = static_cast<int>(chunk);
    p.n_chunks = static_cast<int>((cand + chunk - 1) / chunk);
    p.chain = 4 * SelShape<D>::CPL;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = dependent_launch(rows * p.n_chunks, kScoreThreads, s, attr);
    cfg.dynamicSmemBytes = SelShape<D>::SMEM;
    const cudaError_t e = bf16 ? allow_score_smem<D, true, QB>() : allow_score_smem<D, false, QB>();
    if (e != cudaSuccess) return e;
    return bf16 ? cudaLaunchKernelEx(&cfg, score_pages_kernel<D, true, QB>, p)
                : cudaLaunchKernelEx(&cfg, score_pages_kernel<D, false, QB>, p);
}

template <int D>
cudaError_t launch_score(SelectParams& p, bool bf16, int num_sms, cudaStream_t s) {
    if (p.q_len >= 3) return launch_score_q<D, 4>(p, bf16, num_sms, s);
    return p.q_len == 2 ? launch_score_q<D, 2>(p, bf16, num_sms, s) : launch_score_q<D, 1>(p, bf16, num_sms, s);
}

template <bool BF16, int NW>
cudaError_t launch_choose_type(const SelectParams& p, cudaStream_t s) {
    static std::atomic<unsigned long long> done{0};  // shared memory allowed: one bit per device
    constexpr int bytes = static_cast<int>(sizeof(ChooseShared<NW>));
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (bytes > 48 * 1024 && (dev >= 64 || !(done.load(std::memory_order_acquire) & (1ull << dev)))) {
        e = cudaFuncSetAttribute(choose_pages_kernel<BF16, NW>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        if (dev < 64) done.fetch_or(1ull << dev, std::memory_order_release);
    }
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = dependent_launch(static_cast<int64_t>(p.batch) * p.q_len * p.hk, NW * 32, s, attr);
    cfg.dynamicSmemBytes = bytes;
    return cudaLaunchKernelEx(&cfg, choose_pages_kernel<BF16, NW>, p);
}

template <int NW>
cudaError_t launch_choose(const SelectParams& p, bool bf16, cudaStream_t s) {
    return bf16 ? launch_choose_type<true, NW>(p, s) : launch_choose_type<false, NW>(p, s);
}

}  // namespace

int64_t select_abs_stride(int64_t max_pages) { return (max_pages + kMinChunk - 1) / kMinChunk; }

cudaError_t launch_select_pages(SelectParams p, int head_dim, bool bf16, int num_sms, cudaStream_t s) {
    p.head_dim = head_dim;
    cudaError_t e;
    switch (head_dim) {
        case 64: e = launch_score<64>(p, bf16, num_sms, s); break;
        case 128: e = launch_score<128>(p, bf16, num_sms, s); break;
        case 192: e = launch_score<192>(p, bf16, num_sms, s); break;
        case 256: e = launch_score<256>(p, bf16, num_sms, s); break;
        case 512: e = launch_score<512>(p, bf16, num_sms, s); break;
        default: return cudaErrorInvalidValue;
    }
    if (e != cudaSuccess) return e;
    // More threads a row where there are at most as many rows as SMs: 4 rows of 4096 pages
    // take 9.8 us with 1024 threads each, 10.3 with 512, 12.1 with 256; 128 rows of 512 pages
    // 13.8 with 512, 14.5 with 256.  With more rows 256 threads (512 rows of up to 2048 pages:
    // 67 against 72 with 512; 608 rows of 4096: 66 against 70), but 512 while two rows an SM
    // are all there are (304 rows of 4096: 61 against 64) and for pages past 256 threads' tile
    // (304 rows of 8192: 99 against 108).
    const int64_t rows = static_cast<int64_t>(p.batch) * p.q_len * p.hk;
    if (rows > num_sms) {
        const bool wide = p.max_pages > ChooseShared<8>::TILE || (p.max_pages > 2048 && rows <= 2 * num_sms);
        return wide ? launch_choose<16>(p, bf16, s) : launch_choose<8>(p, bf16, s);
    }
    return p.max_pages > 1024 ? launch_choose<32>(p, bf16, s) : launch_choose<16>(p, bf16, s);
}

}  // namespace fdec
