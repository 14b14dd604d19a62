// norm_rope.cu -- the rows of new tokens on their way into attention: RMS norm of
// every query and key head, rotation by the token's position, and the paged write of
// the keys and values, in one pass.
//
//   y = x * rsqrt(mean(x^2) + eps) * w          (q and k heads; w per element, or 1)
//   (a, b) -> (a cos - b sin, b cos + a sin)     pairs of the first rot elements:
//                                                (e, e + rot/2), or (2e, 2e + 1)
//   q -> q_out;  k, v -> page table[b][t / P], slot t % P (16-bit, or E4M3 of x / scale)
//
// The sum of squares, the norm and the rotation are fp32 and the result is rounded
// once, as it is stored.  HBM-bound: a token's rows are read once and written once.
// A lane holds two 16-byte chunks of a row, those whose elements rotate together (c and
// c + rot/16; chunks past rot pair up among themselves), so nothing but the sum of
// squares crosses lanes, and weight x cosine, weight x sine are computed once a token
// and kept for its rows: a row then costs two packed products and a scaling per
// element pair.  (The first form, one chunk a lane with the partner's chunk, weight and
// angle read again for every row, was bound by instructions.)  GB300, 32768 tokens of
// 32/8 heads of 128 (822 MB): 141 us, 5.8 TB/s, 0.86 of the measured copy bandwidth; the
// first form 269 us.  One token: 2.8 us a call in a stream, which is launch and three
// dependent reads (position, page id, angle).
#include <algorithm>
#include <atomic>
#include <cstdint>
#include <type_traits>

#include <cuda_fp8.h>

#include "../../include/fdec.h"
#include "device_utils.cuh"
#include "fdec_internal.h"

namespace fdec {

namespace {

constexpr int kRowsThreads = 256;
constexpr int kRowsCtas = 2;  // an SM: 128 registers a thread

template <int D>
struct RowLanes {
    static constexpr int PAIRS = D / 16;                                          // chunk pairs of a row
    static constexpr int LPR = PAIRS <= 4 ? 4 : PAIRS <= 8 ? 8 : PAIRS <= 16 ? 16 : 32;  // lanes per row
    static constexpr int RPW = 32 / LPR;                                          // rows per warp
};

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& w, float2 (&x)[4]) {
    x[0] = unpack2<BF16>(w.x);
    x[1] = unpack2<BF16>(w.y);
    x[2] = unpack2<BF16>(w.z);
    x[3] = unpack2<BF16>(w.w);
}

// |a| at most 65536, with a's sign; NaN stays NaN.
__device__ __forceinline__ float at_most_65536(float a) {
    float v;
    asm("min.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(v) : "f"(a), "f"(65536.f));
    return v;
}

// Eight values divided by the scale and rounded to E4M3 codes (saturating at 448); inv is
// the rounded 1 / scale.  The quotient is the rounded one: the values are 16-bit ones or
// products of them, so quotients half way between two codes do occur, and x inv, an ulp
// off, puts those on the wrong side (scale 7/256: 60 of the finite bf16 values).  It is
// q + (x - q scale) inv, q = x inv, with fused multiply-adds (P. Markstein, Computation of
// elementary functions on the IBM RISC System/6000 processor, 1990): exact residual, hence
// rounded once, for scales in [2^-60, 2^60].  (32768 tokens of 32/8 heads of 128 137.8 us,
// with the product alone 135.3, with __fdiv_rn 160.7.)
__device__ __forceinline__ uint2 codes8(const float2 (&x)[4], float scale, float inv) {
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 q = __fmul2_rn(x[i], make_float2(inv, inv));
        q = make_float2(at_most_65536(q.x), at_most_65536(q.y));  // (an infinite q would have no residual)
        const float2 r = __ffma2_rn(q, make_float2(-scale, -scale), x[i]);
        c[i] = __nv_cvt_float2_to_fp8x2(__ffma2_rn(r, make_float2(inv, inv), q), __NV_SATFINITE, __NV_E4M3);
    }
    return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

// One lane's coefficients for the q rows or the k rows of a token: output chunk 0 is
// x0 a0 + m0 b0 and chunk 1 is x1 a1 + m1 b1, with m the other element of each pair.
struct Coef {
    float2 a0[4], b0[4], a1[4], b1[4];
};

template <bool BF16, bool INTER>
__device__ __forceinline__ void make_coef(Coef& f, const uint16_t* weight, const float* cs, int half, int c0, int c1,
                                          bool rotated) {
    float2 w0[4], w1[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) w0[k] = w1[k] = make_float2(1.f, 1.f);
    if (weight != nullptr) {
        unpack8<BF16>(*reinterpret_cast<const uint4*>(weight + 8 * c0), w0);
        unpack8<BF16>(*reinterpret_cast<const uint4*>(weight + 8 * c1), w1);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        f.a0[k] = w0[k], f.a1[k] = w1[k];
        f.b0[k] = f.b1[k] = make_float2(0.f, 0.f);
    }
    if (!rotated) return;
    if constexpr (INTER) {  // pairs within a chunk: four angles each
        const float4 p0 = *reinterpret_cast<const float4*>(cs + 4 * c0), q0 = *reinterpret_cast<const float4*>(cs + half + 4 * c0);
        const float4 p1 = *reinterpret_cast<const float4*>(cs + 4 * c1), q1 = *reinterpret_cast<const float4*>(cs + half + 4 * c1);
        const float cc0[4] = {p0.x, p0.y, p0.z, p0.w}, ss0[4] = {q0.x, q0.y, q0.z, q0.w};
        const float cc1[4] = {p1.x, p1.y, p1.z, p1.w}, ss1[4] = {q1.x, q1.y, q1.z, q1.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            f.a0[k] = make_float2(w0[k].x * cc0[k], w0[k].y * cc0[k]);
            f.b0[k] = make_float2(-w0[k].y * ss0[k], w0[k].x * ss0[k]);
            f.a1[k] = make_float2(w1[k].x * cc1[k], w1[k].y * cc1[k]);
            f.b1[k] = make_float2(-w1[k].y * ss1[k], w1[k].x * ss1[k]);
        }
    } else {  // element e of chunk 0 with element e of chunk 1: eight angles
#pragma unroll
        for (int k2 = 0; k2 < 2; ++k2) {
            const float4 p = *reinterpret_cast<const float4*>(cs + 8 * c0 + 4 * k2);
            const float4 q = *reinterpret_cast<const float4*>(cs + half + 8 * c0 + 4 * k2);
            const float2 cc[2] = {make_float2(p.x, p.y), make_float2(p.z, p.w)};
            const float2 ss[2] = {make_float2(q.x, q.y), make_float2(q.z, q.w)};
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int k = 2 * k2 + y;
                f.a0[k] = make_float2(w0[k].x * cc[y].x, w0[k].y * cc[y].y);
                f.b0[k] = make_float2(-w1[k].x * ss[y].x, -w1[k].y * ss[y].y);
                f.a1[k] = make_float2(w1[k].x * cc[y].x, w1[k].y * cc[y].y);
                f.b1[k] = make_float2(w0[k].x * ss[y].x, w0[k].y * ss[y].y);
            }
        }
    }
}

// U: row groups a warp loads at once, the next U while it computes these.  PRE: its first q,
// k and v rows are requested together.
template <int D, bool BF16, bool KV8, bool INTER, int U, bool PRE>
__global__ void __launch_bounds__(kRowsThreads, kRowsCtas) norm_rope_kernel(const __grid_constant__ NormRopeParams p, int wpt) {
    using R = RowLanes<D>;
    constexpr int LPR = R::LPR, RPW = R::RPW;
    const int lane = threadIdx.x & 31;
    const int sub = lane / LPR;
    // head_dim 192 needs 12 of 16 lanes: the others go along with the last one's chunks, but
    // add nothing to the sum and store nothing.
    const bool on = lane - sub * LPR < R::PAIRS;
    const int l = on ? lane - sub * LPR : R::PAIRS - 1;
    const int64_t warp0 = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    const int64_t nwarps = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5;
    const int64_t n_work = static_cast<int64_t>(p.n_tokens) * wpt;
    const int half = p.rot / 2;
    const int page_mask = (1 << p.page_shift) - 1;
    const int n_rot = p.rot / 16;  // chunk pairs that rotate
    const bool rotated = l < n_rot;
    const int c0 = rotated ? l : n_rot + l;
    const int c1 = rotated ? l + n_rot : c0 + (D / 16 - n_rot);
    // Row groups of the q, k and v rows; a warp takes every wpt-th over all three.
    const int groups_q = (p.hq + RPW - 1) / RPW, groups_kv = (p.hk + RPW - 1) / RPW;

    // A programmatic dependent of the kernel before it on the stream (the projection):
    // nothing is read or written before that kernel has completed.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    int b_next = 0, t_next = 0, rt_next = 0;
    auto fetch = [&](int64_t w) {
        if (w >= n_work) return;
        const int64_t i = w / wpt;
        b_next = p.batch_indices[i];
        t_next = p.positions[i];
        rt_next = p.rope_positions != nullptr ? p.rope_positions[i] : t_next;
    };
    fetch(warp0);
    for (int64_t w = warp0; w < n_work; w += nwarps) {
        const int64_t i = w / wpt;
        const int part = static_cast<int>(w - i * wpt);
        const int b = b_next, t = t_next, rt = rt_next;
        fetch(w + nwarps);
        const int pi = t >> p.page_shift;
        if (t < 0 || pi >= p.pt_stride || b < 0 || b >= p.batch || (p.rot > 0 && (rt < 0 || rt >= p.cos_rows))) {
            if (lane == 0 && part == 0 && p.err != nullptr) atomicOr(p.err, FDEC_DEVERR_SEQ_LEN);
            continue;
        }
        const int page = p.page_table[static_cast<int64_t>(b) * p.pt_stride + pi];
        // Not waited for here: the query rows' loads do not depend on it, only what is stored.
        const bool page_ok = page >= 0 && page < p.k_pages && page < p.v_pages;
        const int64_t slot = t & page_mask;
        const float* cs = p.cos_sin + static_cast<int64_t>(rt) * p.rot;
        // this warp's first group of the kind whose groups start at `from`
        auto first_group = [&](int from) {
            const int back = part - from;
            return back >= 0 ? back : back + (-back + wpt - 1) / wpt * wpt;
        };
        auto load_rows = [&](const uint8_t* src, int64_t src_h, int heads, int at, uint4 (&a)[U], uint4 (&c)[U]) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = (at + u * wpt) * RPW + sub;
                a[u] = c[u] = make_uint4(0u, 0u, 0u, 0u);
                if (h < heads) {
                    a[u] = *reinterpret_cast<const uint4*>(src + h * src_h + 16 * c0);
                    c[u] = *reinterpret_cast<const uint4*>(src + h * src_h + 16 * c1);
                }
            }
        };
        // The q rows or the k rows: norm and rotation of rows h < heads at src + h * src_h, the
        // first of them in r0, r1 with PRE.
        auto normed = [&](const uint8_t* src, int64_t src_h, uint8_t* dst, int64_t dst_h, int heads, int from, int groups,
                          const uint16_t* weight, auto codes, uint4 (&r0)[U], uint4 (&r1)[U]) {
            constexpr bool CODES = decltype(codes)::value;
            int g = first_group(from);
            if (g >= groups) return;
            uint4 n0[U], n1[U];
            auto load = [&](int at, uint4 (&a)[U], uint4 (&c)[U]) { load_rows(src, src_h, heads, at, a, c); };
            if constexpr (!PRE) load(g, r0, r1);
            Coef f;
            make_coef<BF16, INTER>(f, weight, cs, half, c0, c1, rotated);
            for (; g < groups; g += U * wpt) {
                // (a lane stores only chunks that it has loaded itself, so q_out may be q)
                load(g + U * wpt, n0, n1);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float2 x0[4], x1[4];
                    unpack8<BF16>(r0[u], x0);
                    unpack8<BF16>(r1[u], x1);
                    float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
                    for (int k = 0; k < 4; ++k) s2 = __ffma2_rn(x1[k], x1[k], __ffma2_rn(x0[k], x0[k], s2));
                    float sum = on ? s2.x + s2.y : 0.f;
#pragma unroll
                    for (int o = LPR / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    const float rs = rsqrtf(sum * (1.f / D) + p.eps);
                    const float2 rs2 = make_float2(rs, rs);
                    float2 y0[4], y1[4];
                    if (rotated) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float2 m0 = INTER ? make_float2(x0[k].y, x0[k].x) : x1[k];
                            const float2 m1 = INTER ? make_float2(x1[k].y, x1[k].x) : x0[k];
                            y0[k] = __fmul2_rn(__ffma2_rn(x0[k], f.a0[k], __fmul2_rn(m0, f.b0[k])), rs2);
                            y1[k] = __fmul2_rn(__ffma2_rn(x1[k], f.a1[k], __fmul2_rn(m1, f.b1[k])), rs2);
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            y0[k] = __fmul2_rn(__fmul2_rn(x0[k], f.a0[k]), rs2);
                            y1[k] = __fmul2_rn(__fmul2_rn(x1[k], f.a1[k]), rs2);
                        }
                    }
                    const int h = (g + u * wpt) * RPW + sub;
                    if (!on || h >= heads || !page_ok) continue;
                    uint8_t* to = dst + h * dst_h;
                    if constexpr (CODES) {
                        *reinterpret_cast<uint2*>(to + 8 * c0) = codes8(y0, p.k_scale, p.k_inv);
                        *reinterpret_cast<uint2*>(to + 8 * c1) = codes8(y1, p.k_scale, p.k_inv);
                    } else {
                        *reinterpret_cast<uint4*>(to + 16 * c0) =
                            make_uint4(pack2<BF16>(y0[0].x, y0[0].y), pack2<BF16>(y0[1].x, y0[1].y),
                                       pack2<BF16>(y0[2].x, y0[2].y), pack2<BF16>(y0[3].x, y0[3].y));
                        *reinterpret_cast<uint4*>(to + 16 * c1) =
                            make_uint4(pack2<BF16>(y1[0].x, y1[0].y), pack2<BF16>(y1[1].x, y1[1].y),
                                       pack2<BF16>(y1[2].x, y1[2].y), pack2<BF16>(y1[3].x, y1[3].y));
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) r0[u] = n0[u], r1[u] = n1[u];
            }
        };
        const int gv0 = first_group(groups_q + groups_kv);
        uint4 q0[U], q1[U], k0[U], k1[U], v0[U], v1[U];
        if constexpr (PRE) {
            load_rows(p.q + i * p.q_st, p.q_sh, p.hq, first_group(0), q0, q1);
            load_rows(p.k_new + i * p.k_new_st, p.k_new_sh, p.hk, first_group(groups_q), k0, k1);
            load_rows(p.v_new + i * p.v_new_st, p.v_new_sh, p.hk, gv0, v0, v1);
        }
        normed(p.q + i * p.q_st, p.q_sh, p.q_out + i * p.q_out_st, p.q_out_sh, p.hq, 0, groups_q, p.q_weight,
               std::false_type{}, q0, q1);
        normed(p.k_new + i * p.k_new_st, p.k_new_sh, p.k_base + page * p.k_sp + slot * p.k_st, p.k_sh, p.hk, groups_q,
               groups_kv, p.k_weight, std::bool_constant<KV8>{}, k0, k1);
        if (!page_ok) {
            if (lane == 0 && part == 0 && p.err != nullptr) atomicOr(p.err, FDEC_DEVERR_PAGE_ID);
            continue;
        }
        // The v rows: as they are, or scaled and rounded to codes.
        const uint8_t* src = p.v_new + i * p.v_new_st;
        uint8_t* dst = p.v_base + page * p.v_sp + slot * p.v_st;
        for (int g = gv0; g < groups_kv; g += wpt) {
            const int h = g * RPW + sub;
            if (!on || h >= p.hk) continue;
            uint4 r0, r1;
            if (PRE && g == gv0) {
                r0 = v0[0], r1 = v1[0];
            } else {
                r0 = *reinterpret_cast<const uint4*>(src + h * p.v_new_sh + 16 * c0);
                r1 = *reinterpret_cast<const uint4*>(src + h * p.v_new_sh + 16 * c1);
            }
            uint8_t* to = dst + h * p.v_sh;
            if constexpr (KV8) {
                float2 x0[4], x1[4];
                unpack8<BF16>(r0, x0);
                unpack8<BF16>(r1, x1);
                *reinterpret_cast<uint2*>(to + 8 * c0) = codes8(x0, p.v_scale, p.v_inv);
                *reinterpret_cast<uint2*>(to + 8 * c1) = codes8(x1, p.v_scale, p.v_inv);
            } else {
                *reinterpret_cast<uint4*>(to + 16 * c0) = r0;
                *reinterpret_cast<uint4*>(to + 16 * c1) = r1;
            }
        }
    }
}

template <int D, bool BF16, bool KV8>
cudaError_t launch_rows(const NormRopeParams& p, bool pairs, int num_sms, cudaStream_t s) {
    using R = RowLanes<D>;
    const int groups = (p.hq + R::RPW - 1) / R::RPW + 2 * ((p.hk + R::RPW - 1) / R::RPW);
    const int64_t slots = static_cast<int64_t>(num_sms) * kRowsCtas * (kRowsThreads / 32);
    // Warps per token (a warp takes every wpt-th group of rows, and computes the token's
    // coefficients again): all the groups' own while they fit the machine at once, else the
    // number with the least (rounds of the machine) x (a token's set-up, about four groups,
    // + a warp's groups).  One warp each, 2036 tokens take 12.6 us, with two 14.5; but 2457
    // tokens of 24 groups, a little over one round, 38.7 us with one.
    int wpt = groups;
    if (static_cast<int64_t>(p.n_tokens) * groups > slots) {
        int64_t best = INT64_MAX;
        for (int w = 1; w <= std::min(groups, 8); ++w) {
            const int64_t rounds = (static_cast<int64_t>(p.n_tokens) * w + slots - 1) / slots;
            const int64_t cost = rounds * (4 + (groups + w - 1) / w);
            if (cost < best) {
                best = cost;
                wpt = w;
            }
        }
    }
    // A warp has two groups at most: the form without loads ahead is shorter code, which a
    // call of a few tokens mostly waits to fetch (64 tokens: 3.2 against 3.6 us).  Up to four:
    // its q, k and v rows together, as a token's latency decides (32768 tokens of 4/1 heads of
    // 128 51 against 62 us; in every call, one token 3.1 against 2.8).
    const int per_warp = (groups + wpt - 1) / wpt;
    const int64_t warps = static_cast<int64_t>(p.n_tokens) * wpt;
    const int64_t blocks =
        std::min<int64_t>((warps * 32 + kRowsThreads - 1) / kRowsThreads, static_cast<int64_t>(num_sms) * kRowsCtas);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
    cfg.blockDim = dim3(kRowsThreads, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto launch = [&](auto u, auto pre) {
        constexpr int U = decltype(u)::value;
        constexpr bool PRE = decltype(pre)::value;
        return pairs ? cudaLaunchKernelEx(&cfg, norm_rope_kernel<D, BF16, KV8, true, U, PRE>, p, wpt)
                     : cudaLaunchKernelEx(&cfg, norm_rope_kernel<D, BF16, KV8, false, U, PRE>, p, wpt);
    };
    using One = std::integral_constant<int, 1>;
    if (per_warp <= 2) return launch(One{}, std::false_type{});
    if (per_warp <= 4) return launch(One{}, std::true_type{});
    return launch(std::integral_constant<int, 2>{}, std::false_type{});
}

template <int D>
cudaError_t launch_rows_d(const NormRopeParams& p, bool bf16, bool kv8, bool pairs, int num_sms, cudaStream_t s) {
    if (kv8) {
        if constexpr (D == 128 || D == 256)
            return bf16 ? launch_rows<D, true, true>(p, pairs, num_sms, s)
                        : launch_rows<D, false, true>(p, pairs, num_sms, s);
        return cudaErrorInvalidValue;
    }
    return bf16 ? launch_rows<D, true, false>(p, pairs, num_sms, s)
                : launch_rows<D, false, false>(p, pairs, num_sms, s);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams& p, int head_dim, bool bf16, bool kv8, bool pairs, int num_sms,
                             cudaStream_t s) {
    if (p.n_tokens == 0) return cudaSuccess;
    switch (head_dim) {
        case 64: return launch_rows_d<64>(p, bf16, kv8, pairs, num_sms, s);
        case 128: return launch_rows_d<128>(p, bf16, kv8, pairs, num_sms, s);
        case 192: return launch_rows_d<192>(p, bf16, kv8, pairs, num_sms, s);
        case 256: return launch_rows_d<256>(p, bf16, kv8, pairs, num_sms, s);
        case 512: return launch_rows_d<512>(p, bf16, kv8, pairs, num_sms, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace fdec
