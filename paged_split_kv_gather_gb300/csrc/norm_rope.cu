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
// A row of D elements is held by D/8 lanes (16 bytes each; 3 or 2 chunks per lane at
// head_dim 192 and 512), so a load instruction of a warp covers up to four whole rows
// and the sum of squares is a shuffle among the lanes of a row.
#include <algorithm>
#include <atomic>
#include <cstdint>

#include <cuda_fp8.h>

#include "../../include/fdec.h"
#include "device_utils.cuh"
#include "fdec_internal.h"

namespace fdec {

namespace {

constexpr int kRowsThreads = 256;

template <int D>
struct RowLanes {
    static constexpr int CHUNKS = D / 8;
    static constexpr int LPR = D == 192 ? 8 : (CHUNKS > 32 ? 32 : CHUNKS);  // lanes per row
    static constexpr int CPL = CHUNKS / LPR;                                // chunks per lane
    static constexpr int RPW = 32 / LPR;                                    // rows per warp
};

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2<BF16>(v[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

// Eight values divided by the scale and rounded to E4M3 codes (saturating at 448).
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float scale) {
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const __nv_fp8x2_storage_t c =
            __nv_cvt_float2_to_fp8x2(make_float2(x[i] / scale, x[i + 1] / scale), __NV_SATFINITE, __NV_E4M3);
        w[i >> 2] |= static_cast<uint32_t>(c) << (8 * (i & 3));
    }
    return make_uint2(w[0], w[1]);
}

template <int D, bool BF16, bool KV8, bool PAIRS>
__global__ void __launch_bounds__(kRowsThreads) norm_rope_kernel(const __grid_constant__ NormRopeParams p, int wpt) {
    using R = RowLanes<D>;
    constexpr int CPL = R::CPL, LPR = R::LPR, RPW = R::RPW;
    const int lane = threadIdx.x & 31;
    const int sub = lane / LPR, l = lane - sub * LPR;
    const int64_t warp0 = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    const int64_t nwarps = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5;
    const int rows = p.hq + 2 * p.hk;
    const int groups = (rows + RPW - 1) / RPW;
    const int half = p.rot / 2;
    const int page_mask = (1 << p.page_shift) - 1;

    // A programmatic dependent of the kernel before it on the stream (the projection):
    // nothing is read or written before that kernel has completed.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    for (int64_t w = warp0; w < static_cast<int64_t>(p.n_tokens) * wpt; w += nwarps) {
        const int64_t i = w / wpt;
        const int part = static_cast<int>(w - i * wpt);
        const int b = p.batch_indices[i];
        const int t = p.positions[i];
        const int rt = p.rope_positions != nullptr ? p.rope_positions[i] : t;
        const int pi = t >> p.page_shift;
        if (t < 0 || pi >= p.pt_stride || b < 0 || b >= p.batch || (p.rot > 0 && (rt < 0 || rt >= p.cos_rows))) {
            if (lane == 0 && part == 0 && p.err != nullptr) atomicOr(p.err, FDEC_DEVERR_SEQ_LEN);
            continue;
        }
        const int page = p.page_table[static_cast<int64_t>(b) * p.pt_stride + pi];
        if (page < 0 || page >= p.k_pages || page >= p.v_pages) {
            if (lane == 0 && part == 0 && p.err != nullptr) atomicOr(p.err, FDEC_DEVERR_PAGE_ID);
            continue;
        }
        const int64_t slot = t & page_mask;
        const float* cs = p.cos_sin + static_cast<int64_t>(rt) * p.rot;
        for (int g = part; g < groups; g += wpt) {
            const int r = g * RPW + sub;
            const bool live = r < rows;
            const int kind = r < p.hq ? 0 : (r < p.hq + p.hk ? 1 : 2);  // q, k or v row
            const int h = kind == 0 ? r : (kind == 1 ? r - p.hq : r - p.hq - p.hk);
            const uint8_t* src = kind == 0 ? p.q + i * p.q_st + h * p.q_sh
                                           : (kind == 1 ? p.k_new + i * p.k_new_st + h * p.k_new_sh
                                                        : p.v_new + i * p.v_new_st + h * p.v_new_sh);
            const uint16_t* weight = kind == 0 ? p.q_weight : p.k_weight;
            uint4 raw[CPL], mate[CPL];
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < CPL; ++j) {
                const int e0 = 8 * (l + LPR * j);
                raw[j] = mate[j] = make_uint4(0u, 0u, 0u, 0u);
                if (live) {
                    raw[j] = *reinterpret_cast<const uint4*>(src + 2 * e0);
                    // the other half of this chunk's pairs (rot / 2 is a multiple of 8)
                    if (!PAIRS && kind < 2 && e0 < p.rot)
                        mate[j] = *reinterpret_cast<const uint4*>(src + 2 * (e0 < half ? e0 + half : e0 - half));
                }
            }
#pragma unroll
            for (int j = 0; j < CPL; ++j) {
                float x[8];
                unpack8<BF16>(raw[j], x);
#pragma unroll
                for (int e = 0; e < 8; ++e) sum = fmaf(x[e], x[e], sum);
            }
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            const float rs = rsqrtf(sum * (1.f / D) + p.eps);
            __syncwarp();  // every lane has read its row (q_out may be q)
            if (!live) continue;
            uint8_t* dst = kind == 0 ? p.q_out + i * p.q_out_st + h * p.q_out_sh
                                     : (kind == 1 ? p.k_base + page * p.k_sp + h * p.k_sh + slot * p.k_st
                                                  : p.v_base + page * p.v_sp + h * p.v_sh + slot * p.v_st);
#pragma unroll
            for (int j = 0; j < CPL; ++j) {
                const int e0 = 8 * (l + LPR * j);
                if (kind == 2) {
                    if constexpr (KV8) {
                        float x[8];
                        unpack8<BF16>(raw[j], x);
                        *reinterpret_cast<uint2*>(dst + e0) = codes8(x, p.v_scale);
                    } else {
                        *reinterpret_cast<uint4*>(dst + 2 * e0) = raw[j];
                    }
                    continue;
                }
                float x[8], wt[8];
                unpack8<BF16>(raw[j], x);
#pragma unroll
                for (int e = 0; e < 8; ++e) wt[e] = 1.f;
                if (weight != nullptr) unpack8<BF16>(__ldg(reinterpret_cast<const uint4*>(weight + e0)), wt);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] *= rs * wt[e];
                if (e0 < p.rot) {
                    if constexpr (PAIRS) {
                        const float4 c = *reinterpret_cast<const float4*>(cs + e0 / 2);
                        const float4 s = *reinterpret_cast<const float4*>(cs + half + e0 / 2);
                        const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float a = x[2 * e], bb = x[2 * e + 1];
                            x[2 * e] = a * cc[e] - bb * ss[e];
                            x[2 * e + 1] = bb * cc[e] + a * ss[e];
                        }
                    } else {
                        const int f0 = e0 < half ? e0 : e0 - half;  // index of the pairs
                        const float sign = e0 < half ? -1.f : 1.f;
                        float m[8];
                        unpack8<BF16>(mate[j], m);
#pragma unroll
                        for (int e = 0; e < 8; ++e) wt[e] = 1.f;
                        if (weight != nullptr)
                            unpack8<BF16>(__ldg(reinterpret_cast<const uint4*>(weight + (e0 < half ? e0 + half : f0))), wt);
#pragma unroll
                        for (int q4 = 0; q4 < 2; ++q4) {
                            const float4 c = *reinterpret_cast<const float4*>(cs + f0 + 4 * q4);
                            const float4 s = *reinterpret_cast<const float4*>(cs + half + f0 + 4 * q4);
                            const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int k = 4 * q4 + e;
                                x[k] = x[k] * cc[e] + sign * (m[k] * (rs * wt[k])) * ss[e];
                            }
                        }
                    }
                }
                if (KV8 && kind == 1) {
                    *reinterpret_cast<uint2*>(dst + e0) = codes8(x, p.k_scale);
                } else {
                    *reinterpret_cast<uint4*>(dst + 2 * e0) =
                        make_uint4(pack2<BF16>(x[0], x[1]), pack2<BF16>(x[2], x[3]), pack2<BF16>(x[4], x[5]),
                                   pack2<BF16>(x[6], x[7]));
                }
            }
        }
    }
}

template <int D, bool BF16, bool KV8>
cudaError_t launch_rows(const NormRopeParams& p, bool pairs, int num_sms, cudaStream_t s) {
    using R = RowLanes<D>;
    const int groups = (p.hq + 2 * p.hk + R::RPW - 1) / R::RPW;
    const int64_t full_warps = static_cast<int64_t>(num_sms) * 8 * (kRowsThreads / 32);
    // Warps per token: one while the tokens alone fill the machine, else enough that
    // they do (a warp then takes every wpt-th group of rows).
    int wpt = 1;
    while (wpt < groups && static_cast<int64_t>(p.n_tokens) * wpt < full_warps) wpt *= 2;
    wpt = std::min(wpt, groups);
    const int64_t warps = static_cast<int64_t>(p.n_tokens) * wpt;
    const int64_t blocks =
        std::min<int64_t>((warps * 32 + kRowsThreads - 1) / kRowsThreads, static_cast<int64_t>(num_sms) * 8);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
    cfg.blockDim = dim3(kRowsThreads, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return pairs ? cudaLaunchKernelEx(&cfg, norm_rope_kernel<D, BF16, KV8, true>, p, wpt)
                 : cudaLaunchKernelEx(&cfg, norm_rope_kernel<D, BF16, KV8, false>, p, wpt);
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
