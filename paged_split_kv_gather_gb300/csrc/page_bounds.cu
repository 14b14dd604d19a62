// page_bounds.cu -- elementwise minimum and maximum of the keys of each page.
//
//   bounds[page, h, 0, :] = min over the page's tokens below L of K[page, h, slot, :]
//   bounds[page, h, 1, :] = max   (a NaN key element gives NaN)
//
// for the pages that hold positions [begin, L) of each sequence.  Exact: a minimum
// rounds nothing, and E4M3 values are 16-bit values.  HBM-bound: a page's keys are
// read once (2 D bytes a token), its two rows written.  A page and KV head is one unit:
// one warp, or the four warps of a CTA for long pages and where there are too few units to
// fill the machine (a batch's newest pages); D/8 lanes hold a row, several rows in flight.
// GB300: the pages of 131072 tokens, 4 heads of 128 (138 MB), 23.1 us, 0.88 of the
// measured copy bandwidth; the newest pages of 64 sequences 2.7 us.
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include <cuda_fp8.h>

#include "../../include/fdec.h"
#include "device_utils.cuh"
#include "fdec_internal.h"

namespace fdec {

namespace {

constexpr int kBoundsWarps = 4;

template <bool BF16>
using Pair = std::conditional_t<BF16, __nv_bfloat162, __half2>;

template <typename P2>
__device__ __forceinline__ P2 as_pair(uint32_t w) {
    return *reinterpret_cast<P2*>(&w);
}
template <typename P2>
__device__ __forceinline__ uint32_t as_word(P2 v) {
    return *reinterpret_cast<uint32_t*>(&v);
}

// The keys' arithmetic type: their own 16-bit type, or binary16 for E4M3 codes (every
// E4M3 value is a binary16 value).
template <int D, bool BF16, bool KV8>
struct BoundsShape {
    using P2 = Pair<BF16 && !KV8>;
    static constexpr int ROW_BYTES = D * (KV8 ? 1 : 2);
    static constexpr int CHUNKS = ROW_BYTES / 16;
    static constexpr int LPR = CHUNKS == 24 ? 8 : (CHUNKS > 32 ? 32 : CHUNKS);
    static constexpr int CPL = CHUNKS / LPR;
    static constexpr int RPW = 32 / LPR;
    static constexpr int NP = KV8 ? 8 : 4;   // pairs per chunk
    static constexpr int U = 8 / CPL;        // row groups in flight
};

template <int D, bool BF16, bool KV8, int WPU>
__global__ void __launch_bounds__(kBoundsWarps * 32) page_bounds_kernel(const __grid_constant__ BoundsParams p) {
    using S = BoundsShape<D, BF16, KV8>;
    using P2 = typename S::P2;
    constexpr int NP = S::NP, CPL = S::CPL, LPR = S::LPR, RPW = S::RPW, U = S::U;
    __shared__ uint32_t s_part[WPU > 1 ? kBoundsWarps : 1][2][WPU > 1 ? NP * CPL : 1][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane / LPR, l = lane - sub * LPR;
    const int ww = WPU > 1 ? warp : 0;
    const int64_t unit = WPU > 1 ? blockIdx.x : static_cast<int64_t>(blockIdx.x) * kBoundsWarps + warp;
    const int64_t units = static_cast<int64_t>(p.batch) * p.span * p.hk;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (unit >= units) return;
    const int h = static_cast<int>(unit % p.hk);
    const int64_t bj = unit / p.hk;
    const int j0 = static_cast<int>(bj % p.span);
    const int b = static_cast<int>(bj / p.span);
    int64_t L = p.seq_lens[b];
    int64_t begin = p.begins != nullptr ? p.begins[b] : 0;
    const int64_t room = p.pt_stride << p.page_shift;
    if (L < 0 || L > room || begin < 0) {
        if (lane == 0 && ww == 0 && p.err != nullptr) atomicOr(p.err, FDEC_DEVERR_SEQ_LEN);
        L = L < 0 ? 0 : min(L, room);
        begin = max(begin, static_cast<int64_t>(0));
    }
    const int P = 1 << p.page_shift;
    // span: pages of one sequence that the launch has CTAs for; a longer range is walked
    for (int64_t j = (begin >> p.page_shift) + j0; j * P < L; j += p.span) {
        const int page = p.page_table[static_cast<int64_t>(b) * p.pt_stride + j];
        if (page < 0 || page >= p.k_pages || page >= p.b_pages) {
            if (lane == 0 && ww == 0 && p.err != nullptr) atomicOr(p.err, FDEC_DEVERR_PAGE_ID);
            continue;
        }
        const int n = static_cast<int>(min(static_cast<int64_t>(P), L - j * P));  // >= 1
        const uint8_t* rows = p.k_base + page * p.k_sp + h * p.k_sh;
        P2 lo[CPL][NP], hi[CPL][NP];
        bool first = true;
        for (int r0 = ww * RPW; r0 < n || first; r0 += WPU * RPW * U) {
            uint4 raw[U][CPL];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                // rows past the page's last token repeat it
                const int r = min(r0 + u * WPU * RPW + sub, n - 1);
#pragma unroll
                for (int c = 0; c < CPL; ++c)
                    raw[u][c] = *reinterpret_cast<const uint4*>(rows + r * p.k_st + 16 * (l + LPR * c));
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int c = 0; c < CPL; ++c) {
                    const uint32_t w[4] = {raw[u][c].x, raw[u][c].y, raw[u][c].z, raw[u][c].w};
                    P2 v[NP];
#pragma unroll
                    for (int k = 0; k < NP; ++k) {
                        if constexpr (KV8) {
                            const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(
                                static_cast<__nv_fp8x2_storage_t>(w[k >> 1] >> (16 * (k & 1))), __NV_E4M3);
                            v[k] = *reinterpret_cast<const P2*>(&hr);
                        } else {
                            v[k] = as_pair<P2>(w[k]);
                        }
                        lo[c][k] = first && u == 0 ? v[k] : __hmin2_nan(lo[c][k], v[k]);
                        hi[c][k] = first && u == 0 ? v[k] : __hmax2_nan(hi[c][k], v[k]);
                    }
                }
            first = false;
        }
        // the lanes that hold other rows of the same chunk
#pragma unroll
        for (int o = LPR; o < 32; o <<= 1)
#pragma unroll
            for (int c = 0; c < CPL; ++c)
#pragma unroll
                for (int k = 0; k < NP; ++k) {
                    lo[c][k] = __hmin2_nan(lo[c][k], as_pair<P2>(__shfl_xor_sync(0xffffffffu, as_word(lo[c][k]), o)));
                    hi[c][k] = __hmax2_nan(hi[c][k], as_pair<P2>(__shfl_xor_sync(0xffffffffu, as_word(hi[c][k]), o)));
                }
        if constexpr (WPU > 1) {
            __syncthreads();  // the previous page's values have been read
#pragma unroll
            for (int c = 0; c < CPL; ++c)
#pragma unroll
                for (int k = 0; k < NP; ++k) {
                    s_part[warp][0][c * NP + k][lane] = as_word(lo[c][k]);
                    s_part[warp][1][c * NP + k][lane] = as_word(hi[c][k]);
                }
            __syncthreads();
            if (warp != 0) continue;
#pragma unroll
            for (int w = 1; w < WPU; ++w)
#pragma unroll
                for (int c = 0; c < CPL; ++c)
#pragma unroll
                    for (int k = 0; k < NP; ++k) {
                        lo[c][k] = __hmin2_nan(lo[c][k], as_pair<P2>(s_part[w][0][c * NP + k][lane]));
                        hi[c][k] = __hmax2_nan(hi[c][k], as_pair<P2>(s_part[w][1][c * NP + k][lane]));
                    }
        }
        if (sub == 0) {
            uint8_t* out = p.b_base + page * p.b_sp + h * p.b_sh;
#pragma unroll
            for (int side = 0; side < 2; ++side)
#pragma unroll
                for (int c = 0; c < CPL; ++c) {
                    uint32_t w[NP];
#pragma unroll
                    for (int k = 0; k < NP; ++k) {
                        const P2 v = side == 0 ? lo[c][k] : hi[c][k];
                        if constexpr (KV8 && BF16) {
                            const float2 f = __half22float2(v);
                            w[k] = pack2<true>(f.x, f.y);  // exact
                        } else {
                            w[k] = as_word(v);
                        }
                    }
#pragma unroll
                    for (int k = 0; k < NP; k += 4)
                        *reinterpret_cast<uint4*>(out + side * p.b_st + (l + LPR * c) * NP * 4 + k * 4) =
                            make_uint4(w[k], w[k + 1], w[k + 2], w[k + 3]);
                }
        }
    }
}

template <int D, bool BF16, bool KV8>
cudaError_t launch_bounds(const BoundsParams& p, int num_sms, cudaStream_t s) {
    using S = BoundsShape<D, BF16, KV8>;
    const int64_t units = static_cast<int64_t>(p.batch) * p.span * p.hk;
    // Four warps for one page where its rows are more than one round of a warp's loads and
    // single warps would leave the machine empty, or are eight rounds and more.  Measured
    // (head_dim 128, us, four warps / one): 8 pages of 64 tokens 1.9 / 2.9, 512 of 256
    // 4.4 / 7.6, 2400 of 256 15.9 / 18.6; 2048 of 64 5.0 / 4.3, 8192 of 64 23.9 / 23.1.
    const int rounds = (1 << p.page_shift) / (S::RPW * S::U);
    const bool wide = rounds >= 8 || (rounds >= 2 && units < static_cast<int64_t>(num_sms) * 8);
    const int64_t blocks = wide ? units : (units + kBoundsWarps - 1) / kBoundsWarps;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
    cfg.blockDim = dim3(kBoundsWarps * 32, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return wide ? cudaLaunchKernelEx(&cfg, page_bounds_kernel<D, BF16, KV8, kBoundsWarps>, p)
                : cudaLaunchKernelEx(&cfg, page_bounds_kernel<D, BF16, KV8, 1>, p);
}

template <int D>
cudaError_t launch_bounds_d(const BoundsParams& p, bool bf16, bool kv8, int num_sms, cudaStream_t s) {
    if (kv8) {
        if constexpr (D == 128 || D == 256)
            return bf16 ? launch_bounds<D, true, true>(p, num_sms, s) : launch_bounds<D, false, true>(p, num_sms, s);
        return cudaErrorInvalidValue;
    }
    return bf16 ? launch_bounds<D, true, false>(p, num_sms, s) : launch_bounds<D, false, false>(p, num_sms, s);
}

}  // namespace

cudaError_t launch_page_bounds(const BoundsParams& p, int head_dim, bool bf16, bool kv8, int num_sms, cudaStream_t s) {
    switch (head_dim) {
        case 64: return launch_bounds_d<64>(p, bf16, kv8, num_sms, s);
        case 128: return launch_bounds_d<128>(p, bf16, kv8, num_sms, s);
        case 192: return launch_bounds_d<192>(p, bf16, kv8, num_sms, s);
        case 256: return launch_bounds_d<256>(p, bf16, kv8, num_sms, s);
        case 512: return launch_bounds_d<512>(p, bf16, kv8, num_sms, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace fdec
