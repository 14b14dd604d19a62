// tree_attention.cu -- attention of drafted trees, joined with the prefix's state.
//
//   z_j = scale q.K_j over a node and its ancestors, M = max(lse_p, max z),
//   w = exp(lse_p - M), l = w + sum exp(z_j - M),  out = (w o_p + sum exp(z_j - M) V_j) / l
//
// A CTA takes one sequence and KV head and some of its query rows (row = node x group +
// head).  The tree's keys and values, at most 64 rows, are staged once in shared memory;
// a warp then takes 16 query rows at a time with mma.sync.m16n8k16: S of 16 x 64 in
// registers, the ancestors a 64-bit word a node, one maximum and sum (every key is there,
// so nothing is rescaled), P V in blocks of 64 columns.  The prefix's state enters as one
// more key, whose value is o_p.
//
// Bytes: 2 D of q, 4 D of o_p, 4 D or 2 D of the result for a query row, against 4 D x 64
// operations or less, so the call is bound by HBM; mma.sync keeps S and P in registers
// and costs less than the bytes, where a tcgen05 tile of 128 rows would be mostly empty
// for trees of a few nodes.
//
// The probabilities of a bf16 cache enter P V as three bf16 values (24 bits) and those of
// an f16 cache as two f16 values (22 bits, scaled by 2^15 so that the small ones stay
// normal): the result is as good as fp32 sums.  With one value less of each it would be
// off by 2^-17 (bf16), with a single one by 2^-9.
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

// Pitches of the staged rows in bytes.  K is read 16 bytes a lane, four lanes a row: rows
// 64 bytes apart modulo 128 keep the eight lanes of a phase on different banks.  V is read
// by ldmatrix: rows 16 bytes apart modulo 128.
template <int D>
struct TreeShape {
    static constexpr int PK = 2 * D + 64, PV = 2 * D + 16;
    static size_t smem(int nodes) { return static_cast<size_t>((nodes + 15) / 16 * 16) * (PK + PV); }
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

// Whether one of the two values of a word is infinite or NaN.
template <bool BF16>
__device__ __forceinline__ bool not_finite(uint32_t w) {
    constexpr uint32_t m = BF16 ? 0x7f80u : 0x7c00u;
    return (w & m) == m || ((w >> 16) & m) == m;
}

// x, y as a sum of TERMS 16-bit values each, the largest first.
template <bool BF16, int TERMS>
__device__ __forceinline__ void split_terms(float x, float y, uint32_t (&out)[TERMS]) {
#pragma unroll
    for (int i = 0; i < TERMS; ++i) {
        out[i] = pack2<BF16>(x, y);
        const float2 r = unpack2<BF16>(out[i]);
        x -= r.x;
        y -= r.y;
    }
}

template <int D, bool BF16, bool KV8>
__global__ void __launch_bounds__(kTreeThreads, 3) tree_attention_kernel(const TreeParams p) {
    using S = TreeShape<D>;
    constexpr int TERMS = BF16 ? 3 : 2;
    constexpr float kPScale = BF16 ? 1.f : 32768.f;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ uint64_t s_anc[kMaxNodes];
    __shared__ int64_t s_k[kMaxNodes], s_v[kMaxNodes];  // byte offsets of the nodes' rows, or -1
    __shared__ unsigned s_valid[2];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int N = p.nodes, g = p.group;
    const int tiles_max = (N * g + 15) / 16;
    const int blocks = (tiles_max + kTreeWarps * p.tiles_per_warp - 1) / (kTreeWarps * p.tiles_per_warp);
    const int blk = blockIdx.x % blocks;
    const int bh = blockIdx.x / blocks;
    const int kvh = bh % p.hk, b = bh / p.hk;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    const bool reports = blk == 0 && kvh == 0 && p.err != nullptr;  // one CTA a sequence
    int n = p.node_counts != nullptr ? p.node_counts[b] : N;
    if (n < 0 || n > N) {
        if (reports && tid == 0) atomicOr(p.err, FDEC_DEVERR_SEQ_LEN);
        n = min(max(n, 0), N);
    }
    const int R = n * g;
    if (blk * kTreeWarps * p.tiles_per_warp * 16 >= R) return;

    // ancestors: bits of a node's path, by pointer doubling (a path has at most 63 steps)
    if (warp == 0) {
        uint64_t anc[2];
        int up[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = lane + 32 * h;
            int par = i - 1;
            if (p.parents != nullptr) par = i < n ? p.parents[static_cast<int64_t>(b) * N + i] : -1;
            if (par < -1 || par >= i) {
                if (reports) atomicOr(p.err, FDEC_DEVERR_TREE);
                par = -1;
            }
            up[h] = par;
            anc[h] = uint64_t{1} << i;
        }
#pragma unroll
        for (int step = 0; step < 6; ++step) {
            uint64_t a[2];
            int u[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int from = up[h] & 31;
                const uint64_t a0 = __shfl_sync(0xffffffffu, anc[0], from), a1 = __shfl_sync(0xffffffffu, anc[1], from);
                const int u0 = __shfl_sync(0xffffffffu, up[0], from), u1 = __shfl_sync(0xffffffffu, up[1], from);
                a[h] = up[h] < 0 ? 0 : up[h] < 32 ? a0 : a1;
                u[h] = up[h] < 0 ? -1 : up[h] < 32 ? u0 : u1;
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                anc[h] |= a[h];
                up[h] = u[h];
            }
        }
        s_anc[lane] = anc[0];
        s_anc[lane + 32] = anc[1];
    } else if (warp <= 2) {  // where the nodes' rows lie
        const int j = tid - 32;
        bool ok = false;
        if (j < n) {
            int64_t prefix = p.prefix_lens[b];
            if (prefix < 0) {
                if (reports) atomicOr(p.err, FDEC_DEVERR_SEQ_LEN);
                prefix = 0;
            }
            const int64_t pos = prefix + j, pi = pos >> p.page_shift;
            const int64_t slot = pos & ((1 << p.page_shift) - 1);
            if (pi >= p.pt_stride) {
                if (reports) atomicOr(p.err, FDEC_DEVERR_SEQ_LEN);
            } else {
                const int64_t page = p.page_table[static_cast<int64_t>(b) * p.pt_stride + pi];
                ok = page >= 0 && page < p.k_pages && page < p.v_pages;
                if (!ok && reports) atomicOr(p.err, FDEC_DEVERR_PAGE_ID);
                s_k[j] = page * p.k_sp + slot * p.k_st + kvh * p.k_sh;
                s_v[j] = page * p.v_sp + slot * p.v_st + kvh * p.v_sh;
            }
        }
        const unsigned bits = __ballot_sync(0xffffffffu, ok);
        if (lane == 0) s_valid[warp - 1] = bits;
    }
    __syncthreads();

    // K and V rows, widened to 16 bits; rows past the tree and unreadable ones are zeros
    const int rows16 = (n + 15) & ~15;
    const uint64_t valid = s_valid[0] | static_cast<uint64_t>(s_valid[1]) << 32;
    uint8_t* sm_k = smem;
    uint8_t* sm_v = smem + rows16 * S::PK;
    bool odd = false;  // an infinite or NaN value
    {
        constexpr int CH = KV8 ? D / 16 : D / 8;  // 16-byte chunks of a stored row
        constexpr int U = 4;
        for (int c0 = tid; c0 < rows16 * CH; c0 += U * kTreeThreads) {
            uint4 kk[U], vv[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = c0 + u * kTreeThreads, j = c / CH;
                kk[u] = vv[u] = make_uint4(0, 0, 0, 0);
                if (c < rows16 * CH && (valid >> j & 1)) {
                    kk[u] = *reinterpret_cast<const uint4*>(p.k_base + s_k[j] + (c - j * CH) * 16);
                    vv[u] = *reinterpret_cast<const uint4*>(p.v_base + s_v[j] + (c - j * CH) * 16);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = c0 + u * kTreeThreads, j = c / CH;
                if (c >= rows16 * CH) break;
                if constexpr (KV8) {
                    const uint32_t kw[4] = {kk[u].x, kk[u].y, kk[u].z, kk[u].w};
                    const uint32_t vw[4] = {vv[u].x, vv[u].y, vv[u].z, vv[u].w};
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint2 ka = widen4<BF16>(kw[2 * h]), kb = widen4<BF16>(kw[2 * h + 1]);
                        const uint2 va = widen4<BF16>(vw[2 * h]), vb = widen4<BF16>(vw[2 * h + 1]);
                        *reinterpret_cast<uint4*>(sm_k + j * S::PK + (c - j * CH) * 32 + h * 16) =
                            make_uint4(ka.x, ka.y, kb.x, kb.y);
                        *reinterpret_cast<uint4*>(sm_v + j * S::PV + (c - j * CH) * 32 + h * 16) =
                            make_uint4(va.x, va.y, vb.x, vb.y);
                        odd |= not_finite<BF16>(va.x) || not_finite<BF16>(va.y) || not_finite<BF16>(vb.x) ||
                               not_finite<BF16>(vb.y);
                    }
                } else {
                    *reinterpret_cast<uint4*>(sm_k + j * S::PK + (c - j * CH) * 16) = kk[u];
                    *reinterpret_cast<uint4*>(sm_v + j * S::PV + (c - j * CH) * 16) = vv[u];
                    odd |= not_finite<BF16>(vv[u].x) || not_finite<BF16>(vv[u].y) || not_finite<BF16>(vv[u].z) ||
                           not_finite<BF16>(vv[u].w);
                }
            }
        }
    }
    odd = __syncthreads_or(odd);

    const int gq = lane >> 2, t = lane & 3;
    const uint32_t k_addr = smem_addr(sm_k) + gq * S::PK + t * 16;
    const uint32_t v_addr = smem_addr(sm_v) + ((lane & 7) + ((lane >> 3) & 1) * 8) * S::PV + (lane >> 4) * 16;
    const int tiles = (R + 15) / 16;
    for (int it = 0; it < p.tiles_per_warp; ++it) {
        const int T = (blk * p.tiles_per_warp + it) * kTreeWarps + warp;
        if (T >= tiles) break;
        // the lane's two rows
        int64_t row[2];  // (token, head) index of out and lse, -1 past the last row
        const uint16_t* q[2];
        uint64_t vis[2];
        float lse2[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = T * 16 + gq + 8 * h;
            row[h] = -1;
            vis[h] = 0;
            lse2[h] = -INFINITY;
            q[h] = nullptr;
            if (r < R) {
                const int i = r / g, head = kvh * g + (r - i * g);
                const int64_t tok = static_cast<int64_t>(b) * N + i;
                row[h] = tok * p.hq + head;
                q[h] = p.q + tok * p.q_st + head * p.q_sh;
                vis[h] = s_anc[i] & valid;
                if (p.lse_prefix != nullptr) lse2[h] = p.lse_prefix[row[h]] * 1.4426950408889634f;
            }
        }
        const int keys = min(n, (min(T * 16 + 15, R - 1)) / g + 1);  // no node sees a later one
        const int nt = (keys + 7) >> 3;

        // the prefix's rows, 64 columns ahead of their use: the first block while S is computed
        float2 op[2][8];
        const auto load_prefix = [&](int cb) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const bool has = p.o_prefix != nullptr && lse2[h] != -INFINITY;
                const float* at = p.o_prefix + row[h] * D + cb * 64 + 2 * t;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    op[h][j] = has ? *reinterpret_cast<const float2*>(at + j * 8) : make_float2(0.f, 0.f);
            }
        };
        load_prefix(0);

        float s[8][4];
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[j][e] = 0.f;
        // S = Q K^T, 32 dims at a time: lane t of a row's four holds dims 8t .. 8t + 7 of
        // both operands, so the k order of the products is permuted alike in both
#pragma unroll 4
        for (int c = 0; c < D / 32; ++c) {
            uint4 qa = make_uint4(0, 0, 0, 0), qb = qa;
            if (q[0] != nullptr) qa = *reinterpret_cast<const uint4*>(q[0] + c * 32 + t * 8);
            if (q[1] != nullptr) qb = *reinterpret_cast<const uint4*>(q[1] + c * 32 + t * 8);
            const uint32_t a0[4] = {qa.x, qb.x, qa.y, qb.y}, a1[4] = {qa.z, qb.z, qa.w, qb.w};
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < nt) {
                    const uint4 kk = lds128<0>(k_addr + j * 8 * S::PK + c * 64);
                    mma_16816<BF16>(s[j], a0, kk.x, kk.y);
                    mma_16816<BF16>(s[j], a1, kk.z, kk.w);
                }
        }

        float m[2], inv[2], w[2], lse_out[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float top = lse2[h];
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const bool sees = vis[h] >> (j * 8 + 2 * t + e) & 1;
                    float& z = s[j][2 * h + e];
                    z = sees ? z * p.scale_log2 : -INFINITY;
                    top = fmaxf(top, z);
                }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            m[h] = top == -INFINITY ? 0.f : top;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float& z = s[j][2 * h + e];
                    z = exp2_approx(z - m[h]);
                    sum += z;
                }
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            w[h] = exp2_approx(lse2[h] - m[h]);
            sum += w[h];
            inv[h] = sum == 0.f ? 0.f : 1.f / sum;
            lse_out[h] = sum == 0.f ? -INFINITY : m[h] * 0.6931471805599453f + logf(sum);
        }

        // O in blocks of 64 columns
        const auto finish = [&](int cb, const float (&acc)[8][4]) {
            const float vs = p.v_scale / kPScale;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (row[h] < 0) continue;
                const int64_t at = row[h] * D + cb * 64 + 2 * t;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float x = (w[h] * op[h][j].x + vs * acc[j][2 * h]) * inv[h];
                    const float y = (w[h] * op[h][j].y + vs * acc[j][2 * h + 1]) * inv[h];
                    if (p.out_type == kOutF32)
                        *reinterpret_cast<float2*>(p.out + at + j * 8) = make_float2(x, y);
                    else
                        *reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(p.out) + at + j * 8) = pack2<BF16>(x, y);
                }
            }
        };
        if (!odd) {
            uint32_t pf[4][TERMS][4];
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t terms[TERMS];
                    const float* z = &s[2 * ks + (e >> 1)][2 * (e & 1)];
                    split_terms<BF16, TERMS>(z[0] * kPScale, z[1] * kPScale, terms);
#pragma unroll
                    for (int i = 0; i < TERMS; ++i) pf[ks][i][e] = terms[i];
                }
#pragma unroll 1
            for (int cb = 0; cb < D / 64; ++cb) {
                if (cb > 0) load_prefix(cb);
                float acc[8][4];
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    if (ks * 2 < nt) {
#pragma unroll
                        for (int dp = 0; dp < 4; ++dp) {
                            uint32_t r0, r1, r2, r3;
                            ldmatrix_x4_trans(v_addr + ks * 16 * S::PV + cb * 128 + dp * 32, r0, r1, r2, r3);
#pragma unroll
                            for (int i = TERMS - 1; i >= 0; --i) {
                                mma_16816<BF16>(acc[2 * dp], pf[ks][i], r0, r1);
                                mma_16816<BF16>(acc[2 * dp + 1], pf[ks][i], r2, r3);
                            }
                        }
                    }
                finish(cb, acc);
            }
        } else {
            // 0 x infinity and 0 x NaN: a product with a row that is not seen must not be made
#pragma unroll 1
            for (int cb = 0; cb < D / 64; ++cb) {
                if (cb > 0) load_prefix(cb);
                float acc[8][4];
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
#pragma unroll
                for (int jt = 0; jt < 8; ++jt)
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk) {
                        const int key = jt * 8 + kk, from = (lane & ~3) | (kk >> 1);
                        const float p0 = __shfl_sync(0xffffffffu, s[jt][kk & 1], from) * kPScale;
                        const float p1 = __shfl_sync(0xffffffffu, s[jt][2 + (kk & 1)], from) * kPScale;
                        if (key < keys) {
                            const bool sees0 = vis[0] >> key & 1, sees1 = vis[1] >> key & 1;
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const float2 v = unpack2<BF16>(*reinterpret_cast<const uint32_t*>(
                                    sm_v + key * S::PV + cb * 128 + j * 16 + t * 4));
                                if (sees0) {
                                    acc[j][0] += p0 * v.x;
                                    acc[j][1] += p0 * v.y;
                                }
                                if (sees1) {
                                    acc[j][2] += p1 * v.x;
                                    acc[j][3] += p1 * v.y;
                                }
                            }
                        }
                    }
                finish(cb, acc);
            }
        }
        if (p.lse != nullptr && t == 0) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (row[h] >= 0) p.lse[row[h]] = lse_out[h];
        }
    }
}

template <int D, bool BF16, bool KV8>
cudaError_t launch_tree(TreeParams p, int num_sms, cudaStream_t s) {
    static unsigned long long attr_done = 0;  // one bit per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !(__atomic_load_n(&attr_done, __ATOMIC_ACQUIRE) & (1ull << dev))) {
        e = cudaFuncSetAttribute(tree_attention_kernel<D, BF16, KV8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(TreeShape<D>::smem(kMaxNodes)));
        if (e != cudaSuccess) return e;
        if (dev < 64) __atomic_fetch_or(&attr_done, 1ull << dev, __ATOMIC_RELEASE);
    }
    const int tiles = (p.nodes * p.group + 15) / 16;
    const int64_t warp_tiles = static_cast<int64_t>(p.batch) * p.hk * tiles;
    const int64_t slots = static_cast<int64_t>(num_sms) * 3 * kTreeWarps;  // warps resident at once
    p.tiles_per_warp = static_cast<int>(std::max<int64_t>(
        1, std::min<int64_t>((tiles + kTreeWarps - 1) / kTreeWarps, (warp_tiles + slots - 1) / slots)));
    const int blocks = (tiles + kTreeWarps * p.tiles_per_warp - 1) / (kTreeWarps * p.tiles_per_warp);
    const int64_t grid = static_cast<int64_t>(p.batch) * p.hk * blocks;
    if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(kTreeThreads, 1, 1);
    cfg.dynamicSmemBytes = TreeShape<D>::smem(p.nodes);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tree_attention_kernel<D, BF16, KV8>, p);
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

cudaError_t launch_tree_attention(TreeParams p, int head_dim, bool bf16, bool kv8, int num_sms, cudaStream_t s) {
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
