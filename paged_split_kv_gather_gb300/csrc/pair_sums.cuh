// pair_sums.cuh -- sums carried as pairs of fp32 values (about 46 bits), and their reductions
// over a warp.  Plain fp32 operations and warp shuffles only, so that a host test can run them.
#pragma once

namespace fdec {

// A number as a pair of fp32 values.
struct Pair {
    float hi, lo;
    // + (x + e), e small against x
    __device__ __forceinline__ void add(float x, float e) {
        const float sum = __fadd_rn(hi, x);
        const float back = __fsub_rn(sum, hi);
        const float err = __fadd_rn(__fsub_rn(hi, __fsub_rn(sum, back)), __fsub_rn(x, back));
        hi = sum;
        lo = __fadd_rn(lo, __fadd_rn(err, e));
    }
    __device__ __forceinline__ Pair plus(Pair x) const {  // lo small against hi again, whatever has cancelled
        Pair d = *this;
        d.add(x.hi, x.lo);
        const float sum = __fadd_rn(d.hi, d.lo);
        return {sum, __fadd_rn(__fsub_rn(d.hi, sum), d.lo)};
    }
    __device__ __forceinline__ Pair minus(Pair x) const { return plus({-x.hi, -x.lo}); }
    __device__ __forceinline__ Pair times(float x) const {
        const float t = __fmul_rn(hi, x);
        return {t, __fmaf_rn(lo, x, __fmaf_rn(hi, x, -t))};
    }
    __device__ __forceinline__ Pair times(Pair x) const {
        const float t = __fmul_rn(hi, x.hi);
        return {t, __fmaf_rn(lo, x.hi, __fmaf_rn(hi, x.lo, __fmaf_rn(hi, x.hi, -t)))};
    }
    __device__ __forceinline__ bool positive() const { return __fadd_rn(hi, lo) > 0.f; }
    __device__ __forceinline__ bool above(Pair x) const {
        Pair d = *this;
        d.add(-x.hi, -x.lo);
        return d.positive();
    }
};

// The sum over a warp: one pair, the same bits in every lane.  (add() does not commute in its low words, so an
// exchange leaves lanes with sums that differ below 2^-46: the first lane's counts.)
__device__ __forceinline__ Pair warp_sum(Pair v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float hi = __shfl_xor_sync(0xffffffffu, v.hi, o), lo = __shfl_xor_sync(0xffffffffu, v.lo, o);
        v.add(hi, lo);
    }
    return {__shfl_sync(0xffffffffu, v.hi, 0), __shfl_sync(0xffffffffu, v.lo, 0)};
}

__device__ __forceinline__ Pair warp_scan(Pair v) {  // inclusive
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float hi = __shfl_up_sync(0xffffffffu, v.hi, o), lo = __shfl_up_sync(0xffffffffu, v.lo, o);
        if (lane >= o) v.add(hi, lo);
    }
    return v;
}

// max(p - s q, 0) added to a sum.  UNIT: s is 1.
template <bool UNIT>
__device__ __forceinline__ void add_rest(Pair& sum, float p, float q, Pair s) {
    if constexpr (UNIT) {
        const float t = fminf(q, p);
        const float d = __fsub_rn(p, t);
        sum.add(d, __fsub_rn(__fsub_rn(p, d), t));  // (exact: p >= t >= 0)
    } else {
        const float t = __fmul_rn(s.hi, q);
        const float te = __fmaf_rn(s.lo, q, __fmaf_rn(s.hi, q, -t));
        float d = __fsub_rn(p, t);
        float e = __fsub_rn(__fsub_rn(__fsub_rn(p, d), t), te);  // exact where p >= t, and else d < 0
        if (!(__fadd_rn(d, e) > 0.f)) d = e = 0.f;
        sum.add(d, e);
    }
}

}  // namespace fdec
