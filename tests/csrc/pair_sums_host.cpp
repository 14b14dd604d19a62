// The reductions of pair_sums.cuh on the host: 32 threads stand for a warp's lanes, a shuffle is
// an exchange through an array between two barriers, and fp32 operations are the host's (IEEE,
// uncontracted).
#include <algorithm>
#include <barrier>
#include <cmath>
#include <random>
#include <thread>
#include <vector>

#define __device__
#define __forceinline__ inline

namespace {

constexpr int kLanes = 32;
std::barrier<>* g_meet;
float g_slots[kLanes];
thread_local struct {
    int x;
} threadIdx;

float exchange(float v, int from) {
    g_slots[threadIdx.x] = v;
    g_meet->arrive_and_wait();
    const float got = g_slots[from];
    g_meet->arrive_and_wait();
    return got;
}

float __fadd_rn(float a, float b) { return a + b; }
float __fsub_rn(float a, float b) { return a - b; }
float __fmul_rn(float a, float b) { return a * b; }
float __fmaf_rn(float a, float b, float c) { return std::fmaf(a, b, c); }
float __shfl_sync(unsigned, float v, int lane) { return exchange(v, lane); }
float __shfl_xor_sync(unsigned, float v, int o) { return exchange(v, threadIdx.x ^ o); }
float __shfl_up_sync(unsigned, float v, int o) { return exchange(v, threadIdx.x >= o ? threadIdx.x - o : threadIdx.x); }

}  // namespace

#include "../../paged_split_kv_gather_gb300/csrc/pair_sums.cuh"

using fdec::Pair;

namespace {

template <typename F>
void warp(F&& f) {
    std::barrier<> meet(kLanes);
    g_meet = &meet;
    std::vector<std::thread> lanes;
    for (int l = 0; l < kLanes; ++l)
        lanes.emplace_back([&, l] {
            threadIdx.x = l;
            f(l);
        });
    for (auto& t : lanes) t.join();
}

}  // namespace

extern "C" {

// Every lane's sum of max(p - s q, 0) (q null: of p) over each run of the vocabulary: sums [runs][32] pairs.
void run_sums(const float* p, const float* q, int vocab, int chunk, int runs, float s_hi, float s_lo, float* sums) {
    warp([&](int lane) {
        for (int run = 0; run < runs; ++run) {
            const long begin = static_cast<long>(run) * chunk, end = std::min<long>(vocab, begin + chunk);
            Pair sum = {0.f, 0.f};
            for (long v = begin + lane; v < end; v += kLanes) {
                if (q == nullptr)
                    sum.add(p[v], 0.f);
                else if (s_hi == 1.f && s_lo == 0.f)
                    fdec::add_rest<true>(sum, p[v], q[v], {s_hi, s_lo});
                else
                    fdec::add_rest<false>(sum, p[v], q[v], {s_hi, s_lo});
            }
            sum = fdec::warp_sum(sum);
            sums[(run * kLanes + lane) * 2] = sum.hi;
            sums[(run * kLanes + lane) * 2 + 1] = sum.lo;
        }
    });
}

// Whether a token of probability p_child stands against u W in each of 8 CTAs, CTA c with the sums of lane c; W is
// the row's sum less the probability that has fallen.  Two runs a lane.
void decisions(const float* sums, float p_gone, float p_child, float u, int* stands) {
    warp([&](int lane) {
        for (int cta = 0; cta < 8; ++cta) {
            Pair upto = {0.f, 0.f};
            for (int k = 0; k < 2; ++k) {
                const float* at = sums + ((2 * lane + k) * kLanes + cta) * 2;
                upto.add(at[0], at[1]);
            }
            upto = fdec::warp_scan(upto);
            const Pair total = {__shfl_sync(~0u, upto.hi, 31), __shfl_sync(~0u, upto.lo, 31)};
            const Pair W = total.minus(Pair{0.f, 0.f}.plus({p_gone, 0.f}));
            if (lane == 0) stands[cta] = Pair{p_child, 0.f}.above(W.times(Pair{u, 0.f}.times(1.f)));
        }
    });
}

// exp(3 N(0, 1)) of a seeded generator, divided by its sum.
void seeded_row(int vocab, int seed, float* p) {
    std::mt19937_64 g(seed);
    std::normal_distribution<float> normal(0.f, 3.f);
    double sum = 0;
    for (int i = 0; i < vocab; ++i) sum += p[i] = std::exp(normal(g));
    for (int i = 0; i < vocab; ++i) p[i] = static_cast<float>(p[i] / sum);
}

}  // extern "C"
