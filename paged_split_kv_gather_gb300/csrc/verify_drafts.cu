// verify_drafts.cu -- verification of drafted tokens against the target's probabilities.
//
// The walk through a tree needs p and q at the children's tokens and, whenever a child
// falls, the sum of what the target has left: W = sum_v max(p(v) - s q(v), 0).  After k
// falls at one node the target left over is max(p - s q, 0) / W, because
//   max(max(p - s q, 0) / W - q, 0) = max(p - (s + W) q, 0) / W      (q >= 0),
// so one number s stands for all of them and every sum reads the same two rows.
//
// A cluster of eight CTAs (one, for a small vocabulary) takes one sequence; each warp sums a run
// of the vocabulary.  The first
// CTA reads what the walk goes by, all children's p and q among it, and copies it into the
// others' shared memory; every warp's sum goes to all CTAs.  Each CTA then walks for itself on the
// same bits, so all of them agree, even on inputs that change under them: a sum costs one
// barrier of the cluster, and the draw none.  (Orders of the first CTA to the others, a second
// barrier a sum: 2.6 us more for 16 trees.)
//
// A token is the first whose cumulative weight passes u W, among 10^5 borders, so sums of
// fp32 rounding would often give another token than exact ones.  Each term p - s q is
// taken as a pair of fp32 values (Dekker's and Knuth's error-free sums and products) and
// added up in pairs, about 46 bits, 13 to 20 fp32 instructions a term.  fp64 units do two
// products a clock and SM here: with the warps' sums and the search in a run in fp64, 64 rows
// of 131072 took 31 us instead of 21, and with the walk, which one warp does while the others
// wait, in fp64 16 trees 14.6 instead of 11.5.
//
// Bytes: the rows p and q of the last node, once from HBM.  64 sequences, p and q of 131072 in
// fp32: 18.6 us, 3.2 TB/s; all sequences read their tokens, sum and search at the same time,
// so most of the 7 us that one sequence takes come on top of the 9 us for the bytes.
#include <algorithm>
#include <cstdint>

#include <cooperative_groups.h>

#include "../../include/fdec.h"
#include "device_utils.cuh"
#include "fdec_internal.h"
#include "pair_sums.cuh"

namespace cg = cooperative_groups;

namespace fdec {

namespace {

constexpr int kVerifyWarps = 8;
constexpr int kVerifyThreads = kVerifyWarps * 32;
constexpr int kMostCtas = 8;  // of a sequence
// A sequence's CTAs each have kVerifyWarps runs of the vocabulary, a warp's each.
constexpr int kMostRuns = kMostCtas * kVerifyWarps;

// Vectors of each row in flight a lane.  (Eight, with two CTAs an SM instead of four: one sequence of 32768 tokens 7.1 us
// instead of 6.7, 64 of 4096 7.7 instead of 7.1; 16 trees over 50021 tokens 11.5 instead of 11.7.)
constexpr int kAhead = 4;

enum Op : int { kSum = 0, kDraw = 1, kStop = 2 };

__device__ __forceinline__ float value(const float* p) { return *p; }
__device__ __forceinline__ float value(const __half* p) { return __half2float(*p); }
__device__ __forceinline__ float value(const __nv_bfloat16* p) { return __bfloat162float(*p); }

__device__ __forceinline__ void value4(const float* p, float (&v)[4]) {
    const float4 x = *reinterpret_cast<const float4*>(p);
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
}
__device__ __forceinline__ void value4(const __half* p, float (&v)[4]) {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    const float2 a = unpack2<false>(x.x), b = unpack2<false>(x.y);
    v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
}
__device__ __forceinline__ void value4(const __nv_bfloat16* p, float (&v)[4]) {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    const float2 a = unpack2<true>(x.x), b = unpack2<true>(x.y);
    v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
}

// A probability as it counts: in [0, 2], NaN as 0.
__device__ __forceinline__ float bounded(float x, bool& bad) {
    const float y = fminf(fmaxf(x, 0.f), 2.f);
    bad |= !(y == x);
    return y;
}

struct Order {       // what comes next
    int op;
    int node;        // whose rows
    int run;         // kDraw: the warp's run of the vocabulary that holds the token
    int place;       // index of the next token in out_tokens
    Pair s;          // weight of q
    Pair target;     // kDraw: cumulative weight to pass, from the run's begin
    uint64_t gone;   // without draft rows: children whose tokens have lost their weight
};

// A drafted token as the walk sees it.
struct Node {
    int tok, par;
    float p, q, u;  // at its token, in its parent's rows; its random number
};

// Whether token v is that of one of the children `gone`.
__device__ __forceinline__ bool is_gone(int v, const Node* nodes, uint64_t gone) {
    for (uint64_t m = gone; m != 0; m &= m - 1)
        if (nodes[__ffsll(static_cast<long long>(m)) - 1].tok == v) return true;
    return false;
}

// What is left of the target at token v, added to a sum.
__device__ __forceinline__ void add_token(Pair& sum, float p, float q, bool drafted, int v, Pair s, const Node* nodes,
                                          uint64_t gone) {
    bool bad = false;
    const float x = bounded(p, bad);
    if (drafted)
        add_rest<false>(sum, x, bounded(q, bad), s);
    else if (!is_gone(v, nodes, gone))
        sum.add(x, 0.f);
}

// One lane's part of a warp's sum over tokens [begin, end).  PLAIN: probabilities are taken as they are, and the
// largest of their bits are noted (as unsigned numbers, all that are not in [0, 2] are above those of 2).
template <typename T, bool VEC, int MODE, bool PLAIN, int AHEAD>  // MODE 0: p, 1: max(p - q, 0), 2: max(p - s q, 0)
__device__ __forceinline__ Pair lane_sum(const T* p, const T* q, int begin, int end, Pair s, uint32_t& most,
                                         bool& bad) {
    const int lane = threadIdx.x & 31;
    Pair sum = {};
    const auto term = [&](float a, float c) {
        if constexpr (PLAIN) {
            most = max(most, __float_as_uint(a));
            if constexpr (MODE > 0) most = max(most, __float_as_uint(c));
        } else {
            a = bounded(a, bad);
            if constexpr (MODE > 0) c = bounded(c, bad);
        }
        if constexpr (MODE > 0)
            add_rest<MODE == 1>(sum, a, c, s);
        else
            sum.add(a, 0.f);
    };
    if constexpr (VEC) {
        constexpr int U = MODE > 0 ? AHEAD : 2 * AHEAD;
        for (int v0 = begin + lane * 4; v0 < end; v0 += U * 128) {
            float a[U][4], c[U][4];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int v = v0 + u * 128;
                a[u][0] = a[u][1] = a[u][2] = a[u][3] = 0.f;
                c[u][0] = c[u][1] = c[u][2] = c[u][3] = 0.f;
                if (v < end) {
                    value4(p + v, a[u]);
                    if constexpr (MODE > 0) value4(q + v, c[u]);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int k = 0; k < 4; ++k) term(a[u][k], c[u][k]);
        }
    } else {
        constexpr int U = (MODE > 0 ? 2 : 4) * AHEAD;
        for (int v0 = begin + lane; v0 < end; v0 += U * 32) {
            float a[U], c[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int v = v0 + u * 32;
                a[u] = v < end ? value(p + v) : 0.f;
                c[u] = 0.f;
                if constexpr (MODE > 0) c[u] = v < end ? value(q + v) : 0.f;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) term(a[u], c[u]);
        }
    }
    return sum;
}

template <typename T, bool VEC, int MODE>
__device__ __forceinline__ Pair mode_sum(const T* p, const T* q, int begin, int end, Pair s, bool& bad) {
    uint32_t most = 0;
    Pair sum = lane_sum<T, VEC, MODE, true, kAhead>(p, q, begin, end, s, most, bad);
    if (__any_sync(0xffffffffu, most > 0x40000000u))
        sum = lane_sum<T, VEC, MODE, false, 2>(p, q, begin, end, s, most, bad);
    return sum;
}

// One warp's sum over tokens [begin, end).
template <typename T, bool VEC>
__device__ __forceinline__ Pair run_sum(const T* p, const T* q, int begin, int end, Pair s, const Node* nodes,
                                        uint64_t gone, bool& bad) {
    const int lane = threadIdx.x & 31;
    Pair sum = {};
    bool hit = false;  // a token without weight lies in here
    if (q == nullptr && gone != 0) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = lane + 32 * h;
            hit |= (gone >> i & 1) && nodes[i].tok >= begin && nodes[i].tok < end;
        }
    }
    if (__any_sync(0xffffffffu, hit)) {
        constexpr int U = 8;
        for (int v0 = begin + lane; v0 < end; v0 += U * 32) {
            float a[U];
#pragma unroll
            for (int u = 0; u < U; ++u) a[u] = v0 + u * 32 < end ? value(p + v0 + u * 32) : 0.f;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float x = bounded(a[u], bad);
                sum.add(is_gone(v0 + u * 32, nodes, gone) ? 0.f : x, 0.f);
            }
        }
    } else if (q == nullptr) {
        sum = mode_sum<T, VEC, 0>(p, q, begin, end, sum, bad);
    } else if (s.hi == 1.f && s.lo == 0.f) {  // the first to fall: nearly all sums
        sum = mode_sum<T, VEC, 1>(p, q, begin, end, sum, bad);
    } else {
        sum = mode_sum<T, VEC, 2>(p, q, begin, end, s, bad);
    }
    return warp_sum(sum);
}

// What a walk goes by: the same bits in every CTA.
struct Tree {
    int n;
    Node node[kMaxNodes];
};

struct Walk {
    Tree tree;
    Pair sum[2][kMostRuns];  // every warp's sum, of even and of odd rounds
    int path[kMaxNodes];
    Pair s;
    // Without draft rows: the target's row is summed once, and a token that falls is taken from that sum.  The
    // difference keeps the sum's absolute error: where it is small (exact), the row is summed without the tokens.
    Pair row_total, row_gone;
    uint64_t weighed;   // the children whose tokens make up row_gone, each token once
    uint64_t gone, left;  // children that have fallen, that are still to try
    int x, len;
    bool have_row, exact;
    bool whole;  // the target's row itself is summed, whatever has fallen
};

// The run of the vocabulary that holds the next token (o.run, o.target), from every warp's sum (a lane's `mine`, their
// sum, the sum up to the lane), less the tokens of the children `weighed`.  A warp; false where nothing is left.
constexpr int kRunsPerLane = kMostRuns / 32;
__device__ __forceinline__ bool draw_run(const Tree& tree, Pair (&mine)[kRunsPerLane], Pair upto, uint64_t weighed,
                                         int chunk, Order& o) {
    const int lane = threadIdx.x & 31;
    constexpr int PER = kRunsPerLane;
    if (weighed != 0) {
        for (uint64_t m = weighed; m != 0; m &= m - 1) {
            const int c = __ffsll(static_cast<long long>(m)) - 1;
            const int run = tree.node[c].tok / chunk;
#pragma unroll
            for (int k = 0; k < PER; ++k)
                if (run == lane * PER + k) {
                    const Pair rest = mine[k].minus({tree.node[c].p, 0.f});
                    mine[k] = rest.hi > mine[k].hi * 0x1p-42f ? rest : Pair{0.f, 0.f};  // (what rounding left is nothing)
                }
        }
        Pair part = mine[0];
#pragma unroll
        for (int k = 1; k < PER; ++k) part.add(mine[k].hi, mine[k].lo);
        upto = warp_scan(part);
    }
    const Pair W = {__shfl_sync(0xffffffffu, upto.hi, 31), __shfl_sync(0xffffffffu, upto.lo, 31)};
    if (!W.positive()) return false;
    const Pair goal = W.times(tree.node[0].u);
    int run = -1, last = -1;
    Pair at = {__shfl_up_sync(0xffffffffu, upto.hi, 1), __shfl_up_sync(0xffffffffu, upto.lo, 1)}, from = {0.f, 0.f};
    if (lane == 0) at = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const Pair before = at;
        at.add(mine[k].hi, mine[k].lo);
        if (mine[k].hi > 0.f) {
            last = lane * PER + k;
            if (run < 0 && at.above(goal)) {
                run = last;
                from = before;
            }
        }
    }
    const unsigned found = __ballot_sync(0xffffffffu, run >= 0);
    const unsigned any = __ballot_sync(0xffffffffu, last >= 0);
    o.op = kDraw;
    if (found != 0) {
        const int who = __ffs(found) - 1;
        o.run = __shfl_sync(0xffffffffu, run, who);
        o.target = goal.minus({__shfl_sync(0xffffffffu, from.hi, who), __shfl_sync(0xffffffffu, from.lo, who)});
    } else {  // (only by rounding: the last run with weight, its last token)
        o.run = __shfl_sync(0xffffffffu, last, 31 - __clz(any));
        o.target = W.times(4.f);
    }
    return true;
}

// What comes next: a CTA's first warp, at the beginning (no sums) and whenever all sums (`runs` of them) have come.
__device__ __noinline__ Order next_order(Walk& walk, const Pair* sums, int runs, bool drafted, int chunk) {
    const int lane = threadIdx.x & 31;
    constexpr int PER = kRunsPerLane;
    const Tree& tree = walk.tree;
    // (nodes past the last have not been given)
    const bool has0 = lane < tree.n, has1 = lane + 32 < tree.n;
    const int par0 = has0 ? tree.node[lane].par : -1, par1 = has1 ? tree.node[lane + 32].par : -1;
    const int tok0 = has0 ? tree.node[lane].tok : -1, tok1 = has1 ? tree.node[lane + 32].tok : -1;
    const auto children = [&](int node) {
        return static_cast<uint64_t>(__ballot_sync(0xffffffffu, par0 == node)) |
               static_cast<uint64_t>(__ballot_sync(0xffffffffu, par1 == node)) << 32;
    };
    int x = 0, len = 1;
    Pair s = {0.f, 0.f}, W = {1.f, 0.f}, row_total = {0.f, 0.f}, row_gone = {0.f, 0.f};
    uint64_t gone = 0, left = 0, weighed = 0;
    bool have_row = false, exact = false, summed = false, whole = false;
    if (sums != nullptr) {
        x = walk.x, len = walk.len;
        s = walk.s, row_total = walk.row_total, row_gone = walk.row_gone;
        gone = walk.gone, left = walk.left, weighed = walk.weighed;
        have_row = walk.have_row, exact = walk.exact, whole = walk.whole;
    } else {
        left = children(0);
        if (lane == 0) walk.path[0] = 0;
    }
    Order o = {};
    o.op = kStop;
    Pair mine[PER] = {}, upto = {0.f, 0.f};
    if (tree.n > 0) {
        bool ask = false;
        if (sums != nullptr) {  // the sums that were asked for
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                if (lane * PER + k < runs) mine[k] = sums[lane * PER + k];
                upto.add(mine[k].hi, mine[k].lo);
            }
            upto = warp_scan(upto);
            W = {__shfl_sync(0xffffffffu, upto.hi, 31), __shfl_sync(0xffffffffu, upto.lo, 31)};
            summed = true;
            if (!drafted && !exact && !whole) {
                row_total = W;
                have_row = true;
                W = row_total.minus(row_gone);
                if (!(W.hi * 64.f > row_total.hi)) ask = exact = true;
            }
            if (!ask && !W.positive()) left = 0;
        }
        while (left != 0 && !ask) {
            const int c = __ffsll(static_cast<long long>(left)) - 1;
            left &= left - 1;
            const int t = tree.node[c].tok;
            const float q = tree.node[c].q;
            Pair rest = {tree.node[c].p, 0.f};
            if (drafted) {
                rest = rest.minus(s.times(q));
                if (!rest.positive()) rest = {0.f, 0.f};
            } else {
                const uint64_t same = static_cast<uint64_t>(__ballot_sync(0xffffffffu, tok0 == t)) |
                                      static_cast<uint64_t>(__ballot_sync(0xffffffffu, tok1 == t)) << 32;
                if (same & gone) rest = {0.f, 0.f};
            }
            if (rest.above(W.times(Pair{tree.node[c].u, 0.f}.times(q)))) {
                x = c;
                if (lane == 0) walk.path[len] = c;
                ++len;
                s = {0.f, 0.f}, W = {1.f, 0.f}, gone = 0, summed = false;
                row_gone = {0.f, 0.f}, weighed = 0, have_row = exact = false;
                left = children(c);
            } else {
                s = s.plus(W);
                gone |= uint64_t{1} << c;
                if (!drafted && rest.hi > 0.f) {
                    row_gone = row_gone.plus(rest);
                    weighed |= uint64_t{1} << c;
                }
                W = row_total.minus(row_gone);
                if (drafted || !have_row || exact || !(W.hi * 64.f > row_total.hi)) ask = true;
                if (ask && have_row) exact = true;
            }
        }
        const bool plain = drafted || exact || whole;  // (the sums are those of what is left)
        if (!ask && !(summed && draw_run(tree, mine, upto, plain ? 0 : weighed, chunk, o))) {  // no child stands
            if (summed) {  // nothing is left: the target's row itself, if that is not it already
                ask = !whole;
                s = {0.f, 0.f}, gone = 0;
            } else {  // no child has fallen here
                ask = true;
            }
            whole = true;
        }
        if (ask) o.op = kSum;
        o.node = x;
        o.s = s;
        // (a plain sum of the row first; without its tokens where it must be exact)
        o.gone = o.op == kSum && !exact ? 0 : gone;
        o.place = len - 1;
    }
    __syncwarp();
    if (lane == 0) {
        walk.x = x, walk.len = len;
        walk.s = s, walk.row_total = row_total, walk.row_gone = row_gone;
        walk.gone = gone, walk.left = left, walk.weighed = weighed;
        walk.have_row = have_row, walk.exact = exact, walk.whole = whole;
    }
    __syncwarp();
    return o;
}

// CTAS: of a sequence.
template <typename T, bool VEC, int CTAS>
__global__ void __launch_bounds__(kVerifyThreads, 4) verify_drafts_kernel(const VerifyParams p) {
    __shared__ Walk s_walk;
    __shared__ Pair s_warp[kVerifyWarps];
    __shared__ int s_first, s_last, s_any;
    __shared__ Order s_order;

    cg::cluster_group cluster = cg::this_cluster();
    const int rank = CTAS > 1 ? static_cast<int>(cluster.block_rank()) : 0;
    const auto meet = [&] {  // all threads of the sequence's CTAs
        if constexpr (CTAS > 1)
            cluster.sync();
        else
            __syncthreads();
    };
    const int b = blockIdx.x / CTAS;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int N = p.nodes;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if constexpr (CTAS > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // this CTA runs

    const T* target = static_cast<const T*>(p.target) + static_cast<int64_t>(b) * p.t_seq;
    const T* draft = p.draft != nullptr ? static_cast<const T*>(p.draft) + static_cast<int64_t>(b) * p.d_seq : nullptr;
    unsigned flags = 0;
    if (rank == 0 && tid < kMaxNodes) {
        int n = p.node_counts != nullptr ? p.node_counts[b] : N;
        int par = tid - 1, tok = -1;
        float u = 0.f;
        if (tid < N) {  // (read before n is there)
            const int64_t at = static_cast<int64_t>(b) * N + tid;
            tok = p.tokens[at];
            if (p.parents != nullptr) par = p.parents[at];
            u = p.uniforms[at];
        }
        if (n < 0 || n > N) {
            flags |= FDEC_DEVERR_SEQ_LEN;
            n = min(max(n, 0), N);
        }
        if (tid >= n) par = -1;
        if (par < -1 || par >= tid) {
            flags |= FDEC_DEVERR_TREE;
            par = -1;
        }
        float pv = 0.f, qv = 1.f;
        if (tid > 0 && tid < n && par >= 0) {
            if (tok < 0 || tok >= p.vocab) {
                flags |= FDEC_DEVERR_TREE;
                par = -1;
            } else {
                bool bad = false;
                pv = bounded(value(target + par * p.t_node + tok), bad);
                if (draft != nullptr) qv = bounded(value(draft + par * p.d_node + tok), bad);
                if (bad) flags |= FDEC_DEVERR_PROB;
            }
        }
        Node& node = s_walk.tree.node[tid];
        node.tok = tid < n && tid > 0 ? tok : -1;
        node.par = par;
        node.p = pv;
        node.q = qv;
        node.u = u >= 0.f ? fminf(u, 0.99999994f) : 0.f;
        if (tid == 0) s_walk.tree.n = n;
    }
    __syncthreads();
    if constexpr (CTAS > 1) {
        asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // the other CTAs run: their memory is written next
        if (rank == 0 && warp > 0 && warp < CTAS) {
            const int* from = reinterpret_cast<const int*>(&s_walk.tree);
            int* to = reinterpret_cast<int*>(cluster.map_shared_rank(&s_walk.tree, warp));
            const int words = 1 + s_walk.tree.n * static_cast<int>(sizeof(Node) / 4);
            for (int i = lane; i < words; i += 32) to[i] = from[i];
        }
        cluster.sync();
    }

    const int n = s_walk.tree.n;
    // (at most two sums for every child and two for the draw)
    for (int round = 0; round < 2 * kMaxNodes + 3; ++round) {
        if (warp == 0) {
            const Pair* sums = round > 0 ? s_walk.sum[(round - 1) & 1] : nullptr;
            const Order next = next_order(s_walk, sums, CTAS * kVerifyWarps, draft != nullptr, p.chunk);
            if (lane == 0) s_order = next;
        }
        __syncthreads();
        const Order o = s_order;
        if (o.op != kSum) break;
        const T* prow = target + o.node * p.t_node;
        // (the target's row itself needs no q; a leaf has none)
        const T* qrow = draft != nullptr && o.s.hi != 0.f ? draft + o.node * p.d_node : nullptr;
        const int run = rank * kVerifyWarps + warp;
        const int64_t begin = static_cast<int64_t>(run) * p.chunk;
        Pair sum = {};
        bool bad = false;
        if (begin < p.vocab) {
            const int end = static_cast<int>(min(static_cast<int64_t>(p.vocab), begin + p.chunk));
            sum = run_sum<T, VEC>(prow, qrow, static_cast<int>(begin), end, o.s, s_walk.tree.node, o.gone, bad);
        }
        if (bad) flags |= FDEC_DEVERR_PROB;
        if constexpr (CTAS > 1) {
            if (lane < CTAS) cluster.map_shared_rank(&s_walk, lane)->sum[round & 1][run] = sum;
        } else if (lane == 0) {
            s_walk.sum[round & 1][run] = sum;
        }
        meet();
    }

    const Order o = s_order;
    const int64_t out = static_cast<int64_t>(b) * N;
    if (rank == 0) {
        if (tid < N) {  // (len is the first warp's: the order's place tells the others)
            const int steps = n > 0 ? o.place + 1 : 0;
            p.path[out + tid] = tid < steps ? s_walk.path[tid] : -1;
            if (tid + 1 < steps)
                p.out_tokens[out + tid] = s_walk.tree.node[s_walk.path[tid + 1]].tok;
            else if (o.op != kDraw || tid != o.place)
                p.out_tokens[out + tid] = -1;
            if (tid == 0) p.path_lens[b] = steps;
        }
        if (n > 0 && o.op != kDraw) flags |= FDEC_DEVERR_PROB;
    }
    if (o.op == kDraw && o.run / kVerifyWarps == rank) {
        // the run's tokens, a stretch for each thread in their order
        const T* prow = target + o.node * p.t_node;
        const T* qrow = draft != nullptr && o.s.hi != 0.f ? draft + o.node * p.d_node : nullptr;
        const int64_t begin = static_cast<int64_t>(o.run) * p.chunk;
        const int end = static_cast<int>(min(static_cast<int64_t>(p.vocab), begin + p.chunk));
        const int per = (p.chunk + kVerifyThreads - 1) / kVerifyThreads;
        const int v0 = static_cast<int>(min(static_cast<int64_t>(end), begin + static_cast<int64_t>(tid) * per));
        const int v1 = min(end, v0 + per);
        constexpr int U = 8;
        const Pair weight = o.s, target_sum = o.target;
        Pair mine = {};
        for (int v = v0; v < v1; v += U) {
            float a[U], c[U];
#pragma unroll
            for (int k = 0; k < U; ++k) {
                a[k] = v + k < v1 ? value(prow + v + k) : 0.f;
                c[k] = v + k < v1 && qrow != nullptr ? value(qrow + v + k) : 0.f;
            }
#pragma unroll
            for (int k = 0; k < U; ++k)
                if (v + k < v1) add_token(mine, a[k], c[k], qrow != nullptr, v + k, weight, s_walk.tree.node, o.gone);
        }
        const bool some = mine.hi > 0.f;
        const Pair scan = warp_scan(mine);
        if (lane == 31) s_warp[warp] = scan;
        if (tid == 0) {
            s_first = kVerifyThreads;
            s_last = -1;
            s_any = p.vocab;
        }
        __syncthreads();
        Pair before = {};
        for (int k = 0; k < warp; ++k) before.add(s_warp[k].hi, s_warp[k].lo);
        Pair upto = before;
        upto.add(scan.hi, scan.lo);
        if (some) {
            if (upto.above(target_sum)) atomicMin(&s_first, tid);
            atomicMax(&s_last, tid);
        }
        const Pair prior = {__shfl_up_sync(0xffffffffu, scan.hi, 1), __shfl_up_sync(0xffffffffu, scan.lo, 1)};
        if (lane > 0) before.add(prior.hi, prior.lo);
        __syncthreads();
        if (tid == (s_first < kVerifyThreads ? s_first : s_last)) {
            int token = -1;
            for (int v = v0; v < v1; ++v) {
                Pair here = {};
                add_token(here, value(prow + v), qrow != nullptr ? value(qrow + v) : 0.f, qrow != nullptr, v, weight,
                          s_walk.tree.node, o.gone);
                if (!(here.hi > 0.f)) continue;
                token = v;
                before.add(here.hi, here.lo);
                if (before.above(target_sum)) break;
            }
            p.out_tokens[out + o.place] = token;
        }
        if (s_last < 0) {  // (only by rounding: the run has no weight after all; the first token that has some)
            for (int v = tid; v < p.vocab; v += kVerifyThreads) {
                Pair here = {};
                add_token(here, value(prow + v), qrow != nullptr ? value(qrow + v) : 0.f, qrow != nullptr, v, weight,
                          s_walk.tree.node, o.gone);
                if (here.hi > 0.f) atomicMin(&s_any, v);
            }
            __syncthreads();
            if (tid == 0) p.out_tokens[out + o.place] = s_any < p.vocab ? s_any : -1;
        }
    }
    if (flags != 0 && p.err != nullptr) atomicOr(p.err, flags);
}

template <typename T>
bool vectors(const VerifyParams& p) {
    const auto ok = [](const void* base, int64_t a, int64_t b) {
        return reinterpret_cast<uintptr_t>(base) % (4 * sizeof(T)) == 0 && a % 4 == 0 && b % 4 == 0;
    };
    return p.vocab % 4 == 0 && ok(p.target, p.t_seq, p.t_node) && ok(p.draft, p.d_seq, p.d_node);
}

template <typename T, bool VEC, int CTAS>
cudaError_t launch_verify_one(VerifyParams p, cudaStream_t s) {
    constexpr int kRuns = CTAS * kVerifyWarps;
    p.chunk = ((p.vocab + kRuns - 1) / kRuns + 127) / 128 * 128;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.batch) * CTAS, 1, 1);
    cfg.blockDim = dim3(kVerifyThreads, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CTAS;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CTAS > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, verify_drafts_kernel<T, VEC, CTAS>, p);
}

template <typename T, bool VEC>
cudaError_t launch_verify_v(const VerifyParams& p, cudaStream_t s) {
    // A small vocabulary is one CTA's, which needs no cluster: 64 sequences 7.1 us against 9.3 at 4096 and 7.7 against 9.4 at
    // 8192 tokens, 16 trees 8.7 against 10.5 and 9.7 against 10.2; at 16384 tokens (eight vectors ahead) 9.6 against 9.5
    // and 12.8 against 10.3.
    // (Clusters of 4 CTAs 1.5 us more for 16 trees over 50021 tokens, of 16 9 more.)
    if (p.vocab <= 8192) return launch_verify_one<T, VEC, 1>(p, s);
    return launch_verify_one<T, VEC, kMostCtas>(p, s);
}

template <typename T>
cudaError_t launch_verify(const VerifyParams& p, cudaStream_t s) {
    return vectors<T>(p) ? launch_verify_v<T, true>(p, s) : launch_verify_v<T, false>(p, s);
}

}  // namespace

cudaError_t launch_verify_drafts(const VerifyParams& p, int prob_dtype, cudaStream_t s) {
    switch (prob_dtype) {
        case FDEC_PROB_F16: return launch_verify<__half>(p, s);
        case FDEC_PROB_BF16: return launch_verify<__nv_bfloat16>(p, s);
        case FDEC_PROB_F32: return launch_verify<float>(p, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace fdec
