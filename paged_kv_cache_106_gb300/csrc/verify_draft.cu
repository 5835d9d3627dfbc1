// Verification of drafted tokens against the target's probabilities
// (pa_verify_draft): which drafted nodes are accepted, and the next token,
// from given uniform numbers.
//
// Mathematics (speculative sampling on a tree).  At a node v the target's
// next-token weights start as w = p_v (its row of probabilities), Z = 1.  The
// children c of v are tried in index order: token x = x_c is accepted if
//     u_c q_v(x) Z < w(x)
// and the walk goes on at c; otherwise
//     w <- max(w - Z q_v, 0),   Z <- sum w   (unless that sum is 0),
// which is the distribution that, mixed with the accepted share of q_v, gives
// p_v again.  Where no child is accepted the next token is the first i whose
// running sum of w passes u_s sum w.  Without draft probabilities q_v is 1 at
// the child's token (a drafter that picks one token): a rejected token's
// weight becomes 0.
//
// Exactness.  A running sum crosses an edge at every token, so rounding of
// 2^-24 in it would move the answer once in some hundred samples at 50 k
// tokens.  All weights and sums are therefore pairs of fp32 (value + error
// term), added with error-free transformations; in fp64 the additions alone
// would take three times a row's bytes (this GPU does two fp64 operations a clock
// and SM).  What a pair cannot hold, with u = 2^-24 and W the row's sum: after j
// terms of `plus` the error term is j u W at most and its two roundings 2 j u^2 W,
// so a lane's m terms of a segment make m^2 u^2 W (m is 16 up to 131072 tokens;
// in trials it is 2^-46 W for 16 terms, 2^-44 W for 64); each `add` makes 3 u^2 W
// at most, and there are 5 over the lanes, up to 32 over the segments and some 25
// over the warps and in the search, 2^-40 W in all.  A rejection is exact the
// first time and makes some 2^-44 W after that, beside Z's own error.  No atomics:
// the result depends only on the inputs.
//
// What bounds it: the rows it has to read (one target row, and one draft row
// once something is rejected, 4 V bytes each) for a large batch; the chain of
// dependent loads and barriers for a small one.  Per sequence one cluster of
// up to 8 CTAs shares a row: first the scalars p_parent(x), q_parent(x), u of
// all nodes are gathered at once, so the walk itself touches no memory (a
// chain never needs a pass over a row before the last one), then each pass over
// a row is split evenly over the cluster's warps, contiguous spans in order of
// index, whose sums go to every CTA of the cluster.  A warp keeps the sums of up
// to 32 segments of its span, so the one in whose span the target falls goes
// through one segment again, then scans 128 tokens.  All loads of a round come
// before any of them is used (256 chains: 44 -> 30 us).  The code is kept short: a
// CTA goes through it about once, and with everything unrolled its instructions
// came slower than the data (112 us).
//
// Measured (in a graph): 256 chains of 5 to 9 nodes, 50272 tokens, fp32 31 us (the
// rows that have to be read take 15 at 6.78 TB/s); 64 trees of 10 to 26 nodes,
// 100003 tokens, fp16 62 us (4; two to three passes one after another, each of
// which applies all rejections so far to every element); one chain of 8, 32000 tokens,
// 9.0 us (launch, gather, walk, sum, search: each waits for the one before).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <climits>
#include <type_traits>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pagedkv {

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kWarps = 8, kThreads = kWarps * 32, kPerSm = 4;
constexpr int kMaxCluster = 8;
constexpr int kPerLane = kMaxCluster * kWarps / 32;   // warps' sums a lane of warp 0 takes
constexpr int kRound = 4;                             // rows of 128 tokens a warp loads at a time
constexpr int kSegments = 32;                         // sums a warp keeps of its span
constexpr int kNodes = PA_TREE_MAX_NODES;

struct VerifyParams {
    int32_t *path, *path_lens, *next_tokens;
    const void *p, *q;
    const int32_t *tokens, *parents, *q_starts;
    const float *u_accept, *u_sample;
    int32_t max_q, q_rows, vocab;
    int32_t rows, segment;   // rows of 128 a warp owns, and of one of its segments (a multiple of kRound)
    int32_t *status;
};

// A nonnegative weight as an unevaluated sum of two fp32.
struct __align__(8) Pair {
    float hi, lo;
};

__device__ __forceinline__ Pair two_sum(float a, float b) {
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}

__device__ __forceinline__ Pair add(Pair a, Pair b) {
    Pair t = two_sum(a.hi, b.hi);
    const float lo = __fadd_rn(t.lo, __fadd_rn(a.lo, b.lo)), hi = __fadd_rn(t.hi, lo);
    return {hi, __fsub_rn(lo, __fsub_rn(hi, t.hi))};
}

__device__ __forceinline__ bool above(Pair a, Pair b) {
    if (b.hi == INFINITY) return false;
    const Pair d = two_sum(a.hi, -b.hi);
    return __fadd_rn(d.hi, __fadd_rn(d.lo, __fsub_rn(a.lo, b.lo))) > 0.f;
}

// The running sum a and one weight more; a.lo collects the errors.
__device__ __forceinline__ Pair plus(Pair a, Pair w) {
    const Pair t = two_sum(a.hi, w.hi);
    return {t.hi, __fadd_rn(a.lo, __fadd_rn(t.lo, w.lo))};
}

// max(p - q, 0), exact: what is left where p > q has p as the larger term.
__device__ __forceinline__ Pair less(float p, float q) {
    const float d = __fsub_rn(p, q), e = __fsub_rn(__fsub_rn(p, d), q);
    return d > 0.f ? Pair{d, e} : Pair{0.f, 0.f};
}

// a b z
__device__ __forceinline__ Pair times(float a, float b, Pair z) {
    const float p = __fmul_rn(a, b), e = __fmaf_rn(a, b, -p);
    const float h = __fmul_rn(p, z.hi);
    const float l = __fadd_rn(__fmaf_rn(p, z.hi, -h), __fmaf_rn(p, z.lo, __fmul_rn(e, z.hi)));
    return {h, l};
}

// max(w - z q, 0), z = zh + zl
__device__ __forceinline__ Pair reject(Pair w, float q, float zh, float zl) {
    const float ph = __fmul_rn(q, zh);
    const float pl = __fmaf_rn(q, zl, __fmaf_rn(q, zh, -ph));
    Pair d = two_sum(w.hi, -ph);
    d.lo = __fadd_rn(d.lo, __fsub_rn(w.lo, pl));
    const float hi = __fadd_rn(d.hi, d.lo);
    d.lo = __fsub_rn(d.lo, __fsub_rn(hi, d.hi));
    d.hi = hi;
    if (!(d.hi > 0.f)) d.hi = d.lo = 0.f;
    return d;
}

// Probabilities that are not positive and finite count as 0.
__device__ __forceinline__ float clean(float x) {
    return __float_as_uint(x) < 0x7f800000u ? x : 0.f;   // (negative: the top bit; NaN: above infinity)
}

__device__ __forceinline__ float value(const float *p) { return clean(__ldg(p)); }
__device__ __forceinline__ float value(const __half *p) { return clean(__half2float(__ldg(p))); }
__device__ __forceinline__ float value(const __nv_bfloat16 *p) { return clean(__bfloat162float(__ldg(p))); }

// Elements x .. x + 3 of a row of V, 0 outside it, one by one.
template <typename T>
__device__ __noinline__ float4 edge4(const T *row, int x, int V) {
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = x + i >= 0 && x + i < V ? value(row + x + i) : 0.f;
    return make_float4(v[0], v[1], v[2], v[3]);
}
// Four elements as they lie in memory.
template <typename T>
struct Raw {
    using type = uint2;
};
template <>
struct Raw<float> {
    using type = uint4;
};
__device__ __forceinline__ float4 unpack(const uint4 &r, float) {
    return make_float4(clean(__uint_as_float(r.x)), clean(__uint_as_float(r.y)), clean(__uint_as_float(r.z)),
                       clean(__uint_as_float(r.w)));
}
template <typename T>
__device__ __forceinline__ float4 unpack(const uint2 &r, T) {
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint16_t b = (uint16_t)((i < 2 ? r.x : r.y) >> (16 * (i & 1)));
        if constexpr (std::is_same<T, __half>::value) v[i] = clean(__half2float(__ushort_as_half(b)));
        else v[i] = clean(__bfloat162float(__ushort_as_bfloat16(b)));
    }
    return make_float4(v[0], v[1], v[2], v[3]);
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void store_cluster(Pair *local, uint32_t rank, Pair v) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(local)), "r"(rank));
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(a), "f"(v.hi), "f"(v.lo) : "memory");
}

struct Shared {
    float pu[kNodes], qu[kNodes], u[kNodes];   // of a node: its token's weight in its parent's rows
    int32_t up[kNodes], tok[kNodes];
    float zh[kNodes], zl[kNodes];              // Z before each rejection at the current node
    int32_t out[kNodes];                       // the tokens rejected there
    Pair sums[2][kMaxCluster * kWarps];        // the row's sums by warp, in order; by parity of the pass
    Pair seg[kWarps][kSegments];               // of this CTA's warps' segments
    int32_t cur, k;                            // the row to add up: its node, rejections there
    int32_t owner;                             // the warp that finds the next token, or:
    Pair left;                                 // of the target, within the owner's span
};
enum { kAgain = -1, kNone = -2 };

template <typename T, bool DRAFT, bool VEC>
__global__ void __launch_bounds__(kThreads, kPerSm) verify_draft_kernel(const VerifyParams a) {
    __shared__ Shared sh;
    const uint32_t rank = cluster_rank(), C = cluster_size();
    const int s = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int V = a.vocab;
    const int row0 = a.q_starts[s], n = a.q_starts[s + 1] - row0;
    const bool bad = row0 < 0 || n < 0 || n > a.max_q || (long long)row0 + n > a.q_rows;
    if (bad || n == 0) {   // the whole cluster alike
        if (rank == 0) {
            for (int i = tid; i < a.max_q; i += kThreads) a.path[(size_t)s * a.max_q + i] = -1;
            if (tid == 0) {
                a.path_lens[s] = 0;
                a.next_tokens[s] = -1;
                if (bad) report(a.status, PA_ERR_INVALID_ARG);
            }
        }
        return;
    }
    cluster_arrive();      // waited for before the first store to another CTA: all have started then
    const T *P = static_cast<const T *>(a.p) + (size_t)row0 * V;
    const T *Q = DRAFT ? static_cast<const T *>(a.q) + (size_t)row0 * V : nullptr;
    const float us = a.u_sample[s];

    // ---- what the walk needs of every node
    if (tid < n) {
        const int i = tid;
        int up = i - 1;
        if (a.parents && i > 0) {
            up = a.parents[row0 + i];
            if (up < -1 || up >= i) {
                report(a.status, PA_ERR_INVALID_ARG);
                up = -1;
            }
        }
        if (i == 0) up = -1;
        const int x = i > 0 ? a.tokens[row0 + i] : 0;
        float pu = 0.f, qu = 0.f;
        bool in = x >= 0 && x < V;
        if (i > 0 && !in) report(a.status, PA_ERR_INVALID_ARG);
        if (up >= 0 && in) {
            pu = value(P + (size_t)up * V + x);
            qu = DRAFT ? value(Q + (size_t)up * V + x) : 1.f;
        }
        sh.up[i] = in ? up : -1;      // a token outside the vocabulary is never reached
        sh.tok[i] = x;
        sh.pu[i] = pu;
        sh.qu[i] = qu;
        sh.u[i] = a.u_accept[row0 + i];
    }
    __syncthreads();
    cluster_wait();

    // Spans are counted from the vector boundary at or before the row's start.
    const int gw = (int)rank * kWarps + warp;          // this warp's place in the row
    const int lo = gw * a.rows * 128 + lane * 4;       // this lane's first tokens of it

    struct Row {
        const T *p, *q;
        int shift, k;                                  // elements before the row; rejections
    };
    auto row_of = [&](int v, int k) {
        const long long at = (long long)v * V;
        return Row{P + at, DRAFT ? Q + at : nullptr, VEC ? (int)(((long long)row0 * V + at) & 3) : 0, k};
    };
    // This lane's four weights of a 128, from their probabilities; x: the first's token.
    auto weights = [&](const Row &r, int x, const float4 &pv, const float4 &qv, Pair (&w)[4]) {
        w[0] = {pv.x, 0.f};
        w[1] = {pv.y, 0.f};
        w[2] = {pv.z, 0.f};
        w[3] = {pv.w, 0.f};
        if (DRAFT && r.k > 0) {          // (Z is 1 for the first rejection)
            w[0] = less(pv.x, qv.x);
            w[1] = less(pv.y, qv.y);
            w[2] = less(pv.z, qv.z);
            w[3] = less(pv.w, qv.w);
        }
#pragma unroll 1
        for (int i = DRAFT ? 1 : 0; i < r.k; ++i) {
            if (DRAFT) {
                const float zh = sh.zh[i], zl = sh.zl[i];
                w[0] = reject(w[0], qv.x, zh, zl);
                w[1] = reject(w[1], qv.y, zh, zl);
                w[2] = reject(w[2], qv.z, zh, zl);
                w[3] = reject(w[3], qv.w, zh, zl);
            } else {
                const int out = sh.out[i] - x;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (out == e) w[e] = {0.f, 0.f};
            }
        }
    };
    // This lane's sums of kRound rows of 128 from row j on.
    auto round_sums = [&](const Row &r, int j, Pair (&t)[kRound]) {
        // every load first, each on its own: nothing between them waits for one
        typename Raw<T>::type pr[kRound] = {}, qr[kRound] = {};
#pragma unroll
        for (int b = 0; b < kRound; ++b) {
            const int x = lo + (j + b) * 128 - r.shift;
            if (VEC && j + b < a.rows && x >= 0 && x + 4 <= V) {
                pr[b] = __ldg(reinterpret_cast<const typename Raw<T>::type *>(r.p + x));
                if (DRAFT && r.k > 0) qr[b] = __ldg(reinterpret_cast<const typename Raw<T>::type *>(r.q + x));
            }
        }
#pragma unroll
        for (int b = 0; b < kRound; ++b) {
            const int x = lo + (j + b) * 128 - r.shift;
            float4 pv = unpack(pr[b], T()), qv = unpack(qr[b], T());
            if (j + b < a.rows && (!VEC || x < 0 || x + 4 > V) && x < V) {   // a row's ends
                pv = edge4(r.p, x, V);
                if (DRAFT && r.k > 0) qv = edge4(r.q, x, V);
            }
            Pair w[4];
            weights(r, x, pv, qv, w);
            t[b] = plus(plus(plus(w[0], w[1]), w[2]), w[3]);
        }
    };
    auto over_lanes = [&](Pair v) {
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1)
            v = add(v, {__shfl_xor_sync(kAll, v.hi, off), __shfl_xor_sync(kAll, v.lo, off)});
        return v;
    };
    // Running sums over a warp's lanes.
    auto scan = [&](Pair incl) {
#pragma unroll 1
        for (int off = 1; off < 32; off <<= 1) {
            const Pair y = {__shfl_up_sync(kAll, incl.hi, off), __shfl_up_sync(kAll, incl.lo, off)};
            if (lane >= off) incl = add(incl, y);
        }
        return incl;
    };
    auto from_lane = [&](const Pair &v, int l) { return Pair{__shfl_sync(kAll, v.hi, l), __shfl_sync(kAll, v.lo, l)}; };

    // Warp 0 of every CTA walks (alike) up to where the sum of a row is needed,
    // all warps add up that row, warp 0 goes on.
    int i = 1, cur = 0, k = 0, len = 1;
    bool pending = false;       // the last rejection's sum is not known yet
    Pair z = {1.f, 0.f};
    int32_t *path = a.path + (size_t)s * a.max_q;
    const bool writer = rank == 0 && tid == 0;
    if (writer) path[0] = 0;
    for (int parity = 0;; parity ^= 1) {
        if (warp == 0) {
            for (; i < n; ++i) {
                if (sh.up[i] != cur) continue;
                if (pending) break;
                Pair w = {sh.pu[i], 0.f};
                const float qx = sh.qu[i];
                if (DRAFT) {
                    for (int r = 0; r < k; ++r) w = reject(w, qx, sh.zh[r], sh.zl[r]);
                } else {
                    for (int r = 0; r < k; ++r)
                        if (sh.out[r] == sh.tok[i]) w = {0.f, 0.f};
                }
                if (above(w, times(sh.u[i], qx, z))) {
                    cur = i;
                    k = 0;
                    z = {1.f, 0.f};
                    if (writer) path[len] = i;
                    ++len;
                } else {
                    __syncwarp();       // every lane has read the list's earlier entries
                    if (lane == 0) {
                        sh.zh[k] = z.hi;
                        sh.zl[k] = z.lo;
                        sh.out[k] = sh.tok[i];
                    }
                    __syncwarp();
                    ++k;
                    pending = true;
                }
            }
            if (lane == 0) {
                sh.cur = cur;
                sh.k = k;
            }
        }
        __syncthreads();
        const Row row = row_of(sh.cur, sh.k);
        Pair acc = {0.f, 0.f};
#pragma unroll 1
        for (int j = 0, g = 0; j < a.rows; ++g) {
            Pair sum = {0.f, 0.f};
#pragma unroll 1
            for (const int end = j + a.segment; j < end; j += kRound) {
                Pair t[kRound];
                round_sums(row, j, t);
#pragma unroll
                for (int b = 0; b < kRound; ++b) sum = plus(sum, t[b]);
            }
            sum = over_lanes(sum);
            if (lane == 0) sh.seg[warp][g] = sum;
            acc = add(acc, sum);
        }
        // to every CTA; two buffers, since a CTA of the cluster may still read the
        // last pass's (none can be two passes behind)
        if (lane < (int)C) store_cluster(&sh.sums[parity][gw], (uint32_t)lane, acc);
        __syncwarp();
        cluster_arrive();
        cluster_wait();
        if (warp == 0) {
            // lane l: the sums of warps kPerLane l .. of the row
            const Pair zero = {0.f, 0.f};
            Pair run[kPerLane];
            bool weighs[kPerLane];
            int positive = -1;
#pragma unroll
            for (int e = 0; e < kPerLane; ++e) {
                const int w = kPerLane * lane + e;
                const Pair v = w < (int)C * kWarps ? sh.sums[parity][w] : zero;
                weighs[e] = v.hi > 0.f;
                if (weighs[e]) positive = w;
                run[e] = e ? add(run[e - 1], v) : v;
            }
            const Pair incl = scan(run[kPerLane - 1]), total = from_lane(incl, 31);
            int owner = kAgain;
            if (pending && !(total.hi > 0.f)) {  // nothing would be left: the weights stay
                --k;
                pending = false;
            } else if (i < n) {                  // on with the next child
                if (pending) z = total;
                pending = false;
            } else if (!(total.hi > 0.f)) {
                owner = kNone;
                if (writer) report(a.status, PA_ERR_INVALID_ARG);
            } else {
                // the warp whose span the target falls into finds the token; the
                // last one with any weight where the target rounds to the total
                // (the sums before a span are added up in another order than those
                // up to the span before it, so a target on the border of two can
                // seem to lie between them: in no span without weight)
                const Pair target = times(us, 1.f, total);
                Pair before = {__shfl_up_sync(kAll, incl.hi, 1), __shfl_up_sync(kAll, incl.lo, 1)}, from = zero;
                if (lane == 0) before = zero;
                int mine = INT_MAX;
#pragma unroll
                for (int e = kPerLane - 1; e >= 0; --e) {
                    if (weighs[e] && above(add(before, run[e]), target)) {
                        mine = kPerLane * lane + e;
                        from = e ? add(before, run[e > 0 ? e - 1 : 0]) : before;
                    }
                }
                owner = __reduce_min_sync(kAll, mine);
                const bool past = owner == INT_MAX;
                if (past) owner = __reduce_max_sync(kAll, positive);
                if (lane == owner / kPerLane)
                    sh.left = past ? Pair{INFINITY, 0.f} : add(target, {-from.hi, -from.lo});
            }
            if (lane == 0) sh.owner = owner;
        }
        __syncthreads();
        if (sh.owner == kAgain) continue;

        if (writer) {
            a.path_lens[s] = len;
            if (sh.owner == kNone) a.next_tokens[s] = -1;
        }
        if (rank == 0 && warp == 0)
            for (int x = len + lane; x < a.max_q; x += 32) path[x] = -1;
        if (gw == sh.owner) {
            // The first token at which the span's running sum passes what is
            // left: its segment, its 128, itself.  (Rounding can leave the last
            // ones short: then the last one of positive weight.)
            const Pair left = sh.left, zero = {0.f, 0.f};
            __syncwarp();
            const Pair seg = lane * a.segment < a.rows ? sh.seg[warp][lane] : zero, upto = scan(seg);
            unsigned m = __ballot_sync(kAll, seg.hi > 0.f && above(upto, left));
            if (!m) m = 1u << (31 - __clz(__ballot_sync(kAll, seg.hi > 0.f) | 1u));
            const int g = __ffs(m) - 1;
            Pair before = g ? from_lane(upto, g - 1) : zero;
            int in = -1;
            Pair base = before;
#pragma unroll 1
            for (int j = g * a.segment; j < (g + 1) * a.segment; j += kRound) {
                Pair t[kRound];
                round_sums(row, j, t);
#pragma unroll
                for (int b = 0; b < kRound; ++b) t[b] = over_lanes(t[b]);
#pragma unroll
                for (int b = 0; b < kRound; ++b) {
                    // (the first one of any weight even where `base` seems past it)
                    if (t[b].hi > 0.f && (in < 0 || !above(base, left))) {
                        in = j + b;
                        before = base;
                    }
                    base = add(base, t[b]);
                }
            }
            const int x = lo + in * 128 - row.shift;
            float4 qv = make_float4(0.f, 0.f, 0.f, 0.f);
            const float4 pv = edge4(row.p, x, V);
            if (DRAFT && row.k > 0) qv = edge4(row.q, x, V);
            Pair w[4];
            weights(row, x, pv, qv, w);
            int found = INT_MAX, last = -1;
            const Pair incl = scan(add(add(w[0], w[1]), add(w[2], w[3])));
            Pair run = {__shfl_up_sync(kAll, incl.hi, 1), __shfl_up_sync(kAll, incl.lo, 1)};
            run = lane == 0 ? before : add(before, run);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                run = add(run, w[e]);
                if (w[e].hi > 0.f) {
                    last = x + e;
                    if (found == INT_MAX && above(run, left)) found = x + e;
                }
            }
            found = __reduce_min_sync(kAll, found);
            last = __reduce_max_sync(kAll, last);
            if (lane == 0) a.next_tokens[s] = found != INT_MAX ? found : last;
        }
        return;
    }
}

template <typename T, bool DRAFT>
cudaError_t launch_vec(const VerifyParams &a, bool vec, const cudaLaunchConfig_t &cfg) {
    return vec ? cudaLaunchKernelEx(&cfg, verify_draft_kernel<T, DRAFT, true>, a)
               : cudaLaunchKernelEx(&cfg, verify_draft_kernel<T, DRAFT, false>, a);
}
template <typename T>
cudaError_t launch_type(const VerifyParams &a, bool vec, const cudaLaunchConfig_t &cfg) {
    return a.q ? launch_vec<T, true>(a, vec, cfg) : launch_vec<T, false>(a, vec, cfg);
}

}  // namespace

int launch_verify_draft(int32_t *path, int32_t *path_lens, int32_t *next_tokens, const void *target_probs,
                        const void *draft_probs, int32_t dtype, const int32_t *draft_tokens,
                        const int32_t *parents, const int32_t *q_starts, const float *u_accept,
                        const float *u_sample, int32_t n_seqs, int32_t max_q_len, int32_t q_rows,
                        int32_t vocab, int32_t *status, void *stream) {
    const char *who = "pa_verify_draft";
    if (dtype != PA_DTYPE_F16 && dtype != PA_DTYPE_F32 && dtype != PA_DTYPE_BF16)
        return fail(PA_ERR_INVALID_ARG, "%s: dtype %d", who, dtype);
    if (n_seqs < 0 || n_seqs > 65535 || q_rows < 0 || vocab < 1)
        return fail(PA_ERR_INVALID_ARG, "%s: n_seqs=%d (<= 65535), q_rows=%d, vocab=%d", who, n_seqs, q_rows, vocab);
    if (max_q_len < 1 || max_q_len > PA_TREE_MAX_NODES)
        return fail(PA_ERR_INVALID_ARG, "%s: max_q_len=%d (1 to %d)", who, max_q_len, PA_TREE_MAX_NODES);
    if (n_seqs == 0) return PA_OK;
    const int size = dtype == PA_DTYPE_F32 ? 4 : 2;
    auto mis = [](const void *ptr, int n) { return (reinterpret_cast<uintptr_t>(ptr) & (n - 1)) != 0; };
    if (!path || !path_lens || !next_tokens || !target_probs || !draft_tokens || !q_starts || !u_accept || !u_sample)
        return fail(PA_ERR_INVALID_ARG, "%s: NULL pointer", who);
    if (mis(target_probs, size) || mis(draft_probs, size) || mis(path, 4) || mis(path_lens, 4) ||
        mis(next_tokens, 4) || mis(draft_tokens, 4) || mis(parents, 4) || mis(q_starts, 4) ||
        mis(u_accept, 4) || mis(u_sample, 4) || mis(status, 4))
        return fail(PA_ERR_INVALID_ARG, "%s: misaligned pointer", who);
    const bool vec = !mis(target_probs, 4 * size) && !mis(draft_probs, 4 * size);
    // Clusters of up to 8 CTAs, each CTA with 2048 tokens or more, and no more
    // CTAs than the GPU holds at once: a sequence's fixed part (loads that wait
    // on one another, barriers) is as long as its share of a row then.  (256 chains of
    // 50272 tokens: clusters of 2, this rule's, 30 us, of 8 43 us, single CTAs 33 us; 64
    // trees: of 8 62 us, single CTAs 242 us; one chain: of 8 9 us, a single CTA 17 us.)
    int sms = 152, dev = 0, C = 1;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    while (C < kMaxCluster && (int64_t)C * 2048 < vocab && (int64_t)n_seqs * C * 2 <= (int64_t)sms * kPerSm) C *= 2;
    VerifyParams a{};
    a.path = path;
    a.path_lens = path_lens;
    a.next_tokens = next_tokens;
    a.p = target_probs;
    a.q = draft_probs;
    a.tokens = draft_tokens;
    a.parents = parents;
    a.q_starts = q_starts;
    a.u_accept = u_accept;
    a.u_sample = u_sample;
    a.max_q = max_q_len;
    a.q_rows = q_rows;
    a.vocab = vocab;
    const int64_t warps = (int64_t)C * kWarps;
    if (vocab > INT32_MAX / 2) return fail(PA_ERR_INVALID_ARG, "%s: vocab=%d too large", who, vocab);
    a.rows = (int32_t)((((int64_t)vocab + 3 + warps - 1) / warps + 127) / 128);   // (3: up to a row's vector boundary)
    a.segment = ((a.rows + kSegments - 1) / kSegments + kRound - 1) / kRound * kRound;
    a.status = status;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)C, (unsigned)n_seqs, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)C;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = dtype == PA_DTYPE_F32   ? launch_type<float>(a, vec, cfg)
                          : dtype == PA_DTYPE_F16 ? launch_type<__half>(a, vec, cfg)
                                                  : launch_type<__nv_bfloat16>(a, vec, cfg);
    if (e != cudaSuccess) return fail(PA_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
    return PA_OK;
}

}  // namespace pagedkv
