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
// tokens.  All weights are therefore pairs of fp32 (value + error term, 2^-48),
// added with error-free transformations; only the joining of the warps' sums
// and the tests of single tokens are in fp64, in one warp (this GPU does two
// fp64 operations a clock and SM: with sums joined in fp64 by every thread
// 256 rows of 50 k tokens took 342 us, this way ...).  No atomics: the result depends
// only on the inputs.
//
// What bounds it: the rows it has to read (one target row, and one draft row
// once something is rejected, 4 V bytes each) for a large batch; the chain of
// dependent loads for a small one.  Per sequence one cluster of up to 8 CTAs
// shares a row: first the scalars p_parent(x), q_parent(x), u of all nodes are
// gathered at once, so the walk itself touches no memory (a chain never needs
// a pass over a row before the last one), then each pass over a row is split
// evenly over the cluster's warps, contiguous spans in order of index, and the
// warps' sums are exchanged through distributed shared memory.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <climits>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pagedkv {

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kMaxCluster = 8;
static_assert(kMaxCluster * kWarps <= 64, "a lane of warp 0 takes two warps' sums");
constexpr int kNodes = PA_TREE_MAX_NODES;

struct VerifyParams {
    int32_t *path, *path_lens, *next_tokens;
    const void *p, *q;
    const int32_t *tokens, *parents, *q_starts;
    const float *u_accept, *u_sample;
    int32_t max_q, q_rows, vocab, span;   // span: elements a warp owns
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
__device__ __forceinline__ float clean(float x) { return x > 0.f && x <= FLT_MAX ? x : 0.f; }

__device__ __forceinline__ float value(const float *p) { return clean(__ldg(p)); }
__device__ __forceinline__ float value(const __half *p) { return clean(__half2float(__ldg(p))); }
__device__ __forceinline__ float value(const __nv_bfloat16 *p) { return clean(__bfloat162float(__ldg(p))); }

// VEC consecutive values (one load when VEC > 1).
template <typename T, int VEC>
__device__ __forceinline__ void values(const T *p, float (&v)[VEC]) {
    if constexpr (VEC == 1) {
        v[0] = value(p);
    } else if constexpr (sizeof(T) == 4) {
        const float4 x = __ldg(reinterpret_cast<const float4 *>(p));
        v[0] = clean(x.x);
        v[1] = clean(x.y);
        v[2] = clean(x.z);
        v[3] = clean(x.w);
    } else {
        const uint2 x = __ldg(reinterpret_cast<const uint2 *>(p));
        T h[4];
        *reinterpret_cast<uint2 *>(h) = x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (std::is_same<T, __half>::value) v[i] = clean(__half2float(h[i]));
            else v[i] = clean(__bfloat162float(h[i]));
        }
    }
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
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
__device__ __forceinline__ double load_cluster(const Pair *local, uint32_t rank) {
    uint32_t a;
    Pair v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(local)), "r"(rank));
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.hi), "=f"(v.lo) : "r"(a) : "memory");
    return (double)v.hi + (double)v.lo;
}

struct Shared {
    float pu[kNodes], qu[kNodes], u[kNodes];   // of a node: its token's weight in its parent's rows
    int32_t up[kNodes], tok[kNodes];
    float zh[kNodes], zl[kNodes];              // Z before each rejection at the current node
    int32_t out[kNodes];                       // the tokens rejected there
    Pair wsum[2][kWarps];                      // this CTA's warps' sums, by parity of the pass
    int32_t cur, k;                            // the row to add up: its node, rejections there
    int32_t owner;                             // the warp that finds the next token, or:
    Pair left;                                 // of the target, within the owner's span
};
enum { kAgain = -1, kNone = -2 };

template <typename T, bool DRAFT, int VEC>
__global__ void __launch_bounds__(kThreads) verify_draft_kernel(const VerifyParams a) {
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

    const int gw = (int)rank * kWarps + warp;          // this warp's place in the row
    const int lo = (int)min((long long)V, (long long)gw * a.span);
    const int hi = (int)min((long long)V, (long long)lo + a.span);

    // The weights of VEC tokens from i on, after k rejections at node v.
    auto weights = [&](int v, int k, int i, Pair (&w)[VEC]) {
        float pv[VEC];
        values<T, VEC>(P + (size_t)v * V + i, pv);
#pragma unroll
        for (int e = 0; e < VEC; ++e) w[e] = {pv[e], 0.f};
        if (k > 0) {
            if (DRAFT) {
                float qv[VEC];
                values<T, VEC>(Q + (size_t)v * V + i, qv);
                for (int r = 0; r < k; ++r) {
                    const float zh = sh.zh[r], zl = sh.zl[r];
#pragma unroll
                    for (int e = 0; e < VEC; ++e) w[e] = reject(w[e], qv[e], zh, zl);
                }
            } else {
                for (int r = 0; r < k; ++r) {
                    const int x = sh.out[r] - i;
#pragma unroll
                    for (int e = 0; e < VEC; ++e)
                        if (x == e) w[e] = {0.f, 0.f};
                }
            }
        }
    };

    // Warp 0 of every CTA walks (alike, in fp64: a few operations a node; the
    // other warps would only queue for the fp64 unit) up to where the sum of a
    // row is needed, all warps add up that row, warp 0 goes on.
    int i = 1, cur = 0, k = 0, len = 1;
    bool pending = false;       // the last rejection's sum is not known yet
    double z = 1.;
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
                // (u q is exact in fp64)
                if ((double)sh.u[i] * (double)qx * z < (double)w.hi + (double)w.lo) {
                    cur = i;
                    k = 0;
                    z = 1.;
                    if (writer) path[len] = i;
                    ++len;
                } else {
                    __syncwarp();       // every lane has read the list's earlier entries
                    if (lane == 0) {
                        sh.zh[k] = (float)z;
                        sh.zl[k] = (float)(z - (double)(float)z);
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
        const int v = sh.cur, kk = sh.k;
        Pair acc = {0.f, 0.f};
#pragma unroll 4
        for (int x = lo + lane * VEC; x < hi; x += 32 * VEC) {
            Pair w[VEC];
            weights(v, kk, x, w);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const Pair t = two_sum(acc.hi, w[e].hi);
                acc = {t.hi, __fadd_rn(acc.lo, __fadd_rn(t.lo, w[e].lo))};
            }
        }
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1)
            acc = add(acc, {__shfl_xor_sync(kAll, acc.hi, off), __shfl_xor_sync(kAll, acc.lo, off)});
        if (lane == 0) sh.wsum[parity][warp] = acc;
        cluster_sync();
        if (warp == 0) {
            // lane l: the sums of warps 2l and 2l + 1 of the row
            double w0 = 0., w1 = 0.;
            const int g0 = 2 * lane, g1 = g0 + 1, all = (int)C * kWarps;
            if (g0 < all) w0 = load_cluster(&sh.wsum[parity][g0 % kWarps], (uint32_t)(g0 / kWarps));
            if (g1 < all) w1 = load_cluster(&sh.wsum[parity][g1 % kWarps], (uint32_t)(g1 / kWarps));
            double incl = w0 + w1;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const double y = __shfl_up_sync(kAll, incl, off);
                if (lane >= off) incl += y;
            }
            const double total = __shfl_sync(kAll, incl, 31);
            int owner = kAgain;
            if (pending && !(total > 0.)) {      // nothing would be left: the weights stay
                --k;
                pending = false;
            } else if (i < n) {                  // on with the next child
                if (pending) z = total;
                pending = false;
            } else if (!(total > 0.)) {
                owner = kNone;
                if (writer) report(a.status, PA_ERR_INVALID_ARG);
            } else {
                // the warp whose span the target falls into finds the token
                const double target = (double)us * total, before = incl - (w0 + w1);
                const unsigned m0 = __ballot_sync(kAll, before + w0 > target);
                const unsigned m1 = __ballot_sync(kAll, incl > target);
                const unsigned p0 = __ballot_sync(kAll, w0 > 0.), p1 = __ballot_sync(kAll, w1 > 0.);
                const int f0 = m0 ? 2 * (__ffs(m0) - 1) : INT_MAX, f1 = m1 ? 2 * (__ffs(m1) - 1) + 1 : INT_MAX;
                owner = min(f0, f1);
                const bool past = owner == INT_MAX;   // the target rounds to the total or more
                if (past)
                    owner = max(p0 ? 2 * (31 - __clz(p0)) : 0, p1 ? 2 * (31 - __clz(p1)) + 1 : 0);
                if (lane == owner / 2) {
                    const double left = past ? INFINITY : target - (owner & 1 ? before + w0 : before);
                    sh.left = {(float)left, past ? 0.f : (float)(left - (double)(float)left)};
                }
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
            // the first token at which the span's running sum passes what is left
            const Pair left = sh.left;
            int found = INT_MAX, positive = -1;
            Pair base = {0.f, 0.f};
            for (int x0 = lo; x0 < hi && found == INT_MAX; x0 += 32 * VEC) {
                const int x = x0 + lane * VEC;
                Pair w[VEC], run[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) w[e] = {0.f, 0.f};
                if (x < hi) weights(v, kk, x, w);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    run[e] = e ? add(run[e - 1], w[e]) : w[e];
                    if (w[e].hi > 0.f) positive = x + e;
                }
                Pair incl = run[VEC - 1];
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const Pair y = {__shfl_up_sync(kAll, incl.hi, off), __shfl_up_sync(kAll, incl.lo, off)};
                    if (lane >= off) incl = add(incl, y);
                }
                Pair excl = {__shfl_up_sync(kAll, incl.hi, 1), __shfl_up_sync(kAll, incl.lo, 1)};
                excl = lane == 0 ? base : add(base, excl);
#pragma unroll
                for (int e = VEC - 1; e >= 0; --e)
                    if (w[e].hi > 0.f && above(add(excl, run[e]), left)) found = x + e;
                base = add(base, {__shfl_sync(kAll, incl.hi, 31), __shfl_sync(kAll, incl.lo, 31)});
                found = __reduce_min_sync(kAll, found);
            }
            positive = __reduce_max_sync(kAll, positive);
            // (rounding can leave the last element short of the warp's sum)
            if (lane == 0) a.next_tokens[s] = found != INT_MAX ? found : positive;
        }
        break;
    }
    cluster_sync();   // no CTA leaves while another may read its sums
}

template <typename T, bool DRAFT>
cudaError_t launch_vec(const VerifyParams &a, bool vec, const cudaLaunchConfig_t &cfg) {
    return vec ? cudaLaunchKernelEx(&cfg, verify_draft_kernel<T, DRAFT, 4>, a)
               : cudaLaunchKernelEx(&cfg, verify_draft_kernel<T, DRAFT, 1>, a);
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
    // every row starts on a vector boundary
    const bool vec = vocab % 4 == 0 && !mis(target_probs, 4 * size) && !mis(draft_probs, 4 * size);
    const int step = vec ? 128 : 32;
    // a CTA for every 2048 tokens, up to a cluster of 8
    int C = 1;
    while (C < kMaxCluster && (int64_t)C * 2048 < vocab) C *= 2;
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
    const int64_t span = ((vocab + warps - 1) / warps + step - 1) / step * step;
    if (span > INT32_MAX / 2) return fail(PA_ERR_INVALID_ARG, "%s: vocab=%d too large", who, vocab);
    a.span = (int32_t)span;
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
