// Attention of several drafted tokens per sequence over the paged cache
// (pa_tree_attention), and decode attention that also returns what weight
// each cached position received (pa_decode_attention_weights).
//
// Mathematics.  The n_s query rows of sequence s are its last n_s positions
// (nodes of a draft tree, node i at position ctx_s - n_s + i).  Node i sees
// every position before the nodes, itself, and its ancestors:
//     x_ip = scale * q_i . k_p   (p visible, else -inf)
//     o_i  = sum_p 2^(x'_ip - m_i) v_p / l_i,   x' = x log2 e,
//     m_i = max_p x'_ip, l_i = sum_p 2^(x'_ip - m_i)
// kept online over the positions and, for a context cut into parts, joined
// by the parts' (m, l, sum).  The weight of position p is 2^(x'_p - m) / l.
//
// What bounds it: every key and value is read once for all n rows of a
// sequence, 4 D bytes against 4 n D operations a position, so up to the 64
// rows allowed the bytes bound it (64 flops a byte against 286 the tensor
// cores could do).  The products run on the tensor cores all the same (a
// row's dot products on the plain pipes would be 16 times slower than the
// bytes at n = 16): m16n8k16 products with queries in M.
//
// Layout.  One persistent CTA an SM slot: a producer warp streams the unit's
// blocks by TMA (GH adjacent heads of a block are one box, 128-byte swizzled)
// into a ring; consumer warp (g, mw) owns head g and query rows
// [16 mw, 16 mw + 16) for the whole unit, so nothing is combined between
// warps.  In the swizzled layout every fragment comes by plain 16-byte shared
// loads without bank conflicts:
//   * keys (B of S = Q K^T): lane (g, c) takes the 8 dims [16c + 8u, +8) of
//     token g; a product's k index is any order of the dims that Q shares;
//   * values (B of O = P V): lane (g, c) takes 8 dims of its four tokens and
//     interleaves them pairwise (byte permutes), so column g of n-tile e is
//     dim 8g + e: the accumulators of a lane are 16 consecutive dims.
// Scores stay in registers from the first product to the second: the
// accumulator layout of S is the A layout of P.
//
// Rounding: products of fp16 values are exact in the fp32 accumulators; the
// running maximum is exact, so P is in [0, 1] and enters the second product
// as fp16 (half a unit in 2^-11 of each weight, like the fp16 output's own
// rounding); sums and the join of parts are fp32.
//
// Work plan (the same in every CTA): sequences longer than P blocks are cut
// into even parts, P such that the units fill the slots once (few sequences)
// or about twice over (many); cut sequences first, then the others by size.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <mutex>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pagedkv {

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kHeaderBytes = 256;    // workspace head: unit ticket, number of cut sequences
constexpr int kUnitSlots = 3;        // units a CTA has open
constexpr int kMinPartTokens = 64;

struct TreeParams {
    __half *out;
    const __half *q;
    const int32_t *block_tables;
    const int32_t *ctx_lens;
    const int32_t *q_starts;   // NULL (weights form): one query a sequence
    const int32_t *parents;    // NULL: a chain
    int32_t *header;           // [0] unit tickets, [1] cut sequences
    int4 *cut;                 // [cap] cut sequences: s, first part, parts, rows
    float2 *ws_ml;             // [cap][H][NR] (max, sum) of a part's rows
    float *ws_acc;             // [cap][H][NR][D] unnormalised output
    // weights form
    int2 *plan;                // [S] first part (cut) and parts of each sequence
    float2 *ml_one;            // [S][H] (max, sum) of an uncut sequence
    float *scores;             // [S][H][score_stride] scores in log2 units
    int32_t *status;
    int32_t n_seqs, num_heads, num_blocks, max_blocks, bshift, max_q, q_rows, cap;
    int32_t stages, stage_tokens;
    int32_t score_stride, weight_len;
    float qscale;              // scale * log2(e)
};

struct TreeMaps {
    CUtensorMap k, v;
};

// ---------------------------------------------------------------- helpers

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// d += a b: 16 x 16 fp16 (row) times 16 x 8 fp16 (column), fp32 accumulators.
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr));
    return v;
}

__device__ __forceinline__ uint32_t word_of(const uint4 &v, int i) {
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, int c3, uint32_t bar,
                                            uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
        "[%0], [%1, {%2, %2, %2, %3}], [%4], %5;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(c3), "r"(bar), "l"(policy)
        : "memory");
}

// Rows and length of sequence s; 0 rows: nothing to do (or refused, reported).
struct SeqRows {
    int n, row0, ctx;
};
template <bool SCORES>
__device__ __forceinline__ SeqRows rows_of(const TreeParams &p, int s, bool tell) {
    SeqRows r;
    r.ctx = p.ctx_lens[s];
    if (SCORES) {
        r.row0 = s;
        r.n = r.ctx > 0 ? 1 : 0;
        if (r.ctx > p.weight_len) {
            if (tell) report(p.status, PA_ERR_INVALID_ARG);
            r.n = 0;
        }
    } else {
        const int a = p.q_starts[s], b = p.q_starts[s + 1];
        r.row0 = a;
        r.n = b - a;
        if (a < 0 || b < a || b > p.q_rows || b - a > p.max_q || b - a > max(r.ctx, 0)) {
            if (tell) report(p.status, PA_ERR_INVALID_ARG);
            r.n = 0;
        }
    }
    if (r.n > 0 && r.ctx > ((int64_t)p.max_blocks << p.bshift)) {
        if (tell) report(p.status, PA_ERR_BAD_BLOCK);
        r.n = 0;
    }
    return r;
}

__device__ __forceinline__ int warp_incl_scan(int v, int lane) {
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(kAll, v, off);
        if (lane >= off) v += y;
    }
    return v;
}

// ------------------------------------------------------------ main kernel

template <int D, int GH, int MW>
struct TreeCfg {
    static constexpr int NP = D / 64;                       // 64-column panels of a row
    static constexpr int NR = 16 * MW;                      // query rows, padded
    static constexpr int WARPS = GH * MW;                   // consumer warps
    static constexpr int THREADS = (WARPS + 1) * 32;
    static constexpr int PER_SM = WARPS >= 8 ? 1 : WARPS >= 4 ? 2 : WARPS >= 2 ? 3 : 4;
    static constexpr int MAX_STAGES = 16;
    // fixed shared memory before the ring (1024-byte aligned)
    static constexpr int SDESC = 0;                                   // int4 per stage
    static constexpr int BARS = SDESC + MAX_STAGES * 16;              // full, empty, unit empty
    static constexpr int VARS = BARS + (2 * MAX_STAGES + kUnitSlots) * 8 + 8;
    static constexpr int UNITS = (VARS + 16 + 15) / 16 * 16;          // 64 B per slot
    static constexpr int MASKS = UNITS + kUnitSlots * 64;             // 64 x u64 per slot
    static constexpr int PLAN = MASKS + kUnitSlots * 64 * 8;          // pre[S+1], len[S], order[S]
    static int plan_bytes(int S) { return (S + 1) * 4 + S * 4 + (S + 1) / 2 * 4; }
    static int bytes(int S, int ring) { return PLAN + plan_bytes(S) + 1024 + ring; }
};

enum { FLAG_FIRST = 1, FLAG_LAST = 2, FLAG_END = 4 };

template <int D, int GH, int MW, bool SCORES>
__global__ void __launch_bounds__((GH * MW + 1) * 32, (TreeCfg<D, GH, MW>::PER_SM))
    tree_attention_kernel(const TreeParams p, const __grid_constant__ TreeMaps maps) {
    using Cfg = TreeCfg<D, GH, MW>;
    constexpr int NP = Cfg::NP, NR = Cfg::NR;
    const uint32_t HALF = (uint32_t)GH * p.stage_tokens * D * 2, STAGE = 2 * HALF;   // keys, then values
    extern __shared__ __align__(16) uint8_t smem[];
    int4 *sdesc = reinterpret_cast<int4 *>(smem + Cfg::SDESC);
    const uint32_t bar_full = smem_addr(smem + Cfg::BARS);
    const uint32_t bar_empty = bar_full + Cfg::MAX_STAGES * 8;
    const uint32_t bar_unit = bar_empty + Cfg::MAX_STAGES * 8;
    int32_t *vars = reinterpret_cast<int32_t *>(smem + Cfg::VARS);   // ordered, cut sequences
    int32_t *units = reinterpret_cast<int32_t *>(smem + Cfg::UNITS);
    uint64_t *masks = reinterpret_cast<uint64_t *>(smem + Cfg::MASKS);
    const int S = p.n_seqs, H = p.num_heads, HG = H / GH;
    int32_t *pre = reinterpret_cast<int32_t *>(smem + Cfg::PLAN);    // parts before the i-th in order
    int32_t *len = pre + S + 1;                                      // blocks of sequence s
    uint16_t *order = reinterpret_cast<uint16_t *>(len + S);
    const uint32_t ring = (smem_addr(order + S) + 1023u) & ~1023u;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int stages = p.stages, bshift = p.bshift, B = 1 << bshift;

    // ---- the plan
    if (tid == 0) {
        for (int i = 0; i < stages; ++i) {
            mbar_init(bar_full + 8 * i, 1);
            mbar_init(bar_empty + 8 * i, Cfg::WARPS);
        }
        for (int i = 0; i < kUnitSlots; ++i) mbar_init(bar_unit + 8 * i, Cfg::WARPS);
        fence_barrier_init();
    }
    for (int s = tid; s < S; s += Cfg::THREADS) {
        const SeqRows r = rows_of<SCORES>(p, s, blockIdx.x == 0);
        len[s] = r.n > 0 ? (r.ctx + B - 1) >> bshift : 0;
    }
    __syncthreads();
    if (warp == 0) {
        const int per = (S + 31) / 32, lo_s = min(S, lane * per), hi_s = min(S, lo_s + per);
        long long total = 0;
        int some = 0, longest = 0;
        for (int s = lo_s; s < hi_s; ++s) {
            total += len[s];
            some += len[s] > 0;
            longest = max(longest, len[s]);
        }
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) {
            total += __shfl_xor_sync(kAll, total, off);
            some += __shfl_xor_sync(kAll, some, off);
            longest = max(longest, __shfl_xor_sync(kAll, longest, off));
        }
        const int slots = gridDim.x;
        const int share = (int)((total * HG + slots - 1) / slots);   // blocks a slot has to read
        int P = max(1, kMinPartTokens >> bshift);
        if ((long long)some * HG < slots) {
            // few sequences: the smallest part size whose units fit the slots
            // at once; every lane tries one size of a grid
            int lo = max(P, share), hi = max(lo, longest);
            while (lo < hi) {
                const int step = (hi - lo + 30) / 31, cand = min(hi, lo + lane * step);
                long long units_n = 0;
                for (int s = 0; s < S; ++s) units_n += (len[s] + cand - 1) / cand;
                const unsigned fits = __ballot_sync(kAll, units_n * HG <= slots || cand == hi);
                const int f = __ffs(fits) - 1;   // (lane 31 reaches hi)
                const int nhi = min(hi, lo + f * step);
                lo = f == 0 ? nhi : min(hi, lo + (f - 1) * step + 1);
                hi = nhi;
            }
            P = hi;
        } else {
            P = max(P, (share + 1) / 2);
        }
        int ncls[5], cut_parts;
        while (true) {   // (the cap is never passed: parts of at least half a share each)
            cut_parts = 0;
#pragma unroll
            for (int k = 0; k < 5; ++k) ncls[k] = 0;
            for (int s = lo_s; s < hi_s; ++s) {
                const int l = len[s];
                if (l > P) cut_parts += (l + P - 1) / P;
                const int cls = l > P ? 0 : 4 * (long long)l > 3ll * P ? 1 : 2ll * l > P ? 2 : 4ll * l > P ? 3 : 4;
#pragma unroll
                for (int k = 0; k < 5; ++k) ncls[k] += l > 0 && cls == k;
            }
            if (__reduce_add_sync(kAll, cut_parts) <= p.cap) break;
            P *= 2;
        }
        int base[5], start = 0, n_cut = 0;
#pragma unroll
        for (int k = 0; k < 5; ++k) {
            const int incl = warp_incl_scan(ncls[k], lane);
            base[k] = start + incl - ncls[k];
            start += __shfl_sync(kAll, incl, 31);
            if (k == 0) n_cut = start;
        }
        for (int s = lo_s; s < hi_s; ++s) {
            const int l = len[s];
            if (l == 0) continue;
            const int cls = l > P ? 0 : 4 * (long long)l > 3ll * P ? 1 : 2ll * l > P ? 2 : 4ll * l > P ? 3 : 4;
            int r = 0;
#pragma unroll
            for (int k = 0; k < 5; ++k)
                if (cls == k) r = base[k]++;
            order[r] = (uint16_t)s;
        }
        __syncwarp();
        const int n_ord = start, per2 = (n_ord + 31) / 32;
        const int lo_i = min(n_ord, lane * per2), hi_i = min(n_ord, lo_i + per2);
        int mine = 0;
        for (int i = lo_i; i < hi_i; ++i) mine += (len[order[i]] + P - 1) / P;
        int run = warp_incl_scan(mine, lane) - mine;
        for (int i = lo_i; i < hi_i; ++i) {
            pre[i] = run;
            run += (len[order[i]] + P - 1) / P;
        }
        if (hi_i == n_ord) pre[n_ord] = run;   // (lanes past the end hold the total too)
        if (lane == 0) {
            vars[0] = n_ord;
            vars[1] = n_cut;
        }
    }
    __syncthreads();
    const int n_ord = vars[0], n_units = pre[n_ord] * HG;
    if (blockIdx.x == 0) {   // for the kernels that join the parts
        const int n_cut = vars[1];
        if (tid == 0) p.header[1] = n_cut;
        for (int i = tid; i < n_cut; i += Cfg::THREADS) {
            const int s = order[i];
            const SeqRows r = rows_of<SCORES>(p, s, false);
            p.cut[i] = make_int4(s, pre[i], pre[i + 1] - pre[i], r.n);
        }
        if (SCORES) {
            for (int s = tid; s < S; s += Cfg::THREADS)
                if (len[s] == 0) p.plan[s] = make_int2(0, 0);
            for (int i = tid; i < n_ord; i += Cfg::THREADS)
                p.plan[order[i]] = make_int2(pre[i], pre[i + 1] - pre[i]);
        }
    }

    if (warp == Cfg::WARPS) {
        // ================================================ producer warp
        const uint64_t policy = l2_evict_first_policy();
        const int bps = p.stage_tokens >> bshift;                    // blocks a stage
        const uint32_t blk_bytes = (uint32_t)GH * D * 2u << bshift;
        const int groups_per_run = GH << bshift >> 3;    // 8-row groups of a box
        const int groups_per_block = (H << bshift) >> 3;
        bool ok = true;
        int st = 0;
        uint32_t use = 0;        // times the ring has wrapped
        int k_unit = 0, issued = 0;

        struct Pending {
            int ticket, s, h0, gp, parts, b0, nb, tbl;
            SeqRows r;
        };
        // Names the unit of a ticket and starts the loads it needs.
        auto prepare = [&](int ticket) {
            Pending u;
            u.ticket = ticket;
            u.s = u.h0 = u.gp = u.parts = u.b0 = u.nb = 0;
            u.tbl = -1;
            u.r.n = u.r.row0 = u.r.ctx = 0;
            if (ticket >= n_units) return u;
            u.gp = ticket / HG;
            u.h0 = (ticket - u.gp * HG) * GH;
            int lo = 0, hi = n_ord - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (pre[mid] <= u.gp) lo = mid; else hi = mid - 1;
            }
            u.s = order[lo];
            u.parts = pre[lo + 1] - pre[lo];
            const int part = u.gp - pre[lo], l = len[u.s];
            u.b0 = (int)((long long)part * l / u.parts);
            u.nb = (int)((long long)(part + 1) * l / u.parts) - u.b0;
            if (lane < u.nb) u.tbl = p.block_tables[(size_t)u.s * p.max_blocks + u.b0 + lane];
            u.r = rows_of<SCORES>(p, u.s, false);
            return u;
        };

        int t_next = 0;
        Pending cur = prepare(blockIdx.x);
        if (lane == 0) t_next = (int)gridDim.x + atomicAdd(p.header, 1);
        while (ok && cur.ticket < n_units) {
            const int tn = __shfl_sync(kAll, t_next, 0);
            if (lane == 0 && tn < n_units) t_next = (int)gridDim.x + atomicAdd(p.header, 1);
            const Pending nxt = prepare(tn);
            const int slot = k_unit % kUnitSlots, slot_use = k_unit / kUnitSlots;
            if (slot_use > 0 && !mbar_wait_bounded(bar_unit + 8 * slot, (uint32_t)(slot_use - 1) & 1u,
                                                   p.status, true)) {
                report(p.status, PA_ERR_TIMEOUT);
                ok = false;
            }
            ok = __all_sync(kAll, ok);
            if (!ok) break;
            int32_t *u = units + slot * 16;
            const int base = cur.r.ctx - cur.r.n;
            if (lane == 0) {
                u[0] = cur.s;
                u[1] = cur.h0;
                u[2] = cur.gp;
                u[3] = cur.parts;
                u[4] = cur.r.ctx;
                u[5] = base;
                u[6] = cur.r.n;
                u[7] = cur.r.row0;
            }
            if ((cur.b0 + cur.nb) << bshift > base) {
                // which nodes each node sees: its ancestors and itself, by
                // doubling the parent links
                uint64_t m[2];
                int up[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int i = lane + 32 * e;
                    up[e] = i - 1;
                    if (!SCORES && p.parents && i < cur.r.n) {
                        up[e] = p.parents[cur.r.row0 + i];
                        if (up[e] < -1 || up[e] >= i) {
                            report(p.status, PA_ERR_INVALID_ARG);
                            up[e] = -1;
                        }
                    }
                    m[e] = 1ull << i;
                }
                if (SCORES || !p.parents) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) m[e] |= (1ull << (lane + 32 * e)) - 1;
                } else {
                    for (int k = 1; k < cur.r.n; k <<= 1) {
                        uint64_t add[2];
                        int far[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int t = up[e] & 31;
                            const bool second = up[e] >= 32;
                            const uint64_t a = __shfl_sync(kAll, m[0], t), b = __shfl_sync(kAll, m[1], t);
                            const int fa = __shfl_sync(kAll, up[0], t), fb = __shfl_sync(kAll, up[1], t);
                            add[e] = up[e] < 0 ? 0 : (second ? b : a);
                            far[e] = up[e] < 0 ? -1 : (second ? fb : fa);
                        }
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            m[e] |= add[e];
                            up[e] = far[e];
                        }
                    }
                }
                masks[slot * 64 + lane] = m[0];
                masks[slot * 64 + 32 + lane] = m[1];
            }
            __syncwarp();
            const int32_t *trow = p.block_tables + (size_t)cur.s * p.max_blocks + cur.b0;
            int tbl = cur.tbl;
            for (int b = 0; b < cur.nb; b += bps) {
                if (b > 0 && (b & 31) == 0) tbl = b + lane < cur.nb ? trow[b + lane] : -1;
                const int here = min(bps, cur.nb - b);
                // one lane a block of the stage
                const int phys = __shfl_sync(kAll, tbl, (b & 31) + (lane < here ? lane : 0));
                const bool good = lane < here && phys >= 0 && phys < p.num_blocks;
                const unsigned goods = __ballot_sync(kAll, good);
                if (lane < here && !good) report(p.status, PA_ERR_BAD_BLOCK);
                const uint32_t full = bar_full + 8 * st;
                if (use > 0 && !mbar_wait_bounded(bar_empty + 8 * st, (use - 1) & 1u, p.status, true)) {
                    report(p.status, PA_ERR_TIMEOUT);
                    ok = false;
                }
                ok = __all_sync(kAll, ok);
                if (!ok) break;
                if (lane == 0) {
                    const int tok0 = (cur.b0 + b) << bshift;
                    const int nv = min(here << bshift, cur.r.ctx - tok0);
                    const int flags = (b == 0 ? FLAG_FIRST : 0) | (b + bps >= cur.nb ? FLAG_LAST : 0);
                    sdesc[st] = make_int4(slot, flags, tok0, nv);
                    const uint32_t bytes = (uint32_t)__popc(goods) * 2u * blk_bytes;
                    if (bytes) mbar_arrive_expect_tx(full, bytes);
                    else mbar_arrive(full);
                }
                __syncwarp();
                if (good) {
                    const uint32_t dst = ring + st * STAGE + lane * blk_bytes;
                    const int grp = phys * groups_per_block + (cur.h0 / GH) * groups_per_run;
                    tma_load_4d(dst, &maps.k, grp, full, policy);
                    tma_load_4d(dst + HALF, &maps.v, grp, full, policy);
                }
                ++issued;
                if (++st == stages) {
                    st = 0;
                    ++use;
                }
            }
            ++k_unit;
            cur = nxt;
        }
        if (ok) {   // the end of the stream
            if (use > 0 && !mbar_wait_bounded(bar_empty + 8 * st, (use - 1) & 1u, p.status, true)) {
                report(p.status, PA_ERR_TIMEOUT);
                ok = false;
            }
            ok = __all_sync(kAll, ok);
            if (ok && lane == 0) {
                sdesc[st] = make_int4(0, FLAG_END, 0, 0);
                mbar_arrive(bar_full + 8 * st);
            }
        }
        if (!ok) {   // every issued copy lands before the CTA can exit
            for (int k = max(0, issued - stages); k < issued; ++k)
                mbar_wait_bounded(bar_full + 8 * (k % stages), (uint32_t)(k / stages) & 1u, p.status, false);
        }
        return;
    }

    // ==================================================== consumer warps
    const int hw = warp / MW, mw = warp - hw * MW;       // head of the group, row tile
    const int g = lane >> 2, c = lane & 3;
    uint4 ql[NP][2], qh[NP][2];                          // rows g and g + 8: dims 64 pn + 16c + 8u ..
    float o[NP][8][4];
    float m0 = 0.f, m1 = 0.f, l0 = 0.f, l1 = 0.f;
    int u_s = 0, u_h = 0, u_gp = 0, u_parts = 0, u_base = 0, u_n = 0, u_row0 = 0;
    const uint32_t koff0 = (uint32_t)g * 128u + (uint32_t)((2 * c) ^ g) * 16u;   // u = 0; u = 1: ^ 16
    const uint32_t voff0 = (uint32_t)(2 * c) * 128u + (uint32_t)(g ^ (2 * c)) * 16u;
    const uint32_t voff1 = (uint32_t)(2 * c + 1) * 128u + (uint32_t)(g ^ (2 * c + 1)) * 16u;
    const uint32_t blk_bytes = (uint32_t)GH * D * 2u << bshift;
    const int r0 = mw * 16 + g;                          // this lane's rows: r0, r0 + 8

    int st = 0;
    uint32_t use = 0;
    while (true) {
        if (!mbar_wait_bounded(bar_full + 8 * st, use & 1u, p.status, true)) {
            report(p.status, PA_ERR_TIMEOUT);
            return;
        }
        const int4 d = sdesc[st];
        if (d.y & FLAG_END) return;
        if (d.y & FLAG_FIRST) {
            const int32_t *u = units + d.x * 16;
            u_s = u[0];
            u_h = u[1] + hw;
            u_gp = u[2];
            u_parts = u[3];
            u_base = u[5];
            u_n = u[6];
            u_row0 = u[7];
            m0 = m1 = -INFINITY;
            l0 = l1 = 0.f;
#pragma unroll
            for (int pn = 0; pn < NP; ++pn)
#pragma unroll
                for (int e = 0; e < 8; ++e)
#pragma unroll
                    for (int k = 0; k < 4; ++k) o[pn][e][k] = 0.f;
            const uint4 zero = make_uint4(0, 0, 0, 0);
            const uint4 *qr = reinterpret_cast<const uint4 *>(
                p.q + ((size_t)(u_row0 + r0) * H + u_h) * D + 16 * c);
#pragma unroll
            for (int pn = 0; pn < NP; ++pn)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    ql[pn][e] = r0 < u_n ? qr[pn * 8 + e] : zero;
                    qh[pn][e] = r0 + 8 < u_n ? qr[(size_t)8 * H * (D / 8) + pn * 8 + e] : zero;
                }
        }
        if (mw * 16 < u_n) {
            const uint32_t kst = ring + st * STAGE + (uint32_t)hw * ((uint32_t)D * 2u << bshift);
            for (int t0 = 0; t0 < d.w; t0 += 16) {
                // byte offsets of the chunk's two 8-token groups
                uint32_t grp[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int t = t0 + 8 * j;
                    grp[j] = kst + (uint32_t)(t >> bshift) * blk_bytes +
                             (uint32_t)((t & (B - 1)) >> 3) * (NP * 1024u);
                }
                float x[2][4];
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int k = 0; k < 4; ++k) x[j][k] = 0.f;
#pragma unroll
                for (int pn = 0; pn < NP; ++pn)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const uint4 kk = lds128(grp[j] + pn * 1024u + (koff0 ^ (e * 16u)));
                            mma16816(x[j], ql[pn][e].x, qh[pn][e].x, ql[pn][e].y, qh[pn][e].y, kk.x, kk.y);
                            mma16816(x[j], ql[pn][e].z, qh[pn][e].z, ql[pn][e].w, qh[pn][e].w, kk.z, kk.w);
                        }
                const int pos0 = d.z + t0;
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int k = 0; k < 4; ++k) x[j][k] *= p.qscale;
                // drafted positions, or slots past the unit's end (which may hold anything)
                const bool tail = t0 + 16 > d.w;
                if (pos0 + 16 > u_base || tail) {
                    const uint64_t ma = masks[d.x * 64 + r0], mb = masks[d.x * 64 + r0 + 8];
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const int t = t0 + 8 * j + 2 * c + k, node = d.z + t - u_base;
                            const bool out = t >= d.w;
                            if (out || (node >= 0 && !((ma >> node) & 1))) x[j][k] = -INFINITY;
                            if (out || (node >= 0 && !((mb >> node) & 1))) x[j][2 + k] = -INFINITY;
                        }
                }
                if (SCORES && mw == 0 && g == 0) {
                    float *sc = p.scores + ((size_t)u_s * H + u_h) * p.score_stride + pos0 + 2 * c;
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        if (t0 + 8 * j + 2 * c < d.w)   // (the stride covers whole blocks)
                            *reinterpret_cast<float2 *>(sc + 8 * j) = make_float2(x[j][0], x[j][1]);
                }
                float n0 = fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[1][0], x[1][1]));
                float n1 = fmaxf(fmaxf(x[0][2], x[0][3]), fmaxf(x[1][2], x[1][3]));
                n0 = fmaxf(n0, __shfl_xor_sync(kAll, n0, 1));
                n1 = fmaxf(n1, __shfl_xor_sync(kAll, n1, 1));
                n0 = fmaxf(n0, __shfl_xor_sync(kAll, n0, 2));
                n1 = fmaxf(n1, __shfl_xor_sync(kAll, n1, 2));
                if (__any_sync(kAll, n0 > m0 || n1 > m1)) {
                    n0 = fmaxf(n0, m0);
                    n1 = fmaxf(n1, m1);
                    const float a0 = n0 == -INFINITY ? 1.f : ex2(m0 - n0);
                    const float a1 = n1 == -INFINITY ? 1.f : ex2(m1 - n1);
                    m0 = n0;
                    m1 = n1;
                    l0 *= a0;
                    l1 *= a1;
#pragma unroll
                    for (int pn = 0; pn < NP; ++pn)
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            o[pn][e][0] *= a0;
                            o[pn][e][1] *= a0;
                            o[pn][e][2] *= a1;
                            o[pn][e][3] *= a1;
                        }
                }
                // a row that has seen nothing yet keeps m = -inf: its terms are 2^-inf = 0
                const float f0 = m0 == -INFINITY ? 0.f : m0, f1 = m1 == -INFINITY ? 0.f : m1;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    x[j][0] = ex2(x[j][0] - f0);
                    x[j][1] = ex2(x[j][1] - f0);
                    x[j][2] = ex2(x[j][2] - f1);
                    x[j][3] = ex2(x[j][3] - f1);
                    l0 += x[j][0] + x[j][1];
                    l1 += x[j][2] + x[j][3];
                }
                const uint32_t a0 = pack_half2(x[0][0], x[0][1]), a1 = pack_half2(x[0][2], x[0][3]);
                const uint32_t a2 = pack_half2(x[1][0], x[1][1]), a3 = pack_half2(x[1][2], x[1][3]);
#pragma unroll
                for (int pn = 0; pn < NP; ++pn) {
                    uint4 v00 = lds128(grp[0] + HALF + pn * 1024u + voff0);
                    uint4 v01 = lds128(grp[0] + HALF + pn * 1024u + voff1);
                    uint4 v10 = lds128(grp[1] + HALF + pn * 1024u + voff0);
                    uint4 v11 = lds128(grp[1] + HALF + pn * 1024u + voff1);
                    if (tail) {
                        const uint4 zero = make_uint4(0, 0, 0, 0);
                        const int t = t0 + 2 * c;
                        if (t >= d.w) v00 = zero;
                        if (t + 1 >= d.w) v01 = zero;
                        if (t + 8 >= d.w) v10 = zero;
                        if (t + 9 >= d.w) v11 = zero;
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint32_t sel = e & 1 ? 0x7632u : 0x5410u;
                        mma16816(o[pn][e], a0, a1, a2, a3,
                                 __byte_perm(word_of(v00, e >> 1), word_of(v01, e >> 1), sel),
                                 __byte_perm(word_of(v10, e >> 1), word_of(v11, e >> 1), sel));
                    }
                }
            }
        }
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(bar_empty + 8 * st);
            if (d.y & FLAG_LAST) mbar_arrive(bar_unit + 8 * d.x);
        }
        if ((d.y & FLAG_LAST) && mw * 16 < u_n) {
            l0 += __shfl_xor_sync(kAll, l0, 1);
            l1 += __shfl_xor_sync(kAll, l1, 1);
            l0 += __shfl_xor_sync(kAll, l0, 2);
            l1 += __shfl_xor_sync(kAll, l1, 2);
            if (u_parts == 1) {
                const float i0 = 1.f / l0, i1 = 1.f / l1;
#pragma unroll
                for (int e = 0; e < 2; ++e) {            // rows r0, r0 + 8
                    if (r0 + 8 * e >= u_n) continue;
                    const float inv = e ? i1 : i0;
                    uint4 *dst = reinterpret_cast<uint4 *>(
                        p.out + ((size_t)(u_row0 + r0 + 8 * e) * H + u_h) * D + 16 * c);
#pragma unroll
                    for (int pn = 0; pn < NP; ++pn)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            uint32_t w[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                w[i] = pack_half2(o[pn][2 * i][2 * e + k] * inv,
                                                  o[pn][2 * i + 1][2 * e + k] * inv);
                            dst[pn * 8 + k] = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                }
                if (SCORES && lane == 0 && mw == 0)
                    p.ml_one[(size_t)u_s * H + u_h] = make_float2(m0, l0);
            } else {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (r0 + 8 * e >= u_n) continue;
                    const size_t row = ((size_t)u_gp * H + u_h) * NR + r0 + 8 * e;
                    if (c == 0) p.ws_ml[row] = e ? make_float2(m1, l1) : make_float2(m0, l0);
                    float4 *dst = reinterpret_cast<float4 *>(p.ws_acc + row * D + 16 * c);
#pragma unroll
                    for (int pn = 0; pn < NP; ++pn)
#pragma unroll
                        for (int k = 0; k < 2; ++k)
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                dst[pn * 16 + k * 2 + i] =
                                    make_float4(o[pn][4 * i][2 * e + k], o[pn][4 * i + 1][2 * e + k],
                                                o[pn][4 * i + 2][2 * e + k], o[pn][4 * i + 3][2 * e + k]);
                }
            }
        }
        if (++st == stages) {
            st = 0;
            ++use;
        }
    }
}

// -------------------------------------------------------- joining the parts

// One warp per (cut sequence, head, row): m = max m_p, l = sum 2^(m_p - m) l_p,
// o = sum 2^(m_p - m) acc_p / l.
template <int D>
__global__ void __launch_bounds__(256) tree_join_kernel(const TreeParams p, int NR) {
    constexpr int DL = D / 32;
    const int lane = threadIdx.x & 31, H = p.num_heads;
    const long long items = (long long)p.header[1] * H * NR;
    const long long step = (long long)gridDim.x * 8;
    for (long long it = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); it < items; it += step) {
        const int row = (int)(it % NR);
        const long long sh = it / NR;
        const int h = (int)(sh % H);
        const int4 e = p.cut[sh / H];
        if (row >= e.w) continue;
        const size_t at = ((size_t)e.y * H + h) * NR + row, part = (size_t)H * NR;
        float M = -INFINITY;
        for (int q = lane; q < e.z; q += 32) M = fmaxf(M, p.ws_ml[at + q * part].x);
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) M = fmaxf(M, __shfl_xor_sync(kAll, M, off));
        float L = 0.f, o[DL];
#pragma unroll
        for (int k = 0; k < DL; ++k) o[k] = 0.f;
#pragma unroll 4
        for (int q = 0; q < e.z; ++q) {
            const float2 ml = p.ws_ml[at + q * part];
            const float w = ex2(ml.x - M);
            L = fmaf(w, ml.y, L);
#pragma unroll
            for (int k = 0; k < DL; ++k)
                o[k] = fmaf(w, p.ws_acc[(at + q * part) * D + 32 * k + lane], o[k]);
        }
        const float inv = 1.f / L;
        __half *dst = p.out + ((size_t)(p.q_starts[e.x] + row) * H + h) * D;
#pragma unroll
        for (int k = 0; k < DL; ++k) dst[32 * k + lane] = __float2half(o[k] * inv);
    }
}

constexpr int kWeightChunk = 2048;   // positions a block of the weights kernel covers

// One block per (head, sequence, chunk of positions): the sequence's (m, l),
// its output where it was cut, and weights_out = weights_in + 2^(x - m) / l.
template <int D, bool VEC>
__global__ void __launch_bounds__(256)
    decode_weights_kernel(const TreeParams p, int NR, float *w_out, const float *w_in) {
    const int h = blockIdx.x, s = blockIdx.y, H = p.num_heads, tid = threadIdx.x, lane = tid & 31;
    const int ctx = p.ctx_lens[s];
    const int p0 = blockIdx.z * kWeightChunk;
    if (ctx <= 0) {      // nothing cached: the output is 0
        if (p0 == 0 && tid < D) p.out[((size_t)s * H + h) * D + tid] = __float2half(0.f);
        return;
    }
    if (p0 >= ctx) return;
    const int2 plan = p.plan[s];
    if (plan.y == 0) return;                 // refused, reported
    float M, L;
    if (plan.y == 1) {
        const float2 ml = p.ml_one[(size_t)s * H + h];
        M = ml.x;
        L = ml.y;
    } else {
        const size_t at = ((size_t)plan.x * H + h) * NR, part = (size_t)H * NR;
        M = -INFINITY;
        for (int q = lane; q < plan.y; q += 32) M = fmaxf(M, p.ws_ml[at + q * part].x);
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) M = fmaxf(M, __shfl_xor_sync(kAll, M, off));
        L = 0.f;
        for (int q = lane; q < plan.y; q += 32) {
            const float2 ml = p.ws_ml[at + q * part];
            L = fmaf(ex2(ml.x - M), ml.y, L);
        }
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) L += __shfl_xor_sync(kAll, L, off);
        if (p0 == 0 && tid < D) {
            float o = 0.f;
#pragma unroll 4
            for (int q = 0; q < plan.y; ++q)
                o = fmaf(ex2(p.ws_ml[at + q * part].x - M), p.ws_acc[(at + q * part) * D + tid], o);
            p.out[((size_t)s * H + h) * D + tid] = __float2half(o / L);
        }
    }
    const float inv = 1.f / L;
    const size_t row = (size_t)s * H + h;
    const float *x = p.scores + row * p.score_stride;
    float *wo = w_out + row * p.weight_len;
    const float *wi = w_in ? w_in + row * p.weight_len : nullptr;
    const int end = min(ctx, p0 + kWeightChunk);
    if (VEC) {
        for (int i = p0 + tid * 4; i < end; i += 1024) {
            const float4 sx = *reinterpret_cast<const float4 *>(x + i);
            float4 w = wi && i + 4 <= end ? *reinterpret_cast<const float4 *>(wi + i) : make_float4(0, 0, 0, 0);
            if (i + 4 <= end) {
                w.x = fmaf(ex2(sx.x - M), inv, w.x);
                w.y = fmaf(ex2(sx.y - M), inv, w.y);
                w.z = fmaf(ex2(sx.z - M), inv, w.z);
                w.w = fmaf(ex2(sx.w - M), inv, w.w);
                *reinterpret_cast<float4 *>(wo + i) = w;
            } else {
                const float a[4] = {sx.x, sx.y, sx.z, sx.w};
                for (int k = 0; i + k < end; ++k)
                    wo[i + k] = fmaf(ex2(a[k] - M), inv, wi ? wi[i + k] : 0.f);
            }
        }
    } else {
        for (int i = p0 + tid; i < end; i += 256)
            wo[i] = fmaf(ex2(x[i] - M), inv, wi ? wi[i] : 0.f);
    }
}

// ------------------------------------------------------------- launching

PFN_cuTensorMapEncodeTiled_v12000 map_encoder() {
    static std::once_flag once;
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    std::call_once(once, [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) ==
                cudaSuccess &&
            r == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    });
    return fn;
}

// A cache as [row / 8][panel][row % 8][64] fp16 with a box of one block's
// rows of GH adjacent heads.
int encode_cache(CUtensorMap *m, const void *base, int64_t groups, int D, int box_groups, const char *who) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = map_encoder();
    if (!enc) return fail(PA_ERR_CUDA, "%s: cuTensorMapEncodeTiled unavailable", who);
    const cuuint64_t dims[4] = {64, 8, (cuuint64_t)(D / 64), (cuuint64_t)groups};
    const cuuint64_t strides[3] = {(cuuint64_t)D * 2, 128, (cuuint64_t)D * 16};
    const cuuint32_t box[4] = {64, 8, (cuuint32_t)(D / 64), (cuuint32_t)box_groups}, elem[4] = {1, 1, 1, 1};
    const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<void *>(base), dims, strides, box,
                           elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(PA_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed (%d)", who, (int)r);
    return PA_OK;
}

constexpr int kMaxDevs = 64;

int sm_count() {
    static std::once_flag once[kMaxDevs];
    static int n[kMaxDevs];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevs) return 152;
    std::call_once(once[dev], [&] {
        n[dev] = 152;
        cudaDeviceGetAttribute(&n[dev], cudaDevAttrMultiProcessorCount, dev);
    });
    return n[dev];
}

// Heads a unit takes: as many adjacent ones as divide H (longer copies), at
// most 4, 2 with 64 query rows (8 consumer warps) and 2 where a stage of 4
// heads would be 64 KB (D = 128, B = 32).
int heads_per_unit(int H, int MW, int D, int B) {
    int gh = H % 4 == 0 ? 4 : H % 2 == 0 ? 2 : 1;
    if (MW == 4 || (D == 128 && B == 32)) gh = std::min(gh, 2);
    return gh;
}
int row_tiles(int max_q) { return max_q <= 16 ? 1 : max_q <= 32 ? 2 : 4; }

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Parts of cut sequences a launch can have: each is at least half a slot's
// share of the blocks, rounded up, and a sequence of k > 1 parts is longer
// than k - 1 of them; at most 4 CTAs an SM take units.
int part_cap(int n_seqs, int max_blocks, int hg) {
    const int64_t slots = (int64_t)sm_count() * 4;
    return (int)std::min<int64_t>(4 * slots / hg + 4, (int64_t)n_seqs * std::max(max_blocks, 1));
}

struct Sections {
    size_t cut, ml, acc, plan, one, scores, total;
};
Sections sections(int n_seqs, int max_blocks, int NR, int cap, bool weights, const pa_pool_desc *d) {
    Sections s{};
    size_t at = kHeaderBytes;
    const size_t rows = (size_t)cap * d->num_heads * NR;
    s.cut = at;
    at += align256((size_t)cap * sizeof(int4));
    s.ml = at;
    at += align256(rows * sizeof(float2));
    s.acc = at;
    at += align256(rows * d->head_dim * sizeof(float));
    if (weights) {
        s.plan = at;
        at += align256((size_t)n_seqs * sizeof(int2));
        s.one = at;
        at += align256((size_t)n_seqs * d->num_heads * sizeof(float2));
        s.scores = at;
        at += align256((size_t)n_seqs * d->num_heads * max_blocks * d->block_size * sizeof(float));
    }
    s.total = at;
    return s;
}

bool tree_geometry_ok(const pa_pool_desc *d, std::string *why) {
    if (!device_geometry_ok(d, why)) return false;
    if (!(d->head_dim == 64 || d->head_dim == 128)) {
        *why = "head_dim must be 64 or 128";
        return false;
    }
    if (d->block_size < 8) {
        *why = "block_size must be 8, 16 or 32";
        return false;
    }
    if (d->num_heads > 65535 || (int64_t)d->num_blocks * d->num_heads * d->block_size / 8 >= (1ll << 31)) {
        *why = "num_heads above 65535, or a cache of 2^34 rows or more";
        return false;
    }
    return true;
}

template <int D, int GH, int MW, bool SCORES>
int launch_tree(TreeParams p, const TreeMaps &maps, const char *who, cudaStream_t st) {
    using Cfg = TreeCfg<D, GH, MW>;
    auto kern = tree_attention_kernel<D, GH, MW, SCORES>;
    constexpr int kSmBytes = 227 * 1024, kMaxBytes = 227 * 1024;
    static std::once_flag once[kMaxDevs];
    static cudaError_t err[kMaxDevs];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevs)
        return fail(PA_ERR_CUDA, "%s: cudaGetDevice failed", who);
    std::call_once(once[dev], [&] {
        err[dev] = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxBytes);
    });
    if (err[dev] != cudaSuccess)
        return fail(PA_ERR_CUDA, "%s: cudaFuncSetAttribute: %s", who, cudaGetErrorString(err[dev]));
    // as many CTAs an SM as leave each at least 3 stages beside its plan
    int per_sm = Cfg::PER_SM, stages = 0;
    // a stage holds whole blocks, 16 tokens at least, and 16 KB
    p.stage_tokens = std::max(std::max(16, 1 << p.bshift), 16384 / (GH * D * 4));
    const int stage_bytes = GH * p.stage_tokens * D * 4;
    for (; per_sm >= 1; --per_sm) {
        const int room = (per_sm == 1 ? kMaxBytes : (kSmBytes + 1024) / per_sm - 1024) - Cfg::bytes(p.n_seqs, 0);
        stages = std::min(Cfg::MAX_STAGES, room / stage_bytes);
        if (stages >= 3) break;
    }
    if (per_sm < 1) return fail(PA_ERR_INVALID_ARG, "%s: the batch's plan does not fit", who);
    p.stages = stages;
    cudaError_t e = cudaMemsetAsync(p.header, 0, 8, st);
    if (e != cudaSuccess) return fail(PA_ERR_CUDA, "%s: memset: %s", who, cudaGetErrorString(e));
    kern<<<sm_count() * per_sm, Cfg::THREADS, Cfg::bytes(p.n_seqs, stages * stage_bytes), st>>>(p, maps);
    e = cudaGetLastError();
    if (e != cudaSuccess) return fail(PA_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
    return PA_OK;
}

template <int D, int MW, bool SCORES>
int launch_heads(int gh, const TreeParams &p, const TreeMaps &maps, const char *who, cudaStream_t st) {
    if constexpr (MW < 4)
        if (gh == 4) return launch_tree<D, 4, MW, SCORES>(p, maps, who, st);
    if (gh == 2) return launch_tree<D, 2, MW, SCORES>(p, maps, who, st);
    return launch_tree<D, 1, MW, SCORES>(p, maps, who, st);
}

// Checks and the main launch that both entry points share.
int launch_common(const char *who, bool weights, TreeParams &p, const void *k_cache, const void *v_cache,
                  void *workspace, size_t workspace_bytes, int max_q, const pa_pool_desc *d, cudaStream_t st) {
    const int MW = row_tiles(max_q), NR = 16 * MW, B = d->block_size;
    const int gh = heads_per_unit(d->num_heads, MW, d->head_dim, B);
    p.cap = part_cap(p.n_seqs, p.max_blocks, d->num_heads / gh);
    const Sections s = sections(p.n_seqs, p.max_blocks, NR, p.cap, weights, d);
    if (!workspace || workspace_bytes < s.total)
        return fail(PA_ERR_INVALID_ARG, "%s: workspace of %zu bytes needed, %zu given", who, s.total,
                    workspace ? workspace_bytes : (size_t)0);
    if (reinterpret_cast<uintptr_t>(workspace) & 255)
        return fail(PA_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", who);
    char *ws = static_cast<char *>(workspace);
    p.header = reinterpret_cast<int32_t *>(ws);
    p.cut = reinterpret_cast<int4 *>(ws + s.cut);
    p.ws_ml = reinterpret_cast<float2 *>(ws + s.ml);
    p.ws_acc = reinterpret_cast<float *>(ws + s.acc);
    if (weights) {
        p.plan = reinterpret_cast<int2 *>(ws + s.plan);
        p.ml_one = reinterpret_cast<float2 *>(ws + s.one);
        p.scores = reinterpret_cast<float *>(ws + s.scores);
        p.score_stride = p.max_blocks * B;
    }
    p.num_heads = d->num_heads;
    p.num_blocks = d->num_blocks;
    p.bshift = B == 8 ? 3 : B == 16 ? 4 : 5;
    p.max_q = max_q;
    TreeMaps maps;
    const int64_t groups = (int64_t)d->num_blocks * d->num_heads * B / 8;
    int rc = encode_cache(&maps.k, k_cache, groups, d->head_dim, gh * B / 8, who);
    if (rc == PA_OK) rc = encode_cache(&maps.v, v_cache, groups, d->head_dim, gh * B / 8, who);
    if (rc != PA_OK) return rc;
    if (d->head_dim == 64) {
        if (weights) return launch_heads<64, 1, true>(gh, p, maps, who, st);
        return MW == 1 ? launch_heads<64, 1, false>(gh, p, maps, who, st)
             : MW == 2 ? launch_heads<64, 2, false>(gh, p, maps, who, st)
                       : launch_heads<64, 4, false>(gh, p, maps, who, st);
    }
    if (weights) return launch_heads<128, 1, true>(gh, p, maps, who, st);
    return MW == 1 ? launch_heads<128, 1, false>(gh, p, maps, who, st)
         : MW == 2 ? launch_heads<128, 2, false>(gh, p, maps, who, st)
                   : launch_heads<128, 4, false>(gh, p, maps, who, st);
}

bool mis(const void *ptr, int n) { return (reinterpret_cast<uintptr_t>(ptr) & (n - 1)) != 0; }

}  // namespace

size_t tree_workspace_bytes(int32_t n_seqs, int32_t max_blocks, int32_t max_q_len, const pa_pool_desc *d) {
    std::string why;
    if (!d || n_seqs <= 0 || n_seqs > PA_TREE_MAX_SEQS || max_blocks < 0 || max_q_len < 1 ||
        max_q_len > PA_TREE_MAX_NODES || !tree_geometry_ok(d, &why))
        return 0;
    const int MW = row_tiles(max_q_len);
    const int hg = d->num_heads / heads_per_unit(d->num_heads, MW, d->head_dim, d->block_size);
    return sections(n_seqs, max_blocks, 16 * MW, part_cap(n_seqs, max_blocks, hg), false, d).total;
}

size_t decode_weights_workspace_bytes(int32_t n_seqs, int32_t max_blocks, const pa_pool_desc *d) {
    std::string why;
    if (!d || n_seqs <= 0 || n_seqs > PA_TREE_MAX_SEQS || max_blocks < 0 || !tree_geometry_ok(d, &why)) return 0;
    const int hg = d->num_heads / heads_per_unit(d->num_heads, 1, d->head_dim, d->block_size);
    return sections(n_seqs, max_blocks, 16, part_cap(n_seqs, max_blocks, hg), true, d).total;
}

int launch_tree_attention(void *out, const void *q, const void *k_cache, const void *v_cache,
                          const int32_t *block_tables, const int32_t *ctx_lens, const int32_t *q_starts,
                          const int32_t *parents, int32_t n_seqs, int32_t max_blocks, int32_t max_q_len,
                          int32_t q_rows, float scale, void *workspace, size_t workspace_bytes,
                          int32_t *status, const pa_pool_desc *d, void *stream) {
    const char *who = "pa_tree_attention";
    std::string why;
    if (!d) return fail(PA_ERR_INVALID_ARG, "%s: NULL desc", who);
    if (!tree_geometry_ok(d, &why)) return fail(PA_ERR_INVALID_ARG, "%s: %s", who, why.c_str());
    if (n_seqs < 0 || n_seqs > PA_TREE_MAX_SEQS || max_blocks < 0 || q_rows < 0)
        return fail(PA_ERR_INVALID_ARG, "%s: n_seqs=%d (<= %d), max_blocks=%d, q_rows=%d", who, n_seqs,
                    PA_TREE_MAX_SEQS, max_blocks, q_rows);
    if (max_q_len < 0 || max_q_len > PA_TREE_MAX_NODES)
        return fail(PA_ERR_INVALID_ARG, "%s: max_q_len=%d (<= %d)", who, max_q_len, PA_TREE_MAX_NODES);
    if (!std::isfinite(scale)) return fail(PA_ERR_INVALID_ARG, "%s: scale is not finite", who);
    if (n_seqs == 0 || max_q_len == 0 || q_rows == 0) return PA_OK;
    if (!out || !q || !k_cache || !v_cache || !ctx_lens || !q_starts || !block_tables)
        return fail(PA_ERR_INVALID_ARG, "%s: NULL pointer", who);
    if (mis(out, 16) || mis(q, 16) || mis(k_cache, 16) || mis(v_cache, 16) || mis(block_tables, 4) ||
        mis(ctx_lens, 4) || mis(q_starts, 4) || mis(parents, 4) || mis(status, 4))
        return fail(PA_ERR_INVALID_ARG, "%s: misaligned pointer", who);
    if (d->num_blocks < 1 || max_blocks < 1 || (int64_t)max_blocks * d->block_size > INT32_MAX)
        return fail(PA_ERR_INVALID_ARG, "%s: num_blocks=%d, max_blocks=%d", who, d->num_blocks, max_blocks);
    TreeParams p{};
    p.out = static_cast<__half *>(out);
    p.q = static_cast<const __half *>(q);
    p.block_tables = block_tables;
    p.ctx_lens = ctx_lens;
    p.q_starts = q_starts;
    p.parents = parents;
    p.status = status;
    p.n_seqs = n_seqs;
    p.max_blocks = max_blocks;
    p.q_rows = q_rows;
    p.qscale = scale * kLog2e;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int rc = launch_common(who, false, p, k_cache, v_cache, workspace, workspace_bytes, max_q_len, d, st);
    if (rc != PA_OK) return rc;
    const int NR = 16 * row_tiles(max_q_len);
    const int blocks = (int)std::min<int64_t>((int64_t)p.cap * d->num_heads * NR / 8 + 1, (int64_t)sm_count() * 4);
    if (d->head_dim == 64) tree_join_kernel<64><<<blocks, 256, 0, st>>>(p, NR);
    else tree_join_kernel<128><<<blocks, 256, 0, st>>>(p, NR);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return fail(PA_ERR_CUDA, "%s: join launch: %s", who, cudaGetErrorString(e));
    return PA_OK;
}

int launch_decode_attention_weights(void *out, float *weights_out, const float *weights_in, int32_t weight_len,
                                    const void *q, const void *k_cache, const void *v_cache,
                                    const int32_t *block_tables, const int32_t *ctx_lens, int32_t n_seqs,
                                    int32_t max_blocks, float scale, void *workspace, size_t workspace_bytes,
                                    int32_t *status, const pa_pool_desc *d, void *stream) {
    const char *who = "pa_decode_attention_weights";
    std::string why;
    if (!d) return fail(PA_ERR_INVALID_ARG, "%s: NULL desc", who);
    if (!tree_geometry_ok(d, &why)) return fail(PA_ERR_INVALID_ARG, "%s: %s", who, why.c_str());
    if (n_seqs < 0 || n_seqs > PA_TREE_MAX_SEQS || max_blocks < 0 || weight_len < 0)
        return fail(PA_ERR_INVALID_ARG, "%s: n_seqs=%d (<= %d), max_blocks=%d, weight_len=%d", who, n_seqs,
                    PA_TREE_MAX_SEQS, max_blocks, weight_len);
    if (!std::isfinite(scale)) return fail(PA_ERR_INVALID_ARG, "%s: scale is not finite", who);
    if (n_seqs == 0) return PA_OK;
    if (!out || !q || !k_cache || !v_cache || !ctx_lens || !block_tables || (weight_len > 0 && !weights_out))
        return fail(PA_ERR_INVALID_ARG, "%s: NULL pointer", who);
    if (mis(out, 16) || mis(q, 16) || mis(k_cache, 16) || mis(v_cache, 16) || mis(block_tables, 4) ||
        mis(ctx_lens, 4) || mis(weights_out, 4) || mis(weights_in, 4) || mis(status, 4))
        return fail(PA_ERR_INVALID_ARG, "%s: misaligned pointer", who);
    if (d->num_blocks < 1 || max_blocks < 1 || (int64_t)max_blocks * d->block_size > INT32_MAX)
        return fail(PA_ERR_INVALID_ARG, "%s: num_blocks=%d, max_blocks=%d", who, d->num_blocks, max_blocks);
    const int64_t longest = std::min<int64_t>(weight_len, (int64_t)max_blocks * d->block_size);
    const dim3 grid(d->num_heads, n_seqs, (unsigned)std::max<int64_t>(1, (longest + kWeightChunk - 1) / kWeightChunk));
    if (grid.z > 65535) return fail(PA_ERR_INVALID_ARG, "%s: weight_len=%d too large", who, weight_len);
    TreeParams p{};
    p.out = static_cast<__half *>(out);
    p.q = static_cast<const __half *>(q);
    p.block_tables = block_tables;
    p.ctx_lens = ctx_lens;
    p.status = status;
    p.n_seqs = n_seqs;
    p.max_blocks = max_blocks;
    p.q_rows = n_seqs;
    p.weight_len = weight_len;
    p.qscale = scale * kLog2e;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int rc = launch_common(who, true, p, k_cache, v_cache, workspace, workspace_bytes, 1, d, st);
    if (rc != PA_OK) return rc;
    const bool vec = weight_len % 4 == 0 && !mis(weights_out, 16) && !mis(weights_in, 16);
    auto go = [&](auto kern) { kern<<<grid, 256, 0, st>>>(p, 16, weights_out, weights_in); };
    if (d->head_dim == 64) vec ? go(decode_weights_kernel<64, true>) : go(decode_weights_kernel<64, false>);
    else vec ? go(decode_weights_kernel<128, true>) : go(decode_weights_kernel<128, false>);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return fail(PA_ERR_CUDA, "%s: weights launch: %s", who, cudaGetErrorString(e));
    return PA_OK;
}

}  // namespace pagedkv
