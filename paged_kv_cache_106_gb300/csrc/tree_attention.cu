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
// sequence, 4 D bytes against 4 n D operations a position, so up to the 64 rows
// allowed the bytes bound it (64 operations a byte against the 286 that the
// tensor cores could do in that time).
//
// Products (tcgen05, one tile of 128 tokens at a time).  Tokens, of which there
// are always many, are the 128 lanes of tensor memory and the few rows its
// columns (N = 16, 32 or 64: the rows padded):
//     S (tokens x rows)  = K Q^T,     K and Q as they lie, K-major
//     O (dims x rows)   += V^T P^T,   V and P as they lie, both MN-major
// so nothing is transposed, 8 rows cost little more than 1, and one thread owns
// one token's scores (then one dimension of the output).  With queries in the
// lanes (128 of them, 8 used) the same cases took 242 us instead of 215 (64
// sequences of 128 to 2048 positions, 4 to 16 nodes, 40 heads of 128) and 282
// instead of 214 (3 sequences of 40 to 65 thousand, 31 nodes, 32 heads of 64);
// warp-level products (m16n8k16) 1814 us instead of 762 at 64 nodes (256
// sequences of 128 to 1536 positions).
//
// One persistent CTA an SM.  Its warps:
//   * producer: names the units (sequence, head, part) and streams their blocks
//     by TMA, a block of one head a box, 128-byte swizzled, keys and values of a
//     tile in two stages of a ring that fills what shared memory is left (5 to 12
//     stages, 160 to 196 KB on their way);
//   * products: S of tile t + 1, then O of tile t;
//   * queries: Q of the unit by TMA, and which nodes see each node;
//   * 4 softmax warps up to 16 rows, 8 above (a token's rows halved: 64 nodes
//     945 -> 779 us; at 16 rows 8 gave 22.4 instead of 21.9 us for one sequence,
//     247 instead of 246 us for 64).  Up to 16 rows and with two units a CTA or
//     more there are two groups of 4 that take units in turn (launch_tree).
// Scores are taken relative to a reference per row, 7 binary orders below the
// largest score when it is set, that only moves where a score passes it by 15
// (then O and the sums are rescaled): almost every tile goes without a reduction
// over its tokens.
//
// Rounding: products of fp16 values are exact in the fp32 accumulators; sums,
// references and the join of parts are fp32.  P enters the second product as fp16,
// which is what the tensor cores take beside fp16 values: 2^-11 of each weight at
// most, like the fp16 output's own rounding.  Below 2^-14 fp16 has steps of 2^-24,
// so the references lie where P uses its upper bits: the largest term of a row is
// 2^7 to 2^15, and only weights below 2^-21 of the largest one meet those steps
// (half of one is 2^-32 of the largest weight).  With references at the maximum a
// first position of 20 binary orders above 32 thousand others, its own value 0,
// left the output off by 3 % (now 2^-11).
//
// Work plan (the same in every CTA, no counters to clear): sequences are cut into
// even parts by part_size; cut ones first, then the others by size, dealt to the
// CTAs back and forth.  The kernel that joins the parts is launched ahead and
// waits for this one's end (one sequence: 14.2 instead of 14.5 us).
//
// Measured (in a graph; share of the bytes' time at 6.78 TB/s): 64 sequences of
// 128 to 2048, 4 to 16 nodes, 40 heads of 128: 215 us (98 %); 256 sequences of 128
// to 1536, 64 nodes: 765 us (91 %; the softmax of 64 rows and the end of each
// unit, 3.2 of 3.4 thousand clocks a tile, are what bounds it); 3 of 40 to 65
// thousand, 17 to 31 nodes, 32 heads of 64: 216 us (88 %); 1 of 2048, 8 nodes:
// 14.2 us against 6.2 (two launches, the plan, one round of loads: latency).
// Weights form: 64 sequences 220 us (97 %), 2 of 50 to 65 thousand 381 us (93 %).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <mutex>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "tc_device.cuh"

namespace pagedkv {

namespace tc {
// 16 consecutive 32-bit columns of this thread's lane.
__device__ __forceinline__ void ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
}  // namespace tc

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kHeaderBytes = 256;    // workspace head: number of cut sequences
constexpr int kUnitSlots = 8;        // units a CTA has open (with 3, 256 sequences of 100 positions took 164 instead of 161 us)
constexpr int kTile = 128;           // tokens of a tile: the lanes of tensor memory
constexpr float kBelowLog2 = 7.f;    // how far below its row's largest score a reference is set
constexpr float kRescaleLog2 = 15.f; // how far scores may pass it: P stays in fp16's range

struct TreeParams {
    __half *out;
    const __half *q;
    const __half *k_cache, *v_cache;   // (read around the ring by node_tiles only)
    const int32_t *block_tables;
    const int32_t *ctx_lens;
    const int32_t *q_starts;   // NULL (weights form): one query a sequence
    const int32_t *parents;    // NULL: a chain
    int32_t *header;           // [0] cut sequences
    int4 *cut;                 // [cap] cut sequences: s, first part, parts, rows
    float2 *ws_ml;             // [cap][H][NR] (max, sum) of a part's rows
    float *ws_acc;             // [cap][H][NR][D] unnormalised output
    // weights form
    int2 *plan;                // [S] first part (cut) and parts of each sequence
    float2 *ml_one;            // [S][H] (max, sum) of an uncut sequence
    float *scores;             // [S][H][score_stride] scores in log2 units
    int32_t *status;
    int32_t n_seqs, num_heads, num_blocks, max_blocks, bshift, max_q, q_rows, cap;
    int32_t stages;
    int32_t score_stride, weight_len;
    float qscale;              // scale * log2(e)
};

struct TreeMaps {
    CUtensorMap k, v, q;
};

// ---------------------------------------------------------------- helpers

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
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

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

// Whether a barrier's phase is complete, without waiting for it.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"(bar), "r"(parity)
        : "memory");
    return r != 0;
}

// One lane of a warp whose lanes are all here, always the same.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(r));
    return r != 0;
}

// Lets the kernel launched after this one start (it then waits, at
// wait_for_launch_before, for this one's end).
__device__ __forceinline__ void allow_next_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_launch_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

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

// A lane's candidate for how many tiles a part may have, and what comes of it.
struct Cuts {
    int size;          // tiles of a part, at most
    int units, parts;  // units of all sequences; of them parts of cut ones
    int tiles;         // of the cut ones
    __device__ void take(int l) {
        const int n = (l + size - 1) / size;
        units += n;
        if (n > 1) {
            parts += n;
            tiles += l;
        }
    }
};
// The longest sequence in lane + 1 parts.  (More would serve a long context of
// one head and hurt where rows to join are many: with up to 125 parts, 70000
// positions and 8 rows 29.0 us instead of 31.0, 2 heads' 2 x 30000 and 64 rows
// 29.4 us instead of 27.9.)
__device__ __forceinline__ Cuts candidate(int longest, int lane) {
    return {max(1, (longest + lane) / (lane + 1)), 0, 0, 0};
}

// How many tiles a part may have: the candidate with the earliest end.  (Its
// parts fit the workspace: lane 0 cuts nothing, and parts of a quarter of an SM's
// share are at most two for each such quarter in a cut sequence.)  A unit
// costs its tiles, about one more to get going, and where it is a part of a cut
// sequence the writing and joining of its rows.  The last CTA is done when all
// work would be, evenly shared; or after as many parts as it must take (they
// are alike: 1056 units on 152 CTAs are 7 each, 1440 are 10 where 9.5 would be
// even), or, where whole sequences come last, half one of these late.  (Over
// random batches the choice ends 3 % after the best candidate's end; half a part
// late for every cut ended 5 % after it: 3 sequences of 60000 at 32 heads 241 us
// instead of 232, 2 at 40 heads 393 instead of 386.)
__device__ __forceinline__ int part_size(const TreeParams &p, long long total, int some, int HG, const Cuts &c,
                                         int lane) {
    const int slots = gridDim.x;
    // many units: parts of a quarter of an SM's share
    if ((long long)some * HG >= 4 * slots) return max(1, (int)((total * HG + 4 * slots - 1) / (4 * slots)));
    const float extra = lane ? 1.f + p.max_q * (2.f / kTile) : 1.f;   // in tiles
    const float all = ((float)total * HG + (float)c.units * HG * extra) / slots;
    float end = fmaxf(all, (float)c.size + extra);
    if (c.parts > 0)
        end = fmaxf(end, (float)((c.parts * HG + slots - 1) / slots) * ((float)c.tiles / c.parts + extra));
    if (c.units > c.parts && c.units * HG > slots)
        end = fmaxf(end, all + 0.5f * (float)(total - c.tiles) / (c.units - c.parts));
    if (c.parts > p.cap) end = INFINITY;
    float best = end;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) best = fminf(best, __shfl_xor_sync(kAll, best, off));
    return __shfl_sync(kAll, c.size, __ffs(__ballot_sync(kAll, end == best)) - 1);
}

// What the plan of more than 32 sequences adds up over the warps.
struct PlanSums {
    unsigned long long total;          // tiles
    int some, longest;                 // sequences with work, tiles of the longest
    int units[32], parts[32], tiles[32];   // by candidate
};

// More than 32 sequences: by all warps, in chunks of 32.  (A function of its own:
// its instructions are not in the way of small batches.)
template <bool SCORES>
__device__ __noinline__ void plan_of_many(const TreeParams &p, int32_t *pre, int32_t *len, uint16_t *order,
                                          int32_t *vars, int32_t *counts, int HG) {
    const int S = p.n_seqs, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, n_warps = blockDim.x >> 5;
    PlanSums *sums = reinterpret_cast<PlanSums *>(counts);
    for (int i = tid; i < (int)(sizeof(PlanSums) / 4); i += (int)blockDim.x) counts[i] = 0;
    __syncthreads();
    for (int s0 = warp * 32; s0 < S; s0 += (int)blockDim.x) {
        const int s = s0 + lane;
        int l = 0;
        if (s < S) {
            const SeqRows r = rows_of<SCORES>(p, s, blockIdx.x == 0);
            len[s] = l = r.n > 0 ? (r.ctx + kTile - 1) / kTile : 0;
        }
        const int add = __reduce_add_sync(kAll, l), top = __reduce_max_sync(kAll, l);
        const int n = __popc(__ballot_sync(kAll, l > 0));
        if (lane == 0) {
            atomicAdd(&sums->total, (unsigned long long)add);
            atomicMax(&sums->longest, top);
            atomicAdd(&sums->some, n);
        }
    }
    __syncthreads();
    const int chunks = (S + 31) / 32, some = sums->some, longest = sums->longest;
    const long long total = (long long)sums->total;
    Cuts c = candidate(longest, lane);
    if ((long long)some * HG < 4 * (int)gridDim.x) {
        for (int s = warp; s < S; s += n_warps) c.take(len[s]);
        atomicAdd(&sums->units[lane], c.units);
        atomicAdd(&sums->parts[lane], c.parts);
        atomicAdd(&sums->tiles[lane], c.tiles);
        __syncthreads();
        c.units = sums->units[lane];
        c.parts = sums->parts[lane];
        c.tiles = sums->tiles[lane];
    }
    const int P = part_size(p, total, some, HG, c, lane);
    // counting sort by size class: 0 the cut ones, 1 .. 31 the others, long
    // ones first, in order of index within a class; 32: no work
    int32_t *at = counts + sizeof(PlanSums) / 4;     // [chunk][33]
    const int top = max(1, min(P, longest));
    auto cls = [&](int s) {
        const int l = s < S ? len[s] : 0;
        return l == 0 ? 32 : l > P ? 0 : 1 + (top - l) * 30 / top;   // (below 2^24 tiles)
    };
    auto rank = [&](int k, unsigned &same) {
        same = __match_any_sync(kAll, k);
        return __popc(same & ((1u << lane) - 1));
    };
    unsigned same;
    for (int ch = warp; ch < chunks; ch += n_warps) {
        at[ch * 33 + lane] = 0;
        __syncwarp();
        const int k = cls(ch * 32 + lane), r = rank(k, same);
        if (r == 0 && k < 32) at[ch * 33 + k] = __popc(same);
    }
    __syncthreads();
    if (warp == 0) {                 // lane = class: where its chunks' sequences start
        int mine = 0;
        for (int ch = 0; ch < chunks; ++ch) mine += at[ch * 33 + lane];
        const int incl = warp_incl_scan(mine, lane);
        int run = incl - mine;
        for (int ch = 0; ch < chunks; ++ch) {
            const int n = at[ch * 33 + lane];
            at[ch * 33 + lane] = run;
            run += n;
        }
        if (lane == 31) vars[0] = incl;
        if (lane == 0) vars[1] = incl;
    }
    __syncthreads();
    for (int ch = warp; ch < chunks; ch += n_warps) {
        const int k = cls(ch * 32 + lane), r = rank(k, same);
        if (k < 32) order[at[ch * 33 + k] + r] = (uint16_t)(ch * 32 + lane);
    }
    __syncthreads();
    // running sums of the parts in that order: within chunks, then of chunks
    const int n_ord = vars[0];
    for (int ch = warp; ch * 32 < n_ord; ch += n_warps) {
        const int i = ch * 32 + lane, parts = i < n_ord ? (len[order[i]] + P - 1) / P : 0;
        const int incl = warp_incl_scan(parts, lane);
        if (i < n_ord) pre[i] = incl - parts;
        if (lane == 31) at[ch] = incl;
    }
    __syncthreads();
    if (warp == 0) {
        int base = 0;
        for (int c0 = 0; c0 * 32 < n_ord; c0 += 32) {
            const int n = (c0 + lane) * 32 < n_ord ? at[c0 + lane] : 0, incl = warp_incl_scan(n, lane);
            if ((c0 + lane) * 32 < n_ord) at[c0 + lane] = base + incl - n;
            base += __shfl_sync(kAll, incl, 31);
        }
        if (lane == 0) pre[n_ord] = base;
    }
    __syncthreads();
    for (int i = tid; i < n_ord; i += (int)blockDim.x) pre[i] += at[i >> 5];
}

// The launch's work plan, the same in every CTA, by all its threads: len[s]
// tiles of sequence s (0: no work), order[] the sequences with work, pre[i]
// the parts of those before the i-th; vars: how many have work, how many of
// them are cut.  A part is read once for each of HG head groups.  CTA 0 also
// leaves the cut sequences (weights form: every sequence's parts) for the kernels
// that join them.
template <bool SCORES>
__device__ void make_plan(const TreeParams &p, int32_t *pre, int32_t *len, uint16_t *order, int32_t *vars,
                          int32_t *counts, int HG) {
    const int S = p.n_seqs, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (S > 32) {
        plan_of_many<SCORES>(p, pre, len, order, vars, counts, HG);
    } else if (warp == 0) {
        // a sequence a lane: the same without loops
        int l = 0;
        if (lane < S) {
            const SeqRows r = rows_of<SCORES>(p, lane, blockIdx.x == 0);
            len[lane] = l = r.n > 0 ? (r.ctx + kTile - 1) / kTile : 0;
        }
        __syncwarp();
        const int total = __reduce_add_sync(kAll, l), longest = __reduce_max_sync(kAll, l);
        const int some = __popc(__ballot_sync(kAll, l > 0));
        Cuts c = candidate(longest, lane);
        for (int s = 0; s < S; ++s) c.take(__shfl_sync(kAll, l, s));
        const int P = part_size(p, total, some, HG, c, lane);
        const int parts = (l + P - 1) / P, key = parts > 1 ? INT_MAX : l;
        int rank = 0;
        for (int s = 0; s < S; ++s) {
            const int other = __shfl_sync(kAll, key, s);
            rank += other > key || (other == key && s < lane);
        }
        if (l > 0) {
            order[rank] = (uint16_t)lane;
            counts[rank] = parts;
        }
        __syncwarp();
        const int here = lane < some ? counts[lane] : 0, incl = warp_incl_scan(here, lane);
        if (lane < some) pre[lane] = incl - here;
        if (lane == max(some, 1) - 1) pre[some] = incl;
        const int n_cut = __popc(__ballot_sync(kAll, parts > 1));
        if (lane == 0) {
            vars[0] = some;
            vars[1] = n_cut;
        }
    }
    __syncthreads();
    if (blockIdx.x == 0) {   // for the kernels that join the parts
        const int n_cut = vars[1];
        if (tid == 0) p.header[0] = n_cut;
        for (int i = tid; i < n_cut; i += (int)blockDim.x) {
            const int s = order[i];
            const SeqRows r = rows_of<SCORES>(p, s, false);
            p.cut[i] = make_int4(s, pre[i], pre[i + 1] - pre[i], r.n);
        }
        if (SCORES) {
            for (int s = tid; s < S; s += (int)blockDim.x)
                if (len[s] == 0) p.plan[s] = make_int2(0, 0);
            for (int i = tid; i < vars[0]; i += (int)blockDim.x)
                p.plan[order[i]] = make_int2(pre[i], pre[i + 1] - pre[i]);
        }
    }
}

// Which nodes see each node of a sequence (itself and its descendants): every
// node's ancestors by doubling the parent links (lane l takes nodes l and
// l + 32), then the 64 x 64 bits transposed.
template <bool SCORES>
__device__ __forceinline__ void nodes_seen_by(const TreeParams &p, const SeqRows &r, int lane, uint64_t *out) {
    uint64_t m[2];
    int up[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int i = lane + 32 * e;
        up[e] = i - 1;
        if (!SCORES && p.parents && i < r.n) {
            up[e] = p.parents[r.row0 + i];
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
        for (int k = 1; k < r.n; k <<= 1) {
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
    for (int j = 0; j < r.n; ++j) {
        const uint32_t lo = __ballot_sync(kAll, lane < r.n && ((m[0] >> j) & 1));
        const uint32_t hi = __ballot_sync(kAll, lane + 32 < r.n && ((m[1] >> j) & 1));
        if (lane == 0) out[j] = (uint64_t)hi << 32 | lo;
    }
}

// ------------------------------------------------------------ main kernel

constexpr int kMinStages = 4, kMaxStages = 12;

template <int D, int NQ, int G>
struct TreeCfg {
    static constexpr int NP = D / 64;                        // 64-column panels of a row
    static constexpr int HALF = kTile * D * 2;               // keys or values of a tile: a ring stage
    // softmax warps: a token of the tile a thread, with more than 16 rows two
    // threads a token, each half of the rows; then the warps that stream the
    // ring, issue the products and fetch Q
    // (SW of them).  Two groups of them take units in turn, so that one's end
    // (sums, O, output) is behind the other's tiles: see launch_tree.
    static constexpr int SW = NQ == 16 ? 4 : 8, CQ = NQ / (SW / 4);
    static constexpr int PRODUCER = SW * G, PRODUCTS = PRODUCER + 1, Q_WARP = PRODUCER + 2;
    static constexpr int THREADS = (PRODUCER + 3) * 32;
    // tensor-memory columns: two S, then for each group O, O of the tiles that
    // rows see different nodes of (a power of two in all)
    static constexpr uint32_t S_COL = 0, O_COL = 2 * NQ, COLS = G == 2 ? 8 * NQ : 4 * NQ;
    static constexpr int BARS = 0;                           // full, empty; units; q, s, p, seen, o, done
    static constexpr int VARS = BARS + (2 * kMaxStages + 3 * kUnitSlots + 2 * 2 + 4 + 2 + 2 + 1) * 8;
    static constexpr int UNITS = (VARS + 16 + 15) / 16 * 16;
    static constexpr int SEEN = UNITS + kUnitSlots * 64;     // NQ x u64 per slot
    static constexpr int RED = SEEN + kUnitSlots * NQ * 8;   // per 32 tokens and row
    static constexpr int REF = RED + G * 4 * NQ * 4;    // reference maxima, corrections
    static constexpr int PLAN = REF + G * 2 * NQ * 4;   // pre[S+1], len[S], order[S]
    static constexpr int Q_BYTES = NQ * D * 2;               // [panel][row][128 bytes]
    static constexpr int QB = Q_BYTES > 8192 ? 1 : 2;        // buffers of it
    static constexpr int P_BYTES = kTile * 128;              // [token][128 bytes], rows of 64 columns
    // node_tiles' numbers: a group's own, or where P is
    static constexpr int ODD_BYTES = G == 2 ? NQ * kTile * 4 : 0;
    __host__ __device__ static constexpr int plan_bytes(int S) { return (S + 1) * 4 + S * 4 + (S + 1) / 2 * 4; }
    static constexpr int bytes(int S, int stages) {
        return (PLAN + plan_bytes(S) + 1023) / 1024 * 1024 + G * ODD_BYTES + QB * Q_BYTES + 2 * P_BYTES +
               stages * HALF;
    }
};

// One barrier of a group of softmax warps (N threads).  (A warp comes to a
// barrier, and to the loads and stores of tensor memory, with all its lanes
// together: the instructions are undefined otherwise, and lanes that parted at a
// branch before need not have met again by themselves.)
template <int N>
__device__ __forceinline__ void softmax_sync(int group) {
    __syncwarp();
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(N) : "memory");
}
// The same; whether v held in any (all) of their threads.
template <int N>
__device__ __forceinline__ bool softmax_any(int group, bool v) {
    uint32_t r;
    __syncwarp();
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, %2, %3, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v), "r"(1 + group), "n"(N)
        : "memory");
    return r != 0;
}
template <int N>
__device__ __forceinline__ bool softmax_all(int group, bool v) {
    return !softmax_any<N>(group, !v);
}

// Combines N values over a warp's lanes: on return v[0 .. max(N / 32, 1)) are
// the results for values first, first + 1, ... (every lane has a share).
template <int N, typename Op>
__device__ __forceinline__ int warp_combine(float (&v)[N], int lane, Op op) {
    int first = 0;
#pragma unroll
    for (int k = 0; k < 5; ++k) {
        const int off = 16 >> k, half = N >> (k + 1);
        if (half >= 1) {
            const bool upper = (lane & off) != 0;
#pragma unroll
            for (int i = 0; i < half; ++i) {
                const float send = upper ? v[i] : v[i + half], keep = upper ? v[i + half] : v[i];
                v[i] = op(keep, __shfl_xor_sync(kAll, send, off));
            }
            if (upper) first += half;
        } else {
            v[0] = op(v[0], __shfl_xor_sync(kAll, v[0], off));
        }
    }
    return first;
}

// The part of a unit's output that its tiles with nodes give, without the matrix
// products, by the softmax warps: where a node's value is not finite,
// 0 times it has put NaN into the rows that do not see the node.  Here a row
// adds what it sees and nothing else, in the dimensions that are odd.  Thread =
// token, then dimension, as in the kernel; buf: NQ x kTile.
// Takes 0.1 ms a tile (64 rows), one or two tiles a unit: those tiles have an
// accumulator of their own, so that the rest of a long unit needs no second
// pass.  A look at every tile's values instead costs each unit without such
// values: 256 sequences of 64 nodes took 820 us with it, 788 us so.
template <int D, int NQ, int G>
__device__ __noinline__ void node_tiles(const TreeParams &p, const int32_t *u, const uint64_t *seen,
                                        const float *ref, float *buf, bool odd, float *o) {
    using Cfg = TreeCfg<D, NQ, G>;
    constexpr int CQ = Cfg::CQ, ST = Cfg::SW * 32;
    const int s = u[0], h = u[1], tok_first = u[4], n_tok = u[5], base = u[6], n = u[7], row0 = u[8];
    const int group = G == 2 ? threadIdx.x >> 7 : 0, id = threadIdx.x - group * ST;
    const int H = p.num_heads, tok = id & 127, lane = id & 31, col0 = (id >> 7) * CQ;
    const int32_t *table = p.block_tables + (size_t)s * p.max_blocks;
    // where a position's row is in the caches, -1: in no block of the pool
    auto at = [&](int pos) {
        const int phys = table[pos >> p.bshift];
        return phys < 0 || phys >= p.num_blocks
                   ? -1ll
                   : ((((long long)phys * H + h) << p.bshift) + (pos & ((1 << p.bshift) - 1))) * D;
    };
    auto rows_that_see = [&](int pos) { return (uint64_t)(pos < base ? ~0ull : seen[pos - base]) >> col0; };
    float sum[CQ] = {};
#pragma unroll 1
    for (int t0 = max(0, base - tok_first) / kTile * kTile; t0 < n_tok; t0 += kTile) {
        const int here = min(kTile, n_tok - t0);
        const long long k_at = tok < here ? at(tok_first + t0 + tok) : -1;
        const uint64_t who = k_at >= 0 ? rows_that_see(tok_first + t0 + tok) : 0;
        // (64 dimensions at a time: no registers are left for more)
#pragma unroll 1
        for (int d0 = 0; d0 < D; d0 += 64) {
            uint4 k[8];
#pragma unroll
            for (int d = 0; d < 8; ++d)
                k[d] = k_at >= 0 ? __ldg(reinterpret_cast<const uint4 *>(p.k_cache + k_at + d0) + d) : make_uint4(0, 0, 0, 0);
#pragma unroll 1
            for (int i = 0; i < CQ && col0 + i < n; ++i) {
                const uint4 *q = reinterpret_cast<const uint4 *>(p.q + ((size_t)(row0 + col0 + i) * H + h) * D + d0);
                float *to = buf + (col0 + i) * kTile + tok, x = d0 ? *to : 0.f;
#pragma unroll
                for (int d = 0; d < 8; ++d) {
                    const uint4 q8 = __ldg(q + d);
                    const uint32_t a[4] = {k[d].x, k[d].y, k[d].z, k[d].w}, b[4] = {q8.x, q8.y, q8.z, q8.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 fa = __half22float2(*reinterpret_cast<const __half2 *>(&a[e]));
                        const float2 fb = __half22float2(*reinterpret_cast<const __half2 *>(&b[e]));
                        x = fmaf(fa.x, fb.x, fmaf(fa.y, fb.y, x));
                    }
                }
                if (d0 + 64 == D) x = (who >> i) & 1 ? ex2(fmaf(x, p.qscale, -ref[col0 + i])) : 0.f;
                *to = x;
            }
        }
        softmax_sync<ST>(group);
        if (__any_sync(kAll, odd))
            for (int j0 = 0; j0 < here; j0 += 32) {
                // a token a lane: where it is, and who sees it
                const long long mine = j0 + lane < here ? at(tok_first + t0 + j0 + lane) : -1;
                const uint64_t see = mine >= 0 ? rows_that_see(tok_first + t0 + j0 + lane) : 0;
#pragma unroll 4
                for (int j = 0; j < 32; ++j) {
                    const long long v_at = __shfl_sync(kAll, mine, j);
                    const uint64_t by = __shfl_sync(kAll, see, j);
                    const float v = odd && v_at >= 0 ? __half2float(p.v_cache[v_at + tok]) : 0.f;
#pragma unroll
                    for (int i = 0; i < CQ; ++i)
                        if ((by >> i) & 1) sum[i] = fmaf(buf[(col0 + i) * kTile + j0 + j], v, sum[i]);
                }
            }
        softmax_sync<ST>(group);
    }
    if (odd) {
#pragma unroll
        for (int i = 0; i < CQ; ++i) o[i] = sum[i];
    }
    for (int i = id; i < NQ * kTile; i += ST) buf[i] = 0.f;   // (as P: finite)
    fence_proxy_async_smem();
    softmax_sync<ST>(group);
}

template <int D, int NQ, bool SCORES, int G>
__global__ void __launch_bounds__((TreeCfg<D, NQ, G>::THREADS), 1)
    tree_attention_kernel(const __grid_constant__ TreeParams p, const __grid_constant__ TreeMaps maps) {
    using Cfg = TreeCfg<D, NQ, G>;
    constexpr int NP = Cfg::NP, HALF = Cfg::HALF;
    constexpr int QB = Cfg::QB, SW = Cfg::SW, CQ = Cfg::CQ, ST = SW * 32;
    constexpr int R = SCORES ? 1 : CQ;                   // rows a softmax thread works on
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t bar_full = smem_addr(smem + Cfg::BARS), bar_empty = bar_full + kMaxStages * 8;
    const uint32_t bar_unit = bar_empty + kMaxStages * 8, bar_unit_free = bar_unit + kUnitSlots * 8;
    const uint32_t bar_q = bar_unit_free + kUnitSlots * 8, bar_q_free = bar_q + 16, bar_s = bar_q_free + 16,
                   bar_p = bar_s + 32, bar_seen = bar_p + 16, bar_o = bar_seen + 8 * kUnitSlots, bar_done = bar_o + 16;
    int32_t *vars = reinterpret_cast<int32_t *>(smem + Cfg::VARS);    // [2]: tensor-memory address
    int32_t *units = reinterpret_cast<int32_t *>(smem + Cfg::UNITS);
    uint64_t *seen = reinterpret_cast<uint64_t *>(smem + Cfg::SEEN);
    const int S = p.n_seqs, H = p.num_heads;
    int32_t *pre = reinterpret_cast<int32_t *>(smem + Cfg::PLAN);
    int32_t *len = pre + S + 1;
    uint16_t *order = reinterpret_cast<uint16_t *>(len + S);
    uint8_t *tiles_at = smem + (Cfg::PLAN + Cfg::plan_bytes(S) + 1023) / 1024 * 1024;
    // (the shuffles here and in the products' warp tell the compiler that a warp's lanes agree)
    const int tid = threadIdx.x, warp = __shfl_sync(kAll, tid >> 5, 0), lane = tid & 31;
    const int stages = p.stages, bshift = p.bshift, B = 1 << bshift, bps = kTile >> bshift;
    // (for D = 64 the second half of V^T's rows is whatever lies 1 KB on: the
    // ring is followed by P)
    const uint32_t ring = smem_addr(tiles_at), sP = ring + stages * HALF, sQ = sP + 2 * Cfg::P_BYTES;

    if (tid == 0) {
        for (int i = 0; i < stages; ++i) {
            mbar_init(bar_full + 8 * i, 1);
            mbar_init(bar_empty + 8 * i, 1);
        }
        for (int i = 0; i < kUnitSlots; ++i) {
            mbar_init(bar_unit + 8 * i, 1);
            mbar_init(bar_unit_free + 8 * i, SW + 2);
        }
        for (int i = 0; i < QB; ++i) {
            mbar_init(bar_q + 8 * i, 1);
            mbar_init(bar_q_free + 8 * i, 1);
        }
        for (int i = 0; i < 4; ++i) mbar_init(bar_s + 8 * i, 1);   // group, buffer
        mbar_init(bar_p, SW);
        mbar_init(bar_p + 8, SW);
        for (int i = 0; i < kUnitSlots; ++i) mbar_init(bar_seen + 8 * i, 1);
        mbar_init(bar_o, 1);
        mbar_init(bar_o + 8, 1);
        mbar_init(bar_done, 1);
        fence_barrier_init();
    }
    allow_next_launch();
    if (warp == Cfg::PRODUCTS) tc::alloc(smem_addr(&vars[2]), Cfg::COLS);
    make_plan<SCORES>(p, pre, len, order, vars, reinterpret_cast<int32_t *>(tiles_at), H);
    // columns of P that no row writes have to hold finite numbers
    for (int i = tid; i < 2 * Cfg::P_BYTES / 16; i += Cfg::THREADS)
        reinterpret_cast<uint4 *>(tiles_at + stages * HALF)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = (uint32_t)vars[2];
    const int n_ord = vars[0], n_units = pre[n_ord] * H;
    // First tile of a slot's unit that rows may see different nodes of; INT_MAX: none.
    auto first_node_tile = [&](int slot) {
        const int32_t *u = units + slot * 16;
        return !SCORES && u[7] > 1 && u[4] + u[5] > u[6] ? max(0, u[6] - u[4]) / kTile : INT_MAX;
    };
    bool ok = true;

    if (warp == Cfg::PRODUCER) {
        // ================================================ producer warp
        const uint64_t policy = l2_evict_first_policy();
        const uint32_t blk_bytes = (uint32_t)D * 2u << bshift;
        const int run = B >> 3;                          // 8-row groups of a block's head
        int st = 0, k_unit = 0, issued = 0, tile = 0;    // (tile: of all units so far)
        uint32_t use = 0;
        struct Pending {
            int ticket, s, h, gp, parts, b0, nb, tbl;
            SeqRows r;
        };
        // Names the unit of a ticket and starts the loads it needs.
        auto prepare = [&](int ticket) {
            Pending u;
            u.ticket = ticket;
            u.s = u.h = u.gp = u.parts = u.b0 = u.nb = 0;
            u.tbl = -1;
            u.r.n = u.r.row0 = u.r.ctx = 0;
            if (ticket >= n_units) return u;
            u.gp = ticket / H;
            u.h = ticket - u.gp * H;
            int lo = 0, hi = n_ord - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (pre[mid] <= u.gp) lo = mid; else hi = mid - 1;
            }
            u.s = order[lo];
            u.parts = pre[lo + 1] - pre[lo];
            const int part = u.gp - pre[lo], l = len[u.s];
            // even parts, the first ones a tile longer
            const int even = l / u.parts, more = l - even * u.parts;
            u.b0 = (part * even + min(part, more)) * bps;
            u.nb = (even + (part < more)) * bps;
            // (the sequence's last blocks may be fewer)
            if (u.b0 + lane < p.max_blocks && lane < u.nb)
                u.tbl = p.block_tables[(size_t)u.s * p.max_blocks + u.b0 + lane];
            u.r = rows_of<SCORES>(p, u.s, false);
            return u;
        };
        // The next free stage of the ring.
        auto stage = [&]() {
            if (use > 0) ok = mbar_wait_bounded(bar_empty + 8 * st, (use - 1) & 1u, p.status, true);
            ok = __all_sync(kAll, ok);
            return ok;
        };
        // Units in order of size, back and forth over the CTAs.
        const int n_ctas = gridDim.x;
        Pending cur = prepare(blockIdx.x);
        int ends = 0;
        while (true) {
            const bool last = cur.ticket >= n_units;     // one more descriptor (a group): the end
            const int slot = k_unit % kUnitSlots, slot_use = k_unit / kUnitSlots;
            if (slot_use > 0)
                ok = mbar_wait_bounded(bar_unit_free + 8 * slot, (uint32_t)(slot_use - 1) & 1u, p.status, true);
            ok = __all_sync(kAll, ok);
            if (!ok) break;
            int32_t *u = units + slot * 16;
            const int base = cur.r.ctx - cur.r.n;
            cur.nb = min(cur.nb, ((cur.r.ctx + B - 1) >> bshift) - cur.b0);
            const int n_tok = last ? 0 : min(cur.r.ctx, (cur.b0 + cur.nb) << bshift) - (cur.b0 << bshift);
            if (lane == 0) {
                u[0] = cur.s;
                u[1] = cur.h;
                u[2] = cur.gp;
                u[3] = cur.parts;
                u[4] = cur.b0 << bshift;                     // first token
                u[5] = n_tok;                                // tokens
                u[6] = base;
                u[7] = cur.r.n;
                u[8] = cur.r.row0;
                u[9] = tile;
            }
            if (lane == 0) mbar_arrive(bar_unit + 8 * slot);
            ++k_unit;
            if (last && (++ends == G)) break;
            if (last) continue;
            tile += (n_tok + kTile - 1) / kTile;
            const Pending nxt = prepare(k_unit * n_ctas + (k_unit & 1 ? n_ctas - 1 - (int)blockIdx.x : (int)blockIdx.x));
            const int32_t *trow = p.block_tables + (size_t)cur.s * p.max_blocks + cur.b0;
            int tbl = cur.tbl;
            for (int b = 0; b < cur.nb; b += bps) {
                if (b > 0 && (b & 31) == 0) tbl = b + lane < cur.nb ? trow[b + lane] : -1;
                const int here = min(bps, cur.nb - b);
                // one lane a block of the tile
                const int phys = __shfl_sync(kAll, tbl, (b & 31) + (lane < here ? lane : 0));
                const bool good = lane < here && phys >= 0 && phys < p.num_blocks;
                const uint32_t bytes = (uint32_t)__popc(__ballot_sync(kAll, good)) * blk_bytes;
                if (lane < here && !good) report(p.status, PA_ERR_BAD_BLOCK);
                const int grp = (phys * H + cur.h) * run;
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {         // the keys' stage, the values' stage
                    if (!stage()) break;
                    const uint32_t full = bar_full + 8 * st;
                    if (lane == 0) {
                        if (bytes) mbar_arrive_expect_tx(full, bytes);
                        else mbar_arrive(full);
                    }
                    __syncwarp();
                    if (good)
                        tma_load_4d(ring + st * HALF + lane * blk_bytes, kv ? &maps.v : &maps.k, grp, full, policy);
                    ++issued;
                    if (++st == stages) {
                        st = 0;
                        ++use;
                    }
                }
                if (!ok) break;
            }
            if (!ok) break;
            cur = nxt;
        }
        if (!ok) {   // every issued copy lands before the CTA can exit
            if (lane == 0) report(p.status, PA_ERR_TIMEOUT);
            for (int k = max(0, issued - stages); k < issued; ++k)
                mbar_wait_bounded(bar_full + 8 * (k % stages), (uint32_t)(k / stages) & 1u, p.status, false);
        }
    } else if (warp == Cfg::Q_WARP) {
        // ================================================ queries
        // Q of each unit, and which nodes see each node, by a warp of their own:
        // the unit's keys and values need neither, and are on their way.
        uint32_t k = 0;
        for (;; ++k) {
            const int slot = k % kUnitSlots, buf = k % QB;
            ok = __all_sync(kAll, mbar_wait_bounded(bar_unit + 8 * slot, (k / kUnitSlots) & 1u, p.status, true));
            if (!ok) break;
            const int32_t *u = units + slot * 16;
            const int n_tok = u[5], h = u[1];
            const bool edge = u[4] + n_tok > u[6];           // the unit has nodes among its positions
            const SeqRows r = {u[7], u[8], u[6] + u[7]};
            if (n_tok <= 0) break;
            if (k >= QB) ok = mbar_wait_bounded(bar_q_free + 8 * buf, (k / QB - 1) & 1u, p.status, true);
            ok = __all_sync(kAll, ok);
            if (!ok) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(bar_q + 8 * buf, Cfg::Q_BYTES);
#pragma unroll
                for (int pn = 0; pn < NP; ++pn)
                    tma_load_3d(sQ + buf * Cfg::Q_BYTES + pn * NQ * 128, &maps.q, pn * 64, h, r.row0,
                                bar_q + 8 * buf);
            }
            if (edge) nodes_seen_by<SCORES>(p, r, lane, seen + slot * NQ);
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar_seen + 8 * slot);
                mbar_arrive(bar_unit_free + 8 * slot);
            }
        }
        if (!ok && lane == 0) report(p.status, PA_ERR_TIMEOUT);
        // the last copies have landed
        for (uint32_t i = k >= QB ? k - QB : 0; i < k; ++i)
            mbar_wait_bounded(bar_q + 8 * (i % QB), (i / QB) & 1u, p.status, false);
        __syncwarp();
    } else if (warp == Cfg::PRODUCTS) {
        // ================================================ products
        // Order: S of tile t + 1 before O of tile t, so that the softmax of a
        // tile finds its S ready; S and P have two buffers, taken in turn.  The
        // warp goes along together and one lane issues: its operands then lie
        // in uniform registers.  (With one lane going alone a product took 100
        // clocks to issue, so 60 to 75.)
        constexpr uint32_t idS = tc::idesc_f16(kTile, NQ, false);
        constexpr uint32_t idO = tc::idesc_f16(128, NQ, true) | (1u << 15);   // both MN-major
        int st = 0, st_v = 1;            // stage of the next keys; of the next values
        uint32_t use = 0, use_v = 0, gs = 0, gp = 0;   // tiles whose S, whose O was issued
        uint32_t q_buf = 0, s_set = 0;   // of the unit whose S is issued: its Q, its group
        auto wait = [&](uint32_t bar, uint32_t parity) {
            ok = __all_sync(kAll, ok && mbar_wait_bounded(bar, parity, p.status, true));
            return ok;
        };
        auto step = [&](int &i, uint32_t &n) {
            i += 2;
            if (i >= stages) {
                i -= stages;
                ++n;
            }
        };
        // S (tokens x rows) = K Q^T; the unit's last: Q is not needed any more
        auto issue_s = [&](bool last) {
            if (!wait(bar_full + 8 * st, use & 1u)) return;
            tc::fence_after();
            const uint64_t dk = tc::smem_desc(ring + st * HALF, 16, 1024u * NP);
            const uint64_t dq = tc::smem_desc(sQ + q_buf * Cfg::Q_BYTES, 16, 1024);
            const uint32_t d = tmem + Cfg::S_COL + (gs & 1) * NQ;
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    tc::mma_ss(d, dk + (((kk >> 2) * 1024 + (kk & 3) * 32) >> 4),
                               dq + (((kk >> 2) * NQ * 128 + (kk & 3) * 32) >> 4), idS, kk > 0 ? 1u : 0u);
                tc::commit(bar_empty + 8 * st);
                tc::commit(bar_s + 16 * s_set + 8 * (gs & 1));
                if (last) tc::commit(bar_q_free + 8 * q_buf);
            }
            __syncwarp();
            ++gs;
            step(st, use);
        };
        // O (dims x rows) += V^T P^T: tile t of n of the unit of a group
        auto issue_o = [&](int t, int n, int node_tile, uint32_t group) {
            if (!wait(bar_full + 8 * st_v, use_v & 1u) || !wait(bar_p + 8 * (gp & 1), (gp >> 1) & 1u)) return;
            tc::fence_after();
            const uint64_t dv = tc::smem_desc(ring + st_v * HALF, 1024, 1024u * NP);
            const uint64_t dp = tc::smem_desc(sP + (gp & 1) * Cfg::P_BYTES, 1024, 1024);
            const uint32_t d = tmem + Cfg::O_COL + (2 * group + (t < node_tile ? 0 : 1)) * NQ;
            const uint32_t more = t > 0 && t != node_tile ? 1u : 0u;
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < kTile / 16; ++kk)
                    tc::mma_ss(d, dv + ((kk * 2048u * NP) >> 4), dp + ((kk * 2048u) >> 4), idO, kk > 0 ? 1u : more);
                tc::commit(bar_empty + 8 * st_v);
                if (t + 1 == n) tc::commit(bar_o + 8 * group);
            }
            __syncwarp();
            ++gp;
            step(st_v, use_v);
        };
        uint32_t k = 0;                                  // units begun
        int ns = 0, node_s = 0;                          // the last one's tiles, its first with nodes
        // Begins the next unit; false: there is none.
        auto open = [&]() {
            const int slot = k % kUnitSlots;
            ns = 0;
            if (!wait(bar_unit + 8 * slot, (k / kUnitSlots) & 1u)) return false;
            ns = __shfl_sync(kAll, (units[slot * 16 + 5] + kTile - 1) / kTile, 0);
            node_s = __shfl_sync(kAll, first_node_tile(slot), 0);
            if (lane == 0) mbar_arrive(bar_unit_free + 8 * slot);
            q_buf = k % QB;
            s_set = k % G;
            return ns > 0 && wait(bar_q + 8 * q_buf, (k++ / QB) & 1u);
        };
        if constexpr (G == 1) {
            while (open()) {
                issue_s(ns == 1);
                for (int t = 0; ok && t < ns; ++t) {
                    if (t + 1 < ns) issue_s(t + 2 == ns);
                    issue_o(t, ns, node_s, 0);
                }
            }
        } else {
            // S goes ahead into the next unit, the other group's, where that is
            // at hand.  (One place for each product: with a copy for every case
            // their instructions were waited for, 158 us instead of 151 for 256
            // sequences of 100 positions.)
            int ts = 0, to = 0, no = 0, node_o = 0;      // next tile of S's unit; of O's, its tiles
            int n_before = 0, node_before = 0;           // of the unit before S's
            uint32_t k_o = 0;                            // units whose O was begun
            auto at_hand = [&]() {
                return __all_sync(kAll, mbar_test(bar_unit + 8 * (k % kUnitSlots), (k / kUnitSlots) & 1u) &&
                                            mbar_test(bar_q + 8 * (k % QB), (k / QB) & 1u) &&
                                            mbar_test(bar_full + 8 * st, use & 1u));
            };
            while (ok) {
                if (ts == ns && (gs == gp || at_hand())) {
                    n_before = ns;
                    node_before = node_s;
                    ts = 0;
                    if (!open()) break;                  // (the end has no Q: never at hand before O is done)
                }
                if (ts < ns && gs - gp < 2) {
                    issue_s(++ts == ns);
                    if (gs - gp < 2) continue;
                }
                if (to == no) {
                    const bool latest = k_o + 1 == k;
                    to = 0;
                    no = latest ? ns : n_before;
                    node_o = latest ? node_s : node_before;
                    ++k_o;
                }
                issue_o(to, no, node_o, (k_o - 1) % G);
                ++to;
            }
        }
        if (elect_one()) {
            if (!ok) report(p.status, PA_ERR_TIMEOUT);
            tc::commit(bar_done);   // lets the teardown wait for every product issued
        }
        __syncwarp();
    } else {
        // ================================================ softmax warps
        // Thread = token of the tile (then, for O, dimension of the head) and
        // CQ of the rows.  The warps go through barriers together: a wait that
        // fails only clears ok until the next vote.
        const int group = G == 2 ? warp >> 2 : 0, id = tid - group * ST;
        const int tok = id & 127, col0 = (id >> 7) * CQ;
        float *red = reinterpret_cast<float *>(smem + Cfg::RED) + group * 4 * NQ;
        float *ref = reinterpret_cast<float *>(smem + Cfg::REF) + group * 2 * NQ, *corr = ref + NQ;
        const uint32_t o_col = Cfg::O_COL + group * 2 * NQ;
        // (this group's, so that a wait for a tile to come cannot take an earlier
        // tile of the other group's for it)
        uint32_t s_phase = 0;                            // parities of this group's S barriers
        float *odd_at = reinterpret_cast<float *>(                // for node_tiles
            tiles_at + stages * HALF + (G == 2 ? 2 * Cfg::P_BYTES + QB * Cfg::Q_BYTES + group * Cfg::ODD_BYTES : 0));
        const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const float qs = p.qscale;
        auto wait = [&](uint32_t bar, uint32_t parity) {
            ok = __all_sync(kAll, ok && mbar_wait_bounded(bar, parity, p.status, true));
        };
        // CQ columns of this thread's lane
        auto load_cols = [&](uint32_t col, float (&v)[CQ]) {
            uint32_t r[CQ];
            __syncwarp();
            if constexpr (CQ == 16) tc::ld16(lane_base + col + col0, r);
            else tc::ld32(lane_base + col + col0, r);
            tc::wait_ld();
#pragma unroll
            for (int i = 0; i < CQ; ++i) v[i] = __uint_as_float(r[i]);
        };
        for (uint32_t k = group;; k += G) {
            const int slot = k % kUnitSlots;
            wait(bar_unit + 8 * slot, (k / kUnitSlots) & 1u);
            if (!softmax_all<ST>(group, ok)) break;
            const int32_t *u = units + slot * 16;
            const int s = u[0], h = u[1], part = u[2], parts = u[3], tok_first = u[4], n_tok = u[5], base = u[6],
                      n = u[7], row0 = u[8];
            if (n_tok <= 0) break;                       // the end
            const int have = n - col0;                   // rows of this thread's that exist
            uint32_t g = u[9];                           // tile, counted over all units
            const int node_tile = first_node_tile(slot);
            bool knows = false;                          // who sees the nodes is there
            float l[R], off[R];                          // running sums; minus the rows' references
#pragma unroll
            for (int i = 0; i < R; ++i) l[i] = off[i] = 0.f;
            for (int t0 = 0; t0 < n_tok; t0 += kTile) {
                const int nv = min(kTile, n_tok - t0);
                const int pos = tok_first + t0 + tok;
                const uint32_t b = g & 1;
                wait(bar_s + 16 * group + 8 * b, (G == 1 ? g >> 1 : s_phase >> b) & 1u);
                if (G == 2) s_phase ^= 1u << b;
                tc::fence_after();
                if (tok_first + t0 + kTile > base && !knows) {
                    wait(bar_seen + 8 * slot, (k / kUnitSlots) & 1u);
                    knows = true;
                }
                // -inf where the row does not see this position
                auto hide = [&](auto &x) {
                    if (tok_first + t0 + kTile > base || nv < kTile) {
                        // who sees it: every row before the nodes, then the node
                        // itself and its descendants; none past the end
                        const uint64_t v = (tok >= nv ? 0ull : pos < base ? ~0ull : seen[slot * NQ + pos - base]) >> col0;
#pragma unroll
                        for (int i = 0; i < R; ++i)
                            if (!((v >> i) & 1)) x[i] = -INFINITY;
                    }
                };
                // the tile's products, then its scores less the references (by
                // one rounding on every way here, so that a row does not depend
                // on whether another's reference moves)
                float y[CQ];
                auto scores = [&]() {
#pragma unroll
                    for (int i = 0; i < R; ++i) y[i] = fmaf(y[i], qs, off[i]);
                    hide(y);
                };
                load_cols(Cfg::S_COL + b * NQ, y);
                if (SCORES && tok < nv) p.scores[((size_t)s * H + h) * p.score_stride + pos] = y[0] * qs;
                // a row's reference moves when a score passes it by more than 2^15
                bool over = false;
                if (t0 > 0) {
                    scores();
                    float top = -INFINITY;
#pragma unroll
                    for (int c = 0; c < R; c += 8)
                        if (c < have) {
#pragma unroll
                            for (int i = c; i < c + 8 && i < R; ++i) top = fmaxf(top, y[i]);
                        }
                    over = top > kRescaleLog2;
                }
                if (t0 == 0 || softmax_any<ST>(group, over || !ok)) {
                    if (!softmax_all<ST>(group, ok)) break;
                    if (t0 > 0) load_cols(Cfg::S_COL + b * NQ, y);
                    float m[R];                          // the scores themselves
#pragma unroll
                    for (int i = 0; i < R; ++i) m[i] = y[i] * qs;
                    hide(m);
                    const int first = warp_combine(m, lane, [](float a, float c) { return fmaxf(a, c); });
#pragma unroll
                    for (int i = 0; i < (R + 31) / 32; ++i) red[(warp & 3) * NQ + col0 + first + i] = m[i];
                    softmax_sync<ST>(group);
                    if (id < (SCORES ? 1 : NQ)) {
                        const float top = fmaxf(fmaxf(red[id], red[NQ + id]), fmaxf(red[2 * NQ + id], red[3 * NQ + id]));
                        // (a row that has seen nothing yet has reference -2^100: its
                        // terms, if any come, are rescaled from 0; a column that
                        // is no row, and holds the next sequence's scores, has no
                        // terms and never moves)
                        const float old = t0 ? ref[id] : -0x1p100f, now = top > old + kRescaleLog2 ? top - kBelowLog2 : old;
                        ref[id] = id < n ? now : INFINITY;
                        corr[id] = id < n ? ex2(old - now) : 0.f;
                    }
                    softmax_sync<ST>(group);
#pragma unroll
                    for (int i = 0; i < R; ++i) off[i] = -ref[col0 + i];
                    if (t0 > 0) {
#pragma unroll
                        for (int i = 0; i < R; ++i) l[i] *= corr[col0 + i];
                        // O, complete up to the tile before once that gave its
                        // values' stage back
                        const uint32_t v = 2 * g - 1;            // (stage 2 t + 1 of all holds tile t's)
                        wait(bar_empty + 8 * (v % stages), (v / stages) & 1u);
                        tc::fence_after();
#pragma unroll 1
                        for (int half = node_tile == 0; half <= (t0 > node_tile * (int64_t)kTile); ++half) {
                            float o[CQ];
                            load_cols(o_col + half * NQ, o);
#pragma unroll
                            for (int i = 0; i < R; ++i) o[i] *= corr[col0 + i];
                            uint32_t r[CQ];
#pragma unroll
                            for (int i = 0; i < CQ; ++i) r[i] = __float_as_uint(o[i]);
                            __syncwarp();
                            if constexpr (CQ == 16) tc::st16(lane_base + o_col + half * NQ + col0, r);
                            else tc::st32(lane_base + o_col + half * NQ + col0, r);
                        }
                        tc::wait_st();
                    }
                    // (32 rows a thread do not stay in registers up to here: spilled
                    // they cost more than the second load, 785 instead of 771 us
                    // for 256 sequences of 64 nodes)
                    if constexpr (R > 16) load_cols(Cfg::S_COL + b * NQ, y);
                    scores();
                }
                // P of the tile: this token's row, in the second operand's layout
                uint32_t w[(R + 7) / 8 * 4];
                if constexpr (SCORES) {
                    const float p0 = ex2(y[0]);
                    l[0] += p0;
                    w[0] = pack_half2(p0, 0.f);
                    w[1] = w[2] = w[3] = 0;
                } else {
#pragma unroll
                    for (int c = 0; c < R; c += 8)
                        if (c < have) {
#pragma unroll
                            for (int i = c; i < c + 8; i += 2) {
                                const float p0 = ex2(y[i]), p1 = ex2(y[i + 1]);
                                l[i] += p0;
                                l[i + 1] += p1;
                                w[i / 2] = pack_half2(p0, p1);
                            }
                        }
                }
                // (the product that read this buffer's last P is done: this tile's S
                // was issued after it)
                const uint32_t prow = sP + b * Cfg::P_BYTES + (uint32_t)tok * 128u;
#pragma unroll
                for (int c = 0; c < R; c += 8)
                    if (c < have)
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                                         prow + (uint32_t)((((col0 + c) >> 3) ^ (tok & 7)) << 4)),
                                     "r"(w[c / 2]), "r"(w[c / 2 + 1]), "r"(w[c / 2 + 2]), "r"(w[c / 2 + 3])
                                     : "memory");
                if (nv < kTile) {
                    // values past the end meet P = 0 and have to be finite: zeros
                    const uint32_t v = 2 * g + 1, st_v = v % stages;
                    wait(bar_full + 8 * st_v, (v / stages) & 1u);
                    if (tok >= nv && col0 == 0) {
                        const uint32_t row = ring + st_v * HALF + (uint32_t)(tok >> 3) * (NP * 1024u) +
                                             (uint32_t)(tok & 7) * 128u;
#pragma unroll
                        for (int c = 0; c < NP * 8; ++c)
                            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                             row + (uint32_t)(c >> 3) * 1024u + (uint32_t)(c & 7) * 16u),
                                         "r"(0)
                                         : "memory");
                    }
                }
                fence_proxy_async_smem();
                tc::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_p + 8 * b);
                ++g;
            }
            // sums over the tokens
            const int first = warp_combine(l, lane, [](float a, float c) { return a + c; });
#pragma unroll
            for (int i = 0; i < (R + 31) / 32; ++i) red[(warp & 3) * NQ + col0 + first + i] = l[i];
            if (!softmax_all<ST>(group, ok)) break;
            const bool nodes = node_tile != INT_MAX;
            if (lane == 0 && !nodes) mbar_arrive(bar_unit_free + 8 * slot);
            const size_t part_row = ((size_t)part * H + h) * NQ;
            if (id < (SCORES ? 1 : NQ)) {
                const float sum = (red[id] + red[NQ + id]) + (red[2 * NQ + id] + red[3 * NQ + id]);
                corr[id] = 1.f / sum;
                if (parts > 1 && id < n) p.ws_ml[part_row + id] = make_float2(ref[id], sum);
                if (SCORES && parts == 1) p.ml_one[(size_t)s * H + h] = make_float2(ref[0], sum);
            }
            softmax_sync<ST>(group);
            wait(bar_o + 8 * group, (k / G) & 1u);
            tc::fence_after();
            float o[CQ];
            if (!nodes) {
                load_cols(o_col, o);
            } else {
                load_cols(o_col + NQ, o);
                // (0 times a value that is not finite leaves no row's sum finite)
                bool odd = tok < D && have > 0 && !isfinite(o[0]);
                const bool some = softmax_any<ST>(group, odd);
                if (some) {
#pragma unroll
                    for (int i = 0; i < CQ; ++i) odd = odd && (i >= have || !isfinite(o[i]));
                    float again[CQ];
#pragma unroll
                    for (int i = 0; i < CQ; ++i) again[i] = o[i];
                    node_tiles<D, NQ, G>(p, u, seen + slot * NQ, ref,
                                      odd_at, odd, again);
#pragma unroll
                    for (int i = 0; i < CQ; ++i) o[i] = again[i];
                }
                if (lane == 0) mbar_arrive(bar_unit_free + 8 * slot);
                if (node_tile > 0) {
                    float before[CQ];
                    load_cols(o_col, before);
#pragma unroll
                    for (int i = 0; i < CQ; ++i) o[i] += before[i];
                }
            }
            if (tok < D) {                               // thread = dimension
                if (parts == 1) {
                    __half *dst = p.out + ((size_t)(row0 + col0) * H + h) * D + tok;
#pragma unroll
                    for (int i = 0; i < R; ++i)
                        if (i < have) dst[(size_t)i * H * D] = __float2half(o[i] * corr[col0 + i]);
                } else {
                    float *dst = p.ws_acc + (part_row + col0) * D + tok;
#pragma unroll
                    for (int i = 0; i < R; ++i)
                        if (i < have) dst[i * D] = o[i];
                }
            }
            __syncwarp();
        }
        if (!ok && lane == 0) report(p.status, PA_ERR_TIMEOUT);
        __syncwarp();
    }

    // ---- teardown: every product drained (bounded), then tensor memory freed
    __syncwarp();
    tc::fence_before();
    __syncthreads();
    if (warp == Cfg::PRODUCTS) {
        if (lane == 0 && !mbar_wait_bounded(bar_done, 0, p.status, false)) report(p.status, PA_ERR_TIMEOUT);
        __syncwarp();
        tc::fence_after();
        tc::dealloc(tmem, Cfg::COLS);
    }
}

// -------------------------------------------------------- joining the parts

// One warp per (cut sequence, head, row): m = max m_p, l = sum 2^(m_p - m) l_p,
// o = sum 2^(m_p - m) acc_p / l.
template <int D>
__global__ void __launch_bounds__(256) tree_join_kernel(const TreeParams p, int NR) {
    constexpr int DL = D / 32;
    const int lane = threadIdx.x & 31, H = p.num_heads;
    wait_for_launch_before();
    const long long items = (long long)p.header[0] * H * NR;
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
    wait_for_launch_before();
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
// rows of one head.
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

// Queries as [rows][H][D] with a box of 64 columns of one head of box_rows rows.
int encode_queries(CUtensorMap *m, const void *base, int rows, int H, int D, int box_rows, const char *who) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = map_encoder();
    if (!enc) return fail(PA_ERR_CUDA, "%s: cuTensorMapEncodeTiled unavailable", who);
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)rows};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)H * D * 2};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)box_rows}, elem[3] = {1, 1, 1};
    const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void *>(base), dims, strides, box,
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

// Query rows of a launch, padded to what a product's N takes.
int padded_rows(int max_q) { return max_q <= 16 ? 16 : max_q <= 32 ? 32 : 64; }

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Parts of cut sequences a launch can have: each is at least half of a
// quarter of an SM's share of the blocks.
int part_cap(int n_seqs, int max_blocks, int H) {
    return (int)std::min<int64_t>(8ll * sm_count() / H + 8, (int64_t)n_seqs * std::max(max_blocks, 1));
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

// A launch that may begin while the kernel before it ends.
template <typename... Args>
cudaError_t launch_after(void (*kern)(Args...), dim3 grid, cudaStream_t st, Args... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <int D, int NQ, bool SCORES, int G>
int launch_groups(TreeParams p, const TreeMaps &maps, const char *who, cudaStream_t st) {
    using Cfg = TreeCfg<D, NQ, G>;
    auto kern = tree_attention_kernel<D, NQ, SCORES, G>;
    constexpr int kBytes = 227 * 1024;
    static std::once_flag once[kMaxDevs];
    static cudaError_t err[kMaxDevs];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevs)
        return fail(PA_ERR_CUDA, "%s: cudaGetDevice failed", who);
    std::call_once(once[dev], [&] {
        err[dev] = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
    });
    if (err[dev] != cudaSuccess)
        return fail(PA_ERR_CUDA, "%s: cudaFuncSetAttribute: %s", who, cudaGetErrorString(err[dev]));
    p.stages = std::min(kMaxStages, (kBytes - Cfg::bytes(p.n_seqs, 0)) / Cfg::HALF);
    static_assert((kBytes - Cfg::bytes(PA_TREE_MAX_SEQS, 0)) / Cfg::HALF >= kMinStages,
                  "room beside the largest batch's plan");
    kern<<<sm_count(), Cfg::THREADS, Cfg::bytes(p.n_seqs, p.stages), st>>>(p, maps);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return fail(PA_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
    return PA_OK;
}

// Two groups of softmax warps where sequences make two units or more a CTA without
// being cut: 256 sequences x 40 heads of 100 positions 151 us instead of 204, 4096 x
// 2 of 40 137 instead of 170, and no difference where units are long (64 sequences,
// 1000 on average: 218 both).  One where each CTA has a unit or two, all long: 8
// heads' 20000 positions 21.2 us instead of 23.3.  Above 16 rows two groups'
// registers do not fit.
template <int D, int NQ, bool SCORES>
int launch_tree(const TreeParams &p, const TreeMaps &maps, const char *who, cudaStream_t st) {
    if constexpr (NQ == 16)
        if ((int64_t)p.n_seqs * p.num_heads >= 2 * sm_count()) return launch_groups<D, NQ, SCORES, 2>(p, maps, who, st);
    return launch_groups<D, NQ, SCORES, 1>(p, maps, who, st);
}

// Checks and the main launch that both entry points share.
int launch_common(const char *who, bool weights, TreeParams &p, const void *k_cache, const void *v_cache,
                  void *workspace, size_t workspace_bytes, int max_q, const pa_pool_desc *d, cudaStream_t st) {
    const int NR = padded_rows(max_q), B = d->block_size;
    p.cap = part_cap(p.n_seqs, p.max_blocks, d->num_heads);
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
    p.k_cache = static_cast<const __half *>(k_cache);
    p.v_cache = static_cast<const __half *>(v_cache);
    int rc = encode_cache(&maps.k, k_cache, groups, d->head_dim, B / 8, who);
    if (rc == PA_OK) rc = encode_cache(&maps.v, v_cache, groups, d->head_dim, B / 8, who);
    if (rc == PA_OK) rc = encode_queries(&maps.q, p.q, p.q_rows, d->num_heads, d->head_dim, NR, who);
    if (rc != PA_OK) return rc;
    if (d->head_dim == 64) {
        if (weights) return launch_tree<64, 16, true>(p, maps, who, st);
        return NR == 16 ? launch_tree<64, 16, false>(p, maps, who, st)
             : NR == 32 ? launch_tree<64, 32, false>(p, maps, who, st)
                        : launch_tree<64, 64, false>(p, maps, who, st);
    }
    if (weights) return launch_tree<128, 16, true>(p, maps, who, st);
    return NR == 16 ? launch_tree<128, 16, false>(p, maps, who, st)
         : NR == 32 ? launch_tree<128, 32, false>(p, maps, who, st)
                    : launch_tree<128, 64, false>(p, maps, who, st);
}

bool mis(const void *ptr, int n) { return (reinterpret_cast<uintptr_t>(ptr) & (n - 1)) != 0; }

}  // namespace

size_t tree_workspace_bytes(int32_t n_seqs, int32_t max_blocks, int32_t max_q_len, const pa_pool_desc *d) {
    std::string why;
    if (!d || n_seqs <= 0 || n_seqs > PA_TREE_MAX_SEQS || max_blocks < 0 || max_q_len < 1 ||
        max_q_len > PA_TREE_MAX_NODES || !tree_geometry_ok(d, &why))
        return 0;
    return sections(n_seqs, max_blocks, padded_rows(max_q_len), part_cap(n_seqs, max_blocks, d->num_heads), false, d)
        .total;
}

size_t decode_weights_workspace_bytes(int32_t n_seqs, int32_t max_blocks, const pa_pool_desc *d) {
    std::string why;
    if (!d || n_seqs <= 0 || n_seqs > PA_TREE_MAX_SEQS || max_blocks < 0 || !tree_geometry_ok(d, &why)) return 0;
    return sections(n_seqs, max_blocks, padded_rows(1), part_cap(n_seqs, max_blocks, d->num_heads), true, d).total;
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
    if (d->num_blocks < 1 || max_blocks < 1 || (int64_t)max_blocks * d->block_size > INT32_MAX - kTile)
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
    const int NR = padded_rows(max_q_len);
    const int blocks = (int)std::min<int64_t>((int64_t)p.cap * d->num_heads * NR / 8 + 1, (int64_t)sm_count() * 4);
    const cudaError_t e = launch_after(d->head_dim == 64 ? tree_join_kernel<64> : tree_join_kernel<128>, dim3(blocks),
                                       st, p, NR);
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
    if (d->num_blocks < 1 || max_blocks < 1 || (int64_t)max_blocks * d->block_size > INT32_MAX - kTile)
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
    const auto kern = d->head_dim == 64 ? (vec ? decode_weights_kernel<64, true> : decode_weights_kernel<64, false>)
                                        : (vec ? decode_weights_kernel<128, true> : decode_weights_kernel<128, false>);
    const cudaError_t e = launch_after(kern, grid, st, p, padded_rows(1), weights_out, weights_in);
    if (e != cudaSuccess) return fail(PA_ERR_CUDA, "%s: weights launch: %s", who, cudaGetErrorString(e));
    return PA_OK;
}

}  // namespace pagedkv
