// Decode attention over a cache in 8 or 4 bits with grouped query heads
// (definition in include/pagedkv.h).
//
// Mathematics.  With codes c and scales s (32 dimensions a scale, group g of a row),
//     q . k_p = sum_g s_pg (sum_{d in g} q_d c_pd),   o_d = sum_p (w_p s_pg) c_pd / sum_p w_p,
// so both products run on the codes alone, which are exact in fp16, and the
// scales meet a product's result (keys) or a position's weight (values).  The
// weights are 2^(y_p - R) with a reference R that follows the running maximum, and
// in R stands a power of two that lifts weight * scale into the middle of fp16's
// range, where it is rounded once to be the second product's operand.
//
// What bounds it: a position of a key/value head is 144 bytes in 4 bits (D = 128) and
// 256 codes, 47 G positions a second at the copy's rate: the bytes bound it as long as a
// code costs less than an instruction of a lane.  So the codes never leave
// registers: a warp's matrix instructions (m16n8k16) take 16 positions (keys) or 16
// dimensions (values) as rows and up to 8 query heads as columns, their A fragments
// made in place from the packed words by a shift and a three-input logic operation
// that puts a code into an fp16 mantissa (1024 + 4 n or 1024 + 64 n; queries are
// divided by 4 or 64 beforehand, and one more product takes the constants' share off
// the scores), or, for values, one more FMA that centres it.  An
// operand for tcgen05 would have to be widened the same way and then be stored in shared
// or tensor memory, four times the bytes that came in.
//
// Work: a warp of four takes one key/value head (or fewer heads and a share of the
// positions, or 8 more of its query heads) of a stage that a fifth warp fills by
// bulk copies through the block table.  The batch's (sequence, head group, tile of
// positions) are laid end to end and every CTA takes an equal stretch of them, so
// no CTA ends late; a stretch that begins or ends inside a sequence leaves a partial
// result, at most two a CTA, and a second kernel, launched ahead, joins them.
//
// Measured (calls one after another in a graph): 256 sequences of 128 to 4096 positions, 8
// heads of keys for 64 of queries, 8 bits: 181 us, 6.5 TB/s; 64 of 128 to 2048, 40 heads,
// 4 bits: 74.8 us, 5.5 TB/s, where the arithmetic on the codes (56 % of the issue slots with
// twelve warps an SM) no longer hides behind the bytes; one of 2048: 9.0 us, latency. The
// pairs of figures at the choices below are from when each was made.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <mutex>
#include <type_traits>

#include "pa_internal.h"
#include "quant_device.cuh"

namespace pagedkv {

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kWarps = 4;                       // that compute; one more copies
constexpr int kThreads = (kWarps + 1) * 32;
// CTAs of an SM.  Codes of 4 bits take three CTAs' warps to widen as fast as they come (64
// mixed sequences 84 us, two CTAs 94), codes of 8 bits come no faster with three, and
// two leave fewer parts to join (256 grouped ones 198 us, two CTAs 190).
__host__ __device__ constexpr int ctas_of(int bits) { return bits == 4 ? 3 : 2; }
// Shared memory of a CTA, beside what is static.
__host__ __device__ constexpr int smem_of(int bits) { return 233472 / ctas_of(bits) - 1536; }
constexpr int kMaxStages = 8;
constexpr int kMaxCtas = 1024;                  // of a launch
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.f;                   // a weight may grow to 2^8 before R moves
constexpr int kLift = 6;                        // scales are lifted below 2^(kLift + 1)
// Scores (base 2) from here on are rounded to steps that a reference with a lift in it would
// miss: their maximum is taken off first, the lift comes after.
constexpr float kFar = 0x1p22f;

// What the copying warp tells the others of a stretch, a unit's tiles that the CTA takes.
struct Stretch {
    int tiles, positions;     // positions: from its first tile to the context's end
    int seq, unit, part;      // part: -1 for a whole context, otherwise where the partial result goes
};

struct QuantParams {
    void *out;
    const void *q;
    const uint8_t *k, *v;
    const int32_t *tables, *ctx;
    int n_seqs, max_blocks, num_blocks, H, Hq, rep, bshift, rec, bf16;
    float scale, sign;            // |scale|, and its sign
    int lg, lqg, lns;             // log2 of a CTA's heads, column groups, shares of a tile's positions
    int head_groups, col_passes;
    int rows;                     // query rows of a unit, at most
    int code_at[16], scale_at[16];  // where each 8 positions of a warp begin in a stage
    int stages, q_bytes;          // q_bytes: of one of two query buffers
    int4 *jobs;                   // first CTA, parts (below 2: nothing to join), sequence and unit of
    int by_unit;                  // every unit, or of every CTA's last stretch
    float2 *ml;                   // [2 CTA + ..][rows] reference and sum
    float *acc;                   // [..][rows][D]
    int32_t *status;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void mma(float d[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// starting from other sums
__device__ __forceinline__ void mma_from(float d[4], const float z[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(z[0]), "f"(z[1]), "f"(z[2]), "f"(z[3]));
}
__device__ __forceinline__ void mma_zero(float d[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    const float z[4] = {0.f, 0.f, 0.f, 0.f};
    mma_from(d, z, a0, a1, a2, a3, b0, b1);
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// (w & m) | c in one instruction
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t m, uint32_t c) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(w), "r"(m), "r"(c));
    return d;
}
template <int N>
__device__ __forceinline__ void lds(uint32_t at, uint32_t w[N]) {
    if constexpr (N == 1) asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(at));
    else if constexpr (N == 2) asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at));
    else {
#pragma unroll
        for (int i = 0; i < N; i += 4)
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3])
                         : "r"(at + i * 4));
    }
}

// The four fp16 pairs of a word of 8 codes, not centred: 1024 + 4 n for pairs 0
// and 2, 1024 + 64 n for 1 and 3; pair j holds codes j and j + 4.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t p[4]) {
    const uint32_t lo = w << 2, hi = w >> 6;
    p[0] = and_or(lo, 0x003c003cu, 0x64006400u);
    p[1] = and_or(lo, 0x03c003c0u, 0x64006400u);
    p[2] = and_or(hi, 0x003c003cu, 0x64006400u);
    p[3] = and_or(hi, 0x03c003c0u, 0x64006400u);
}

constexpr uint32_t half2_const(int bits) { return (uint32_t)bits << 16 | (uint32_t)bits; }

// A key's piece of 8 codes as four pairs (pair j: codes j and j + 4 of 4-bit ones,
// 2 j and 2 j + 1 of 8-bit ones), and what queries of those pairs are divided by.
template <int BITS>
__device__ __forceinline__ void key_pairs(const uint32_t *w, uint32_t p[4]) {
    if constexpr (BITS == 4) {
        widen4(w[0], p);
    } else {
        p[0] = __byte_perm(w[0], 0x64646464u, 0x4140);       // 1024 + n
        p[1] = __byte_perm(w[0], 0x64646464u, 0x4342);
        p[2] = __byte_perm(w[1], 0x64646464u, 0x4140);
        p[3] = __byte_perm(w[1], 0x64646464u, 0x4342);
    }
}
// what pair j of code 0 looks like
template <int BITS>
__device__ __forceinline__ constexpr uint32_t key_zero(int j) {
    return BITS == 8 ? half2_const(0x6480) : (j & 1) ? half2_const(0x6600) : half2_const(0x6420);  // 1152, 1536, 1056
}
template <int BITS>
__device__ __forceinline__ constexpr float key_divide(int j) {
    return BITS == 8 ? 1.f : (j & 1) ? 1.f / 64 : 1.f / 4;
}

// Codes of 4 dimensions of two positions as pairs (position a, position b), centred; of
// 4-bit ones, codes 0 and 2 with 16 times codes 1 and 3.
template <int BITS>
__device__ __forceinline__ void value_pairs(uint32_t a, uint32_t b, uint32_t pick, uint32_t p[4]) {
    if constexpr (BITS == 4) {
        // Whole bytes 16 n' + n, centred, in the place of the lower codes, which the sums' difference
        // gives at the end (one operation of six fewer than the codes apart: 76.0 us
        // for 64 mixed sequences, 73.7 so).
        const uint32_t x = __byte_perm(a, b, pick), y = __byte_perm(x, 0x64646464u, 0x4341);   // y: 1024 + upper bytes
        p[0] = hadd2(and_or(x, 0x00ff00ffu, 0x64006400u), half2_const(0xe488));                         // - 1160
        p[1] = hfma2(and_or(x, 0x00f000f0u, 0x64006400u), half2_const(0x2c00), half2_const(0xd480));    // / 16 - 72
        p[2] = hadd2(y, half2_const(0xe488));
        p[3] = hfma2(y & 0xfff0fff0u, half2_const(0x2c00), half2_const(0xd480));
    } else {
        const uint32_t lo = __byte_perm(a, b, 0x5140), hi = __byte_perm(a, b, 0x7362);
        p[0] = hadd2(__byte_perm(lo, 0x64646464u, 0x4140), half2_const(0xe480));   // - 1152
        p[1] = hadd2(__byte_perm(lo, 0x64646464u, 0x4342), half2_const(0xe480));
        p[2] = hadd2(__byte_perm(hi, 0x64646464u, 0x4140), half2_const(0xe480));
        p[3] = hadd2(__byte_perm(hi, 0x64646464u, 0x4342), half2_const(0xe480));
    }
}

// What scales up to these bits are lifted by, as a power of two.
__device__ __forceinline__ int lift_of(uint32_t bits) { return kLift + 15 - (int)(bits >> 10); }

__device__ __forceinline__ float half_at(uint32_t w, int i) {
    return __half2float(__ushort_as_half((unsigned short)(i ? w >> 16 : w & 0xffffu)));
}

// The position that row r of a matrix instruction's 8 rows stands for: neighbours
// differ in parity (a warp's 16-byte loads of keys cover all banks), and so do
// the even rows' two halves (values).
__device__ __forceinline__ int row_token(int r) { return r ^ ((r >> 1) & 1); }

// Positions of a sequence that are read; 0: nothing to do or refused.
__device__ __forceinline__ int length_of(const QuantParams &p, int s, bool tell) {
    const int c = p.ctx[s];
    if ((int64_t)c > ((int64_t)p.max_blocks << p.bshift)) {
        if (tell) report(p.status, PA_ERR_BAD_BLOCK);
        return 0;
    }
    return max(c, 0);
}

// Dividing a batch's T tiles, laid end to end, among CTAs: where CTA b's stretch begins,
// and whose stretch tile x is in.
struct Shares {
    unsigned long long each, more;    // tiles of every CTA; of these, how many take one more
    __device__ Shares(unsigned long long T, unsigned n) {
        each = T >> 32 ? T / n : (unsigned)T / n;
        more = T - each * n;
    }
    __device__ unsigned long long begin(unsigned b) const { return b * each + min((unsigned long long)b, more); }
    __device__ unsigned owner(unsigned long long x) const {
        const unsigned long long cut = more * (each + 1);
        const unsigned long long y = x < cut ? x : x - cut, d = x < cut ? each + 1 : each;
        return (unsigned)((y | d) >> 32 ? y / d : (unsigned)y / (unsigned)d) + (x < cut ? 0u : (unsigned)more);
    }
};

__device__ __forceinline__ void allow_next_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_launch_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// A bounded wait whose end is one for the whole warp: lanes see the timer and the
// status at different moments, and what follows a wait takes all lanes or none.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const int32_t *status) {
    return __all_sync(kAll, mbar_wait_bounded(bar, parity, status, true));
}

template <int D>
__device__ __forceinline__ void store4(const QuantParams &p, int64_t row, int d, float a, float b, float c, float e) {
    const uint2 w = p.bf16 ? make_uint2(quant::pack2<__nv_bfloat16>(a, b), quant::pack2<__nv_bfloat16>(c, e))
                           : make_uint2(quant::pack2<__half>(a, b), quant::pack2<__half>(c, e));
    *reinterpret_cast<uint2 *>((char *)p.out + (row * D + d) * 2) = w;
}

// MT: 16-position tiles of a warp in a stage.
// SETS: with 0 a column is a query head and an operand of queries (or of weights times
// scales) belongs to one group of 32 dimensions.  Otherwise a column is a query of one
// group, and SETS operands hold the groups (8 SETS / groups queries fit: up to two with 1
// and four with 2 of D = 128, four with 1 of D = 64).  The keys' products then leave a query's
// group sums side by side in two lanes (one where a set has two groups), which scale and
// add them once, and one operand of weights times scales serves a set's dimensions:
// the arithmetic between the products is a fourth or half of what it is otherwise.
template <int D, int BITS, int MT, int SETS>
__global__ void __launch_bounds__(kThreads, ctas_of(BITS)) quant_attention_kernel(const QuantParams p) {
    constexpr bool PACK = SETS > 0;
    constexpr int GR = D / 32;                 // groups of a row
    constexpr int RB = D * BITS / 8;           // bytes of a row's codes
    constexpr int SB = GR * 2;                 // and of its scales
    constexpr int NW = RB / 16;                // words of a lane's quarter of a row
    constexpr int WP = BITS / 4;               // words of 8 codes
    constexpr int NQ = PACK ? 1 : 2;           // queries of a lane
    constexpr int GS = PACK ? GR / SETS : 1;   // groups of a set
    constexpr int SW = PACK ? SETS : GR / 2;   // words of scales that a lane reads of a row
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages], q_empty[2], merged[kWarps];
    __shared__ Stretch stretch[2];
    __shared__ long long sums[kThreads / 32], start_rest;
    __shared__ int start_seq;                  // and start_rest: where this CTA's stretch begins: sequence, tile of its units

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = 1 << p.lg, NS = 1 << p.lns, B = 1 << p.bshift;
    const int TT = 16 * MT * NS;               // positions of a tile
    const int tshift = 4 + (MT == 1 ? 0 : MT == 2 ? 1 : MT == 4 ? 2 : 3) + p.lns;
    const int run = G * p.rec;                 // bytes of a block's heads
    const int half = (TT >> p.bshift) * run, stage_bytes = 2 * half;
    uint8_t *const q_at = smem + p.stages * stage_bytes;
    float *const merge_at = reinterpret_cast<float *>(q_at + 2 * p.q_bytes);

    allow_next_launch();
    wait_for_launch_before();
    // ---- this CTA's stretch of the batch
    const int per = (p.n_seqs + kThreads - 1) / kThreads, s_lo = min(p.n_seqs, tid * per),
              s_hi = min(p.n_seqs, s_lo + per);
    long long mine = 0;
    for (int s = s_lo; s < s_hi; ++s) mine += (length_of(p, s, blockIdx.x == 0) + TT - 1) >> tshift;
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(kAll, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) sums[warp] = incl;
    if (tid == 0) {
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(smem_addr(full + i), 1);
            mbar_init(smem_addr(empty + i), kWarps);
        }
        for (int i = 0; i < 2; ++i) mbar_init(smem_addr(q_empty + i), kWarps);
        for (int i = 0; i < kWarps; ++i) mbar_init(smem_addr(merged + i), NS);
        fence_barrier_init();
    }
    __syncthreads();
    long long before = incl - mine, total = 0;
    for (int i = 0; i < kThreads / 32; ++i) {
        if (i < warp) before += sums[i];
        total += sums[i];
    }
    const int units = p.head_groups * p.col_passes;
    const long long T = total * units;
    const Shares shares(T, gridDim.x);
    const long long w0 = shares.begin(blockIdx.x), w1 = shares.begin(blockIdx.x + 1);
    if (w1 > w0 && before * units <= w0 && w0 < (before + mine) * units) {
        long long at = before * units;
        for (int s = s_lo; s < s_hi; ++s) {
            const long long n = (long long)((length_of(p, s, false) + TT - 1) >> tshift) * units;
            if (w0 < at + n) {
                start_seq = s;
                start_rest = w0 - at;
                break;
            }
            at += n;
        }
    }
    __syncthreads();
    const int count = (int)(w1 - w0);

    if (warp == kWarps) {
        // ---- copies
        int4 job = make_int4(0, 0, 0, 0);      // a unit that begins here and ends elsewhere
        const uint64_t policy = l2_evict_first_policy();
        const int blocks = TT >> p.bshift;
        int s = start_seq, u = 0, tile = 0, ctx = 0, n = 0, issued = 0, st = 0, round = 0;
        if (count > 0) {
            ctx = length_of(p, s, false);
            n = (ctx + TT - 1) >> tshift;
            u = (int)(start_rest / n);
            tile = (int)(start_rest - (long long)u * n);
        }
        // a lane's block of a tile: its table entry, loaded a tile ahead
        auto entry = [&](int seq, int length, int t) {
            const int b = t * blocks + lane;
            return lane < blocks && b < (length + B - 1) >> p.bshift ? p.tables[(int64_t)seq * p.max_blocks + b] : -1;
        };
        int id = count > 0 ? entry(s, ctx, tile) : -1;
        bool ok = true;
        // (after a wait that gave up it goes on without copies: the second kernel reads
        // the entry of every unit that begins here)
        for (int seg = 0; issued < count; ++seg) {
            const int left = min(n - tile, count - issued), after = issued + left;     // tiles of this unit
            const bool whole = left == n;
            if (tile == 0) {
                // (up to the CTA that its last tile is in)
                const int parts = whole ? 1 : (int)shares.owner(w0 + issued + n - 1) - (int)blockIdx.x + 1;
                job = make_int4(blockIdx.x, parts, s, u);
                if (p.by_unit && lane == 0) p.jobs[(int64_t)s * units + u] = job;
            }
            const int part = whole ? -1 : 2 * (int)blockIdx.x + (tile == 0 ? 1 : 0);
            const int hg = p.col_passes == 1 ? u : u / p.col_passes, cp = p.col_passes == 1 ? 0 : u - hg * p.col_passes;
            const int q_first = hg * G * p.rep + cp * (8 << p.lqg);
            const int q_rows = p.col_passes == 1 ? G * p.rep : min(8 << p.lqg, p.rep - cp * (8 << p.lqg));
            // the unit after this one
            int s2 = s, u2 = u + 1, ctx2 = ctx, n2 = n;
            if (u2 == units) {
                u2 = 0;
                if (issued + left < count) do {
                    ctx2 = length_of(p, ++s2, false);
                    n2 = (ctx2 + TT - 1) >> tshift;
                } while (n2 == 0);
            }
            if (seg >= 2 && ok) ok = warp_wait(smem_addr(q_empty + (seg & 1)), ((seg >> 1) & 1) ^ 1, p.status);
            const int64_t from = (int64_t)hg * G * p.rec, step = (int64_t)p.H * p.rec;
            for (int j = 0; j < left && ok; ++j) {
                const int valid = min(TT, ctx - (tile + j) * TT);
                const bool here = lane < (valid + B - 1) >> p.bshift;
                const bool good = here && (unsigned)id < (unsigned)p.num_blocks;
                if (here && !good) report(p.status, PA_ERR_BAD_BLOCK);
                const int now = id;
                if (j + 1 < left) id = entry(s, ctx, tile + j + 1);
                else if (issued + 1 < count) id = entry(s2, ctx2, 0);
                if (round > 0) ok = warp_wait(smem_addr(empty + st), (round & 1) ^ 1, p.status);
                if (!ok) {
                    report(p.status, PA_ERR_TIMEOUT);
                    break;
                }
                const uint32_t bar = smem_addr(full + st);
                const int copies = __popc(__ballot_sync(kAll, good));
                if (lane == 0) {
                    if (j == 0) stretch[seg & 1] = {left, ctx - tile * TT, s, u, part};
                    mbar_arrive_expect_tx(bar, copies * 2 * run + (j == 0 ? q_rows * D * 2 : 0));
                    if (j == 0)
                        bulk_g2s(smem_addr(q_at + (seg & 1) * p.q_bytes),
                                 (const char *)p.q + ((int64_t)s * p.Hq + q_first) * D * 2, q_rows * D * 2, bar, policy);
                }
                __syncwarp();
                if (good) {
                    const int64_t src = now * step + from;
                    const uint32_t dst = smem_addr(smem + st * stage_bytes + lane * run);
                    bulk_g2s(dst, p.k + src, run, bar, policy);
                    bulk_g2s(dst + half, p.v + src, run, bar, policy);
                }
                ++issued;
                if (++st == p.stages) {
                    st = 0;
                    ++round;
                }
            }
            issued = after;
            s = s2;
            u = u2;
            ctx = ctx2;
            n = n2;
            tile = 0;
        }
        if (!ok) report(p.status, PA_ERR_TIMEOUT);
        if (!p.by_unit && lane == 0) p.jobs[blockIdx.x] = job;
        // no copy is in flight when the CTA ends
        const int copied = round * p.stages + st;
        for (int i = max(0, copied - p.stages); i < copied; ++i)
            if (!mbar_wait_bounded(smem_addr(full + i % p.stages), (i / p.stages) & 1, p.status, false)) {
                report(p.status, PA_ERR_TIMEOUT);
                break;
            }
        return;
    }

    // ---- products: lane = (r, c), rows r and r + 8, columns 2 c and 2 c + 1
    const int r = lane >> 2, c = lane & 3;
    const int ns = warp & (NS - 1), cg = (warp >> p.lns) & ((1 << p.lqg) - 1), g = warp >> (p.lns + p.lqg);
    const int group = warp >> p.lns;          // warps that share a head's tiles
    const int base = ns * 16 * MT;            // this warp's positions in a tile
    const uint32_t head = g * p.rec + (base >> p.bshift) * run, in = base & (B - 1);
    const uint32_t k_lane = head + (in + row_token(r)) * RB + c * (RB / 4);
    const uint32_t s_lane = head + (RB << p.bshift) + (in + row_token(r)) * SB + (GS == 4 ? (c & 1) * 4 : 0);
    // values: 4 dimensions of every group, positions of rows 2 c and 2 c + 1
    const uint32_t v_piece = BITS == 4 ? (r >> 1) * (RB / 4) : (r >> 1) * (RB / 4) + (r & 1) * 4;
    const uint32_t va_lane = half + head + (in + row_token(2 * c)) * RB + v_piece;
    const uint32_t vb_lane = half + head + (in + row_token(2 * c + 1)) * RB + v_piece;
    const uint32_t pick = (r & 1) ? 0x7632u : 0x5410u;   // the halves of a and b

    uint32_t qb[GR][4], zb[2];                // queries; the codes' constants, see below
    float zq[PACK ? SETS : 1][4];
    // (R: minus the reference)
    float mult[NQ], R[NQ], top[NQ], l[NQ], O[2 * GR][4];
#pragma unroll
    for (int j = 0; j < NQ; ++j) mult[j] = R[j] = top[j] = l[j] = 0.f;
    int merges = 0, st = 0, phase = 0;

    bool ok = true;
    for (int done = 0, seg = 0; done < count && ok; ++seg) {
        ok = warp_wait(smem_addr(full + st), phase, p.status);   // the stretch's first tile
        if (!ok) break;
        const Stretch m = stretch[seg & 1];
        done += m.tiles;
        uint32_t vref = 0;                       // the largest scale of values, twice; once where a column is beyond kFar
        int cols = 0;
        {
            const int cp = p.col_passes == 1 ? 0 : m.unit % p.col_passes;
            cols = min(8, p.rep - cp * (8 << p.lqg) - cg * 8);      // may be negative
            // the queries, scaled by a power of two so that their largest is 4 .. 8 (8 bits:
            // 1/2 .. 1) and no sum of constants beyond fp16
            const int query = PACK ? r / GS : r;            // of column r
            const uint8_t *row = q_at + (seg & 1) * p.q_bytes + (g * p.rep + cg * 8 + query) * D * 2;
            constexpr int NG = PACK ? SETS : GR;            // groups of this lane's columns
            float f[NG][8];
            uint32_t big = 0;
#pragma unroll
            for (int k = 0; k < NG; ++k) {
                uint4 w = make_uint4(0, 0, 0, 0);
                if (query < cols) w = *reinterpret_cast<const uint4 *>(row + (32 * (PACK ? GS * k + r % GS : k) + 8 * c) * 2);
                if (p.bf16) quant::unpack8<__nv_bfloat16>(w, f[k]);
                else quant::unpack8<__half>(w, f[k]);
#pragma unroll
                for (int j = 0; j < 8; ++j) big = max(big, __float_as_uint(f[k][j]) & 0x7fffffffu);
            }
#pragma unroll
            for (int o = 1; o < (PACK ? 4 * GS : 4); o <<= 1) big = max(big, __shfl_xor_sync(kAll, big, o));
            // (a query near either end of bf16's range comes 2^32 nearer to 1 first: every power of
            // two here then is a normal number, e within -94 .. 104, infinity and NaN aside)
            const int nearer = big < 32u << 23 ? 32 : big >= 224u << 23 ? -32 : 0;
            if (nearer != 0) {
                const float by = __uint_as_float((uint32_t)(127 + nearer) << 23);
                big = __float_as_uint(__uint_as_float(big) * by);
#pragma unroll
                for (int k = 0; k < NG; ++k)
#pragma unroll
                    for (int j = 0; j < 8; ++j) f[k][j] *= by;
            }
            const int e = max(-126, min((BITS == 4 ? 2 : -1) - ((int)(big >> 23) - 127), 104));
            const float up = __uint_as_float((uint32_t)(e + 127) << 23) * p.sign;
            // (at most 2^96: a score times it stays finite, and any two that differ are far apart)
            const float back = query < cols ? fminf(p.scale * __uint_as_float((uint32_t)(127 - e) << 23) *
                                                        __uint_as_float((uint32_t)(127 - nearer) << 23) * kLog2e, 0x1p96f) : 0.f;
            // (never 0: masked scores are minus infinity before they meet it)
#pragma unroll
            for (int j = 0; j < NQ; ++j)
                mult[j] = fmaxf(__shfl_sync(kAll, back, 4 * (PACK ? 2 * c / GS * GS : 2 * c + j)), 1.1754944e-38f);
#pragma unroll
            for (int k = 0; k < GR; ++k) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float u = up * key_divide<BITS>(j), *x = f[PACK ? k / GS : k];
                    const uint32_t q2 = BITS == 4 ? half2_bits(x[j] * u, x[j + 4] * u)
                                                  : half2_bits(x[2 * j] * u, x[2 * j + 1] * u);
                    qb[k][j] = !PACK || k % GS == r % GS ? q2 : 0;
                }
            }
            // What the codes' constants add to every score, Z_g for each group and column: where a
            // column has one group, its sums start from - Z; otherwise one more product takes it
            // off, a position's scales times - Z_g in three fp16 parts (33 bits), parts
            // 0, 1, 2 of the groups along the product's depth.
            if constexpr (PACK) {
#pragma unroll
                for (int e = 0; e < SETS; ++e) {
                    float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int k = GS * e; k < GS * e + GS; ++k) {
                        mma(d, key_zero<BITS>(0), key_zero<BITS>(0), key_zero<BITS>(1), key_zero<BITS>(1), qb[k][0], qb[k][1]);
                        mma(d, key_zero<BITS>(2), key_zero<BITS>(2), key_zero<BITS>(3), key_zero<BITS>(3), qb[k][2], qb[k][3]);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) zq[e][j] = -d[j];
                }
            } else {
                float z[4][2] = {};          // part 0 .. 2 of this lane's column r and two of its groups
#pragma unroll
                for (int k = 0; k < GR; ++k) {
                    float d[4];
                    mma_zero(d, key_zero<BITS>(0), key_zero<BITS>(0), key_zero<BITS>(1), key_zero<BITS>(1), qb[k][0], qb[k][1]);
                    mma(d, key_zero<BITS>(2), key_zero<BITS>(2), key_zero<BITS>(3), key_zero<BITS>(3), qb[k][2], qb[k][3]);
                    // column r's is with the lanes whose c is r / 2
                    const float even = __shfl_sync(kAll, d[0], r >> 1), odd = __shfl_sync(kAll, d[1], r >> 1);
                    const float Z = -((r & 1) ? odd : even);
                    const float hi = __half2float(__float2half_rn(Z)), mid = __half2float(__float2half_rn(Z - hi));
                    if (GR == 2 || k / 2 == (c & 1)) {
                        z[0][k & 1] = hi;
                        z[1][k & 1] = mid;
                        z[2][k & 1] = Z - hi - mid;
                    }
                }
                // depth 2 c, 2 c + 1: D = 128: parts 0, 0, 1, 1 of groups (0, 1), (2, 3) ..; then part 2, 2, none,
                // none; D = 64: parts 0, 1, 2, none
                if (GR == 4) {
                    zb[0] = c < 2 ? half2_bits(z[0][0], z[0][1]) : half2_bits(z[1][0], z[1][1]);
                    zb[1] = c < 2 ? half2_bits(z[2][0], z[2][1]) : 0;
                } else {
                    zb[0] = c == 0   ? half2_bits(z[0][0], z[0][1])
                            : c == 1 ? half2_bits(z[1][0], z[1][1])
                            : c == 2 ? half2_bits(z[2][0], z[2][1])
                                     : 0;
                    zb[1] = 0;
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(q_empty + (seg & 1)));
#pragma unroll
            for (int k = 0; k < 2 * GR; ++k) O[k][0] = O[k][1] = O[k][2] = O[k][3] = 0.f;
#pragma unroll
            for (int j = 0; j < NQ; ++j) {
                R[j] = INFINITY;
                top[j] = -INFINITY;
                l[j] = 0.f;
            }
        }
        int valid = m.positions - base;          // from this warp's first position of the tile on
        for (int tile = 0; tile < m.tiles; ++tile, valid -= TT) {
        if (tile > 0) ok = warp_wait(smem_addr(full + st), phase, p.status);
        if (!ok) break;
        const uint32_t at = smem_addr(smem) + st * stage_bytes;
        if (valid > 0 && cols > 0) {
            float x[MT][2 * NQ];              // scores of rows r (0 ..) and r + 8 (NQ ..)
            uint32_t vs[MT][2][SW];
            const uint32_t at_k = at + k_lane, at_s = at + s_lane, at_a = at + va_lane, at_b = at + vb_lane;
            // scores
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                uint32_t w[2][NW], ks[2][SW];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    lds<NW>(at_k + p.code_at[2 * t + h], w[h]);
                    lds<SW>(at_s + p.scale_at[2 * t + h], ks[h]);
                    lds<SW>(at_s + half + p.scale_at[2 * t + h], vs[t][h]);
                }
                if constexpr (PACK) {
                    float d[SETS][4];
#pragma unroll
                    for (int k = 0; k < GR; ++k) {
                        uint32_t a[4], b[4];
                        key_pairs<BITS>(w[0] + k * WP, a);
                        key_pairs<BITS>(w[1] + k * WP, b);
                        if (k % GS == 0) mma_from(d[k / GS], zq[k / GS], a[0], b[0], a[1], b[1], qb[k][0], qb[k][1]);
                        else mma(d[k / GS], a[0], b[0], a[1], b[1], qb[k][0], qb[k][1]);
                        mma(d[k / GS], a[2], b[2], a[3], b[3], qb[k][2], qb[k][3]);
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        x[t][h] = half_at(ks[h][0], 0) * d[0][2 * h];
#pragma unroll
                        for (int e = 0; e < SETS; ++e) {
                            if (e > 0) x[t][h] = fmaf(half_at(ks[h][e], 0), d[e][2 * h], x[t][h]);
                            x[t][h] = fmaf(half_at(ks[h][e], 1), d[e][2 * h + 1], x[t][h]);
                        }
                        if (GS == 4) x[t][h] += __shfl_xor_sync(kAll, x[t][h], 1);
                    }
                } else {
                    const uint32_t za = GR == 4 && (c & 1) ? ks[0][SW - 1] : ks[0][0];
                    const uint32_t zc = GR == 4 && (c & 1) ? ks[1][SW - 1] : ks[1][0];
                    mma_zero(x[t], za, zc, za, zc, zb[0], zb[1]);
#pragma unroll
                    for (int k = 0; k < GR; ++k) {
                        uint32_t a[4], b[4];
                        float d[4];
                        key_pairs<BITS>(w[0] + k * WP, a);
                        key_pairs<BITS>(w[1] + k * WP, b);
                        mma_zero(d, a[0], b[0], a[1], b[1], qb[k][0], qb[k][1]);
                        mma(d, a[2], b[2], a[3], b[3], qb[k][2], qb[k][3]);
#pragma unroll
                        for (int j = 0; j < 4; ++j) x[t][j] = fmaf(half_at(ks[j / 2][k / 2], k & 1), d[j], x[t][j]);
                    }
                }
            }
            if (valid < 16 * MT) {           // slots past the context hold anything
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if (16 * t + 8 * h + row_token(r) >= valid) {
#pragma unroll
                            for (int j = 0; j < NQ; ++j) x[t][h * NQ + j] = -INFINITY;
#pragma unroll
                            for (int k = 0; k < SW; ++k) vs[t][h][k] = 0;
                        }
            }
            // the reference
            float big[NQ];
            bool grows = false;
#pragma unroll
            for (int j = 0; j < NQ; ++j) {
                big[j] = fmaxf(x[0][j], x[0][NQ + j]);
#pragma unroll
                for (int t = 1; t < MT; ++t) big[j] = fmaxf(big[j], fmaxf(x[t][j], x[t][NQ + j]));
                big[j] = __fmul_rn(big[j], mult[j]);         // (mult > 0)
                grows |= big[j] > top[j] + kSlack;
            }
            uint32_t v2 = __vmaxu2(vs[0][0][0], vs[0][1][0]);
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int k = t > 0 ? 0 : 1; k < SW; ++k) v2 = __vimax3_u16x2(v2, vs[t][0][k], vs[t][1][k]);
            // (vref 0: the stretch's first positions; scores beyond kFar come here always)
            if (__any_sync(kAll, grows || __vmaxu2(v2, vref) != vref || vref < 0x10000u)) {
                uint32_t vmax = __reduce_max_sync(kAll, max(max(v2 >> 16, v2 & 0xffffu), vref & 0xffffu));
                // a group that is not finite sets no reference for the others (read again: the words
                // at hand would cost registers, four grouped heads 112.6 us, so 117.6)
                if (vmax >= 0x7c00u) {
                    uint32_t most = vref & 0xffffu;
#pragma unroll 1
                    for (int i = 0; i < 2 * MT; ++i) {
                        if (8 * i + row_token(r) >= valid) break;
                        uint32_t w[SW];
                        lds<SW>(at_s + half + p.scale_at[i], w);
#pragma unroll
                        for (int k = 0; k < SW; ++k) {
                            const uint32_t lo = w[k] & 0xffffu, hi = w[k] >> 16;
                            most = max(most, max(lo < 0x7c00u ? lo : 0, hi < 0x7c00u ? hi : 0));
                        }
                    }
                    vmax = __reduce_max_sync(kAll, most);
                }
                const float lift = (float)lift_of(vmax), more = (float)(lift_of(vmax) - lift_of(vref & 0xffffu));
                float f[NQ];
                bool far = false;
#pragma unroll
                for (int j = 0; j < NQ; ++j) {
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) big[j] = fmaxf(big[j], __shfl_xor_sync(kAll, big[j], o));
                    const float was = top[j];
                    top[j] = fmaxf(top[j], big[j]);
                    const bool beyond = fabsf(top[j]) >= kFar;
                    far |= beyond;
                    f[j] = ex2(beyond || fabsf(was) >= kFar ? (was - top[j]) + more : (lift - top[j]) - R[j]);
                    R[j] = beyond ? 0.f : lift - top[j];
                    l[j] *= f[j];
                }
                far = __any_sync(kAll, far);
                vref = vmax * (far ? 1u : 0x10001u);
                if (far) {
#pragma unroll
                    for (int j = 0; j < NQ; ++j) {
                        if (!(fabsf(top[j]) >= kFar)) continue;
                        const float back = 1.f / mult[j];     // (R is 0)
#pragma unroll
                        for (int t = 0; t < MT; ++t) {
                            x[t][j] = ((__fmul_rn(x[t][j], mult[j]) - top[j]) + lift) * back;
                            x[t][NQ + j] = ((__fmul_rn(x[t][NQ + j], mult[j]) - top[j]) + lift) * back;
                        }
                    }
                }
#pragma unroll
                for (int k = 0; k < 2 * GR; ++k)
#pragma unroll
                    for (int j = 0; j < 4; ++j) O[k][j] *= f[PACK ? 0 : j & 1];
            }
            // weights, and the values' product
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                uint32_t w[4][BITS == 4 ? NW : GR];      // positions a, b of rows 0 .. 7, then of 8 .. 15
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t o = p.code_at[2 * t + h];
                    if constexpr (BITS == 4) {
                        lds<NW>(at_a + o, w[2 * h]);
                        lds<NW>(at_b + o, w[2 * h + 1]);
                    } else {
#pragma unroll
                        for (int k = 0; k < GR; ++k) {
                            lds<1>(at_a + o + k * 8, &w[2 * h][k]);
                            lds<1>(at_b + o + k * 8, &w[2 * h + 1][k]);
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < 2 * NQ; ++j) x[t][j] = ex2(fmaf(x[t][j], mult[j % NQ], R[j % NQ]));
#pragma unroll
                for (int j = 0; j < NQ; ++j) l[j] += x[t][j] + x[t][NQ + j];
                uint32_t b0 = 0, b1 = 0;
#pragma unroll
                for (int k = 0; k < GR; ++k) {
                    if constexpr (PACK) {
                        if (k % GS == 0) {
                            const uint32_t lo = vs[t][0][k / GS], hi = vs[t][1][k / GS];
                            b0 = transpose8(half2_bits(x[t][0] * half_at(lo, 0), x[t][0] * half_at(lo, 1)));
                            b1 = transpose8(half2_bits(x[t][1] * half_at(hi, 0), x[t][1] * half_at(hi, 1)));
                        }
                    } else {
                        const float lo = half_at(vs[t][0][k / 2], k & 1), hi = half_at(vs[t][1][k / 2], k & 1);
                        b0 = transpose8(half2_bits(x[t][0] * lo, x[t][1] * lo));
                        b1 = transpose8(half2_bits(x[t][2] * hi, x[t][3] * hi));
                    }
                    uint32_t a[4], b[4];
                    value_pairs<BITS>(w[0][k], w[1][k], pick, a);
                    value_pairs<BITS>(w[2][k], w[3][k], pick, b);
                    mma(O[2 * k], a[0], a[1], b[0], b[1], b0, b1);
                    mma(O[2 * k + 1], a[2], a[3], b[2], b[3], b0, b1);
                }
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(empty + st));
        if (++st == p.stages) {
            st = 0;
            phase ^= 1;
        }
        }
        if (!ok) break;

        // ---- the stretch's end
        if (vref < 0x10000u) {                   // beyond kFar: references without the lift
            const float down = __uint_as_float((uint32_t)(127 - lift_of(vref & 0xffffu)) << 23);
#pragma unroll
            for (int j = 0; j < NQ; ++j) {
                if (!(fabsf(top[j]) >= kFar)) continue;
                R[j] = -top[j];
                l[j] *= down;
#pragma unroll
                for (int k = 0; k < 2 * GR; ++k)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (PACK || (i & 1) == j) O[k][i] *= down;
            }
        }
        if constexpr (BITS == 4) {               // dimensions 0 and 2 of four came with 16 times 1 and 3
#pragma unroll
            for (int k = 0; k < 2 * GR; ++k)
#pragma unroll
                for (int j = 0; j < 2; ++j) O[k][j] = fmaf(-16.f, O[k][j + 2], O[k][j]);
        }
#pragma unroll
        for (int j = 0; j < NQ; ++j)
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) l[j] += __shfl_xor_sync(kAll, l[j], o);
        const int hg = m.unit / p.col_passes, cp = m.unit - hg * p.col_passes;
        const int local = g * p.rep + cg * 8;                 // of the unit's rows
        const int64_t row0 = (int64_t)m.seq * p.Hq + hg * G * p.rep + cp * (8 << p.lqg) + local;
        const int64_t ws0 = (int64_t)max(m.part, 0) * p.rows + local;
        // 4 dimensions of a group: with fn(query, dimension, values, scale of a whole context's sums)
        auto results = [&](auto fn) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if constexpr (PACK) {
                    // (a set of four groups: the upper two are the odd lanes')
                    const bool upper = GS == 4 && (c & 1);
#pragma unroll
                    for (int e = 0; e < SETS; ++e) {
                        const int k = 2 * e + j, up = (k + 2) % GR;       // (up: only where GS == 4)
                        const float4 v = make_float4(upper ? O[2 * up][j] : O[2 * k][j], upper ? O[2 * up][j + 2] : O[2 * k][j + 2],
                                                     upper ? O[2 * up + 1][j] : O[2 * k + 1][j],
                                                     upper ? O[2 * up + 1][j + 2] : O[2 * k + 1][j + 2]);
                        if (2 * c / GS < cols) fn(2 * c / GS, 32 * (upper ? up : k) + 4 * r, v, l[0]);
                    }
                } else if (2 * c + j < cols) {
#pragma unroll
                    for (int k = 0; k < GR; ++k)
                        fn(2 * c + j, 32 * k + 4 * r,
                           make_float4(O[2 * k][j], O[2 * k][j + 2], O[2 * k + 1][j], O[2 * k + 1][j + 2]), l[NQ == 2 ? j : 0]);
                }
            }
        };
        if (NS == 1) {
            if (m.part < 0) {
                results([&](int col, int d, float4 v, float sum) {
                    const float inv = 1.f / sum;
                    store4<D>(p, row0 + col, d, v.x * inv, v.y * inv, v.z * inv, v.w * inv);
                });
            } else {
                results([&](int col, int d, float4 v, float) {
                    *reinterpret_cast<float4 *>(p.acc + (ws0 + col) * D + d) = v;
                });
#pragma unroll
                for (int j = 0; j < NQ; ++j) {
                    const int col = PACK ? 2 * c / GS : 2 * c + j;
                    if (r == 0 && col < cols) p.ml[ws0 + col] = make_float2(-R[j], l[j]);
                }
            }
        } else {
            // warps with shares of the same positions meet in shared memory: 8 columns of D, then references and sums
            float *area = merge_at + (group * NS + ns) * 8 * (D + 2);
            results([&](int col, int d, float4 v, float) { *reinterpret_cast<float4 *>(area + col * D + d) = v; });
#pragma unroll
            for (int j = 0; j < NQ; ++j) {
                const int col = PACK ? 2 * c / GS : 2 * c + j;
                if (r == 0) {
                    area[8 * D + 2 * col] = -R[j];
                    area[8 * D + 2 * col + 1] = l[j];
                }
            }
            const uint32_t bar = smem_addr(merged + group);
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
            if (!warp_wait(bar, merges & 1, p.status)) {
                ok = false;
                break;
            }
            ++merges;
            for (int col = ns; col < cols; col += NS) {
                const float *first = merge_at + group * NS * 8 * (D + 2);
                float M = -INFINITY, L = 0.f;
                for (int w = 0; w < NS; ++w) M = fmaxf(M, first[w * 8 * (D + 2) + 8 * D + 2 * col]);
                float o[D / 32];
#pragma unroll
                for (int k = 0; k < D / 32; ++k) o[k] = 0.f;
                for (int w = 0; w < NS; ++w) {
                    const float *from = first + w * 8 * (D + 2);
                    // (a share without positions: weight 0)
                    const float l_w = from[8 * D + 2 * col + 1];
                    const float f = l_w == 0.f ? 0.f : ex2(from[8 * D + 2 * col] - M);
                    L = fmaf(f, l_w, L);
#pragma unroll
                    for (int k = 0; k < D / 32; ++k) o[k] = fmaf(f, from[col * D + lane * (D / 32) + k], o[k]);
                }
                if (m.part < 0) {
                    const float inv = 1.f / L;
                    char *dst = (char *)p.out + ((row0 + col) * D + lane * (D / 32)) * 2;
#pragma unroll
                    for (int k = 0; k < D / 32; k += 2)
                        *reinterpret_cast<uint32_t *>(dst + 2 * k) =
                            p.bf16 ? quant::pack2<__nv_bfloat16>(o[k] * inv, o[k + 1] * inv)
                                   : quant::pack2<__half>(o[k] * inv, o[k + 1] * inv);
                } else {
#pragma unroll
                    for (int k = 0; k < D / 32; ++k) p.acc[(ws0 + col) * D + lane * (D / 32) + k] = o[k];
                    if (lane == 0) p.ml[ws0 + col] = make_float2(M, L);
                }
            }
            // before anyone writes its share of the next stretch
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
            if (!warp_wait(bar, merges & 1, p.status)) {
                ok = false;
                break;
            }
            ++merges;
        }
    }
    if (!ok) report(p.status, PA_ERR_TIMEOUT);
    // sequences without positions give 0, refused ones nothing
    for (int s = blockIdx.x; s < p.n_seqs; s += gridDim.x) {
        if (length_of(p, s, false) > 0) continue;
        if (p.by_unit)
            for (int k = tid; k < units; k += kWarps * 32) p.jobs[(int64_t)s * units + k] = make_int4(0, 0, 0, 0);
        if (p.ctx[s] <= 0)
            for (int k = tid; k < p.Hq * D / 8; k += kWarps * 32)
                reinterpret_cast<uint4 *>((char *)p.out + (int64_t)s * p.Hq * D * 2)[k] = make_uint4(0, 0, 0, 0);
    }
}

// M = max R_p, o = sum 2^(R_p - M) acc_p / sum 2^(R_p - M) l_p over the parts of every row
// of a unit that is cut: the cutting CTA's last stretch and the first ones of the CTAs
// after it.  Bound by latency: an entry, then all else at once.  A warp takes ROWS rows of
// a unit, 32 / ROWS parts at a time (lane = (row, part) for references and sums, four or two
// dimensions a lane for the rest); `each` warps of a block share a unit's parts, as many
// as the GPU holds at once, and where that leaves warps idle they take one row each (one
// sequence of 32768 positions, 228 parts: 20.8 us with four rows a warp, 17.0 with one).
constexpr int kJoinWarps = 8;
template <int D, int ROWS>
__global__ void __launch_bounds__(kJoinWarps * 32, 2) quant_join_kernel(const QuantParams p, int entries, int each) {
    constexpr int N = D / 32, PARTS = 32 / ROWS, BATCH = 16 / ROWS;
    using Vec = typename std::conditional<N == 4, float4, float2>::type;
    __shared__ float2 part_ml[kJoinWarps][ROWS];
    __shared__ Vec part_o[kJoinWarps][ROWS][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int groups = (p.rows + ROWS - 1) / ROWS, items = entries * groups;
    const int per_block = kJoinWarps / each, share = warp % each;
    allow_next_launch();
    wait_for_launch_before();
    for (int i0 = blockIdx.x * per_block; i0 < items; i0 += gridDim.x * per_block) {
        const int item = min(i0 + warp / each, items - 1), row0 = item % groups * ROWS;
        const int4 job = p.jobs[item / groups];          // first CTA, parts, sequence, unit
        const bool have = i0 + warp / each < items && job.y > 1;
        const int hg = job.w / p.col_passes, cp = job.w - hg * p.col_passes;
        const int rows = p.col_passes == 1 ? p.rows : min(8 << p.lqg, p.rep - cp * (8 << p.lqg));
        auto slot = [&](int k, int row) { return (int64_t)(2 * (job.x + k) + (k == 0)) * p.rows + min(row, rows - 1); };
        const int mn = (job.y + each - 1) / each, k0 = share * mn, k1 = have ? min(job.y, k0 + mn) : 0;
        float M = -INFINITY, L = 0.f;        // of row lane / PARTS
        float o[ROWS][N];
#pragma unroll
        for (int u = 0; u < ROWS; ++u)
#pragma unroll
            for (int j = 0; j < N; ++j) o[u][j] = 0.f;
        for (int kc = k0; kc < k1; kc += PARTS) {
            const int k = kc + lane % PARTS;
            const float2 ml = k < k1 ? p.ml[slot(k, row0 + lane / PARTS)] : make_float2(-INFINITY, 0.f);
            Vec v[BATCH][ROWS];
            auto load = [&](int kk) {
#pragma unroll
                for (int e = 0; e < BATCH; ++e)
#pragma unroll
                    for (int u = 0; u < ROWS; ++u)      // (past the last: the last, with weight 0)
                        v[e][u] = reinterpret_cast<const Vec *>(p.acc + slot(min(kc + kk + e, k1 - 1), row0 + u) * D)[lane];
            };
            load(0);
            float top = fmaxf(M, ml.x);
#pragma unroll
            for (int x = PARTS / 2; x >= 1; x >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, x));
            const float f = k < k1 ? ex2(ml.x - top) : 0.f, old = kc > k0 ? ex2(M - top) : 0.f;
            float sum = f * ml.y;
#pragma unroll
            for (int x = PARTS / 2; x >= 1; x >>= 1) sum += __shfl_xor_sync(kAll, sum, x);
            L = fmaf(L, old, sum);
            M = top;
            if (kc > k0) {
#pragma unroll
                for (int u = 0; u < ROWS; ++u) {
                    const float g = __shfl_sync(kAll, old, PARTS * u);
#pragma unroll
                    for (int j = 0; j < N; ++j) o[u][j] *= g;
                }
            }
#pragma unroll
            for (int kk = 0; kk < PARTS; kk += BATCH) {
                if (kc + kk >= k1) break;
                if (kk > 0) load(kk);
#pragma unroll
                for (int e = 0; e < BATCH; ++e)
#pragma unroll
                    for (int u = 0; u < ROWS; ++u) {
                        const float g = __shfl_sync(kAll, f, PARTS * u + kk + e);
                        const float *x = reinterpret_cast<const float *>(&v[e][u]);
#pragma unroll
                        for (int j = 0; j < N; ++j) o[u][j] = fmaf(g, x[j], o[u][j]);
                    }
            }
        }
        const int64_t out0 = (int64_t)job.z * p.Hq + hg * (p.rep << p.lg) + cp * (8 << p.lqg);
        auto store = [&](int row, const float *x, float sum) {
            const float inv = 1.f / sum;
            uint32_t *dst = reinterpret_cast<uint32_t *>((char *)p.out + ((out0 + row) * D + lane * N) * 2);
#pragma unroll
            for (int j = 0; j < N; j += 2)
                dst[j / 2] = p.bf16 ? quant::pack2<__nv_bfloat16>(x[j] * inv, x[j + 1] * inv)
                                    : quant::pack2<__half>(x[j] * inv, x[j + 1] * inv);
        };
        if (each == 1) {
#pragma unroll
            for (int u = 0; u < ROWS; ++u) {
                const float sum = __shfl_sync(kAll, L, PARTS * u);
                if (have && row0 + u < rows) store(row0 + u, o[u], sum);
            }
            continue;
        }
#pragma unroll
        for (int u = 0; u < ROWS; ++u) {
            float *to = reinterpret_cast<float *>(&part_o[warp][u][lane]);
#pragma unroll
            for (int j = 0; j < N; ++j) to[j] = o[u][j];
        }
        if (lane % PARTS == 0) part_ml[warp][lane / PARTS] = make_float2(M, L);
        __syncthreads();
        for (int u = share; u < ROWS; u += each) {
            if (!have || row0 + u >= rows) break;
            const int n = (job.y + mn - 1) / mn;             // warps that had parts
            float top = -INFINITY, sum = 0.f, x[N];
#pragma unroll
            for (int j = 0; j < N; ++j) x[j] = 0.f;
            for (int w = 0; w < n; ++w) top = fmaxf(top, part_ml[warp - share + w][u].x);
            for (int w = 0; w < n; ++w) {
                const float2 ml = part_ml[warp - share + w][u];
                const float f = ex2(ml.x - top);
                sum = fmaf(f, ml.y, sum);
                const float *from = reinterpret_cast<const float *>(&part_o[warp - share + w][u][lane]);
#pragma unroll
                for (int j = 0; j < N; ++j) x[j] = fmaf(f, from[j], x[j]);
            }
            store(row0 + u, x, sum);
        }
        __syncthreads();
    }
}

bool mis(const void *ptr, int n) { return (reinterpret_cast<uintptr_t>(ptr) & (n - 1)) != 0; }

constexpr int kMaxDevs = 64;

int sm_count() {
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess ? sm_count_of(dev) : 152;
}

// How a CTA's four warps are dealt: 8 query heads of a key/value head each; first
// to more query heads of it, then to further key/value heads (a power of two that
// divides them), the rest to shares of the positions.  Blocks of 32 rows of 128
// bytes fill a stage with two heads' already.
void deal(QuantParams &p, const pa_pool_desc *d) {
    p.H = d->num_heads;
    p.lqg = p.rep <= 8 ? 0 : p.rep <= 16 ? 1 : 2;
    p.lg = 2 - p.lqg;
    if (d->dtype == PA_DTYPE_I8 && d->head_dim == 128 && d->block_size == 32) p.lg = std::max(0, p.lg - 1);
    while (p.H % (1 << p.lg)) --p.lg;
    p.lns = 2 - p.lqg - p.lg;
    p.head_groups = p.H >> p.lg;
    p.col_passes = (p.rep + (8 << p.lqg) - 1) / (8 << p.lqg);
    if (p.col_passes > 1) {      // (lqg is 2, so a unit is one key/value head's 32 query heads)
        p.rows = 8 << p.lqg;
    } else {
        p.rows = p.rep << p.lg;
    }
}

int cta_count(const pa_pool_desc *d) { return std::min(kMaxCtas, sm_count() * ctas_of(d->dtype == PA_DTYPE_I4 ? 4 : 8)); }

struct Sections {
    size_t ml, acc, total;
};
Sections sections(const QuantParams &p, int ctas, int D) {
    Sections s;
    auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
    s.ml = up((size_t)ctas * sizeof(int4));
    s.acc = s.ml + up((size_t)ctas * 2 * p.rows * sizeof(float2));
    s.total = s.acc + up((size_t)ctas * 2 * p.rows * D * sizeof(float));
    return s;
}

bool shape_ok(int32_t n_seqs, int32_t q_heads, const pa_pool_desc *d, std::string *why) {
    if (!quant_geometry_ok(d, why)) return false;
    if (n_seqs < 0 || q_heads < 1 || q_heads > 65535 || q_heads % d->num_heads) {
        *why = "n_seqs < 0, or q_heads no multiple of num_heads from 1 to 65535";
        return false;
    }
    return true;
}

// A launch that may begin while the kernel before it ends (and then waits for its end).
template <typename... Args>
cudaError_t launch_after(void (*kern)(Args...), dim3 grid, int threads, int smem, cudaStream_t st, Args... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Shared memory of a CTA: a stage, and what stands beside the stages.
int stage_bytes_of(const QuantParams &p, int MT) { return 2 * ((16 * MT << p.lns) >> p.bshift) * (p.rec << p.lg); }
int other_bytes_of(const QuantParams &p, int D) {
    return 2 * p.rows * D * 2 + (p.lns > 0 ? kWarps * 8 * (D + 2) * 4 : 0);
}

template <int D, int BITS, int MT, int SETS>
int launch_main(QuantParams p, int ctas, const char *who, cudaStream_t st) {
    auto kern = quant_attention_kernel<D, BITS, MT, SETS>;
    static std::once_flag once[kMaxDevs];
    static cudaError_t err[kMaxDevs];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevs)
        return fail(PA_ERR_CUDA, "%s: cudaGetDevice failed", who);
    std::call_once(once[dev], [&] {
        err[dev] = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_of(BITS));
    });
    if (err[dev] != cudaSuccess)
        return fail(PA_ERR_CUDA, "%s: cudaFuncSetAttribute: %s", who, cudaGetErrorString(err[dev]));
    for (int i = 0; i < 2 * MT; ++i) {
        const int block = (8 * i) >> p.bshift, row = (8 * i) & ((1 << p.bshift) - 1);
        p.code_at[i] = block * (p.rec << p.lg) + row * (D * BITS / 8);
        p.scale_at[i] = block * (p.rec << p.lg) + row * (D / 16);
    }
    const int stage = stage_bytes_of(p, MT), rest = other_bytes_of(p, D);
    p.q_bytes = p.rows * D * 2;
    p.stages = std::min(kMaxStages, (smem_of(BITS) - rest) / stage);
    if (p.stages < 2) return fail(PA_ERR_INVALID_ARG, "%s: no room for two stages", who);
    const cudaError_t e = launch_after(kern, dim3(ctas), kThreads, p.stages * stage + rest, st, p);
    if (e != cudaSuccess) return fail(PA_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
    return PA_OK;
}

int launch_join(const QuantParams &p, int ctas, int D, const char *who, cudaStream_t st) {
    // two blocks an SM hold `warps`
    const int warps = 2 * sm_count() * kJoinWarps;
    const int entries = p.by_unit ? p.n_seqs * p.head_groups * p.col_passes : ctas;
    const int rows = (int64_t)entries * p.rows * kJoinWarps <= warps ? 1 : 4, groups = (p.rows + rows - 1) / rows;
    int each = kJoinWarps;
    while (each > 1 && (int64_t)entries * groups * each > warps) each >>= 1;
    const int64_t blocks = ((int64_t)entries * groups * each + kJoinWarps - 1) / kJoinWarps;
    const dim3 grid((unsigned)std::min<int64_t>(blocks, warps / kJoinWarps));
    const cudaError_t e = launch_after(D == 64 ? (rows == 1 ? quant_join_kernel<64, 1> : quant_join_kernel<64, 4>)
                                               : (rows == 1 ? quant_join_kernel<128, 1> : quant_join_kernel<128, 4>), grid, kJoinWarps * 32, 0,
                                       st, p, entries, each);
    if (e != cudaSuccess) return fail(PA_ERR_CUDA, "%s: join launch: %s", who, cudaGetErrorString(e));
    return PA_OK;
}

}  // namespace

size_t decode_quant_workspace_bytes(int32_t n_seqs, int32_t q_heads, const pa_pool_desc *d) {
    std::string why;
    if (!d || n_seqs <= 0 || !shape_ok(n_seqs, q_heads, d, &why)) return 0;
    QuantParams p{};
    p.rep = q_heads / d->num_heads;
    deal(p, d);
    return sections(p, cta_count(d), d->head_dim).total;
}

int launch_decode_attention_quant(void *out, const void *q, int32_t dtype, int32_t q_heads, const void *k_cache,
                                  const void *v_cache, const int32_t *block_tables, const int32_t *ctx_lens,
                                  int32_t n_seqs, int32_t max_blocks, float scale, void *workspace,
                                  size_t workspace_bytes, int32_t *status, const pa_pool_desc *d, void *stream) {
    const char *who = "pa_decode_attention_quant";
    std::string why;
    if (!d) return fail(PA_ERR_INVALID_ARG, "%s: NULL desc", who);
    if (!shape_ok(n_seqs, q_heads, d, &why)) return fail(PA_ERR_INVALID_ARG, "%s: %s", who, why.c_str());
    if (dtype != PA_DTYPE_F16 && dtype != PA_DTYPE_BF16)
        return fail(PA_ERR_INVALID_ARG, "%s: dtype %d: PA_DTYPE_F16 or PA_DTYPE_BF16", who, dtype);
    if (max_blocks < 0 || (int64_t)max_blocks * d->block_size > INT_MAX - 1024)
        return fail(PA_ERR_INVALID_ARG, "%s: max_blocks=%d", who, max_blocks);
    if (!std::isfinite(scale)) return fail(PA_ERR_INVALID_ARG, "%s: scale is not finite", who);
    if (n_seqs == 0) return PA_OK;
    if (!out || !q || !ctx_lens || (max_blocks > 0 && (!k_cache || !v_cache || !block_tables)))
        return fail(PA_ERR_INVALID_ARG, "%s: NULL pointer", who);
    if (out == q) return fail(PA_ERR_INVALID_ARG, "%s: out and q are one buffer", who);
    if (mis(out, 16) || mis(q, 16) || mis(k_cache, 16) || mis(v_cache, 16) || mis(block_tables, 4) ||
        mis(ctx_lens, 4) || mis(status, 4))
        return fail(PA_ERR_INVALID_ARG, "%s: misaligned pointer", who);
    QuantParams p{};
    p.Hq = q_heads;
    p.rep = q_heads / d->num_heads;
    deal(p, d);
    const int D = d->head_dim, ctas = cta_count(d);
    const Sections sec = sections(p, ctas, D);
    if (!workspace || workspace_bytes < sec.total)
        return fail(PA_ERR_INVALID_ARG, "%s: workspace of %zu bytes needed, %zu given", who, sec.total,
                    workspace ? workspace_bytes : (size_t)0);
    if (mis(workspace, 256)) return fail(PA_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", who);
    char *ws = static_cast<char *>(workspace);
    p.jobs = reinterpret_cast<int4 *>(ws);
    p.ml = reinterpret_cast<float2 *>(ws + sec.ml);
    p.acc = reinterpret_cast<float *>(ws + sec.acc);
    p.by_unit = (int64_t)n_seqs * p.head_groups * p.col_passes <= ctas;
    p.out = out;
    p.q = q;
    p.k = static_cast<const uint8_t *>(k_cache);
    p.v = static_cast<const uint8_t *>(v_cache);
    p.tables = block_tables;
    p.ctx = ctx_lens;
    p.n_seqs = n_seqs;
    p.max_blocks = max_blocks;
    p.num_blocks = d->num_blocks;
    p.bshift = d->block_size == 8 ? 3 : d->block_size == 16 ? 4 : 5;
    p.rec = (int)(block_bytes(d) / d->num_heads);
    p.bf16 = dtype == PA_DTYPE_BF16;
    p.scale = std::fabs(scale);
    p.sign = scale < 0.f ? -1.f : 1.f;
    p.status = status;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    // Positions of a stage: as many as leave two stages (a CTA's three) beside the queries, since
    // every stage costs a warp some 60 instructions beside its positions' own; of 8 bits
    // and D = 128 as few as a block allows, so that five stages are in flight.
    const bool four = d->dtype == PA_DTYPE_I4;
    auto fits = [&](int MT) { return 2 * stage_bytes_of(p, MT) + other_bytes_of(p, D) <= smem_of(4); };
    int rc;
    if (D == 64) {
        if (p.rep > 4) rc = four ? launch_main<64, 4, 4, 0>(p, ctas, who, st) : launch_main<64, 8, 2, 0>(p, ctas, who, st);
        else if (!four) rc = launch_main<64, 8, 2, 1>(p, ctas, who, st);
        else rc = fits(8) ? launch_main<64, 4, 8, 1>(p, ctas, who, st) : launch_main<64, 4, 4, 1>(p, ctas, who, st);
    } else if (four) {
        rc = p.rep > 4   ? launch_main<128, 4, 2, 0>(p, ctas, who, st)
             : p.rep > 2 ? launch_main<128, 4, 2, 2>(p, ctas, who, st)
             : fits(4)   ? launch_main<128, 4, 4, 1>(p, ctas, who, st)
                         : launch_main<128, 4, 2, 1>(p, ctas, who, st);
    } else if ((16 << p.lns) >= d->block_size) {
        rc = p.rep > 4   ? launch_main<128, 8, 1, 0>(p, ctas, who, st)
             : p.rep > 2 ? launch_main<128, 8, 1, 2>(p, ctas, who, st)
                         : launch_main<128, 8, 1, 1>(p, ctas, who, st);
    } else {
        rc = launch_main<128, 8, 2, 0>(p, ctas, who, st);
    }
    if (rc != PA_OK) return rc;
    return launch_join(p, ctas, D, who, st);
}

}  // namespace pagedkv
