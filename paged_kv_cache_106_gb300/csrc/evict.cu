// Keeping part of a cached context: which positions a budget keeps by the
// attention weight they have accumulated (pa_evict_select), and moving kept
// rows of the cache to the front of their sequence (pa_compact_kv), which is
// also how accepted drafts get into place after a verification.
#include <cuda_runtime.h>

#include <algorithm>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pagedkv {

namespace {

constexpr unsigned kAll = 0xffffffffu;

// ---------------------------------------------------------------- selection
//
// For one (sequence, head): the last `recent` of ctx positions and, of the
// others, the budget - recent with the largest sums (ties to the lowest
// position), in ascending order.  One CTA finds the sum of the last one kept on
// order-preserving keys: a histogram of their first 11 bits (sign, exponent and
// 2 mantissa bits, so the sums of one head spread over many bins and the
// shared-memory counters do not queue up), then, where the bin that holds it
// has few keys, each of those counts the ones above it; where it has many
// (equal sums, mostly) two more histograms.  Then the kept positions are written
// in order, with one counting and one writing sweep, each warp over a contiguous
// span.  It reads 4 bytes a position from memory once: contexts up to kCached
// positions stay in shared memory, longer ones are re-read through L2.  Bound
// by the barriers between these steps, so short rows take small CTAs, several
// an SM.
//
// Measured: 64 sequences of 256 to 2048 positions x 40 heads, 512 kept: 24 us (11 MB
// read: 2 us; with the move 212 us, and 237 with 1024 threads a CTA instead of
// 256, 223 with more histograms instead of ranking).  4 of 20 to 32 thousand, 4096
// kept: some 45 us, the move 110 (with more histograms 4 us later; a row in
// shared memory, which leaves one CTA an SM above kCached, 1 us earlier).

constexpr int kBins = 2048;
constexpr int kFew = 512;            // keys of a bin that are ranked one against another (8 bytes each, where the bins were)
constexpr int kShort = 4096;         // positions up to which a CTA has 256 threads, else 1024
constexpr int kCached = 26624;       // positions of a row kept in shared memory (104 KB: two CTAs an SM)

// Larger sums have larger keys; -0 counts as 0, NaN as less than everything.
__device__ __forceinline__ uint32_t key_of(float x) {
    if (x != x) return 0u;
    const uint32_t b = __float_as_uint(x == 0.f ? 0.f : x);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

struct SelectParams {
    int32_t *keep, *keep_lens;
    float *w_out;
    const float *w_in;
    const int32_t *ctx_lens;
    int32_t weight_len, budget, recent, num_heads;
    int32_t *status;
};

// (Six small CTAs an SM, which 42 registers allow: 212 us with the move for 64
// sequences, 214 with the 63 that the compiler takes otherwise.)
template <bool CACHED, int kSelThreads>
__global__ void __launch_bounds__(kSelThreads, kSelThreads == 256 ? 6 : 2) evict_select_kernel(const SelectParams a) {
    constexpr int kSelWarps = kSelThreads / 32;
    extern __shared__ float row_sh[];
    __shared__ __align__(16) uint32_t bins[kBins];   // after a histogram: the few keys of the bin
    __shared__ uint32_t part[kSelWarps], part2[kSelWarps];
    __shared__ uint32_t found[4];      // digit, how many of it are still wanted, how many there are; listed
    const int h = blockIdx.x, s = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int ctx = max(a.ctx_lens[s], 0), budget = a.budget;
    const size_t sh_row = (size_t)s * a.num_heads + h;
    int32_t *keep = a.keep + sh_row * budget;
    const float *w = a.w_in + sh_row * a.weight_len;
    float *wo = a.w_out + sh_row * a.weight_len;
    const bool bad = ctx > a.weight_len;
    const int len = bad ? 0 : min(ctx, budget);
    if (h == 0 && tid == 0) {
        a.keep_lens[s] = len;
        if (bad) report(a.status, PA_ERR_INVALID_ARG);
    }
    for (int j = len + tid; j < budget; j += kSelThreads) keep[j] = -1;
    if (bad) return;
    if (ctx <= budget) {               // everything stays
        for (int j = tid; j < ctx; j += kSelThreads) {
            keep[j] = j;
            wo[j] = w[j];
        }
        return;
    }
    const int old = ctx - a.recent, heavy = budget - a.recent;   // 0 <= heavy < old
    auto at = [&](int j) { return CACHED ? row_sh[j] : w[j]; };
    // f(position, its key) over a warp's span, 32 positions at a time (all lanes
    // come; inside: position < hi), four loads ahead
    auto sweep = [&](int lo, int hi, auto f) {
        for (int j0 = lo; j0 < hi; j0 += 128) {
            float x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] = j0 + 32 * k + lane < hi ? at(j0 + 32 * k + lane) : 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (j0 + 32 * k < hi) f(j0 + 32 * k + lane, key_of(x[k]));
        }
    };

    // ---- the last kept position in the order of sums: its key and position
    // (kept: larger keys, and the same key up to that position), and how many
    // each warp's span keeps
    const int per = (old + kSelWarps * 32 - 1) / (kSelWarps * 32) * 32;
    const int lo = min(old, warp * per), hi = min(old, lo + per);
    uint32_t last = 0;
    int cut = -1;
    if (heavy > 0) {
        uint32_t prefix = 0, mask = 0;
        int want = heavy;
        bool few = false;
#pragma unroll 1
        for (int pass = 0; pass < 3 && !few; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
            const int nb = pass == 2 ? 1024 : 2048;
            for (int b = tid; b < nb; b += kSelThreads) bins[b] = 0;
            __syncthreads();
            if (pass == 0) {
                constexpr int kAtOnce = 4;
                for (int j0 = tid; j0 < ctx; j0 += kAtOnce * kSelThreads) {
                    float x[kAtOnce];
#pragma unroll
                    for (int k = 0; k < kAtOnce; ++k) x[k] = j0 + k * kSelThreads < ctx ? w[j0 + k * kSelThreads] : 0.f;
#pragma unroll
                    for (int k = 0; k < kAtOnce; ++k) {
                        const int j = j0 + k * kSelThreads;
                        if (CACHED && j < ctx) row_sh[j] = x[k];
                        if (j < old) atomicAdd(&bins[key_of(x[k]) >> 21], 1u);
                    }
                }
            } else {
                for (int j = tid; j < old; j += kSelThreads) {
                    const uint32_t key = key_of(at(j));
                    if ((key & mask) == prefix) atomicAdd(&bins[(key >> shift) & (nb - 1)], 1u);
                }
            }
            __syncthreads();
            // bins from the top: thread t owns the bins [nb - (t+1) e, nb - t e)
            const int e = nb / kSelThreads;
            uint32_t mine = 0;
            if (e % 4 == 0) {
                const uint4 *b4 = reinterpret_cast<const uint4 *>(bins + nb - (tid + 1) * e);
                for (int k = 0; k < e / 4; ++k) mine += b4[k].x + b4[k].y + b4[k].z + b4[k].w;
            } else {
                for (int k = 0; k < e; ++k) mine += bins[nb - 1 - (tid * e + k)];
            }
            uint32_t incl = mine;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const uint32_t y = __shfl_up_sync(kAll, incl, off);
                if (lane >= off) incl += y;
            }
            if (lane == 31) part[warp] = incl;
            __syncthreads();
            uint32_t before = incl - mine;
            for (int k = 0; k < warp; ++k) before += part[k];
            if ((int)before < want && (int)(before + mine) >= want) {
                uint32_t run = before;
                for (int k = 0; k < e; ++k) {
                    const int b = nb - 1 - (tid * e + k);
                    if ((int)(run + bins[b]) >= want) {
                        found[0] = (uint32_t)b;
                        found[1] = (uint32_t)want - run;
                        found[2] = bins[b];
                        break;
                    }
                    run += bins[b];
                }
                found[3] = 0;
            }
            __syncthreads();
            prefix |= found[0] << shift;
            mask |= (uint32_t)(nb - 1) << shift;
            want = (int)found[1];
            few = found[2] <= kFew;
        }
        const uint32_t many = found[2];
        __syncthreads();
        uint32_t more = 0, same = 0;       // in this warp's span: surely kept; of the bin
        if (few) {
            // the bin's positions in one number each, larger ones first in order;
            // each counts the ones before it
            unsigned long long *list = reinterpret_cast<unsigned long long *>(bins);
            uint32_t above = 0;
            sweep(lo, hi, [&](int j, uint32_t key) {
                above += j < hi && (key & mask) > prefix;
                if (j < hi && (key & mask) == prefix)
                    list[atomicAdd(&found[3], 1u)] = (unsigned long long)key << 32 | ~(uint32_t)j;
            });
            __syncthreads();
            for (uint32_t i = tid; i < many; i += kSelThreads) {
                const unsigned long long mine = list[i];
                int ahead = 0;
#pragma unroll 8
                for (uint32_t k = 0; k < many; ++k) ahead += list[k] > mine;
                if (ahead == want - 1) {
                    found[0] = (uint32_t)(mine >> 32);
                    found[1] = ~(uint32_t)mine;
                }
            }
            __syncthreads();
            last = found[0];
            cut = (int)found[1];
            const unsigned long long least = (unsigned long long)last << 32 | ~(uint32_t)cut;
            for (uint32_t i = lane; i < many; i += 32) {
                const int j = (int)~(uint32_t)list[i];
                same += list[i] >= least && j >= lo && j < hi;
            }
            more = __reduce_add_sync(kAll, above + same);
        } else {
            // a key that many positions share: the want-th of them in order
            last = prefix;
            sweep(lo, hi, [&](int j, uint32_t key) {
                more += __popc(__ballot_sync(kAll, j < hi && key > last));
                same += __popc(__ballot_sync(kAll, j < hi && key == last));
            });
            if (lane == 0) part2[warp] = same;
            __syncthreads();
            int ahead = 0;
            for (int k = 0; k < warp; ++k) ahead += (int)part2[k];
            if (ahead < want && want <= ahead + (int)same) {      // it lies in this warp's span
                for (int j0 = lo, run = ahead; j0 < hi; j0 += 32) {
                    const int j = j0 + lane;
                    const unsigned eq = __ballot_sync(kAll, j < hi && key_of(at(min(j, hi - 1))) == last);
                    if (run < want && want <= run + __popc(eq)) {
                        if (((eq >> lane) & 1) && run + __popc(eq & ((2u << lane) - 1)) == want) found[1] = (uint32_t)j;
                    }
                    run += __popc(eq);
                }
            }
            __syncthreads();
            cut = (int)found[1];
            more += (uint32_t)max(0, min((int)same, want - ahead));
        }
        if (lane == 0) part[warp] = more;
        __syncthreads();
    } else if (CACHED) {
        for (int j = tid; j < ctx; j += kSelThreads) row_sh[j] = w[j];
        __syncthreads();
    }

    // ---- kept positions in order
    if (heavy > 0) {
        uint32_t out = 0;
        for (int k = 0; k < warp; ++k) out += part[k];
        sweep(lo, hi, [&](int j, uint32_t key) {
            const bool take = j < hi && (key > last || (key == last && j <= cut));
            const unsigned m = __ballot_sync(kAll, take);
            if (take) {
                const uint32_t o = out + __popc(m & ((1u << lane) - 1));
                keep[o] = j;
                if (CACHED) wo[o] = row_sh[j];
            }
            out += __popc(m);
        });
    }
    for (int j = tid; j < a.recent; j += kSelThreads) {
        keep[heavy + j] = old + j;
        if (CACHED) wo[heavy + j] = row_sh[old + j];
    }
    if (!CACHED) {
        // kept sums move down in ascending order, so each chunk is read before
        // anything at or after it is written (the two rows may be one)
        __syncthreads();
        for (int j0 = 0; j0 < len; j0 += kSelThreads) {
            const int j = j0 + tid;
            const float x = j < len ? w[keep[j]] : 0.f;
            __syncthreads();
            if (j < len) wo[j] = x;
            __syncthreads();
        }
    }
    for (int j = len + tid; j < ctx; j += kSelThreads) wo[j] = 0.f;
}

// ---------------------------------------------------------------- compaction
//
// Row j of a sequence's part from position first on becomes the row that was
// at position first + keep[j], keep strictly ascending: keep[j] >= j, so in
// place every row is read before anything is written over it as long as reads
// run ahead of writes in order.  A CTA owns whole columns (16-byte vectors of
// a head's rows) and walks the rows in chunks: where the chunk's rows lie, all
// loads, all stores.  Bound by the bytes: each kept row is read and written
// once; rows already in place are skipped.  Two forms:
//   * a list for each head, or a long one: a head of a cache a CTA, 16 threads a
//     row (D = 128) and so many rows at once, a barrier between loads and stores;
//   * a short list for all heads (accepted drafts; many layers): a thread has a
//     column of all heads' rows to itself, needs no barrier, and moves keys and
//     values by the same row numbers (finding them takes longer than moving a
//     row).  Several layers a CTA, which share that finding, made no difference
//     (174 us).
// Measured: 24 layers x 256 sequences of 1 to 8 accepted rows x 40 heads of 128: 174
// us, 96 % of the bytes' time (by the first form 1641 us: a CTA a head, most of
// them for a row or two).  64 sequences x 40 heads, 512 rows each of its own list:
// 187 us, 1.22 GB at 6.5 TB/s.

constexpr int kMoveThreads = 256;
constexpr int kMaxMoveLayers = 128;
constexpr int kMaxChunk = 512;       // rows of a chunk
constexpr int kShortList = 64;       // entries up to which one list for all heads moves by columns

struct CompactParams {
    const int32_t *src_tables, *dst_tables, *src_lens, *first, *keep, *keep_lens;
    int32_t num_heads, keep_heads, keep_stride, max_blocks, num_blocks, bshift, row_shift;
    int32_t cols, rows, chunk;       // columns and rows a pass of the CTA covers; rows of a chunk
    int32_t *status;
    uint4 *cache[2 * kMaxMoveLayers];   // keys and values of layer 0, 1, ..
};

template <bool SHARED>
__global__ void __launch_bounds__(kMoveThreads) compact_kv_kernel(const __grid_constant__ CompactParams a) {
    constexpr int kUnroll = SHARED ? 4 : 8;
    __shared__ long long from[2][SHARED ? kUnroll : kMaxChunk], to[2][SHARED ? kUnroll : kMaxChunk];   // row numbers, -1: none
    const int s = blockIdx.y, tid = threadIdx.x;
    const int vec = 1 << a.row_shift;                   // vectors of a row
    const int H = a.num_heads, B = 1 << a.bshift, heads = SHARED ? H : 1;   // heads of a list
    // blockIdx.x: group of columns, or head
    const int kh = SHARED ? 0 : blockIdx.x, cg = SHARED ? blockIdx.x : 0;
    const int len = a.keep_lens[s], ctx = a.src_lens[s], first = a.first ? a.first[s] : 0;
    if (len <= 0) return;
    if (len > a.keep_stride || first < 0) {
        if (tid == 0 && blockIdx.x == 0 && blockIdx.z == 0) report(a.status, PA_ERR_INVALID_ARG);
        return;
    }
    const int32_t *keep = a.keep + ((size_t)s * a.keep_heads + (a.keep_heads > 1 ? kh : 0)) * a.keep_stride;
    const int32_t *src = a.src_tables + (size_t)s * a.max_blocks;
    const int32_t *dst = a.dst_tables + (size_t)s * a.max_blocks;

    // Rows (of head kh, or of head 0 of all) that row j of the list moves between.
    auto plan = [&](int buf, int j0) {
        for (int k = tid; k < a.chunk; k += kMoveThreads) {
            long long f = -1, t = -1;
            const int j = j0 + k;
            if (j < len) {
                const int at = keep[j], prev = j > 0 ? keep[j - 1] : -1;
                const long long sp = (long long)first + at, dp = (long long)first + j;
                if (at <= prev || at < j || sp >= ctx) {   // (at >= j: sources lie at or after their targets)
                    report(a.status, PA_ERR_INVALID_ARG);
                } else if ((sp >> a.bshift) >= a.max_blocks) {
                    report(a.status, PA_ERR_BAD_BLOCK);
                } else {
                    const int sb = src[sp >> a.bshift], db = dst[dp >> a.bshift];
                    if (sb < 0 || sb >= a.num_blocks || db < 0 || db >= a.num_blocks) {
                        report(a.status, PA_ERR_BAD_BLOCK);
                    } else if (sb != db || sp != dp) {
                        f = (((long long)sb * H + kh) << a.bshift) + (sp & (B - 1));
                        t = (((long long)db * H + kh) << a.bshift) + (dp & (B - 1));
                    }
                }
            }
            from[buf][k] = f;
            to[buf][k] = t;
        }
    };
    const int c = tid % a.cols, r = tid / a.cols;
    const int col = cg * a.cols + c;                    // vector of the row, over the list's heads
    const bool mine = col < heads * vec && r < a.rows;
    // column col is vector col % vec of head col / vec
    const long long col_off =
        ((long long)(col >> a.row_shift) << (a.bshift + a.row_shift)) + (col & (vec - 1));
    auto load = [&](const uint4 *cache, int buf, uint4 (&x)[kUnroll]) {
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            const int i = r + k * a.rows;
            if (i < a.chunk && from[buf][i] >= 0) x[k] = cache[(from[buf][i] << a.row_shift) + col_off];
        }
    };
    auto store = [&](uint4 *cache, int buf, const uint4 (&x)[kUnroll]) {
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            const int i = r + k * a.rows;
            if (i < a.chunk && to[buf][i] >= 0) cache[(to[buf][i] << a.row_shift) + col_off] = x[k];
        }
    };
    plan(0, 0);
    __syncthreads();
    int buf = 0;
    for (int j0 = 0; j0 < len; j0 += a.chunk, buf ^= 1) {
        uint4 x[kUnroll];
        if (SHARED) {
            if (j0 + a.chunk < len) plan(buf ^ 1, j0 + a.chunk);
            if (mine) {
                uint4 y[kUnroll];
                load(a.cache[2 * blockIdx.z], buf, x);
                load(a.cache[2 * blockIdx.z + 1], buf, y);
                store(a.cache[2 * blockIdx.z], buf, x);
                store(a.cache[2 * blockIdx.z + 1], buf, y);
            }
        } else {
            uint4 *cache = a.cache[blockIdx.z];
            if (mine) load(cache, buf, x);
            if (j0 + a.chunk < len) plan(buf ^ 1, j0 + a.chunk);
            __syncthreads();
            if (mine) store(cache, buf, x);
        }
        __syncthreads();
    }
}

bool mis(const void *ptr, int n) { return (reinterpret_cast<uintptr_t>(ptr) & (n - 1)) != 0; }

}  // namespace

int launch_evict_select(int32_t *keep, int32_t *keep_lens, float *weights_out, const float *weights_in,
                        int32_t weight_len, const int32_t *ctx_lens, int32_t n_seqs, int32_t num_heads,
                        int32_t budget, int32_t recent, int32_t *status, void *stream) {
    const char *who = "pa_evict_select";
    if (n_seqs < 0 || n_seqs > 65535 || num_heads < 1 || weight_len < 0)
        return fail(PA_ERR_INVALID_ARG, "%s: n_seqs=%d (<= 65535), num_heads=%d, weight_len=%d", who, n_seqs,
                    num_heads, weight_len);
    if (budget < 1 || recent < 0 || recent > budget)
        return fail(PA_ERR_INVALID_ARG, "%s: budget=%d (>= 1), recent=%d (0 to budget)", who, budget, recent);
    if (n_seqs == 0) return PA_OK;
    if (!keep || !keep_lens || !ctx_lens || (weight_len > 0 && (!weights_out || !weights_in)))
        return fail(PA_ERR_INVALID_ARG, "%s: NULL pointer", who);
    if (mis(keep, 4) || mis(keep_lens, 4) || mis(weights_out, 4) || mis(weights_in, 4) || mis(ctx_lens, 4) ||
        mis(status, 4))
        return fail(PA_ERR_INVALID_ARG, "%s: misaligned pointer", who);
    SelectParams a{keep, keep_lens, weights_out, weights_in, ctx_lens, weight_len, budget, recent, num_heads, status};
    const dim3 grid((unsigned)num_heads, (unsigned)n_seqs);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    const size_t bytes = (size_t)weight_len * 4;
    if (weight_len <= kShort) {
        evict_select_kernel<true, 256><<<grid, 256, bytes, st>>>(a);
    } else if (weight_len <= kCached) {
        if (bytes > 32 * 1024)       // (beside 8 KB of counters)
            e = cudaFuncSetAttribute(evict_select_kernel<true, 1024>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     kCached * 4);
        if (e == cudaSuccess) evict_select_kernel<true, 1024><<<grid, 1024, bytes, st>>>(a);
    } else {
        evict_select_kernel<false, 1024><<<grid, 1024, 0, st>>>(a);
    }
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return fail(PA_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
    return PA_OK;
}

int launch_compact_kv(void *const *k_caches, void *const *v_caches, int32_t num_layers,
                      const int32_t *src_tables, const int32_t *dst_tables, const int32_t *src_lens,
                      const int32_t *first, const int32_t *keep, const int32_t *keep_lens, int32_t keep_heads,
                      int32_t keep_stride, int32_t n_seqs, int32_t max_blocks, const pa_pool_desc *d,
                      int32_t *status, void *stream) {
    const char *who = "pa_compact_kv";
    std::string why;
    if (!d) return fail(PA_ERR_INVALID_ARG, "%s: NULL desc", who);
    if (!device_geometry_ok(d, &why)) return fail(PA_ERR_INVALID_ARG, "%s: %s", who, why.c_str());
    if (num_layers < 0 || num_layers > kMaxMoveLayers || n_seqs < 0 || n_seqs > 65535 || max_blocks < 0 ||
        keep_stride < 0)
        return fail(PA_ERR_INVALID_ARG,
                    "%s: num_layers=%d (<= %d), n_seqs=%d (<= 65535), max_blocks=%d, keep_stride=%d", who,
                    num_layers, kMaxMoveLayers, n_seqs, max_blocks, keep_stride);
    if (keep_heads != 1 && keep_heads != d->num_heads)
        return fail(PA_ERR_INVALID_ARG, "%s: keep_heads=%d is neither 1 nor num_heads=%d", who, keep_heads,
                    d->num_heads);
    if (num_layers == 0 || n_seqs == 0 || keep_stride == 0) return PA_OK;
    if (!k_caches || !v_caches || !src_tables || !dst_tables || !src_lens || !keep || !keep_lens)
        return fail(PA_ERR_INVALID_ARG, "%s: NULL pointer", who);
    if (mis(src_tables, 4) || mis(dst_tables, 4) || mis(src_lens, 4) || mis(first, 4) || mis(keep, 4) ||
        mis(keep_lens, 4) || mis(status, 4))
        return fail(PA_ERR_INVALID_ARG, "%s: misaligned pointer", who);
    CompactParams a{};
    for (int l = 0; l < num_layers; ++l) {
        if (!k_caches[l] || !v_caches[l] || mis(k_caches[l], 16) || mis(v_caches[l], 16))
            return fail(PA_ERR_INVALID_ARG, "%s: cache pointer of layer %d NULL or not 16-byte aligned", who, l);
        a.cache[2 * l] = static_cast<uint4 *>(k_caches[l]);
        a.cache[2 * l + 1] = static_cast<uint4 *>(v_caches[l]);
    }
    // CTAs of their own move each cache, so none may be there twice
    uintptr_t at[2 * kMaxMoveLayers];
    const uintptr_t bytes = (uintptr_t)d->num_blocks * d->num_heads * d->block_size * d->head_dim * 2;
    for (int i = 0; i < 2 * num_layers; ++i) at[i] = reinterpret_cast<uintptr_t>(a.cache[i]);
    std::sort(at, at + 2 * num_layers);
    for (int i = 1; i < 2 * num_layers; ++i)
        if (at[i] - at[i - 1] < bytes) return fail(PA_ERR_INVALID_ARG, "%s: caches overlap", who);
    a.src_tables = src_tables;
    a.dst_tables = dst_tables;
    a.src_lens = src_lens;
    a.first = first;
    a.keep = keep;
    a.keep_lens = keep_lens;
    a.num_heads = d->num_heads;
    a.keep_heads = keep_heads;
    a.keep_stride = keep_stride;
    a.max_blocks = max_blocks;
    a.num_blocks = d->num_blocks;
    while ((1 << a.bshift) < d->block_size) ++a.bshift;
    while ((8 << a.row_shift) < d->head_dim) ++a.row_shift;
    a.status = status;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const unsigned S = (unsigned)n_seqs;
    if (keep_heads > 1 || keep_stride > kShortList) {
        a.cols = 1 << a.row_shift;
        a.rows = kMoveThreads / a.cols;
        a.chunk = std::min(kMaxChunk, a.rows * 8);
        compact_kv_kernel<false><<<dim3((unsigned)d->num_heads, S, (unsigned)(2 * num_layers)), kMoveThreads, 0, st>>>(a);
    } else {
        const int64_t columns = (int64_t)d->num_heads << a.row_shift;
        a.cols = kMoveThreads;
        a.rows = 1;
        a.chunk = 4;
        const int64_t gx = (columns + a.cols - 1) / a.cols;
        if (gx > INT32_MAX) return fail(PA_ERR_INVALID_ARG, "%s: num_heads * head_dim too large", who);
        compact_kv_kernel<true><<<dim3((unsigned)gx, S, (unsigned)num_layers), kMoveThreads, 0, st>>>(a);
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return fail(PA_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
    return PA_OK;
}

}  // namespace pagedkv
