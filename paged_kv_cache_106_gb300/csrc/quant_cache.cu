// Slot write into a cache of 8 or 4 bits, and reading its rows back
// (definitions in include/pagedkv.h).
//
// Both are streams: the write reads 4 D bytes a (token, head) of keys and values
// and stores 2 (D bits / 8 + D / 16), the read the other way round.  A CTA takes 16
// tokens of 128 dimensions (32 of 64), whose rows are neighbours in a block where
// their slots are, and goes through a range of heads, four of whose loads are in flight at
// once (bound by latency without: the read of 37 thousand tokens x 40 heads into fp16
// blocks 208 us, so 157, 6.2 TB/s).  The write is bound by the issue of the arithmetic
// on its values beside the bytes (69 % of the slots): magnitudes are compared, and
// quotients formed, two at once; 51 thousand tokens x 8 heads into 8 bits take 51 us, 6.3
// TB/s of what they must move, into 4 bits 50 us, 5.3 TB/s.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "pa_internal.h"
#include "quant_device.cuh"

namespace pagedkv {

namespace {

constexpr int kThreads = 256;

struct RowsParams {
    const void *k_in, *v_in;             // write: rows; read: caches
    void *k_out, *v_out;                 // write: caches; read: rows, or fp16 caches
    const int64_t *slots, *out_slots;
    int64_t k_stride, v_stride;          // bytes between tokens (rows)
    int64_t num_slots, out_num_slots;
    int64_t rec;                         // bytes of a (block, head)
    int32_t n_tokens, H, bshift;
    int32_t heads;                       // of a CTA
    int32_t *status;
};

// grid = (16-token tiles (as many rows as a CTA has lanes for), head ranges).  A row
// of lanes keeps its token and goes through the CTA's heads.
template <typename T, int D, int BITS>
__global__ void __launch_bounds__(kThreads) write_quant_kernel(const RowsParams p) {
    using L = quant::Layout<D, BITS>;
    using Piece = typename quant::Codes<BITS>::Piece;
    constexpr int LPR = D / 8, ROWS = kThreads / LPR;
    const int l = threadIdx.x % LPR;
    const int64_t t = (int64_t)blockIdx.x * ROWS + threadIdx.x / LPR;
    int64_t slot = -1;
    if (t < p.n_tokens) {
        slot = p.slots[t];
        if (slot >= p.num_slots) {
            if (l == 0) report(p.status, PA_ERR_BAD_BLOCK);
            slot = -1;
        }
    }
    const int off = (int)(slot & ((1 << p.bshift) - 1));
    const int64_t at = (slot >> p.bshift) * p.H * p.rec;
    const int h0 = blockIdx.y * p.heads, h1 = min(p.H, h0 + p.heads);
    const char *const ks = (const char *)p.k_in + t * p.k_stride + l * 16,
                     *const vs = (const char *)p.v_in + t * p.v_stride + l * 16;
    constexpr int BATCH = 4;                 // heads whose loads are in flight together
    for (int h = h0; h < h1; h += BATCH) {
        uint4 u[BATCH][2];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            u[i][0] = u[i][1] = make_uint4(0, 0, 0, 0);
            if (slot >= 0 && h + i < h1) {
                u[i][0] = *reinterpret_cast<const uint4 *>(ks + (h + i) * (D * 2));
                u[i][1] = *reinterpret_cast<const uint4 *>(vs + (h + i) * (D * 2));
            }
        }
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            if (h + i >= h1) break;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                uint16_t scale;
                const Piece c = quant::encode8<T, BITS>(u[i][kv], scale);
                if (slot >= 0) {
                    char *dst = (char *)(kv ? p.v_out : p.k_out) + at + (h + i) * p.rec;
                    *reinterpret_cast<Piece *>(dst + off * L::kRow + L::piece(l)) = c;
                    if ((l & 3) == 0)
                        *reinterpret_cast<uint16_t *>(dst + (L::kRow << p.bshift) + off * L::kScales + (l >> 2) * 2) =
                            scale;
                }
            }
        }
    }
}

template <typename T, int D, int BITS>
__global__ void __launch_bounds__(kThreads) read_quant_kernel(const RowsParams p) {
    using L = quant::Layout<D, BITS>;
    using Piece = typename quant::Codes<BITS>::Piece;
    constexpr int LPR = D / 8, ROWS = kThreads / LPR;
    const int l = threadIdx.x % LPR;
    const int64_t t = (int64_t)blockIdx.x * ROWS + threadIdx.x / LPR;
    if (t >= p.n_tokens) return;
    const int64_t slot = p.slots[t];
    int64_t to = p.out_slots ? p.out_slots[t] : t;
    if (slot < 0 || to < 0) return;
    if (slot >= p.num_slots || (p.out_slots && to >= p.out_num_slots)) {
        if (l == 0) report(p.status, PA_ERR_BAD_BLOCK);
        return;
    }
    const int mask = (1 << p.bshift) - 1, off = (int)(slot & mask);
    const int64_t at = (slot >> p.bshift) * p.H * p.rec;
    // row of head h in the output: dense rows, or a slot of an fp16 cache
    const int64_t row0 = p.out_slots ? ((to >> p.bshift) * p.H << p.bshift) + (to & mask) : to * p.H;
    const int64_t row_step = p.out_slots ? 1 << p.bshift : 1;
    const int h0 = blockIdx.y * p.heads, h1 = min(p.H, h0 + p.heads);
    const int64_t codes = at + off * L::kRow + L::piece(l), scales = at + (L::kRow << p.bshift) + off * L::kScales + (l >> 2) * 2;
    constexpr int BATCH = 4;                 // heads whose loads are in flight together
    for (int h = h0; h < h1; h += BATCH) {
        Piece c[BATCH][2];
        uint16_t s[BATCH][2];
#pragma unroll
        for (int i = 0; i < BATCH; ++i)
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                const char *src = (const char *)(kv ? p.v_in : p.k_in) + min(h + i, h1 - 1) * p.rec;
                c[i][kv] = *reinterpret_cast<const Piece *>(src + codes);
                s[i][kv] = *reinterpret_cast<const uint16_t *>(src + scales);
            }
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            if (h + i >= h1) break;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                char *dst = (char *)(kv ? p.v_out : p.k_out) + ((row0 + (h + i) * row_step) * D + l * 8) * 2;
                *reinterpret_cast<uint4 *>(dst) = quant::decode8<T, BITS>(c[i][kv], s[i][kv]);
            }
        }
    }
}

bool mis(const void *ptr, int n) { return (reinterpret_cast<uintptr_t>(ptr) & (n - 1)) != 0; }

int sm_count() {
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess ? sm_count_of(dev) : 152;
}

// Heads a CTA goes through: as many as leave 16 CTAs to an SM (40: no difference), at least one.
void grid_of(RowsParams &p, int rows, dim3 &grid) {
    const int64_t tiles = ((int64_t)p.n_tokens + rows - 1) / rows;
    const int64_t want = (int64_t)sm_count() * 16;
    const int64_t ranges = std::min<int64_t>(p.H, std::max<int64_t>(1, (want + tiles - 1) / tiles));
    p.heads = (int)((p.H + ranges - 1) / ranges);
    grid = dim3((unsigned)tiles, (unsigned)((p.H + p.heads - 1) / p.heads));
}

template <bool WRITE, typename T, int D>
void launch_rows(const RowsParams &p0, int bits, cudaStream_t st) {
    RowsParams p = p0;
    dim3 grid;
    grid_of(p, kThreads / (D / 8), grid);
    auto kern = WRITE ? (bits == 4 ? write_quant_kernel<T, D, 4> : write_quant_kernel<T, D, 8>)
                      : (bits == 4 ? read_quant_kernel<T, D, 4> : read_quant_kernel<T, D, 8>);
    kern<<<grid, kThreads, 0, st>>>(p);
}

template <bool WRITE>
int launch_typed(const char *who, const RowsParams &p, int32_t dtype, const pa_pool_desc *d, void *stream) {
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int bits = d->dtype == PA_DTYPE_I8 ? 8 : 4;
    if (dtype == PA_DTYPE_F16)
        d->head_dim == 64 ? launch_rows<WRITE, __half, 64>(p, bits, st) : launch_rows<WRITE, __half, 128>(p, bits, st);
    else
        d->head_dim == 64 ? launch_rows<WRITE, __nv_bfloat16, 64>(p, bits, st)
                          : launch_rows<WRITE, __nv_bfloat16, 128>(p, bits, st);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return fail(PA_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
    return PA_OK;
}

// What both calls check, and the parameters they share.
int common(const char *who, RowsParams &p, int32_t dtype, int32_t n_tokens, const int64_t *slots,
           const pa_pool_desc *d, int32_t *status) {
    std::string why;
    if (!d) return fail(PA_ERR_INVALID_ARG, "%s: NULL desc", who);
    if (!quant_geometry_ok(d, &why)) return fail(PA_ERR_INVALID_ARG, "%s: %s", who, why.c_str());
    if (dtype != PA_DTYPE_F16 && dtype != PA_DTYPE_BF16)
        return fail(PA_ERR_INVALID_ARG, "%s: dtype %d: PA_DTYPE_F16 or PA_DTYPE_BF16", who, dtype);
    if (n_tokens < 0) return fail(PA_ERR_INVALID_ARG, "%s: n_tokens < 0", who);
    if (n_tokens == 0) return PA_OK;
    if (!p.k_in || !p.v_in || !p.k_out || !p.v_out || !slots)
        return fail(PA_ERR_INVALID_ARG, "%s: NULL pointer", who);
    if (mis(p.k_in, 16) || mis(p.v_in, 16) || mis(p.k_out, 16) || mis(p.v_out, 16) || mis(slots, 8) || mis(status, 4))
        return fail(PA_ERR_INVALID_ARG, "%s: misaligned pointer", who);
    p.slots = slots;
    p.num_slots = (int64_t)d->num_blocks * d->block_size;
    p.n_tokens = n_tokens;
    p.H = d->num_heads;
    p.rec = block_bytes(d) / d->num_heads;
    p.bshift = d->block_size == 8 ? 3 : d->block_size == 16 ? 4 : 5;
    p.status = status;
    return PA_OK;
}

}  // namespace

int sm_count_of(int device) {
    static std::atomic<int> counts[64];
    std::atomic<int> *known = device >= 0 && device < 64 ? counts + device : nullptr;
    if (known && known->load(std::memory_order_relaxed) > 0) return known->load(std::memory_order_relaxed);
    int sms = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess || sms <= 0) return 152;
    if (known) known->store(sms, std::memory_order_relaxed);
    return sms;
}

int launch_write_kv_quant(const void *k, const void *v, int32_t dtype, int64_t k_stride, int64_t v_stride,
                          const int64_t *slot_mapping, int32_t n_tokens, void *k_cache, void *v_cache,
                          const pa_pool_desc *d, int32_t *status, void *stream) {
    const char *who = "pa_write_kv_quant";
    RowsParams p{};
    p.k_in = k;
    p.v_in = v;
    p.k_out = k_cache;
    p.v_out = v_cache;
    p.k_stride = k_stride * 2;
    p.v_stride = v_stride * 2;
    const int rc = common(who, p, dtype, n_tokens, slot_mapping, d, status);
    if (rc != PA_OK || n_tokens == 0) return rc;
    if (k_stride < 0 || v_stride < 0 || k_stride % 8 || v_stride % 8 || k_stride > (1ll << 40) || v_stride > (1ll << 40))
        return fail(PA_ERR_INVALID_ARG, "%s: strides %lld and %lld: multiples of 8, not negative", who,
                    (long long)k_stride, (long long)v_stride);
    return launch_typed<true>(who, p, dtype, d, stream);
}

int launch_read_kv_quant(void *k, void *v, int32_t dtype, const int64_t *slot_mapping, const int64_t *out_slots,
                         int32_t out_blocks, int32_t n_tokens, const void *k_cache, const void *v_cache,
                         const pa_pool_desc *d, int32_t *status, void *stream) {
    const char *who = "pa_read_kv_quant";
    RowsParams p{};
    p.k_in = k_cache;
    p.v_in = v_cache;
    p.k_out = k;
    p.v_out = v;
    const int rc = common(who, p, dtype, n_tokens, slot_mapping, d, status);
    if (rc != PA_OK || n_tokens == 0) return rc;
    if (out_slots) {
        if (dtype != PA_DTYPE_F16)
            return fail(PA_ERR_INVALID_ARG, "%s: out_slots go to fp16 caches, dtype is %d", who, dtype);
        if (out_blocks < 0) return fail(PA_ERR_INVALID_ARG, "%s: out_blocks < 0", who);
        if (mis(out_slots, 8)) return fail(PA_ERR_INVALID_ARG, "%s: misaligned pointer", who);
        p.out_slots = out_slots;
        p.out_num_slots = (int64_t)out_blocks * d->block_size;
    }
    return launch_typed<false>(who, p, dtype, d, stream);
}

}  // namespace pagedkv
