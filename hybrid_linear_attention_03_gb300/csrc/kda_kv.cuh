// kda_kv.cuh -- device views of the paged cache and its batch tables, shared
// by the append, read-back and attention kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <utility>

#include "kda_internal.h"

namespace kda {
namespace kv {

constexpr int kMaxGroup = 64;  // query heads per cache head

struct BatchView {
    const int32_t *cu, *lens, *table;
    uint32_t *err;
    int32_t n_seqs, table_stride, max_rows, max_new;
    int32_t num_pages, page_shift;
    int32_t max_len;  // tokens a sequence may have
};

// Positions are 32-bit, and a tile of keys may reach this far past the last one.
constexpr int32_t kMaxPositions = 0x7ffffc00;

struct Seq {
    int row0, T, L;  // first row, new tokens, cache length with them
};

// Reads sequence n's tables; false (and KDA_DEVERR_META when `report`) if
// they are inconsistent.  Of a Seq that passed, rows [row0, row0 + T) are in
// [0, max_rows) and positions [0, L) in the page table's row; a row from
// elsewhere (a search in cu_seqlens) has to be shown to be one of these first.
__device__ __forceinline__ bool load_seq(const BatchView &b, int n, Seq &s, bool report) {
    const int a = b.cu[n], e = b.cu[n + 1], L = b.lens[n];
    const bool ok = a >= 0 && e >= a && e <= b.max_rows && e - a <= b.max_new && L >= e - a &&
                    L <= b.max_len;
    s.row0 = a;
    s.T = ok ? e - a : 0;
    s.L = L;
    if (!ok && report) atomicOr(b.err, KDA_DEVERR_META);
    return ok;
}

// The page that holds position pos of sequence n, or -1 (and
// KDA_DEVERR_PAGE_RANGE) if the table names one outside the cache.
__device__ __forceinline__ int load_page(const BatchView &b, int n, int pos) {
    const int page = b.table[size_t(n) * size_t(b.table_stride) + size_t(pos >> b.page_shift)];
    if (page >= 0 && page < b.num_pages) return page;
    atomicOr(b.err, KDA_DEVERR_PAGE_RANGE);
    return -1;
}

// The last sequence whose first row is at most r (whole warp, every lane gets
// it): each round looks at 32 evenly spaced entries of cu_seqlens, so a few
// hundred sequences take two dependent loads.  n_seqs if r is past the last
// row, -1 if before the first.
__device__ __forceinline__ int find_seq(const BatchView &b, int r, int lane) {
    int lo = 0, len = b.n_seqs + 1;
    bool first = true;
    while (len > 1 || first) {
        first = false;
        const int step = (len + 31) / 32, at = lane * step;
        const unsigned hit = __ballot_sync(0xffffffffu, at < len && b.cu[lo + at] <= r);
        const int k = __popc(hit);
        if (k == 0) return lo - 1;
        lo += (k - 1) * step;
        len = min(step, len - (k - 1) * step);
    }
    return lo;
}

// ---- programmatic dependent launch ----------------------------------------------
__device__ __forceinline__ void wait_prior_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void allow_next_kernel() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ---- e4m3 with a power-of-two scale -----------------------------------------------
// Biased exponent of the smallest 2^e with amax <= 448 * 2^e (448 = 1.75 * 2^8
// is e4m3's largest value); 0 for amax = 0.  A power of two makes scaling
// exact in both directions: the only rounding is the one to e4m3, and a value
// read back is exact in bf16.  It gives up less than one bit of e4m3's range
// at the small end against amax / 448, and its 4 bits of precision not at all.
__device__ __forceinline__ int scale_exponent(float amax) {
    if (amax == 0.f) return 0;
    const uint32_t u = __float_as_uint(amax);
    const int e = int(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return min(max(e, 1), 254);
}
// 2^(127 - e) for the biased exponent e >= 1 (the quantising factor; e = 254
// gives a subnormal, which a finite amax never reaches).
__device__ __forceinline__ float exp2_neg_biased(int e) { return __uint_as_float(uint32_t(254 - e) << 23); }
// 2^(e - 127), e in [0, 254].
__device__ __forceinline__ float exp2_biased(int e) { return __uint_as_float(e == 0 ? 0x400000u : uint32_t(e) << 23); }

__device__ __forceinline__ uint16_t pack_e4m3(float lo, float hi) {  // round to nearest even, saturating
    return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 unpack_e4m3(uint16_t v) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(v, __NV_E4M3);
    return __half22float2(__half2(h));
}

// ---- host ---------------------------------------------------------------------------
inline int page_shift_of(int page_size) { return page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : 7; }

inline BatchView make_view(const kda_kv_cache *c, const kda_kv_batch *b) {
    BatchView v;
    v.cu = b->cu_seqlens;
    v.lens = b->kv_lens;
    v.table = b->page_table;
    v.err = c->err;
    v.n_seqs = b->n_seqs;
    v.table_stride = b->table_stride;
    v.max_rows = b->max_rows;
    v.max_new = b->max_new;
    v.num_pages = c->num_pages;
    v.page_shift = page_shift_of(c->page_size);
    const long long pages_hold = static_cast<long long>(b->table_stride) << v.page_shift;
    v.max_len = pages_hold < kMaxPositions ? int32_t(pages_hold) : kMaxPositions;
    return v;
}

int sm_count();  // of the current device (152 where there is none)

kda_status launch_append(const kda_kv_cache *c, const kda_qk_params *p, const kda_kv_io *io, const kda_kv_batch *b,
                         cudaStream_t stream);
kda_status launch_read(const kda_kv_cache *c, const kda_kv_batch *b, void *k_out, void *v_out, cudaStream_t stream);
size_t attend_workspace_bytes(const kda_kv_cache *c, const kda_kv_batch *b);
kda_status launch_attend(const kda_kv_cache *c, const kda_attn_io *io, const kda_kv_batch *b, void *workspace,
                         cudaStream_t stream);

// A launch that may begin under the preceding kernel (every kernel here waits
// for that kernel's completion before it touches memory).
template <typename... P, typename... A>
inline kda_status launch_overlapped(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                                    A &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(unsigned(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, std::forward<A>(args)...) == cudaSuccess) return KDA_OK;
    cudaGetLastError();
    return KDA_ERR_CUDA;
}

}  // namespace kv
}  // namespace kda
