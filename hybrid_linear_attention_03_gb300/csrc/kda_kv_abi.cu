// kda_kv_abi.cu -- the C ABI of the paged cache: argument checks and dispatch.
// Declarations and contracts are in include/kda.h.
#include <nvtx3/nvToolsExt.h>

#include <cmath>

#include "kda_kv.cuh"

namespace {

struct CallRange {  // an NVTX range over an entry point that enqueues device work
    explicit CallRange(const char *name) { nvtxRangePushA(name); }
    ~CallRange() { nvtxRangePop(); }
    CallRange(const CallRange &) = delete;
    CallRange &operator=(const CallRange &) = delete;
};

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool good(const void *p) { return p && aligned(p, 16); }

kda_status check_cache(const kda_kv_cache *c) {
    if (!c || !good(c->k) || !good(c->v) || !c->err || !aligned(c->err, 4)) return KDA_ERR_INVALID_ARG;
    if (c->num_pages <= 0 || c->page_size <= 0 || c->num_heads <= 0 || c->num_kv_heads <= 0 || c->head_dim <= 0)
        return KDA_ERR_INVALID_ARG;
    if ((c->act != KDA_F32 && c->act != KDA_BF16) || (c->format != KDA_KV_ACT && c->format != KDA_KV_E4M3))
        return KDA_ERR_INVALID_ARG;
    if (c->format == KDA_KV_E4M3 && (!good(c->k_scale) || !good(c->v_scale))) return KDA_ERR_INVALID_ARG;
    if (c->num_heads % c->num_kv_heads != 0) return KDA_ERR_INVALID_ARG;
    const int P = c->page_size, D = c->head_dim;
    if (P != 16 && P != 32 && P != 64 && P != 128) return KDA_ERR_UNSUPPORTED;
    if (D != 16 && D != 32 && D != 64 && D != 128) return KDA_ERR_UNSUPPORTED;
    if (c->num_heads / c->num_kv_heads > kda::kv::kMaxGroup) return KDA_ERR_UNSUPPORTED;
    // page * heads is a 32-bit coordinate of the tile copies, and a row's channels a 32-bit offset
    if (static_cast<long long>(c->num_pages) * c->num_kv_heads > 0x7fffffffLL ||
        static_cast<long long>(c->num_heads) * D > 0x7fffffffLL)
        return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

kda_status check_batch(const kda_kv_batch *b) {
    if (!b || b->n_seqs < 0 || b->max_rows < 0 || b->max_new < 0) return KDA_ERR_INVALID_ARG;
    if (b->n_seqs == 0 || b->max_rows == 0) return KDA_OK;
    if (!b->cu_seqlens || !b->kv_lens || !b->page_table || b->table_stride <= 0 || b->max_new == 0)
        return KDA_ERR_INVALID_ARG;
    if (!aligned(b->cu_seqlens, 4) || !aligned(b->kv_lens, 4) || !aligned(b->page_table, 4)) return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

bool empty(const kda_kv_batch *b) { return b->n_seqs == 0 || b->max_rows == 0; }

// A row tensor: 16-byte rows, wide enough for its heads.
bool good_rows(const void *p, int64_t stride, int heads, const kda_kv_cache *c) {
    const int64_t unit = c->act == KDA_BF16 ? 8 : 4;
    return good(p) && stride >= int64_t(heads) * c->head_dim && stride % unit == 0;
}

bool good_params(const kda_qk_params *p, const kda_kv_cache *c) {
    if (!p) return true;
    if ((p->q_norm_w && !aligned(p->q_norm_w, 16)) || (p->k_norm_w && !aligned(p->k_norm_w, 16))) return false;
    if (!std::isfinite(p->eps) || p->eps < 0.f) return false;
    if (p->rot_dim < 0 || p->rot_dim > c->head_dim || (p->interleaved != 0 && p->interleaved != 1)) return false;
    if (p->rot_dim > 0 && !p->inv_freq) return false;
    for (int i = 0; i < p->rot_dim / 2; ++i)
        if (!std::isfinite(p->inv_freq[i])) return false;
    return true;
}

}  // namespace

extern "C" {

kda_status kda_kv_append(const kda_kv_cache *cache, const kda_qk_params *p, const kda_kv_io *io,
                         const kda_kv_batch *batch, kda_stream_t stream) {
    const CallRange range("kda_kv_append");
    kda_status st = check_cache(cache);
    if (st != KDA_OK || (st = check_batch(batch)) != KDA_OK) return st;
    if (!io || (io->q == nullptr) != (io->q_out == nullptr) || !good_params(p, cache)) return KDA_ERR_INVALID_ARG;
    if (p && p->rot_dim % 8 != 0) return KDA_ERR_UNSUPPORTED;
    if (empty(batch)) return KDA_OK;
    if (!good_rows(io->k, io->k_stride, cache->num_kv_heads, cache) ||
        !good_rows(io->v, io->v_stride, cache->num_kv_heads, cache))
        return KDA_ERR_INVALID_ARG;
    if (io->q && (!good_rows(io->q, io->q_stride, cache->num_heads, cache) ||
                  !good_rows(io->q_out, io->q_out_stride, cache->num_heads, cache)))
        return KDA_ERR_INVALID_ARG;
    if (io->q && io->q == io->q_out && io->q_stride != io->q_out_stride) return KDA_ERR_INVALID_ARG;
    return kda::kv::launch_append(cache, p, io, batch, reinterpret_cast<cudaStream_t>(stream));
}

kda_status kda_kv_read(const kda_kv_cache *cache, const kda_kv_batch *batch, void *k_out, void *v_out,
                       kda_stream_t stream) {
    const CallRange range("kda_kv_read");
    kda_status st = check_cache(cache);
    if (st != KDA_OK || (st = check_batch(batch)) != KDA_OK) return st;
    if (empty(batch)) return KDA_OK;
    if (!good(k_out) || !good(v_out)) return KDA_ERR_INVALID_ARG;
    return kda::kv::launch_read(cache, batch, k_out, v_out, reinterpret_cast<cudaStream_t>(stream));
}

size_t kda_kv_attend_workspace_bytes(const kda_kv_cache *cache, const kda_kv_batch *batch) {
    if (check_cache(cache) != KDA_OK || check_batch(batch) != KDA_OK || empty(batch)) return 0;
    return kda::kv::attend_workspace_bytes(cache, batch);
}

kda_status kda_kv_attend(const kda_kv_cache *cache, const kda_attn_io *io, const kda_kv_batch *batch, void *workspace,
                         size_t workspace_bytes, kda_stream_t stream) {
    const CallRange range("kda_kv_attend");
    kda_status st = check_cache(cache);
    if (st != KDA_OK || (st = check_batch(batch)) != KDA_OK) return st;
    if (!io || !(io->scale > 0.f) || !std::isfinite(io->scale * 1.4426950f)) return KDA_ERR_INVALID_ARG;
    if (empty(batch)) return KDA_OK;
    if (!good_rows(io->q, io->q_stride, cache->num_heads, cache) ||
        !good_rows(io->out, io->out_stride, cache->num_heads, cache) || io->q == io->out)
        return KDA_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < kda::kv::attend_workspace_bytes(cache, batch))
        return KDA_ERR_WORKSPACE;
    return kda::kv::launch_attend(cache, io, batch, workspace, reinterpret_cast<cudaStream_t>(stream));
}

kda_status kda_kv_poll_device_error(const kda_kv_cache *cache, kda_stream_t stream, uint32_t *flags) {
    if (!cache || !cache->err) return KDA_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    uint32_t word = 0;
    if (cudaMemcpyAsync(&word, cache->err, sizeof(word), cudaMemcpyDeviceToHost, s) != cudaSuccess ||
        cudaMemsetAsync(cache->err, 0, sizeof(word), s) != cudaSuccess || cudaStreamSynchronize(s) != cudaSuccess) {
        cudaGetLastError();
        return KDA_ERR_CUDA;
    }
    if (flags) *flags = word;
    return word ? KDA_ERR_DEVICE : KDA_OK;
}

}  // extern "C"
