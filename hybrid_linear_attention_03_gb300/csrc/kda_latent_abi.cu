// kda_latent_abi.cu -- the C ABI of latent attention: argument checks and dispatch.
// Declarations and contracts are in include/kda.h.
#include <nvtx3/nvToolsExt.h>

#include <cmath>

#include "kda_latent.cuh"

namespace {

struct CallRange {  // an NVTX range over an entry point that enqueues device work
    explicit CallRange(const char *name) { nvtxRangePushA(name); }
    ~CallRange() { nvtxRangePop(); }
    CallRange(const CallRange &) = delete;
    CallRange &operator=(const CallRange &) = delete;
};

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool good(const void *p) { return p && aligned(p, 16); }

// What both forms need of a layer's description.
kda_status check_layer(const kda_latent_cache *c) {
    if (!c || !c->err || !aligned(c->err, 4) || c->num_heads <= 0 || c->rope_dim <= 0) return KDA_ERR_INVALID_ARG;
    if (c->act != KDA_F32 && c->act != KDA_BF16) return KDA_ERR_INVALID_ARG;
    if (c->rope_dim != 16 && c->rope_dim != 32 && c->rope_dim != 64) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

kda_status check_cache(const kda_latent_cache *c) {
    if (!c || !good(c->c) || !good(c->kr) || c->num_pages <= 0 || c->page_size <= 0 || c->latent_dim <= 0)
        return KDA_ERR_INVALID_ARG;
    if (c->format != KDA_KV_ACT && c->format != KDA_KV_E4M3) return KDA_ERR_INVALID_ARG;
    if (c->format == KDA_KV_E4M3 && !good(c->c_scale)) return KDA_ERR_INVALID_ARG;
    const kda_status st = check_layer(c);
    if (st != KDA_OK) return st;
    const int P = c->page_size, L = c->latent_dim;
    if (P != 16 && P != 32 && P != 64 && P != 128) return KDA_ERR_UNSUPPORTED;
    if (L != 128 && L != 256 && L != 512) return KDA_ERR_UNSUPPORTED;
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
kda_status check_batch(const kda_latent_prefill_batch *b) {
    if (!b || b->n_seqs < 0 || b->max_rows < 0 || b->max_kv_rows < 0 || b->max_new < 0) return KDA_ERR_INVALID_ARG;
    if (b->n_seqs == 0 || b->max_rows == 0) return KDA_OK;
    if (!b->cu_seqlens || !b->cu_kv || b->max_new == 0 || b->max_kv_rows == 0) return KDA_ERR_INVALID_ARG;
    if (!aligned(b->cu_seqlens, 4) || !aligned(b->cu_kv, 4)) return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

bool empty(const kda_kv_batch *b) { return b->n_seqs == 0 || b->max_rows == 0; }
bool empty(const kda_latent_prefill_batch *b) { return b->n_seqs == 0 || b->max_rows == 0; }

// A stride of vectors of `dim` elements: whole 16-byte pieces, and so short that a row's offset and a tile
// copy's 40-bit byte strides hold it.
bool good_stride(int64_t s, int dim, int act) {
    return s >= dim && s % (act == KDA_BF16 ? 8 : 4) == 0 && s < (int64_t(1) << 37);
}
bool good_rows(const void *p, int64_t stride, int dim, int act) { return good(p) && good_stride(stride, dim, act); }
bool good_heads(const void *p, int64_t stride, int64_t head, int dim, int act) {
    return good_rows(p, stride, dim, act) && good_stride(head, dim, act);
}
bool good_scale(float s) { return s > 0.f && std::isfinite(s * 1.4426950f); }

bool good_params(const kda_latent_params *p, const kda_latent_cache *c) {
    if (!p) return true;
    if (p->c_norm_w && !aligned(p->c_norm_w, 16)) return false;
    if (!std::isfinite(p->eps) || p->eps < 0.f) return false;
    if (p->rot_dim < 0 || p->rot_dim > c->rope_dim || (p->interleaved != 0 && p->interleaved != 1)) return false;
    if (p->rot_dim > 0 && !p->inv_freq) return false;
    for (int i = 0; i < p->rot_dim / 2; ++i)
        if (!std::isfinite(p->inv_freq[i])) return false;
    return true;
}

kda_status check_prefill(const kda_latent_cache *c, const kda_latent_prefill_io *io, const kda_latent_prefill_batch *b) {
    kda_status st = check_layer(c);
    if (st != KDA_OK || (st = check_batch(b)) != KDA_OK) return st;
    if (!io || io->nope_dim <= 0 || io->value_dim <= 0) return KDA_ERR_INVALID_ARG;
    if ((io->nope_dim != 64 && io->nope_dim != 128) || (io->value_dim != 64 && io->value_dim != 128))
        return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

}  // namespace

extern "C" {

kda_status kda_latent_append(const kda_latent_cache *cache, const kda_latent_params *p, const kda_latent_io *io,
                             const kda_kv_batch *batch, kda_stream_t stream) {
    const CallRange range("kda_latent_append");
    kda_status st = check_cache(cache);
    if (st != KDA_OK || (st = check_batch(batch)) != KDA_OK) return st;
    if (!io || (io->q == nullptr) != (io->q_out == nullptr) || !good_params(p, cache)) return KDA_ERR_INVALID_ARG;
    if (p && p->rot_dim % 8 != 0) return KDA_ERR_UNSUPPORTED;
    if (empty(batch)) return KDA_OK;
    const int act = cache->act, R = cache->rope_dim;
    if (!good_rows(io->c, io->c_stride, cache->latent_dim, act) || !good_rows(io->kr, io->kr_stride, R, act))
        return KDA_ERR_INVALID_ARG;
    if (io->q && (!good_heads(io->q, io->q_stride, io->q_head_stride, R, act) ||
                  !good_heads(io->q_out, io->q_out_stride, io->q_out_head_stride, R, act)))
        return KDA_ERR_INVALID_ARG;
    if (io->q && io->q == io->q_out && (io->q_stride != io->q_out_stride || io->q_head_stride != io->q_out_head_stride))
        return KDA_ERR_INVALID_ARG;
    return kda::kv::launch_latent_append(cache, p, io, batch, reinterpret_cast<cudaStream_t>(stream));
}

kda_status kda_latent_read(const kda_latent_cache *cache, const kda_kv_batch *batch, void *c_out, int64_t c_stride,
                           void *kr_out, int64_t kr_stride, kda_stream_t stream) {
    const CallRange range("kda_latent_read");
    kda_status st = check_cache(cache);
    if (st != KDA_OK || (st = check_batch(batch)) != KDA_OK) return st;
    if (empty(batch)) return KDA_OK;
    if (!good_rows(c_out, c_stride, cache->latent_dim, cache->act) || !good_rows(kr_out, kr_stride, cache->rope_dim, cache->act))
        return KDA_ERR_INVALID_ARG;
    return kda::kv::launch_latent_read(cache, batch, c_out, c_stride, kr_out, kr_stride,
                                       reinterpret_cast<cudaStream_t>(stream));
}

size_t kda_latent_attend_workspace_bytes(const kda_latent_cache *cache, const kda_kv_batch *batch) {
    if (check_cache(cache) != KDA_OK || check_batch(batch) != KDA_OK || empty(batch)) return 0;
    return kda::kv::latent_attend_workspace_bytes(cache, batch);
}

kda_status kda_latent_attend(const kda_latent_cache *cache, const kda_latent_attn_io *io, const kda_kv_batch *batch,
                             void *workspace, size_t workspace_bytes, kda_stream_t stream) {
    const CallRange range("kda_latent_attend");
    kda_status st = check_cache(cache);
    if (st != KDA_OK || (st = check_batch(batch)) != KDA_OK) return st;
    if (!io || !good_scale(io->scale)) return KDA_ERR_INVALID_ARG;
    if (empty(batch)) return KDA_OK;
    const int act = cache->act;
    if (!good_heads(io->q_c, io->q_c_stride, io->q_c_head_stride, cache->latent_dim, act) ||
        !good_heads(io->q_r, io->q_r_stride, io->q_r_head_stride, cache->rope_dim, act) ||
        !good_heads(io->out, io->out_stride, io->out_head_stride, cache->latent_dim, act) || io->out == io->q_c ||
        io->out == io->q_r)
        return KDA_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < kda::kv::latent_attend_workspace_bytes(cache, batch))
        return KDA_ERR_WORKSPACE;
    return kda::kv::launch_latent_attend(cache, io, batch, workspace, reinterpret_cast<cudaStream_t>(stream));
}

size_t kda_latent_prefill_workspace_bytes(const kda_latent_cache *cache, const kda_latent_prefill_io *io,
                                          const kda_latent_prefill_batch *batch) {
    if (check_prefill(cache, io, batch) != KDA_OK || empty(batch)) return 0;
    return kda::kv::latent_prefill_workspace_bytes(cache, io, batch);
}

kda_status kda_latent_prefill(const kda_latent_cache *cache, const kda_latent_prefill_io *io,
                              const kda_latent_prefill_batch *batch, void *workspace, size_t workspace_bytes,
                              kda_stream_t stream) {
    const CallRange range("kda_latent_prefill");
    const kda_status st = check_prefill(cache, io, batch);
    if (st != KDA_OK) return st;
    if (!good_scale(io->scale)) return KDA_ERR_INVALID_ARG;
    if (empty(batch)) return KDA_OK;
    const int act = cache->act, dn = io->nope_dim, dv = io->value_dim, R = cache->rope_dim;
    if (!good_heads(io->q_n, io->q_n_stride, io->q_n_head_stride, dn, act) ||
        !good_heads(io->q_r, io->q_r_stride, io->q_r_head_stride, R, act) ||
        !good_heads(io->k, io->k_stride, io->k_head_stride, dn, act) || !good_rows(io->kr, io->kr_stride, R, act) ||
        !good_heads(io->v, io->v_stride, io->v_head_stride, dv, act) ||
        !good_heads(io->out, io->out_stride, io->out_head_stride, dv, act))
        return KDA_ERR_INVALID_ARG;
    for (const void *in : {io->q_n, io->q_r, io->k, io->kr, io->v})
        if (io->out == in) return KDA_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < kda::kv::latent_prefill_workspace_bytes(cache, io, batch))
        return KDA_ERR_WORKSPACE;
    return kda::kv::launch_latent_prefill(cache, io, batch, workspace, reinterpret_cast<cudaStream_t>(stream));
}

kda_status kda_latent_poll_device_error(const kda_latent_cache *cache, kda_stream_t stream, uint32_t *flags) {
    if (!cache || !cache->err) return KDA_ERR_INVALID_ARG;
    kda_kv_cache word = {};
    word.err = cache->err;
    return kda_kv_poll_device_error(&word, stream, flags);
}

}  // extern "C"
