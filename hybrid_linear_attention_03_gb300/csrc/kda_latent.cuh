// kda_latent.cuh -- latent attention: device views, the parameters of its kernels and
// their host entry points.  How the keys of a call are shared out over the CTAs, the
// records of the shares and the walk over items are those of kda_attend.cuh:
//   absorbed  an item is (sequence, group of heads, run of tokens); all heads share a key,
//             so the cache's "heads" are groups of as many as a row tile holds (the last group
//             may have fewer: rows for heads past the last one are worked on as that one's, and not written);
//   expanded  an item is (sequence, head, run of tokens).
#pragma once

#include "kda_attend.cuh"

namespace kda {
namespace kv {

// ---- expanded form: keys and values in rows --------------------------------------
struct RowsView {
    const int32_t *cu, *cu_kv;
    uint32_t *err;
    int32_t n_seqs, max_rows, max_kv_rows, max_new;
};
// As for pages (kda_kv.cuh); of a Seq that passed, rows [cu_kv[n], cu_kv[n] + L) are in [0, max_kv_rows).
__device__ __forceinline__ bool load_seq(const RowsView &b, int n, Seq &s, bool report) {
    const int a = b.cu[n], e = b.cu[n + 1], ka = b.cu_kv[n], ke = b.cu_kv[n + 1];
    const bool ok = a >= 0 && e >= a && e <= b.max_rows && e - a <= b.max_new && ka >= 0 && ke >= ka &&
                    ke <= b.max_kv_rows && ke - ka >= e - a && ke - ka <= kMaxPositions;
    s.row0 = a;
    s.T = ok ? e - a : 0;
    s.L = ok ? ke - ka : 0;
    if (!ok && report) atomicOr(b.err, KDA_DEVERR_META);
    return ok;
}

// What both forms' kernels know of a call's rows and items.
struct LatentRows {
    const void *q_a, *q_r;  // the heads' own part (latent_dim or nope_dim channels), the part that meets kr
    void *out;
    long long qa_stride, qa_head, qr_stride, qr_head, out_stride, out_head;
    int32_t hkv, group;                               // groups of heads, heads of one (the last may have fewer)
    int32_t tile_tokens, key_step, item_cost, min_keys;  // as in AttendParams
    int32_t rope;
    float scale_log2;
    Part *parts;
    float *part_data;
    uint32_t group_inv;
    int32_t heads;  // of all groups
    __device__ __forceinline__ int token_of(int r) const { return int(uint32_t(r) * group_inv >> 16); }
    // token and head of row r of an item (absorbed: one from `heads` on is none)
    __device__ __forceinline__ void locate(const Item &it, int r, long long &row, long long &head) const {
        const int t = token_of(r);
        row = it.row0 + it.tok0 + t, head = it.h * group + r - t * group;
    }
    // likewise; false, and the last head, where the group has no such one
    __device__ __forceinline__ bool locate_head(const Item &it, int r, long long &row, long long &head) const {
        const int t = token_of(r), h = it.h * group + r - t * group;
        row = it.row0 + it.tok0 + t, head = min(h, heads - 1);
        return h < heads;
    }
};
struct LatentParams : LatentRows {
    BatchView b;
    const void *c, *kr;
    const uint8_t *sc;
};
struct PrefillRowsParams : LatentRows {
    RowsView b;
    const void *k, *kr, *v;
    long long k_stride, k_head, kr_stride, v_stride, v_head;
};

inline BatchView make_view(const kda_latent_cache *c, const kda_kv_batch *b) {
    kda_kv_cache pages = {};
    pages.err = c->err, pages.num_pages = c->num_pages, pages.page_size = c->page_size;
    return make_view(&pages, b);
}

// Heads of a group, and groups: the fewest that leave each at most `most` heads, and those as even as that allows.
// (Equal groups only: 67 heads would be 67 groups of one and read the cache as often, 64 single tokens over 4001 to 16384 7010 us.)
struct HeadGroups {
    int each, groups;
};
inline HeadGroups head_groups(int heads, int most) {
    const int n = (heads - 1) / most + 1, each = (heads - 1) / n + 1;
    return {each, (heads - 1) / each + 1};
}

kda_status launch_latent_append(const kda_latent_cache *c, const kda_latent_params *p, const kda_latent_io *io,
                                const kda_kv_batch *b, cudaStream_t stream);
kda_status launch_latent_read(const kda_latent_cache *c, const kda_kv_batch *b, void *c_out, long long c_stride, void *kr_out,
                              long long kr_stride, cudaStream_t stream);
size_t latent_attend_workspace_bytes(const kda_latent_cache *c, const kda_kv_batch *b);
kda_status launch_latent_attend(const kda_latent_cache *c, const kda_latent_attn_io *io, const kda_kv_batch *b,
                                void *workspace, cudaStream_t stream);
size_t latent_prefill_workspace_bytes(const kda_latent_cache *c, const kda_latent_prefill_io *io,
                                      const kda_latent_prefill_batch *b);
kda_status launch_latent_prefill(const kda_latent_cache *c, const kda_latent_prefill_io *io, const kda_latent_prefill_batch *b,
                                 void *workspace, cudaStream_t stream);

// The kernels (see AttendPlan).
bool latent_tile_plan(const kda_latent_cache *c, AttendPlan *plan);
kda_status latent_tile_launch(const kda_latent_cache *c, LatentParams &p, const AttendPlan &plan, cudaStream_t stream);
bool prefill_tile_plan(const kda_latent_cache *c, const kda_latent_prefill_batch *b, AttendPlan *plan);
kda_status prefill_tile_launch(const kda_latent_cache *c, const kda_latent_prefill_io *io, PrefillRowsParams &p,
                               const AttendPlan &plan, cudaStream_t stream);
void latent_generic_plan(int latent, AttendPlan *plan);  // 0: the expanded form
kda_status latent_generic_launch(const kda_latent_cache *c, LatentParams &p, const AttendPlan &plan, cudaStream_t stream);
kda_status prefill_generic_launch(const kda_latent_cache *c, const kda_latent_prefill_io *io, PrefillRowsParams &p,
                                  const AttendPlan &plan, cudaStream_t stream);

}  // namespace kv
}  // namespace kda
