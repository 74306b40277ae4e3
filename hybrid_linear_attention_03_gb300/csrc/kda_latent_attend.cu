// kda_latent_attend.cu -- kda_latent_attend and kda_latent_prefill: the choice of kernel,
// the workspace and the kernel that joins an item's parts (see kda_attend.cuh for the
// sharing-out).
#include <algorithm>

#include "kda_latent.cuh"

namespace kda {
namespace kv {
namespace {

constexpr int kCombineThreads = 256;
constexpr int kSlice = 128;  // channels that a warp joins of a row, four a lane (64 of values of 64)

// Block (c, y): of the item whose first part CTA c left, eight (row, slice of channels)
// pairs, one a warp: with M the largest of the parts' maxima,
//   out = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i,
// in the order of the parts.  The blocks of CTAs that cut no item return after one load; the others are a
// chain of three round trips to L2, so the outputs of 16 parts are asked for at a time.
template <typename Act, int D>
__global__ void __launch_bounds__(kCombineThreads) latent_combine_kernel(const __grid_constant__ LatentRows p, int bm,
                                                                         int n_cta) {
    constexpr int W = D < kSlice ? D : kSlice, kSlices = D / W, CPL = W / 32, kAhead = 16;
    const int c = int(blockIdx.x), lane = int(threadIdx.x) & 31;
    const int at = int(blockIdx.y) * (kCombineThreads / 32) + int(threadIdx.x >> 5);
    const int r = at / kSlices, ch = at % kSlices * W + lane * CPL;
    wait_prior_kernel();
    allow_next_kernel();
    const Part first = p.parts[2 * c + 1];
    // the parts after CTA c's last one: the first parts of the CTAs behind it, up to the item's end
    const int state = c + 1 + lane < n_cta ? p.parts[2 * (c + 1 + lane)].state : 2;
    if (first.state != 1 || r >= first.rows) return;
    unsigned ends = __ballot_sync(0xffffffffu, state != 1);
    int n_parts = 1 + (ends ? __ffs(ends) : 32);
    for (int base = c + 33; !ends && base < n_cta; base += 32) {
        ends = __ballot_sync(0xffffffffu, base + lane >= n_cta || p.parts[2 * (base + lane)].state != 1);
        n_parts += ends ? __ffs(ends) : 32;
    }
    n_parts = min(n_parts, n_cta - c);
    const size_t stride = size_t(bm) * (D + 2);
    const float *data = p.part_data + size_t(2 * c) * stride;  // part i > 0 at 2 i strides, part 0 at one
    float M = -INFINITY, l = 0.f, acc[CPL];
#pragma unroll
    for (int e = 0; e < CPL; ++e) acc[e] = 0.f;
    for (int base = 0; base < n_parts; base += 32) {  // 32 parts a round, one statistics pair a lane
        const int i = base + lane;
        float m = -INFINITY, li = 0.f;
        if (i < n_parts) {
            const float *d = data + size_t(i == 0 ? 1 : 2 * i) * stride + size_t(bm) * D;
            m = d[r], li = d[bm + r];
        }
        float top = m;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        top = fmaxf(top, M);
        const float ref = top == -INFINITY ? 0.f : top, back = exp2f(M - ref);
        const float f = i < n_parts ? exp2f(m - ref) : 0.f;
        M = top;
        l = l * back + f * li;
#pragma unroll
        for (int e = 0; e < CPL; ++e) acc[e] *= back;
        const int cnt = min(32, n_parts - base);
        for (int i0 = 0; i0 < cnt; i0 += kAhead) {
            float v[kAhead][CPL];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int ii = base + i0 + k;
                const float *d = data + size_t(ii == 0 ? 1 : 2 * ii) * stride + size_t(r) * D + ch;
#pragma unroll
                for (int e = 0; e < CPL; ++e) v[k][e] = 0.f;
                if (i0 + k < cnt) {
                    if constexpr (CPL == 4) {
                        const float4 t = *reinterpret_cast<const float4 *>(d);
                        v[k][0] = t.x, v[k][1] = t.y, v[k][2] = t.z, v[k][3] = t.w;
                    } else {
                        const float2 t = *reinterpret_cast<const float2 *>(d);
                        v[k][0] = t.x, v[k][1] = t.y;
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const float fk = __shfl_sync(0xffffffffu, f, (i0 + k) & 31);
                if (i0 + k < cnt)
#pragma unroll
                    for (int e = 0; e < CPL; ++e) acc[e] = fmaf(fk, v[k][e], acc[e]);
            }
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    const float inv = l > 0.f || l != l ? 1.0f / l : 0.f;
    const int t = p.token_of(r);
    Act *dst = static_cast<Act *>(p.out) + (static_cast<long long>(first.row) + t) * p.out_stride +
               (static_cast<long long>(first.h) * p.group + r - t * p.group) * p.out_head + ch;
#pragma unroll
    for (int e = 0; e < CPL; ++e) dst[e] = from_f32<Act>(acc[e] * inv);
}

template <typename Act, int D>
kda_status combine_d(const LatentRows &p, const AttendPlan &plan, long long rows, cudaStream_t stream) {
    const long long work = rows * (D < kSlice ? 1 : D / kSlice);
    const ProfScope prof(KDA_KERNEL_LATENT_COMBINE, stream);
    return launch_overlapped(latent_combine_kernel<Act, D>,
                             dim3(unsigned(plan.n_cta), unsigned((work + kCombineThreads / 32 - 1) / (kCombineThreads / 32))),
                             kCombineThreads, 0, stream, p, plan.bm, plan.n_cta);
}
template <typename Act> kda_status combine_t(int D, const LatentRows &p, const AttendPlan &plan, long long rows, cudaStream_t s) {
    switch (D) {
        case 64: return combine_d<Act, 64>(p, plan, rows, s);
        case 128: return combine_d<Act, 128>(p, plan, rows, s);
        case 256: return combine_d<Act, 256>(p, plan, rows, s);
        case 512: return combine_d<Act, 512>(p, plan, rows, s);
    }
    return KDA_ERR_UNSUPPORTED;
}
// rows: of a tile, at most
kda_status combine(int act, int D, const LatentRows &p, const AttendPlan &plan, int max_new, cudaStream_t s) {
    const long long rows = std::min<long long>(p.tile_tokens, max_new) * p.group;
    return act == KDA_BF16 ? combine_t<__nv_bfloat16>(D, p, plan, rows, s) : combine_t<float>(D, p, plan, rows, s);
}

void set_items(LatentRows &p, const AttendPlan &plan, int groups, int group, float scale, void *workspace) {
    p.hkv = groups, p.group = group;
    p.group_inv = (65536u + uint32_t(group) - 1) / uint32_t(group);
    p.tile_tokens = plan.bm / group;
    p.scale_log2 = scale * kLog2e;
    p.parts = static_cast<Part *>(workspace);
    p.part_data = reinterpret_cast<float *>(static_cast<char *>(workspace) + parts_bytes(plan.n_cta));
}

}  // namespace

// The kernel of a call, from its sizes and types alone.
struct LatentChoice {
    AttendPlan plan;
    kda_status (*launch)(const kda_latent_cache *, LatentParams &, const AttendPlan &, cudaStream_t);
};
static LatentChoice choose(const kda_latent_cache *c) {
    LatentChoice ch;
    if (latent_tile_plan(c, &ch.plan)) ch.launch = latent_tile_launch;
    else latent_generic_plan(&ch.plan), ch.launch = latent_generic_launch;
    return ch;
}

size_t latent_attend_workspace_bytes(const kda_latent_cache *c, const kda_kv_batch *) {
    const AttendPlan plan = choose(c).plan;
    return share_bytes(plan.n_cta, plan.bm, c->latent_dim);
}

kda_status launch_latent_attend(const kda_latent_cache *c, const kda_latent_attn_io *io, const kda_kv_batch *b,
                                void *workspace, cudaStream_t stream) {
    const LatentChoice ch = choose(c);
    const AttendPlan &plan = ch.plan;
    LatentParams p = {};
    p.b = make_view(c, b);
    p.q_a = io->q_c, p.q_r = io->q_r, p.out = io->out;
    p.qa_stride = io->q_c_stride, p.qa_head = io->q_c_head_stride;
    p.qr_stride = io->q_r_stride, p.qr_head = io->q_r_head_stride;
    p.out_stride = io->out_stride, p.out_head = io->out_head_stride;
    p.c = c->c, p.kr = c->kr, p.sc = c->c_scale, p.rope = c->rope_dim;
    const int groups = head_groups(c->num_heads, plan.bm);
    set_items(p, plan, groups, c->num_heads / groups, io->scale, workspace);
    const kda_status st = ch.launch(c, p, plan, stream);
    if (st != KDA_OK || p.b.max_len <= p.key_step) return st;  // sequences of one key step are never cut
    return combine(c->act, c->latent_dim, p, plan, b->max_new, stream);
}

static AttendPlan choose(const kda_latent_cache *c, const kda_latent_prefill_io *, const kda_latent_prefill_batch *) {
    AttendPlan plan;
    (void)c;
    latent_generic_plan(&plan);
    return plan;
}

size_t latent_prefill_workspace_bytes(const kda_latent_cache *c, const kda_latent_prefill_io *io,
                                      const kda_latent_prefill_batch *b) {
    const AttendPlan plan = choose(c, io, b);
    return share_bytes(plan.n_cta, plan.bm, io->value_dim);
}

kda_status launch_latent_prefill(const kda_latent_cache *c, const kda_latent_prefill_io *io, const kda_latent_prefill_batch *b,
                                 void *workspace, cudaStream_t stream) {
    const AttendPlan plan = choose(c, io, b);
    PrefillRowsParams p = {};
    p.b = RowsView{b->cu_seqlens, b->cu_kv, c->err, b->n_seqs, b->max_rows, b->max_kv_rows, b->max_new};
    p.q_a = io->q_n, p.q_r = io->q_r, p.out = io->out;
    p.qa_stride = io->q_n_stride, p.qa_head = io->q_n_head_stride;
    p.qr_stride = io->q_r_stride, p.qr_head = io->q_r_head_stride;
    p.out_stride = io->out_stride, p.out_head = io->out_head_stride;
    p.k = io->k, p.kr = io->kr, p.v = io->v, p.rope = c->rope_dim;
    p.k_stride = io->k_stride, p.k_head = io->k_head_stride, p.kr_stride = io->kr_stride;
    p.v_stride = io->v_stride, p.v_head = io->v_head_stride;
    set_items(p, plan, c->num_heads, 1, io->scale, workspace);
    const kda_status st = prefill_generic_launch(c, io, p, plan, stream);
    if (st != KDA_OK || b->max_kv_rows <= p.key_step) return st;
    return combine(c->act, io->value_dim, p, plan, b->max_new, stream);
}

}  // namespace kv
}  // namespace kda
