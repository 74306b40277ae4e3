// kda_attend.cu -- kda_kv_attend: the choice of kernel, the workspace and the
// kernel that joins an item's parts (see kda_attend.cuh for the sharing-out).
#include "kda_attend.cuh"

namespace kda {
namespace kv {
namespace {

constexpr int kCombineThreads = 256;
constexpr int kCombineRows = 16;  // rows of a block: two per warp

// Block (c, y): joins the item whose first part CTA c left, rows
// [16 y, 16 y + 16).  A row is one warp's: with M the largest of the parts'
// maxima, out = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i.  Reads each
// part once; the calls that cut few items return after one load.
template <typename Act, int D>
__global__ void __launch_bounds__(kCombineThreads) attend_combine_kernel(const __grid_constant__ AttendParams p, int bm,
                                                                         int n_cta) {
    constexpr int CPL = D >= 32 ? D / 32 : 1;  // channels per lane
    const int c = int(blockIdx.x), lane = int(threadIdx.x) & 31, warp = int(threadIdx.x) >> 5;
    wait_prior_kernel();
    allow_next_kernel();
    const Part first = p.parts[2 * c + 1];
    if (first.state != 1) return;
    int n_parts = 1;  // CTA c's last part, then the first parts of the CTAs after it up to the item's end
    for (int base = c + 1; base < n_cta; base += 32) {
        const int state = base + lane < n_cta ? p.parts[2 * (base + lane)].state : 2;
        const unsigned ends = __ballot_sync(0xffffffffu, state != 1);
        n_parts += ends ? __ffs(ends) : 32;
        if (ends) break;
    }
    n_parts = min(n_parts, n_cta - c);
    Seq sq;
    if (!load_seq(p.b, first.n, sq, false)) return;
    const int tok0 = first.tile * p.tile_tokens, rows = min(p.tile_tokens, sq.T - tok0) * p.group;
    const size_t stride = size_t(bm) * (D + 2);
    auto part_data = [&](int i) { return p.part_data + (size_t(c + i) * 2 + (i == 0 ? 1 : 0)) * stride; };
    for (int r = int(blockIdx.y) * kCombineRows + warp; r < min(rows, int(blockIdx.y + 1) * kCombineRows);
         r += kCombineThreads / 32) {
        float M = -INFINITY;
        for (int i = lane; i < n_parts; i += 32) M = fmaxf(M, part_data(i)[bm * D + r]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        const float ref = M == -INFINITY ? 0.f : M;
        float l = 0.f, acc[CPL];
#pragma unroll
        for (int e = 0; e < CPL; ++e) acc[e] = 0.f;
        for (int base = 0; base < n_parts; base += 32) {
            float f = 0.f;
            if (base + lane < n_parts) {
                const float *d = part_data(base + lane) + bm * D;
                f = exp2f(d[r] - ref);
                l = fmaf(f, d[bm + r], l);
            }
            const int cnt = min(32, n_parts - base);
#pragma unroll 4
            for (int i = 0; i < cnt; ++i) {
                const float fi = __shfl_sync(0xffffffffu, f, i);
                const float *d = part_data(base + i) + size_t(r) * D;
                if constexpr (D >= 32) {
#pragma unroll
                    for (int e = 0; e < CPL; ++e) acc[e] = fmaf(fi, d[e * 32 + lane], acc[e]);
                } else {
                    if (lane < D) acc[0] = fmaf(fi, d[lane], acc[0]);
                }
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        const float inv = l > 0.f || l != l ? 1.0f / l : 0.f;
        Act *dst = static_cast<Act *>(p.out) + size_t(sq.row0 + tok0 + r / p.group) * size_t(p.out_stride) +
                   size_t(first.h * p.group + r % p.group) * D;
#pragma unroll
        for (int e = 0; e < CPL; ++e)
            if (e * 32 + lane < D) dst[e * 32 + lane] = from_f32<Act>(acc[e] * inv);
    }
}

template <typename Act, int D>
kda_status combine_d(const AttendParams &p, const AttendPlan &plan, cudaStream_t stream) {
    const ProfScope prof(KDA_KERNEL_KV_COMBINE, stream);
    return launch_overlapped(attend_combine_kernel<Act, D>,
                             dim3(unsigned(plan.n_cta), unsigned(plan.bm / kCombineRows)), kCombineThreads, 0, stream, p,
                             plan.bm, plan.n_cta);
}

template <typename Act>
kda_status combine(int D, const AttendParams &p, const AttendPlan &plan, cudaStream_t stream) {
    switch (D) {
        case 16: return combine_d<Act, 16>(p, plan, stream);
        case 32: return combine_d<Act, 32>(p, plan, stream);
        case 64: return combine_d<Act, 64>(p, plan, stream);
        case 128: return combine_d<Act, 128>(p, plan, stream);
    }
    return KDA_ERR_UNSUPPORTED;
}

}  // namespace

size_t attend_workspace_bytes(const kda_kv_cache *c, const kda_kv_batch *b) {
    AttendPlan plan;
    if (!tile_plan(c, b, &plan)) generic_plan(c, b, &plan);
    return share_bytes(plan.n_cta, plan.bm, c->head_dim);
}

kda_status launch_attend(const kda_kv_cache *c, const kda_attn_io *io, const kda_kv_batch *b, void *workspace,
                         cudaStream_t stream) {
    AttendPlan plan;
    const bool tile = tile_plan(c, b, &plan);
    if (!tile) generic_plan(c, b, &plan);
    AttendParams p = {};
    p.b = make_view(c, b);
    p.q = io->q, p.out = io->out, p.q_stride = io->q_stride, p.out_stride = io->out_stride;
    p.pk = c->k, p.pv = c->v, p.sk = c->k_scale, p.sv = c->v_scale;
    p.hq = c->num_heads, p.hkv = c->num_kv_heads, p.group = c->num_heads / c->num_kv_heads;
    p.tile_tokens = plan.bm / p.group;
    p.scale_log2 = io->scale * kLog2e;
    p.parts = static_cast<Part *>(workspace);
    p.part_data = reinterpret_cast<float *>(static_cast<char *>(workspace) + parts_bytes(plan.n_cta));
    const kda_status st = tile ? tile_launch(c, p, plan, stream) : generic_launch(c, p, plan, stream);
    if (st != KDA_OK) return st;
    return c->act == KDA_BF16 ? combine<__nv_bfloat16>(c->head_dim, p, plan, stream)
                              : combine<float>(c->head_dim, p, plan, stream);
}

}  // namespace kv
}  // namespace kda
