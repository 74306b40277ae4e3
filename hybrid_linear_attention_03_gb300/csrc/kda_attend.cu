// kda_attend.cu -- kda_kv_attend: the choice of kernel, the workspace and the
// kernel that joins an item's parts (see kda_attend.cuh for the sharing-out).
#include <algorithm>

#include "kda_attend.cuh"

namespace kda {
namespace kv {
namespace {

constexpr int kCombineThreads = 256;
constexpr int kCombineRows = kCombineThreads / 32;  // rows of a block: one a warp

// Block (c, y): joins the item whose first part CTA c left, rows
// [8 y, 8 y + 8), a row a warp: with M the largest of the parts' maxima,
//   out = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i.
// Each part is read once.  The blocks of CTAs that cut no item return after one
// load; the others are a chain of three round trips to L2 (records, statistics,
// outputs), so the outputs of 8 parts are asked for at a time.
template <typename Act, int D>
__global__ void __launch_bounds__(kCombineThreads) attend_combine_kernel(const __grid_constant__ AttendParams p, int bm,
                                                                         int n_cta) {
    constexpr int CPL = D >= 32 ? D / 32 : 1, kAhead = 8;  // channels per lane, parts in flight
    const int c = int(blockIdx.x), lane = int(threadIdx.x) & 31, warp = int(threadIdx.x) >> 5;
    const int r = int(blockIdx.y) * kCombineRows + warp;
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
    const int ch = lane * CPL;  // this lane's channels
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
                if (i0 + k < cnt && ch < D) {
                    if constexpr (CPL == 4) {
                        const float4 t = *reinterpret_cast<const float4 *>(d);
                        v[k][0] = t.x, v[k][1] = t.y, v[k][2] = t.z, v[k][3] = t.w;
                    } else if constexpr (CPL == 2) {
                        const float2 t = *reinterpret_cast<const float2 *>(d);
                        v[k][0] = t.x, v[k][1] = t.y;
                    } else {
                        v[k][0] = d[0];
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
    if (ch < D) {
        const int t = p.token_of(r);
        Act *dst = static_cast<Act *>(p.out) + size_t(first.row + t) * size_t(p.out_stride) +
                   size_t(first.h * p.group + r - t * p.group) * D + ch;
#pragma unroll
        for (int e = 0; e < CPL; ++e) dst[e] = from_f32<Act>(acc[e] * inv);
    }
}

template <typename Act, int D>
kda_status combine_d(const AttendParams &p, const AttendPlan &plan, cudaStream_t stream) {
    const long long rows = std::min<long long>(plan.bm, static_cast<long long>(p.b.max_new) * p.group);
    const ProfScope prof(KDA_KERNEL_KV_COMBINE, stream);
    return launch_overlapped(attend_combine_kernel<Act, D>,
                             dim3(unsigned(plan.n_cta), unsigned((rows + kCombineRows - 1) / kCombineRows)),
                             kCombineThreads, 0, stream, p, plan.bm, plan.n_cta);
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

// The kernel of a call, from its sizes and types alone.
struct Choice {
    AttendPlan plan;
    kda_status (*launch)(const kda_kv_cache *, AttendParams &, const AttendPlan &, cudaStream_t);
};
static Choice choose(const kda_kv_cache *c, const kda_kv_batch *b) {
    Choice ch;
    if (few_plan(c, b, &ch.plan)) ch.launch = few_launch;
    else if (lanes_plan(c, b, &ch.plan)) ch.launch = lanes_launch;
    else if (tile_plan(c, b, &ch.plan)) ch.launch = tile_launch;
    else generic_plan(c, b, &ch.plan), ch.launch = generic_launch;
    return ch;
}

size_t attend_workspace_bytes(const kda_kv_cache *c, const kda_kv_batch *b) {
    const AttendPlan plan = choose(c, b).plan;
    return share_bytes(plan.n_cta, plan.bm, c->head_dim);
}

kda_status launch_attend(const kda_kv_cache *c, const kda_attn_io *io, const kda_kv_batch *b, void *workspace,
                         cudaStream_t stream) {
    const Choice ch = choose(c, b);
    const AttendPlan &plan = ch.plan;
    AttendParams p = {};
    p.b = make_view(c, b);
    p.q = io->q, p.out = io->out, p.q_stride = io->q_stride, p.out_stride = io->out_stride;
    p.pk = c->k, p.pv = c->v, p.sk = c->k_scale, p.sv = c->v_scale;
    p.hq = c->num_heads, p.hkv = c->num_kv_heads, p.group = c->num_heads / c->num_kv_heads, p.dim = c->head_dim;
    p.group_inv = (65536u + uint32_t(p.group) - 1) / uint32_t(p.group);
    p.tile_tokens = plan.bm / p.group;
    p.scale_log2 = io->scale * kLog2e;
    p.parts = static_cast<Part *>(workspace);
    p.part_data = reinterpret_cast<float *>(static_cast<char *>(workspace) + parts_bytes(plan.n_cta));
    const kda_status st = ch.launch(c, p, plan, stream);
    // sequences that fit in one key step are never cut: nothing to join (such calls take 8 to 10 us, with it 12)
    if (st != KDA_OK || p.b.max_len <= p.key_step) return st;
    return c->act == KDA_BF16 ? combine<__nv_bfloat16>(c->head_dim, p, plan, stream)
                              : combine<float>(c->head_dim, p, plan, stream);
}

}  // namespace kv
}  // namespace kda
