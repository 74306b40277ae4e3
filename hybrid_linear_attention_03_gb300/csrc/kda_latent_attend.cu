// kda_latent_attend.cu -- kda_latent_attend and kda_latent_prefill: the choice of kernel,
// the workspace and the kernel that joins an item's parts (see kda_attend.cuh for the
// sharing-out).
#include <algorithm>
#include <type_traits>

#include "kda_latent.cuh"

namespace kda {
namespace kv {
namespace {

constexpr int kCombineThreads = 256;
constexpr int kMaxCtas = 320;  // of an attention kernel's grid

// A load that stays where it is written: the compiler moves plain ones to their uses, one after the other.
__device__ __forceinline__ float2 load_now(const float *p) {
    float2 v;
    asm volatile("ld.global.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "l"(p) : "memory");
    return v;
}

// Block (x, y): of the x-th item that was cut, eight (row, slice of channels) pairs, one a
// warp, or two, four warps sharing a pair's parts: with M the largest of the parts' maxima,
//   out = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i,
// in the order of the parts (of the four warps').  A chain of three round trips to L2 (all CTAs' records, statistics,
// outputs), so 16 loads of a lane are asked for at a time: of 16 parts where a slice is 64 channels, of
// fewer where it is a whole row (many items: their blocks are then one wave).  Blocks go by items
// that may be there and not by CTAs: empty ones took longer than the joining (one item: 14 us with them).
template <typename Act, int D, int kSlice, int kShare>
__global__ void __launch_bounds__(kCombineThreads) latent_combine_kernel(const __grid_constant__ LatentRows p, int bm,
                                                                         int n_cta) {
    constexpr int kSlices = D / kSlice, kPieces = kSlice / 64, kMost = 16 / kPieces, kWords = kMaxCtas / 32;
    constexpr int kPairs = kCombineThreads / 32 / kShare;
    static_assert(kShare == 1 || kPieces == 1, "shared sums of one piece a lane");
    __shared__ float s_stat[kPairs][kShare][2];
    __shared__ float2 s_acc[kPairs][kShare][32];
    const int lane = int(threadIdx.x) & 31, pair = int(threadIdx.x >> 5) / kShare, share = int(threadIdx.x >> 5) % kShare;
    const int at = int(blockIdx.y) * kPairs + pair;
    const int r = at / kSlices, ch = at % kSlices * kSlice + lane * 2;
    wait_prior_kernel();
    allow_next_kernel();
    // bit i of word w: CTA 32 w + i left an item's first part, or one in its middle
    uint32_t begins[kWords], goes_on[kWords];
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
        const int i = 32 * w + lane;
        int first = 0, next = 0;
        if (i < n_cta) first = p.parts[2 * i + 1].state, next = p.parts[2 * i].state;
        begins[w] = __ballot_sync(0xffffffffu, first == 1);
        goes_on[w] = __ballot_sync(0xffffffffu, next == 1);
    }
    int skip = int(blockIdx.x), c = -1;
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
        const int n = __popc(begins[w]);
        if (c < 0 && skip < n) {
            uint32_t left = begins[w];
            for (; skip > 0; --skip) left &= left - 1;
            c = 32 * w + __ffs(left) - 1;
        }
        skip -= n;
    }
    if (c < 0) return;
    const Part first = p.parts[2 * c + 1];
    if (kShare == 1 && r >= first.rows) return;
    // its parts: CTA c's last one, then the first ones of the CTAs behind it up to one that ends the item
    int n_parts = 2;
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
        const int from = c + n_parts - 1 - 32 * w;  // the next CTA to look at, in this word
        if (from < 0 || from > 31) continue;
        const uint32_t ends = ~goes_on[w] >> from;
        n_parts += ends ? __ffs(ends) - 1 : 32 - from;
    }
    n_parts = min(n_parts, n_cta - c);
    const size_t stride = size_t(bm) * (D + 2);
    const float *data = p.part_data + size_t(2 * c) * stride;  // part i > 0 at 2 i strides, part 0 at one
    float M = -INFINITY, l = 0.f;
    float2 acc[kPieces];
#pragma unroll
    for (int e = 0; e < kPieces; ++e) acc[e] = make_float2(0.f, 0.f);
    const int per = (n_parts + kShare - 1) / kShare, begin = share * per, end = r < first.rows ? min(begin + per, n_parts) : begin;
    for (int base = begin; base < end; base += 32) {  // 32 parts a round, one statistics pair a lane
        const int i = base + lane, cnt = min(32, end - base);
        float m = -INFINITY, li = 0.f;
        if (i < end) {
            const float *d = data + size_t(i == 0 ? 1 : 2 * i) * stride + size_t(bm) * D;
            m = d[r], li = d[bm + r];
        }
        float top = m;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        top = fmaxf(top, M);
        const float ref = top == -INFINITY ? 0.f : top, back = exp2f(M - ref);
        const float f = i < end ? exp2f(m - ref) : 0.f;
        M = top;
        l = l * back + f * li;
#pragma unroll
        for (int e = 0; e < kPieces; ++e) acc[e].x *= back, acc[e].y *= back;
        // outputs of N parts at a time, past the last one it again
        auto add = [&](auto n, int k0) {
            constexpr int N = decltype(n)::value;
            float2 v[N][kPieces];
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const int ii = base + min(k0 + k, cnt - 1);
                const float *d = data + size_t(ii == 0 ? 1 : 2 * ii) * stride + size_t(r) * D + ch;
#pragma unroll
                for (int e = 0; e < kPieces; ++e) v[k][e] = load_now(d + e * 64);
            }
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const float fk = __shfl_sync(0xffffffffu, f, (k0 + k) & 31);
                if (k0 + k < cnt)
#pragma unroll
                    for (int e = 0; e < kPieces; ++e)
                        acc[e].x = fmaf(fk, v[k][e].x, acc[e].x), acc[e].y = fmaf(fk, v[k][e].y, acc[e].y);
            }
        };
        int k0 = 0;
        if constexpr (kMost > 4)
            for (; cnt - k0 > 4; k0 += kMost) add(std::integral_constant<int, kMost>(), k0);
        constexpr int kRest = kMost < 4 ? kMost : 4;
        for (; k0 < cnt; k0 += kRest) add(std::integral_constant<int, kRest>(), k0);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if constexpr (kShare > 1) {
        if (lane == 0) s_stat[pair][share][0] = M, s_stat[pair][share][1] = l;
        s_acc[pair][share][lane] = acc[0];
        __syncthreads();
        if (share != 0 || r >= first.rows) return;
#pragma unroll
        for (int g = 0; g < kShare; ++g) M = fmaxf(M, s_stat[pair][g][0]);
        const float ref = M == -INFINITY ? 0.f : M;
        l = 0.f, acc[0] = make_float2(0.f, 0.f);
#pragma unroll
        for (int g = 0; g < kShare; ++g) {
            const float f = exp2f(s_stat[pair][g][0] - ref);
            const float2 v = s_acc[pair][g][lane];
            l = fmaf(f, s_stat[pair][g][1], l);
            acc[0].x = fmaf(f, v.x, acc[0].x), acc[0].y = fmaf(f, v.y, acc[0].y);
        }
    }
    const float inv = l > 0.f || l != l ? 1.0f / l : 0.f;
    const int t = p.token_of(r), head = first.h * p.group + r - t * p.group;
    if (head >= p.heads) return;
    Act *dst = static_cast<Act *>(p.out) + (static_cast<long long>(first.row) + t) * p.out_stride +
               static_cast<long long>(head) * p.out_head + ch;
#pragma unroll
    for (int e = 0; e < kPieces; ++e) {
        if constexpr (sizeof(Act) == 2)
            *reinterpret_cast<__nv_bfloat162 *>(dst + e * 64) = __floats2bfloat162_rn(acc[e].x * inv, acc[e].y * inv);
        else
            *reinterpret_cast<float2 *>(dst + e * 64) = make_float2(acc[e].x * inv, acc[e].y * inv);
    }
}

template <typename Act, int D, int kSlice, int kShare>
kda_status combine_as(const LatentRows &p, const AttendPlan &plan, long long rows, long long cut, cudaStream_t stream) {
    constexpr int kPer = kCombineThreads / 32 / kShare;
    const dim3 grid(unsigned(cut), unsigned((rows * (D / kSlice) + kPer - 1) / kPer));
    // The blocks come as the attention's CTAs leave, and as many to an SM as it holds: shared memory that they do not
    // use spreads them over the SMs (without it 64 of them met on 8 SMs: one sequence of 65536 tokens 84 us against 49).
    const int per_sm = int((static_cast<long long>(grid.x) * grid.y + sm_count() - 1) / sm_count());
    const size_t smem = per_sm >= 8 ? 0 : size_t(200 * 1024 / per_sm) & ~size_t(1023);
    if (!allow_smem<latent_combine_kernel<Act, D, kSlice, kShare>>(200 * 1024)) return KDA_ERR_CUDA;
    return launch_overlapped(latent_combine_kernel<Act, D, kSlice, kShare>, grid, kCombineThreads, smem, stream, p, plan.bm,
                             plan.n_cta);
}
template <typename Act, int D>
kda_status combine_d(const LatentRows &p, const AttendPlan &plan, long long rows, long long items, cudaStream_t stream) {
    const long long cut = std::min<long long>(items, plan.n_cta), one_wave = 8LL * 8 * sm_count();  // warps
    const ProfScope prof(KDA_KERNEL_LATENT_COMBINE, stream);
    // Few items, of many parts each: four warps share a slice's; many: a warp has a whole row.  The joining alone (L2 cold),
    // us, shared, by slices and by rows (64 rows of 512 channels): 1 item 12, 18, 65; 4 items 15.9, 11.8, 26; 12 items 26, 11.8, 13.9;
    // 16 items 32, 13.9, 12.0; 64 items 112, 26, 13.
    if (cut * rows * (D / 64) * 8 <= one_wave) return combine_as<Act, D, 64, 4>(p, plan, rows, cut, stream);
    if constexpr (D > 64)
        if (cut * rows * (D / 64) * 4 > one_wave * 3) return combine_as<Act, D, D, 1>(p, plan, rows, cut, stream);
    return combine_as<Act, D, 64, 1>(p, plan, rows, cut, stream);
}
template <typename Act>
kda_status combine_t(int D, const LatentRows &p, const AttendPlan &plan, long long rows, long long items, cudaStream_t s) {
    switch (D) {
        case 64: return combine_d<Act, 64>(p, plan, rows, items, s);
        case 128: return combine_d<Act, 128>(p, plan, rows, items, s);
        case 256: return combine_d<Act, 256>(p, plan, rows, items, s);
        case 512: return combine_d<Act, 512>(p, plan, rows, items, s);
    }
    return KDA_ERR_UNSUPPORTED;
}
// max_new and n_seqs bound the rows of a tile and the items there may be
kda_status combine(int act, int D, const LatentRows &p, const AttendPlan &plan, int max_new, int n_seqs, cudaStream_t s) {
    const long long rows = std::min<long long>(p.tile_tokens, max_new) * p.group;
    const long long items = static_cast<long long>(n_seqs) * p.hkv * ((max_new - 1) / p.tile_tokens + 1);
    return act == KDA_BF16 ? combine_t<__nv_bfloat16>(D, p, plan, rows, items, s) : combine_t<float>(D, p, plan, rows, items, s);
}

void set_items(LatentRows &p, const AttendPlan &plan, int heads, HeadGroups g, float scale, void *workspace) {
    p.hkv = g.groups, p.group = g.each, p.heads = heads;
    p.group_inv = (65536u + uint32_t(g.each) - 1) / uint32_t(g.each);
    p.tile_tokens = plan.bm / g.each;
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
    else latent_generic_plan(c->latent_dim, &ch.plan), ch.launch = latent_generic_launch;
    ch.plan.n_cta = std::min(ch.plan.n_cta, kMaxCtas);
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
    set_items(p, plan, c->num_heads, head_groups(c->num_heads, plan.bm), io->scale, workspace);
    const kda_status st = ch.launch(c, p, plan, stream);
    if (st != KDA_OK || p.b.max_len <= p.key_step) return st;  // sequences of one key step are never cut
    return combine(c->act, c->latent_dim, p, plan, b->max_new, b->n_seqs, stream);
}

struct PrefillChoice {
    AttendPlan plan;
    kda_status (*launch)(const kda_latent_cache *, const kda_latent_prefill_io *, PrefillRowsParams &, const AttendPlan &,
                         cudaStream_t);
};
static PrefillChoice choose(const kda_latent_cache *c, const kda_latent_prefill_batch *b) {
    PrefillChoice ch;
    if (prefill_tile_plan(c, b, &ch.plan)) ch.launch = prefill_tile_launch;
    else latent_generic_plan(0, &ch.plan), ch.launch = prefill_generic_launch;
    ch.plan.n_cta = std::min(ch.plan.n_cta, kMaxCtas);
    return ch;
}

size_t latent_prefill_workspace_bytes(const kda_latent_cache *c, const kda_latent_prefill_io *io,
                                      const kda_latent_prefill_batch *b) {
    const AttendPlan plan = choose(c, b).plan;
    return share_bytes(plan.n_cta, plan.bm, io->value_dim);
}

kda_status launch_latent_prefill(const kda_latent_cache *c, const kda_latent_prefill_io *io, const kda_latent_prefill_batch *b,
                                 void *workspace, cudaStream_t stream) {
    const PrefillChoice ch = choose(c, b);
    const AttendPlan &plan = ch.plan;
    PrefillRowsParams p = {};
    p.b = RowsView{b->cu_seqlens, b->cu_kv, c->err, b->n_seqs, b->max_rows, b->max_kv_rows, b->max_new};
    p.q_a = io->q_n, p.q_r = io->q_r, p.out = io->out;
    p.qa_stride = io->q_n_stride, p.qa_head = io->q_n_head_stride;
    p.qr_stride = io->q_r_stride, p.qr_head = io->q_r_head_stride;
    p.out_stride = io->out_stride, p.out_head = io->out_head_stride;
    p.k = io->k, p.kr = io->kr, p.v = io->v, p.rope = c->rope_dim;
    p.k_stride = io->k_stride, p.k_head = io->k_head_stride, p.kr_stride = io->kr_stride;
    p.v_stride = io->v_stride, p.v_head = io->v_head_stride;
    set_items(p, plan, c->num_heads, HeadGroups{1, c->num_heads}, io->scale, workspace);
    const kda_status st = ch.launch(c, io, p, plan, stream);
    if (st != KDA_OK || b->max_kv_rows <= p.key_step) return st;
    return combine(c->act, io->value_dim, p, plan, b->max_new, b->n_seqs, stream);
}

}  // namespace kv
}  // namespace kda
