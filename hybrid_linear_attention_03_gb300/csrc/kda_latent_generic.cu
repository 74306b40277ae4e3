// kda_latent_generic.cu -- latent attention in 32 bits on the CUDA cores, both forms
// (the tensor cores have no 32-bit products).
//
// One pass over the keys with a softmax's running maximum and sum, as in
// kda_attend_generic.cu.  A CTA holds 32 rows and walks 32 keys a step through shared
// memory: 16 threads side by side share two rows of the scores with two keys each; then
// 64 threads share 8 rows of the outputs, DV / 64 channels each, in registers.  In the
// absorbed form a key's first channels are its value, so the tile is read once for both.  Bound by the
// reads of shared memory behind its multiplications: 8 of them for 48 bytes of scores, 8 for 16 of outputs.
#include <algorithm>
#include <type_traits>

#include "kda_latent.cuh"

namespace kda {
namespace kv {
namespace {

constexpr int BM = 32, KS = 32, kThreads = 256;
// In place of the weight of a key that the row does not see (or that scores -inf), whose value may be anything.  Not 0: a key
// that the row does see may weigh that little, and 0 * infinity is NaN in every tile.
constexpr float kUnseen = -1.f;

__device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 load4(const uint8_t *p) {
    const uint32_t r = *reinterpret_cast<const uint32_t *>(p);
    const float2 a = unpack_e4m3(uint16_t(r)), b = unpack_e4m3(uint16_t(r >> 16));
    return make_float4(a.x, a.y, b.x, b.y);
}

// Where a key's parts are, by form.
struct KeyAt {
    long long line;  // vector index (absorbed) or row (expanded), -1 where there is none
    float unit;      // e4m3: the vector's scale
};

// DA: channels of the heads' own part; DV: of a value; kExpanded: values apart from keys.
template <int DA, int DV, bool kExpanded> struct Smem {
    static constexpr int DK = DA + 64;  // and the shared part, up to 64 channels
    static constexpr int P = DK + 4;    // an odd number of 16-byte pieces: no bank is met twice
    float q[BM][P];
    float k[KS][P];
    float v[kExpanded ? KS : 1][DV];
    float p[KS][BM + 4];
    float f[BM];
    KeyAt at[KS];
    Cursor piece[2];
    int has;
};

template <typename P, typename Kv, int DA, int DV>
__global__ void __launch_bounds__(kThreads) latent_generic_kernel(const __grid_constant__ P p) {
    constexpr bool kExpanded = std::is_same_v<P, PrefillRowsParams>;
    using S = Smem<DA, DV, kExpanded>;
    constexpr int CT = DV / 64, CV = CT >= 4 ? 4 : CT;  // channels of a thread, side by side
    extern __shared__ __align__(16) unsigned char smem_raw[];
    S &s = *reinterpret_cast<S *>(smem_raw);
    const int tid = int(threadIdx.x), ty = tid >> 4, tx = tid & 15, cta = int(blockIdx.x);
    const int r0 = (tid >> 6) * 8, cx = tid & 63;  // of the outputs: first row, place among channels
    wait_prior_kernel();
    allow_next_kernel();
    if (tid < 2) p.parts[2 * cta + tid].state = 0;
    if (tid < 32) {
        Cursor a, z;
        const bool has = find_piece(p, cta, int(gridDim.x), tid, a, z);
        if (tid == 0) s.piece[0] = a, s.piece[1] = z, s.has = has;
    }
    __syncthreads();
    if (!s.has) return;
    ItemWalk walk(s.piece[0], s.piece[1]);
    Item it;
    const int dk = DA + p.rope, kq = dk / 4;
    while (walk.next(p, it)) {
        __syncthreads();
        for (int i = tid; i < BM * kq; i += kThreads) {
            const int r = i / kq, c = (i - r * kq) * 4;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < it.rows) {
                long long row, head;
                p.locate(it, r, row, head);
                if constexpr (!kExpanded) head = min(int(head), p.heads - 1);
                x = c < DA ? load4(static_cast<const float *>(p.q_a) + row * p.qa_stride + head * p.qa_head + c)
                           : load4(static_cast<const float *>(p.q_r) + row * p.qr_stride + head * p.qr_head + (c - DA));
            }
            *reinterpret_cast<float4 *>(&s.q[r][c]) =
                make_float4(x.x * p.scale_log2, x.y * p.scale_log2, x.z * p.scale_log2, x.w * p.scale_log2);
        }
        float o[8][CT], m[2], l[2];
        int lim[2];  // last key a row sees
#pragma unroll
        for (int a = 0; a < 8; ++a)
#pragma unroll
            for (int c = 0; c < CT; ++c) o[a][c] = 0.f;
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            m[a] = -INFINITY, l[a] = 0.f;
            lim[a] = 2 * ty + a < it.rows ? it.ctx + it.tok0 + p.token_of(2 * ty + a) : -1;
        }
        for (int kb = it.k0; kb < it.k1; kb += KS) {
            __syncthreads();  // the previous step's keys and values are done with
            bool hidden = false;  // this thread's key is absent, or behind some row's position
            if (tid < KS) {
                const int j = kb + tid;
                KeyAt at = {-1, 1.f};
                if (j < it.k1) {
                    if constexpr (kExpanded) {
                        at.line = static_cast<long long>(p.b.cu_kv[it.n]) + j;
                    } else {
                        const int page = load_page(p.b, it.n, j);
                        if (page >= 0) {
                            at.line = (static_cast<long long>(page) << p.b.page_shift) + (j & ((1 << p.b.page_shift) - 1));
                            if (sizeof(Kv) == 1) at.unit = exp2_biased(p.sc[at.line]);
                        }
                    }
                }
                s.at[tid] = at;
                hidden = at.line < 0 || j > it.ctx + it.tok0;
            }
            const bool masked = __syncthreads_or(hidden);
#pragma unroll 4
            for (int i = tid; i < KS * kq; i += kThreads) {
                const int j = i / kq, c = (i - j * kq) * 4;
                const KeyAt at = s.at[j];
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                if (at.line >= 0) {
                    if constexpr (kExpanded) {
                        x = c < DA ? load4(static_cast<const float *>(p.k) + at.line * p.k_stride + it.h * p.k_head + c)
                                   : load4(static_cast<const float *>(p.kr) + at.line * p.kr_stride + (c - DA));
                    } else if (c < DA) {
                        x = load4(static_cast<const Kv *>(p.c) + at.line * DA + c);
                        x = make_float4(x.x * at.unit, x.y * at.unit, x.z * at.unit, x.w * at.unit);
                    } else {
                        x = load4(static_cast<const float *>(p.kr) + at.line * p.rope + (c - DA));
                    }
                }
                *reinterpret_cast<float4 *>(&s.k[j][c]) = x;
            }
            if constexpr (kExpanded) {
#pragma unroll 4
                for (int i = tid; i < KS * DV / 4; i += kThreads) {
                    const int j = i / (DV / 4), c = i % (DV / 4) * 4;
                    const long long line = s.at[j].line;
                    *reinterpret_cast<float4 *>(&s.v[j][c]) =
                        line >= 0 ? load4(static_cast<const float *>(p.v) + line * p.v_stride + it.h * p.v_head + c)
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
                }
            }
            __syncthreads();
            float2 x2[2][2] = {};
#pragma unroll 4
            for (int c = 0; c < dk; c += 4) {
                float4 kk[2], qq[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) kk[e] = *reinterpret_cast<const float4 *>(&s.k[tx + 16 * e][c]);
#pragma unroll
                for (int a = 0; a < 2; ++a) qq[a] = *reinterpret_cast<const float4 *>(&s.q[2 * ty + a][c]);
#pragma unroll
                for (int a = 0; a < 2; ++a)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        x2[a][e] = fma2(make_float2(qq[a].x, qq[a].y), make_float2(kk[e].x, kk[e].y), x2[a][e]);
                        x2[a][e] = fma2(make_float2(qq[a].z, qq[a].w), make_float2(kk[e].z, kk[e].w), x2[a][e]);
                    }
            }
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                float x[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    x[e] = x2[a][e].x + x2[a][e].y;
                    if (masked && (s.at[tx + 16 * e].line < 0 || kb + tx + 16 * e > lim[a])) x[e] = -INFINITY;
                }
                float mx = fmaxf(x[0], x[1]);
#pragma unroll
                for (int d = 8; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                const float mn = fmaxf(m[a], mx), ref = mn == -INFINITY ? 0.f : mn, f = exp2f(m[a] - ref);
                float sum = 0.f;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float w = exp2f(x[e] - ref);
                    sum += w;
                    s.p[tx + 16 * e][2 * ty + a] = masked && x[e] == -INFINITY ? kUnseen : w;
                }
#pragma unroll
                for (int d = 8; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                l[a] = l[a] * f + sum;
                m[a] = mn;
                if (tx == 0) s.f[2 * ty + a] = f;
            }
            __syncthreads();
            if (r0 >= it.rows) continue;
#pragma unroll
            for (int a = 0; a < 8; ++a) {
                const float f = s.f[r0 + a];
#pragma unroll
                for (int c = 0; c < CT; ++c) o[a][c] *= f;
            }
#pragma unroll 2
            for (int j = 0; j < KS; ++j) {
                const float4 t = *reinterpret_cast<const float4 *>(&s.p[j][r0]), u = *reinterpret_cast<const float4 *>(&s.p[j][r0 + 4]);
                const float w[8] = {t.x, t.y, t.z, t.w, u.x, u.y, u.z, u.w};
                const float *src = kExpanded ? s.v[j] : s.k[j];
                float vv[CT];
#pragma unroll
                for (int g = 0; g < CT / CV; ++g)
#pragma unroll
                    for (int e = 0; e < CV; ++e) vv[g * CV + e] = src[g * 64 * CV + cx * CV + e];
#pragma unroll
                for (int a = 0; a < 8; ++a) {
                    if (masked && w[a] == kUnseen) continue;
#pragma unroll
                    for (int c = 0; c < CT; ++c) o[a][c] = fmaf(w[a], vv[c], o[a][c]);
                }
            }
        }
        const bool whole = it.whole();
        float *data = p.part_data + (size_t(cta) * 2 + it.slot()) * size_t(BM) * (DV + 2);
        __syncthreads();
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            const int r = 2 * ty + a;
            if (tx == 0) s.f[r] = !whole ? 1.f : l[a] > 0.f || l[a] != l[a] ? 1.0f / l[a] : 0.f;
            if (!whole && tx == 0 && r < it.rows) data[BM * DV + r] = m[a], data[BM * DV + BM + r] = l[a];
        }
        if (!whole && tid == 0) p.parts[2 * cta + it.slot()] = it.part();
        __syncthreads();
#pragma unroll
        for (int a = 0; a < 8; ++a) {
            const int r = r0 + a;
            if (r >= it.rows) continue;
            long long row, head;
            p.locate(it, r, row, head);
            if constexpr (!kExpanded)
                if (head >= p.heads) continue;
            float *dst = static_cast<float *>(p.out) + row * p.out_stride + head * p.out_head;
            const float f = s.f[r];
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                const int ch = c / CV * 64 * CV + cx * CV + c % CV;
                if (whole) dst[ch] = o[a][c] * f;
                else data[size_t(r) * DV + ch] = o[a][c];
            }
        }
    }
}

// CTAs of an SM by the latent's channels (0: the expanded form): two where shared memory holds two, as eight warps
// leave the SM waiting at their barriers (five sequences of 800 tokens at most, 12 heads: 54 us with one, 47 with
// two; three prompts of 700 at most 219 and 163).
constexpr int ctas_of_sm(int latent) { return latent == 512 ? 1 : 2; }

template <typename P, typename Kv, int DA, int DV>
kda_status launch(P &p, const AttendPlan &plan, cudaStream_t stream) {
    auto kern = latent_generic_kernel<P, Kv, DA, DV>;
    // As much that the CTAs of an SM are kCtas: launched while the kernel before still holds some SMs, a grid that leaves
    // room would crowd the others (three prompts of 700 tokens at most: 456 us for what takes 233).
    constexpr bool kExpanded = std::is_same_v<P, PrefillRowsParams>;
    constexpr int kNeeds = int(sizeof(Smem<DA, DV, kExpanded>)), kCtas = ctas_of_sm(kExpanded ? 0 : DA);
    constexpr int smem = std::max(kNeeds, (kCtas == 1 ? 120 : 80) * 1024);
    static_assert(kCtas * (smem + 1024) <= 228 * 1024, "they fit");
    static_assert(smem <= 232448, "shared memory of a CTA");
    if (!allow_smem<latent_generic_kernel<P, Kv, DA, DV>>(smem)) return KDA_ERR_CUDA;
    p.key_step = KS;
    p.item_cost = KS;
    p.min_keys = 2 * KS;
    const ProfScope prof(std::is_same_v<P, LatentParams> ? KDA_KERNEL_LATENT_ATTEND : KDA_KERNEL_LATENT_PREFILL, stream);
    return launch_overlapped(kern, dim3(unsigned(plan.n_cta)), kThreads, size_t(smem), stream, p);
}

template <typename Kv>
kda_status by_latent(int L, LatentParams &p, const AttendPlan &plan, cudaStream_t s) {
    switch (L) {
        case 128: return launch<LatentParams, Kv, 128, 128>(p, plan, s);
        case 256: return launch<LatentParams, Kv, 256, 256>(p, plan, s);
        case 512: return launch<LatentParams, Kv, 512, 512>(p, plan, s);
    }
    return KDA_ERR_UNSUPPORTED;
}

kda_status by_heads(int dn, int dv, PrefillRowsParams &p, const AttendPlan &plan, cudaStream_t s) {
    if (dn == 64 && dv == 64) return launch<PrefillRowsParams, float, 64, 64>(p, plan, s);
    if (dn == 64 && dv == 128) return launch<PrefillRowsParams, float, 64, 128>(p, plan, s);
    if (dn == 128 && dv == 64) return launch<PrefillRowsParams, float, 128, 64>(p, plan, s);
    if (dn == 128 && dv == 128) return launch<PrefillRowsParams, float, 128, 128>(p, plan, s);
    return KDA_ERR_UNSUPPORTED;
}

}  // namespace

void latent_generic_plan(int latent, AttendPlan *plan) {
    plan->bm = BM;
    plan->n_cta = ctas_of_sm(latent) * sm_count();
}

kda_status latent_generic_launch(const kda_latent_cache *c, LatentParams &p, const AttendPlan &plan, cudaStream_t stream) {
    return c->format == KDA_KV_E4M3 ? by_latent<uint8_t>(c->latent_dim, p, plan, stream)
                                    : by_latent<float>(c->latent_dim, p, plan, stream);
}

kda_status prefill_generic_launch(const kda_latent_cache *, const kda_latent_prefill_io *io, PrefillRowsParams &p,
                                  const AttendPlan &plan, cudaStream_t stream) {
    return by_heads(io->nope_dim, io->value_dim, p, plan, stream);
}

}  // namespace kv
}  // namespace kda
