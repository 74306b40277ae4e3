// kda_attend_generic.cu -- kda_kv_attend for more than 16 rows a cache head in
// 32 bits, on the CUDA cores (the tensor cores have no 32-bit products).
//
// One pass over the keys with the running row maximum m and sum l of a
// softmax (in powers of two, x = scale * log2(e) * q . k):
//   m' = max(m, max_j x_j),  l <- l 2^(m - m') + sum_j 2^(x_j - m'),
//   o <- o 2^(m - m') + sum_j 2^(x_j - m') v_j,   out = o / l.
// A CTA holds a tile of BM rows (query heads of one cache head, consecutive
// tokens) and walks 64 keys a step through shared memory; 16 threads side by
// side share 8 rows, each with 4 of the keys of the scores and D / 16 channels
// of the output in registers.  Multiply-adds go two to an instruction (scores sum
// even and odd channels apart).  They bound it, with the shared memory reads that
// feed them close behind: at 4 rows a thread the reads came first (ragged prompts
// of 777 to 1500 tokens, 12 heads of 64: 305 us against 258 at 8; 237 now, 33 TFLOP/s).
// 64 rows on 128 threads leave room for three CTAs an SM, whose loads and sums
// cover each other; head size 128 takes 128 rows on 256 threads, one CTA an SM.
#include <type_traits>

#include "kda_attend.cuh"

namespace kda {
namespace kv {
namespace {

constexpr int KS = 64;  // keys a step
constexpr int threads_of(int bm) { return bm * 2; }  // 16 threads for 8 rows

// Four channels of a key or value; e4m3 times their scale.
__device__ __forceinline__ float4 widen4(const uint4 &r, float) {
    return make_float4(__uint_as_float(r.x), __uint_as_float(r.y), __uint_as_float(r.z), __uint_as_float(r.w));
}
__device__ __forceinline__ float4 widen4(uint32_t r, float f) {
    const float2 a = unpack_e4m3(uint16_t(r)), b = unpack_e4m3(uint16_t(r >> 16));
    return make_float4(a.x * f, a.y * f, b.x * f, b.y * f);
}

// Rows are padded to an odd number of 16-byte pieces, so that the 8 lanes of a
// read that take one piece of 8 rows meet no bank twice.
template <int BM, int D> struct Smem {
    float q[BM][D + 4];
    float k[KS][D + 4];
    float v[KS][D];
    float p[KS][BM + 4];
    int64_t line[KS];  // vector index of each key's line, -1 where there is none
    Cursor piece[2];
    int has;
};

template <typename Kv, int BM, int D>
__global__ void __launch_bounds__(threads_of(BM), BM == 64 ? 3 : 1) attend_generic_kernel(const __grid_constant__ AttendParams p) {
    constexpr int kThreads = threads_of(BM), RT = 8, CT = D / 16, CV = CT >= 4 ? 4 : CT;  // rows and channels of a thread
    extern __shared__ __align__(16) unsigned char smem_raw[];
    Smem<BM, D> &s = *reinterpret_cast<Smem<BM, D> *>(smem_raw);
    const int tid = int(threadIdx.x), ty = tid >> 4, tx = tid & 15;
    const int cta = int(blockIdx.x);
    wait_prior_kernel();
    allow_next_kernel();
    Part *my_parts = p.parts + 2 * cta;
    if (tid < 2) my_parts[tid].state = 0;
    if (tid < 32) {
        Cursor a, z;
        const bool has = find_piece(p, cta, int(gridDim.x), tid, a, z);
        if (tid == 0) s.piece[0] = a, s.piece[1] = z, s.has = has;
    }
    __syncthreads();
    if (!s.has) return;
    ItemWalk walk(s.piece[0], s.piece[1]);
    Item it;
    const int page_mask = (1 << p.b.page_shift) - 1;

    while (walk.next(p, it)) {
        __syncthreads();
#pragma unroll 8
        for (int i = tid; i < BM * D / 4; i += kThreads) {
            const int r = i / (D / 4), c = i % (D / 4) * 4;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < it.rows)
                x = *reinterpret_cast<const float4 *>(static_cast<const float *>(p.q) + it.at(r, p, p.q_stride, D) + c);
            *reinterpret_cast<float4 *>(&s.q[r][c]) =
                make_float4(x.x * p.scale_log2, x.y * p.scale_log2, x.z * p.scale_log2, x.w * p.scale_log2);
        }
        float o[RT][CT], m[RT], l[RT];
#pragma unroll
        for (int a = 0; a < RT; ++a) {
            m[a] = -INFINITY, l[a] = 0.f;
#pragma unroll
            for (int c = 0; c < CT; ++c) o[a][c] = 0.f;
        }
        int lim[RT];  // last key a row sees
#pragma unroll
        for (int a = 0; a < RT; ++a) {
            const int r = ty * RT + a;
            lim[a] = r < it.rows ? it.ctx + it.tok0 + p.token_of(r) : -1;
        }
        for (int kb = it.k0; kb < it.k1; kb += KS) {
            __syncthreads();  // the previous step's keys and values are done with
            bool hidden = false;  // this thread's key is absent, or behind some row's position
            if (tid < KS) {
                const int j = kb + tid;
                int64_t line = -1;
                if (j < it.k1) {
                    const int page = load_page(p.b, it.n, j);
                    if (page >= 0)
                        line = ((int64_t(page) * p.hkv + it.h) << p.b.page_shift) + (j & page_mask);
                }
                s.line[tid] = line;
                hidden = line < 0 || j > it.ctx + it.tok0;
            }
            const bool masked = __syncthreads_or(hidden);
            // all of a thread's pieces are asked for before the first is put down
            using Raw = std::conditional_t<sizeof(Kv) == 1, uint32_t, uint4>;
            constexpr int kPieces = KS * D / 4 / kThreads;
            Raw rk[kPieces], rv[kPieces];
            float fk[kPieces], fv[kPieces];
#pragma unroll
            for (int u = 0; u < kPieces; ++u) {
                const int i = tid + u * kThreads, j = i / (D / 4), c = i % (D / 4) * 4;
                const int64_t line = s.line[j];
                rk[u] = rv[u] = Raw{};
                fk[u] = fv[u] = 1.f;
                if (line >= 0) {
                    rk[u] = *reinterpret_cast<const Raw *>(static_cast<const Kv *>(p.pk) + line * D + c);
                    rv[u] = *reinterpret_cast<const Raw *>(static_cast<const Kv *>(p.pv) + line * D + c);
                    if constexpr (sizeof(Kv) == 1) fk[u] = exp2_biased(p.sk[line]), fv[u] = exp2_biased(p.sv[line]);
                }
            }
#pragma unroll
            for (int u = 0; u < kPieces; ++u) {
                const int i = tid + u * kThreads, j = i / (D / 4), c = i % (D / 4) * 4;
                *reinterpret_cast<float4 *>(&s.k[j][c]) = widen4(rk[u], fk[u]);
                *reinterpret_cast<float4 *>(&s.v[j][c]) = widen4(rv[u], fv[u]);
            }
            __syncthreads();
            // keys of a thread: tx, tx + 16, tx + 32, tx + 48
            float2 x2[RT][4];
#pragma unroll
            for (int a = 0; a < RT; ++a)
#pragma unroll
                for (int e = 0; e < 4; ++e) x2[a][e] = make_float2(0.f, 0.f);
#pragma unroll 1
            for (int c = 0; c < D; c += 4) {
                float4 kk[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) kk[e] = *reinterpret_cast<const float4 *>(&s.k[tx + 16 * e][c]);
#pragma unroll
                for (int a = 0; a < RT; ++a) {
                    const float4 qq = *reinterpret_cast<const float4 *>(&s.q[ty * RT + a][c]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        x2[a][e] = fma2(make_float2(qq.x, qq.y), make_float2(kk[e].x, kk[e].y), x2[a][e]);
                        x2[a][e] = fma2(make_float2(qq.z, qq.w), make_float2(kk[e].z, kk[e].w), x2[a][e]);
                    }
                }
            }
            float x[RT][4];
#pragma unroll
            for (int a = 0; a < RT; ++a)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[a][e] = x2[a][e].x + x2[a][e].y;
            if (masked) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const bool there = s.line[tx + 16 * e] >= 0;
#pragma unroll
                    for (int a = 0; a < RT; ++a)
                        if (!there || kb + tx + 16 * e > lim[a]) x[a][e] = -INFINITY;
                }
            }
#pragma unroll
            for (int a = 0; a < RT; ++a) {
                float mx = fmaxf(fmaxf(x[a][0], x[a][1]), fmaxf(x[a][2], x[a][3]));
#pragma unroll
                for (int d = 8; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                const float mn = fmaxf(m[a], mx), ref = mn == -INFINITY ? 0.f : mn;
                const float f = exp2f(m[a] - ref);
                float sum = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[a][e] = exp2f(x[a][e] - ref);
                    sum += x[a][e];
                }
#pragma unroll
                for (int d = 8; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                l[a] = l[a] * f + sum;
                m[a] = mn;
#pragma unroll
                for (int c = 0; c < CT; ++c) o[a][c] *= f;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float *dst = &s.p[tx + 16 * e][ty * RT];
                reinterpret_cast<float4 *>(dst)[0] = make_float4(x[0][e], x[1][e], x[2][e], x[3][e]);
                reinterpret_cast<float4 *>(dst)[1] = make_float4(x[4][e], x[5][e], x[6][e], x[7][e]);
            }
            __syncwarp();  // a row's weights are written and read by the same half warp
            // channels of a thread: groups of four (or the D / 16 there are) 16 groups apart
#pragma unroll 1
            for (int j = 0; j < KS; ++j) {
                const float4 t = *reinterpret_cast<const float4 *>(&s.p[j][ty * 8]);
                const float4 u = *reinterpret_cast<const float4 *>(&s.p[j][ty * 8 + 4]);
                const float w[RT] = {t.x, t.y, t.z, t.w, u.x, u.y, u.z, u.w};
                float vv[CT];
#pragma unroll
                for (int g = 0; g < CT / CV; ++g)
#pragma unroll
                    for (int e = 0; e < CV; ++e) vv[g * CV + e] = s.v[j][g * 16 * CV + tx * CV + e];
                if (!masked) {
#pragma unroll
                    for (int a = 0; a < RT; ++a) {
                        if constexpr (CT >= 2) {
#pragma unroll
                            for (int c = 0; c < CT; c += 2) {
                                const float2 t = fma2(make_float2(w[a], w[a]), make_float2(vv[c], vv[c + 1]),
                                                      make_float2(o[a][c], o[a][c + 1]));
                                o[a][c] = t.x, o[a][c + 1] = t.y;
                            }
                        } else {
                            o[a][0] = fmaf(w[a], vv[0], o[a][0]);
                        }
                    }
                } else {  // a value of a key that the row does not see may be anything
#pragma unroll
                    for (int a = 0; a < RT; ++a)
#pragma unroll
                        for (int c = 0; c < CT; ++c) o[a][c] = w[a] != 0.f ? fmaf(w[a], vv[c], o[a][c]) : o[a][c];
                }
            }
        }
        const bool whole = it.whole();
        float *data = p.part_data + (size_t(cta) * 2 + it.slot()) * size_t(BM) * (D + 2);
        if (!whole && tid == 0) my_parts[it.slot()] = it.part();
#pragma unroll
        for (int a = 0; a < RT; ++a) {
            const int r = ty * RT + a;
            if (r >= it.rows) continue;
            const float inv = l[a] > 0.f || l[a] != l[a] ? 1.0f / l[a] : 0.f;
            float *dst = static_cast<float *>(p.out) + it.at(r, p, p.out_stride, D);
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                const int ch = c / CV * 16 * CV + tx * CV + c % CV;
                if (whole) dst[ch] = o[a][c] * inv;
                else data[size_t(r) * D + ch] = o[a][c];
            }
            if (!whole && tx == 0) data[BM * D + r] = m[a], data[BM * D + BM + r] = l[a];
        }
    }
}

template <typename Kv, int BM, int D>
kda_status launch(AttendParams &p, const AttendPlan &plan, cudaStream_t stream) {
    auto kern = attend_generic_kernel<Kv, BM, D>;
    const int smem = int(sizeof(Smem<BM, D>));
    if (!allow_smem<attend_generic_kernel<Kv, BM, D>>(smem)) return KDA_ERR_CUDA;
    p.key_step = KS;
    // Measured at 0, 64, 128, 256, 1024: 16 sequences of 30 to 60 new tokens behind 100 to 1500, heads of 128,
    // take 512, 460, 478, 495, 630 us (before all of a step's loads went out together; 369 since).
    p.item_cost = KS;
    p.min_keys = 2 * KS;
    const ProfScope prof(KDA_KERNEL_KV_ATTEND, stream);
    return launch_overlapped(kern, dim3(unsigned(plan.n_cta)), threads_of(BM), size_t(smem), stream, p);
}

template <typename Kv> kda_status by_size(int D, AttendParams &p, const AttendPlan &plan, cudaStream_t s) {
    switch (D) {
        case 16: return launch<Kv, 64, 16>(p, plan, s);
        case 32: return launch<Kv, 64, 32>(p, plan, s);
        case 64: return launch<Kv, 64, 64>(p, plan, s);
        case 128: return launch<Kv, 128, 128>(p, plan, s);
    }
    return KDA_ERR_UNSUPPORTED;
}

}  // namespace

bool generic_plan(const kda_kv_cache *c, const kda_kv_batch *b, AttendPlan *plan) {
    plan->bm = c->head_dim == 128 ? 128 : 64;
    plan->n_cta = (plan->bm == 128 ? 1 : 3) * sm_count();
    return true;
}

kda_status generic_launch(const kda_kv_cache *c, AttendParams &p, const AttendPlan &plan, cudaStream_t stream) {
    return c->format == KDA_KV_E4M3 ? by_size<uint8_t>(c->head_dim, p, plan, stream)
                                    : by_size<float>(c->head_dim, p, plan, stream);
}

}  // namespace kv
}  // namespace kda
