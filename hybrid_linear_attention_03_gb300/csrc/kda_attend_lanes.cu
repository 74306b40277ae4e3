// kda_attend_lanes.cu -- kda_kv_attend for few rows a cache head where the
// tensor-core kernels do not pay: 32-bit rows (up to 16), and bf16 rows (up to 4)
// of head sizes 16 and 32.
//
// The softmax of kda_attend_generic.cu in one pass, without shared memory: a key
// and its value are held by the lanes that load them 16 bytes at a time (8 for
// e4m3), a lane keeps the rows' queries and outputs for its channels in 32-bit
// registers, and a score is the sum of its lanes' products, formed by shuffles.
// Every group of lanes has running maxima, sums and outputs of its own over the
// keys that it met; they are joined at the item's end.  A warp takes 32 keys at
// a time: each lane looks up one key's page (and, e4m3, its scales), a chunk
// ahead, and the groups then fetch kAhead keys and values each before they use
// them.  So the memory bounds it while rows are few; a row costs a lane group
// about 20 instructions a key, which takes over from 4 rows on.  Every 4 rows have
// warps of their own (registers), which read the same keys again, from L1.
// Measured on 32 sequences of 3001 to 8192 tokens, 4 cache heads: 32-bit pages of
// 128 channels 126 us for one or two rows (5.7 TB/s), 274 us for 8, 539 us for 16
// (the tiles of kda_attend_generic.cu, which have room for more rows, 540 us for
// any of these); bf16 pages of 32 channels 33 us for 2 rows, 50 for 4, 81 for 8,
// where kda_attend_tile.cu takes 42 us for any number (borders: lanes_plan).
#include "kda_attend.cuh"

namespace kda {
namespace kv {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kChunk = 32;  // keys a warp takes at a time

// A lane's channels of a key or value.
template <typename Kv, int N> struct Piece;
template <> struct Piece<float, 4> {
    using Raw = uint4;
    static __device__ __forceinline__ void unpack(const uint4 &r, float2 (&x)[2]) {
        x[0] = make_float2(__uint_as_float(r.x), __uint_as_float(r.y));
        x[1] = make_float2(__uint_as_float(r.z), __uint_as_float(r.w));
    }
};
template <> struct Piece<__nv_bfloat16, 8> {
    using Raw = uint4;
    static __device__ __forceinline__ void unpack(const uint4 &r, float2 (&x)[4]) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
};
template <> struct Piece<uint8_t, 8> {
    using Raw = uint2;
    static __device__ __forceinline__ void unpack(const uint2 &r, float2 (&x)[4]) {
        x[0] = unpack_e4m3(uint16_t(r.x)), x[1] = unpack_e4m3(uint16_t(r.x >> 16));
        x[2] = unpack_e4m3(uint16_t(r.y)), x[3] = unpack_e4m3(uint16_t(r.y >> 16));
    }
};

__device__ __forceinline__ void load_channels(const float *src, float2 (&x)[2]) {
    Piece<float, 4>::unpack(*reinterpret_cast<const uint4 *>(src), x);
}
__device__ __forceinline__ void load_channels(const __nv_bfloat16 *src, float2 (&x)[4]) {
    Piece<__nv_bfloat16, 8>::unpack(*reinterpret_cast<const uint4 *>(src), x);
}
__device__ __forceinline__ void load_channels(const float *src, float2 (&x)[4]) {
    float2 a[2], b[2];
    load_channels(src, a), load_channels(src + 4, b);
    x[0] = a[0], x[1] = a[1], x[2] = b[0], x[3] = b[1];
}

// R: rows of an item (2, 4, 8 or 16)
template <typename Act, typename Kv, int D, int R>
__global__ void __launch_bounds__(kThreads, 2) attend_lanes_kernel(const __grid_constant__ AttendParams p) {
    constexpr int N = sizeof(Kv) == 4 ? 4 : 8, LPH = D / N, KPW = 32 / LPH;  // channels a lane, lanes a key, keys at once
    constexpr int RW = R < 4 ? R : 4, kSets = R / RW, kSetWarps = kWarps / kSets;
    constexpr int kAhead = LPH < 4 ? LPH : 4;  // keys a lane group has in flight
    constexpr bool kE4m3 = sizeof(Kv) == 1;
    using P = Piece<Kv, N>;
    __shared__ float join[kWarps][RW][D + 2];
    __shared__ Cursor piece[2];
    __shared__ int has_piece;
    const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5, cta = int(blockIdx.x);
    const int set = warp % kSets, sw = warp / kSets;  // the warp's rows, and its place among the warps of these rows
    const int group = lane / LPH, c0 = lane % LPH * N;
    wait_prior_kernel();
    allow_next_kernel();
    Part *my_parts = p.parts + 2 * cta;
    if (tid < 2) my_parts[tid].state = 0;
    if (warp == 0) {
        Cursor a, z;
        const bool has = find_piece(p, cta, int(gridDim.x), lane, a, z);
        if (lane == 0) piece[0] = a, piece[1] = z, has_piece = has;
    }
    __syncthreads();
    if (!has_piece) return;
    ItemWalk walk(piece[0], piece[1]);
    Item it;
    const int page_mask = (1 << p.b.page_shift) - 1;

    while (walk.next(p, it)) {
        float2 q[RW][N / 2], o[RW][N / 2];
        float m[RW], l[RW];
        int lim[RW];  // last key a row sees
#pragma unroll
        for (int a = 0; a < RW; ++a) {
            const int r = set * RW + a;
            m[a] = -INFINITY, l[a] = 0.f;
            lim[a] = r < it.rows ? it.ctx + it.tok0 + p.token_of(r) : -1;
#pragma unroll
            for (int i = 0; i < N / 2; ++i) q[a][i] = o[a][i] = make_float2(0.f, 0.f);
            if (r < it.rows) load_channels(static_cast<const Act *>(p.q) + it.at(r, p, p.q_stride, D) + c0, q[a]);
#pragma unroll
            for (int i = 0; i < N / 2; ++i) q[a][i].x *= p.scale_log2, q[a][i].y *= p.scale_log2;
        }
        // the line of key j, or -1
        auto find_line = [&](int j) {
            int64_t line = -1;
            if (j < it.k1) {
                const int page = load_page(p.b, it.n, j);
                if (page >= 0) line = ((int64_t(page) * p.hkv + it.h) << p.b.page_shift) + (j & page_mask);
            }
            return line;
        };
        int64_t next_line = find_line(it.k0 + sw * kChunk + lane);
        for (int kb = it.k0 + sw * kChunk; kb < it.k1; kb += kSetWarps * kChunk) {
            const int64_t line = next_line;
            next_line = find_line(kb + kSetWarps * kChunk + lane);
            float fk = 1.f, fv = 1.f;
            if (kE4m3 && line >= 0) fk = exp2_biased(p.sk[line]), fv = exp2_biased(p.sv[line]);
            // some row does not see some key of the chunk
            const bool masked = __any_sync(0xffffffffu, line < 0 || kb + lane > it.ctx + it.tok0);
#pragma unroll 1
            for (int s0 = 0; s0 < LPH; s0 += kAhead) {
                typename P::Raw kr[kAhead], vr[kAhead];
                bool there[kAhead];
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const int64_t at = __shfl_sync(0xffffffffu, line, (s0 + u) * KPW + group);
                    there[u] = at >= 0;
                    kr[u] = vr[u] = typename P::Raw{};
                    if (there[u]) {
                        kr[u] = *reinterpret_cast<const typename P::Raw *>(static_cast<const Kv *>(p.pk) + at * D + c0);
                        vr[u] = *reinterpret_cast<const typename P::Raw *>(static_cast<const Kv *>(p.pv) + at * D + c0);
                    }
                }
                float x[kAhead][RW];
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    float2 k[N / 2];
                    P::unpack(kr[u], k);
                    const float unit = kE4m3 ? __shfl_sync(0xffffffffu, fk, (s0 + u) * KPW + group) : 1.f;
#pragma unroll
                    for (int a = 0; a < RW; ++a) {
                        float2 s = make_float2(0.f, 0.f);
#pragma unroll
                        for (int i = 0; i < N / 2; ++i) s = fma2(q[a][i], k[i], s);
                        x[u][a] = s.x + s.y;
                    }
#pragma unroll
                    for (int a = 0; a < RW; ++a) {
#pragma unroll
                        for (int d = LPH / 2; d > 0; d >>= 1) x[u][a] += __shfl_xor_sync(0xffffffffu, x[u][a], d);
                        if constexpr (kE4m3) x[u][a] *= unit;
                        if (masked && (!there[u] || kb + (s0 + u) * KPW + group > lim[a])) x[u][a] = -INFINITY;
                    }
                }
#pragma unroll
                for (int a = 0; a < RW; ++a) {
                    float top = m[a];
#pragma unroll
                    for (int u = 0; u < kAhead; ++u) top = fmaxf(top, x[u][a]);
                    const float ref = top == -INFINITY ? 0.f : top, back = exp2f(m[a] - ref);
                    m[a] = top;
                    l[a] *= back;
#pragma unroll
                    for (int i = 0; i < N / 2; ++i) o[a][i].x *= back, o[a][i].y *= back;
#pragma unroll
                    for (int u = 0; u < kAhead; ++u) {
                        x[u][a] = exp2f(x[u][a] - ref);
                        l[a] += x[u][a];
                    }
                }
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    float2 v[N / 2];
                    P::unpack(vr[u], v);
                    if constexpr (kE4m3) {
                        const float unit = __shfl_sync(0xffffffffu, fv, (s0 + u) * KPW + group);
#pragma unroll
                        for (int i = 0; i < N / 2; ++i) v[i].x *= unit, v[i].y *= unit;
                    }
#pragma unroll
                    for (int a = 0; a < RW; ++a) {
                        // a value of a key that the row does not see may be anything
                        if (masked && x[u][a] == 0.f) continue;
#pragma unroll
                        for (int i = 0; i < N / 2; ++i) o[a][i] = fma2(make_float2(x[u][a], x[u][a]), v[i], o[a][i]);
                    }
                }
            }
        }
        // the warp's lane groups joined, then the warps of the same rows
#pragma unroll
        for (int a = 0; a < RW; ++a) {
            float top = m[a];
#pragma unroll
            for (int d = 16; d >= LPH; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            const float f = exp2f(m[a] - (top == -INFINITY ? 0.f : top));
            l[a] *= f;
#pragma unroll
            for (int i = 0; i < N / 2; ++i) o[a][i].x *= f, o[a][i].y *= f;
#pragma unroll
            for (int d = 16; d >= LPH; d >>= 1) {
                l[a] += __shfl_xor_sync(0xffffffffu, l[a], d);
#pragma unroll
                for (int i = 0; i < N / 2; ++i) {
                    o[a][i].x += __shfl_xor_sync(0xffffffffu, o[a][i].x, d);
                    o[a][i].y += __shfl_xor_sync(0xffffffffu, o[a][i].y, d);
                }
            }
            if (group == 0) {
#pragma unroll
                for (int i = 0; i < N / 2; ++i)
                    *reinterpret_cast<float2 *>(&join[warp][a][c0 + 2 * i]) = o[a][i];
                if (lane == 0) join[warp][a][D] = top, join[warp][a][D + 1] = l[a];
            }
        }
        __syncthreads();
        const bool whole = it.whole();
        float *data = p.part_data + (size_t(cta) * 2 + it.slot()) * size_t(R) * (D + 2);
        if (!whole && tid == 0) my_parts[it.slot()] = it.part();
        for (int i = tid; i < it.rows * D; i += kThreads) {
            const int r = i / D, ch = i % D, of = r / RW, a = r % RW;
            float top = -INFINITY, sum = 0.f, out = 0.f;
#pragma unroll
            for (int w = 0; w < kSetWarps; ++w) top = fmaxf(top, join[w * kSets + of][a][D]);
            const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
            for (int w = 0; w < kSetWarps; ++w) {
                const float f = exp2f(join[w * kSets + of][a][D] - ref);
                sum = fmaf(f, join[w * kSets + of][a][D + 1], sum);
                out = fmaf(f, join[w * kSets + of][a][ch], out);
            }
            if (whole) {
                const float inv = sum > 0.f || sum != sum ? 1.0f / sum : 0.f;
                static_cast<Act *>(p.out)[it.at(r, p, p.out_stride, D) + ch] = from_f32<Act>(out * inv);
            } else {
                data[i] = out;
                if (ch == 0) data[R * D + r] = top, data[R * D + R + r] = sum;
            }
        }
        __syncthreads();
    }
}

template <typename Act, typename Kv, int D, int R> kda_status launch(AttendParams &p, const AttendPlan &plan, cudaStream_t stream) {
    p.key_step = kChunk;
    // Keys that take as long as an item's start and output.  Measured at 0, 128, 256, 1024: 128 sequences of
    // 100 to 1500 tokens and 32-bit heads of 64 take 101, 90, 84, 96 us.
    p.item_cost = 8 * kChunk;
    p.min_keys = kWarps * kChunk;
    const ProfScope prof(KDA_KERNEL_KV_ATTEND, stream);
    return launch_overlapped(attend_lanes_kernel<Act, Kv, D, R>, dim3(unsigned(plan.n_cta)), kThreads, 0, stream, p);
}

template <typename Act, typename Kv, int D> kda_status by_rows(AttendParams &p, const AttendPlan &plan, cudaStream_t s) {
    if (plan.bm == 2) return launch<Act, Kv, D, 2>(p, plan, s);
    if (plan.bm == 4) return launch<Act, Kv, D, 4>(p, plan, s);
    if constexpr (sizeof(Act) == 4) {
        if (plan.bm == 8) return launch<Act, Kv, D, 8>(p, plan, s);
        if (plan.bm == 16) return launch<Act, Kv, D, 16>(p, plan, s);
    }
    return KDA_ERR_UNSUPPORTED;
}

template <typename Act, typename Kv> kda_status by_size(int D, AttendParams &p, const AttendPlan &plan, cudaStream_t s) {
    if (D == 16) return by_rows<Act, Kv, 16>(p, plan, s);
    if (D == 32) return by_rows<Act, Kv, 32>(p, plan, s);
    if constexpr (sizeof(Act) == 4) {
        if (D == 64) return by_rows<Act, Kv, 64>(p, plan, s);
        if (D == 128) return by_rows<Act, Kv, 128>(p, plan, s);
    }
    return KDA_ERR_UNSUPPORTED;
}

}  // namespace

// The borders.  32 bits: where the kernel for more rows catches up (figures above).  bf16: us here and with
// kda_attend_tile.cu, for 32 sequences of 3001 to 8192 tokens, and for 128 of 100 to 1500:
//   channels  rows  bf16 pages             e4m3 pages
//   16        2     23 / 40   20 / 42      23 / 59   20 / 62
//   16        4     32 / 40   27 / 42      29 / 59   27 / 62
//   32        2     33 / 42   25 / 45      30 / 60   22 / 64
//   32        4     50 / 42   38 / 45      38 / 60   30 / 64
//   64        2     48 / 44   36 / 47      55 / 62   39 / 66
//   64        4     67 / 44   53 / 48      73 / 62   54 / 66
// (3 rows as 4; one sequence of 3001 tokens: 14 to 17 us on either side up to 32 channels).  Up to 4 rows of at most
// 32 channels is ahead in all but one of these, 32 channels of bf16 with 3 or 4 rows over long caches.
bool lanes_plan(const kda_kv_cache *c, const kda_kv_batch *b, AttendPlan *plan) {
    const long long rows = static_cast<long long>(b->max_new) * (c->num_heads / c->num_kv_heads);
    if (c->act == KDA_BF16 ? rows > 4 || c->head_dim > 32 : rows > 16) return false;
    plan->bm = rows <= 2 ? 2 : rows <= 4 ? 4 : rows <= 8 ? 8 : 16;
    plan->n_cta = 2 * sm_count();
    return true;
}

kda_status lanes_launch(const kda_kv_cache *c, AttendParams &p, const AttendPlan &plan, cudaStream_t stream) {
    const int D = c->head_dim;
    const bool e4 = c->format == KDA_KV_E4M3;
    if (c->act == KDA_BF16)
        return e4 ? by_size<__nv_bfloat16, uint8_t>(D, p, plan, stream)
                  : by_size<__nv_bfloat16, __nv_bfloat16>(D, p, plan, stream);
    return e4 ? by_size<float, uint8_t>(D, p, plan, stream) : by_size<float, float>(D, p, plan, stream);
}

}  // namespace kv
}  // namespace kda
