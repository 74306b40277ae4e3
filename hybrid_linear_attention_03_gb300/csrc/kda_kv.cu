// kda_kv.cu -- the paged cache's writers and readers: kda_kv_append (per-head
// RMSNorm, position rotation and the quantised page write in one pass) and
// kda_kv_read.  Formulas, layout and contracts: include/kda.h.
//
// Both only move data: append reads (Hq + 2 Hkv) d values a token and writes
// as many (half for e4m3 pages), about 10 operations each, so HBM bounds
// them.  A vector of head_dim channels is owned by the head_dim * size / 16
// lanes that hold it in 16-byte loads; its sum of squares, its largest
// magnitude and its rotation partners move by shuffles, and nothing but the
// rotation's cosines (once per row) passes through shared memory.
#include "kda_kv.cuh"

#include <cmath>

namespace kda {
namespace kv {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsPerCta = 4;  // many rows: the rows of a CTA, which share one set of cosines
constexpr int kUnroll = 4;      // 16-byte loads in flight per thread
// Cosine / sine pairs of one row: 32 chunks of two pairs, chunk c at
// (c & 3) * 18 + (c >> 2), which the 16-byte reads of 8 neighbouring lanes
// meet without a bank conflict in both pair orders.
constexpr int kCsChunks = 4 * 18;
__device__ __forceinline__ int cs_at(int c) { return (c & 3) * 18 + (c >> 2); }

struct AppendParams {
    BatchView b;
    const void *q, *k, *v;
    void *q_out, *pk, *pv;
    uint8_t *sk, *sv;
    const void *wq, *wk;
    long long q_stride, k_stride, v_stride, qo_stride;
    int32_t hq, hkv;          // hq = 0 when the call has no queries
    int32_t rows_per_cta, heads_per_cta;
    int32_t half_rot, interleaved;
    float eps;
    uint64_t turn[64];  // inv_freq / (2 pi) mod 1, in units of 2^-64 turns
};

template <typename Act> struct Vec;  // 16 bytes of activations
template <> struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void unpack(const uint4 &r, float (&x)[4]) {
        x[0] = __uint_as_float(r.x), x[1] = __uint_as_float(r.y);
        x[2] = __uint_as_float(r.z), x[3] = __uint_as_float(r.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[4]) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
};
template <> struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void unpack(const uint4 &r, float (&x)[8]) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

template <int N> __device__ __forceinline__ void store_e4m3(void *dst, const float (&y)[N]) {
    uint32_t w[N / 4];
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
        w[i] = uint32_t(pack_e4m3(y[4 * i], y[4 * i + 1])) | uint32_t(pack_e4m3(y[4 * i + 2], y[4 * i + 3])) << 16;
    if constexpr (N == 8)
        *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
    else
        *reinterpret_cast<uint32_t *>(dst) = w[0];
}

// One CTA: rows_per_cta rows x heads_per_cta of the hq + 2 hkv heads.
template <typename Act, int D, bool kE4m3>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const __grid_constant__ AppendParams p) {
    using V = Vec<Act>;
    constexpr int N = V::N, LPH = D / N;  // values per lane, lanes per head
    __shared__ float4 cs[kRowsPerCta][kCsChunks];
    __shared__ int s_pos[kRowsPerCta], s_page[kRowsPerCta];
    const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5;
    const int row_base = int(blockIdx.x) * p.rows_per_cta;
    wait_prior_kernel();
    allow_next_kernel();

    if (warp < p.rows_per_cta) {
        const int r = row_base + warp;
        int pos = -1, page = -1;
        const int n = r < p.b.max_rows ? find_seq(p.b, r, lane) : -1;
        if (lane == 0 && n >= 0 && n < p.b.n_seqs) {
            Seq s;
            if (load_seq(p.b, n, s, true)) {
                pos = s.L - s.T + (r - s.row0);
                page = load_page(p.b, n, pos);
            }
        }
        if (lane == 0) s_pos[warp] = pos, s_page[warp] = page;
    }
    __syncthreads();
    if (p.half_rot) {
        // angle p * f in turns is a 64-bit product mod 2^64: exact for any position
        for (int i = tid; i < p.rows_per_cta * p.half_rot; i += kThreads) {
            const int row = i / p.half_rot, pair = i % p.half_rot;
            const uint64_t ph = uint64_t(uint32_t(max(s_pos[row], 0))) * p.turn[pair];
            float sn, cn;
            sincospif(float(int64_t(ph)) * 0x1p-63f, &sn, &cn);
            reinterpret_cast<float2 *>(&cs[row][cs_at(pair >> 1)])[pair & 1] = make_float2(cn, sn);
        }
        __syncthreads();
    }

    const int heads = p.hq + 2 * p.hkv;
    const int h0 = int(blockIdx.y) * p.heads_per_cta, nh = min(p.heads_per_cta, heads - h0);
    const int l = tid % LPH, c0 = l * N;
    const int items = p.rows_per_cta * nh;
    const int mine = tid / LPH;
    uint4 wq = make_uint4(0, 0, 0, 0), wk = wq;
    const bool norm_q = p.wq != nullptr, norm_k = p.wk != nullptr;
    if (norm_q) wq = __ldg(reinterpret_cast<const uint4 *>(p.wq) + l);
    if (norm_k) wk = __ldg(reinterpret_cast<const uint4 *>(p.wk) + l);

    for (int base = 0; base < items; base += kUnroll * (kThreads / LPH)) {
        uint4 raw[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int it = base + u * (kThreads / LPH) + mine;
            raw[u] = make_uint4(0, 0, 0, 0);
            if (it >= items) continue;
            const int row = it / nh, h = h0 + it % nh;
            if (s_pos[row] < 0) continue;
            const size_t r = size_t(row_base + row);
            const Act *src;
            if (h < p.hq) src = static_cast<const Act *>(p.q) + r * size_t(p.q_stride) + size_t(h) * D;
            else if (h < p.hq + p.hkv) src = static_cast<const Act *>(p.k) + r * size_t(p.k_stride) + size_t(h - p.hq) * D;
            else src = static_cast<const Act *>(p.v) + r * size_t(p.v_stride) + size_t(h - p.hq - p.hkv) * D;
            raw[u] = *reinterpret_cast<const uint4 *>(src + c0);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            // every lane of the warp takes part in the shuffles; the branches below are uniform
            const int it = base + u * (kThreads / LPH) + mine;
            const bool live = it < items;
            const int row = live ? it / nh : 0, h = live ? h0 + it % nh : 0;
            const bool is_q = h < p.hq, is_v = h >= p.hq + p.hkv;
            float x[N];
            V::unpack(raw[u], x);
            if (norm_q || norm_k) {
                float ss = 0.f;
#pragma unroll
                for (int e = 0; e < N; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
                for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                if (!is_v && (is_q ? norm_q : norm_k)) {
                    const float rs = 1.0f / sqrtf(ss * (1.0f / D) + p.eps);
                    float w[N];
                    V::unpack(is_q ? wq : wk, w);
#pragma unroll
                    for (int e = 0; e < N; ++e) x[e] = x[e] * rs * w[e];
                }
            }
            if (p.half_rot) {
                const float4 *c = cs[row];
                if (p.interleaved) {
                    if (!is_v && c0 < 2 * p.half_rot) {
#pragma unroll
                        for (int e = 0; e < N; e += 4) {
                            const float4 t = c[cs_at((c0 + e) >> 2)];  // pairs (c0 + e) / 2 and the next
                            const float a0 = x[e], b0 = x[e + 1], a1 = x[e + 2], b1 = x[e + 3];
                            x[e] = a0 * t.x - b0 * t.y, x[e + 1] = a0 * t.y + b0 * t.x;
                            x[e + 2] = a1 * t.z - b1 * t.w, x[e + 3] = a1 * t.w + b1 * t.z;
                        }
                    }
                } else {
                    // partner of channel i: i + half (first half) or i - half; half is a
                    // multiple of 4, so with 8 values a lane it may sit 4 further along
                    const int q = p.half_rot / N, sh = p.half_rot % N;
                    float y[N];
#pragma unroll
                    for (int e = 0; e < N; ++e) {
                        const bool first = c0 + e < p.half_rot;
                        const int carry = sh ? (first ? (e >= 4 ? 1 : 0) : (e < 4 ? 1 : 0)) : 0;
                        const int src = first ? l + q + carry : l - q - carry;
                        const float v0 = sh ? x[(e + 4) % N] : x[e];
                        y[e] = __shfl_sync(0xffffffffu, v0, src, LPH);
                    }
#pragma unroll
                    for (int e = 0; e < N; e += 2) {
                        const int i = c0 + e;
                        if (!is_v && i < 2 * p.half_rot) {
                            const bool first = i < p.half_rot;
                            const float4 t = c[cs_at((first ? i : i - p.half_rot) >> 1)];
                            x[e] = first ? x[e] * t.x - y[e] * t.y : x[e] * t.x + y[e] * t.y;
                            x[e + 1] = first ? x[e + 1] * t.z - y[e + 1] * t.w : x[e + 1] * t.z + y[e + 1] * t.w;
                        }
                    }
                }
            }
            int ex = 0;
            if constexpr (kE4m3) {
                float m = 0.f;
#pragma unroll
                for (int e = 0; e < N; ++e) m = fmaxf(m, isfinite(x[e]) ? fabsf(x[e]) : 0.f);
#pragma unroll
                for (int o = LPH / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                ex = scale_exponent(m);
            }
            if (!live || s_pos[row] < 0) continue;
            if (is_q) {
                Act *dst = static_cast<Act *>(p.q_out) + size_t(row_base + row) * size_t(p.qo_stride) + size_t(h) * D + c0;
                *reinterpret_cast<uint4 *>(dst) = V::pack(x);
                continue;
            }
            if (s_page[row] < 0) continue;
            const int line = s_pos[row] & ((1 << p.b.page_shift) - 1), hk = is_v ? h - p.hq - p.hkv : h - p.hq;
            const size_t vec = ((size_t(s_page[row]) * size_t(p.hkv) + size_t(hk)) << p.b.page_shift) + size_t(line);
            void *pages = is_v ? p.pv : p.pk;
            if constexpr (kE4m3) {
                const float f = exp2_neg_biased(max(ex, 1));
#pragma unroll
                for (int e = 0; e < N; ++e) x[e] = isfinite(x[e]) ? x[e] * f : __int_as_float(0x7fffffff);
                store_e4m3<N>(static_cast<uint8_t *>(pages) + vec * D + c0, x);
                if (l == 0) (is_v ? p.sv : p.sk)[vec] = uint8_t(ex);
            } else {
                *reinterpret_cast<uint4 *>(static_cast<Act *>(pages) + vec * D + c0) = V::pack(x);
            }
        }
    }
}

struct ReadParams {
    BatchView b;
    const void *pk, *pv;
    const uint8_t *sk, *sv;
    void *k_out, *v_out;
    int32_t hkv, rows_per_cta;
};

template <typename Act, int D, bool kE4m3>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const ReadParams p) {
    using V = Vec<Act>;
    constexpr int N = V::N, LPH = D / N;
    __shared__ int s_pos[kRowsPerCta], s_page[kRowsPerCta];
    const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5;
    const int row_base = int(blockIdx.x) * p.rows_per_cta;
    wait_prior_kernel();
    allow_next_kernel();
    if (warp < p.rows_per_cta) {
        const int r = row_base + warp;
        int pos = -1, page = -1;
        const int n = r < p.b.max_rows ? find_seq(p.b, r, lane) : -1;
        if (lane == 0 && n >= 0 && n < p.b.n_seqs) {
            Seq s;
            if (load_seq(p.b, n, s, true)) {
                pos = s.L - s.T + (r - s.row0);
                page = load_page(p.b, n, pos);
            }
        }
        if (lane == 0) s_pos[warp] = pos, s_page[warp] = page;
    }
    __syncthreads();
    const int items = p.rows_per_cta * 2 * p.hkv, mine = tid / LPH, c0 = (tid % LPH) * N;
    for (int base = 0; base < items; base += kUnroll * (kThreads / LPH)) {
        uint4 raw[kUnroll];
        int ex[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int it = base + u * (kThreads / LPH) + mine;
            raw[u] = make_uint4(0, 0, 0, 0);
            ex[u] = 0;
            if (it >= items) continue;
            const int row = it / (2 * p.hkv), j = it % (2 * p.hkv), hk = j % p.hkv;
            if (s_pos[row] < 0 || s_page[row] < 0) continue;
            const bool is_v = j >= p.hkv;
            const int line = s_pos[row] & ((1 << p.b.page_shift) - 1);
            const size_t vec = ((size_t(s_page[row]) * size_t(p.hkv) + size_t(hk)) << p.b.page_shift) + size_t(line);
            const void *pages = is_v ? p.pv : p.pk;
            if constexpr (kE4m3) {
                const uint8_t *src = static_cast<const uint8_t *>(pages) + vec * D + c0;
                if constexpr (N == 8) {
                    const uint2 t = *reinterpret_cast<const uint2 *>(src);
                    raw[u].x = t.x, raw[u].y = t.y;
                } else {
                    raw[u].x = *reinterpret_cast<const uint32_t *>(src);
                }
                ex[u] = (is_v ? p.sv : p.sk)[vec];
            } else {
                raw[u] = *reinterpret_cast<const uint4 *>(static_cast<const Act *>(pages) + vec * D + c0);
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int it = base + u * (kThreads / LPH) + mine;
            if (it >= items) continue;
            const int row = it / (2 * p.hkv), j = it % (2 * p.hkv), hk = j % p.hkv;
            if (s_pos[row] < 0) continue;
            uint4 o = raw[u];
            if constexpr (kE4m3) {
                const float f = exp2_biased(ex[u]);
                const uint32_t w[2] = {raw[u].x, raw[u].y};
                float x[N];
#pragma unroll
                for (int e = 0; e < N; e += 2) {
                    const float2 t = unpack_e4m3(uint16_t(w[e / 4] >> ((e & 2) * 8)));
                    x[e] = t.x * f, x[e + 1] = t.y * f;
                }
                o = V::pack(x);
            }
            Act *dst = static_cast<Act *>(j >= p.hkv ? p.v_out : p.k_out);
            *reinterpret_cast<uint4 *>(dst + (size_t(row_base + row) * size_t(p.hkv) + size_t(hk)) * D + c0) = o;
        }
    }
}

// Few rows: one row a CTA and its heads spread over CTAs so that every thread
// has one 16-byte item (latency).  Many rows: kRowsPerCta rows a CTA.  The
// border is where one item per thread fills every SM once.
template <typename Act, int D> bool few_rows(int rows, int heads) {
    return static_cast<long long>(rows) * heads * (D / Vec<Act>::N) <= 2048LL * sm_count();
}

template <typename Act, int D, bool kE4m3>
kda_status append_d(AppendParams &p, int rows, cudaStream_t stream) {
    const int heads = p.hq + 2 * p.hkv;
    const bool few = few_rows<Act, D>(rows, heads);
    p.rows_per_cta = few ? 1 : kRowsPerCta;
    p.heads_per_cta = few ? kThreads / (D / Vec<Act>::N) : heads;
    const dim3 grid(unsigned((rows + p.rows_per_cta - 1) / p.rows_per_cta),
                    unsigned((heads + p.heads_per_cta - 1) / p.heads_per_cta));
    const ProfScope prof(KDA_KERNEL_KV_APPEND, stream);
    return launch_overlapped(kv_append_kernel<Act, D, kE4m3>, grid, kThreads, 0, stream, p);
}

template <typename Act, int D, bool kE4m3>
kda_status read_d(ReadParams &p, int rows, cudaStream_t stream) {
    p.rows_per_cta = few_rows<Act, D>(rows, 2 * p.hkv) ? 1 : kRowsPerCta;
    const ProfScope prof(KDA_KERNEL_KV_READ, stream);
    return launch_overlapped(kv_read_kernel<Act, D, kE4m3>, dim3(unsigned((rows + p.rows_per_cta - 1) / p.rows_per_cta)),
                             kThreads, 0, stream, p);
}

template <typename Act, bool kE4m3, typename P, typename F>
kda_status by_dim(int D, P &p, F f) {
    switch (D) {
        case 16: return f(std::integral_constant<int, 16>(), p);
        case 32: return f(std::integral_constant<int, 32>(), p);
        case 64: return f(std::integral_constant<int, 64>(), p);
        case 128: return f(std::integral_constant<int, 128>(), p);
    }
    return KDA_ERR_UNSUPPORTED;
}

template <typename Act, bool kE4m3>
kda_status append_t(int D, AppendParams &p, int rows, cudaStream_t s) {
    return by_dim<Act, kE4m3>(D, p, [&](auto d, AppendParams &q) { return append_d<Act, decltype(d)::value, kE4m3>(q, rows, s); });
}
template <typename Act, bool kE4m3>
kda_status read_t(int D, ReadParams &p, int rows, cudaStream_t s) {
    return by_dim<Act, kE4m3>(D, p, [&](auto d, ReadParams &q) { return read_d<Act, decltype(d)::value, kE4m3>(q, rows, s); });
}

}  // namespace

int sm_count() {
    static int cached[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        cudaGetLastError();
        return 152;
    }
    int sms = cached[dev];
    if (sms == 0 && cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess) cached[dev] = sms;
    return sms > 0 ? sms : 152;
}

kda_status launch_append(const kda_kv_cache *c, const kda_qk_params *qp, const kda_kv_io *io, const kda_kv_batch *b,
                         cudaStream_t stream) {
    AppendParams p = {};
    p.b = make_view(c, b);
    p.q = io->q, p.k = io->k, p.v = io->v, p.q_out = io->q_out;
    p.pk = c->k, p.pv = c->v, p.sk = c->k_scale, p.sv = c->v_scale;
    p.q_stride = io->q_stride, p.k_stride = io->k_stride, p.v_stride = io->v_stride, p.qo_stride = io->q_out_stride;
    p.hq = io->q ? c->num_heads : 0, p.hkv = c->num_kv_heads;
    if (qp) {
        p.wq = qp->q_norm_w, p.wk = qp->k_norm_w, p.eps = qp->eps;
        p.half_rot = qp->rot_dim / 2, p.interleaved = qp->interleaved;
        for (int i = 0; i < p.half_rot; ++i) {
            const double t = qp->inv_freq[i] / 6.283185307179586476925286766559, f = t - std::floor(t);
            p.turn[i] = f < 1.0 ? uint64_t(f * 0x1p64) : 0;
        }
    }
    const int rows = b->max_rows, D = c->head_dim;
    const bool e4 = c->format == KDA_KV_E4M3;
    if (c->act == KDA_BF16)
        return e4 ? append_t<__nv_bfloat16, true>(D, p, rows, stream) : append_t<__nv_bfloat16, false>(D, p, rows, stream);
    return e4 ? append_t<float, true>(D, p, rows, stream) : append_t<float, false>(D, p, rows, stream);
}

kda_status launch_read(const kda_kv_cache *c, const kda_kv_batch *b, void *k_out, void *v_out, cudaStream_t stream) {
    ReadParams p = {};
    p.b = make_view(c, b);
    p.pk = c->k, p.pv = c->v, p.sk = c->k_scale, p.sv = c->v_scale;
    p.k_out = k_out, p.v_out = v_out, p.hkv = c->num_kv_heads;
    const int rows = b->max_rows, D = c->head_dim;
    const bool e4 = c->format == KDA_KV_E4M3;
    if (c->act == KDA_BF16)
        return e4 ? read_t<__nv_bfloat16, true>(D, p, rows, stream) : read_t<__nv_bfloat16, false>(D, p, rows, stream);
    return e4 ? read_t<float, true>(D, p, rows, stream) : read_t<float, false>(D, p, rows, stream);
}

}  // namespace kv
}  // namespace kda
