// kda_latent.cu -- the latent cache's writers and readers: kda_latent_append (RMSNorm of
// the latents, position rotation of the shared key part and the queries, the quantised
// page write) and kda_latent_read.  Formulas, layout and contracts: include/kda.h.
//
// Both only move data.  A token has one latent (a warp holds it: 16 bytes a lane and
// step, sums and maxima by shuffles) and num_heads + 1 short vectors that turn, of
// which the queries' are most of the bytes (64 heads of 64 channels: 16 KB read and
// written, beside 2 KB for the cache).  A thread takes two places of 4 or 8 channels of
// such a vector that turn together, so no partner has to be fetched from another lane.
// Bound by memory: 32768 tokens at 64 heads with e4m3 pages 99 us, 6.0 TB/s, reading as many back 12.9 us, 4.6 TB/s
// (in a graph, one after another over tensors that do not fit L2; a call alone behind an emptied L2, launch included, 106 and
// 20 us).  One token: 3.5 us like that, called one after another from the host 5.6: the chain from the tables to a
// row's place and angles.
#include "kda_latent.cuh"
#include "kda_rows.cuh"

namespace kda {
namespace kv {
namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;
constexpr int kMaxHalf = 32;  // pairs that turn

struct LatentAppendParams {
    BatchView b;
    const void *c, *kr, *q, *w;
    void *q_out, *pc, *pkr;
    uint8_t *sc;
    long long c_stride, kr_stride, q_stride, q_head, qo_stride, qo_head;
    int32_t heads;  // 0 when the call has no queries
    int32_t latent, rope, half_rot, interleaved, rows_per_cta;
    int32_t slot_shift;  // log2 of the places pairs of a vector
    float eps;
    uint64_t turn[kMaxHalf];  // inv_freq / (2 pi) mod 1, in units of 2^-64
};

// W channels as they lie in memory.
template <typename Act, int W> struct Place;
template <> struct Place<float, 4> {
    using Raw = uint4;
    static __device__ __forceinline__ void unpack(const Raw &r, float (&x)[4]) { Vec<float>::unpack(r, x); }
    static __device__ __forceinline__ Raw pack(const float (&x)[4]) { return Vec<float>::pack(x); }
};
template <> struct Place<__nv_bfloat16, 8> {
    using Raw = uint4;
    static __device__ __forceinline__ void unpack(const Raw &r, float (&x)[8]) { Vec<__nv_bfloat16>::unpack(r, x); }
    static __device__ __forceinline__ Raw pack(const float (&x)[8]) { return Vec<__nv_bfloat16>::pack(x); }
};
template <> struct Place<__nv_bfloat16, 4> {
    using Raw = uint2;
    static __device__ __forceinline__ void unpack(const Raw &r, float (&x)[4]) {
        x[0] = __uint_as_float(r.x << 16), x[1] = __uint_as_float(r.x & 0xffff0000u);
        x[2] = __uint_as_float(r.y << 16), x[3] = __uint_as_float(r.y & 0xffff0000u);
    }
    static __device__ __forceinline__ Raw pack(const float (&x)[4]) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
        return make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    }
};

// a <- a + b, what the sum loses to rest (a and b of any sizes).
__device__ __forceinline__ void two_sum(float &a, float &rest, float b) {
    const float s = __fadd_rn(a, b), b_in = __fsub_rn(s, a);
    rest += __fadd_rn(__fsub_rn(a, __fsub_rn(s, b_in)), __fsub_rn(b, b_in));
    a = s;
}

// A warp's latent: normalised, to its line of the pages.
template <typename Act, bool kE4m3>
__device__ __forceinline__ void latent_to_page(const LatentAppendParams &p, size_t row, int page, int line, int lane) {
    using V = Vec<Act>;
    constexpr int N = V::N, kPieces = 512 / N / 32;
    const int n = p.latent / N;  // 16-byte pieces of the vector
    uint4 raw[kPieces], w_raw[kPieces];
    const Act *src = static_cast<const Act *>(p.c) + row * size_t(p.c_stride);
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
        const int i = lane + 32 * k;
        raw[k] = w_raw[k] = make_uint4(0, 0, 0, 0);
        if (i < n) {
            raw[k] = *reinterpret_cast<const uint4 *>(src + i * N);
            if (p.w) w_raw[k] = __ldg(static_cast<const uint4 *>(p.w) + i);
        }
    }
    float x[kPieces][N];
#pragma unroll
    for (int k = 0; k < kPieces; ++k) V::unpack(raw[k], x[k]);
    if (p.w) {
        // Latents on their way to e4m3 pages carry every rounding but the last along: next to a border of e4m3 a last
        // bit becomes a whole step.  So their sum of squares is one of two floats, ss + rest.
        float ss = 0.f, rest = 0.f;
#pragma unroll
        for (int k = 0; k < kPieces; ++k)
#pragma unroll
            for (int e = 0; e < N; ++e) {
                if constexpr (kE4m3) {
                    const float sq = __fmul_rn(x[k][e], x[k][e]);
                    rest += fmaf(x[k][e], x[k][e], -sq);
                    two_sum(ss, rest, sq);
                } else {
                    ss = fmaf(x[k][e], x[k][e], ss);
                }
            }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float other = __shfl_xor_sync(0xffffffffu, ss, o);
            if constexpr (kE4m3) {
                rest += __shfl_xor_sync(0xffffffffu, rest, o);
                two_sum(ss, rest, other);
            } else {
                ss += other;
            }
        }
        const float inv = 1.0f / float(p.latent);  // a power of two
        float y = ss * inv, y_rest = rest * inv, rs_rest = 0.f;
        if constexpr (kE4m3) two_sum(y, y_rest, p.eps);
        else y += p.eps;
        const float rs = 1.0f / sqrtf(y);
        if (kE4m3) {  // 1 / sqrt(y + y_rest) = rs + rs_rest: half of what (y + y_rest) rs^2 misses of one
            const float t = __fmul_rn(y, rs), miss = fmaf(-t, rs, 1.0f) - fmaf(y, rs, -t) * rs - y_rest * rs * rs;
            rs_rest = isfinite(miss) ? 0.5f * rs * miss : 0.f;
        }
#pragma unroll
        for (int k = 0; k < kPieces; ++k) {
            float w[N];
            V::unpack(w_raw[k], w);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float xw = __fmul_rn(x[k][e], w[e]);
                if (kE4m3) {
                    const float lost = fmaf(x[k][e], w[e], -xw), z = fmaf(xw, rs, fmaf(xw, rs_rest, lost * rs));
                    x[k][e] = isfinite(z) ? z : xw * rs;
                } else {
                    x[k][e] = xw * rs;
                }
            }
        }
    }
    if (page < 0) return;
    const size_t vec = (size_t(page) << p.b.page_shift) + size_t(line);
    if constexpr (kE4m3) {
        float m = 0.f;
#pragma unroll
        for (int k = 0; k < kPieces; ++k)
#pragma unroll
            for (int e = 0; e < N; ++e) m = fmaxf(m, isfinite(x[k][e]) ? fabsf(x[k][e]) : 0.f);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const int ex = scale_exponent(m);
        const float f = exp2_neg_biased(max(ex, 1));
        uint8_t *dst = static_cast<uint8_t *>(p.pc) + vec * size_t(p.latent);
#pragma unroll
        for (int k = 0; k < kPieces; ++k) {
            const int i = lane + 32 * k;
#pragma unroll
            for (int e = 0; e < N; ++e) x[k][e] = isfinite(x[k][e]) ? x[k][e] * f : __int_as_float(0x7fffffff);
            if (i < n) store_e4m3<N>(dst + i * N, x[k]);
        }
        if (lane == 0) p.sc[vec] = uint8_t(ex);
    } else {
        Act *dst = static_cast<Act *>(p.pc) + vec * size_t(p.latent);
#pragma unroll
        for (int k = 0; k < kPieces; ++k) {
            const int i = lane + 32 * k;
            if (i < n) *reinterpret_cast<uint4 *>(dst + i * N) = p.w ? V::pack(x[k]) : raw[k];
        }
    }
}

// A row is one warp's, or two or all four warps of a CTA share its vectors (few rows: latency); the last of them
// has the latent.  A thread's places are the same in all its vectors, so it keeps their cosines and sines in
// registers (from shared memory for each vector, a CTA's warps sharing all its rows: 119 us for 32768 tokens and
// 53 for eight prompts of 500 to 2000, against 111 and 43; with four vectors in flight instead of three 135 and 53; between
// events around single calls behind an emptied L2, which is longer than the kernel).
// W: channels of a place, 8 (bf16, 16 bytes) where half the channels that turn are a multiple of it, else 4.
template <typename Act, bool kE4m3, int W>
__global__ void __launch_bounds__(kThreads) latent_append_kernel(const __grid_constant__ LatentAppendParams p) {
    using Pl = Place<Act, W>;
    using Raw = typename Pl::Raw;
    constexpr int kUnroll = 3;
    __shared__ float2 cs[kWarps][kMaxHalf];
    const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5;
    const int per_row = kWarps / p.rows_per_cta, part = warp % per_row;  // warps of a row
    const long long at_row = static_cast<long long>(blockIdx.x) * p.rows_per_cta + warp / per_row;
    const int row = int(min(at_row, static_cast<long long>(p.b.max_rows)));
    wait_prior_kernel();
    allow_next_kernel();
    if (warp == 0) report_seqs(p.b, lane);
    if (row >= p.b.max_rows) return;
    int pos, page;
    find_row(p.b, row, lane, pos, page);
    pos = __shfl_sync(0xffffffffu, pos, 0), page = __shfl_sync(0xffffffffu, page, 0);
    if (pos < 0) return;
    const int line = pos & ((1 << p.b.page_shift) - 1);

    // this thread's two places of a vector, and which of them turn
    const int s = lane & ((1 << p.slot_shift) - 1), rot = 2 * p.half_rot;
    int ch[2];
    bool on[2];
    if (p.interleaved) {
        ch[0] = 2 * s * W, ch[1] = ch[0] + W;
        on[0] = ch[0] < rot, on[1] = ch[1] < rot;
    } else {
        const int turning = p.half_rot / W;  // of the places, pairs that turn
        const bool t = s < turning;
        ch[0] = t ? s * W : rot + 2 * (s - turning) * W, ch[1] = ch[0] + (t ? p.half_rot : W);
        on[0] = on[1] = t;
    }
    // vector 0 is kr, the others the query heads
    const int n_vec = p.heads + 1, step = per_row * (32 >> p.slot_shift);
    const Act *q = static_cast<const Act *>(p.q) + size_t(row) * size_t(p.q_stride);
    Act *q_out = static_cast<Act *>(p.q_out) + size_t(row) * size_t(p.qo_stride);
    Raw raw[kUnroll][2];
    auto load = [&](int v) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u, v += step) {
            raw[u][0] = raw[u][1] = Raw{};
            if (v >= n_vec) continue;
            const Act *src = v == 0 ? static_cast<const Act *>(p.kr) + size_t(row) * size_t(p.kr_stride)
                                    : q + size_t(v - 1) * size_t(p.q_head);
            raw[u][0] = *reinterpret_cast<const Raw *>(src + ch[0]);
            raw[u][1] = *reinterpret_cast<const Raw *>(src + ch[1]);
        }
    };
    int v = part * (32 >> p.slot_shift) + (lane >> p.slot_shift);
    load(v);
    // angle p * f in turns is a 64-bit product mod 2^64, as good as the frequency there times the position
    if (lane < p.half_rot) cs[warp][lane] = cos_sin(uint64_t(uint32_t(pos)) * p.turn[lane]);
    __syncwarp();
    float2 f[W];  // interleaved: of the first place's pairs and of the second's
#pragma unroll
    for (int e = 0; e < W; ++e) {
        const int i = p.interleaved ? ch[e / (W / 2)] / 2 + e % (W / 2) : ch[0] + e;
        f[e] = cs[warp][min(i, kMaxHalf - 1)];
    }
    for (; v < n_vec; v += kUnroll * step, load(v)) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int vec = v + u * step;
            if (vec >= n_vec || (vec == 0 && page < 0)) continue;
            Act *dst = vec == 0 ? static_cast<Act *>(p.pkr) + ((size_t(page) << p.b.page_shift) + size_t(line)) * size_t(p.rope)
                                : q_out + size_t(vec - 1) * size_t(p.qo_head);
            float a[W], b[W];
            Pl::unpack(raw[u][0], a), Pl::unpack(raw[u][1], b);
            if (p.interleaved) {
#pragma unroll
                for (int e = 0; e < W; e += 2) {
                    const float2 g = f[e / 2], h = f[W / 2 + e / 2];
                    const float x = a[e], y = a[e + 1], z = b[e], w = b[e + 1];
                    a[e] = x * g.x - y * g.y, a[e + 1] = fmaf(x, g.y, y * g.x);
                    b[e] = z * h.x - w * h.y, b[e + 1] = fmaf(z, h.y, w * h.x);
                }
            } else {
#pragma unroll
                for (int e = 0; e < W; ++e) {
                    const float x = a[e], y = b[e];
                    a[e] = x * f[e].x - y * f[e].y, b[e] = fmaf(x, f[e].y, y * f[e].x);
                }
            }
            // channels that do not turn go as they are
            *reinterpret_cast<Raw *>(dst + ch[0]) = on[0] ? Pl::pack(a) : raw[u][0];
            *reinterpret_cast<Raw *>(dst + ch[1]) = on[1] ? Pl::pack(b) : raw[u][1];
        }
    }
    if (part == per_row - 1) latent_to_page<Act, kE4m3>(p, size_t(row), page, line, lane);
}

struct LatentReadParams {
    BatchView b;
    const void *pc, *pkr;
    const uint8_t *sc;
    void *c_out, *kr_out;
    long long c_stride, kr_stride;
    int32_t latent, rope;
};

// A warp a row.  64 heads' cache, bf16 / e4m3 pages, in a graph one after another: 1 row 1.7 / 1.6 us, 1216 2.8 / 2.5, 4864 4.2 /
// 4.1, 9728 5.9 / 5.8, 32768 13.9 / 12.9 (floors 11.1 and 8.6).
template <typename Act, bool kE4m3>
__global__ void __launch_bounds__(kThreads) latent_read_kernel(const LatentReadParams p) {
    using V = Vec<Act>;
    constexpr int N = V::N, NC = kE4m3 ? 16 : N, kPieces = 512 / NC / 32;  // channels of a loaded piece of c
    const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5;
    const long long at_row = static_cast<long long>(blockIdx.x) * kWarps + warp;
    const int row = int(min(at_row, static_cast<long long>(p.b.max_rows)));
    const int n = p.latent / NC, nr = p.rope / N;
    wait_prior_kernel();
    allow_next_kernel();
    if (warp == kWarps - 1) report_seqs(p.b, lane);
    if (row >= p.b.max_rows) return;
    int pos, page;
    find_row(p.b, row, lane, pos, page);
    pos = __shfl_sync(0xffffffffu, pos, 0), page = __shfl_sync(0xffffffffu, page, 0);
    if (pos < 0) return;
    const size_t vec = (size_t(max(page, 0)) << p.b.page_shift) + size_t(pos & ((1 << p.b.page_shift) - 1));
    uint4 raw[kPieces], rr = make_uint4(0, 0, 0, 0);
    int ex = 0;
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
        raw[k] = make_uint4(0, 0, 0, 0);
        if (page >= 0 && lane + 32 * k < n)
            raw[k] = *reinterpret_cast<const uint4 *>(static_cast<const unsigned char *>(p.pc) +
                                                      (vec * size_t(p.latent) + size_t(lane + 32 * k) * NC) *
                                                          (kE4m3 ? 1 : sizeof(Act)));
    }
    if (page >= 0) {
        if (lane < nr)
            rr = *reinterpret_cast<const uint4 *>(static_cast<const Act *>(p.pkr) + vec * size_t(p.rope) + lane * N);
        if constexpr (kE4m3) ex = p.sc[vec];
    }
    Act *dst = static_cast<Act *>(p.c_out) + size_t(row) * size_t(p.c_stride);
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
        const int at = lane + 32 * k;
        if (at >= n) continue;
        if constexpr (kE4m3) {
            const float f = exp2_biased(ex);
            const uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
#pragma unroll
            for (int j = 0; j < NC / N; ++j) {
                float x[N];
#pragma unroll
                for (int e = 0; e < N; e += 2) {
                    const int c = j * N + e;
                    const float2 t = unpack_e4m3(uint16_t(w[c / 4] >> ((c & 2) * 8)));
                    x[e] = t.x * f, x[e + 1] = t.y * f;
                }
                *reinterpret_cast<uint4 *>(dst + at * NC + j * N) = V::pack(x);
            }
        } else {
            *reinterpret_cast<uint4 *>(dst + at * N) = raw[k];
        }
    }
    if (lane < nr)
        *reinterpret_cast<uint4 *>(static_cast<Act *>(p.kr_out) + size_t(row) * size_t(p.kr_stride) + lane * N) = rr;
}

template <typename Act, bool kE4m3> kda_status append_t(LatentAppendParams &p, int rows, cudaStream_t stream) {
    // The fewest rows a CTA that leave one wave (an SM holds six CTAs), else a warp each.  With norm and rotation, latents of
    // 512 to pages in bf16 / e4m3, in a graph one after another, us with one, two and four rows a CTA:
    //   64 heads  912 rows 6.0 / 6.4, 6.6 / 7.0, 7.6 / 8.0; 1064 8.5 / 9.4, 7.4 / 8.0, 7.9 / 8.2;
    //             1824 10.4 / 11.1, 8.6 / 9.1, 9.4 / 9.9; 2128 12.5 / 13.5, 11.8 / 12.8, 10.6 / 11.9; 9728 40 / 44, 35 / 38, 31 / 34
    //   8 heads   912 rows 4.5 / 4.9, 4.6 / 5.0, 4.6 / 5.0; 1064 6.6 / 7.4, 4.9 / 5.5, 4.6 / 5.0;
    //             1824 7.9 / 8.6, 5.2 / 5.8, 4.9 / 5.6; 2128 9.5 / 10.6, 7.8 / 8.8, 5.6 / 7.0; 9728 30 / 34, 21 / 24, 14 / 17
    p.rows_per_cta = rows <= 6 * sm_count() ? 1 : rows <= 12 * sm_count() ? 2 : kWarps;
    const dim3 grid(unsigned((rows - 1) / p.rows_per_cta + 1));
    constexpr int N = Vec<Act>::N;
    const bool wide = p.half_rot % N == 0;
    const int places = p.rope / (2 * (wide ? N : 4));
    p.slot_shift = places >= 8 ? 3 : places >= 4 ? 2 : places >= 2 ? 1 : 0;
    const ProfScope prof(KDA_KERNEL_LATENT_APPEND, stream);
    if constexpr (N == 8)
        if (!wide) return launch_overlapped(latent_append_kernel<Act, kE4m3, 4>, grid, kThreads, 0, stream, p);
    return launch_overlapped(latent_append_kernel<Act, kE4m3, N>, grid, kThreads, 0, stream, p);
}

template <typename Act, bool kE4m3> kda_status read_t(LatentReadParams &p, int rows, cudaStream_t stream) {
    const ProfScope prof(KDA_KERNEL_LATENT_READ, stream);
    return launch_overlapped(latent_read_kernel<Act, kE4m3>, dim3(unsigned((rows - 1) / kWarps + 1)), kThreads, 0, stream,
                             p);
}

}  // namespace

kda_status launch_latent_append(const kda_latent_cache *c, const kda_latent_params *lp, const kda_latent_io *io,
                                const kda_kv_batch *b, cudaStream_t stream) {
    LatentAppendParams p = {};
    p.b = make_view(c, b);
    p.c = io->c, p.kr = io->kr, p.q = io->q, p.q_out = io->q_out;
    p.pc = c->c, p.pkr = c->kr, p.sc = c->c_scale;
    p.c_stride = io->c_stride, p.kr_stride = io->kr_stride;
    p.q_stride = io->q_stride, p.q_head = io->q_head_stride;
    p.qo_stride = io->q_out_stride, p.qo_head = io->q_out_head_stride;
    p.heads = io->q ? c->num_heads : 0, p.latent = c->latent_dim, p.rope = c->rope_dim;
    if (lp) {
        p.w = lp->c_norm_w, p.eps = lp->eps, p.half_rot = lp->rot_dim / 2, p.interleaved = lp->interleaved;
        for (int i = 0; i < p.half_rot; ++i) p.turn[i] = turn_of(lp->inv_freq[i]);
    }
    const bool e4 = c->format == KDA_KV_E4M3;
    if (c->act == KDA_BF16)
        return e4 ? append_t<__nv_bfloat16, true>(p, b->max_rows, stream) : append_t<__nv_bfloat16, false>(p, b->max_rows, stream);
    return e4 ? append_t<float, true>(p, b->max_rows, stream) : append_t<float, false>(p, b->max_rows, stream);
}

kda_status launch_latent_read(const kda_latent_cache *c, const kda_kv_batch *b, void *c_out, long long c_stride, void *kr_out,
                              long long kr_stride, cudaStream_t stream) {
    LatentReadParams p = {};
    p.b = make_view(c, b);
    p.pc = c->c, p.pkr = c->kr, p.sc = c->c_scale;
    p.c_out = c_out, p.kr_out = kr_out, p.c_stride = c_stride, p.kr_stride = kr_stride;
    p.latent = c->latent_dim, p.rope = c->rope_dim;
    const bool e4 = c->format == KDA_KV_E4M3;
    if (c->act == KDA_BF16)
        return e4 ? read_t<__nv_bfloat16, true>(p, b->max_rows, stream) : read_t<__nv_bfloat16, false>(p, b->max_rows, stream);
    return e4 ? read_t<float, true>(p, b->max_rows, stream) : read_t<float, false>(p, b->max_rows, stream);
}

}  // namespace kv
}  // namespace kda
