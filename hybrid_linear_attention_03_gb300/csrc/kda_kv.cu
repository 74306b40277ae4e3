// kda_kv.cu -- the paged cache's writers and readers: kda_kv_append (per-head
// RMSNorm, position rotation and the quantised page write in one pass) and
// kda_kv_read.  Formulas, layout and contracts: include/kda.h.
//
// Both only move data: append reads (Hq + 2 Hkv) d values a token and writes
// as many (half for e4m3 pages), about 10 operations each, so HBM bounds them
// as long as the instructions around a 16-byte load stay few.  A vector of
// head_dim channels is owned by the head_dim * size / 16 lanes that hold it in
// 16-byte loads (a lane group).  A group keeps to one row: the row's position,
// page and cosines are worked out once, and then its heads go by with no more
// than a pointer step between them.  Sums of squares, largest magnitudes and
// rotation partners move by shuffles.
// Measured, 64 heads over 8 cache heads of 128 in bf16: 8 ragged prompts of 511 to
// 2049 tokens written in 82 us (5.3 TB/s, 79 % of the measured copy rate); 32768
// tokens written in e4m3 and read back 318 us (4.4 TB/s: beside the bytes there is
// the search for a vector's largest magnitude, and the keys' roundings are carried
// along, which takes 13 us and halves the share of values that a rounding before
// the last puts on the wrong side of an e4m3 border); one token 4.6 us, 64 of them
// written and read in e4m3 9 us (launches).
#include "kda_rows.cuh"

#include <atomic>

namespace kda {
namespace kv {
namespace {

constexpr int kThreads = 256;
// Most rows of a CTA, for lane groups of `lanes` lanes.
constexpr int max_rows_per_cta(int lanes) { return kThreads / lanes < 32 ? kThreads / lanes : 32; }
constexpr int kUnroll = 4;      // 16-byte loads in flight per thread

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
    uint64_t turn[64];  // inv_freq / (2 pi) mod 1, in units of 2^-64
};

// x <- x c + t where `on`, as one instruction under a predicate (32768 tokens written and
// read in bf16: 282 us this way, 285 with a select or a branch, 280 if every channel turned).
__device__ __forceinline__ void fma_where(bool on, float &x, float c, float t) {
    asm("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %3, 0;\n\t@p fma.rn.f32 %0, %0, %1, %2;\n\t}"
        : "+f"(x)
        : "f"(c), "f"(t), "r"(uint32_t(on)));
}

enum { kNoRot = 0, kHalves = 1, kPairs = 2 };  // rotation: none, channels (i, i + half), channels (2i, 2i + 1)

// One CTA: rows_per_cta rows x heads_per_cta of the hq + 2 hkv heads.  Four CTAs an
// SM (64 registers) against three at 72: 307 against 330 us for the 32768 tokens
// (before the keys carried their roundings).
template <typename Act, int D, bool kE4m3, int kRot>
__global__ void __launch_bounds__(kThreads, 4) kv_append_kernel(const __grid_constant__ AppendParams p) {
    using V = Vec<Act>;
    constexpr int N = V::N, LPH = D / N, kGroups = kThreads / LPH;  // values per lane, lanes per group
    constexpr int kRows = max_rows_per_cta(LPH);
    __shared__ float2 cs[kRows][D / 2];
    __shared__ int s_pos[kRows], s_page[kRows];
    const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5;
    const int row_base = int(blockIdx.x) * p.rows_per_cta;
    wait_prior_kernel();
    allow_next_kernel();
    for (int i = warp; i < p.rows_per_cta; i += kThreads / 32) {
        int pos, page;
        find_row(p.b, row_base + i, lane, pos, page);
        if (lane == 0) s_pos[i] = pos, s_page[i] = page;
    }
    if (blockIdx.y == 0 && warp == kThreads / 32 - 1) report_seqs(p.b, lane);
    __syncthreads();
    if constexpr (kRot != kNoRot) {
        // angle p * f in turns is a 64-bit product mod 2^64, as good as the frequency there times the position
        for (int i = tid; i < p.rows_per_cta * p.half_rot; i += kThreads) {
            const int row = i / p.half_rot, pair = i % p.half_rot;
            const uint64_t ph = uint64_t(uint32_t(max(s_pos[row], 0))) * p.turn[pair];
            cs[row][pair] = cos_sin(ph);
        }
        __syncthreads();
    }

    // This lane group: row `row`, heads j, j + step, ...  Groups of a warp may have different rows and
    // head counts, so the loops below run to the same end for all and the lanes' work is masked.
    const int step = kGroups / p.rows_per_cta, row = (tid / LPH) / step, j = (tid / LPH) % step;
    const int l = tid % LPH, c0 = l * N;
    const int pos = s_pos[row], page = s_page[row];
    const size_t r = size_t(row_base + row);
    const bool turns = c0 < 2 * p.half_rot;  // all of this lane's channels or none: rot_dim is a multiple of 8
    float cn[N], sn[N];  // of this lane's channels; the sine with the sign it takes
    if constexpr (kRot != kNoRot) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const int c = c0 + e;
            const bool second = kRot == kPairs ? (e & 1) != 0 : c >= p.half_rot;
            const int pair = !turns ? 0 : kRot == kPairs ? c / 2 : second ? c - p.half_rot : c;
            const float2 t = turns ? cs[row][pair] : make_float2(1.f, 0.f);
            cn[e] = t.x, sn[e] = second ? t.y : -t.y;
        }
    }
    // halves: the partner of channel i is i +- half; half is a multiple of 4, so with 8 values a lane
    // it may sit 4 further along (odd4)
    const int q = p.half_rot / N;
    const bool odd4 = p.half_rot % N != 0, first = c0 < p.half_rot;

    // x: 16 bytes of a q or k head -> normalised and rotated.  fine: every rounding but the last is carried along
    // (keys that go to e4m3 pages).
    auto norm_rotate = [&](float (&x)[N], const uint4 &w_raw, bool norm, bool fine) {
        float rs = 1.f, rs_rest = 0.f;
        if (norm) {
            float sq[N / 2];
#pragma unroll
            for (int e = 0; e < N / 2; ++e) sq[e] = fmaf(x[e], x[e], x[e + N / 2] * x[e + N / 2]);
            float ss = N == 8 ? (sq[0] + sq[1]) + (sq[N / 2 - 2] + sq[N / 2 - 1]) : sq[0] + sq[1];
#pragma unroll
            for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const float y = fmaf(ss, 1.0f / D, p.eps);
            rs = 1.0f / sqrtf(y);
            if (fine) {  // 1 / sqrt(y) = rs + rs_rest: half of what y rs^2 misses of one
                const float t = __fmul_rn(y, rs), miss = fmaf(-t, rs, 1.0f) - fmaf(y, rs, -t) * rs;
                rs_rest = isfinite(miss) ? 0.5f * rs * miss : 0.f;
            }
            float w[N];
            V::unpack(w_raw, w);
#pragma unroll
            for (int e = 0; e < N; ++e) x[e] = fine ? x[e] * w[e] : x[e] * w[e] * rs;  // the first product is exact in bf16
        }
        float y[N] = {};  // the partners
        if constexpr (kRot == kPairs) {
#pragma unroll
            for (int e = 0; e < N; e += 2) y[e] = x[e + 1], y[e + 1] = x[e];
        } else if constexpr (kRot == kHalves) {
            if (!odd4) {
                const int src = first ? l + q : l - q;
#pragma unroll
                for (int e = 0; e < N; ++e) y[e] = __shfl_sync(0xffffffffu, x[e], src, LPH);
            } else {
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const bool fst = c0 + e < p.half_rot;
                    const int src = fst ? l + q + (e >= 4 ? 1 : 0) : l - q - (e < 4 ? 1 : 0);
                    y[e] = __shfl_sync(0xffffffffu, x[(e + 4) % N], src, LPH);
                }
            }
        }
        // channels that do not turn get no multiple of a partner, which may be an infinity or NaN
#pragma unroll
        for (int e = 0; e < N; ++e) {
            if (!fine) {
                if (kRot != kNoRot) fma_where(turns, x[e], cn[e], y[e] * sn[e]);
                continue;
            }
            float sum = x[e], rest = 0.f;
            if (kRot != kNoRot) {
                const float other = turns ? y[e] : 0.f;
                const float a = __fmul_rn(x[e], cn[e]), b = __fmul_rn(other, sn[e]);
                sum = __fadd_rn(a, b);
                const float b_in = __fsub_rn(sum, a);  // and what the sum lost of either
                rest = __fadd_rn(__fsub_rn(a, __fsub_rn(sum, b_in)), __fsub_rn(b, b_in)) + fmaf(x[e], cn[e], -a) +
                       fmaf(other, sn[e], -b);
            }
            const float z = fmaf(sum, rs, fmaf(sum, rs_rest, rest * rs));
            x[e] = isfinite(z) ? z : sum * rs;  // infinities come as they are
        }
    };
    // x to head h of the pages
    const int line = pos & ((1 << p.b.page_shift) - 1);
    const size_t vec0 = (size_t(max(page, 0)) * size_t(p.hkv) << p.b.page_shift) + size_t(max(line, 0));
    auto to_page = [&](float (&x)[N], int h, void *pages, uint8_t *scales, bool live) {
        const size_t vec = vec0 + (size_t(h) << p.b.page_shift);
        if constexpr (kE4m3) {
            float m = 0.f;
#pragma unroll
            for (int e = 0; e < N; ++e) m = fmaxf(m, isfinite(x[e]) ? fabsf(x[e]) : 0.f);
#pragma unroll
            for (int o = LPH / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            const int ex = scale_exponent(m);
            const float f = exp2_neg_biased(max(ex, 1));
#pragma unroll
            for (int e = 0; e < N; ++e) x[e] = isfinite(x[e]) ? x[e] * f : __int_as_float(0x7fffffff);
            if (live) {
                store_e4m3<N>(static_cast<uint8_t *>(pages) + vec * D + c0, x);
                if (l == 0) scales[vec] = uint8_t(ex);
            }
        } else if (live) {
            *reinterpret_cast<uint4 *>(static_cast<Act *>(pages) + vec * D + c0) = V::pack(x);
        }
    };
    // heads [lo, hi) of this CTA among one kind's n heads at `src`; f(x, head, live) for each
    const int cta0 = int(blockIdx.y) * p.heads_per_cta, cta1 = cta0 + p.heads_per_cta;
    auto each_head = [&](const void *base, long long stride, int kind0, int n, auto f) {
        const int lo = max(cta0 - kind0, 0), hi = min(cta1 - kind0, n);
        const Act *src = static_cast<const Act *>(base) + r * size_t(stride) + c0;
        for (int h0 = lo; h0 < hi; h0 += kUnroll * step) {
            uint4 raw[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int h = h0 + u * step + j;
                raw[u] = make_uint4(0, 0, 0, 0);
                if (h < hi && pos >= 0) raw[u] = *reinterpret_cast<const uint4 *>(src + size_t(h) * D);
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                if (h0 + u * step >= hi) break;
                const int h = h0 + u * step + j;
                float x[N];
                V::unpack(raw[u], x);
                f(x, h, h < hi && pos >= 0);
            }
        }
    };

    uint4 wq = make_uint4(0, 0, 0, 0), wk = wq;
    const bool norm_q = p.wq != nullptr, norm_k = p.wk != nullptr;
    if (norm_q) wq = __ldg(reinterpret_cast<const uint4 *>(p.wq) + l);
    if (norm_k) wk = __ldg(reinterpret_cast<const uint4 *>(p.wk) + l);
    Act *q_out = static_cast<Act *>(p.q_out) + r * size_t(p.qo_stride) + c0;
    each_head(p.q, p.q_stride, 0, p.hq, [&](float (&x)[N], int h, bool live) {
        norm_rotate(x, wq, norm_q, false);
        if (live) *reinterpret_cast<uint4 *>(q_out + size_t(h) * D) = V::pack(x);
    });
    each_head(p.k, p.k_stride, p.hq, p.hkv, [&](float (&x)[N], int h, bool live) {
        norm_rotate(x, wk, norm_k, kE4m3);
        to_page(x, h, p.pk, p.sk, live && page >= 0);
    });
    each_head(p.v, p.v_stride, p.hq + p.hkv, p.hkv,
              [&](float (&x)[N], int h, bool live) { to_page(x, h, p.pv, p.sv, live && page >= 0); });
}

struct ReadParams {
    BatchView b;
    const void *pk, *pv;
    const uint8_t *sk, *sv;
    void *k_out, *v_out;
    int32_t hkv, rows_per_cta;
};

// Lane groups as above, each 16 bytes of a page line per lane.
template <typename Act, int D, bool kE4m3>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const ReadParams p) {
    constexpr int N = kE4m3 ? 16 : Vec<Act>::N, LPH = D / N, kGroups = kThreads / LPH;
    constexpr int kRows = max_rows_per_cta(LPH);
    __shared__ int s_pos[kRows], s_page[kRows];
    const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5;
    const int row_base = int(blockIdx.x) * p.rows_per_cta;
    wait_prior_kernel();
    allow_next_kernel();
    for (int i = warp; i < p.rows_per_cta; i += kThreads / 32) {
        int pos, page;
        find_row(p.b, row_base + i, lane, pos, page);
        if (lane == 0) s_pos[i] = pos, s_page[i] = page;
    }
    if (warp == kThreads / 32 - 1) report_seqs(p.b, lane);
    __syncthreads();
    const int step = kGroups / p.rows_per_cta, row = (tid / LPH) / step, j = (tid / LPH) % step;
    const int c0 = (tid % LPH) * N, pos = s_pos[row], page = s_page[row];
    if (pos < 0) return;
    const int line = pos & ((1 << p.b.page_shift) - 1);
    const size_t vec0 = (size_t(max(page, 0)) * size_t(p.hkv) << p.b.page_shift) + size_t(line);
    // head h of both: 2 hkv lines, keys first
    auto load = [&](int h, uint4 &raw, int &ex) {
        raw = make_uint4(0, 0, 0, 0);
        ex = 0;
        if (page < 0 || h >= 2 * p.hkv) return;
        const bool is_v = h >= p.hkv;
        const size_t vec = vec0 + (size_t(is_v ? h - p.hkv : h) << p.b.page_shift);
        const size_t at = (vec * D + size_t(c0)) * (kE4m3 ? 1 : sizeof(Act));
        raw = *reinterpret_cast<const uint4 *>(static_cast<const unsigned char *>(is_v ? p.pv : p.pk) + at);
        if constexpr (kE4m3) ex = (is_v ? p.sv : p.sk)[vec];
    };
    auto store = [&](int h, const uint4 &raw, int ex) {
        if (h >= 2 * p.hkv) return;
        const bool is_v = h >= p.hkv;
        Act *dst = static_cast<Act *>(is_v ? p.v_out : p.k_out) +
                   (size_t(row_base + row) * size_t(p.hkv) + size_t(is_v ? h - p.hkv : h)) * D + c0;
        if constexpr (kE4m3) {
            const float f = exp2_biased(ex);
            const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
            constexpr int M = Vec<Act>::N;
#pragma unroll
            for (int i = 0; i < N / M; ++i) {
                float x[M];
#pragma unroll
                for (int e = 0; e < M; e += 2) {
                    const int at = i * M + e;
                    const float2 t = unpack_e4m3(uint16_t(w[at / 4] >> ((at & 2) * 8)));
                    x[e] = t.x * f, x[e + 1] = t.y * f;
                }
                *reinterpret_cast<uint4 *>(dst + i * M) = Vec<Act>::pack(x);
            }
        } else {
            *reinterpret_cast<uint4 *>(dst) = raw;
        }
    };
    for (int h0 = j; h0 < 2 * p.hkv; h0 += kUnroll * step) {
        uint4 raw[kUnroll];
        int ex[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) load(h0 + u * step, raw[u], ex[u]);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) store(h0 + u * step, raw[u], ex[u]);
    }
}

// Rows of a CTA.  Few rows: as few as leave every thread one 16-byte piece of
// the row's heads (latency); the border is where one piece per thread fills every
// SM once (64 heads over 8 of 128 in bf16, 240 rows: 9.5 us this way, 11.1 the
// other; 320 rows: 12.4 and 11.1).  Many rows: 4, and 8 where that still gives every
// place for a CTA four of them (32768 rows written and read in bf16 282 us against
// 300, 10700 rows written 85 against 82).  More where a row's heads of one kind (at
// most `kind`) are fewer than the lane groups that it would get (32768 rows of one
// head and one cache head of 32 channels: 57 us at 4 rows a CTA, 17 at 32).
struct RowSplit {
    int rows_per_cta;
    bool few;
};
inline RowSplit split_rows(int rows, int lanes, int heads, int kind) {
    const int groups = kThreads / lanes, most = max_rows_per_cta(lanes);
    RowSplit s = {1, static_cast<long long>(rows) * heads * lanes <= 2048LL * sm_count()};
    const int many = rows >= 8 * 16 * sm_count() ? 8 : 4;
    if (!s.few) s.rows_per_cta = most < many ? most : many;
    while (s.rows_per_cta < most && groups / s.rows_per_cta / 2 >= (s.few ? heads : kind)) s.rows_per_cta *= 2;
    return s;
}

template <typename Act, int D, bool kE4m3>
kda_status append_d(AppendParams &p, int rows, cudaStream_t stream) {
    const int heads = p.hq + 2 * p.hkv;
    constexpr int lanes = D / Vec<Act>::N;
    const RowSplit split = split_rows(rows, lanes, heads, p.hq > p.hkv ? p.hq : p.hkv);
    p.rows_per_cta = split.rows_per_cta;
    p.heads_per_cta = split.few ? kThreads / lanes / split.rows_per_cta : heads;
    const dim3 grid(unsigned((rows + p.rows_per_cta - 1) / p.rows_per_cta),
                    unsigned((heads + p.heads_per_cta - 1) / p.heads_per_cta));
    auto kern = p.half_rot == 0   ? kv_append_kernel<Act, D, kE4m3, kNoRot>
                : p.interleaved ? kv_append_kernel<Act, D, kE4m3, kPairs>
                                : kv_append_kernel<Act, D, kE4m3, kHalves>;
    const ProfScope prof(KDA_KERNEL_KV_APPEND, stream);
    return launch_overlapped(kern, grid, kThreads, 0, stream, p);
}

template <typename Act, int D, bool kE4m3>
kda_status read_d(ReadParams &p, int rows, cudaStream_t stream) {
    constexpr int lanes = D / (kE4m3 ? 16 : Vec<Act>::N);
    p.rows_per_cta = split_rows(rows, lanes, 2 * p.hkv, 2 * p.hkv).rows_per_cta;
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
    static std::atomic<int> cached[64] = {};  // calls may come from several threads
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        cudaGetLastError();
        return 152;
    }
    int sms = cached[dev].load(std::memory_order_relaxed);
    if (sms == 0 && cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess)
        cached[dev].store(sms, std::memory_order_relaxed);
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
        for (int i = 0; i < p.half_rot; ++i) p.turn[i] = turn_of(qp->inv_freq[i]);
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
