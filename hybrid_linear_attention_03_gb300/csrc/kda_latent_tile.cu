// kda_latent_tile.cu -- kda_latent_attend for bf16 rows on the tensor cores.
//
// All heads share a key, and a key's first L channels are its value, so a tile of 64
// keys lands in shared memory once and is read twice by the tensor cores: as it is for
// the scores and, channels for rows, for the outputs,
//   X = Q K^T  (64 rows x 64 keys, L + 64 channels),   O^T += C^T P^T  (L channels x rows).
// Turned like that, O of 64 rows takes half of tensor memory (L / 128 times 64 columns);
// the other way round 64 rows would take all of it and leave the scores no place.
// Softmax in one pass as in kda_attend_tile.cu: a row's reference is its maximum at
// the time it was last moved, and only moves when a score exceeds it by more than 8 (then the
// eight warps meet and scale O); until then a tile costs one vote.  The weights, bf16,
// take the place of the tile's shared key part, which the scores have used by then.
//
// A tile comes, is multiplied and leaves in parts of 128 channels, each with barriers of
// its own: shared memory holds two tiles of 512 channels, and in whole ones the copies would wait
// for the products and the products for the copies.
//
// Warps: eight for the softmax, then one that issues the scores, one that fetches pages by TMA, and
// one that issues the outputs (so that neither product waits for what the other needs).  In
// the softmax four threads share a row; for O a thread is a channel.
//
// e4m3 pages go to both products as they are.  The scores take them against Q as the sum of two e4m3 terms,
// 2^e (q1 + q2) (exact to about 2^-18 of a row's largest value), beside those of the bf16 key parts; the outputs
// against the weights as three e5m2 terms, p1 + p2 + p3, each what the ones before leave: off by
// (1/9)^3 after the 2^-11 of the f16 they are split from, together less than the 2^-8 of bf16 weights, and
// e5m2 reaches down to 2^-22 of the largest weight where e4m3 would end at 2^-18.  The
// keys' scales (one more warp makes numbers of them) multiply the scores, and the weights before they are split,
// in units that follow the largest scale a row has met.  Eight more warps bring and split the rows of
// Q.  (Latents widened to f16 for the outputs: 64 verifies of 8 tokens 715 us against 434; to bf16, 835:
// two tiles and a wide one fill shared memory, and one tile's widening, products and copies wait in turn.)
// For latents of 512 over e4m3 pages, 144 registers of a softmax thread are 48 bytes too few (spilled, 88 read back).
//
// What bounds it (latents of 512, pages of 64): single tokens, the cache's bytes: 64 sequences of 4001
// to 16384 tokens at 64 heads take 144 us, 5.3 TB/s.  Verifies in e4m3, the reads of shared memory:
// a product of 64 x 64 scores reads 4 KB in its 32.5 cycles and one of 128 channels 6 KB in 48.5 (measured), 2330 cycles
// a tile and 320 for its copy; a tile takes 2900.  One sequence of 4096 tokens: 16 us, of them
// 3.5 before the first page is asked for and 3.5 for writing the parts.
//
// A latent behind a row's position weighs nothing, but 0 * NaN is NaN in the product.
// So in the few tiles where some row does not see some key, the softmax warps zero the
// latents of absent keys and the non-finite ones that not every row sees, once the scores
// are there: a row that does see such a key has NaN for its weight, which is what
// remains (or 0, for a score of -inf).
#include "kda_latent_tc.cuh"

namespace kda {
namespace kv {
namespace {

constexpr int KL = 64, BM = 64;       // keys of a tile, rows of an item
constexpr int kSoftThreads = 256, kFirst = kSoftThreads / 32;  // two groups of four softmax warps; the first warp behind them
constexpr int kBlock = 64 * 128;      // 64 rows of 64 channels, bf16, swizzled over 128 bytes
constexpr float kRefSlack = 8.f;
// e4m3: weights (up to 2^8) times scales (up to p_unit) are split in units of p_unit / 2^7: no more than 2^15, and what the
// last term leaves below its normal range, 2^-17, no more than 2^-22 of the largest scale's whole weight (p_unit is up to four
// times that scale).
constexpr float kPUnits = 128.f, kLeastUnit = 0x1p-120f;  // kPUnits / p_unit stays finite

template <int L, bool kE4m3> struct Cfg {
    static constexpr int NB = L / 64, MT = L / 128;  // blocks of a latent, its parts of 128 channels (matrix rows of O^T)
    // e4m3: eight more warps, that bring the rows of Q, and registers split by four warps
    static constexpr int kRowWarps = 8;
    static constexpr int kThreads = kSoftThreads + (kE4m3 ? 128 + 32 * kRowWarps : 96), kLaunch = 96, kSoftmax = 144, kOther = 64;
    static_assert(2 * kSoftmax + 3 * kOther <= 5 * kLaunch, "the split takes no more than the launch has");
    static constexpr int kQBytes = (NB + 1) * kBlock;
    static constexpr int kThird = kE4m3 ? kBlock : 0;  // e4m3: the weights' third terms, of two tiles
    static constexpr int kPart = kE4m3 ? kBlock : 2 * kBlock;  // 128 channels of a tile as they come
    static constexpr int kKrAt = MT * kPart, kStage = kKrAt + kBlock;  // the shared key part, later the weights
    static constexpr int kRoom = 232448 - 1024 - 4096 - kQBytes - kThird;
    static constexpr int kStages = kRoom / kStage < 6 ? kRoom / kStage : 6;
    static constexpr int kThirdAt = kQBytes, kRingAt = kThirdAt + kThird, kMiscAt = kRingAt + kStages * kStage;
    // tensor memory: scores by tile parity (e4m3: of the latents, of the key parts), O
    static constexpr int kScores = kE4m3 ? 2 * KL : KL, kOAt = 2 * kScores, kColumns = kOAt + MT * BM > 256 ? 512 : 256;
    static_assert(kOAt + MT * BM <= kColumns && kStages >= 2, "room for two tiles");
};

struct alignas(16) Misc {
    uint64_t full[6][5], empty[6][5];            // by stage, the parts of the latents and the shared key parts
    uint64_t unit_full[2];                       // by tile parity: the scales are numbers
    uint64_t s_full[2], p_ready[2], o_done[2];   // by tile parity
    uint64_t q_full, q_free, done[2];            // q_free (e4m3): an item's scores are there
    uint32_t tmem;
    int has;
    Cursor piece[2];
    alignas(16) float back[BM], inv[BM];  // what a move of the reference scales O by; an item's end: the rows' factors
    long long out_at[BM];                 // element offsets of the rows in out, -1 for one of no head
    alignas(16) uint8_t scale[6][KL];     // e4m3, by stage: the keys' scale exponents
    alignas(16) float unit[2][KL];        // by tile parity: the scales
    float unit_top[2];                    // and the largest of them
    float q_unit[4][BM];                  // by item: the rows' scales
    float top[2][BM], scale_top[2][BM], sum[BM];  // what the two groups of softmax warps tell one another of a row
    uint64_t rows_full[4];                // and that they are there
};

struct LatentMaps {
    CUtensorMap c, kr;
};

// Instruction descriptor as idesc_e4m3_f32, of A e4m3 with its rows' values apart (a_mn of idesc_bf16_f32) and B e5m2.
constexpr uint32_t idesc_e4m3_e5m2_f32(int M, int N) {
    return (1u << 4) | (1u << 10) | (1u << 15) | (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24);
}
// Two numbers as the sums of three e5m2 terms each (the first of a pair in the low byte).
__device__ __forceinline__ void split_e5m2(float lo, float hi, uint32_t (&o)[3]) {
    __half2 r = __floats2half2_rn(lo, hi);
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        o[i] = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(r), __NV_SATFINITE, __NV_E5M2);
        const uint32_t back = __byte_perm(o[i], 0, 0x1404);  // an e5m2 value is the upper byte of the same f16 value
        if (i < 2) r = __hsub2(r, *reinterpret_cast<const __half2 *>(&back));
    }
}

// Lane l < 16 gets row l's columns [c, c + 16), lane l + 16 its columns [c + 32, c + 48), of the 16 rows a warp's
// quarter of tensor memory holds of a product of 64.
__device__ __forceinline__ void tmem_ld_rows16(uint32_t taddr, float (&v)[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.16x32bx2.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16], 32;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// Four neighbouring lanes hold four values each: lane i of them gets everyone's i-th, in the order of the lanes.
__device__ __forceinline__ void swap_4x4(float &a, float &b, float &c, float &d, int lane) {
    auto swap = [&](float &x, float &y, int bit) {  // the lower lane's y for the upper one's x
        const float t = __shfl_xor_sync(0xffffffffu, lane & bit ? x : y, bit);
        if (lane & bit) x = t;
        else y = t;
    };
    swap(a, b, 1), swap(c, d, 1), swap(a, c, 2), swap(b, d, 2);
}

// Barriers of the hardware's: 1 the votes, 2 the meetings of the softmax threads.
template <int kThreads>
__device__ __forceinline__ bool any_of(bool mine) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(uint32_t(mine)), "n"(kThreads)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ int tiles_of(const Item &it) { return (it.k1 - it.k0 + KL - 1) / KL; }
// The table's entry for keys [kb + 16 lane, kb + 16 lane + 16) of the tile at kb (page 0 where there are none),
// asked for a tile ahead.
__device__ __forceinline__ int peek_page(const LatentParams &p, const Item &it, int kb, int lane) {
    const int j = kb + lane * 16;
    if (lane >= KL / 16 || j >= it.k1) return 0;
    return p.b.table[size_t(it.n) * size_t(p.b.table_stride) + size_t(j >> p.b.page_shift)];
}

// Asks for the rows of Q that `threads` threads bring (16-byte copies; rows past the item's, up to a warp's 16, are
// zeros): all of them, or only the part that meets kr.
template <int L, bool kOnlyKr, int kThreads>
__device__ __forceinline__ void ask_q(const LatentParams &p, const Item &it, unsigned char *q_img, int tid) {
    const int c = tid & 7;
    const bool in = c * 8 < p.rope;
#pragma unroll 1
    for (int r = tid >> 3; r < ((it.rows + 15) & ~15); r += kThreads / 8) {
        long long row, head;
        p.locate_head(it, min(r, it.rows - 1), row, head);
        const bool there = r < it.rows;
        const __nv_bfloat16 *b = static_cast<const __nv_bfloat16 *>(p.q_r) + row * p.qr_stride + head * p.qr_head;
        unsigned char *dst = q_img + sw128_chunk(r, c, 64);
        if constexpr (!kOnlyKr) {
            const __nv_bfloat16 *a = static_cast<const __nv_bfloat16 *>(p.q_a) + row * p.qa_stride + head * p.qa_head + c * 8;
#pragma unroll
            for (int k = 0; k < L / 64; ++k) cp_async16_or_zero(dst + k * kBlock, a + k * 64, there);
        }
        cp_async16_or_zero(dst + (L / 64) * kBlock, b + (in ? c * 8 : 0), there && in);
    }
}
// e4m3 pages: rows [r0, r0 + 8) of Q, one warp: those for the latents as 2^e (q1 + q2), two e4m3 terms, as in
// kda_attend_tile.cu.
template <int L>
__device__ __forceinline__ void split_q(const LatentParams &p, const Item &it, unsigned char *q_img, float *q_unit, int r0, int lane) {
    constexpr int kPieces = L / 8 > 32 ? L / 8 / 32 : 1, kB = 2;  // of 16 bytes, of a lane; rows at a time
#pragma unroll 1
    for (int g = 0; g < 8 && r0 + g < it.rows; g += kB) {
        uint4 raw[kB][kPieces];
#pragma unroll
        for (int i = 0; i < kB; ++i) {
            long long row, head;
            p.locate_head(it, min(r0 + g + i, it.rows - 1), row, head);
            const __nv_bfloat16 *a = static_cast<const __nv_bfloat16 *>(p.q_a) + row * p.qa_stride + head * p.qa_head;
#pragma unroll
            for (int k = 0; k < kPieces; ++k) {
                const int at = (lane + 32 * k) * 8;
                raw[i][k] = r0 + g + i < it.rows && at < L ? *reinterpret_cast<const uint4 *>(a + at) : make_uint4(0, 0, 0, 0);
            }
        }
        uint32_t m[kB];  // the largest magnitude as a bf16 pattern
#pragma unroll
        for (int i = 0; i < kB; ++i) {
            m[i] = 0;
#pragma unroll
            for (int k = 0; k < kPieces; ++k) {
                const uint4 &w = raw[i][k];
                const uint32_t t = __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu),
                                            __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
                m[i] = max(m[i], max(t & 0xffffu, t >> 16));
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < kB; ++i) m[i] = max(m[i], __shfl_xor_sync(0xffffffffu, m[i], o));
#pragma unroll
        for (int i = 0; i < kB; ++i) {
            const int e = m[i] >= 0x7f80u ? -1 : max(scale_exponent(__uint_as_float(m[i] << 16)), 1), r = r0 + g + i;
            if (lane == 0) q_unit[r] = exp2_biased(e < 0 ? 127 : e);
#pragma unroll
            for (int k = 0; k < kPieces; ++k) {
                const int pc = lane + 32 * k;  // the row's piece of eight values
                if (pc * 8 >= L) continue;
                uint32_t w1[2], w2[2];
                split_row(raw[i][k], e, w1, w2);
                unsigned char *at = q_img + (pc >> 4) * kBlock + row8_piece<128>(r, (pc & 15) >> 1) + (pc & 1) * 8;
                *reinterpret_cast<uint2 *>(at) = make_uint2(w1[0], w1[1]);
                *reinterpret_cast<uint2 *>(at + (L / 128) * kBlock) = make_uint2(w2[0], w2[1]);
            }
        }
    }
}

// A tile in which some row does not see some key: zeroes the latents of absent keys and the non-finite ones that
// not every row sees.  Four threads a key.
template <int L, bool kE4m3>
__device__ __noinline__ void look_over(const Item &it, int kb, uint32_t absent, unsigned char *tile, int tid) {
    constexpr int kPieces = kE4m3 ? L / 16 : L / 8;  // of 16 bytes, eight of them in a block's row
    constexpr int kEach = kSoftThreads / KL;
    const int key = tid / kEach, j = kb + key, first = tid % kEach;
    const bool gone = j >= it.k1 || (absent >> (key / 16) & 1);
    unsigned char *img = tile + key * 128;
    auto piece = [&](int c) { return reinterpret_cast<uint4 *>(img + (c >> 3) * kBlock + (((c & 7) ^ (key & 7)) << 4)); };
    bool bad = false;
    if (!gone && j > it.ctx + it.tok0)
        for (int c = first; c < kPieces; c += kEach) bad |= kE4m3 ? nan_codes(*piece(c)) != 0 : odd_bf16(*piece(c));
#pragma unroll
    for (int o = 1; o < kEach; o *= 2) bad |= __shfl_xor_sync(0xffffffffu, bad, o);
    if (gone || bad)
        for (int c = first; c < kPieces; c += kEach) *piece(c) = make_uint4(0, 0, 0, 0);
}

template <int L, bool kE4m3>
__global__ void __launch_bounds__(Cfg<L, kE4m3>::kThreads, 1)
    latent_tile_kernel(const __grid_constant__ LatentParams p, const __grid_constant__ LatentMaps maps) {
    using C = Cfg<L, kE4m3>;
    constexpr int NS = C::kStages, MT = C::MT;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Misc &ms = *reinterpret_cast<Misc *>(smem + C::kMiscAt);
    unsigned char *ring = smem + C::kRingAt, *third = smem + C::kThirdAt;
    const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5, cta = int(blockIdx.x);

    if (tid == 0) {
        for (int i = 0; i < NS; ++i)
            for (int c = 0; c <= MT; ++c)
                mbar_init(&ms.full[i][c], 1), mbar_init(&ms.empty[i][c], 1);
        for (int i = 0; i < 2; ++i) mbar_init(&ms.s_full[i], 1), mbar_init(&ms.p_ready[i], kFirst), mbar_init(&ms.o_done[i], 1), mbar_init(&ms.unit_full[i], 1);
        for (int i = 0; i < 4; ++i) mbar_init(&ms.rows_full[i], C::kRowWarps);
        mbar_init(&ms.q_full, kE4m3 ? C::kRowWarps : kFirst), mbar_init(&ms.q_free, 1), mbar_init(&ms.done[0], 1), mbar_init(&ms.done[1], 1);
        fence_mbar_init();
    }
    if (tid == 32) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.c) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.kr) : "memory");
    }
    if (warp == kFirst) tmem_alloc(&ms.tmem, C::kColumns);
    wait_prior_kernel();
    allow_next_kernel();
    if (tid < 2) p.parts[2 * cta + tid].state = 0;
    if (warp == kFirst + 1) {
        Cursor a, z;
        const bool has = find_piece(p, cta, int(gridDim.x), lane, a, z);
        if (lane == 0) ms.piece[0] = a, ms.piece[1] = z, ms.has = has;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = ms.tmem, tm_o = tm + C::kOAt;
    uint32_t *err = p.b.err;
    bool ok = true;  // of this thread's waits

    if (warp < kFirst) {
        if constexpr (kE4m3) set_regs<C::kSoftmax, C::kLaunch>();
        // ---- softmax: four threads a row, 16 keys each; for O: thread = channel of each 128, the groups take 16 rows
        // in turn ----
        constexpr int kKeys = 16;
        const int quarter = warp & 3, group = warp >> 2;
        const int row = 16 * quarter + (lane & 15), key0 = (lane >> 4) * 32 + group * kKeys;
        const uint32_t lanes = uint32_t(quarter * 32) << 16;
        ItemWalk walk(ms.piece[0], ms.piece[1]);
        Item it = {};
        uint32_t tile = 0;
        uint32_t n_it = 0;  // items so far
        auto put_q = [&] {
            if (kE4m3) return;  // others bring them
            cp_async_wait_all();
            fence_proxy_async_smem();
            __syncwarp();
            if (ok && lane == 0) mbar_arrive(&ms.q_full);
        };
        // O holds the product of tile t
        auto wait_o = [&](uint32_t t) {
            wait_for(ok, &ms.o_done[t & 1], (t >> 1) & 1, err);
            __syncwarp();
            tc_fence_after();
        };
        bool more = ms.has && walk.next(p, it);
        auto ask = [&] {
            if constexpr (!kE4m3) ask_q<L, false, kSoftThreads>(p, it, smem, tid);
        };
        if (more) ask(), put_q();
        for (; more; ++n_it) {
            const int nt = tiles_of(it), n_cols = (it.rows + 15) & ~15;
            const bool live = 16 * quarter < it.rows;  // this warp has rows of the item
            const int lim = it.ctx + it.tok0 + p.token_of(min(row, it.rows - 1));  // last key the row sees
            float ref = -INFINITY, l = 0.f;
            // e4m3: what weights times their keys' scales are in units of, before they become f16 (a power of two)
            float p_unit = kLeastUnit, q_unit = 0.f;
            if constexpr (kE4m3) {
                wait_for(ok, &ms.rows_full[n_it & 3], (n_it >> 2) & 1, err);
                __syncwarp();
                q_unit = fmaxf(p.scale_log2 * ms.q_unit[n_it & 3][row], 0x1p-149f);
            }
            int page = peek_page(p, it, it.k0, lane);
            for (int v = 0; v < nt; ++v, ++tile) {
                const int kb = it.k0 + v * KL;
                const uint32_t absent = __ballot_sync(0xffffffffu, uint32_t(page) >= uint32_t(p.b.num_pages));
                const bool check = absent != 0 || kb + KL - 1 > it.ctx + it.tok0;  // some row does not see some key
                page = peek_page(p, it, kb + KL, lane);
                unsigned char *stage = ring + tile % NS * C::kStage;
                wait_for(ok, &ms.s_full[tile & 1], (tile >> 1) & 1, err);
                // (in order, so that no later wait for these barriers is two phases ahead)
                if (tile >= 2) wait_for(ok, &ms.o_done[tile & 1], ((tile >> 1) - 1) & 1, err);
                __syncwarp();
                tc_fence_after();
                float x[kKeys];
                bool move = false;
                float top = -INFINITY, unit_top = 0.f;
                if constexpr (kE4m3) wait_for(ok, &ms.unit_full[tile & 1], (tile >> 1) & 1, err), __syncwarp();
                const float *unit = ms.unit[tile & 1] + key0;
                if (live) {
                    tmem_ld_rows16(tm + lanes + (tile & 1) * C::kScores + group * kKeys, x);
                    if constexpr (kE4m3) {
                        // scores in powers of two: the latents' times their scales, and the key parts'
                        float y[kKeys];
                        tmem_ld_rows16(tm + lanes + (tile & 1) * C::kScores + KL + group * kKeys, y);
                        const float2 f2 = make_float2(q_unit, q_unit), sc = make_float2(p.scale_log2, p.scale_log2);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < kKeys; i += 4) {
                            const float4 u = *reinterpret_cast<const float4 *>(unit + i);
                            const float2 a = fma2(mul2(make_float2(u.x, u.y), f2), make_float2(x[i], x[i + 1]),
                                                  mul2(make_float2(y[i], y[i + 1]), sc));
                            const float2 b = fma2(mul2(make_float2(u.z, u.w), f2), make_float2(x[i + 2], x[i + 3]),
                                                  mul2(make_float2(y[i + 2], y[i + 3]), sc));
                            x[i] = a.x, x[i + 1] = a.y, x[i + 2] = b.x, x[i + 3] = b.y;
                        }
                        if (!check) unit_top = ms.unit_top[tile & 1];
                    } else {
                        tmem_wait_ld();
                    }
                    if (check) {
#pragma unroll
                        for (int i = 0; i < kKeys; ++i) {
                            const int j = kb + key0 + i;
                            if (j > lim || j >= it.k1 || (absent >> ((key0 + i) / 16) & 1)) x[i] = -INFINITY;
                            else if (kE4m3) unit_top = fmaxf(unit_top, unit[i]);
                        }
                    }
                    float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                    for (int i = 4; i < kKeys; i += 4)
#pragma unroll
                        for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], x[i + e]);
                    top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * (kE4m3 ? 1.f : p.scale_log2);
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                    move = top > ref + kRefSlack;
                    if constexpr (kE4m3) {
                        unit_top = fmaxf(unit_top, __shfl_xor_sync(0xffffffffu, unit_top, 16));
                        move = move || unit_top > p_unit;
                    }
                }
                if (any_of<kSoftThreads>(move)) {
                    // the row's maxima over both groups' keys
                    if (lane < 16) ms.top[group][row] = top, ms.scale_top[group][row] = unit_top;
                    named_sync<2, kSoftThreads>();
                    top = fmaxf(top, ms.top[group ^ 1][row]), unit_top = fmaxf(unit_top, ms.scale_top[group ^ 1][row]);
                    const float to = top > ref + kRefSlack ? top : ref;
                    float f = to != ref ? ex2(ref - to) : 1.f;
                    l *= f, ref = to;
                    if constexpr (kE4m3) {
                        // (with room for scales four times as large)
                        const float unit_to = unit_top > p_unit ? fminf(4.f * unit_top, 0x1p127f) : p_unit;
                        f = f * (p_unit / unit_to), p_unit = unit_to;
                    }
                    if (live && lane < 16) ms.back[row] = f;  // (the same number from both groups)
                    named_sync<2, kSoftThreads>();
                    if (v > 0) {
                        wait_o(tile - 1);
#pragma unroll 1
                        for (int c = 16 * group; c < n_cols; c += 32) {
                            float b[16];
#pragma unroll
                            for (int i = 0; i < 16; i += 4) {
                                const float4 t = *reinterpret_cast<const float4 *>(&ms.back[c + i]);
                                b[i] = t.x, b[i + 1] = t.y, b[i + 2] = t.z, b[i + 3] = t.w;
                            }
#pragma unroll
                            for (int m = 0; m < MT; ++m) {
                                float o[16];
                                tmem_ld16(tm_o + lanes + uint32_t(m * BM + c), o);
                                tmem_wait_ld();
#pragma unroll
                                for (int i = 0; i < 16; ++i) o[i] *= b[i];
                                tmem_st16(tm_o + lanes + uint32_t(m * BM + c), o);
                            }
                        }
                        tmem_wait_st();
                    }
                }
                if (live) {
                    const float base = ref == -INFINITY ? 0.f : ref;
                    const float one = kE4m3 ? 1.f : p.scale_log2, per = kE4m3 ? kPUnits / p_unit : 1.f;
                    const float2 sc = make_float2(one, one), sh = make_float2(-base, -base), per2 = make_float2(per, per);
                    float2 sum = make_float2(0.f, 0.f);
                    unsigned char *p_row = stage + C::kKrAt + row * 128;
                    constexpr int kStep = kE4m3 ? 16 : 8;  // keys whose weights, or terms of them, fill 16 bytes
#pragma unroll
                    for (int i = 0; i < kKeys; i += kStep) {
                        uint32_t w[kE4m3 ? 3 : 1][4];
#pragma unroll
                        for (int e = 0; e < kStep / 2; ++e) {
                            float2 t = fma2(make_float2(x[i + 2 * e], x[i + 2 * e + 1]), sc, sh);
                            t.x = ex2(t.x), t.y = ex2(t.y);
                            sum = add2(sum, t);
                            if constexpr (kE4m3) {
                                const float2 u = *reinterpret_cast<const float2 *>(unit + i + 2 * e);
                                const float2 z = mul2(t, mul2(u, per2));
                                // the scale of a key that the row does not see may be anything
                                t = check ? make_float2(t.x == 0.f ? 0.f : z.x, t.y == 0.f ? 0.f : z.y) : z;
                                uint32_t h[3];
                                split_e5m2(t.x, t.y, h);
#pragma unroll
                                for (int k = 0; k < 3; ++k) w[k][e >> 1] = e & 1 ? w[k][e >> 1] | h[k] << 16 : h[k];
                            } else {
                                w[0][e] = pack_bf16(t.x, t.y);
                            }
                        }
                        const int c = (key0 + i) / kStep;  // the piece of 16 bytes
                        auto put = [&](unsigned char *to, int c, const uint32_t (&v)[4]) {
                            *reinterpret_cast<uint4 *>(to + ((c ^ (row & 7)) << 4)) = make_uint4(v[0], v[1], v[2], v[3]);
                        };
                        put(p_row, c, w[0]);
                        if constexpr (kE4m3)
                            put(p_row, 4 + c, w[1]), put(third + row * 128, int(tile & 1) * 4 + c, w[2]);
                    }
                    l += sum.x + sum.y;
                }
                if (check) {
                    const Item copy = it;
                    look_over<L, kE4m3>(copy, kb, absent, stage, tid);
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (ok && lane == 0) mbar_arrive(&ms.p_ready[tile & 1]);
            }
            l += __shfl_xor_sync(0xffffffffu, l, 16);
            if (group == 1 && lane < 16) ms.sum[row] = l;
            named_sync<2, kSoftThreads>();
            l += ms.sum[row];  // (of use to the first group)
            // the item's scores are all there, so the rows of the next may take the place of its own
            const Item was = it;
            more = walk.next(p, it);
            if (more) ask();

            // ---- output -----------------------------------------------------------------
            const bool whole = was.whole();
            float *data = p.part_data + (size_t(cta) * 2 + was.slot()) * size_t(BM) * (L + 2);
            if (live && group == 0 && lane < 16) {
                const float up = kE4m3 ? p_unit / kPUnits : 1.f;
                ms.inv[row] = !whole ? up : l > 0.f || l != l ? up / l : 0.f;
                if (row < was.rows) {
                    long long token, head;
                    const bool there = p.locate_head(was, row, token, head);
                    ms.out_at[row] = there ? token * p.out_stride + head * p.out_head : -1;
                    if (!whole) data[BM * L + row] = ref, data[BM * L + BM + row] = l;
                }
            }
            if (!whole && tid == 0) p.parts[2 * cta + was.slot()] = was.part();
            wait_o(tile - 1);
            named_sync<2, kSoftThreads>();
            if (more) put_q();
            // a thread gets 16 rows of its channel; four neighbours swap them for four channels of a row each
            const int ch0 = quarter * 32 + (lane & ~3);
#pragma unroll 1
            for (int c = 16 * group; c < n_cols; c += 32) {
                float o[MT][16];
#pragma unroll
                for (int m = 0; m < MT; ++m) tmem_ld16(tm_o + lanes + uint32_t(m * BM + c), o[m]);
                tmem_wait_ld();
#pragma unroll
                for (int g = 0; g < 16; g += 4) {
#pragma unroll
                    for (int m = 0; m < MT; ++m) swap_4x4(o[m][g], o[m][g + 1], o[m][g + 2], o[m][g + 3], lane);
                    const int r = c + g + (lane & 3);
                    if (r < was.rows) {
                        const long long at = ms.out_at[r];
                        if (at < 0) {  // a row of no head
                        } else if (whole) {
                            const float f = ms.inv[r];
                            __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out) + at + ch0;
#pragma unroll
                            for (int m = 0; m < MT; ++m)
                                *reinterpret_cast<uint2 *>(dst + m * 128) = make_uint2(
                                    pack_bf16(o[m][g] * f, o[m][g + 1] * f), pack_bf16(o[m][g + 2] * f, o[m][g + 3] * f));
                        } else {
#pragma unroll
                            for (int m = 0; m < MT; ++m) {
                                const float f = kE4m3 ? ms.inv[r] : 1.f;
                                *reinterpret_cast<float4 *>(data + size_t(r) * L + ch0 + m * 128) =
                                    make_float4(o[m][g] * f, o[m][g + 1] * f, o[m][g + 2] * f, o[m][g + 3] * f);
                            }
                        }
                    }
                    __syncwarp();
                }
            }
            tc_fence_before();  // the next item's products rewrite O
            named_sync<2, kSoftThreads>();  // and its end the rows' factors and places
        }
    } else if (kE4m3 && warp >= kFirst + 4) {
        // ---- rows of Q (e4m3), once the last item's scores are there.  Those are at most two tiles
        // ahead of the outputs, so nobody reads the scales of four items before ------------------
        if constexpr (kE4m3) set_regs<C::kOther, C::kLaunch>();
        ItemWalk walk(ms.piece[0], ms.piece[1]);
        Item it = {};
        for (uint32_t n_it = 0; ms.has && walk.next(p, it); ++n_it) {
            if (n_it > 0) wait_for(ok, &ms.q_free, (n_it - 1) & 1, err);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            ask_q<L, true, 32 * C::kRowWarps>(p, it, smem, tid - 32 * (kFirst + 4));
            split_q<L>(p, it, smem, ms.q_unit[n_it & 3], (warp - kFirst - 4) * 8, lane);
            cp_async_wait_all();
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ms.q_full), mbar_arrive(&ms.rows_full[n_it & 3]);
        }
    } else {
        if constexpr (kE4m3) set_regs<C::kOther, C::kLaunch>();
        if (!ms.has) {
        } else if (warp == kFirst) {
            // ---- scores (converged warp, one lane issues; descriptors count 16-byte units) -------
            const uint32_t id_s = idesc_bf16_f32(64, KL), id_8 = idesc_e4m3_f32(64, KL);
            const uint32_t q_desc = desc_k(smem_u32(smem)), k_desc = desc_k(smem_u32(ring));
            ItemWalk walk(ms.piece[0], ms.piece[1]);
            Item it = {};
            uint32_t t = 0, n_q = 0;
            while (ok && walk.next(p, it)) {
                wait_for(ok, &ms.q_full, n_q++ & 1, err);
                ok = __all_sync(0xffffffffu, ok);
                for (int v = tiles_of(it); v > 0 && ok; --v, ++t) {
                    const uint32_t s = t % NS, t_s = tm + (t & 1) * C::kScores;
                    if (t >= 2) wait_for(ok, &ms.p_ready[t & 1], ((t >> 1) - 1) & 1, err);  // those before have been read
                    const uint32_t kd = k_desc + s * uint32_t(C::kStage >> 4);
#pragma unroll
                    for (int c = 0; c <= MT; ++c) {
                        wait_for(ok, &ms.full[s][c], (t / NS) & 1, err);
                        ok = __all_sync(0xffffffffu, ok);
                        tc_fence_after();
                        if (ok && elect_one()) {
                            if (kE4m3 && c < MT) {
#pragma unroll
                                for (int k = 0; k < 8; ++k)  // both terms of Q against the same keys
                                    mma_lo_e4m3(t_s, q_desc + uint32_t((c + k / 4 * MT) * (kBlock >> 4) + (k & 3) * 2),
                                                kd + uint32_t(c * (C::kPart >> 4) + (k & 3) * 2), id_8, c > 0 || k > 0);
                            } else {
#pragma unroll
                                for (int k = 0; k < (c < MT ? 8 : 4); ++k) {
                                    const uint32_t in = uint32_t((k >> 2) * (kBlock >> 4) + (k & 3) * 2);
                                    mma_lo(t_s + (kE4m3 ? KL : 0), q_desc + in + uint32_t(c * (2 * kBlock >> 4)),
                                           kd + in + uint32_t(c * (C::kPart >> 4)), id_s, (!kE4m3 && c > 0) || k > 0);
                                }
                            }
                            if (c == MT) {
                                mma_commit(&ms.s_full[t & 1]);
                                if (kE4m3 && v == 1) mma_commit(&ms.q_free);
                            }
                        }
                        __syncwarp();
                    }
                }
            }
            // nothing of this CTA's is in flight when its tensor memory goes
            if (elect_one()) mma_commit(&ms.done[0]);
            __syncwarp();
            mbar_wait(&ms.done[0], 0, err);
        } else if (warp == kFirst + 2) {
            // ---- outputs, likewise ------------------------------------------------------------
            const uint32_t v_desc = desc_mn(smem_u32(ring), kBlock), p_desc = desc_k(smem_u32(ring + C::kKrAt)), p3_desc = desc_k(smem_u32(third));
            ItemWalk walk(ms.piece[0], ms.piece[1]);
            Item it = {};
            uint32_t t = 0;
            while (ok && walk.next(p, it)) {
                const int nt = tiles_of(it);
                const int cols = (it.rows + 15) & ~15;
                const uint32_t id_o = kE4m3 ? idesc_e4m3_e5m2_f32(128, cols) : idesc_bf16_f32(128, cols, true, false);
                for (int v = 0; v < nt && ok; ++v, ++t) {
                    const uint32_t s = t % NS;
                    wait_for(ok, &ms.p_ready[t & 1], (t >> 1) & 1, err);
                    if (!(ok = __all_sync(0xffffffffu, ok))) break;
                    tc_fence_after();
                    const uint32_t stage = s * uint32_t(C::kStage >> 4), vd = v_desc + stage, pd = p_desc + stage;
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        if (ok && elect_one()) {
                            if constexpr (kE4m3) {
#pragma unroll
                                for (int k = 0; k < 6; ++k)  // 32 keys, a term of their weights
                                    mma_lo_e4m3(tm_o + uint32_t(m * BM), vd + uint32_t(m * (kBlock >> 4) + (k & 1) * 256),
                                                (k < 4 ? pd + uint32_t(k * 2) : p3_desc + (t & 1) * 4 + uint32_t((k & 1) * 2)), id_o,
                                                k > 0 || v > 0);
                            } else {
#pragma unroll
                                for (int k = 0; k < KL / 16; ++k)
                                    mma_lo(tm_o + uint32_t(m * BM), vd + uint32_t(m * 2 * (kBlock >> 4) + k * 128), pd + uint32_t(k * 2),
                                           id_o, k > 0 || v > 0);
                            }
                            mma_commit(&ms.empty[s][m]);
                            if (m + 1 == MT) mma_commit(&ms.o_done[t & 1]), mma_commit(&ms.empty[s][MT]);
                        }
                        __syncwarp();
                    }
                }
            }
            if (elect_one()) mma_commit(&ms.done[1]);
            __syncwarp();
            mbar_wait(&ms.done[1], 0, err);
        } else if (warp == kFirst + 1) {
            // ---- page fetches ------------------------------------------------------------------
            const int page_size = 1 << p.b.page_shift, box = min(page_size, KL);
            ItemWalk walk(ms.piece[0], ms.piece[1]);
            Item it = {};
            uint32_t t = 0, asked = 0;  // tiles, and parts of them asked for
            while (ok && walk.next(p, it)) {
                auto page_at = [&](int kb) {
                    const int j = kb + lane * box;
                    return lane * box < KL && j < it.k1 ? load_page(p.b, it.n, j) : -1;
                };
                int next = page_at(it.k0);
                for (int kb = it.k0; kb < it.k1 && ok; kb += KL, ++t) {
                    const int page = next, line = kb & (page_size - 1);  // a tile starts a box
                    next = page_at(kb + KL);
                    const uint32_t s = t % NS;
                    const uint32_t there = __popc(__ballot_sync(0xffffffffu, page >= 0));
                    unsigned char *dst = ring + s * C::kStage;
                    // a part at a time, as the outputs leave them: a lane a box
                    for (int c = 0; c <= MT; ++c) {
                        const bool two = !kE4m3 && c < MT;  // bf16 latents: a box holds half of a part's channels
                        const int i = two ? lane >> 1 : lane, b = two ? lane & 1 : 0;
                        const int pg = __shfl_sync(0xffffffffu, page, i);
                        if (t >= NS) wait_for(ok, &ms.empty[s][c], (t / NS - 1) & 1, err);
                        if (!(ok = __all_sync(0xffffffffu, ok))) break;
                        if (lane == 0)
                            mbar_arrive_expect_tx(&ms.full[s][c], there * uint32_t(box * ((two ? 256 : 128) + (kE4m3 && c == MT ? 1 : 0))));
                        ++asked;
                        __syncwarp();
                        if (i < KL / box && pg >= 0) {
                            unsigned char *to = dst + c * C::kPart + b * kBlock + i * box * 128;
                            if (c < MT) tma_load_3d(to, &maps.c, &ms.full[s][c], c * 128 + b * 64, line, pg);
                            else tma_load_3d(to, &maps.kr, &ms.full[s][c], 0, line, pg);
                            if (kE4m3 && c == MT)
                                bulk_load(&ms.scale[s][i * box], p.sc + (size_t(pg) << p.b.page_shift) + line, uint32_t(box), &ms.full[s][c]);
                        }
                        __syncwarp();
                    }
                    if (!ok) break;
                }
            }
            // whichever role gives up, no copy is in flight when the CTA ends
            for (uint32_t i = asked - min(asked, uint32_t(NS * (MT + 1))); i < asked; ++i) {
                const uint32_t of = i / (MT + 1);
                mbar_wait(&ms.full[of % NS][i % (MT + 1)], (of / NS) & 1, err);
            }
        } else if (kE4m3 && warp == kFirst + 3) {
            // ---- scales as numbers, and the largest --------------------------------------------
            ItemWalk walk(ms.piece[0], ms.piece[1]);
            Item it = {};
            uint32_t t = 0;
            while (ok && walk.next(p, it)) {
                for (int v = tiles_of(it); v > 0 && ok; --v, ++t) {
                    const uint32_t s = t % NS;
                    if (t >= 2) wait_for(ok, &ms.p_ready[t & 1], ((t >> 1) - 1) & 1, err);  // those before have been used
                    wait_for(ok, &ms.full[s][MT], (t / NS) & 1, err);
                    if (!(ok = __all_sync(0xffffffffu, ok))) break;
                    const float a = exp2_biased(ms.scale[s][lane]), b = exp2_biased(ms.scale[s][lane + 32]);
                    ms.unit[t & 1][lane] = a, ms.unit[t & 1][lane + 32] = b;
                    float top = fmaxf(a, b);
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                    if (lane == 0) ms.unit_top[t & 1] = top;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ms.unit_full[t & 1]);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kFirst) tmem_dealloc(tm, C::kColumns);
}

// [num_pages][page_size][channels]; a box is a tile's part of one page, 64 channels of it (zeros past the last
// one: a shared key part of 16 or 32), swizzled over 128 bytes.
inline bool latent_map(CUtensorMap *m, const void *base, const kda_latent_cache *c, int channels, bool e4m3) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t D = cuuint64_t(channels), P = cuuint64_t(c->page_size), esize = e4m3 ? 1 : 2;
    const cuuint64_t dims[3] = {D, P, cuuint64_t(c->num_pages)};
    const cuuint64_t strides[2] = {D * esize, D * P * esize};
    const cuuint32_t box[3] = {e4m3 ? 128u : 64u, cuuint32_t(c->page_size < KL ? c->page_size : KL), 1u};
    const cuuint32_t estr[3] = {1u, 1u, 1u};
    return fn(m, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int L, bool kE4m3>
kda_status launch(const kda_latent_cache *c, LatentParams &p, const AttendPlan &plan, cudaStream_t stream) {
    using C = Cfg<L, kE4m3>;
    LatentMaps maps;
    if (!latent_map(&maps.c, c->c, c, L, kE4m3) || !latent_map(&maps.kr, c->kr, c, c->rope_dim, false)) return KDA_ERR_CUDA;
    constexpr size_t smem = 1024 + C::kMiscAt + sizeof(Misc);
    static_assert(smem <= 232448, "shared memory of a CTA");
    if (!allow_smem<latent_tile_kernel<L, kE4m3>>(int(smem))) return KDA_ERR_CUDA;
    p.key_step = KL;
    p.item_cost = 8 * KL;  // (64 verifies over e4m3 pages: 440 us with 2 or 3, 432 with 5 to 8, 438 with 12)
    p.min_keys = KL;  // (two tiles or more a CTA: one token over 4096 takes 16.8 us instead of 16.3, four 18.3)
    const ProfScope prof(KDA_KERNEL_LATENT_ATTEND, stream);
    return launch_overlapped(latent_tile_kernel<L, kE4m3>, dim3(unsigned(plan.n_cta)), C::kThreads, smem, stream, p, maps);
}

template <bool kE4m3>
kda_status by_latent(const kda_latent_cache *c, LatentParams &p, const AttendPlan &plan, cudaStream_t stream) {
    switch (c->latent_dim) {
        case 128: return launch<128, kE4m3>(c, p, plan, stream);
        case 256: return launch<256, kE4m3>(c, p, plan, stream);
        case 512: return launch<512, kE4m3>(c, p, plan, stream);
    }
    return KDA_ERR_UNSUPPORTED;
}

}  // namespace

bool latent_tile_plan(const kda_latent_cache *c, AttendPlan *plan) {
    if (c->act != KDA_BF16) return false;
    plan->bm = BM;
    plan->n_cta = sm_count();
    return true;
}

kda_status latent_tile_launch(const kda_latent_cache *c, LatentParams &p, const AttendPlan &plan, cudaStream_t stream) {
    return c->format == KDA_KV_E4M3 ? by_latent<true>(c, p, plan, stream) : by_latent<false>(c, p, plan, stream);
}

}  // namespace kv
}  // namespace kda
