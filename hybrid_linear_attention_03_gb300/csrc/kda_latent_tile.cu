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
// four warps meet and scale O); until then a tile costs one vote.  The weights, bf16,
// take the place of the tile's shared key part, which the scores have used by then.
//
// A tile comes, is multiplied and leaves in parts of 128 channels, each with barriers of
// its own: shared memory holds two tiles, and in whole ones the copies would wait
// for the products and the products for the copies.
//
// Warps: 0-3 softmax (two threads a row, later a thread a channel) and the rows of Q, 4
// issues the scores, 5 fetches pages by TMA, 6 issues the outputs (a warp of its own, so that
// neither product waits for what the other needs).
//
// e4m3 pages: eight more warps make one bf16 tile of the latents, scale included and
// exact, a part at a time as the outputs of the tile before give its place back.
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
constexpr int kBlock = 64 * 128;      // 64 rows of 64 channels, bf16, swizzled over 128 bytes
constexpr float kRefSlack = 8.f;

template <int L, bool kE4m3> struct Cfg {
    static constexpr int NB = L / 64, MT = L / 128;  // blocks of a latent, its parts of 128 channels (matrix rows of O^T)
    // e4m3: eight warps that widen, and registers split by groups of four warps
    static constexpr int kWiden = 8, kThreads = kE4m3 ? 512 : 224, kLaunch = 128, kSoftmax = 200, kOther = 104;
    static_assert(kSoftmax + 3 * kOther <= 4 * kLaunch, "the split takes no more than the launch has");
    static constexpr int kQBytes = (NB + 1) * kBlock;
    static constexpr int kWide = kE4m3 ? NB * kBlock : 0;  // e4m3: one tile of latents as bf16
    static constexpr int kPart = kE4m3 ? kBlock : 2 * kBlock;  // 128 channels of a tile as they come
    static constexpr int kKrAt = MT * kPart, kStage = kKrAt + kBlock;  // the shared key part, later the weights
    static constexpr int kRoom = 232448 - 1024 - 4096 - kQBytes - kWide;
    static constexpr int kStages = kRoom / kStage < 6 ? kRoom / kStage : 6;
    static constexpr int kWideAt = kQBytes, kRingAt = kWideAt + kWide, kMiscAt = kRingAt + kStages * kStage;
    static constexpr int kColumns = L == 512 ? 512 : 256;  // tensor memory: scores by tile parity, O
    static_assert(2 * KL + MT * BM <= kColumns && kStages >= 2, "room for two tiles");
};

struct alignas(16) Misc {
    uint64_t full[6][5], empty[6][5];            // by stage, the parts of the latents and the shared key parts
    uint64_t wide_full[4], wide_free[4];         // e4m3, by part
    uint64_t s_full[2], p_ready[2], o_done[2];   // by tile parity
    uint64_t q_full, done[2];
    uint32_t tmem;
    int has;
    Cursor piece[2];
    alignas(16) float back[BM], inv[BM];  // what a move of the reference scales O by; an item's end: the rows' factors
    long long out_at[BM];                 // element offsets of the rows in out
    alignas(16) uint8_t scale[6][KL];     // e4m3, by stage: the keys' scale exponents
};

struct LatentMaps {
    CUtensorMap c, kr;
};

// Lane l < 16 gets row l's columns [c, c + 32), lane l + 16 its columns [c + 32, c + 64), of the 16 rows a warp's
// quarter of tensor memory holds of a product of 64.
__device__ __forceinline__ void tmem_ld_rows16(uint32_t taddr, float (&v)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.16x32bx2.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32], 32;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
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

// Barriers of the hardware's: 1 the votes, 2 the meetings of the 128 softmax threads.
__device__ __forceinline__ bool any_of_128(bool mine) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(uint32_t(mine))
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

// Asks for the rows of Q (16-byte copies; rows past the item's, up to a warp's 16, are zeros).
template <int L>
__device__ __forceinline__ void ask_q(const LatentParams &p, const Item &it, unsigned char *q_img, int tid) {
    const int c = tid & 7;
    const bool in = c * 8 < p.rope;
#pragma unroll 1
    for (int r = tid >> 3; r < ((it.rows + 15) & ~15); r += 16) {
        long long row, head;
        p.locate(it, min(r, it.rows - 1), row, head);
        const bool there = r < it.rows;
        const __nv_bfloat16 *a = static_cast<const __nv_bfloat16 *>(p.q_a) + row * p.qa_stride + head * p.qa_head + c * 8;
        const __nv_bfloat16 *b = static_cast<const __nv_bfloat16 *>(p.q_r) + row * p.qr_stride + head * p.qr_head;
        unsigned char *dst = q_img + sw128_chunk(r, c, 64);
#pragma unroll
        for (int k = 0; k < L / 64; ++k) cp_async16_or_zero(dst + k * kBlock, a + k * 64, there);
        cp_async16_or_zero(dst + (L / 64) * kBlock, b + (in ? c * 8 : 0), there && in);
    }
}

// 16 e4m3 values times 2^(e - 127) as bf16, exactly.  Their sign, exponent and fraction in the places of a bf16's
// are the value times 2^-120 (below e4m3's normal range too), so a packed product makes two.  NaN and factors past
// bf16's range go by way of f16 and 32 bits.
__device__ __forceinline__ void widen_bits(const uint4 &q, uint32_t e, uint32_t (&o)[8]) {
    if (nan_codes(q) != 0 || e > 134) {
        widen_e4m3(q, exp2_biased(int(e)), o);
        return;
    }
    const uint32_t f = (e + 120) << 7 | (e + 120) << 23, in[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t t = __byte_perm(in[i / 2], 0, i & 1 ? 0x3424 : 0x1404);
        const uint32_t v = (t >> 4 & 0x07f007f0u) | (t & 0x80008000u);
        const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&v), *reinterpret_cast<const __nv_bfloat162 *>(&f));
        o[i] = *reinterpret_cast<const uint32_t *>(&y);
    }
}

// A tile in which some row does not see some key: zeroes the latents of absent keys and the non-finite ones that
// not every row sees.  Two threads a key.
template <int L>
__device__ __noinline__ void look_over(const Item &it, int kb, uint32_t absent, unsigned char *tile, int tid) {
    const int key = tid >> 1, j = kb + key, half = tid & 1;
    const bool gone = j >= it.k1 || (absent >> (key / 16) & 1);
    unsigned char *img = tile + key * 128;
    auto piece = [&](int c) { return reinterpret_cast<uint4 *>(img + (c >> 3) * kBlock + (((c & 7) ^ (key & 7)) << 4)); };
    bool bad = false;
    if (!gone && j > it.ctx + it.tok0)
        for (int c = half; c < L / 8; c += 2) bad |= odd_bf16(*piece(c));
    bad |= __shfl_xor_sync(0xffffffffu, bad, 1);
    if (gone || bad)
        for (int c = half; c < L / 8; c += 2) *piece(c) = make_uint4(0, 0, 0, 0);
}

template <int L, bool kE4m3>
__global__ void __launch_bounds__(Cfg<L, kE4m3>::kThreads, 1)
    latent_tile_kernel(const __grid_constant__ LatentParams p, const __grid_constant__ LatentMaps maps) {
    using C = Cfg<L, kE4m3>;
    constexpr int NS = C::kStages, MT = C::MT;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Misc &ms = *reinterpret_cast<Misc *>(smem + C::kMiscAt);
    unsigned char *ring = smem + C::kRingAt, *wide = smem + C::kWideAt;
    const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5, cta = int(blockIdx.x);

    if (tid == 0) {
        for (int i = 0; i < NS; ++i)
            for (int c = 0; c <= MT; ++c)
                mbar_init(&ms.full[i][c], 1), mbar_init(&ms.empty[i][c], kE4m3 && c < MT ? C::kWiden / MT : 1);
        for (int c = 0; c < MT; ++c) mbar_init(&ms.wide_full[c], C::kWiden / MT), mbar_init(&ms.wide_free[c], 1);
        for (int i = 0; i < 2; ++i) mbar_init(&ms.s_full[i], 1), mbar_init(&ms.p_ready[i], 4), mbar_init(&ms.o_done[i], 1);
        mbar_init(&ms.q_full, 4), mbar_init(&ms.done[0], 1), mbar_init(&ms.done[1], 1);
        fence_mbar_init();
    }
    if (tid == 32) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.c) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.kr) : "memory");
    }
    if (warp == 4) tmem_alloc(&ms.tmem, C::kColumns);
    wait_prior_kernel();
    allow_next_kernel();
    if (tid < 2) p.parts[2 * cta + tid].state = 0;
    if (warp == 5) {
        Cursor a, z;
        const bool has = find_piece(p, cta, int(gridDim.x), lane, a, z);
        if (lane == 0) ms.piece[0] = a, ms.piece[1] = z, ms.has = has;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = ms.tmem, tm_o = tm + 2 * KL;
    uint32_t *err = p.b.err;
    bool ok = true;  // of this thread's waits

    if (warp < 4) {
        if constexpr (kE4m3) set_regs<C::kSoftmax, C::kLaunch>();
        // ---- softmax: two threads a row, 32 keys each; for O: thread = channel of each 128 ----
        const int row = 16 * warp + (lane & 15), key0 = (lane >> 4) * 32;
        const uint32_t lanes = uint32_t(warp * 32) << 16;
        ItemWalk walk(ms.piece[0], ms.piece[1]);
        Item it = {};
        uint32_t tile = 0;
        auto put_q = [&] {
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
        if (more) ask_q<L>(p, it, smem, tid), put_q();
        while (more) {
            const int nt = tiles_of(it), n_cols = (it.rows + 15) & ~15;
            const bool live = 16 * warp < it.rows;  // this warp has rows of the item
            const int lim = it.ctx + it.tok0 + p.token_of(min(row, it.rows - 1));  // last key the row sees
            float ref = -INFINITY, l = 0.f;
            int page = peek_page(p, it, it.k0, lane);
            for (int v = 0; v < nt; ++v, ++tile) {
                const int kb = it.k0 + v * KL;
                const uint32_t absent = __ballot_sync(0xffffffffu, uint32_t(page) >= uint32_t(p.b.num_pages));
                const bool check = absent != 0 || kb + KL - 1 > it.ctx + it.tok0;  // some row does not see some key
                page = peek_page(p, it, kb + KL, lane);
                unsigned char *stage = ring + tile % NS * C::kStage;
                wait_for(ok, &ms.s_full[tile & 1], (tile >> 1) & 1, err);
                __syncwarp();
                tc_fence_after();
                float x[32];
                bool move = false;
                float top = -INFINITY;
                if (live) {
                    tmem_ld_rows16(tm + lanes + (tile & 1) * KL, x);
                    tmem_wait_ld();
                    if (check) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const int j = kb + key0 + i;
                            if (j > lim || j >= it.k1 || (absent >> ((key0 + i) / 16) & 1)) x[i] = -INFINITY;
                        }
                    }
                    float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                    for (int i = 4; i < 32; i += 4)
#pragma unroll
                        for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], x[i + e]);
                    top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                    move = top > ref + kRefSlack;
                }
                if (any_of_128(move)) {
                    const float f = move ? ex2(ref - top) : 1.f;
                    if (live && lane < 16) ms.back[row] = f;
                    if (move) ref = top, l *= f;
                    named_sync<2, 128>();
                    if (v > 0) {
                        wait_o(tile - 1);
#pragma unroll 1
                        for (int c = 0; c < n_cols; c += 16) {
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
                    const float2 sc = make_float2(p.scale_log2, p.scale_log2), sh = make_float2(-base, -base);
                    float2 sum = make_float2(0.f, 0.f);
                    unsigned char *p_row = stage + C::kKrAt + row * 128;
#pragma unroll
                    for (int i = 0; i < 32; i += 8) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float2 t = fma2(make_float2(x[i + 2 * e], x[i + 2 * e + 1]), sc, sh);
                            t.x = ex2(t.x), t.y = ex2(t.y);
                            sum = add2(sum, t);
                            w[e] = pack_bf16(t.x, t.y);
                        }
                        *reinterpret_cast<uint4 *>(p_row + ((((key0 + i) >> 3) ^ (row & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    l += sum.x + sum.y;
                }
                if (check) {
                    const Item copy = it;
                    look_over<L>(copy, kb, absent, kE4m3 ? wide : stage, tid);
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (ok && lane == 0) mbar_arrive(&ms.p_ready[tile & 1]);
            }
            l += __shfl_xor_sync(0xffffffffu, l, 16);
            // the item's scores are all there, so the rows of the next may take the place of its own
            const Item was = it;
            more = walk.next(p, it);
            if (more) ask_q<L>(p, it, smem, tid);

            // ---- output -----------------------------------------------------------------
            const bool whole = was.whole();
            float *data = p.part_data + (size_t(cta) * 2 + was.slot()) * size_t(BM) * (L + 2);
            if (live && lane < 16) {
                ms.inv[row] = !whole ? 1.f : l > 0.f || l != l ? 1.0f / l : 0.f;
                if (row < was.rows) {
                    long long token, head;
                    p.locate(was, row, token, head);
                    ms.out_at[row] = token * p.out_stride + head * p.out_head;
                    if (!whole) data[BM * L + row] = ref, data[BM * L + BM + row] = l;
                }
            }
            if (!whole && tid == 0) p.parts[2 * cta + was.slot()] = was.part();
            wait_o(tile - 1);
            named_sync<2, 128>();
            if (more) put_q();
            // a thread gets 16 rows of its channel; four neighbours swap them for four channels of a row each
            const int ch0 = warp * 32 + (lane & ~3);
#pragma unroll 1
            for (int c = 0; c < n_cols; c += 16) {
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
                        if (whole) {
                            const float f = ms.inv[r];
                            __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out) + ms.out_at[r] + ch0;
#pragma unroll
                            for (int m = 0; m < MT; ++m)
                                *reinterpret_cast<uint2 *>(dst + m * 128) = make_uint2(
                                    pack_bf16(o[m][g] * f, o[m][g + 1] * f), pack_bf16(o[m][g + 2] * f, o[m][g + 3] * f));
                        } else {
#pragma unroll
                            for (int m = 0; m < MT; ++m)
                                *reinterpret_cast<float4 *>(data + size_t(r) * L + ch0 + m * 128) =
                                    make_float4(o[m][g], o[m][g + 1], o[m][g + 2], o[m][g + 3]);
                        }
                    }
                    __syncwarp();
                }
            }
            tc_fence_before();  // the next item's products rewrite O
            named_sync<2, 128>();  // and its end the rows' factors and places
        }
    } else if (kE4m3 && warp >= 8) {
        // ---- latents made bf16, scale included and exact: a warp has some keys of one part; 8 neighbouring lanes take
        // the same 16-byte piece of 8 keys, which both tiles' swizzles put into different banks ------
        if constexpr (kE4m3) set_regs<C::kOther, C::kLaunch>();
        const int c = (warp - 8) % MT, key = (warp - 8) / MT * (8 * MT) + (lane & 7), pc = lane >> 3;
        unsigned char *to = wide + 2 * c * kBlock + key * 128;
        ItemWalk walk(ms.piece[0], ms.piece[1]);
        Item it = {};
        uint32_t t = 0;
        while (ok && ms.has && walk.next(p, it)) {
            for (int v = tiles_of(it); v > 0 && ok; --v, ++t) {
                const uint32_t s = t % NS;
                if (c > 0) wait_for(ok, &ms.full[s][0], (t / NS) & 1, err);  // the scales
                wait_for(ok, &ms.full[s][c], (t / NS) & 1, err);
                __syncwarp();
                const unsigned char *raw = ring + s * C::kStage + c * kBlock;
                uint4 x[MT][2];
                uint32_t e[MT];
#pragma unroll
                for (int g = 0; g < MT; ++g) {
                    e[g] = ms.scale[s][key + 8 * g];
#pragma unroll
                    for (int u = 0; u < 2; ++u)
                        x[g][u] = *reinterpret_cast<const uint4 *>(raw + row8_piece<128>(key + 8 * g, pc + 4 * u));
                }
                if (t > 0) wait_for(ok, &ms.wide_free[c], (t - 1) & 1, err);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
#pragma unroll
                for (int g = 0; g < MT; ++g)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {  // pieces 0-3 are the first 64 channels
                        uint32_t o[8];
                        widen_bits(x[g][u], e[g], o);
                        unsigned char *at = to + u * kBlock + g * 1024;
                        *reinterpret_cast<uint4 *>(at + (((2 * pc) ^ (key & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                        *reinterpret_cast<uint4 *>(at + (((2 * pc + 1) ^ (key & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
                    }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ms.wide_full[c]), mbar_arrive(&ms.empty[s][c]);
            }
        }
    } else {
        if constexpr (kE4m3) set_regs<C::kOther, C::kLaunch>();
        if (!ms.has) {
        } else if (warp == 4) {
            // ---- scores (converged warp, one lane issues; descriptors count 16-byte units) -------
            const uint32_t id_s = idesc_bf16_f32(64, KL);
            const uint32_t q_desc = desc_k(smem_u32(smem)), k_desc = desc_k(smem_u32(kE4m3 ? wide : ring));
            const uint32_t kr_desc = desc_k(smem_u32(ring + C::kKrAt));
            ItemWalk walk(ms.piece[0], ms.piece[1]);
            Item it = {};
            uint32_t t = 0, n_q = 0;
            while (ok && walk.next(p, it)) {
                wait_for(ok, &ms.q_full, n_q++ & 1, err);
                for (int v = tiles_of(it); v > 0 && ok; --v, ++t) {
                    const uint32_t s = t % NS;
                    // The scores before in this place have been read, and their product is done: so whoever sees
                    // the scores of tile t knows that o_done is at most a tile behind.
                    if (t >= 2) wait_for(ok, &ms.o_done[t & 1], ((t >> 1) - 1) & 1, err);
                    const uint32_t stage = s * uint32_t(C::kStage >> 4), kd = k_desc + (kE4m3 ? 0 : stage), krd = kr_desc + stage;
#pragma unroll
                    for (int c = 0; c <= MT; ++c) {
                        if (kE4m3 && c < MT) wait_for(ok, &ms.wide_full[c], t & 1, err);
                        else wait_for(ok, &ms.full[s][c], (t / NS) & 1, err);
                        ok = __all_sync(0xffffffffu, ok);
                        tc_fence_after();
                        if (ok && elect_one()) {
#pragma unroll
                            for (int k = 0; k < (c < MT ? 8 : 4); ++k) {
                                const uint32_t in = uint32_t((k >> 2) * (kBlock >> 4) + (k & 3) * 2), at = in + c * (2 * kBlock >> 4);
                                mma_lo(tm + (t & 1) * KL, q_desc + at, c < MT ? kd + at : krd + in, id_s, c > 0 || k > 0);
                            }
                            if (c == MT) mma_commit(&ms.s_full[t & 1]);
                        }
                        __syncwarp();
                    }
                }
            }
            // nothing of this CTA's is in flight when its tensor memory goes
            if (elect_one()) mma_commit(&ms.done[0]);
            __syncwarp();
            mbar_wait(&ms.done[0], 0, err);
        } else if (warp == 6) {
            // ---- outputs, likewise ------------------------------------------------------------
            const uint32_t v_desc = desc_mn(smem_u32(kE4m3 ? wide : ring), kBlock), p_desc = desc_k(smem_u32(ring + C::kKrAt));
            ItemWalk walk(ms.piece[0], ms.piece[1]);
            Item it = {};
            uint32_t t = 0;
            while (ok && walk.next(p, it)) {
                const int nt = tiles_of(it);
                const uint32_t id_o = idesc_bf16_f32(128, (it.rows + 15) & ~15, true, false);
                for (int v = 0; v < nt && ok; ++v, ++t) {
                    const uint32_t s = t % NS;
                    wait_for(ok, &ms.p_ready[t & 1], (t >> 1) & 1, err);
                    if (!(ok = __all_sync(0xffffffffu, ok))) break;
                    tc_fence_after();
                    if (elect_one()) {
                        const uint32_t stage = s * uint32_t(C::kStage >> 4), vd = v_desc + (kE4m3 ? 0 : stage), pd = p_desc + stage;
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
#pragma unroll
                            for (int k = 0; k < KL / 16; ++k)
                                mma_lo(tm_o + uint32_t(m * BM), vd + uint32_t(m * 2 * (kBlock >> 4) + k * 128), pd + uint32_t(k * 2),
                                       id_o, k > 0 || v > 0);
                            mma_commit(kE4m3 ? &ms.wide_free[m] : &ms.empty[s][m]);
                        }
                        mma_commit(&ms.o_done[t & 1]);
                        mma_commit(&ms.empty[s][MT]);
                    }
                    __syncwarp();
                }
            }
            if (elect_one()) mma_commit(&ms.done[1]);
            __syncwarp();
            mbar_wait(&ms.done[1], 0, err);
        } else if (warp == 5) {
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
                            mbar_arrive_expect_tx(&ms.full[s][c], there * uint32_t(box * ((two ? 256 : 128) + (kE4m3 && c == 0 ? 1 : 0))));
                        ++asked;
                        __syncwarp();
                        if (i < KL / box && pg >= 0) {
                            unsigned char *to = dst + c * C::kPart + b * kBlock + i * box * 128;
                            if (c < MT) tma_load_3d(to, &maps.c, &ms.full[s][c], c * 128 + b * 64, line, pg);
                            else tma_load_3d(to, &maps.kr, &ms.full[s][c], 0, line, pg);
                            if (kE4m3 && c == 0)
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
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 4) tmem_dealloc(tm, C::kColumns);
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
    p.item_cost = 2 * KL;
    p.min_keys = 2 * KL;
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
