// kda_latent_prefill.cu -- kda_latent_prefill for bf16 rows on the tensor cores.
//
// Per head, scores X = Q K^T over nope_dim channels of its own and up to 64 shared by all
// heads (128 rows x 128 keys a product), one thread a row turns them, 64 at a time, into weights
// P = 2^(scale log2e X - ref) and leaves them as bf16 where the scores were, and
// O += P V reads them from there: the softmax and the sides of kda_attend_tile.cu,
//   sides by rows  (more than 128 tokens a sequence): side s has rows [128 s, 128 s + 128) of a
//                  tile of 256 and both read every key tile;
//   sides by keys  (at most 128): both have all rows, side s has the key tiles of its
//                  parity, joined at the item's end.
// Scores of 128 keys come from one product: with 64 a product of 16 channels takes 48 cycles for the 6 KB that
// it reads from shared memory where its multiplications take 32, with 128 it is level (measured: 48.5 and 64.6
// cycles).  A side then has one place for scores, worked on in two halves of 64 keys: while its threads turn one into
// weights, the product of the other and the other side's are under way.  So that two tiles of keys fit beside 256
// rows of Q of 192 channels, values come in half tiles.  ref moves, and O and the sums with it, when the
// weights of a half sum to more than 2^16.
// A prompt of 8192 tokens at 64 heads of 128 + 64 / 128 takes 1090 to 1130 us from one GB300 to another (1210 to 1260 TFLOP/s), 512 tokens
// behind 32256 537 to 553 us: 4050 cycles for
// 128 keys of both sides, where their products' multiplications and reads take 2660 and a thread's softmax about 3000, the two
// waiting for each other by turns.  Five of the eight forms spill 4 to 12 bytes at the registers of the split (12 to 156 read back,
// most where the heads' own channels are 64 and the sides go by keys).
//
// Warps: 0-3 side 0, 4-7 side 1 (a thread a row); 8 and 9 issue a side's products each;
// 10 and 11 fetch the rows of Q, keys and values by TMA; 12-15 look values over:
// where some row does not see some key, values past the item's keys (the next sequence's) are
// zeroed and non-finite ones taken out; rows that do see those add them one by one.
#include "kda_latent_tc.cuh"

namespace kda {
namespace kv {
namespace {

constexpr int KP = 64;  // keys of a half tile
constexpr int kSideRows = 128;
constexpr int kBlock = KP * 128;  // 64 keys of 64 channels
constexpr int kKBlock = KT * 128, kQBlock = kSideRows * 128;
constexpr int kThreads = 512, kLaunch = 128, kSoftmax = 184, kIssue = 72, kRows = 72;  // registers after the split
static_assert(8 * kSoftmax + 4 * kIssue + 4 * kRows == 16 * kLaunch, "the split uses what the launch has");
constexpr float kSumLimit = 65536.f;

template <int DN, int DV, bool kByKeys> struct Cfg {
    static constexpr int NK = DN / 64 + 1, NV = DV / 64;  // blocks of 64 channels
    static constexpr int kQImages = kByKeys ? 1 : 2, kQBytes = NK * kQBlock;
    static constexpr int kKBytes = NK * kKBlock, kVBytes = NV * kBlock;
    static constexpr int kRoom = 232448 - 1024 - 1792 - kQImages * kQBytes;
    static constexpr int kStagesK = kRoom - 3 * kKBytes >= 4 * kVBytes ? 3 : 2;
    static constexpr int kStagesV = (kRoom - kStagesK * kKBytes) / kVBytes < 6 ? (kRoom - kStagesK * kKBytes) / kVBytes : 6;
    static constexpr int kKAt = kQImages * kQBytes, kVAt = kKAt + kStagesK * kKBytes, kMiscAt = kVAt + kStagesV * kVBytes;
    static_assert(kStagesV >= 2 && kStagesV < kBars, "a tile's barrier is free before its stage");
};
struct alignas(16) Misc {
    uint64_t k_full[kBars], k_empty[kBars], v_full[kBars], v_empty[kBars], clean[kBars];
    uint64_t s_full[2], p_ready[2][2], pv_done[2][2];  // by side, and half
    uint64_t q_full[2], q_free[2], done[2];
    uint32_t tmem;
    int has, rows_gave_up[2];
    uint32_t turn;  // at issuing scores
    Cursor piece[2];
    uint32_t odd[kBars][2];  // by half tile: keys whose value row was taken out of it
    float m[kSideRows], l[kSideRows];  // side 1's row statistics, for the join
};
static_assert(sizeof(Misc) <= 1792, "room left for it");
struct PrefillMaps {
    CUtensorMap qn, qr, k, kr, v;
};

// Key tiles of an item's share that side s computes, and the v-th of them.
template <bool kByKeys> __device__ __forceinline__ int side_tiles(const Item &it, int s) {
    if (kByKeys) return (item_tiles(it) - s + 1) / 2;
    return s * kSideRows < it.rows ? item_tiles(it) : 0;
}
template <bool kByKeys> __device__ __forceinline__ int side_tile(int s, int v) { return kByKeys ? 2 * v + s : v; }
__device__ __forceinline__ bool some_unseen(const Item &it, int kb) { return kb + KP - 1 > it.ctx + it.tok0; }

// Adds the value rows that were taken out of a tile to O, for the rows that see them (a row's weight is read back
// from its bf16 place over the scores).  Rare, so short rather than fast.  Whole warp.
template <int DV>
__device__ __noinline__ void add_odd_rows(const PrefillRowsParams &p, const Item &it, int kb, int lim, const uint32_t *odd,
                                          uint32_t t_s, uint32_t t_o, bool fresh) {
    if (fresh) {
        const float z[16] = {};
        for (int c = 0; c < DV; c += 16) tmem_st16(t_o + uint32_t(c), z);
        tmem_wait_st();
    }
    for (int g = 0; g < KP / 32; ++g) {
        for (uint32_t left = odd[g]; left; left &= left - 1) {
            const int c = g * 32 + __ffs(left) - 1, j = kb + c;
            const uint32_t pw = tmem_ld1(t_s + uint32_t(c / 2));
            tmem_wait_ld();
            const float w = __uint_as_float(c & 1 ? pw & 0xffff0000u : pw << 16);
            const __nv_bfloat16 *val = static_cast<const __nv_bfloat16 *>(p.v) +
                                       (static_cast<long long>(p.b.cu_kv[it.n]) + j) * p.v_stride + it.h * p.v_head;
            for (int ch = 0; ch < DV; ch += 16) {
                float o[16];
                tmem_ld16(t_o + uint32_t(ch), o);
                tmem_wait_ld();
                if (j <= lim) {  // (also where it weighs 0: as in a tile that every row sees, 0 * infinity is NaN)
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[i] = fmaf(w, __bfloat162float(val[ch + i]), o[i]);
                }
                __syncwarp();
                tmem_st16(t_o + uint32_t(ch), o);
                tmem_wait_st();
            }
        }
    }
}

// Warp w of four looks over 16 keys of a value tile, two lanes a key.
template <int DV>
__device__ __forceinline__ void look_over(const Item &it, int kb, unsigned char *tile, int w, int lane, uint32_t *odd) {
    uint32_t out = 0;
    if (some_unseen(it, kb)) {
        const int key = w * 16 + (lane & 15), j = kb + key;
        unsigned char *img = tile + key * 128;
        auto piece = [&](int c) { return reinterpret_cast<uint4 *>(img + (c >> 3) * kBlock + (((c & 7) ^ (key & 7)) << 4)); };
        const bool gone = j >= it.k1;
        bool bad = false;
        for (int c = lane >> 4; c < DV / 8; c += 2) bad |= odd_bf16(*piece(c));
        bad |= __shfl_xor_sync(0xffffffffu, bad, 16);
        bad = bad && !gone && j > it.ctx + it.tok0;  // rows that every query sees stay
        if (gone || bad)
            for (int c = lane >> 4; c < DV / 8; c += 2) *piece(c) = make_uint4(0, 0, 0, 0);
        out = __ballot_sync(0xffffffffu, bad) & 0xffffu;
        fence_proxy_async_smem();
    }
    if (lane == 0) reinterpret_cast<uint16_t *>(odd)[w] = uint16_t(out);
    __syncwarp();
}

// Why the waits by parity are sound (see kBars: when someone waits for tile t, tile t - 8 is past, and t + 8 is not).
// Here the warp that fetches keys brings Q too, once q_free says that the last item's scores are done, while that item's
// values may still be on their way.
//   Not two past: t + 8 takes a stage that is free after t's, which all who wait for t have to say first.
//   Keys.  A tile is asked for when the one kStagesK (at most 3) before it is free, so if tile i was asked for, those up to
// i - 3 are past.  By rows both issuing warps wait for every tile, also of items that a side sits out.  By keys a side waits
// for its own: inside an item t - 2 was asked for before; at its start, q_full: Q is asked for behind all keys of the items before.
//   Values (half tiles 2 t and 2 t + 1).  The warps that look them over wait for each in turn: the one before was asked for, so
// those up to 7 before are free.  So `clean` completes in order, and whoever has seen it of one knows all before it past, of
// v_full and of clean.  By rows a side's issuing warp waits for clean of every one, and issues an item's scores
// after that, which are what its softmax waits for first.  By keys, inside an item, a side has seen clean of both halves of
// t - 2 before it issues the scores of t.  At its start, b being its first tile, side 0 goes on to wait for 2 b and side 1
// for 2 b + 2, so those up to 2 b - 5 (1 + 2 (b - 3), the latest for 2 b + 3) have to be past.  q_full is behind q_free of the item
// before, which both sides give, and tile b - 3 is either in that item, where its side also has the last tile, b - 1, whose scores
// (and q_free) it issues after it has seen b - 3 clean; or in one before that, which its side was through with before.
template <int DN, int DV, bool kByKeys>
__global__ void __launch_bounds__(kThreads, 1)
    latent_prefill_kernel(const __grid_constant__ PrefillRowsParams p, const __grid_constant__ PrefillMaps maps) {
    using C = Cfg<DN, DV, kByKeys>;
    constexpr int NSK = C::kStagesK, NSV = C::kStagesV, NK = C::NK, BM = kByKeys ? kSideRows : 2 * kSideRows;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Misc &ms = *reinterpret_cast<Misc *>(smem + C::kMiscAt);
    const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5, cta = int(blockIdx.x);
    unsigned char *k_ring = smem + C::kKAt, *v_ring = smem + C::kVAt;

    if (tid == 0) {
        for (int i = 0; i < kBars; ++i) {
            mbar_init(&ms.k_full[i], 1), mbar_init(&ms.v_full[i], 1), mbar_init(&ms.clean[i], 4);
            // by rows both sides are done with a tile
            mbar_init(&ms.k_empty[i], kByKeys ? 1 : 2), mbar_init(&ms.v_empty[i], kByKeys ? 1 : 2);
        }
        for (int i = 0; i < 2; ++i) {
            for (int h = 0; h < 2; ++h) mbar_init(&ms.p_ready[i][h], 4), mbar_init(&ms.pv_done[i][h], 1);
            mbar_init(&ms.s_full[i], 1), mbar_init(&ms.q_full[i], 1), mbar_init(&ms.q_free[i], kByKeys ? 2 : 1), mbar_init(&ms.done[i], 1);
        }
        fence_mbar_init();
    }
    if (tid == 32) {
        for (const CUtensorMap *m : {&maps.qn, &maps.qr, &maps.k, &maps.kr, &maps.v})
            asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
    }
    if (warp == 8) tmem_alloc(&ms.tmem, 512);
    wait_prior_kernel();
    allow_next_kernel();
    if (tid < 2) p.parts[2 * cta + tid].state = 0;
    if (warp == 10) {
        Cursor a, z;
        const bool has = find_piece(p, cta, int(gridDim.x), lane, a, z);
        if (lane == 0) ms.piece[0] = a, ms.piece[1] = z, ms.has = has, ms.rows_gave_up[0] = ms.rows_gave_up[1] = 0, ms.turn = 0;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = ms.tmem;
    uint32_t *err = p.b.err;
    bool ok = true;  // of this thread's waits

    if (warp < 8) {
        set_regs<kSoftmax, kLaunch>();
        if (ms.has) {
            // ---- softmax: thread = row -------------------------------------------------
            const int s = warp >> 2, row = tid & 127;
            const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
            const uint32_t t_s = tm + lanes + uint32_t(s) * 128u, t_o = tm + lanes + 256u + uint32_t(s) * 128u;
            const int r = (kByKeys ? 0 : s * kSideRows) + row;
            ItemWalk walk(ms.piece[0], ms.piece[1]);
            Item it = {};
            uint32_t n = 0, tile_base = 0;  // tiles of this side, of all: barrier phases
            // O holds this side's products up to half h of its tile i
            auto wait_o = [&](uint32_t i, int h) {
                wait_for(ok, &ms.pv_done[s][h], i & 1, err);
                __syncwarp();
                tc_fence_after();
            };
            while (walk.next(p, it)) {
                const int nv = side_tiles<kByKeys>(it, s);
                const int lim = it.ctx + it.tok0 + min(r, it.rows - 1);  // last key this row sees
                const bool live = r - lane < it.rows;  // this warp has rows of the item
                const float scale = p.scale_log2;
                float ref = -INFINITY, l = 0.f;
                for (int v = 0; v < nv; ++v, ++n) {
                    const int t = side_tile<kByKeys>(s, v);
                    // Scores of a tile are issued after the last product of the one before, so whoever sees them
                    // knows that O holds it.
                    wait_for(ok, &ms.s_full[s], n & 1, err);
                    __syncwarp();
                    tc_fence_after();
#pragma unroll 1
                    for (int h = 0; h < 2; ++h) {
                        const int kb = it.k0 + t * KT + h * KP;
                        const bool check = some_unseen(it, kb);
                        const uint32_t t_h = t_s + uint32_t(h) * KP;
                        if (live) {
                            float x[KP];
#pragma unroll
                            for (int c = 0; c < KP; c += 32) tmem_ld32(t_h + uint32_t(c), x + c);
                            tmem_wait_ld();
                            if (check) {
#pragma unroll
                                for (int c = 0; c < KP; ++c)
                                    if (kb + c > lim) x[c] = -INFINITY;
                            }
                            const bool started = v > 0 || h > 0;  // O is new with the first product
                            // the reference of a row that needs it moves up to the row's maximum in x, where that is above it
                            // (of no other: what a row gives does not depend on its neighbours)
                            auto move_ref = [&](bool need) {
                                float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                                for (int c = 4; c < KP; c += 4)
#pragma unroll
                                    for (int i = 0; i < 4; ++i) mx[i] = fmaxf(mx[i], x[c + i]);
                                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale;
                                const bool move = need && top > ref;
                                if (!__any_sync(0xffffffffu, move)) return;
                                const float to = move ? top : ref, f = move ? ex2(ref - to) : 1.f;
                                if (started) {
                                    if (h > 0) wait_o(n, 0);
#pragma unroll 1
                                    for (int c = 0; c < DV; c += 16) {
                                        float o[16];
                                        tmem_ld16(t_o + uint32_t(c), o);
                                        tmem_wait_ld();
#pragma unroll
                                        for (int i = 0; i < 16; ++i) o[i] *= f;
                                        tmem_st16(t_o + uint32_t(c), o);
                                    }
                                }
                                l *= f;
                                ref = to;
                            };
                            // weights to the place of the scores; their sum
                            auto weigh = [&] {
                                const float base = ref == -INFINITY ? 0.f : ref;
                                const float2 sc = make_float2(scale, scale), sh = make_float2(-base, -base);
                                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                                for (int c = 0; c < KP; c += 32) {
                                    uint32_t w[16];
#pragma unroll
                                    for (int i = 0; i < 16; ++i) {
                                        float2 e = fma2(make_float2(x[c + 2 * i], x[c + 2 * i + 1]), sc, sh);
                                        e.x = ex2(e.x), e.y = ex2(e.y);
                                        sum[i & 1] = add2(sum[i & 1], e);
                                        w[i] = pack_bf16(e.x, e.y);
                                    }
                                    tmem_st16u(t_h + uint32_t(c / 2), w);
                                }
                                return (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                            };
                            if (!started) move_ref(true);
                            float sum_h = weigh();
                            // past the limit (or NaN), or a row without a reference yet
                            const bool need = r < it.rows && (!(sum_h <= kSumLimit) || ref == -INFINITY);
                            if (__any_sync(0xffffffffu, need)) {
                                move_ref(need);
                                tmem_wait_st();
                                sum_h = weigh();
                            }
                            tmem_wait_st();
                            l += sum_h;
                            if (check) {
                                const uint32_t u = 2 * (tile_base + uint32_t(t)) + uint32_t(h);
                                wait_tile(ok, ms.clean, u, err);
                                ok = __all_sync(0xffffffffu, ok);
                                const uint32_t *odd = ms.odd[u % kBars];
                                if (ok && any_odd(odd)) {
                                    if (h > 0) wait_o(n, 0);
                                    const Item copy = it;
                                    add_odd_rows<DV>(p, copy, kb, lim, odd, t_h, t_o, !started);
                                }
                            }
                        }  // else rows of nobody: their weights may be anything
                        tc_fence_before();
                        __syncwarp();
                        if (ok && lane == 0) mbar_arrive(&ms.p_ready[s][h]);
                    }
                }
                tile_base += uint32_t(item_tiles(it));

                // ---- output ----------------------------------------------------------------
                const int nv_other = kByKeys ? side_tiles<kByKeys>(it, 1 - s) : 0;
                if (nv > 0) wait_o(n - 1, 1);
                float f0 = 1.f, f1 = 0.f;
                if (kByKeys) {
                    if (s == 1) ms.m[row] = ref, ms.l[row] = l;  // its products are done: side 0 may read both
                    tc_fence_before();
                    named_sync<1, 256>();
                    if (s == 0 && nv_other > 0) {
                        const float m1 = ms.m[row], top = fmaxf(ref, m1), base = top == -INFINITY ? 0.f : top;
                        f0 = ex2(ref - base), f1 = ex2(m1 - base);
                        l = l * f0 + ms.l[row] * f1;
                        ref = top;
                    }
                }
                tc_fence_after();
                if (!(kByKeys && s == 1) && nv > 0) {
                    const float inv = l > 0.f || l != l ? 1.0f / l : 0.f;
                    const bool whole = it.whole(), writes = r < it.rows;
                    float *data = p.part_data + (size_t(cta) * 2 + it.slot()) * size_t(BM) * size_t(DV + 2);
                    __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out) +
                                         (static_cast<long long>(it.row0) + it.tok0 + min(r, it.rows - 1)) * p.out_stride +
                                         it.h * p.out_head;
                    const bool wide =
                        ((reinterpret_cast<uintptr_t>(p.out) | uintptr_t(p.out_stride * 2) | uintptr_t(p.out_head * 2)) & 31) == 0;
#pragma unroll 1
                    for (int c = 0; c < DV; c += 32) {
                        float o[32];
                        tmem_ld32(t_o + uint32_t(c), o);
                        if (kByKeys && nv_other > 0) {
                            float o1[32];
                            tmem_ld32(t_o + 128u + uint32_t(c), o1);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] = o[i] * f0 + o1[i] * f1;
                        } else {
                            tmem_wait_ld();
                        }
                        if (!writes) continue;
                        if (whole) {
#pragma unroll
                            for (int e = 0; e < 32; e += 16) {
                                uint32_t w[8];
#pragma unroll
                                for (int i = 0; i < 8; ++i) w[i] = pack_bf16(o[e + 2 * i] * inv, o[e + 2 * i + 1] * inv);
                                if (wide) {
                                    store32(dst + c + e, w);
                                } else {
                                    *reinterpret_cast<uint4 *>(dst + c + e) = make_uint4(w[0], w[1], w[2], w[3]);
                                    *reinterpret_cast<uint4 *>(dst + c + e + 8) = make_uint4(w[4], w[5], w[6], w[7]);
                                }
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; i += 8) {
                                uint32_t w[8];
#pragma unroll
                                for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(o[i + e]);
                                store32(data + size_t(r) * DV + c + i, w);
                            }
                        }
                    }
                    if (!whole) {
                        if (writes) data[BM * DV + r] = ref, data[BM * DV + BM + r] = l;
                        if (s == 0 && row == 0) p.parts[2 * cta + it.slot()] = it.part();
                    }
                }
                tc_fence_before();  // the next item's products rewrite O
                if (kByKeys) named_sync<1, 256>();
            }
        }
    } else if (warp < 12) {
        set_regs<kIssue, kLaunch>();
        if (ms.has && warp < 10) {
            // ---- products of a side (converged warp, one lane issues; descriptors count 16-byte units) ---
            const int s = warp - 8, qi = kByKeys ? 0 : s;  // the image of Q
            const uint32_t id_s = idesc_bf16_f32(128, KT), id_o = idesc_bf16_f32(128, DV, false, true);
            const uint32_t t_s = tm + uint32_t(s) * 128u, t_o = tm + 256u + uint32_t(s) * 128u;
            const uint32_t q_desc = desc_k(smem_u32(smem) + uint32_t(qi) * C::kQBytes), k_desc = desc_k(smem_u32(k_ring));
            const uint32_t v_desc = desc_mn(smem_u32(v_ring), kBlock);
            ItemWalk walk(ms.piece[0], ms.piece[1]);
            Item it = {};
            uint32_t base = 0, n_q = 0, n = 0;
            int nv = 0;
            // scores of the side's v-th tile
            auto scores = [&](int v) {
                const uint32_t tg = base + uint32_t(side_tile<kByKeys>(s, v));
                wait_tile(ok, ms.k_full, tg, err);
                if (!(ok = __all_sync(0xffffffffu, ok))) return;
                tc_fence_after();
                if (elect_one()) {
                    take_turn(&ms.turn);
                    const uint32_t kd = k_desc + tg % NSK * uint32_t(C::kKBytes >> 4);
#pragma unroll
                    for (int k = 0; k < NK * 4; ++k)
                        mma_lo(t_s, q_desc + uint32_t((k >> 2) * (kQBlock >> 4) + (k & 3) * 2),
                               kd + uint32_t((k >> 2) * (kKBlock >> 4) + (k & 3) * 2), id_s, k > 0);
                    end_turn(&ms.turn);
                    mma_commit(&ms.s_full[s]);
                    mma_commit(&ms.k_empty[tg % kBars]);
                    if (v + 1 == nv) mma_commit(&ms.q_free[qi]);
                }
                __syncwarp();
            };
            while (ok && walk.next(p, it)) {
                nv = side_tiles<kByKeys>(it, s);
                if (kByKeys || nv > 0) wait_for(ok, &ms.q_full[qi], n_q++ & 1, err);
                if (nv > 0) {
                    scores(0);
                } else if (kByKeys) {
                    if (!(ok = __all_sync(0xffffffffu, ok))) break;
                    if (lane == 0) mbar_arrive(&ms.q_free[0]);
                }
                for (int v = 0; v < nv && ok; ++v, ++n) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t u = 2 * (base + uint32_t(side_tile<kByKeys>(s, v))) + uint32_t(h);
                        wait_all(ok, err, Awaited{&ms.p_ready[s][h], n & 1}, of_tile(ms.v_full, u), of_tile(ms.clean, u));
                        if (!(ok = __all_sync(0xffffffffu, ok))) break;
                        tc_fence_after();
                        // the first product starts O, unless value rows were added to it by hand
                        const uint32_t acc = v > 0 || any_odd(ms.odd[u % kBars]);
                        if (elect_one()) {
                            const uint32_t vd = v_desc + u % NSV * uint32_t(C::kVBytes >> 4);
#pragma unroll
                            for (int k = 0; k < KP / 16; ++k)
                                mma_lo_ta(t_o, t_s + uint32_t(h * KP + k * 8), vd + uint32_t(k * 128), id_o, h > 0 || k > 0 || acc);
                            mma_commit(&ms.pv_done[s][h]);
                            mma_commit(&ms.v_empty[u % kBars]);
                        }
                        __syncwarp();
                    }
                    if (ok && v + 1 < nv) scores(v + 1);
                }
                if (!kByKeys && nv == 0) {  // a tile is free once both sides have said so
                    for (int i = 0; i < item_tiles(it) && ok; ++i) {
                        const uint32_t tg = base + uint32_t(i);
                        wait_tile(ok, ms.k_full, tg, err);
                        if (ok && lane == 0) mbar_arrive(&ms.k_empty[tg % kBars]);
                        for (uint32_t u = 2 * tg; u < 2 * tg + 2; ++u) {  // (and passes no barrier by)
                            wait_tile(ok, ms.v_full, u, err);
                            wait_tile(ok, ms.clean, u, err);
                            if (!(ok = __all_sync(0xffffffffu, ok))) break;
                            if (lane == 0) mbar_arrive(&ms.v_empty[u % kBars]);
                        }
                    }
                }
                base += uint32_t(item_tiles(it));
            }
            // nothing of this side's is in flight when the tensor memory goes
            if (elect_one()) mma_commit(&ms.done[s]);
            __syncwarp();
            mbar_wait(&ms.done[s], 0, err);
        } else if (ms.has) {
            // ---- fetches: rows of Q and keys, or values ----------------------------------------
            const bool values = warp == 11;
            uint64_t *full = values ? ms.v_full : ms.k_full, *empty = values ? ms.v_empty : ms.k_empty;
            ItemWalk walk(ms.piece[0], ms.piece[1]);
            Item it = {};
            uint32_t t = 0, asked[2] = {0, 0};  // of tiles, and images of Q
            while (ok && walk.next(p, it)) {
                const int row0 = p.b.cu_kv[it.n];
                // the rows of Q, once the last item's scores have read theirs (rows of nobody are the next sequence's,
                // or zeros past the last)
                for (int s = 0; s < (values ? 0 : C::kQImages); ++s) {
                    if (side_tiles<kByKeys>(it, s) == 0) continue;
                    wait_for(ok, &ms.q_free[s], (asked[s] & 1) ^ 1, err);
                    if (!(ok = __all_sync(0xffffffffu, ok))) break;
                    ++asked[s];
                    if (lane == 0) mbar_arrive_expect_tx(&ms.q_full[s], uint32_t(C::kQBytes));
                    __syncwarp();
                    if (lane < NK)
                        tma_load_3d(smem + s * C::kQBytes + lane * kQBlock, lane < NK - 1 ? &maps.qn : &maps.qr, &ms.q_full[s],
                                    lane < NK - 1 ? lane * 64 : 0, it.h, it.row0 + it.tok0 + s * kSideRows);
                    __syncwarp();
                }
                // (whole tiles of both: their second halves may lie past the item's keys)
                const int end = it.k0 + item_tiles(it) * KT, step = values ? KP : KT;
                for (int kb = it.k0; kb < end && ok; kb += step, ++t) {
                    if (values) wait_stage<NSV>(ok, empty, t, err);
                    else wait_stage<NSK>(ok, empty, t, err);
                    if (!(ok = __all_sync(0xffffffffu, ok))) break;
                    uint64_t *bar = &full[t % kBars];
                    if (lane == 0) mbar_arrive_expect_tx(bar, uint32_t(values ? C::kVBytes : C::kKBytes));
                    __syncwarp();
                    if (values) {
                        if (lane < C::NV)
                            tma_load_3d(v_ring + t % NSV * C::kVBytes + lane * kBlock, &maps.v, bar, lane * 64, it.h, row0 + kb);
                    } else if (lane < NK - 1) {
                        tma_load_3d(k_ring + t % NSK * C::kKBytes + lane * kKBlock, &maps.k, bar, lane * 64, it.h, row0 + kb);
                    } else if (lane == NK - 1) {
                        tma_load_3d(k_ring + t % NSK * C::kKBytes + lane * kKBlock, &maps.kr, bar, 0, 0, row0 + kb);
                    }
                    __syncwarp();
                }
            }
            // whichever role gives up, no copy is in flight when the CTA ends
            for (uint32_t i = t - min(t, uint32_t(values ? NSV : NSK)); i < t; ++i) mbar_wait(&full[i % kBars], (i / kBars) & 1, err);
            for (int s = 0; s < 2; ++s)
                if (asked[s] > 0) mbar_wait(&ms.q_full[s], (asked[s] - 1) & 1, err);
        }
    } else {
        set_regs<kRows, kLaunch>();
        if (ms.has) {
            // ---- values looked over ---------------------------------------------------------------
            const int w = warp - 12;
            ItemWalk walk(ms.piece[0], ms.piece[1]);
            Item it = {};
            uint32_t tile = 0, turn = 0;  // half tiles so far
            // Only the first of these warps waits by polling, which takes issue slots; the others
            // meet it at a barrier of the hardware's, and learn there whether it gave up.
            // (by turns two words: the first may be an appointment ahead of a warp that still reads)
            auto meet = [&] {
                if (w == 0 && !ok) ms.rows_gave_up[turn] = 1;
                named_sync<4, 128>();
                ok = ms.rows_gave_up[turn] == 0;
                turn ^= 1;
            };
            while (ok && walk.next(p, it)) {
                const int end = it.k0 + item_tiles(it) * KT;
                for (int kb = it.k0; kb < end && ok; kb += KP, ++tile) {
                    if (w == 0) wait_tile(ok, ms.v_full, tile, err);
                    meet();
                    if (!ok) break;
                    look_over<DV>(it, kb, v_ring + tile % NSV * C::kVBytes, w, lane, ms.odd[tile % kBars]);
                    if (lane == 0) mbar_arrive(&ms.clean[tile % kBars]);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 8) tmem_dealloc(tm, 512);
}

// [rows][heads][channels]; a box is 64 channels of some rows of one head (zeros past the last channel or row).
inline bool rows_map(CUtensorMap *m, const void *base, int channels, int heads, long long head, int rows, long long stride,
                     int box_rows) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {cuuint64_t(channels), cuuint64_t(heads), cuuint64_t(rows)};
    const cuuint64_t strides[2] = {cuuint64_t(head) * 2, cuuint64_t(stride) * 2};
    const cuuint32_t box[3] = {64u, 1u, cuuint32_t(box_rows)}, estr[3] = {1u, 1u, 1u};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DN, int DV, bool kByKeys>
kda_status launch(PrefillRowsParams &p, const AttendPlan &plan, cudaStream_t stream) {
    using C = Cfg<DN, DV, kByKeys>;
    PrefillMaps maps;
    const int rows = p.b.max_kv_rows;
    if (!rows_map(&maps.qn, p.q_a, DN, p.hkv, p.qa_head, p.b.max_rows, p.qa_stride, kSideRows) ||
        !rows_map(&maps.qr, p.q_r, p.rope, p.hkv, p.qr_head, p.b.max_rows, p.qr_stride, kSideRows) ||
        !rows_map(&maps.k, p.k, DN, p.hkv, p.k_head, rows, p.k_stride, KT) ||
        !rows_map(&maps.kr, p.kr, p.rope, 1, p.kr_stride, rows, p.kr_stride, KT) ||
        !rows_map(&maps.v, p.v, DV, p.hkv, p.v_head, rows, p.v_stride, KP))
        return KDA_ERR_CUDA;
    constexpr size_t smem = 1024 + C::kMiscAt + sizeof(Misc);
    static_assert(smem <= 232448, "shared memory of a CTA");
    if (!allow_smem<latent_prefill_kernel<DN, DV, kByKeys>>(int(smem))) return KDA_ERR_CUDA;
    p.key_step = KT;
    p.item_cost = 512;
    p.min_keys = (kByKeys ? 2 : 1) * KT;
    const ProfScope prof(KDA_KERNEL_LATENT_PREFILL, stream);
    return launch_overlapped(latent_prefill_kernel<DN, DV, kByKeys>, dim3(unsigned(plan.n_cta)), kThreads, smem, stream, p, maps);
}

template <int DN, int DV> kda_status by_sides(PrefillRowsParams &p, const AttendPlan &plan, cudaStream_t s) {
    return plan.bm == kSideRows ? launch<DN, DV, true>(p, plan, s) : launch<DN, DV, false>(p, plan, s);
}

}  // namespace

bool prefill_tile_plan(const kda_latent_cache *c, const kda_latent_prefill_batch *b, AttendPlan *plan) {
    if (c->act != KDA_BF16) return false;
    // By keys and by rows, us: 128 tokens behind 16000 101 and 114, 16 sequences of 128 behind 1000 134 and 147, of 16
    // 101 and 117.
    plan->bm = b->max_new <= kSideRows ? kSideRows : 2 * kSideRows;
    plan->n_cta = sm_count();
    return true;
}

kda_status prefill_tile_launch(const kda_latent_cache *, const kda_latent_prefill_io *io, PrefillRowsParams &p,
                               const AttendPlan &plan, cudaStream_t s) {
    if (io->nope_dim == 64) return io->value_dim == 64 ? by_sides<64, 64>(p, plan, s) : by_sides<64, 128>(p, plan, s);
    return io->value_dim == 64 ? by_sides<128, 64>(p, plan, s) : by_sides<128, 128>(p, plan, s);
}

}  // namespace kv
}  // namespace kda
