// kda_attend_tile.cu -- kda_kv_attend for bf16 rows on the tensor cores: the
// kernel of chunks, verifies and wide groups (all bf16 calls but those of few
// rows, see kda_attend_few.cu and kda_attend_lanes.cu).  Heads of 16 and 32
// channels are worked on as if they had 64, the others zero: the products cost
// more than they need, but the softmax bounds such calls.
//
// Softmax in one pass, as in kda_attend_generic.cu: scores X = Q K^T (128 rows
// x 128 keys) land in tensor memory, one thread per row turns them into weights
// P = 2^(scale log2e X - ref) and leaves them as bf16 where the scores were,
// and O += P V reads them from there.  Two of these run side by side so that
// one's products cover the other's exponentials:
//   sides by rows  (row tiles of 256): side s has rows [128 s, 128 s + 128) and
//                  both read every key tile (half the L2 traffic per product);
//   sides by keys  (at most 128 rows an item): both have all rows, side s has
//                  the key tiles of its parity, joined at the item's end.
// A tile is worked on in two halves of 64 keys, each with its own score columns:
// while the threads of a side turn one half into weights, the other half's
// product and the scores that follow in its place are under way, so the threads
// seldom wait and the tensor cores seldom idle.
// ref is the row's maximum at the time it was last moved.  bf16 pages: it moves
// (and O and the sums are scaled by 2^(ref - ref')) when the weights of a half of
// a tile sum to more than 2^16, which shows once they are formed; then they are
// formed again.  e4m3 pages: when a half's maximum exceeds it by more than 8.
// Weights of 2^16 cost no precision in bf16 and fp32, so most tiles leave O in
// tensor memory untouched, and in bf16 need no maximum at all (the 8192-token
// prompt with heads of 64: 653 us against 720 with a maximum for each half; with
// heads of 128 783 either way; in e4m3 the registers are short for it, and verifies
// take 261 us against 224).  P is rounded to bf16 (2^-8 relative, the
// size of the output's own rounding, and not correlated between keys); scores,
// sums and O stay in 32 bits.
//
// Warps: 0-3 side 0, 4-7 side 1 (a thread a row); 8 and 9 issue a side's
// products each; 10 and 11 fetch pages by TMA into rings of key and value tiles;
// 12-15 bring the rows of Q and look value tiles over (below).
//
// e4m3 pages: keys go to the tensor cores as they are, against Q as the sum of
// two e4m3 terms, which is Q itself (as many cycles as bf16 products take), and
// the keys' scales multiply the scores.  Values meet bf16 weights, so warps
// 12-19 turn raw value tiles into bf16 ones, scale included and exact.
//
// A value behind a row's position weighs nothing, but 0 * NaN is NaN in the
// product.  So in the few tiles where some row does not see some key, warps
// 12-15 zero the rows of absent keys in the value tile, and take non-finite
// value rows out of it; the row threads that do see those add them one by one.
//
// What bounds it: a half's products wait for its weights and its weights for its
// scores; two sides with two halves each cover most of that, and tensor memory has
// no columns for more (heads of 128: the tensor pipe is active in 65 % of the
// cycles; heads of 64 leave 128 columns idle, there the softmax threads are the slower
// part).  Measured at 2070 MHz, 64
// heads over 8 cache heads of 128: a prompt of 8192 tokens 771 us (1430 TFLOP/s,
// 74 % of the measured bf16 peak), 512 tokens behind 32256 410 us (69 %); kept up for
// seconds, under the power cap, 800 us at 1972 MHz and 437 us at 1762 MHz.  In e4m3
// pages the prompt takes 1102 us, bound by the threads that widen values and scale
// scores and by the second term of Q.  64 verifies of 8 tokens over 1000 to 8192
// in e4m3 take 208 us (3.0 TB/s).  Heads of 64: the prompt 670 us.
#include "kda_attend_tc.cuh"

namespace kda {
namespace kv {
namespace {

constexpr int KH = KT / 2;        // keys of a half
constexpr int kSideRows = 128;   // rows of a side
// Warps: 8 of softmax, 4 that issue, then those of Q and the value tiles (8 where
// these are e4m3 and have to be widened).  Registers a thread after the split,
// of 128 (bf16) or 96 (e4m3) at launch.
template <bool kE4m3> struct Warps {
    static constexpr int kRowWarps = kE4m3 ? 8 : 4, kThreads = (12 + kRowWarps) * 32, kLaunch = kE4m3 ? 96 : 128;
    static constexpr int kSoftmax = kE4m3 ? 144 : 200, kIssue = kE4m3 ? 48 : 56, kRows = kE4m3 ? 72 : 56;
    static_assert(8 * kSoftmax + 4 * kIssue + kRowWarps * kRows == (12 + kRowWarps) * kLaunch, "the split uses what the launch has");
};
// When a row's reference moves (see above): a maximum this far above it, or a sum of a half's weights.
constexpr float kRefSlack = 8.f, kSumLimit = 65536.f;
// Keys that take as long as an item's start and output.  Measured at 0, 128, 256,
// 512, 1024: 8 sequences of 300 to 700 new tokens behind 100 to 1500 take 237, 216,
// 201, 183, 187 us, 64 verifies of 8 tokens there 86, 75, 69, 64, 63 us.
constexpr int kItemCost = 512;

template <int D, bool kE4m3, bool kByKeys> struct Cfg {
    static constexpr int kQBytes = kSideRows * D * 2;            // bf16, or two e4m3 terms
    static constexpr int kKBytes = KT * D * (kE4m3 ? 1 : 2), kVBytes = KT * D * 2, kRawBytes = KT * D;
    // Shared memory: the rows of Q once (by keys) or a side (by rows), and rings
    // of key tiles, bf16 value tiles and (e4m3) raw value tiles.  By keys the
    // bytes in flight set the pace (HBM latency), by rows the products do.
    static constexpr int kQImages = kByKeys ? 1 : 2;
    static constexpr int kStagesK = D == 64 ? 6 : 3;
    static constexpr int kStagesV = D == 64 ? 6 : kE4m3 ? 2 : kByKeys ? 3 : 2;
    static constexpr int kStagesRaw = !kE4m3 ? 1 : D == 64 ? 4 : kByKeys ? 4 : 2;
    static constexpr int kKAt = kQImages * kQBytes;
    static constexpr int kVAt = kKAt + kStagesK * kKBytes;
    static constexpr int kRawAt = kVAt + kStagesV * kVBytes;
    static constexpr int kMiscAt = kRawAt + (kE4m3 ? kStagesRaw * kRawBytes : 0);
};
template <typename C> struct alignas(16) Misc {
    uint64_t k_full[kBars], k_empty[kBars], v_full[kBars], v_empty[kBars], clean[kBars];
    uint64_t raw_full[kBars], raw_empty[kBars], unit_full[kBars];
    uint64_t s_full[2][2], p_ready[2][2], pv_done[2][2];  // by side and half
    uint64_t q_full[2], q_free[2], done[2];
    uint64_t row_unit[2][2];  // e4m3, by image and item parity: the rows' scales are there
    uint32_t tmem;
    int has, rows_gave_up[2];
    Cursor piece[2];
    uint32_t odd[kBars][4];                        // by tile: keys whose value row was taken out of it
    float m[kSideRows], l[kSideRows];              // side 1's row statistics, for the join
};
// A tile's key scales are written once its keys have landed, in a stage that the
// scores of the tile kStagesK before have left; those come after the same side's
// weights of two tiles before that, so kUnits sets are enough.
constexpr int kUnits = 8;
template <typename C> struct ScaleMisc {  // e4m3 pages only
    alignas(16) uint8_t k[C::kStagesK][KT];  // the tiles' scale exponents
    alignas(16) uint8_t v[C::kStagesRaw][KT];
    alignas(16) float k_unit[kUnits][KT];    // by tile, the keys' scales
    float q_unit[2][2][kSideRows];           // by item parity and image, the rows' scales
};

template <typename C, bool kE4m3> constexpr size_t smem_bytes() {
    return 1024 + C::kMiscAt + (kE4m3 ? sizeof(ScaleMisc<C>) : 0) + sizeof(Misc<C>);
}

// Key tiles of an item's share that side s computes, and the v-th of them.
template <bool kByKeys> __device__ __forceinline__ int side_tiles(const Item &it, int s) {
    if (kByKeys) return (item_tiles(it) - s + 1) / 2;
    return s * kSideRows < it.rows ? item_tiles(it) : 0;
}
template <bool kByKeys> __device__ __forceinline__ int side_tile(int s, int v) { return kByKeys ? 2 * v + s : v; }

// Adds the value rows that were taken out of a tile to O, for the rows that see
// them (a row's weight is read back from its bf16 place over the scores).  Rare,
// so short rather than fast.  Whole warp.
// Channels of a head: images of 64 also hold heads of 16 and 32.
template <int D> __device__ __forceinline__ int head_dim(const AttendParams &p) { return D == 64 ? p.dim : D; }
template <int D, bool kE4m3>
__device__ __noinline__ void add_odd_rows(const AttendParams &p, const Item &it, int kb, int lim, const uint32_t *odd,
                                          uint32_t t_s, uint32_t t_o, bool fresh) {
    if (fresh) {
        const float z[16] = {};
        for (int c = 0; c < D; c += 16) tmem_st16(t_o + uint32_t(c), z);
        tmem_wait_st();
    }
    const int dim = head_dim<D>(p);
    for (int g = 0; g < KH / 32; ++g) {
        for (uint32_t left = odd[g]; left; left &= left - 1) {
            const int c = g * 32 + __ffs(left) - 1, j = kb + c;
            const uint32_t pw = tmem_ld1(t_s + uint32_t(c / 2));
            tmem_wait_ld();
            const float w = __uint_as_float(c & 1 ? pw & 0xffff0000u : pw << 16);
            const int page = load_page(p.b, it.n, j);
            const size_t vec = ((size_t(max(page, 0)) * size_t(p.hkv) + size_t(it.h)) << p.b.page_shift) +
                               size_t(j & ((1 << p.b.page_shift) - 1));
            for (int ch = 0; ch < dim; ch += 16) {
                float o[16];
                tmem_ld16(t_o + uint32_t(ch), o);
                tmem_wait_ld();
                if (j <= lim && w != 0.f) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float val;
                        if constexpr (kE4m3)
                            val = unpack_e4m3(static_cast<const uint8_t *>(p.pv)[vec * size_t(dim) + ch + i]).x * exp2_biased(p.sv[vec]);
                        else
                            val = __bfloat162float(static_cast<const __nv_bfloat16 *>(p.pv)[vec * size_t(dim) + ch + i]);
                        o[i] = fmaf(w, val, o[i]);
                    }
                }
                __syncwarp();
                tmem_st16(t_o + uint32_t(ch), o);
                tmem_wait_st();
            }
        }
    }
}

// The scales of 32 keys, all loads in flight together (one by one, as they are used,
// they took longer than the exponentials), and 32 scores times them.
__device__ __forceinline__ void load_units(float4 (&u)[8], const float *src) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(u[i].x), "=f"(u[i].y), "=f"(u[i].z), "=f"(u[i].w)
                     : "r"(smem_u32(src + 4 * i))
                     : "memory");
}
__device__ __forceinline__ void scale_keys(float *x, const float4 (&u)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 a = mul2(make_float2(x[4 * i], x[4 * i + 1]), make_float2(u[i].x, u[i].y));
        const float2 b = mul2(make_float2(x[4 * i + 2], x[4 * i + 3]), make_float2(u[i].z, u[i].w));
        x[4 * i] = a.x, x[4 * i + 1] = a.y, x[4 * i + 2] = b.x, x[4 * i + 3] = b.y;
    }
}

template <int D, bool kE4m3, bool kByKeys>
__global__ void __launch_bounds__(Warps<kE4m3>::kThreads, 1)
    attend_tile_kernel(const __grid_constant__ AttendParams p, const __grid_constant__ TileMaps maps) {
    using C = Cfg<D, kE4m3, kByKeys>;
    using W = Warps<kE4m3>;
    constexpr int NK = C::kStagesK, NV = C::kStagesV, NR = C::kStagesRaw, BM = kByKeys ? kSideRows : 2 * kSideRows;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Misc<C> &ms = *reinterpret_cast<Misc<C> *>(smem + C::kMiscAt);
    ScaleMisc<C> &sc8 = *reinterpret_cast<ScaleMisc<C> *>(smem + C::kMiscAt + sizeof(Misc<C>));  // kE4m3 only
    const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5, cta = int(blockIdx.x);
    unsigned char *k_ring = smem + C::kKAt, *v_ring = smem + C::kVAt, *raw_ring = smem + C::kRawAt;

    if (tid == 0) {
        for (int i = 0; i < kBars; ++i) {
            mbar_init(&ms.k_full[i], 1), mbar_init(&ms.v_full[i], kE4m3 ? W::kRowWarps : 1);
            // by rows both sides are done with a tile
            mbar_init(&ms.k_empty[i], (kByKeys ? 1 : 2) + (kE4m3 ? W::kRowWarps : 0));  // and the scales read
            mbar_init(&ms.v_empty[i], kByKeys ? 1 : 2);
            mbar_init(&ms.clean[i], 4), mbar_init(&ms.raw_full[i], 1), mbar_init(&ms.raw_empty[i], W::kRowWarps);
            mbar_init(&ms.unit_full[i], W::kRowWarps);
        }
        for (int i = 0; i < 2; ++i) {
            for (int h = 0; h < 2; ++h)
                mbar_init(&ms.s_full[i][h], 1), mbar_init(&ms.p_ready[i][h], 4), mbar_init(&ms.pv_done[i][h], 1);
            mbar_init(&ms.q_full[i], W::kRowWarps), mbar_init(&ms.q_free[i], kByKeys ? 2 : 1);
            mbar_init(&ms.done[i], 1);
            for (int h = 0; h < 2; ++h) mbar_init(&ms.row_unit[i][h], W::kRowWarps);
        }
        fence_mbar_init();
    }
    if (tid == 32) prefetch_maps(maps);
    if (warp == 8) tmem_alloc(&ms.tmem, 512);
    wait_prior_kernel();
    allow_next_kernel();
    if (tid < 2) p.parts[2 * cta + tid].state = 0;
    if (warp == 10) {
        Cursor a, z;
        const bool has = find_piece(p, cta, int(gridDim.x), lane, a, z);
        if (lane == 0) ms.piece[0] = a, ms.piece[1] = z, ms.has = has, ms.rows_gave_up[0] = ms.rows_gave_up[1] = 0;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = ms.tmem;
    uint32_t *err = p.b.err;
    bool ok = true;  // of this thread's waits

    if (warp < 8) {
        set_regs<W::kSoftmax, W::kLaunch>();
        if (ms.has) {
            // ---- softmax: thread = row -------------------------------------------------
            const int s = warp >> 2, row = tid & 127;
            const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
            const uint32_t t_s = tm + lanes + uint32_t(s) * 128u, t_o = tm + lanes + 256u + uint32_t(s) * 128u;
            const int r = (kByKeys ? 0 : s * kSideRows) + row;
            ItemWalk walk(ms.piece[0], ms.piece[1]);
            Item it = {};
            uint32_t n_s = 0, n_it = 0, tile_base = 0;  // tiles and items so far: barrier phases
            // O holds this side's products up to half h of its n-th tile
            auto wait_o = [&](uint32_t n, int h) {
                wait_for(ok, &ms.pv_done[s][h], n & 1, err);
                __syncwarp();
                tc_fence_after();
            };
            while (walk.next(p, it)) {
                const int nv = side_tiles<kByKeys>(it, s);
                const int lim = it.ctx + it.tok0 + p.token_of(min(r, it.rows - 1));  // last key this row sees
                const bool live = r - lane < it.rows;  // this warp has rows of the item
                float ref = -INFINITY, l = 0.f, scale = p.scale_log2;
                if constexpr (kE4m3) {
                    if (nv > 0) {
                        // by item parity: Q may be an item ahead of this side's threads, never two
                        const int qi = kByKeys ? 0 : s;
                        wait_for(ok, &ms.row_unit[qi][n_it & 1], (n_it >> 1) & 1, err);
                        // (never 0, which would make NaN of a masked score: rows of zeros have 2^-126 as their scale)
                        scale = fmaxf(scale * sc8.q_unit[n_it & 1][qi][row], 0x1p-149f);
                    }
                    if (kByKeys || nv > 0) ++n_it;
                }
                int page = peek_page(p, it, it.k0 + side_tile<kByKeys>(s, 0) * KT, lane);
                for (int v = 0; v < nv; ++v, ++n_s) {
                    const int t = side_tile<kByKeys>(s, v), kb = it.k0 + t * KT;
                    const uint32_t absent = absent_groups(p, page);
                    page = peek_page(p, it, it.k0 + side_tile<kByKeys>(s, v + 1) * KT, lane);
                    const bool check = partly_seen(it, kb, absent);
                    const uint32_t tg = tile_base + uint32_t(t);
                    if constexpr (kE4m3) wait_tile(ok, ms.unit_full, tg, err);
#pragma unroll 1
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t t_h = t_s + uint32_t(h) * KH;
                        const int kh = kb + h * KH;
                        // Scores of a half are issued after its last product, so a half's barriers are
                        // never more than a phase ahead.
                        wait_for(ok, &ms.s_full[s][h], n_s & 1, err);
                        __syncwarp();
                        tc_fence_after();
                        if (live) {
                            float x[KH];
#pragma unroll
                            for (int c = 0; c < KH; c += 32) tmem_ld32(t_h + uint32_t(c), x + c);
                            float4 unit[8];
                            if constexpr (kE4m3) load_units(unit, &sc8.k_unit[tg % kUnits][h * KH]);
                            tmem_wait_ld();
                            if constexpr (kE4m3) {
                                scale_keys(&x[0], unit);
                                load_units(unit, &sc8.k_unit[tg % kUnits][h * KH + 32]);
                                scale_keys(&x[32], unit);
                            }
                            if (check) {
#pragma unroll
                                for (int c = 0; c < KH; ++c)
                                    if (kh + c > lim || (absent >> (h * (KH / 16) + c / 16) & 1)) x[c] = -INFINITY;
                            }
                            const bool started = v > 0 || h > 0;  // O is new with the first product
                            // the reference moves up to a row's maximum in x, where that is more than `slack` above it
                            auto move_ref = [&](float slack) {
                                float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                                for (int c = 4; c < KH; c += 8)
#pragma unroll
                                    for (int i = 0; i < 4; ++i)
                                        mx[i] = c + 4 + i < KH ? fmaxf(fmaxf(mx[i], x[c + i]), x[c + 4 + i]) : fmaxf(mx[i], x[c + i]);
                                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale;
                                const bool move = top > ref + slack;
                                if (!__any_sync(0xffffffffu, move)) return;
                                const float to = move ? top : ref, f = move ? ex2(ref - to) : 1.f;
                                if (started) {
                                    wait_o(h == 0 ? n_s - 1 : n_s, h ^ 1);
#pragma unroll 1
                                    for (int c = 0; c < D; c += 16) {
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
                                for (int c = 0; c < KH; c += 32) {
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
                            float sum_h;
                            if constexpr (kE4m3) {
                                move_ref(kRefSlack);
                                sum_h = weigh();
                            } else {
                                sum_h = weigh();
                                // past the limit (or NaN), or a row without a reference yet
                                if (__any_sync(0xffffffffu, !(sum_h <= kSumLimit) || ref == -INFINITY)) {
                                    move_ref(0.f);
                                    tmem_wait_st();
                                    sum_h = weigh();
                                }
                            }
                            tmem_wait_st();
                            l += sum_h;
                            if (check) {
                                wait_tile(ok, kE4m3 ? ms.v_full : ms.clean, tg, err);
                                ok = __all_sync(0xffffffffu, ok);
                                const uint32_t *odd = &ms.odd[tg % kBars][h * (KH / 32)];
                                if (ok && any_odd(odd)) {
                                    if (started) wait_o(h == 0 ? n_s - 1 : n_s, h ^ 1);
                                    const Item copy = it;
                                    add_odd_rows<D, kE4m3>(p, copy, kh, lim, odd, t_h, t_o, !started);
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
                if (nv > 0) wait_o(n_s - 1, 1);
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
                    const bool wide = ((reinterpret_cast<uintptr_t>(p.out) | uintptr_t(p.out_stride * 2)) & 31) == 0;
                    const int dim = head_dim<D>(p);
                    float *data = p.part_data + (size_t(cta) * 2 + it.slot()) * size_t(BM) * size_t(dim + 2);
                    __nv_bfloat16 *dst =
                        static_cast<__nv_bfloat16 *>(p.out) + it.at(min(r, it.rows - 1), p, p.out_stride, dim);
#pragma unroll 2
                    for (int c = 0; c < dim; c += 16) {
                        float o[16];
                        tmem_ld16(t_o + uint32_t(c), o);
                        if (kByKeys && nv_other > 0) {
                            float o1[16];
                            tmem_ld16(t_o + 128u + uint32_t(c), o1);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = o[i] * f0 + o1[i] * f1;
                        } else {
                            tmem_wait_ld();
                        }
                        if (!writes) continue;
                        if (whole) {
                            uint32_t w[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) w[i] = pack_bf16(o[2 * i] * inv, o[2 * i + 1] * inv);
                            if (wide) {
                                store32(dst + c, w);
                            } else {
                                *reinterpret_cast<uint4 *>(dst + c) = make_uint4(w[0], w[1], w[2], w[3]);
                                *reinterpret_cast<uint4 *>(dst + c + 8) = make_uint4(w[4], w[5], w[6], w[7]);
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 16; i += 8) {
                                uint32_t w[8];
#pragma unroll
                                for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(o[i + e]);
                                store32(data + size_t(r) * size_t(dim) + c + i, w);
                            }
                        }
                    }
                    if (!whole) {
                        if (writes) data[BM * dim + r] = ref, data[BM * dim + BM + r] = l;
                        if (s == 0 && row == 0) p.parts[2 * cta + it.slot()] = it.part();
                    }
                }
                tc_fence_before();  // the next item's products rewrite O
                if (kByKeys) named_sync<1, 256>();
            }
        }
    } else if (warp < 12) {
        set_regs<W::kIssue, W::kLaunch>();
        if (ms.has && warp < 10) {
            // ---- products of a side (converged warp, one lane issues) ----------------------
            const int s = warp - 8;
            const uint32_t id_s = kE4m3 ? idesc_e4m3_f32(128, KH) : idesc_bf16_f32(128, KH);
            const uint32_t id_o = idesc_bf16_f32(128, D, false, true);
            const uint32_t t_s = tm + uint32_t(s) * 128u, t_o = tm + 256u + uint32_t(s) * 128u;
            const int qi = kByKeys ? 0 : s;  // the image of Q
            const uint32_t q_at = smem_u32(smem) + uint32_t(qi) * C::kQBytes;
            const uint64_t q_desc = kE4m3 ? sdesc_row8<D>(q_at) : sdesc_sw128(q_at);
            const uint64_t k_desc = kE4m3 ? sdesc_row8<D>(smem_u32(k_ring)) : sdesc_sw128(smem_u32(k_ring));
            const uint64_t v_desc = sdesc_sw128_mn(smem_u32(v_ring), KT * 128u);
            ItemWalk walk(ms.piece[0], ms.piece[1]);
            Item it = {};
            uint32_t base = 0, n_q = 0, n_p = 0;
            int nv = 0;
            // scores of half h of the side's v-th tile (descriptors count 16-byte units)
            auto scores = [&](int v, int h) {
                const uint32_t tg = base + uint32_t(side_tile<kByKeys>(s, v));
                if (h == 0) wait_tile(ok, ms.k_full, tg, err);
                if (!(ok = __all_sync(0xffffffffu, ok))) return;
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t t_h = t_s + uint32_t(h) * KH;
                    const uint64_t kd = k_desc + uint64_t(tg % NK * uint32_t(C::kKBytes >> 4)) +
                                        uint64_t(h * (KH * (kE4m3 ? D : 128) >> 4));
                    if constexpr (kE4m3) {
#pragma unroll
                        for (int k = 0; k < 2 * D / 32; ++k)  // both terms of Q against the same keys
                            mma_e4m3(t_h, q_desc + uint64_t((k / (D / 32)) * (kSideRows * D / 16) + (k % (D / 32)) * 2),
                                     kd + uint64_t((k % (D / 32)) * 2), id_s, k > 0);
                    } else {
#pragma unroll
                        for (int k = 0; k < D / 16; ++k)
                            mma_bf16(t_h, q_desc + uint64_t((k >> 2) * (kSideRows * 8) + (k & 3) * 2),
                                     kd + uint64_t((k >> 2) * (KT * 8) + (k & 3) * 2), id_s, k > 0);
                    }
                    mma_commit(&ms.s_full[s][h]);
                    if (h == 1) {
                        mma_commit(&ms.k_empty[tg % kBars]);
                        if (v + 1 == nv) mma_commit(&ms.q_free[qi]);
                    }
                }
                __syncwarp();
            };
            while (ok && walk.next(p, it)) {
                nv = side_tiles<kByKeys>(it, s);
                if (kByKeys || nv > 0) wait_for(ok, &ms.q_full[qi], n_q++ & 1, err);
                if (nv > 0) {
                    scores(0, 0), scores(0, 1);
                } else if (kByKeys) {
                    if (!(ok = __all_sync(0xffffffffu, ok))) break;
                    if (lane == 0) mbar_arrive(&ms.q_free[0]);
                }
                for (int v = 0; v < nv && ok; ++v, ++n_p) {
                    const uint32_t tg = base + uint32_t(side_tile<kByKeys>(s, v));
                    wait_tile(ok, ms.v_full, tg, err);
                    if (!kE4m3) wait_tile(ok, ms.clean, tg, err);
                    // the first product starts O, unless value rows were added to it by hand
                    const uint32_t acc = v > 0 || any_odd(ms.odd[tg % kBars]);
                    const uint64_t vd = v_desc + uint64_t(tg % NV * uint32_t(C::kVBytes >> 4));
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        wait_for(ok, &ms.p_ready[s][h], n_p & 1, err);
                        if (!(ok = __all_sync(0xffffffffu, ok))) break;
                        tc_fence_after();
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < KH / 16; ++k)
                                mma_bf16_ta(t_o, t_s + uint32_t(h) * KH + uint32_t(k) * 8u,
                                            vd + uint64_t((h * (KH / 16) + k) * 128), id_o, h > 0 || k > 0 || acc);
                            mma_commit(&ms.pv_done[s][h]);
                            if (h == 1) mma_commit(&ms.v_empty[tg % kBars]);
                        }
                        __syncwarp();
                        if (v + 1 < nv) scores(v + 1, h);
                    }
                }
                if (!kByKeys && nv == 0) {  // a tile is free once both sides have said so
                    for (int i = 0; i < item_tiles(it) && ok; ++i) {
                        const uint32_t tg = base + uint32_t(i);
                        wait_tile(ok, ms.k_full, tg, err);
                        wait_tile(ok, ms.v_full, tg, err);
                        if (!(ok = __all_sync(0xffffffffu, ok))) break;
                        if (lane == 0) mbar_arrive(&ms.k_empty[tg % kBars]), mbar_arrive(&ms.v_empty[tg % kBars]);
                    }
                }
                base += uint32_t(item_tiles(it));
            }
            // nothing of this side's is in flight when the tensor memory goes
            if (elect_one()) mma_commit(&ms.done[s]);
            __syncwarp();
            mbar_wait(&ms.done[s], 0, err);
        } else if (ms.has) {
            // ---- page fetches: keys, or values ------------------------------------------------
            fetch_pages<D, kE4m3>(p, maps, ms.piece[0], ms.piece[1], warp == 11, ok, [&](uint32_t t, bool values) {
                if (!values) {
                    wait_stage<NK>(ok, ms.k_empty, t, err);
                    return Landing{&ms.k_full[t % kBars], k_ring + t % NK * C::kKBytes, sc8.k[t % NK]};
                }
                if constexpr (kE4m3) {
                    wait_stage<NR>(ok, ms.raw_empty, t, err);
                    return Landing{&ms.raw_full[t % kBars], raw_ring + t % NR * C::kRawBytes, sc8.v[t % NR]};
                }
                wait_stage<NV>(ok, ms.v_empty, t, err);
                return Landing{&ms.v_full[t % kBars], v_ring + t % NV * C::kVBytes, nullptr};
            }, warp == 11 ? (kE4m3 ? ms.raw_full : ms.v_full) : ms.k_full, warp == 11 ? (kE4m3 ? NR : NV) : NK);
        }
    } else {
        set_regs<W::kRows, W::kLaunch>();
        if (ms.has) {
            // ---- rows of Q; value tiles looked over, and (e4m3) made bf16 ---------------------
            const int w = warp - 12, qt = tid - 384;
            constexpr int kRowThreads = W::kRowWarps * 32;
            ItemWalk walk(ms.piece[0], ms.piece[1]);
            Item it = {};
            uint32_t n_q[2] = {0, 0}, tile = 0;
            // Only the first of these warps waits by polling, which takes issue slots; the others
            // meet it at a barrier of the hardware's, and learn there whether it gave up.
            // (by turns two words: the first may be an appointment ahead of a warp that still reads)
            uint32_t turn = 0;
            auto meet = [&] {
                if (w == 0 && !ok) ms.rows_gave_up[turn] = 1;
                named_sync<4, kRowThreads>();
                ok = ms.rows_gave_up[turn] == 0;
                turn ^= 1;
            };
            while (ok && walk.next(p, it)) {
                for (int s = 0; s < C::kQImages; ++s) {
                    if (side_tiles<kByKeys>(it, s) == 0) continue;
                    unsigned char *q_img = smem + s * C::kQBytes;
                    constexpr int CPR = D / 8, RPP = kRowThreads / CPR;  // 16-byte pieces of a row, rows a pass
                    const int c = qt % CPR, dim = head_dim<D>(p);
                    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.q) + c * 8;
                    auto row_at = [&](int row) {  // this thread's piece of a row of the item
                        return q + it.at(min((kByKeys ? 0 : s * kSideRows) + row, it.rows - 1), p, p.q_stride, dim);
                    };
                    auto is_there = [&](int row) { return (kByKeys ? 0 : s * kSideRows) + row < it.rows && c * 8 < dim; };
                    auto wait_image = [&] {  // the last item's scores have read it
                        if (w == 0) wait_for(ok, &ms.q_free[s], (n_q[s] & 1) ^ 1, err);
                        meet();
                    };
                    if constexpr (kE4m3) {
                        // a row as 2^e (q1 + q2): e4m3 keeps 4 significant bits, so q1 and what q1 leaves
                        // hold all 8 of a bf16 (down to 2^-18 of the row's largest value)
                        constexpr int kBatch = 4;
#pragma unroll 1
                        for (int r0 = qt / CPR; r0 < kSideRows; r0 += RPP * kBatch) {
                            uint4 raw[kBatch];
#pragma unroll
                            for (int b = 0; b < kBatch; ++b) {
                                const int row = r0 + b * RPP;
                                raw[b] = is_there(row) ? *reinterpret_cast<const uint4 *>(row_at(row)) : make_uint4(0, 0, 0, 0);
                            }
                            if (r0 < RPP) wait_image();
                            if (!ok) break;
                            int e[kBatch];
                            row_exponents<CPR>(raw, e);
#pragma unroll
                            for (int b = 0; b < kBatch; ++b) {
                                const int row = r0 + b * RPP;
                                uint32_t w1[2], w2[2];
                                split_row(raw[b], e[b], w1, w2);
                                const uint32_t at = row8_piece<D>(row, c >> 1) + uint32_t(c & 1) * 8u;
                                *reinterpret_cast<uint2 *>(q_img + at) = make_uint2(w1[0], w1[1]);
                                *reinterpret_cast<uint2 *>(q_img + kSideRows * D + at) = make_uint2(w2[0], w2[1]);
                                if (c == 0) sc8.q_unit[n_q[s] & 1][s][row] = exp2_biased(e[b] < 0 ? 127 : e[b]);
                            }
                        }
                        __syncwarp();
                        if (ok && lane == 0) mbar_arrive(&ms.row_unit[s][n_q[s] & 1]);
                    } else {
                        wait_image();
                        if (ok) {
#pragma unroll 4
                            for (int row = qt / CPR; row < kSideRows; row += RPP)
                                cp_async16_or_zero(q_img + sw128_chunk(row, c, kSideRows), row_at(row), is_there(row));
                            cp_async_wait_all();
                        }
                    }
                    if (!ok) break;
                    ++n_q[s];
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ms.q_full[s]);
                }
                int page = peek_page(p, it, it.k0, lane);
                for (int kb = it.k0; kb < it.k1 && ok; kb += KT, ++tile) {
                    const uint32_t absent = absent_groups(p, page);
                    page = peek_page(p, it, kb + KT, lane);
                    unsigned char *dst = v_ring + tile % NV * C::kVBytes;
                    if (w == 0) {
                        if constexpr (kE4m3) {
                            wait_tile(ok, ms.k_full, tile, err), wait_tile(ok, ms.raw_full, tile, err);
                            wait_stage<NV>(ok, ms.v_empty, tile, err);
                        } else {
                            wait_tile(ok, ms.v_full, tile, err);
                        }
                    }
                    meet();
                    if (!ok) break;
                    if constexpr (kE4m3) {
                        if (qt < KT) sc8.k_unit[tile % kUnits][qt] = exp2_biased(sc8.k[tile % NK][qt]);  // as numbers
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&ms.unit_full[tile % kBars]), mbar_arrive(&ms.k_empty[tile % kBars]);
                        widen_tile<D>(p, it, kb, absent, raw_ring + tile % NR * C::kRawBytes, dst, sc8.v[tile % NR], w, lane,
                                      ms.odd[tile % kBars]);
                        if (lane == 0) mbar_arrive(&ms.v_full[tile % kBars]), mbar_arrive(&ms.raw_empty[tile % kBars]);
                    } else {
                        look_over_tile<D>(it, kb, absent, dst, w, lane, ms.odd[tile % kBars]);
                        if (lane == 0) mbar_arrive(&ms.clean[tile % kBars]);
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 8) tmem_dealloc(tm, 512);
}

template <int D, bool kE4m3, bool kByKeys>
kda_status launch(const kda_kv_cache *c, AttendParams &p, const AttendPlan &plan, cudaStream_t stream) {
    using C = Cfg<D, kE4m3, kByKeys>;
    TileMaps maps;
    if (!page_map(&maps.k, c->k, c, kE4m3) || !page_map(&maps.v, c->v, c, kE4m3)) return KDA_ERR_CUDA;
    auto kern = attend_tile_kernel<D, kE4m3, kByKeys>;
    constexpr size_t smem = smem_bytes<C, kE4m3>();
    static_assert(smem <= 232448, "shared memory of a CTA");
    if (!allow_smem<attend_tile_kernel<D, kE4m3, kByKeys>>(int(smem))) return KDA_ERR_CUDA;
    p.key_step = KT;
    p.item_cost = kItemCost;
    p.min_keys = (kByKeys ? 2 : 1) * KT;
    const ProfScope prof(KDA_KERNEL_KV_ATTEND, stream);
    return launch_overlapped(kern, dim3(unsigned(plan.n_cta)), Warps<kE4m3>::kThreads, smem, stream, p, maps);
}

template <int D>
kda_status by_type(const kda_kv_cache *c, AttendParams &p, const AttendPlan &plan, cudaStream_t s) {
    const bool by_keys = plan.bm == kSideRows;
    if (c->format == KDA_KV_E4M3)
        return by_keys ? launch<D, true, true>(c, p, plan, s) : launch<D, true, false>(c, p, plan, s);
    return by_keys ? launch<D, false, true>(c, p, plan, s) : launch<D, false, false>(c, p, plan, s);
}

}  // namespace

// Sides by keys up to a side's rows, by rows past it: 32 sequences of 4000 to 8192
// tokens, 128 rows an item, take 145 us by keys and 153 by rows (e4m3 160 and 191),
// 16 of them with 136 rows 138 and 107.
bool tile_plan(const kda_kv_cache *c, const kda_kv_batch *b, AttendPlan *plan) {
    const long long rows = static_cast<long long>(b->max_new) * (c->num_heads / c->num_kv_heads);
    if (c->act != KDA_BF16) return false;
    plan->bm = rows <= kSideRows ? kSideRows : 2 * kSideRows;
    plan->n_cta = sm_count();
    return true;
}

kda_status tile_launch(const kda_kv_cache *c, AttendParams &p, const AttendPlan &plan, cudaStream_t stream) {
    return c->head_dim <= 64 ? by_type<64>(c, p, plan, stream) : by_type<128>(c, p, plan, stream);
}

}  // namespace kv
}  // namespace kda
