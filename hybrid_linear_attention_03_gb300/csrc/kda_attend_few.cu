// kda_attend_few.cu -- kda_kv_attend for bf16 rows and few of them: decode, at
// most 16 rows an item (query heads of one cache head x new tokens), head size
// 128.
//
// HBM bounds these calls, if nothing around the cache's bytes is slower.  So the
// products are turned: keys and value channels, of which there are always 128,
// take the tensor cores' long side, and the few rows the short one,
//   X^T = K Q^T  (128 keys x 16 rows),   O^T += V^T P^T  (128 channels x 16 rows),
// which costs an eighth of what the tile kernel spends on them, and spreads a
// row's exponentials over the 128 threads of a key tile.  Softmax in one pass as
// in kda_attend_tile.cu: a row's reference is its maximum at the time it was last
// moved, and only moves when a score exceeds it by more than 8 (then the 4 warps
// meet, find the maxima over the keys and rescale O); until then a tile costs one
// vote.  Weights go to shared memory as bf16 (rows x keys), scores and weights are
// double-buffered, sums stay with each thread's keys up to the item's end.
// Measured, 64 heads over 8 cache heads: 64 sequences of 4001 to 16384 tokens
// 398 us (6.7 TB/s, 99 % of the measured copy rate); the same in e4m3 318 us
// (4.2 TB/s: widening the values and storing the weights bound it) against 447 with
// the tile kernel; one sequence of 65536 in e4m3 46 us, of 1024 in bf16 13 us (launch,
// one tile a CTA and the joining of parts).
// The border at 16 rows, us here and with the tile kernel: 128 sequences of 100 to 1500
// tokens 91 and 100 (1 row: 83 and 97), in e4m3 107 and 146; 32 sequences of 8001 to 16384
// 241 and 236 (1 row: 238 and 233), in e4m3 192 and 242.  So bf16 over long caches is level
// from the first row on.  With 32 or 64 rows a thread's share of a tile grows and the
// tile kernel is ahead everywhere (247 against 237 us at 32 rows over 8K to 16K).
//
// Warps: 0-3 softmax (a thread a key, later a channel), 4 issues the products, 5
// and 6 fetch pages by TMA, 8-11 bring the rows of Q and look value tiles over, as in
// kda_attend_tile.cu.  e4m3 pages: keys meet Q as two e4m3 terms, eight row warps
// widen the values, and these slow the softmax so much that it takes two groups of
// four warps, one for the tiles of either parity, each with references, sums and
// an O of its own, joined at an item's end (359 us with one group).
#include "kda_attend_tc.cuh"

namespace kda {
namespace kv {
namespace {

constexpr int D = 128, N = 16;  // channels, rows of an item
constexpr float kRefSlack = 8.f;
// Keys that take as long as an item's start and output.  Measured at 0, 128, 256,
// 1024: 128 sequences of 100 to 1500 tokens take 101, 93, 89, 90 us.
constexpr int kItemCost = 256;

template <bool kE4m3> struct Cfg {
    // e4m3: two groups of softmax warps, one for the tiles of either parity
    static constexpr int kGroups = kE4m3 ? 2 : 1, kSoftWarps = 4 * kGroups, kRowWarps = kE4m3 ? 8 : 4;
    static constexpr int kThreads = (kSoftWarps + 4 + kRowWarps) * 32;
    // registers a thread at launch and after the split (e4m3 only)
    static constexpr int kLaunch = 96, kSoftmax = 136, kIssue = 56, kRows = 72;
    static_assert(!kE4m3 || kSoftWarps * kSoftmax + 4 * kIssue + kRowWarps * kRows <= kThreads / 32 * kLaunch,
                  "the split takes no more than the launch has");
    static constexpr int kQBytes = N * D * 2;  // bf16, or two e4m3 terms
    static constexpr int kPBytes = N * KT * 2;
    static constexpr int kKBytes = KT * D * (kE4m3 ? 1 : 2), kVBytes = KT * D * 2, kRawBytes = KT * D;
    static constexpr int kStagesK = kE4m3 ? 4 : 3;
    static constexpr int kStagesV = kE4m3 ? 2 : 3;
    static constexpr int kStagesRaw = kE4m3 ? 4 : 1;
    static constexpr int kPAt = kQBytes;
    static constexpr int kKAt = kPAt + 2 * kPBytes;
    static constexpr int kVAt = kKAt + kStagesK * kKBytes;
    static constexpr int kRawAt = kVAt + kStagesV * kVBytes;
    static constexpr int kMiscAt = kRawAt + (kE4m3 ? kStagesRaw * kRawBytes : 0);
    static constexpr int kColumns = 64;  // tensor memory: scores by tile parity, O by group
    static_assert(kStagesK < kBars && kStagesV < kBars && kStagesRaw < kBars, "a tile's barrier is free before its stage");
};

template <typename C> struct alignas(16) Misc {
    uint64_t k_full[kBars], k_empty[kBars], v_full[kBars], v_empty[kBars], clean[kBars], raw_full[kBars], raw_empty[kBars];
    uint64_t s_full[2], p_ready[2], pv_done[2];  // by tile parity
    uint64_t q_full, q_free, done;
    uint64_t row_unit[2];  // by item parity
    uint32_t tmem;
    int has, rows_gave_up[2];
    Cursor piece[2];
    uint32_t odd[kBars][4];                  // by tile: keys whose value row was taken out of it
    alignas(16) uint8_t k_scale[C::kStagesK][KT];  // e4m3: the tiles' scale exponents
    alignas(16) uint8_t v_scale[C::kStagesRaw][KT];
    alignas(16) float row_scale[2][N];       // by item parity: scale * log2(e), with e4m3 times the row's scale
    // by group: rows' references, what the last move scaled by, and (by warp) maxima, then sums
    alignas(16) float ref[2][N], back[2][N];
    float tops[2][4][N];
    // an item's end, by group (the first for an item of both): the rows' factors of either group's O, their
    // sums and references
    alignas(16) float f[2][2][N], sum[2][N], top[2][N];
};

template <typename C> constexpr size_t smem_bytes() { return 1024 + C::kMiscAt + sizeof(Misc<C>); }

// Barriers of the hardware's: 1 and 2 the votes, 3 and 4 the meetings of a group's 128 threads, 5 the
// row warps, 6 both groups.
__device__ __forceinline__ void meet_128(int g) { asm volatile("bar.sync %0, 128;" ::"r"(3 + g) : "memory"); }
// Whether any of a group's 128 softmax threads says so (which all meet here).
__device__ __forceinline__ bool any_of_128(bool mine, int g) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(uint32_t(mine)), "r"(1 + g)
        : "memory");
    return r != 0;
}

// Joins 16 values a lane over the warp's lanes, halving the values with each
// step: 16 shuffles instead of 80.  Lane l gets that of value l / 2.
template <typename Op> __device__ __forceinline__ float join_lanes(const float (&v)[N], int lane, Op op) {
    float a[8];
    const bool b4 = lane & 16, b3 = lane & 8, b2 = lane & 4, b1 = lane & 2;
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = op(b4 ? v[i + 8] : v[i], __shfl_xor_sync(0xffffffffu, b4 ? v[i] : v[i + 8], 16));
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = op(b3 ? a[i + 4] : a[i], __shfl_xor_sync(0xffffffffu, b3 ? a[i] : a[i + 4], 8));
#pragma unroll
    for (int i = 0; i < 2; ++i) a[i] = op(b2 ? a[i + 2] : a[i], __shfl_xor_sync(0xffffffffu, b2 ? a[i] : a[i + 2], 4));
    a[0] = op(b1 ? a[1] : a[0], __shfl_xor_sync(0xffffffffu, b1 ? a[0] : a[1], 2));
    return op(a[0], __shfl_xor_sync(0xffffffffu, a[0], 1));
}

template <bool kE4m3>
__global__ void __launch_bounds__(Cfg<kE4m3>::kThreads, 1)
    attend_few_kernel(const __grid_constant__ AttendParams p, const __grid_constant__ TileMaps maps) {
    using C = Cfg<kE4m3>;
    constexpr int kG = C::kGroups, kMma = C::kSoftWarps, kRow0 = kMma + 4;  // groups; first warps of the other roles
    constexpr int NK = C::kStagesK, NV = C::kStagesV, NR = C::kStagesRaw;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Misc<C> &ms = *reinterpret_cast<Misc<C> *>(smem + C::kMiscAt);
    const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5, cta = int(blockIdx.x);
    unsigned char *k_ring = smem + C::kKAt, *v_ring = smem + C::kVAt, *raw_ring = smem + C::kRawAt;

    if (tid == 0) {
        for (int i = 0; i < kBars; ++i) {
            mbar_init(&ms.k_full[i], 1), mbar_init(&ms.k_empty[i], kE4m3 ? 5 : 1);  // and the scales read
            mbar_init(&ms.v_full[i], kE4m3 ? C::kRowWarps : 1), mbar_init(&ms.v_empty[i], 1);
            mbar_init(&ms.clean[i], C::kRowWarps);
            mbar_init(&ms.raw_full[i], 1), mbar_init(&ms.raw_empty[i], C::kRowWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ms.s_full[i], 1), mbar_init(&ms.p_ready[i], 4), mbar_init(&ms.pv_done[i], 1);
            mbar_init(&ms.row_unit[i], C::kRowWarps);
        }
        mbar_init(&ms.q_full, C::kRowWarps), mbar_init(&ms.q_free, 1), mbar_init(&ms.done, 1);
        fence_mbar_init();
    }
    if (tid == 32) prefetch_maps(maps);
    if (warp == kMma) tmem_alloc(&ms.tmem, C::kColumns);
    wait_prior_kernel();
    allow_next_kernel();
    if (tid < 2) p.parts[2 * cta + tid].state = 0;
    if (warp == kMma + 1) {
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

    if (warp < kMma) {
        if constexpr (kE4m3) set_regs<C::kSoftmax, C::kLaunch>();
        if (ms.has) {
            // ---- softmax of a group's tiles: thread = key of the tile; at an item's end = channel ----
            const int g = kG == 2 ? warp >> 2 : 0, key = tid & 127;
            const uint32_t lanes = uint32_t(warp % 4 * 32) << 16;
            const uint32_t t_o = tm + lanes + 2u * N + uint32_t(g) * N;
            float *ref = ms.ref[g], *back = ms.back[g];
            ItemWalk walk(ms.piece[0], ms.piece[1]);
            Item it = {};
            uint32_t base = 0, n_it = 0;  // tiles and items so far
            // O holds the product of this group's tile t
            auto wait_o = [&](uint32_t t) {
                wait_for(ok, &ms.pv_done[t & 1], (t >> 1) & 1, err);
                __syncwarp();
                tc_fence_after();
            };
            for (; walk.next(p, it); ++n_it) {
                const int first_lim = it.ctx + it.tok0, nt = item_tiles(it), v0 = kG == 2 ? int(base & 1) ^ g : 0;
                const uint32_t tile0 = base;
                base += uint32_t(nt);
                if (v0 >= nt) continue;  // one tile, of the other group
                // (a group sits out one item at most, so it misses no phase that could be mistaken)
                wait_for(ok, &ms.row_unit[n_it & 1], (n_it >> 1) & 1, err);
                __syncwarp();
                const float *row_scale = ms.row_scale[n_it & 1];
                if (key < N) ref[key] = -INFINITY;
                float l[N];
#pragma unroll
                for (int c = 0; c < N; ++c) l[c] = 0.f;
                meet_128(g);
                uint32_t tile = tile0 + uint32_t(v0);
                int page = peek_page(p, it, it.k0 + v0 * KT, lane);
                for (int v = v0; v < nt; v += kG, tile += kG) {
                    const bool started = v >= kG;  // O is new with the first product
                    const int kb = it.k0 + v * KT, j = kb + key;
                    const uint32_t absent = absent_groups(p, page);
                    const bool check = partly_seen(it, kb, absent);
                    page = peek_page(p, it, kb + kG * KT, lane);
                    int hidden = 0;  // rows before this one do not see the thread's key
                    if (check) {
                        hidden = max(j - first_lim, 0) * p.group;
                        if (j >= it.k1 || (absent >> (key / 16) & 1)) hidden = N;
                    }
                    float unit = 1.f;
                    if constexpr (kE4m3) {
                        wait_tile(ok, ms.k_full, tile, err);
                        unit = exp2_biased(ms.k_scale[tile % NK][key]);
                        __syncwarp();
                        if (ok && lane == 0) mbar_arrive(&ms.k_empty[tile % kBars]);
                    }
                    wait_for(ok, &ms.s_full[tile & 1], (tile >> 1) & 1, err);
                    __syncwarp();
                    tc_fence_after();
                    float x[N];
                    tmem_ld16(tm + lanes + (tile & 1) * N, x);
                    tmem_wait_ld();
                    bool over = false;
#pragma unroll
                    for (int i = 0; i < N; i += 4) {
                        const float4 f = *reinterpret_cast<const float4 *>(row_scale + i);
                        const float4 r = *reinterpret_cast<const float4 *>(ref + i);
                        x[i] *= f.x * unit, x[i + 1] *= f.y * unit, x[i + 2] *= f.z * unit, x[i + 3] *= f.w * unit;
                        if (check) {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (i + e < hidden) x[i + e] = -INFINITY;
                        }
                        over |= x[i] > r.x + kRefSlack || x[i + 1] > r.y + kRefSlack || x[i + 2] > r.z + kRefSlack ||
                                x[i + 3] > r.w + kRefSlack;
                    }
                    if (any_of_128(over, g)) {
                        const float m = join_lanes(x, lane, [](float a, float b) { return fmaxf(a, b); });
                        if ((lane & 1) == 0) ms.tops[g][warp % 4][lane >> 1] = m;
                        meet_128(g);
                        if (key < N) {
                            const float top = fmaxf(fmaxf(ms.tops[g][0][key], ms.tops[g][1][key]),
                                                    fmaxf(ms.tops[g][2][key], ms.tops[g][3][key]));
                            const float was = ref[key], to = top > was + kRefSlack ? top : was;
                            ref[key] = to;
                            back[key] = to == was ? 1.f : ex2(was - to);
                        }
                        meet_128(g);
                        float o[N];
                        if (started) {
                            wait_o(tile - kG);
                            tmem_ld16(t_o, o);
                            tmem_wait_ld();
                        }
#pragma unroll
                        for (int i = 0; i < N; ++i) l[i] *= back[i], o[i] = started ? o[i] * back[i] : 0.f;
                        if (started) {
                            tmem_st16(t_o, o);
                            tmem_wait_st();
                        }
                    }
                    // the weights of the tile before the last one have been used: theirs is the place
                    if (tile >= 2) wait_for(ok, &ms.pv_done[tile & 1], ((tile - 2) >> 1) & 1, err);
                    __syncwarp();
                    unsigned char *p_img = smem + C::kPAt + (tile & 1) * C::kPBytes;
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        const float r = ref[i], w = ex2(x[i] - (r == -INFINITY ? 0.f : r));
                        l[i] += w;
                        *reinterpret_cast<__nv_bfloat16 *>(p_img + sw128_offset(i, key, N)) = __float2bfloat16_rn(w);
                    }
                    if (check) {
                        wait_tile(ok, kE4m3 ? ms.v_full : ms.clean, tile, err);
                        ok = __all_sync(0xffffffffu, ok);
                        const uint32_t *odd = ms.odd[tile % kBars];
                        // (the group has to agree, and once it has met all weights are there)
                        if (any_of_128(ok && (odd[0] | odd[1] | odd[2] | odd[3]) != 0, g)) {
                            // value rows taken out of the tile: thread = channel adds them for the rows that see them
                            float o[N];
                            if (started) {
                                wait_o(tile - kG);
                                tmem_ld16(t_o, o);
                                tmem_wait_ld();
                            }
#pragma unroll
                            for (int i = 0; i < N; ++i) o[i] = started ? o[i] : 0.f;
                            for (int q = 0; q < 4; ++q) {
                                for (uint32_t left = ok ? odd[q] : 0u; left; left &= left - 1) {
                                    const int out = q * 32 + __ffs(left) - 1, jj = kb + out;
                                    const size_t vec =
                                        ((size_t(max(load_page(p.b, it.n, jj), 0)) * size_t(p.hkv) + size_t(it.h))
                                         << p.b.page_shift) +
                                        size_t(jj & ((1 << p.b.page_shift) - 1));
                                    float val;
                                    if constexpr (kE4m3)
                                        val = unpack_e4m3(static_cast<const uint8_t *>(p.pv)[vec * D + key]).x *
                                              exp2_biased(p.sv[vec]);
                                    else
                                        val = __bfloat162float(static_cast<const __nv_bfloat16 *>(p.pv)[vec * D + key]);
#pragma unroll
                                    for (int i = 0; i < N; ++i) {
                                        const float w = __bfloat162float(
                                            *reinterpret_cast<const __nv_bfloat16 *>(p_img + sw128_offset(i, out, N)));
                                        if (w != 0.f && first_lim + p.token_of(i) >= jj) o[i] = fmaf(w, val, o[i]);
                                    }
                                }
                            }
                            __syncwarp();
                            tmem_st16(t_o, o);
                            tmem_wait_st();
                        }
                    }
                    fence_proxy_async_smem();
                    tc_fence_before();
                    __syncwarp();
                    if (ok && lane == 0) mbar_arrive(&ms.p_ready[tile & 1]);
                }

                // ---- output: thread = channel; rows by turns where both groups had tiles ----------
                const bool both = kG == 2 && nt > 1;
                const int at_end = both ? 0 : g;
                const float own = join_lanes(l, lane, [](float a, float b) { return a + b; });
                if ((lane & 1) == 0) ms.tops[g][warp % 4][lane >> 1] = own;
                if (both) named_sync<6, 256>();
                else meet_128(g);
                const bool whole = it.whole();
                if (key < N && (!both || g == 0)) {
                    float s[2] = {0.f, 0.f}, m[2] = {-INFINITY, -INFINITY};
#pragma unroll
                    for (int e = 0; e < kG; ++e) {
                        if (!both && e != g) continue;
                        m[e] = ms.ref[e][key];
                        s[e] = (ms.tops[e][0][key] + ms.tops[e][1][key]) + (ms.tops[e][2][key] + ms.tops[e][3][key]);
                    }
                    const float top = fmaxf(m[0], m[1]), to = top == -INFINITY ? 0.f : top;
                    const float f0 = ex2(m[0] - to), f1 = ex2(m[1] - to), sum = f0 * s[0] + f1 * s[1];
                    const float inv = !whole ? 1.f : sum > 0.f || sum != sum ? 1.0f / sum : 0.f;
                    ms.f[at_end][0][key] = f0 * inv, ms.f[at_end][1][key] = f1 * inv;
                    ms.top[at_end][key] = top, ms.sum[at_end][key] = sum;
                }
                wait_o(tile - kG);
                tc_fence_before();  // and the other group's threads may read it
                if (both) named_sync<6, 256>();
                else meet_128(g);
                tc_fence_after();
                float *data = p.part_data + (size_t(cta) * 2 + it.slot()) * size_t(N) * (D + 2);
                float o[N], f[N];
                tmem_ld16(t_o, o);
                tmem_wait_ld();
#pragma unroll
                for (int r = 0; r < N; r += 4) {
                    const float4 t = *reinterpret_cast<const float4 *>(&ms.f[at_end][g][r]);
                    f[r] = t.x, f[r + 1] = t.y, f[r + 2] = t.z, f[r + 3] = t.w;
                }
#pragma unroll
                for (int r = 0; r < N; ++r) o[r] *= f[r];
                if (both) {
                    float o1[N];
                    tmem_ld16(tm + lanes + 2u * N + uint32_t(g ^ 1) * N, o1);
                    tmem_wait_ld();
#pragma unroll
                    for (int r = 0; r < N; r += 4) {
                        const float4 t = *reinterpret_cast<const float4 *>(&ms.f[at_end][g ^ 1][r]);
                        o[r] = fmaf(o1[r], t.x, o[r]), o[r + 1] = fmaf(o1[r + 1], t.y, o[r + 1]);
                        o[r + 2] = fmaf(o1[r + 2], t.z, o[r + 2]), o[r + 3] = fmaf(o1[r + 3], t.w, o[r + 3]);
                    }
                }
                if (whole) {
                    __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out) + it.at(0, p, p.out_stride, D) + key;
                    int head = 0;  // of the group
#pragma unroll
                    for (int r = 0; r < N; ++r) {
                        if (r >= it.rows) break;
                        if (!both || (r & 1) == g) *dst = __float2bfloat16_rn(o[r]);
                        dst += D;
                        if (++head == p.group) head = 0, dst += p.out_stride - static_cast<long long>(p.group) * D;
                    }
                } else {
#pragma unroll
                    for (int r = 0; r < N; ++r) {
                        if (r >= it.rows) break;
                        if (!both || (r & 1) == g) data[size_t(r) * D + key] = o[r];
                    }
                }
                if (!whole && (!both || g == 0)) {
                    if (key < it.rows) data[N * D + key] = ms.top[at_end][key], data[N * D + N + key] = ms.sum[at_end][key];
                    if (key == 0) p.parts[2 * cta + it.slot()] = it.part();
                }
                tc_fence_before();  // the next item's products rewrite O, and its start the references and sums
                if (both) named_sync<6, 256>();
                else meet_128(g);
            }
        }
    } else if (warp < kRow0) {
        if constexpr (kE4m3) set_regs<C::kIssue, C::kLaunch>();
        if (ms.has && warp == kMma) {
            // ---- products (converged warp, one lane issues; descriptors count 16-byte units) -------
            const uint32_t id_s = kE4m3 ? idesc_e4m3_f32(128, N) : idesc_bf16_f32(128, N);
            const uint32_t id_o = idesc_bf16_f32(128, N, true, false);
            const uint64_t q_desc = kE4m3 ? sdesc_row8<D>(smem_u32(smem)) : sdesc_sw128(smem_u32(smem));
            const uint64_t k_desc = kE4m3 ? sdesc_row8<D>(smem_u32(k_ring)) : sdesc_sw128(smem_u32(k_ring));
            const uint64_t v_desc = sdesc_sw128_mn(smem_u32(v_ring), KT * 128u);
            const uint64_t p_desc = sdesc_sw128(smem_u32(smem + C::kPAt));
            ItemWalk walk(ms.piece[0], ms.piece[1]);
            Item it = {};
            uint32_t base = 0, n_q = 0;
            int nt = 0;
            auto scores = [&](int v) {
                const uint32_t t = base + uint32_t(v);
                wait_tile(ok, ms.k_full, t, err);
                if (!(ok = __all_sync(0xffffffffu, ok))) return;
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t t_s = tm + (t & 1) * N;
                    const uint64_t kd = k_desc + uint64_t(t % NK * uint32_t(C::kKBytes >> 4));
                    if constexpr (kE4m3) {
#pragma unroll
                        for (int k = 0; k < 2 * D / 32; ++k)  // both terms of Q against the same keys
                            mma_e4m3(t_s, kd + uint64_t((k % (D / 32)) * 2),
                                     q_desc + uint64_t((k / (D / 32)) * (N * D / 16) + (k % (D / 32)) * 2), id_s, k > 0);
                    } else {
#pragma unroll
                        for (int k = 0; k < D / 16; ++k)
                            mma_bf16(t_s, kd + uint64_t((k >> 2) * (KT * 8) + (k & 3) * 2),
                                     q_desc + uint64_t((k >> 2) * (N * 8) + (k & 3) * 2), id_s, k > 0);
                    }
                    mma_commit(&ms.s_full[t & 1]);
                    mma_commit(&ms.k_empty[t % kBars]);
                    if (v + 1 == nt) mma_commit(&ms.q_free);
                }
                __syncwarp();
            };
            while (ok && walk.next(p, it)) {
                nt = item_tiles(it);
                wait_for(ok, &ms.q_full, n_q++ & 1, err);
                scores(0);
                if (ok && nt > 1) scores(1);
                for (int v = 0; v < nt && ok; ++v) {
                    const uint32_t t = base + uint32_t(v);
                    wait_tile(ok, ms.v_full, t, err);
                    if (!kE4m3) wait_tile(ok, ms.clean, t, err);
                    wait_for(ok, &ms.p_ready[t & 1], (t >> 1) & 1, err);
                    if (!(ok = __all_sync(0xffffffffu, ok))) break;
                    tc_fence_after();
                    // the first product of a group starts its O, unless value rows were added to it by hand
                    const uint32_t *odd = ms.odd[t % kBars];
                    const uint32_t acc = v >= kG || (odd[0] | odd[1] | odd[2] | odd[3]) != 0;
                    if (elect_one()) {
                        const uint64_t vd = v_desc + uint64_t(t % NV * uint32_t(C::kVBytes >> 4));
                        const uint64_t pd = p_desc + uint64_t((t & 1) * uint32_t(C::kPBytes >> 4));
#pragma unroll
                        for (int k = 0; k < KT / 16; ++k)
                            mma_bf16(tm + (2u + (kG == 2 ? t & 1 : 0)) * N, vd + uint64_t(k * 128),
                                     pd + uint64_t((k >> 2) * (N * 8) + (k & 3) * 2), id_o, k > 0 || acc);
                        mma_commit(&ms.pv_done[t & 1]);
                        mma_commit(&ms.v_empty[t % kBars]);
                    }
                    __syncwarp();
                    if (v + 2 < nt) scores(v + 2);
                }
                base += uint32_t(nt);
            }
            // nothing of this CTA's is in flight when its tensor memory goes
            if (elect_one()) mma_commit(&ms.done);
            __syncwarp();
            mbar_wait(&ms.done, 0, err);
        } else if (ms.has && warp < kMma + 3) {
            const bool fetches_values = warp == kMma + 2;
            // ---- page fetches: keys, or values ------------------------------------------------
            fetch_pages<D, kE4m3>(p, maps, ms.piece[0], ms.piece[1], fetches_values, ok, [&](uint32_t t, bool values) {
                if (!values) {
                    wait_stage<NK>(ok, ms.k_empty, t, err);
                    return Landing{&ms.k_full[t % kBars], k_ring + t % NK * C::kKBytes, ms.k_scale[t % NK]};
                }
                if constexpr (kE4m3) {
                    wait_stage<NR>(ok, ms.raw_empty, t, err);
                    return Landing{&ms.raw_full[t % kBars], raw_ring + t % NR * C::kRawBytes, ms.v_scale[t % NR]};
                }
                wait_stage<NV>(ok, ms.v_empty, t, err);
                return Landing{&ms.v_full[t % kBars], v_ring + t % NV * C::kVBytes, nullptr};
            }, fetches_values ? (kE4m3 ? ms.raw_full : ms.v_full) : ms.k_full, fetches_values ? (kE4m3 ? NR : NV) : NK);
        }
    } else {
        if constexpr (kE4m3) set_regs<C::kRows, C::kLaunch>();
        if (ms.has) {
            // ---- rows of Q; value tiles looked over, or (e4m3) made bf16 -----------------------------
            const int w = warp - kRow0, qt = tid - kRow0 * 32;
            constexpr int kRowThreads = C::kRowWarps * 32, CPR = D / 8, RPP = kRowThreads / CPR;
            const int c = qt % CPR;
            ItemWalk walk(ms.piece[0], ms.piece[1]);
            Item it = {};
            uint32_t n_it = 0, tile = 0;
            // Only the first of these warps waits by polling; the others meet it at a barrier of the
            // hardware's, and learn there whether it gave up.
            // (by turns two words: the first may be an appointment ahead of a warp that still reads)
            uint32_t turn = 0;
            auto meet = [&] {
                if (w == 0 && !ok) ms.rows_gave_up[turn] = 1;
                named_sync<5, kRowThreads>();
                ok = ms.rows_gave_up[turn] == 0;
                turn ^= 1;
            };
            while (ok && walk.next(p, it)) {
                const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.q) + c * 8;
                uint4 raw[N / RPP];
#pragma unroll
                for (int b = 0; b < N / RPP; ++b) {
                    const int row = qt / CPR + b * RPP;
                    raw[b] = row < it.rows ? *reinterpret_cast<const uint4 *>(q + it.at(row, p, p.q_stride, D))
                                           : make_uint4(0, 0, 0, 0);
                }
                if (w == 0) wait_for(ok, &ms.q_free, (n_it & 1) ^ 1, err);  // the last item's scores have read it
                meet();
                if (!ok) break;
                int e[N / RPP];
                if constexpr (kE4m3) row_exponents<CPR>(raw, e);
#pragma unroll
                for (int b = 0; b < N / RPP; ++b) {
                    const int row = qt / CPR + b * RPP;
                    float unit = 1.f;
                    if constexpr (kE4m3) {
                        // a row as 2^e (q1 + q2): e4m3 keeps 4 significant bits, so q1 and what q1 leaves
                        // hold all 8 of a bf16 (down to 2^-18 of the row's largest value)
                        uint32_t w1[2], w2[2];
                        split_row(raw[b], e[b], w1, w2);
                        unit = exp2_biased(e[b] < 0 ? 127 : e[b]);
                        const uint32_t at = row8_piece<D>(row, c >> 1) + uint32_t(c & 1) * 8u;
                        *reinterpret_cast<uint2 *>(smem + at) = make_uint2(w1[0], w1[1]);
                        *reinterpret_cast<uint2 *>(smem + N * D + at) = make_uint2(w2[0], w2[1]);
                    } else {
                        *reinterpret_cast<uint4 *>(smem + sw128_chunk(row, c, N)) = raw[b];
                    }
                    if (c == 0) ms.row_scale[n_it & 1][row] = p.scale_log2 * unit;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ms.q_full), mbar_arrive(&ms.row_unit[n_it & 1]);
                ++n_it;
                int page = peek_page(p, it, it.k0, lane);
                for (int kb = it.k0; kb < it.k1 && ok; kb += KT, ++tile) {
                    const uint32_t absent = absent_groups(p, page);
                    page = peek_page(p, it, kb + KT, lane);
                    if (w == 0) {
                        if constexpr (kE4m3) {
                            wait_tile(ok, ms.raw_full, tile, err);
                            wait_stage<NV>(ok, ms.v_empty, tile, err);
                        } else {
                            wait_tile(ok, ms.v_full, tile, err);
                        }
                    }
                    meet();
                    if (!ok) break;
                    unsigned char *dst = v_ring + tile % NV * C::kVBytes;
                    if constexpr (kE4m3) {
                        widen_tile<D>(p, it, kb, absent, raw_ring + tile % NR * C::kRawBytes, dst, ms.v_scale[tile % NR], w,
                                      lane, ms.odd[tile % kBars]);
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
    if (warp == kMma) tmem_dealloc(tm, C::kColumns);
}

template <bool kE4m3>
kda_status launch(const kda_kv_cache *c, AttendParams &p, const AttendPlan &plan, cudaStream_t stream) {
    using C = Cfg<kE4m3>;
    TileMaps maps;
    if (!page_map(&maps.k, c->k, c, kE4m3) || !page_map(&maps.v, c->v, c, kE4m3)) return KDA_ERR_CUDA;
    constexpr size_t smem = smem_bytes<C>();
    static_assert(smem <= 232448, "shared memory of a CTA");
    if (!allow_smem<attend_few_kernel<kE4m3>>(int(smem))) return KDA_ERR_CUDA;
    p.key_step = KT;
    p.item_cost = kItemCost;
    p.min_keys = KT;
    const ProfScope prof(KDA_KERNEL_KV_ATTEND, stream);
    return launch_overlapped(attend_few_kernel<kE4m3>, dim3(unsigned(plan.n_cta)), C::kThreads, smem, stream, p, maps);
}

}  // namespace

bool few_plan(const kda_kv_cache *c, const kda_kv_batch *b, AttendPlan *plan) {
    const long long rows = static_cast<long long>(b->max_new) * (c->num_heads / c->num_kv_heads);
    if (c->act != KDA_BF16 || c->head_dim != D || rows > N) return false;
    plan->bm = N;
    plan->n_cta = sm_count();
    return true;
}

kda_status few_launch(const kda_kv_cache *c, AttendParams &p, const AttendPlan &plan, cudaStream_t stream) {
    return c->format == KDA_KV_E4M3 ? launch<true>(c, p, plan, stream) : launch<false>(c, p, plan, stream);
}

}  // namespace kv
}  // namespace kda
