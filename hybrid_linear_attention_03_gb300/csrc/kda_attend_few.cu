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
// 397 us (6.7 TB/s, 99 % of the measured copy rate); the same in e4m3 359 us
// (3.7 TB/s: widening the values and storing the weights bound it) against 447 with
// the tile kernel; one sequence of 65536 in e4m3 50 us, of 1024 in bf16 13 us (launch,
// one tile a CTA and the joining of parts).  With 32 or 64 rows a thread's share of a
// tile grows and the tile kernel is faster: 237 against 247 us for 32 sequences of 8K
// to 16K keys at 32 rows.
//
// Warps: 0-3 softmax (a thread a key, later a channel), 4 issues the products, 5
// and 6 fetch pages by TMA, 8-11 (8-15 with e4m3 pages) bring the rows of Q and
// look value tiles over, or widen them, as in kda_attend_tile.cu; keys in e4m3
// meet Q as two e4m3 terms.
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
    static constexpr int kRowWarps = kE4m3 ? 8 : 4, kThreads = (8 + kRowWarps) * 32;
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
    static constexpr int kColumns = 64;  // tensor memory: scores twice, O
    static_assert(kStagesK < kBars && kStagesV < kBars && kStagesRaw < kBars, "a tile's barrier is free before its stage");
};

template <typename C> struct alignas(16) Misc {
    uint64_t k_full[kBars], k_empty[kBars], v_full[kBars], v_empty[kBars], clean[kBars], raw_full[kBars], raw_empty[kBars];
    uint64_t s_full[2], p_ready[2], pv_done[2];  // by tile parity
    uint64_t q_full, q_free, done;
    uint64_t row_unit[2];  // by item parity
    uint32_t tmem;
    int has, rows_gave_up;
    Cursor piece[2];
    uint32_t odd[kBars][4];                  // by tile: keys whose value row was taken out of it
    alignas(16) uint8_t k_scale[C::kStagesK][KT];  // e4m3: the tiles' scale exponents
    alignas(16) uint8_t v_scale[C::kStagesRaw][KT];
    alignas(16) float row_scale[2][N];       // by item parity: scale * log2(e), with e4m3 times the row's scale
    alignas(16) float ref[N], back[N];       // rows' references, and what the last move scaled by
    float tops[4][N];                        // by warp: maxima, then sums
};

template <typename C> constexpr size_t smem_bytes() { return 1024 + C::kMiscAt + sizeof(Misc<C>); }

// Whether any of the 128 softmax threads says so (which all meet here).
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
    if (warp == 4) tmem_alloc(&ms.tmem, C::kColumns);
    wait_prior_kernel();
    allow_next_kernel();
    if (tid < 2) p.parts[2 * cta + tid].state = 0;
    if (warp == 5) {
        Cursor a, z;
        const bool has = find_piece(p, cta, int(gridDim.x), lane, a, z);
        if (lane == 0) ms.piece[0] = a, ms.piece[1] = z, ms.has = has, ms.rows_gave_up = 0;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = ms.tmem;
    uint32_t *err = p.b.err;
    bool ok = true;  // of this thread's waits

    if (ms.has && warp < 4) {
        // ---- softmax: thread = key of the tile; at an item's end = channel ------------------
        const uint32_t lanes = uint32_t(warp * 32) << 16, t_o = tm + lanes + 2u * N;
        ItemWalk walk(ms.piece[0], ms.piece[1]);
        Item it = {};
        uint32_t tile = 0, n_it = 0;  // tiles and items so far
        // O holds the product of the tile with this count
        auto wait_o = [&](uint32_t t) {
            wait_for(ok, &ms.pv_done[t & 1], (t >> 1) & 1, err);
            __syncwarp();
            tc_fence_after();
        };
        while (walk.next(p, it)) {
            const int first_lim = it.ctx + it.tok0, nt = item_tiles(it);
            wait_for(ok, &ms.row_unit[n_it & 1], (n_it >> 1) & 1, err);
            __syncwarp();
            const float *row_scale = ms.row_scale[n_it & 1];
            ++n_it;
            if (tid < N) ms.ref[tid] = -INFINITY;
            float l[N];
#pragma unroll
            for (int c = 0; c < N; ++c) l[c] = 0.f;
            named_sync<2, 128>();
            int page = peek_page(p, it, it.k0, lane);
            for (int v = 0; v < nt; ++v, ++tile) {
                const int kb = it.k0 + v * KT, j = kb + tid;
                const uint32_t absent = absent_groups(p, page), t_s = tm + lanes + (tile & 1) * N;
                const bool check = partly_seen(it, kb, absent);
                page = peek_page(p, it, kb + KT, lane);
                int hidden = 0;  // rows before this one do not see the thread's key
                if (check) {
                    hidden = max(j - first_lim, 0) * p.group;
                    if (j >= it.k1 || (absent >> (tid / 16) & 1)) hidden = N;
                }
                float unit = 1.f;
                if constexpr (kE4m3) {
                    wait_tile(ok, ms.k_full, tile, err);
                    unit = exp2_biased(ms.k_scale[tile % NK][tid]);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ms.k_empty[tile % kBars]);
                }
                wait_for(ok, &ms.s_full[tile & 1], (tile >> 1) & 1, err);
                __syncwarp();
                tc_fence_after();
                float x[N];
                tmem_ld16(t_s, x);
                tmem_wait_ld();
                bool over = false;
#pragma unroll
                for (int i = 0; i < N; i += 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(row_scale + i);
                    const float4 r = *reinterpret_cast<const float4 *>(ms.ref + i);
                    x[i] *= f.x * unit, x[i + 1] *= f.y * unit, x[i + 2] *= f.z * unit, x[i + 3] *= f.w * unit;
                    if (check) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (i + e < hidden) x[i + e] = -INFINITY;
                    }
                    over |= x[i] > r.x + kRefSlack || x[i + 1] > r.y + kRefSlack || x[i + 2] > r.z + kRefSlack ||
                            x[i + 3] > r.w + kRefSlack;
                }
                if (any_of_128(over)) {
                    const float m = join_lanes(x, lane, [](float a, float b) { return fmaxf(a, b); });
                    if ((lane & 1) == 0) ms.tops[warp][lane >> 1] = m;
                    named_sync<2, 128>();
                    if (tid < N) {
                        const float top = fmaxf(fmaxf(ms.tops[0][tid], ms.tops[1][tid]), fmaxf(ms.tops[2][tid], ms.tops[3][tid]));
                        const float was = ms.ref[tid], to = top > was + kRefSlack ? top : was;
                        ms.ref[tid] = to;
                        ms.back[tid] = to == was ? 1.f : ex2(was - to);
                    }
                    named_sync<2, 128>();
                    float o[N];
                    if (v > 0) {  // O is new with the first product
                        wait_o(tile - 1);
                        tmem_ld16(t_o, o);
                        tmem_wait_ld();
                    }
#pragma unroll
                    for (int i = 0; i < N; ++i) l[i] *= ms.back[i], o[i] = v > 0 ? o[i] * ms.back[i] : 0.f;
                    if (v > 0) {
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
                    const float r = ms.ref[i], w = ex2(x[i] - (r == -INFINITY ? 0.f : r));
                    l[i] += w;
                    *reinterpret_cast<__nv_bfloat16 *>(p_img + sw128_offset(i, tid, N)) = __float2bfloat16_rn(w);
                }
                if (check) {
                    wait_tile(ok, kE4m3 ? ms.v_full : ms.clean, tile, err);
                    __syncwarp();
                    const uint32_t *odd = ms.odd[tile % kBars];
                    if ((odd[0] | odd[1] | odd[2] | odd[3]) != 0) {
                        // value rows taken out of the tile: thread = channel adds them for the rows that see them
                        named_sync<2, 128>();  // all weights are there
                        float o[N];
                        if (v > 0) {
                            wait_o(tile - 1);
                            tmem_ld16(t_o, o);
                            tmem_wait_ld();
                        }
#pragma unroll
                        for (int i = 0; i < N; ++i) o[i] = v > 0 ? o[i] : 0.f;
                        for (int g = 0; g < 4; ++g) {
                            for (uint32_t left = odd[g]; left; left &= left - 1) {
                                const int out = g * 32 + __ffs(left) - 1, jj = kb + out;
                                const size_t vec = ((size_t(max(load_page(p.b, it.n, jj), 0)) * size_t(p.hkv) + size_t(it.h))
                                                    << p.b.page_shift) + size_t(jj & ((1 << p.b.page_shift) - 1));
                                float val;
                                if constexpr (kE4m3)
                                    val = unpack_e4m3(static_cast<const uint8_t *>(p.pv)[vec * D + tid]).x * exp2_biased(p.sv[vec]);
                                else
                                    val = __bfloat162float(static_cast<const __nv_bfloat16 *>(p.pv)[vec * D + tid]);
#pragma unroll
                                for (int i = 0; i < N; ++i) {
                                    const float w = __bfloat162float(
                                        *reinterpret_cast<const __nv_bfloat16 *>(p_img + sw128_offset(i, out, N)));
                                    if (w != 0.f && first_lim + i / p.group >= jj) o[i] = fmaf(w, val, o[i]);
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
                if (lane == 0) mbar_arrive(&ms.p_ready[tile & 1]);
            }

            // ---- output: thread = channel --------------------------------------------------
            const float sum = join_lanes(l, lane, [](float a, float b) { return a + b; });
            if ((lane & 1) == 0) ms.tops[warp][lane >> 1] = sum;
            named_sync<2, 128>();
            if (tid < N) ms.back[tid] = (ms.tops[0][tid] + ms.tops[1][tid]) + (ms.tops[2][tid] + ms.tops[3][tid]);
            wait_o(tile - 1);
            named_sync<2, 128>();
            const bool whole = it.whole();
            float *data = p.part_data + (size_t(cta) * 2 + it.slot()) * size_t(N) * (D + 2);
            float o[N];
            tmem_ld16(t_o, o);
            tmem_wait_ld();
            __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out) + it.at(0, p, p.out_stride, D) + tid;
            int g = 0;  // query head of the group
#pragma unroll
            for (int r = 0; r < N; ++r) {
                if (r >= it.rows) break;
                if (whole) {
                    const float sum = ms.back[r], inv = sum > 0.f || sum != sum ? 1.0f / sum : 0.f;
                    *dst = __float2bfloat16_rn(o[r] * inv);
                    dst += D;
                    if (++g == p.group) g = 0, dst += p.out_stride - static_cast<long long>(p.group) * D;
                } else {
                    data[size_t(r) * D + tid] = o[r];
                }
            }
            if (!whole) {
                if (tid < it.rows) data[N * D + tid] = ms.ref[tid], data[N * D + N + tid] = ms.back[tid];
                if (tid == 0) p.parts[2 * cta + it.slot()] = it.part();
            }
            tc_fence_before();  // the next item's products rewrite O
            named_sync<2, 128>();  // and its start the references and sums
        }
    } else if (ms.has && warp == 4) {
        // ---- products (converged warp, one lane issues; descriptors count 16-byte units) -------
        const uint32_t id_s = kE4m3 ? idesc_e4m3_f32(128, N) : idesc_bf16_f32(128, N), id_o = idesc_bf16_f32(128, N, true, false);
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
                // the first product starts O, unless value rows were added to it by hand
                const uint32_t *odd = ms.odd[t % kBars];
                const uint32_t acc = v > 0 || (odd[0] | odd[1] | odd[2] | odd[3]) != 0;
                if (elect_one()) {
                    const uint64_t vd = v_desc + uint64_t(t % NV * uint32_t(C::kVBytes >> 4));
                    const uint64_t pd = p_desc + uint64_t((t & 1) * uint32_t(C::kPBytes >> 4));
#pragma unroll
                    for (int k = 0; k < KT / 16; ++k)
                        mma_bf16(tm + 2u * N, vd + uint64_t(k * 128), pd + uint64_t((k >> 2) * (N * 8) + (k & 3) * 2), id_o,
                                 k > 0 || acc);
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
        bool end_ok = true;
        wait_for(end_ok, &ms.done, 0, err);
    } else if (ms.has && (warp == 5 || warp == 6)) {
        const bool fetches_values = warp == 6;
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
    } else if (ms.has && warp >= 8) {
        // ---- rows of Q; value tiles looked over, or (e4m3) made bf16 -----------------------------
        const int w = warp - 8, qt = tid - 256;
        constexpr int kRowThreads = C::kRowWarps * 32, CPR = D / 8, RPP = kRowThreads / CPR;
        const int c = qt % CPR;
        ItemWalk walk(ms.piece[0], ms.piece[1]);
        Item it = {};
        uint32_t n_it = 0, tile = 0;
        // Only the first of these warps waits by polling; the others meet it at a barrier of the
        // hardware's, and learn there whether it gave up.
        auto meet = [&] {
            if (w == 0 && !ok) ms.rows_gave_up = 1;
            named_sync<3, kRowThreads>();
            ok = ms.rows_gave_up == 0;
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
#pragma unroll
            for (int b = 0; b < N / RPP; ++b) {
                const int row = qt / CPR + b * RPP;
                float unit = 1.f;
                if constexpr (kE4m3) {
                    // a row as 2^e (q1 + q2): e4m3 keeps 4 significant bits, so q1 and what q1 leaves
                    // hold all 8 of a bf16 (down to 2^-18 of the row's largest value)
                    uint32_t w1[2], w2[2];
                    unit = exp2_biased(split_row<CPR>(raw[b], w1, w2));
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
                    widen_tile<D>(p, it, kb, absent, raw_ring + tile % NR * C::kRawBytes, dst, ms.v_scale[tile % NR], w, lane,
                                  ms.odd[tile % kBars]);
                    if (lane == 0) mbar_arrive(&ms.v_full[tile % kBars]), mbar_arrive(&ms.raw_empty[tile % kBars]);
                } else {
                    look_over_tile<D>(it, kb, absent, dst, w, lane, ms.odd[tile % kBars]);
                    if (lane == 0) mbar_arrive(&ms.clean[tile % kBars]);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 4) tmem_dealloc(tm, C::kColumns);
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
