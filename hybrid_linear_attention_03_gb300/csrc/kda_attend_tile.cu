// kda_attend_tile.cu -- kda_kv_attend for bf16 rows on the tensor cores: the
// kernel of chunks, verifies and wide groups (more than 16 rows an item,
// head sizes 64 and 128).
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
// The weights are handed over in two halves, so the product of the first runs
// under the exponentials of the second.
// ref is the row's maximum so far, but only moved (and O and the sums scaled
// by 2^(ref - ref')) when a tile exceeds it by more than 8: weights then reach
// 2^8 at most, which costs no precision in bf16 and fp32, and most tiles leave
// O in tensor memory untouched.  P is rounded to bf16 (2^-9 relative, the
// size of the output's own rounding, and not correlated between keys); scores,
// sums and O stay in 32 bits.
//
// Warps: 0-3 side 0, 4-7 side 1 (a thread a row); 8 and 9 issue a side's
// products each; 10 fetches pages by TMA into a ring of tiles (K_0, V_0, K_1,
// V_1, ...); 12-15 bring the rows of Q and look value tiles over (below); with
// e4m3 pages warp 10 fetches them raw with their scales, and warps 16-19 turn
// them into exact bf16 tiles.
//
// A value behind a row's position weighs nothing, but 0 * NaN is NaN in the
// product.  So in the few tiles where some row does not see some key, warps
// 12-15 zero the rows of absent keys in the value tile, and take non-finite
// value rows out of it; the row threads that do see those add them one by one.
#include <cudaTypedefs.h>

#include <mutex>

#include "kda_attend.cuh"
#include "kda_sm100.cuh"

namespace kda {
namespace kv {
namespace {

using namespace sm100;

constexpr int KT = 128;          // keys of a tile
constexpr int kSideRows = 128;   // rows of a side
constexpr float kRefSlack = 8.f;
#ifndef ITEM_COST
#define ITEM_COST 384
#endif
constexpr int kItemCost = ITEM_COST;

template <int D, bool kE4m3> struct Cfg {
    static constexpr int kThreads = kE4m3 ? 640 : 512;
    // Registers a thread after the split: every SM quarter holds two softmax
    // warps and two (bf16) or three (e4m3) others, 128 or 96 registers each at
    // launch: 256 * 200 + 256 * 56 = 512 * 128, 256 * 152 + 384 * 56 < 640 * 96.
    static constexpr int kRegsSoftmax = kE4m3 ? 152 : 200;
    static constexpr int kRegsOther = 56;
    static constexpr int kTileBytes = KT * D * 2;
    static constexpr int kQBytes = kSideRows * D * 2;
    static constexpr int kStages = D == 128 ? (kE4m3 ? 4 : 5) : 8;
    static constexpr int kRawStages = kE4m3 ? 2 : 0;
    static constexpr int kRawBytes = KT * D;
    static constexpr int kRingAt = 2 * kQBytes;
    static constexpr int kRawAt = kRingAt + kStages * kTileBytes;
    static constexpr int kMiscAt = kRawAt + kRawStages * kRawBytes;
};

// Barriers of the ring's fills, more than it has stages: fill f (K and V tiles
// in turn) lands in stage f % stages but reports on barrier f % kFills.  A wait
// by parity is only sound for a thread that sees every phase of its barrier, and
// a side or a look-over that takes every second tile, or only the V tiles, sees
// every phase of every barrier it uses (kFills is a multiple of 4), whatever the
// number of stages and the order in which copies land.
constexpr int kFills = 16;
constexpr int kLooked = kFills / 2;  // of value tiles looked over

struct Misc {
    uint64_t full[kFills], empty[kFills], clean[kLooked], raw_full[2], raw_empty[2];
    uint64_t s_full[2], p_ready[2][2], q_full[2], q_free[2], o_full[2], done[2];
    uint32_t tmem;
    int has;
    Cursor piece[2];
    uint32_t odd[kLooked][4];          // by tile: keys whose value row was taken out of it
    alignas(16) uint8_t scale[2][KT];  // e4m3: the raw tile's scale exponents
    float m[kSideRows], l[kSideRows];  // side 1's row statistics, for the join
};

template <int D, bool kE4m3> constexpr size_t smem_bytes() { return 1024 + Cfg<D, kE4m3>::kMiscAt + sizeof(Misc); }

// ---- PTX of this kernel ---------------------------------------------------------
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float *v) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15, %16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
__device__ __forceinline__ uint32_t tmem_ld1(uint32_t taddr) {
    uint32_t r;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr));
    return r;
}
// D[tmem] (+)= A[tmem] * B[smem], A bf16 with two K values a column.
__device__ __forceinline__ void mma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// 16-byte asynchronous copy, or zeros.
__device__ __forceinline__ void cp_async16_or_zero(void *smem_dst, const void *gsrc, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(smem_dst)), "l"(gsrc), "r"(there ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
template <int N> __device__ __forceinline__ void reg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void reg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int kId, int kThreads> __device__ __forceinline__ void named_sync() {
    asm volatile("bar.sync %0, %1;" ::"n"(kId), "n"(kThreads) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Two 32-bit multiply-adds in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\t"
        "mov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\t"
        "mov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// Any bf16 infinity or NaN among eight.
__device__ __forceinline__ bool odd_bf16(const uint4 &w) {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
    bool odd = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) odd |= (x[i] & 0x7f80u) == 0x7f80u || (x[i] & 0x7f800000u) == 0x7f800000u;
    return odd;
}

// A bounded wait that is skipped once one has given up.  The row warps then run
// on with whatever is there (all in bounds, the error word is set), so that the
// CTA's own barriers are met; the other roles stop issuing.  Each try sleeps for
// up to a millisecond: a thread that polls takes issue slots from the others, and
// reading the clock takes longer than most waits.
__device__ __forceinline__ void wait_for(bool &ok, uint64_t *bar, uint32_t parity, uint32_t *err) {
    if (!ok) return;
    uint64_t t0 = 0;
    for (;;) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(smem_u32(bar)), "r"(parity), "r"(1000000u)
            : "memory");
        if (done) return;
        const uint64_t now = global_timer_ns();
        if (t0 == 0) t0 = now;
        if (now - t0 > 2000000000ull) break;
    }
    atomicOr(err, KDA_DEVERR_TIMEOUT);
    ok = false;
}
// The stage of fill f is free: the fill that was there before has been used.
template <int kStages> __device__ __forceinline__ void wait_stage(bool &ok, uint64_t *empty, uint32_t f, uint32_t *err) {
    if (f >= kStages) wait_for(ok, &empty[(f - kStages) % kFills], ((f - kStages) / kFills) & 1, err);
}
// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(one));
    return one != 0;
}

// 32 bytes, one whole sector, to a 32-byte aligned place.
__device__ __forceinline__ void store32(void *dst, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}
__device__ __forceinline__ bool any_odd(const uint32_t *odd) { return (odd[0] | odd[1] | odd[2] | odd[3]) != 0; }

struct TileMaps {
    CUtensorMap k, v;
};

__device__ __forceinline__ int item_tiles(const Item &it) { return (it.k1 - it.k0 + KT - 1) / KT; }
// Key tiles of an item's share that side s computes, and the v-th of them.
template <bool kByKeys> __device__ __forceinline__ int side_tiles(const Item &it, int s) {
    if (kByKeys) return (item_tiles(it) - s + 1) / 2;
    return s * kSideRows < it.rows ? item_tiles(it) : 0;
}
template <bool kByKeys> __device__ __forceinline__ int side_tile(int s, int v) { return kByKeys ? 2 * v + s : v; }

// Bit g: keys [kb + 16 g, kb + 16 g + 16) are in a page outside the cache.
__device__ __forceinline__ uint32_t absent_groups(const AttendParams &p, const Item &it, int kb, int lane) {
    bool bad = false;
    if (lane < KT / 16 && kb + lane * 16 < it.k1) bad = load_page(p.b, it.n, kb + lane * 16) < 0;
    return __ballot_sync(0xffffffffu, bad);
}
// Some row of the item does not see some key of the tile at kb.
__device__ __forceinline__ bool partly_seen(const Item &it, int kb, uint32_t absent) {
    return absent != 0 || kb + KT - 1 > it.ctx + it.tok0;
}

// Adds the value rows that were taken out of a tile to O, for the rows that see
// them (a row's weight is read back from its bf16 place over the scores).  Rare,
// so short rather than fast.  Whole warp.
template <int D, bool kE4m3>
__device__ __noinline__ void add_odd_rows(const AttendParams &p, const Item &it, int kb, int lim, const uint32_t *odd,
                                          uint32_t t_s, uint32_t t_o, bool fresh) {
    if (fresh) {
        const float z[16] = {};
        for (int c = 0; c < D; c += 16) tmem_st16(t_o + uint32_t(c), z);
        tmem_wait_st();
    }
    for (int g = 0; g < KT / 32; ++g) {
        for (uint32_t left = odd[g]; left; left &= left - 1) {
            const int c = g * 32 + __ffs(left) - 1, j = kb + c;
            const uint32_t pw = tmem_ld1(t_s + uint32_t(c / 2));
            tmem_wait_ld();
            const float w = __uint_as_float(c & 1 ? pw & 0xffff0000u : pw << 16);
            const int page = load_page(p.b, it.n, j);
            const size_t vec = ((size_t(max(page, 0)) * size_t(p.hkv) + size_t(it.h)) << p.b.page_shift) +
                               size_t(j & ((1 << p.b.page_shift) - 1));
            for (int ch = 0; ch < D; ch += 16) {
                float o[16];
                tmem_ld16(t_o + uint32_t(ch), o);
                tmem_wait_ld();
                if (j <= lim && w != 0.f) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float val;
                        if constexpr (kE4m3)
                            val = unpack_e4m3(static_cast<const uint8_t *>(p.pv)[vec * D + ch + i]).x * exp2_biased(p.sv[vec]);
                        else
                            val = __bfloat162float(static_cast<const __nv_bfloat16 *>(p.pv)[vec * D + ch + i]);
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

template <int D, bool kE4m3, bool kByKeys>
__global__ void __launch_bounds__(Cfg<D, kE4m3>::kThreads, 1)
    attend_tile_kernel(const __grid_constant__ AttendParams p, const __grid_constant__ TileMaps maps) {
    using C = Cfg<D, kE4m3>;
    constexpr int NST = C::kStages, NRAW = kE4m3 ? C::kRawStages : 1, BM = kByKeys ? kSideRows : 2 * kSideRows;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Misc &ms = *reinterpret_cast<Misc *>(smem + C::kMiscAt);
    const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5, cta = int(blockIdx.x);
    unsigned char *ring = smem + C::kRingAt;

    if (tid == 0) {
        for (int i = 0; i < kFills; ++i) {
            mbar_init(&ms.full[i], kE4m3 ? 4 : 1);
            mbar_init(&ms.empty[i], kByKeys ? 1 : 2);  // by rows both sides are done with a tile
        }
        for (int i = 0; i < kLooked; ++i) mbar_init(&ms.clean[i], 4);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ms.raw_full[i], 1), mbar_init(&ms.raw_empty[i], 4);
            mbar_init(&ms.s_full[i], 1), mbar_init(&ms.p_ready[i][0], 4), mbar_init(&ms.p_ready[i][1], 4);
            mbar_init(&ms.q_full[i], 4), mbar_init(&ms.q_free[i], 1);
            mbar_init(&ms.o_full[i], 1), mbar_init(&ms.done[i], 1);
        }
        fence_mbar_init();
    }
    if (warp == 8) tmem_alloc(&ms.tmem, 512);
    wait_prior_kernel();
    allow_next_kernel();
    if (tid < 2) p.parts[2 * cta + tid].state = 0;
    if (warp == 10) {
        Cursor a, z;
        const bool has = find_piece(p, cta, int(gridDim.x), lane, a, z);
        if (lane == 0) ms.piece[0] = a, ms.piece[1] = z, ms.has = has;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = ms.tmem;
    uint32_t *err = p.b.err;
    bool ok = true;  // of this thread's waits

    if (warp < 8) {
        reg_inc<C::kRegsSoftmax>();
        if (ms.has) {
            // ---- softmax: thread = row -------------------------------------------------
            const int s = warp >> 2, row = tid & 127;
            const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
            const uint32_t t_s = tm + lanes + uint32_t(s) * 128u, t_o = tm + lanes + 256u + uint32_t(s) * 128u;
            const int r = (kByKeys ? 0 : s * kSideRows) + row;
            ItemWalk walk(ms.piece[0], ms.piece[1]);
            Item it;
            uint32_t n_s = 0, n_o = 0, tile_base = 0;  // tiles and items so far: barrier phases
            while (walk.next(p, it)) {
                const int nv = side_tiles<kByKeys>(it, s);
                const int lim = it.ctx + it.tok0 + min(r, it.rows - 1) / p.group;  // last key this row sees
                float ref = -INFINITY, l = 0.f;
                for (int v = 0; v < nv; ++v, ++n_s) {
                    const int t = side_tile<kByKeys>(s, v), kb = it.k0 + t * KT;
                    const uint32_t absent = absent_groups(p, it, kb, lane);
                    const bool check = partly_seen(it, kb, absent);
                    wait_for(ok, &ms.s_full[s], n_s & 1, err);  // and with it the product before
                    __syncwarp();
                    tc_fence_after();
                    float x[KT];
#pragma unroll
                    for (int c = 0; c < KT; c += 32) tmem_ld32(t_s + uint32_t(c), x + c);
                    tmem_wait_ld();
                    if (check) {
#pragma unroll
                        for (int c = 0; c < KT; ++c)
                            if (kb + c > lim || (absent >> (c / 16) & 1)) x[c] = -INFINITY;
                    }
                    float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                    for (int c = 4; c < KT; c += 8) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            mx[i] = c + 4 + i < KT ? fmaxf(fmaxf(mx[i], x[c + i]), x[c + 4 + i]) : fmaxf(mx[i], x[c + i]);
                    }
                    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
                    const bool move = top > ref + kRefSlack;
                    if (__any_sync(0xffffffffu, move)) {
                        const float to = move ? top : ref, f = move ? ex2(ref - to) : 1.f;
                        if (v > 0) {  // O is new with the first product
#pragma unroll
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
                    }
                    const float base = ref == -INFINITY ? 0.f : ref;
                    const float2 sc = make_float2(p.scale_log2, p.scale_log2), sh = make_float2(-base, -base);
                    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                    for (int c = 0; c < KT; c += 32) {
                        uint32_t w[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float2 e = fma2(make_float2(x[c + 2 * i], x[c + 2 * i + 1]), sc, sh);
                            e.x = ex2(e.x), e.y = ex2(e.y);
                            sum[i & 1] = add2(sum[i & 1], e);
                            w[i] = pack_bf16(e.x, e.y);
                        }
                        tmem_st16u(t_s + uint32_t(c / 2), w);
                        if (c == KT / 2 - 32 && !check) {
                            tmem_wait_st();
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&ms.p_ready[s][0]);
                        }
                    }
                    l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                    tmem_wait_st();
                    if (check) {
                        const uint32_t at = tile_base + uint32_t(t), lk = at % kLooked;
                        wait_for(ok, &ms.clean[lk], (at / kLooked) & 1, err);
                        __syncwarp();
                        if (any_odd(ms.odd[lk])) add_odd_rows<D, kE4m3>(p, it, kb, lim, ms.odd[lk], t_s, t_o, v == 0);
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (check) mbar_arrive(&ms.p_ready[s][0]);
                        mbar_arrive(&ms.p_ready[s][1]);
                    }
                }
                tile_base += uint32_t(item_tiles(it));

                // ---- output ----------------------------------------------------------------
                const int nv_other = kByKeys ? side_tiles<kByKeys>(it, 1 - s) : 0;
                if (nv > 0) wait_for(ok, &ms.o_full[s], n_o++ & 1, err);
                __syncwarp();
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
                    float *data = p.part_data + (size_t(cta) * 2 + it.slot()) * size_t(BM) * (D + 2);
                    __nv_bfloat16 *dst =
                        static_cast<__nv_bfloat16 *>(p.out) + it.at(min(r, it.rows - 1), p.group, p.out_stride, D);
#pragma unroll
                    for (int c = 0; c < D; c += 16) {
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
                                store32(data + size_t(r) * D + c + i, w);
                            }
                        }
                    }
                    if (!whole) {
                        if (writes) data[BM * D + r] = ref, data[BM * D + BM + r] = l;
                        if (s == 0 && row == 0) p.parts[2 * cta + it.slot()] = it.part();
                    }
                }
                tc_fence_before();  // the next item's products rewrite O
                if (kByKeys) named_sync<1, 256>();
            }
        }
    } else {
        reg_dec<C::kRegsOther>();
        if (ms.has && warp < 10) {
            // ---- products of a side (converged warp, one lane issues) ----------------------
            const int s = warp - 8;
            const uint32_t id_s = idesc_bf16_f32(128, KT), id_o = idesc_bf16_f32(128, D, false, true);
            const uint32_t t_s = tm + uint32_t(s) * 128u, t_o = tm + 256u + uint32_t(s) * 128u;
            const uint64_t q_desc = sdesc_sw128(smem_u32(smem) + uint32_t(s) * C::kQBytes);
            const uint64_t k_desc = sdesc_sw128(smem_u32(ring)), v_desc = sdesc_sw128_mn(smem_u32(ring), KT * 128u);
            ItemWalk walk(ms.piece[0], ms.piece[1]);
            Item it;
            uint32_t base = 0, n_q = 0, n_p = 0;
            int nv = 0;
            // scores of the side's v-th tile (descriptors count 16-byte units)
            auto scores = [&](int v) {
                const uint32_t fill = base + 2u * uint32_t(side_tile<kByKeys>(s, v)), st = fill % NST;
                wait_for(ok, &ms.full[fill % kFills], (fill / kFills) & 1, err);
                if (!(ok = __all_sync(0xffffffffu, ok))) return;
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t kd = k_desc + uint64_t(st * (C::kTileBytes >> 4));
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        mma_bf16(t_s, q_desc + uint64_t((k >> 2) * (kSideRows * 8) + (k & 3) * 2),
                                 kd + uint64_t((k >> 2) * (KT * 8) + (k & 3) * 2), id_s, k > 0);
                    mma_commit(&ms.s_full[s]);
                    mma_commit(&ms.empty[fill % kFills]);
                    if (v + 1 == nv) mma_commit(&ms.q_free[s]);
                }
                __syncwarp();
            };
            while (ok && walk.next(p, it)) {
                nv = side_tiles<kByKeys>(it, s);
                if (nv > 0) {
                    wait_for(ok, &ms.q_full[s], n_q++ & 1, err);
                    scores(0);
                }
                for (int v = 0; v < nv && ok; ++v, ++n_p) {
                    const uint32_t fill = base + 2u * uint32_t(side_tile<kByKeys>(s, v)) + 1u, st = fill % NST;
                    wait_for(ok, &ms.full[fill % kFills], (fill / kFills) & 1, err);
                    const uint32_t lk = (fill >> 1) % kLooked;
                    wait_for(ok, &ms.clean[lk], ((fill >> 1) / kLooked) & 1, err);
                    // the first product starts O, unless value rows were added to it by hand
                    const uint32_t acc = v > 0 || any_odd(ms.odd[lk]);
                    const uint64_t vd = v_desc + uint64_t(st * (C::kTileBytes >> 4));
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        wait_for(ok, &ms.p_ready[s][half], n_p & 1, err);
                        if (!(ok = __all_sync(0xffffffffu, ok))) break;
                        tc_fence_after();
                        if (elect_one()) {
#pragma unroll
                            for (int k = half * (KT / 32); k < (half + 1) * (KT / 32); ++k)
                                mma_bf16_ta(t_o, t_s + uint32_t(k) * 8u, vd + uint64_t(k * 128), id_o, k > 0 || acc);
                            if (half == 1) {
                                mma_commit(&ms.empty[fill % kFills]);
                                if (v + 1 == nv) mma_commit(&ms.o_full[s]);
                            }
                        }
                        __syncwarp();
                    }
                    if (ok && v + 1 < nv) scores(v + 1);
                }
                if (!kByKeys && nv == 0) {  // a tile is free once both sides have said so
                    for (int i = 0; i < 2 * item_tiles(it) && ok; ++i) {
                        const uint32_t fill = base + uint32_t(i);
                        wait_for(ok, &ms.full[fill % kFills], (fill / kFills) & 1, err);
                        if (!(ok = __all_sync(0xffffffffu, ok))) break;
                        if (lane == 0) mbar_arrive(&ms.empty[fill % kFills]);
                    }
                }
                base += 2u * uint32_t(item_tiles(it));
            }
            // nothing of this side's is in flight when the tensor memory goes
            if (elect_one()) mma_commit(&ms.done[s]);
            __syncwarp();
            bool end_ok = true;
            wait_for(end_ok, &ms.done[s], 0, err);
        } else if (ms.has && warp == 10) {
            // ---- page fetches ------------------------------------------------------------
            const int page_size = 1 << p.b.page_shift, box = min(page_size, KT);
            ItemWalk walk(ms.piece[0], ms.piece[1]);
            Item it;
            uint32_t fill = 0;
            while (ok && walk.next(p, it)) {
                for (int kb = it.k0; kb < it.k1 && ok; kb += KT) {
                    const int j = kb + lane * box, line = j & (page_size - 1);
                    int page = -1;
                    if (lane * box < KT && j < it.k1) page = load_page(p.b, it.n, j);
                    const int there = __popc(__ballot_sync(0xffffffffu, page >= 0)) * box;
                    const int plane = page * p.hkv + it.h;  // below 2^31 (checked on the host)
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv, ++fill) {
                        const CUtensorMap *map = kv ? &maps.v : &maps.k;
                        if constexpr (kE4m3) {
                            const uint32_t st = fill % NRAW;
                            wait_for(ok, &ms.raw_empty[st], ((fill / NRAW) & 1) ^ 1, err);
                            if (!(ok = __all_sync(0xffffffffu, ok))) break;
                            if (lane == 0) mbar_arrive_expect_tx(&ms.raw_full[st], uint32_t(there * (D + 1)));
                            __syncwarp();
                            if (page >= 0) {
                                tma_load_3d(smem + C::kRawAt + st * C::kRawBytes + lane * box * D, map, &ms.raw_full[st], 0,
                                            line, plane);
                                bulk_load(&ms.scale[st][lane * box],
                                          (kv ? p.sv : p.sk) + (size_t(plane) << p.b.page_shift) + line, uint32_t(box),
                                          &ms.raw_full[st]);
                            }
                        } else {
                            const uint32_t st = fill % NST;
                            uint64_t *full = &ms.full[fill % kFills];
                            wait_stage<NST>(ok, ms.empty, fill, err);
                            if (!(ok = __all_sync(0xffffffffu, ok))) break;
                            if (lane == 0) mbar_arrive_expect_tx(full, uint32_t(there * D * 2));
                            __syncwarp();
                            if (page >= 0) {
                                unsigned char *dst = ring + st * C::kTileBytes + lane * box * 128;
#pragma unroll
                                for (int c = 0; c < D / 64; ++c)
                                    tma_load_3d(dst + c * KT * 128, map, full, c * 64, line, plane);
                            }
                        }
                    }
                }
            }
            // a given-up wait elsewhere may leave copies in flight: they land before the CTA ends
            if (!ok) {
                constexpr uint32_t kDepth = kE4m3 ? NRAW : NST;
                for (uint32_t i = 1; i <= kDepth && i <= fill; ++i) {
                    const uint32_t c = fill - i;
                    if (kE4m3) mbar_wait(&ms.raw_full[c % NRAW], (c / NRAW) & 1, err);
                    else mbar_wait(&ms.full[c % kFills], (c / kFills) & 1, err);
                }
            }
        } else if (ms.has && warp >= 12 && warp < 16) {
            // ---- rows of Q, and value tiles looked over ------------------------------------
            const int w = warp - 12, qt = tid - 384;
            ItemWalk walk(ms.piece[0], ms.piece[1]);
            Item it;
            uint32_t n_q[2] = {0, 0}, tile = 0;
            while (ok && walk.next(p, it)) {
                for (int s = 0; s < 2; ++s) {
                    if (side_tiles<kByKeys>(it, s) == 0) continue;
                    wait_for(ok, &ms.q_free[s], (n_q[s]++ & 1) ^ 1, err);  // the last item's scores have read it
                    if (!(ok = __all_sync(0xffffffffu, ok))) break;
                    unsigned char *q_img = smem + s * C::kQBytes;
                    constexpr int CPR = D / 8;  // 16-byte pieces of a row
                    const int c = qt % CPR;
                    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.q) + c * 8;
#pragma unroll 4
                    for (int row = qt / CPR; row < kSideRows; row += 128 / CPR) {
                        const int r = (kByKeys ? 0 : s * kSideRows) + row;
                        cp_async16_or_zero(q_img + sw128_chunk(row, c, kSideRows),
                                           q + it.at(min(r, it.rows - 1), p.group, p.q_stride, D), r < it.rows);
                    }
                    cp_async_wait_all();
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ms.q_full[s]);
                }
                for (int kb = it.k0; kb < it.k1 && ok; kb += KT, ++tile) {
                    const uint32_t absent = absent_groups(p, it, kb, lane), fill = 2u * tile + 1u, st = fill % NST;
                    wait_for(ok, &ms.full[fill % kFills], (fill / kFills) & 1, err);
                    if (!(ok = __all_sync(0xffffffffu, ok))) break;
                    uint32_t odd = 0;
                    if (partly_seen(it, kb, absent)) {
                        // a lane looks over one value row, each at a bank of its own
                        const int row = w * 32 + lane, j = kb + row;
                        unsigned char *img = ring + st * C::kTileBytes + row * 128;
                        const bool gone = j >= it.k1 || (absent >> (row / 16) & 1);
                        bool bad = false;
                        for (int c = 0; c < D / 8; ++c)
                            bad |= odd_bf16(*reinterpret_cast<const uint4 *>(img + (c >> 3) * KT * 128 +
                                                                             (((c & 7) ^ (lane & 7)) << 4)));
                        bad = bad && !gone && j > it.ctx + it.tok0;  // rows that every query sees stay
                        if (gone || bad) {
                            for (int c = 0; c < D / 8; ++c)
                                *reinterpret_cast<uint4 *>(img + (c >> 3) * KT * 128 + (((c & 7) ^ (lane & 7)) << 4)) =
                                    make_uint4(0, 0, 0, 0);
                        }
                        odd = __ballot_sync(0xffffffffu, bad);
                        fence_proxy_async_smem();
                    }
                    const uint32_t lk = tile % kLooked;
                    if (lane == 0) ms.odd[lk][w] = odd;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ms.clean[lk]);
                }
            }
        } else if (kE4m3 && ms.has && warp >= 16) {
            // ---- e4m3 tiles to bf16 ---------------------------------------------------------
            constexpr int UPK = D / 16;             // 16-byte pieces of a key
            constexpr int UPT = KT * UPK / 128;     // of a thread
            const int ct = tid - 512;
            ItemWalk walk(ms.piece[0], ms.piece[1]);
            Item it;
            uint32_t fill = 0;
            while (ok && walk.next(p, it)) {
                const int fills = 2 * item_tiles(it);
                for (int i = 0; i < fills && ok; ++i, ++fill) {
                    const uint32_t rs = fill % NRAW, st = fill % NST;
                    wait_for(ok, &ms.raw_full[rs], (fill / NRAW) & 1, err);
                    wait_stage<NST>(ok, ms.empty, fill, err);
                    if (!(ok = __all_sync(0xffffffffu, ok))) break;
                    const uint4 *raw = reinterpret_cast<const uint4 *>(smem + C::kRawAt + rs * C::kRawBytes);
                    unsigned char *dst = ring + st * C::kTileBytes;
#pragma unroll
                    for (int u = 0; u < UPT; ++u) {
                        const int key = (u * 128 + ct) / UPK, c = ct % UPK;
                        const uint4 q = raw[u * 128 + ct];
                        const float f = exp2_biased(ms.scale[rs][key]);
                        const uint32_t in[4] = {q.x, q.y, q.z, q.w};
                        uint32_t o[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float2 t = unpack_e4m3(uint16_t(in[e / 2] >> ((e & 1) * 16)));
                            o[e] = pack_bf16(t.x * f, t.y * f);
                        }
                        *reinterpret_cast<uint4 *>(dst + sw128_chunk(key, 2 * c, KT)) = make_uint4(o[0], o[1], o[2], o[3]);
                        *reinterpret_cast<uint4 *>(dst + sw128_chunk(key, 2 * c + 1, KT)) = make_uint4(o[4], o[5], o[6], o[7]);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ms.full[fill % kFills]), mbar_arrive(&ms.raw_empty[rs]);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 8) tmem_dealloc(tm, 512);
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    });
    return fn;
}

// [num_pages * num_kv_heads][page_size][head_dim]; a box is a tile's part of
// one page and head (64 channels of it for bf16, whose tiles are 128-byte
// swizzled).
bool page_map(CUtensorMap *m, const void *base, const kda_kv_cache *c, bool e4m3) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t esize = e4m3 ? 1 : 2, D = cuuint64_t(c->head_dim), P = cuuint64_t(c->page_size);
    const cuuint64_t dims[3] = {D, P, cuuint64_t(c->num_pages) * cuuint64_t(c->num_kv_heads)};
    const cuuint64_t strides[2] = {D * esize, D * P * esize};
    const cuuint32_t box[3] = {cuuint32_t(e4m3 ? c->head_dim : 64), cuuint32_t(c->page_size < KT ? c->page_size : KT), 1u};
    const cuuint32_t estr[3] = {1u, 1u, 1u};
    return fn(m, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims,
              strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              e4m3 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool kE4m3, bool kByKeys>
kda_status launch(const kda_kv_cache *c, AttendParams &p, const AttendPlan &plan, cudaStream_t stream) {
    TileMaps maps;
    if (!page_map(&maps.k, c->k, c, kE4m3) || !page_map(&maps.v, c->v, c, kE4m3)) return KDA_ERR_CUDA;
    auto kern = attend_tile_kernel<D, kE4m3, kByKeys>;
    constexpr size_t smem = smem_bytes<D, kE4m3>();
    static_assert(smem <= 232448, "shared memory of a CTA");
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)) != cudaSuccess) {
        cudaGetLastError();
        return KDA_ERR_CUDA;
    }
    p.key_step = KT;
    p.item_cost = kItemCost;
    p.min_keys = (kByKeys ? 2 : 1) * KT;
    const ProfScope prof(KDA_KERNEL_KV_ATTEND, stream);
    return launch_overlapped(kern, dim3(unsigned(plan.n_cta)), Cfg<D, kE4m3>::kThreads, smem, stream, p, maps);
}

template <int D>
kda_status by_type(const kda_kv_cache *c, AttendParams &p, const AttendPlan &plan, cudaStream_t s) {
    const bool by_keys = plan.bm == kSideRows;
    if (c->format == KDA_KV_E4M3)
        return by_keys ? launch<D, true, true>(c, p, plan, s) : launch<D, true, false>(c, p, plan, s);
    return by_keys ? launch<D, false, true>(c, p, plan, s) : launch<D, false, false>(c, p, plan, s);
}

}  // namespace

bool tile_plan(const kda_kv_cache *c, const kda_kv_batch *b, AttendPlan *plan) {
    const long long rows = static_cast<long long>(b->max_new) * (c->num_heads / c->num_kv_heads);
    if (c->act != KDA_BF16 || (c->head_dim != 64 && c->head_dim != 128) || rows <= 16) return false;
    plan->bm = rows <= kSideRows ? kSideRows : 2 * kSideRows;
    plan->n_cta = sm_count();
    return true;
}

kda_status tile_launch(const kda_kv_cache *c, AttendParams &p, const AttendPlan &plan, cudaStream_t stream) {
    return c->head_dim == 64 ? by_type<64>(c, p, plan, stream) : by_type<128>(c, p, plan, stream);
}

}  // namespace kv
}  // namespace kda
