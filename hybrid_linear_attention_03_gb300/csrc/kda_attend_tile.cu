// kda_attend_tile.cu -- kda_kv_attend for bf16 rows on the tensor cores: the
// kernel of chunks, verifies and wide groups (more than 16 rows an item,
// head sizes 64 and 128).
//
// Softmax in one pass, as in kda_attend_generic.cu: scores X = Q K^T (128 rows
// x 128 keys) land in tensor memory, one thread per row turns them into
// weights P = 2^(scale log2e X - ref) and leaves them as bf16 where the scores
// were, and O += P V reads them from there.  Two of these run side by side so
// that one's products cover the other's exponentials:
//   sides by rows  (row tiles of 256): side s has rows [128 s, 128 s + 128) and
//                  both read every key tile (half the L2 traffic per product);
//   sides by keys  (at most 128 rows an item): both have all rows, side s has
//                  the key tiles of its parity, joined at the item's end.
// ref is the row's maximum so far, but only moved (and O and the sums scaled
// by 2^(ref - ref')) when a tile exceeds it by more than 8: weights then reach
// 2^8 at most, which costs no precision in bf16 and fp32, and most tiles leave
// O in tensor memory untouched.  P is rounded to bf16 (2^-9 relative, the
// size of the output's own rounding, and not correlated between keys); scores,
// sums and O stay in 32 bits.
//
// Warps: 0-3 side 0, 4-7 side 1 (a thread a row), 8 issues the products, 9
// fetches pages by TMA into a ring of tiles (K_0, V_0, K_1, V_1, ...), 10 and 11
// fill the warpgroup; with
// e4m3 pages warp 9 fetches them raw and warps 12-15 turn them into exact bf16
// tiles.  Page sizes divide the tile, so a tile is 1 to 8 page boxes.
//
// A value behind a row's position weighs nothing, but 0 * NaN is NaN in the
// product: in the few tiles where some row does not see some key, keys that
// are absent are zeroed in the tile, and non-finite value rows are taken out of
// it too and added by the threads whose rows do see them.
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

template <int D, bool kE4m3> struct Cfg {
    static constexpr int kThreads = kE4m3 ? 512 : 384;
    // Registers a thread after the split: every SM quarter holds two softmax
    // warps and one (bf16) or two (e4m3) others, 168 or 128 registers each at
    // launch: 256 * 216 + 128 * 72 = 384 * 168, 256 * 192 + 256 * 64 = 512 * 128.
    static constexpr int kRegsSoftmax = kE4m3 ? 192 : 216;
    static constexpr int kRegsOther = kE4m3 ? 64 : 72;
    static constexpr int kTileBytes = KT * D * 2;
    static constexpr int kQBytes = kSideRows * D * 2;
    static constexpr int kStages = D == 128 ? (kE4m3 ? 4 : 5) : 8;
    static constexpr int kRawStages = kE4m3 ? 2 : 0;
    static constexpr int kRawBytes = KT * D;
    static constexpr int kRingAt = 2 * kQBytes;
    static constexpr int kRawAt = kRingAt + kStages * kTileBytes;
    static constexpr int kMiscAt = kRawAt + kRawStages * kRawBytes;
};

struct Misc {
    uint64_t full[8], empty[8], raw_full[2], raw_empty[2];
    uint64_t s_full[2], p_ready[2], q_full[2], o_full[2], done;
    uint32_t tmem;
    int has;
    Cursor piece[2];
    uint32_t odd[2][4];     // per side: keys of the tile whose value row was taken out
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
// D[tmem] += A[tmem] * B[smem], A bf16 with two K values a column.
__device__ __forceinline__ void mma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, 1, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc)
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
// CTA's own barriers are met; the other roles stop issuing.
__device__ __forceinline__ void wait_for(bool &ok, uint64_t *bar, uint32_t parity, uint32_t *err) {
    if (ok) ok = mbar_wait(bar, parity, err);
}

struct TileMaps {
    CUtensorMap k, v;
};

// Key tiles of an item's share that side s computes.
template <bool kByKeys> __device__ __forceinline__ int side_tiles(const Item &it, int s) {
    const int nt = (it.k1 - it.k0 + KT - 1) / KT;
    if (kByKeys) return (nt - s + 1) / 2;
    return s * kSideRows < it.rows ? nt : 0;
}

template <int D, bool kE4m3, bool kByKeys>
__global__ void __launch_bounds__(Cfg<D, kE4m3>::kThreads, 1)
    attend_tile_kernel(const __grid_constant__ AttendParams p, const __grid_constant__ TileMaps maps) {
    using C = Cfg<D, kE4m3>;
    constexpr int NST = C::kStages, BM = kByKeys ? kSideRows : 2 * kSideRows;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Misc &ms = *reinterpret_cast<Misc *>(smem + C::kMiscAt);
    const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5, cta = int(blockIdx.x);
    unsigned char *ring = smem + C::kRingAt;

    if (tid == 0) {
        for (int i = 0; i < NST; ++i) mbar_init(&ms.full[i], kE4m3 ? 4 : 1), mbar_init(&ms.empty[i], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ms.raw_full[i], 1), mbar_init(&ms.raw_empty[i], 4);
            mbar_init(&ms.s_full[i], 1), mbar_init(&ms.p_ready[i], 4);
            mbar_init(&ms.q_full[i], 4), mbar_init(&ms.o_full[i], 1);
        }
        mbar_init(&ms.done, 1);
        fence_mbar_init();
    }
    if (warp == 8) tmem_alloc(&ms.tmem, 512);
    wait_prior_kernel();
    allow_next_kernel();
    if (tid < 2) p.parts[2 * cta + tid].state = 0;
    if (warp == 9) {
        Cursor a, z;
        const bool has = find_piece(p, cta, int(gridDim.x), lane, a, z);
        if (lane == 0) ms.piece[0] = a, ms.piece[1] = z, ms.has = has;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = ms.tmem;
    uint32_t *err = p.b.err;

    if (warp < 8) {
        reg_inc<C::kRegsSoftmax>();
        if (ms.has) {
            // ---- softmax: thread = row -------------------------------------------------
            const int s = warp >> 2, row = tid & 127;
            const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
            const uint32_t t_s = tm + lanes + uint32_t(s) * 128u, t_o = tm + lanes + 256u + uint32_t(s) * 128u;
            unsigned char *q_img = smem + s * C::kQBytes;
            const int rb = kByKeys ? 0 : s * kSideRows, r = rb + row;
            ItemWalk walk(ms.piece[0], ms.piece[1]);
            Item it, nx;
            bool ok = true, has = walk.next(p, it);
            uint32_t n_s = 0, n_o = 0, n_o2 = 0;  // visits and items so far: barrier phases
            uint32_t ring_base = 0;

            auto load_q = [&](const Item &x) {
                if (side_tiles<kByKeys>(x, s) == 0) return;
                const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.q) +
                                                                   x.at(min(r, x.rows - 1), p.group, p.q_stride, D));
#pragma unroll
                for (int c0 = 0; c0 < D / 8; c0 += 8) {
                    uint4 w[8];
#pragma unroll
                    for (int c = 0; c < 8; ++c) w[c] = r < x.rows ? src[c0 + c] : make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        *reinterpret_cast<uint4 *>(q_img + sw128_chunk(row, c0 + c, kSideRows)) = w[c];
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ms.q_full[s]);
            };

            if (has) load_q(it);
            while (has) {
                const int nv = side_tiles<kByKeys>(it, s), nt = (it.k1 - it.k0 + KT - 1) / KT;
                const int lim = it.ctx + it.tok0 + min(r, it.rows - 1) / p.group;  // last key this row sees
                const int first_lim = it.ctx + it.tok0;                           // ... and the item's first row
                float ref = -INFINITY, l = 0.f;
                if (nv > 0) {
                    uint32_t z[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) z[i] = 0;
#pragma unroll
                    for (int c = 0; c < D; c += 16) tmem_st16u(t_o + uint32_t(c), z);
                    tmem_wait_st();
                }
                for (int v = 0; v < nv; ++v) {
                    const int t = kByKeys ? 2 * v + s : v, kb = it.k0 + t * KT;
                    // pages of the tile, 16 keys a lane
                    bool bad = false;
                    if (lane < KT / 16 && kb + lane * 16 < it.k1) bad = load_page(p.b, it.n, kb + lane * 16) < 0;
                    const uint32_t absent = __ballot_sync(0xffffffffu, bad);
                    const bool check = absent != 0 || kb + KT - 1 > first_lim;
                    wait_for(ok, &ms.s_full[s], n_s++ & 1, err);
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
                        for (int i = 0; i < 4; ++i) mx[i] = c + 4 + i < KT ? fmaxf(fmaxf(mx[i], x[c + i]), x[c + 4 + i]) : fmaxf(mx[i], x[c + i]);
                    }
                    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
                    const bool move = top > ref + kRefSlack;
                    if (__any_sync(0xffffffffu, move)) {
                        const float to = move ? top : ref, f = move ? ex2(ref - to) : 1.f;
                        if (v > 0) {  // O holds zeros until the first product
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
                    }
                    l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                    tmem_wait_st();
                    if (check) {
                        // this thread's key: absent, or a non-finite value row behind some row's position
                        const int j = kb + row;
                        const uint32_t slot = ring_base + 2u * uint32_t(t) + 1u;
                        unsigned char *v_img = ring + (slot % NST) * C::kTileBytes;
                        const int page = j < it.k1 && !(absent >> (row / 16) & 1) ? load_page(p.b, it.n, j) : -1;
                        const size_t vec = page < 0 ? 0 : ((size_t(page) * size_t(p.hkv) + size_t(it.h)) << p.b.page_shift) +
                                                              size_t(j & ((1 << p.b.page_shift) - 1));
                        bool odd = false;
                        if (page >= 0 && j > first_lim) {
                            if constexpr (kE4m3) {
                                const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(p.pv) + vec * D);
                                for (int c = 0; c < D / 16; ++c) {
                                    const uint4 w = src[c];
                                    odd |= ((__vcmpeq4(w.x & 0x7f7f7f7fu, 0x7f7f7f7fu) | __vcmpeq4(w.y & 0x7f7f7f7fu, 0x7f7f7f7fu) |
                                             __vcmpeq4(w.z & 0x7f7f7f7fu, 0x7f7f7f7fu) | __vcmpeq4(w.w & 0x7f7f7f7fu, 0x7f7f7f7fu)) != 0);
                                }
                                odd |= p.sv[vec] >= 247;  // 448 * 2^(247 - 127) is past bf16's range
                            } else {
                                const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.pv) + vec * D);
                                for (int c = 0; c < D / 8; ++c) odd |= odd_bf16(src[c]);
                            }
                        }
                        const uint32_t word = __ballot_sync(0xffffffffu, odd);
                        if (lane == 0) ms.odd[s][warp & 3] = word;
                        wait_for(ok, &ms.full[slot % NST], (slot / NST) & 1, err);
                        __syncwarp();
                        if (page < 0 || odd) {
#pragma unroll
                            for (int c = 0; c < D / 8; ++c)
                                *reinterpret_cast<uint4 *>(v_img + sw128_chunk(row, c, KT)) = make_uint4(0, 0, 0, 0);
                        }
                        fence_proxy_async_smem();
                        if (s) named_sync<2, 128>();
                        else named_sync<1, 128>();
                        for (int g = 0; g < 4; ++g) {
                            for (uint32_t left = ms.odd[s][g]; left; left &= left - 1) {
                                const int c = g * 32 + __ffs(left) - 1, jj = kb + c;
                                const uint32_t pw = tmem_ld1(t_s + uint32_t(c / 2));
                                tmem_wait_ld();
                                const float w = __uint_as_float(c & 1 ? pw & 0xffff0000u : pw << 16);
                                const int pg = load_page(p.b, it.n, jj);
                                const size_t at = ((size_t(pg) * size_t(p.hkv) + size_t(it.h)) << p.b.page_shift) +
                                                  size_t(jj & ((1 << p.b.page_shift) - 1));
                                for (int ch = 0; ch < D; ch += 16) {
                                    float o[16];
                                    tmem_ld16(t_o + uint32_t(ch), o);
                                    tmem_wait_ld();
                                    if (jj <= lim && w != 0.f) {
                                        for (int i = 0; i < 16; ++i) {
                                            float val;
                                            if constexpr (kE4m3)
                                                val = unpack_e4m3(static_cast<const uint8_t *>(p.pv)[at * D + ch + i]).x *
                                                      exp2_biased(p.sv[at]);
                                            else
                                                val = __bfloat162float(static_cast<const __nv_bfloat16 *>(p.pv)[at * D + ch + i]);
                                            o[i] = fmaf(w, val, o[i]);
                                        }
                                    }
                                    tmem_st16(t_o + uint32_t(ch), o);
                                }
                                tmem_wait_st();
                            }
                        }
                        if (s) named_sync<2, 128>();
                        else named_sync<1, 128>();  // odd[s] is rewritten by the next such tile
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ms.p_ready[s]);
                }
                has = walk.next(p, nx);
                if (has) load_q(nx);  // every score product of this side has completed
                ring_base += 2u * uint32_t(nt);

                // ---- output ----------------------------------------------------------------
                const int nv_other = kByKeys ? side_tiles<kByKeys>(it, 1 - s) : 0;
                if (nv > 0) wait_for(ok, &ms.o_full[s], n_o++ & 1, err);
                __syncwarp();
                bool writes = nv > 0 && r < it.rows;
                float f0 = 1.f, f1 = 0.f;
                if (kByKeys) {
                    if (s == 1) {
                        ms.m[row] = ref, ms.l[row] = l;
                        writes = false;
                    } else if (nv_other > 0) {
                        wait_for(ok, &ms.o_full[1], n_o2++ & 1, err);
                        __syncwarp();
                    }
                    tc_fence_before();
                    named_sync<3, 256>();
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
                    const bool whole = it.whole();
                    float *data = p.part_data + (size_t(cta) * 2 + it.slot()) * size_t(BM) * (D + 2);
                    __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out) + it.at(min(r, it.rows - 1), p.group, p.out_stride, D);
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
                            *reinterpret_cast<uint4 *>(dst + c) = make_uint4(w[0], w[1], w[2], w[3]);
                            *reinterpret_cast<uint4 *>(dst + c + 8) = make_uint4(w[4], w[5], w[6], w[7]);
                        } else {
#pragma unroll
                            for (int i = 0; i < 16; i += 4)
                                *reinterpret_cast<float4 *>(data + size_t(r) * D + c + i) =
                                    make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                        }
                    }
                    if (!whole) {
                        if (writes) data[BM * D + r] = ref, data[BM * D + BM + r] = l;
                        if (s == 0 && row == 0) p.parts[2 * cta + it.slot()] = it.part();
                    }
                }
                if (kByKeys) {
                    tc_fence_before();
                    named_sync<3, 256>();  // side 1 clears its O for the next item
                    tc_fence_after();
                }
                it = nx;
            }
        }
    } else {
        reg_dec<C::kRegsOther>();
        if (ms.has && warp == 8 && lane == 0) {
            // ---- products --------------------------------------------------------------
            const uint32_t id_s = idesc_bf16_f32(128, KT), id_o = idesc_bf16_f32(128, D, false, true);
            const uint32_t q_at = smem_u32(smem), ring_at = smem_u32(ring);
            ItemWalk walk(ms.piece[0], ms.piece[1]);
            Item it;
            bool ok = true;
            uint32_t base = 0, n_q[2] = {0, 0}, n_p[2] = {0, 0};
            auto scores = [&](int s, int t, bool last_user) {
                const uint32_t slot = base + 2u * uint32_t(t), st = slot % NST;
                wait_for(ok, &ms.full[st], (slot / NST) & 1, err);
                if (!ok) return;
                tc_fence_after();
                const uint32_t a = q_at + uint32_t(s) * C::kQBytes, b = ring_at + st * C::kTileBytes;
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t off = uint32_t(k >> 2) * (128u * 128u) + uint32_t(k & 3) * 32u;
                    mma_bf16(tm + uint32_t(s) * 128u, sdesc_sw128(a + off), sdesc_sw128(b + off), id_s, k > 0);
                }
                if (last_user) mma_commit(&ms.empty[st]);
                mma_commit(&ms.s_full[s]);
            };
            while (ok && walk.next(p, it)) {
                const int nv[2] = {side_tiles<kByKeys>(it, 0), side_tiles<kByKeys>(it, 1)};
                const int last_side = kByKeys ? -1 : (nv[1] > 0 ? 1 : 0);  // the last user of a shared tile
                for (int s = 0; s < 2 && ok; ++s) {
                    if (nv[s] == 0) continue;
                    wait_for(ok, &ms.q_full[s], n_q[s]++ & 1, err);
                    scores(s, kByKeys ? s : 0, kByKeys || s == last_side);
                }
                for (int v = 0; v < max(nv[0], nv[1]) && ok; ++v) {
                    for (int s = 0; s < 2 && ok; ++s) {
                        if (v >= nv[s]) continue;
                        const int t = kByKeys ? 2 * v + s : v;
                        const uint32_t slot = base + 2u * uint32_t(t) + 1u, st = slot % NST;
                        wait_for(ok, &ms.p_ready[s], n_p[s]++ & 1, err);
                        wait_for(ok, &ms.full[st], (slot / NST) & 1, err);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t b = ring_at + st * C::kTileBytes;
#pragma unroll
                        for (int k = 0; k < KT / 16; ++k)
                            mma_bf16_ta(tm + 256u + uint32_t(s) * 128u, tm + uint32_t(s) * 128u + uint32_t(k) * 8u,
                                        sdesc_sw128_mn(b + uint32_t(k) * 2048u, KT * 128u), id_o);
                        if (kByKeys || s == last_side) mma_commit(&ms.empty[st]);
                        if (v + 1 < nv[s]) scores(s, kByKeys ? t + 2 : t + 1, kByKeys || s == last_side);
                        else mma_commit(&ms.o_full[s]);
                    }
                }
                base += 2u * uint32_t((it.k1 - it.k0 + KT - 1) / KT);
            }
            mma_commit(&ms.done);  // nothing of this CTA's is in flight when its tensor memory goes
            mbar_wait(&ms.done, 0, err);
        } else if (ms.has && warp == 9) {
            // ---- page fetches ------------------------------------------------------------
            const int page_rows = 1 << p.b.page_shift, boxes = KT >> p.b.page_shift;
            ItemWalk walk(ms.piece[0], ms.piece[1]);
            Item it;
            bool ok = true;
            uint32_t slot = 0;
            while (ok && walk.next(p, it)) {
                for (int kb = it.k0; kb < it.k1 && ok; kb += KT) {
                    int page = -1;
                    if (lane < boxes && kb + lane * page_rows < it.k1) page = load_page(p.b, it.n, kb + lane * page_rows);
                    const int there = __popc(__ballot_sync(0xffffffffu, page >= 0));
                    const int plane = page * p.hkv + it.h;  // below 2^31 (checked on the host)
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv, ++slot) {
                        const CUtensorMap *map = kv ? &maps.v : &maps.k;
                        if constexpr (kE4m3) {
                            const uint32_t st = slot % 2;
                            wait_for(ok, &ms.raw_empty[st], ((slot / 2) & 1) ^ 1, err);
                            if (!(ok = __all_sync(0xffffffffu, ok))) break;
                            if (lane == 0) mbar_arrive_expect_tx(&ms.raw_full[st], uint32_t(there * page_rows * D));
                            __syncwarp();
                            if (page >= 0)
                                tma_load_3d(smem + C::kRawAt + st * C::kRawBytes + lane * page_rows * D, map, &ms.raw_full[st],
                                            0, 0, plane);
                        } else {
                            const uint32_t st = slot % NST;
                            wait_for(ok, &ms.empty[st], ((slot / NST) & 1) ^ 1, err);
                            if (!(ok = __all_sync(0xffffffffu, ok))) break;
                            if (lane == 0) mbar_arrive_expect_tx(&ms.full[st], uint32_t(there * page_rows * D * 2));
                            __syncwarp();
                            if (page >= 0) {
                                unsigned char *dst = ring + st * C::kTileBytes + lane * page_rows * 128;
#pragma unroll
                                for (int c = 0; c < D / 64; ++c)
                                    tma_load_3d(dst + c * KT * 128, map, &ms.full[st], c * 64, 0, plane);
                            }
                        }
                    }
                }
            }
            // a given-up wait elsewhere may leave copies in flight: they land before the CTA ends
            if (!ok) {
                for (uint32_t i = 1; i <= (kE4m3 ? 2u : uint32_t(NST)) && i <= slot; ++i) {
                    const uint32_t c = slot - i;
                    if (kE4m3) mbar_wait(&ms.raw_full[c % 2], (c / 2) & 1, err);
                    else mbar_wait(&ms.full[c % NST], (c / NST) & 1, err);
                }
            }
        } else if (kE4m3 && ms.has && warp >= 12) {
            // ---- e4m3 tiles to bf16 ---------------------------------------------------------
            constexpr int UPK = D / 16;  // 16-byte pieces of a key
            const int ct = tid - 384;
            ItemWalk walk(ms.piece[0], ms.piece[1]);
            Item it;
            bool ok = true;
            uint32_t slot = 0;
            while (ok && walk.next(p, it)) {
                for (int kb = it.k0; kb < it.k1 && ok; kb += KT) {
#pragma unroll 1
                    for (int kv = 0; kv < 2; ++kv, ++slot) {
                        // scales first: thread i looks up key i's, and the pieces get theirs by shuffle or memory
                        const uint8_t *scales = kv ? p.sv : p.sk;
                        float f[UPK];
#pragma unroll
                        for (int i = 0; i < UPK; ++i) {
                            const int key = (i * 128 + ct) / UPK, j = kb + key;
                            f[i] = 0.f;
                            if (j < it.k1) {
                                const int page = p.b.table[size_t(it.n) * size_t(p.b.table_stride) + size_t(j >> p.b.page_shift)];
                                if (page >= 0 && page < p.b.num_pages)
                                    f[i] = exp2_biased(scales[((size_t(page) * size_t(p.hkv) + size_t(it.h)) << p.b.page_shift) +
                                                              size_t(j & ((1 << p.b.page_shift) - 1))]);
                            }
                        }
                        const uint32_t rs = slot % 2, st = slot % NST;
                        wait_for(ok, &ms.raw_full[rs], (slot / 2) & 1, err);
                        wait_for(ok, &ms.empty[st], ((slot / NST) & 1) ^ 1, err);
                        if (!(ok = __all_sync(0xffffffffu, ok))) break;
                        const uint4 *raw = reinterpret_cast<const uint4 *>(smem + C::kRawAt + rs * C::kRawBytes);
                        unsigned char *dst = ring + st * C::kTileBytes;
#pragma unroll
                        for (int i = 0; i < UPK; ++i) {
                            const int key = (i * 128 + ct) / UPK, c = (i * 128 + ct) % UPK;
                            const uint4 w = raw[i * 128 + ct];
                            const uint32_t in[4] = {w.x, w.y, w.z, w.w};
                            uint32_t o[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const float2 t = unpack_e4m3(uint16_t(in[e / 2] >> ((e & 1) * 16)));
                                o[e] = pack_bf16(t.x * f[i], t.y * f[i]);
                            }
                            *reinterpret_cast<uint4 *>(dst + sw128_chunk(key, 2 * c, KT)) = make_uint4(o[0], o[1], o[2], o[3]);
                            *reinterpret_cast<uint4 *>(dst + sw128_chunk(key, 2 * c + 1, KT)) = make_uint4(o[4], o[5], o[6], o[7]);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&ms.full[st]), mbar_arrive(&ms.raw_empty[rs]);
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

// [num_pages * num_kv_heads][page_size][head_dim]; a box is one page of one
// head (64 channels of it for bf16, whose tiles are 128-byte swizzled).
bool page_map(CUtensorMap *m, const void *base, const kda_kv_cache *c, bool e4m3) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t esize = e4m3 ? 1 : 2, D = cuuint64_t(c->head_dim), P = cuuint64_t(c->page_size);
    const cuuint64_t dims[3] = {D, P, cuuint64_t(c->num_pages) * cuuint64_t(c->num_kv_heads)};
    const cuuint64_t strides[2] = {D * esize, D * P * esize};
    const cuuint32_t box[3] = {cuuint32_t(e4m3 ? c->head_dim : 64), cuuint32_t(c->page_size), 1u};
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
    p.min_keys = (kByKeys ? 4 : 2) * KT;
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
