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
// A tile is worked on in two halves of 64 keys, each with its own score columns:
// while the threads of a side turn one half into weights, the other half's
// product and the scores that follow in its place are under way, so the threads
// seldom wait and the tensor cores seldom idle.
// ref is the row's maximum so far, but only moved (and O and the sums scaled
// by 2^(ref - ref')) when a tile exceeds it by more than 8: weights then reach
// 2^8 at most, which costs no precision in bf16 and fp32, and most tiles leave
// O in tensor memory untouched.  P is rounded to bf16 (2^-9 relative, the
// size of the output's own rounding, and not correlated between keys); scores,
// sums and O stay in 32 bits.
//
// Warps: 0-3 side 0, 4-7 side 1 (a thread a row); 8 and 9 issue a side's
// products each; 10 and 11 fetch
// pages by TMA into rings of key and value tiles; 12-15 bring the rows of Q and
// look value tiles over (below).
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
#include <cudaTypedefs.h>

#include <mutex>

#include "kda_attend.cuh"
#include "kda_sm100.cuh"

namespace kda {
namespace kv {
namespace {

using namespace sm100;

constexpr int KT = 128;          // keys of a tile
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
constexpr float kRefSlack = 8.f;
constexpr int kItemCost = 512;  // keys that take as long as an item's start and output

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
// Barriers of a ring's tiles, more than it has stages: tile t lands in stage
// t % stages but reports on barrier t % kBars.  A wait by parity is only sound for
// a thread that sees every phase of its barrier, and a side that takes every
// second tile sees every phase of every barrier it uses (kBars is even), whatever
// the number of stages and the order in which copies land.
constexpr int kBars = 8;

template <typename C> struct alignas(16) Misc {
    uint64_t k_full[kBars], k_empty[kBars], v_full[kBars], v_empty[kBars], clean[kBars];
    uint64_t raw_full[kBars], raw_empty[kBars], unit_full[kBars];
    uint64_t s_full[2][2], p_ready[2][2], pv_done[2][2];  // by side and half
    uint64_t q_full[2], q_free[2], done[2];
    uint64_t row_unit[2][2];  // e4m3, by image and item parity: the rows' scales are there
    uint32_t tmem;
    int has, rows_gave_up;
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
// D[tmem] (+)= A[smem] * B[smem]^T, e4m3 inputs (32 K values an instruction).
__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Instruction descriptor: e4m3 A and B, both K-major, fp32 D.
constexpr uint32_t idesc_e4m3_f32(int M, int N) { return (1u << 4) | (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24); }
// Rows of D e4m3 values, K-major, swizzled over their 128 or 64 bytes: byte
// offset of a row's 16-byte piece, and the operand descriptor (8 rows a group).
template <int D> __host__ __device__ __forceinline__ uint32_t row8_piece(int row, int c) {
    return uint32_t(row * D) + uint32_t((D == 128 ? c ^ (row & 7) : c ^ ((row >> 1) & 3)) << 4);
}
template <int D> __device__ __forceinline__ uint64_t sdesc_row8(uint32_t saddr) {
    return uint64_t((saddr & 0x3FFFFu) >> 4) | uint64_t(1) << 16 | uint64_t(8 * D >> 4) << 32 | uint64_t(1) << 46 |
           uint64_t(D == 128 ? 2 : 4) << 61;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 d, a, b;\n\t"
        "mov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
// 16-byte asynchronous copy, or zeros.
__device__ __forceinline__ void cp_async16_or_zero(void *smem_dst, const void *gsrc, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(smem_dst)), "l"(gsrc), "r"(there ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
template <int N, int kLaunch> __device__ __forceinline__ void set_regs() {
    if constexpr (N > kLaunch) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int kId, int kCount> __device__ __forceinline__ void named_sync() {
    asm volatile("bar.sync %0, %1;" ::"n"(kId), "n"(kCount) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
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
// 16 e4m3 values times a power of two as bf16, exactly.  (Moving the bits by
// integer instructions and one packed product takes as long and loses the ALU
// time that the softmax wants.)
__device__ __forceinline__ void widen_e4m3(const uint4 &q, float f, uint32_t (&o)[8]) {
    const uint32_t in[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 t = mul2(unpack_e4m3(uint16_t(in[i / 2] >> ((i & 1) * 16))), make_float2(f, f));
        o[i] = pack_bf16(t.x, t.y);
    }
}
// Eight bf16 of a row of Q, of which kLanes neighbouring lanes hold one row, as
// two e4m3 terms times a power of two; returns its biased exponent.
template <int kLanes> __device__ __forceinline__ int split_row(const uint4 &raw, uint32_t (&w1)[2], uint32_t (&w2)[2]) {
    const uint32_t in[4] = {raw.x, raw.y, raw.z, raw.w};
    // the largest magnitude as a bf16 pattern, of finite values (a row with others is NaN all the same)
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __vmaxu2(m, in[i] & 0x7fff7fffu);
    m = max(m & 0xffffu, m >> 16);
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    const bool odd = m >= 0x7f80u;
    const int e = odd ? 127 : max(scale_exponent(__uint_as_float(m << 16)), 1);
    const float f = odd ? NAN : exp2_neg_biased(e);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = __uint_as_float(in[i] << 16) * f, b = __uint_as_float(in[i] & 0xffff0000u) * f;
        const uint16_t h1 = pack_e4m3(a, b);
        const float2 t = unpack_e4m3(h1);
        const uint16_t h2 = pack_e4m3(a - t.x, b - t.y);
        if (i % 2 == 0) w1[i / 2] = h1, w2[i / 2] = h2;
        else w1[i / 2] |= uint32_t(h1) << 16, w2[i / 2] |= uint32_t(h2) << 16;
    }
    return e;
}
// Bit 7 of a byte is set where one of the 16 codes is NaN.
__device__ __forceinline__ uint32_t nan_codes(const uint4 &q) {
    return (((q.x & 0x7f7f7f7fu) + 0x01010101u) | ((q.y & 0x7f7f7f7fu) + 0x01010101u) |
            ((q.z & 0x7f7f7f7fu) + 0x01010101u) | ((q.w & 0x7f7f7f7fu) + 0x01010101u)) & 0x80808080u;
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
// Tile t's barrier of a ring has been passed.
__device__ __forceinline__ void wait_tile(bool &ok, uint64_t *bars, uint32_t t, uint32_t *err) {
    wait_for(ok, &bars[t % kBars], (t / kBars) & 1, err);
}
// The stage that tile t will take is free: the tile before it there has been used.
template <int kStages> __device__ __forceinline__ void wait_stage(bool &ok, uint64_t *empty, uint32_t t, uint32_t *err) {
    static_assert(kStages < kBars, "a tile's barrier is free before its stage");
    if (t >= kStages) wait_tile(ok, empty, t - kStages, err);
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
__device__ __forceinline__ bool any_odd(const uint32_t *odd) { return (odd[0] | odd[1]) != 0; }  // of a half

struct TileMaps {
    CUtensorMap k, v;
};

// ItemWalk::next out of line (every role has a copy of the walk); the caller's
// item stays in its registers.
__device__ __forceinline__ bool next_item_call(const AttendParams &p, ItemWalk *walk, Item *it) { return walk->next(p, *it); }
__device__ __forceinline__ bool next_item(const AttendParams &p, ItemWalk &walk, Item &it) {
    Item got;
    const bool has = next_item_call(p, &walk, &got);
    if (has) it = got;
    return has;
}
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
    for (int g = 0; g < KH / 32; ++g) {
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

// Piece u of a lane in the widening of a raw e4m3 tile: a warp has 16 keys, and
// 8 neighbouring lanes take the same 16-byte piece of 8 keys, which both tiles'
// swizzles put into different banks.
template <int D> struct RawPiece {
    static constexpr int kPerKey = D / 64, kCount = 2 * kPerKey;  // of a key, of a lane
    int key;
    uint32_t from, to;  // byte offsets in the raw and the wide tile (whose next 16 bytes are at to ^ 16)
    __device__ __forceinline__ RawPiece(int w, int lane, int u) {
        const int c = lane >> 3, k0 = w * 16 + (lane & 7), g = u / kPerKey, i = u % kPerKey;
        key = k0 + 8 * g;
        from = (row8_piece<D>(k0, c) ^ uint32_t(i * 64)) + uint32_t(8 * g * D);
        to = sw128_chunk(k0, 2 * c, KT) + uint32_t(g * 1024 + i * KT * 128);
    }
};
// A widened tile of which some row does not see some key: zeroes the rows of
// absent keys and takes out the non-finite ones that not every row sees.
// Returns the keys taken out, a bit each of the warp's 16.
template <int D>
__device__ __noinline__ uint32_t look_over_raw(const AttendParams &p, const Item &it, int kb, uint32_t absent,
                                               const unsigned char *raw, unsigned char *dst, const uint8_t *scale, int w,
                                               int lane) {
    uint32_t odd = 0;
#pragma unroll 1
    for (int g = 0; g < 2; ++g) {
        const int key = w * 16 + 8 * g + (lane & 7), j = kb + key;
        uint32_t nan = scale[key] >= 247;  // 448 * 2^(247 - 127) is past bf16's range, and 255 is NaN
        for (int i = 0; i < RawPiece<D>::kPerKey; ++i)
            nan |= nan_codes(*reinterpret_cast<const uint4 *>(raw + RawPiece<D>(w, lane, g * RawPiece<D>::kPerKey + i).from));
        nan |= __shfl_xor_sync(0xffffffffu, nan, 8);
        nan |= __shfl_xor_sync(0xffffffffu, nan, 16);
        const bool gone = j >= it.k1 || (absent >> (key / 16) & 1);
        const bool out = !gone && nan != 0 && j > it.ctx + it.tok0;
        odd |= (__ballot_sync(0xffffffffu, out) & 0xffu) << (8 * g);
        if (gone || out) {
            for (int i = 0; i < RawPiece<D>::kPerKey; ++i) {
                const uint32_t to = RawPiece<D>(w, lane, g * RawPiece<D>::kPerKey + i).to;
                *reinterpret_cast<uint4 *>(dst + to) = make_uint4(0, 0, 0, 0);
                *reinterpret_cast<uint4 *>(dst + (to ^ 16u)) = make_uint4(0, 0, 0, 0);
            }
        }
    }
    return odd;
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
    if (warp == 8) tmem_alloc(&ms.tmem, 512);
    wait_prior_kernel();
    allow_next_kernel();
    if (tid < 2) p.parts[2 * cta + tid].state = 0;
    if (warp == 10) {
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
            while (next_item(p, walk, it)) {
                const int nv = side_tiles<kByKeys>(it, s);
                const int lim = it.ctx + it.tok0 + min(r, it.rows - 1) / p.group;  // last key this row sees
                const bool live = r - lane < it.rows;  // this warp has rows of the item
                float ref = -INFINITY, l = 0.f, scale = p.scale_log2;
                if constexpr (kE4m3) {
                    if (nv > 0) {
                        // by item parity: Q may be an item ahead of this side's threads, never two
                        const int qi = kByKeys ? 0 : s;
                        wait_for(ok, &ms.row_unit[qi][n_it & 1], (n_it >> 1) & 1, err);
                        scale *= sc8.q_unit[n_it & 1][qi][row];
                    }
                    if (kByKeys || nv > 0) ++n_it;
                }
                for (int v = 0; v < nv; ++v, ++n_s) {
                    const int t = side_tile<kByKeys>(s, v), kb = it.k0 + t * KT;
                    const uint32_t absent = absent_groups(p, it, kb, lane);
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
                            tmem_wait_ld();
                            if constexpr (kE4m3) {
#pragma unroll
                                for (int c = 0; c < KH; c += 4) {
                                    const float4 u = *reinterpret_cast<const float4 *>(&sc8.k_unit[tg % kUnits][h * KH + c]);
                                    const float2 a = mul2(make_float2(x[c], x[c + 1]), make_float2(u.x, u.y));
                                    const float2 b = mul2(make_float2(x[c + 2], x[c + 3]), make_float2(u.z, u.w));
                                    x[c] = a.x, x[c + 1] = a.y, x[c + 2] = b.x, x[c + 3] = b.y;
                                }
                            }
                            if (check) {
#pragma unroll
                                for (int c = 0; c < KH; ++c)
                                    if (kh + c > lim || (absent >> (h * (KH / 16) + c / 16) & 1)) x[c] = -INFINITY;
                            }
                            float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                            for (int c = 4; c < KH; c += 8)
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    mx[i] = c + 4 + i < KH ? fmaxf(fmaxf(mx[i], x[c + i]), x[c + 4 + i]) : fmaxf(mx[i], x[c + i]);
                            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale;
                            const bool move = top > ref + kRefSlack;
                            const bool started = v > 0 || h > 0;  // O is new with the first product
                            if (__any_sync(0xffffffffu, move)) {
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
                            }
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
                            l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                            tmem_wait_st();
                            if (check) {
                                wait_tile(ok, kE4m3 ? ms.v_full : ms.clean, tg, err);
                                __syncwarp();
                                const uint32_t *odd = &ms.odd[tg % kBars][h * (KH / 32)];
                                if (any_odd(odd)) {
                                    if (started) wait_o(h == 0 ? n_s - 1 : n_s, h ^ 1);
                                    const Item copy = it;
                                    add_odd_rows<D, kE4m3>(p, copy, kh, lim, odd, t_h, t_o, !started);
                                }
                            }
                        }  // else rows of nobody: their weights may be anything
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&ms.p_ready[s][h]);
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
                    float *data = p.part_data + (size_t(cta) * 2 + it.slot()) * size_t(BM) * (D + 2);
                    __nv_bfloat16 *dst =
                        static_cast<__nv_bfloat16 *>(p.out) + it.at(min(r, it.rows - 1), p.group, p.out_stride, D);
#pragma unroll 2
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
            while (ok && next_item(p, walk, it)) {
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
            bool end_ok = true;
            wait_for(end_ok, &ms.done[s], 0, err);
        } else if (ms.has) {
            // ---- page fetches: keys, or values ------------------------------------------------
            const bool values = warp == 11;
            const CUtensorMap *map = values ? &maps.v : &maps.k;
            const int page_size = 1 << p.b.page_shift, box = min(page_size, KT);
            ItemWalk walk(ms.piece[0], ms.piece[1]);
            Item it = {};
            uint32_t tg = 0;
            auto fetch = [&](int kb, uint64_t *full, unsigned char *dst, uint8_t *scales) {
                const int j = kb + lane * box, line = j & (page_size - 1);
                int page = -1;
                if (lane * box < KT && j < it.k1) page = load_page(p.b, it.n, j);
                const int there = __popc(__ballot_sync(0xffffffffu, page >= 0)) * box;
                const int plane = page * p.hkv + it.h;  // below 2^31 (checked on the host)
                if (lane == 0) mbar_arrive_expect_tx(full, uint32_t(there * (kE4m3 ? D + 1 : 2 * D)));
                __syncwarp();
                if (page < 0) return;
                if constexpr (kE4m3) {
                    tma_load_3d(dst + lane * box * D, map, full, 0, line, plane);
                    bulk_load(scales + lane * box, (values ? p.sv : p.sk) + (size_t(plane) << p.b.page_shift) + line,
                              uint32_t(box), full);
                } else {
#pragma unroll
                    for (int c = 0; c < D / 64; ++c)
                        tma_load_3d(dst + lane * box * 128 + c * KT * 128, map, full, c * 64, line, plane);
                }
            };
            while (ok && next_item(p, walk, it)) {
                for (int kb = it.k0; kb < it.k1 && ok; kb += KT, ++tg) {
                    if (!values) wait_stage<NK>(ok, ms.k_empty, tg, err);
                    else if (kE4m3) wait_stage<NR>(ok, ms.raw_empty, tg, err);
                    else wait_stage<NV>(ok, ms.v_empty, tg, err);
                    if (!(ok = __all_sync(0xffffffffu, ok))) break;
                    if (!values) fetch(kb, &ms.k_full[tg % kBars], k_ring + tg % NK * C::kKBytes, sc8.k[tg % NK]);
                    else if (kE4m3) fetch(kb, &ms.raw_full[tg % kBars], raw_ring + tg % NR * C::kRawBytes, sc8.v[tg % NR]);
                    else fetch(kb, &ms.v_full[tg % kBars], v_ring + tg % NV * C::kVBytes, nullptr);
                }
            }
            // a given-up wait elsewhere may leave copies in flight: they land before the CTA ends
            if (!ok) {
                uint64_t *bars = !values ? ms.k_full : kE4m3 ? ms.raw_full : ms.v_full;
                const uint32_t depth = uint32_t(!values ? NK : kE4m3 ? NR : NV);
                bool end_ok = true;
                for (uint32_t t = tg - min(tg, depth); t < tg; ++t) wait_tile(end_ok, bars, t, err);
            }
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
            auto meet = [&] {
                if (w == 0 && !ok) ms.rows_gave_up = 1;
                named_sync<4, kRowThreads>();
                ok = ms.rows_gave_up == 0;
            };
            while (ok && next_item(p, walk, it)) {
                for (int s = 0; s < C::kQImages; ++s) {
                    if (side_tiles<kByKeys>(it, s) == 0) continue;
                    unsigned char *q_img = smem + s * C::kQBytes;
                    constexpr int CPR = D / 8, RPP = kRowThreads / CPR;  // 16-byte pieces of a row, rows a pass
                    const int c = qt % CPR;
                    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.q) + c * 8;
                    auto row_at = [&](int row) {  // this thread's piece of a row of the item
                        return q + it.at(min((kByKeys ? 0 : s * kSideRows) + row, it.rows - 1), p.group, p.q_stride, D);
                    };
                    auto is_there = [&](int row) { return (kByKeys ? 0 : s * kSideRows) + row < it.rows; };
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
#pragma unroll
                            for (int b = 0; b < kBatch; ++b) {
                                const int row = r0 + b * RPP;
                                uint32_t w1[2], w2[2];
                                const int e = split_row<CPR>(raw[b], w1, w2);
                                const uint32_t at = row8_piece<D>(row, c >> 1) + uint32_t(c & 1) * 8u;
                                *reinterpret_cast<uint2 *>(q_img + at) = make_uint2(w1[0], w1[1]);
                                *reinterpret_cast<uint2 *>(q_img + kSideRows * D + at) = make_uint2(w2[0], w2[1]);
                                if (c == 0) sc8.q_unit[n_q[s] & 1][s][row] = exp2_biased(e);
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
                for (int kb = it.k0; kb < it.k1 && ok; kb += KT, ++tile) {
                    const uint32_t absent = absent_groups(p, it, kb, lane);
                    unsigned char *dst = v_ring + tile % NV * C::kVBytes;
                    uint32_t odd = 0;  // keys taken out, of this warp's
                    if constexpr (kE4m3) {
                        using RP = RawPiece<D>;
                        const unsigned char *raw = raw_ring + tile % NR * C::kRawBytes;
                        const uint8_t *scale = sc8.v[tile % NR];
                        if (w == 0) {
                            wait_tile(ok, ms.k_full, tile, err), wait_tile(ok, ms.raw_full, tile, err);
                            wait_stage<NV>(ok, ms.v_empty, tile, err);
                        }
                        meet();
                        if (!ok) break;
                        if (qt < KT) sc8.k_unit[tile % kUnits][qt] = exp2_biased(sc8.k[tile % NK][qt]);  // as numbers
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&ms.unit_full[tile % kBars]), mbar_arrive(&ms.k_empty[tile % kBars]);
                        uint4 x[RP::kCount];
                        float f[2];
#pragma unroll
                        for (int u = 0; u < RP::kCount; ++u) {
                            const RP r(w, lane, u);
                            x[u] = *reinterpret_cast<const uint4 *>(raw + r.from);
                            if (u % RP::kPerKey == 0) f[u / RP::kPerKey] = exp2_biased(scale[r.key]);
                        }
#pragma unroll
                        for (int u = 0; u < RP::kCount; ++u) {
                            const RP r(w, lane, u);
                            uint32_t o[8];
                            widen_e4m3(x[u], f[u / RP::kPerKey], o);
                            *reinterpret_cast<uint4 *>(dst + r.to) = make_uint4(o[0], o[1], o[2], o[3]);
                            *reinterpret_cast<uint4 *>(dst + (r.to ^ 16u)) = make_uint4(o[4], o[5], o[6], o[7]);
                        }
                        __syncwarp();
                        if (partly_seen(it, kb, absent)) {
                            const Item copy = it;
                            odd = look_over_raw<D>(p, copy, kb, absent, raw, dst, scale, w, lane);
                        }
                        fence_proxy_async_smem();
                        if (lane == 0) reinterpret_cast<uint16_t *>(ms.odd[tile % kBars])[w] = uint16_t(odd);
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&ms.v_full[tile % kBars]), mbar_arrive(&ms.raw_empty[tile % kBars]);
                    } else {
                        if (w == 0) wait_tile(ok, ms.v_full, tile, err);
                        meet();
                        if (!ok) break;
                        if (partly_seen(it, kb, absent)) {
                            // a lane looks over one value row, each at a bank of its own
                            const int row = w * 32 + lane, j = kb + row;
                            unsigned char *img = dst + row * 128;
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
                        if (lane == 0) ms.odd[tile % kBars][w] = odd;
                        __syncwarp();
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
// one page and head (64 channels of it for bf16), swizzled over its row of 128
// or 64 bytes.
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
              e4m3 && c->head_dim == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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

bool tile_plan(const kda_kv_cache *c, const kda_kv_batch *b, AttendPlan *plan) {
    const long long rows = static_cast<long long>(b->max_new) * (c->num_heads / c->num_kv_heads);
    if (c->act != KDA_BF16 || (c->head_dim != 64 && c->head_dim != 128)) return false;
    plan->bm = rows <= kSideRows ? kSideRows : 2 * kSideRows;
    plan->n_cta = sm_count();
    return true;
}

kda_status tile_launch(const kda_kv_cache *c, AttendParams &p, const AttendPlan &plan, cudaStream_t stream) {
    return c->head_dim == 64 ? by_type<64>(c, p, plan, stream) : by_type<128>(c, p, plan, stream);
}

}  // namespace kv
}  // namespace kda
