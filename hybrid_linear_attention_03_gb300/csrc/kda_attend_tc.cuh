// kda_attend_tc.cuh -- building blocks of the attention kernels on the tensor
// cores: rings of key and value tiles, their barriers, e4m3 pages.
#pragma once

#include <cudaTypedefs.h>

#include <mutex>

#include "kda_attend.cuh"
#include "kda_sm100.cuh"

namespace kda {
namespace kv {
namespace {  // every translation unit has its own kernels and their helpers

using namespace sm100;

constexpr int KT = 128;  // keys of a tile

// Barriers of a ring's tiles, more than it has stages: tile t lands in stage
// t % stages but reports on barrier t % kBars.  A wait for tile t by parity is sound
// while the barrier is in t's phase or just past it.
//   Not before: the phase of tile t - kBars has passed.  Inside an item that holds for
// every role that takes all tiles or every second one, which has waited for that tile
// itself (kBars is even).  From item to item, in the kernels over pages of keys and values
// (that of kda_latent_prefill.cu has reasons of its own, given there), it rests on the order of the items: an odd
// number of tiles makes the sides swap barriers, a side may sit an item out, and the
// softmax waits for values only where it checks them.  But nobody waits for an item's
// tiles before its rows of Q (q_full, row_unit) or the scores that need them, and the
// warps that bring those have first been through all value tiles (e4m3 in the tile
// kernel: and key tiles) of the items before, and have waited for all their scores
// (q_free).  Whoever brings Q earlier than that has to give these waits another order.
//   Not two past: tile t + kBars takes a stage that the fetching warp finds free only
// after it found that of tile t free, which t's users say when they are done with it.
constexpr int kBars = 8;

// ---- PTX ---------------------------------------------------------
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
// Biased exponents for kB rows of Q, of each of which kLanes neighbouring lanes
// hold eight bf16 a piece; -1 for a row with an infinity or NaN.  The rows'
// shuffles go by turns, so that they do not wait for each other.
template <int kLanes, int kB> __device__ __forceinline__ void row_exponents(const uint4 (&raw)[kB], int (&e)[kB]) {
    uint32_t m[kB];  // the largest magnitude as a bf16 pattern
#pragma unroll
    for (int b = 0; b < kB; ++b) {
        const uint32_t t = __vmaxu2(__vmaxu2(raw[b].x & 0x7fff7fffu, raw[b].y & 0x7fff7fffu),
                                    __vmaxu2(raw[b].z & 0x7fff7fffu, raw[b].w & 0x7fff7fffu));
        m[b] = max(t & 0xffffu, t >> 16);
    }
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1)
#pragma unroll
        for (int b = 0; b < kB; ++b) m[b] = max(m[b], __shfl_xor_sync(0xffffffffu, m[b], o));
#pragma unroll
    for (int b = 0; b < kB; ++b) e[b] = m[b] >= 0x7f80u ? -1 : max(scale_exponent(__uint_as_float(m[b] << 16)), 1);
}
// Eight bf16 of a row with that exponent as two e4m3 terms times its power of two
// (a row with infinities or NaN as NaN).
__device__ __forceinline__ void split_row(const uint4 &raw, int e, uint32_t (&w1)[2], uint32_t (&w2)[2]) {
    const uint32_t in[4] = {raw.x, raw.y, raw.z, raw.w};
    const float f = e < 0 ? NAN : exp2_neg_biased(e);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = __uint_as_float(in[i] << 16) * f, b = __uint_as_float(in[i] & 0xffff0000u) * f;
        const uint16_t h1 = pack_e4m3(a, b);
        const float2 t = unpack_e4m3(h1);
        const uint16_t h2 = pack_e4m3(a - t.x, b - t.y);
        if (i % 2 == 0) w1[i / 2] = h1, w2[i / 2] = h2;
        else w1[i / 2] |= uint32_t(h1) << 16, w2[i / 2] |= uint32_t(h2) << 16;
    }
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

// ---- waits that may give up ----------------------------------------------
// Every wait is bounded, and skipped once the thread has given up.  A warp whose lane 0
// has given up
//   - arrives at no mbarrier any more, so none completes a phase that its owner did not
//     reach: the roles that still run keep their order, and give up in their turn where
//     they depend on this one (the lanes meet behind each wait, so that lane 0 speaks
//     for all of them);
//   - follows no address that others should have left in shared memory (the lists of keys
//     taken out of a tile; scales, scores and weights may be anything);
//   - meets the hardware's barriers as before (their number follows from the tables alone).
// The issuing and fetching warps then stop, wait for their own products and copies, and
// the CTA ends as usual.  KDA_ATTEND_LOOKS: a build for the test of all this, whose waits
// look that often and no more.
__device__ __forceinline__ void wait_for(bool &ok, uint64_t *bar, uint32_t parity, uint32_t *err) {
#ifndef KDA_ATTEND_LOOKS
    if (ok) ok = mbar_wait(bar, parity, err);
#else
    uint32_t passed = ok ? 0 : 1;
    for (int i = 0; i < KDA_ATTEND_LOOKS && !passed; ++i)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(passed)
            : "r"(smem_u32(bar)), "r"(parity)
            : "memory");
    if (!passed) atomicOr(err, KDA_DEVERR_TIMEOUT), ok = false;
#endif
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
// Has a kernel's maps fetched while it sets up.
__device__ __forceinline__ void prefetch_maps(const TileMaps &m) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&m.k) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&m.v) : "memory");
}

__device__ __forceinline__ int item_tiles(const Item &it) { return (it.k1 - it.k0 + KT - 1) / KT; }
// The table's entry for keys [kb + 16 lane, kb + 16 lane + 16) of the tile at kb (page 0 where there
// are none).  Asked for a tile ahead: a look-up on the way took a fifth of the softmax's time.
__device__ __forceinline__ int peek_page(const AttendParams &p, const Item &it, int kb, int lane) {
    const int j = kb + lane * 16;
    if (lane >= KT / 16 || j >= it.k1) return 0;
    return p.b.table[size_t(it.n) * size_t(p.b.table_stride) + size_t(j >> p.b.page_shift)];
}
// Bit g: keys [kb + 16 g, kb + 16 g + 16) are in a page outside the cache (which the warps that
// fetch pages report).
__device__ __forceinline__ uint32_t absent_groups(const AttendParams &p, int page) {
    return __ballot_sync(0xffffffffu, uint32_t(page) >= uint32_t(p.b.num_pages));
}
// Some row of the item does not see some key of the tile at kb.
__device__ __forceinline__ bool partly_seen(const Item &it, int kb, uint32_t absent) {
    return absent != 0 || kb + KT - 1 > it.ctx + it.tok0;
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

// Where a tile goes: its barrier, its stage, and (e4m3) its scales' place.
struct Landing {
    uint64_t *full;
    unsigned char *dst;
    uint8_t *scales;
};
// One warp fetches the key tiles, or the value tiles, of a piece.  land(t) waits
// for tile t's stage; bars and depth are those of the ring.
template <int D, bool kE4m3, typename F>
__device__ __forceinline__ void fetch_pages(const AttendParams &p, const TileMaps &maps, const Cursor &from, const Cursor &to,
                                            bool values, bool &ok, F land, uint64_t *bars, int depth) {
    const int lane = int(threadIdx.x) & 31, page_size = 1 << p.b.page_shift, box = min(page_size, KT);
    const CUtensorMap *map = values ? &maps.v : &maps.k;
    ItemWalk walk(from, to);
    Item it = {};
    uint32_t t = 0;
    while (ok && walk.next(p, it)) {
        auto page_at = [&](int kb) {
            const int j = kb + lane * box;
            return lane * box < KT && j < it.k1 ? load_page(p.b, it.n, j) : -1;
        };
        int next = page_at(it.k0);
        for (int kb = it.k0; kb < it.k1 && ok; kb += KT, ++t) {
            const int page = next, line = (kb + lane * box) & (page_size - 1);
            next = page_at(kb + KT);
            const Landing to_ring = land(t, values);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            const int there = __popc(__ballot_sync(0xffffffffu, page >= 0)) * box;
            const int plane = page * p.hkv + it.h;  // below 2^31 (checked on the host)
            if (lane == 0) mbar_arrive_expect_tx(to_ring.full, uint32_t(there * (kE4m3 ? D + 1 : 2 * D)));
            __syncwarp();
            if (page >= 0) {
                if constexpr (kE4m3) {
                    tma_load_3d(to_ring.dst + lane * box * D, map, to_ring.full, 0, line, plane);
                    bulk_load(to_ring.scales + lane * box, (values ? p.sv : p.sk) + (size_t(plane) << p.b.page_shift) + line,
                              uint32_t(box), to_ring.full);
                } else {
#pragma unroll
                    for (int c = 0; c < D / 64; ++c)
                        tma_load_3d(to_ring.dst + lane * box * 128 + c * KT * 128, map, to_ring.full, c * 64, line, plane);
                }
            }
            __syncwarp();
        }
    }
    // whichever role gives up, no copy is in flight when the CTA ends
    for (uint32_t i = t - min(t, uint32_t(depth)); i < t; ++i) mbar_wait(&bars[i % kBars], (i / kBars) & 1, p.b.err);
}
// Warp w of eight widens its 16 keys of a raw value tile, and looks them over
// where some row does not see some key; odd: the tile's keys taken out.
template <int D>
__device__ __forceinline__ void widen_tile(const AttendParams &p, const Item &it, int kb, uint32_t absent,
                                           const unsigned char *raw, unsigned char *dst, const uint8_t *scale, int w, int lane, uint32_t *odd) {
    using RP = RawPiece<D>;
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
    uint32_t out = 0;
    if (partly_seen(it, kb, absent)) {
        const Item copy = it;
        __syncwarp();
        out = look_over_raw<D>(p, copy, kb, absent, raw, dst, scale, w, lane);
    }
    fence_proxy_async_smem();
    if (lane == 0) reinterpret_cast<uint16_t *>(odd)[w] = uint16_t(out);
    __syncwarp();
}
// Warp w of four looks over 32 keys of a bf16 value tile, likewise.
template <int D>
__device__ __forceinline__ void look_over_tile(const Item &it, int kb, uint32_t absent, unsigned char *tile, int w, int lane,
                                               uint32_t *odd) {
    uint32_t out = 0;
    if (partly_seen(it, kb, absent)) {
        // a lane looks over one value row, each at a bank of its own
        const int row = w * 32 + lane, j = kb + row;
        unsigned char *img = tile + row * 128;
        const bool gone = j >= it.k1 || (absent >> (row / 16) & 1);
        bool bad = false;
        for (int c = 0; c < D / 8; ++c)
            bad |= odd_bf16(*reinterpret_cast<const uint4 *>(img + (c >> 3) * KT * 128 + (((c & 7) ^ (lane & 7)) << 4)));
        bad = bad && !gone && j > it.ctx + it.tok0;  // rows that every query sees stay
        if (gone || bad) {
            for (int c = 0; c < D / 8; ++c)
                *reinterpret_cast<uint4 *>(img + (c >> 3) * KT * 128 + (((c & 7) ^ (lane & 7)) << 4)) = make_uint4(0, 0, 0, 0);
        }
        out = __ballot_sync(0xffffffffu, bad);
        fence_proxy_async_smem();
    }
    if (lane == 0) odd[w] = out;
    __syncwarp();
}

inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
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
// or 64 bytes.  Heads of 16 or 32 channels fill the first of a box's 64 (the
// copy fills the others with zeros, which add nothing to a product).
inline bool page_map(CUtensorMap *m, const void *base, const kda_kv_cache *c, bool e4m3) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t esize = e4m3 ? 1 : 2, D = cuuint64_t(c->head_dim), P = cuuint64_t(c->page_size);
    const cuuint64_t dims[3] = {D, P, cuuint64_t(c->num_pages) * cuuint64_t(c->num_kv_heads)};
    const cuuint64_t strides[2] = {D * esize, D * P * esize};
    const int image = c->head_dim < 64 ? 64 : c->head_dim;
    const cuuint32_t box[3] = {cuuint32_t(e4m3 ? image : 64), cuuint32_t(c->page_size < KT ? c->page_size : KT), 1u};
    const cuuint32_t estr[3] = {1u, 1u, 1u};
    return fn(m, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims,
              strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              e4m3 && image == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace kv
}  // namespace kda
