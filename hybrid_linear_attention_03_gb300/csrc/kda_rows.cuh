// kda_rows.cuh -- what the kernels that write and read cache lines share: rows and
// their positions, 16 bytes of activations, the angles of a rotation.
#pragma once

#include <cmath>

#include "kda_kv.cuh"

namespace kda {
namespace kv {

template <typename Act> struct Vec;  // 16 bytes of activations
template <> struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void unpack(const uint4 &r, float (&x)[4]) {
        x[0] = __uint_as_float(r.x), x[1] = __uint_as_float(r.y);
        x[2] = __uint_as_float(r.z), x[3] = __uint_as_float(r.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[4]) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
};
template <> struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void unpack(const uint4 &r, float (&x)[8]) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

template <int N> __device__ __forceinline__ void store_e4m3(void *dst, const float (&y)[N]) {
    uint32_t w[N / 4];
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
        w[i] = uint32_t(pack_e4m3(y[4 * i], y[4 * i + 1])) | uint32_t(pack_e4m3(y[4 * i + 2], y[4 * i + 3])) << 16;
    if constexpr (N == 8)
        *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
    else
        *reinterpret_cast<uint32_t *>(dst) = w[0];
}

// The row of a CTA that a warp works on: its position and page, or pos = -1 for
// a row past the last sequence or of one whose tables are inconsistent.  Whole warp.
// The search supposes that cu_seqlens does not decrease.  Where it does it may name a
// sequence that the row is not in, whose position would lie outside the page table.
__device__ __forceinline__ void find_row(const BatchView &b, int r, int lane, int &pos, int &page) {
    pos = page = -1;
    const int n = r < b.max_rows ? find_seq(b, r, lane) : -1;
    if (lane == 0 && n >= 0 && n < b.n_seqs) {
        Seq s;
        if (load_seq(b, n, s, true)) {
            if (r >= s.row0 && r - s.row0 < s.T) {
                pos = s.L - s.T + (r - s.row0);
                page = load_page(b, n, pos);
            } else {
                atomicOr(b.err, KDA_DEVERR_META);
            }
        }
    }
}

// Has the inconsistent sequences reported that no row leads to, as those without rows:
// the grid's columns take 32 sequences a turn each (one warp, beside those that look up rows).
__device__ __forceinline__ void report_seqs(const BatchView &b, int lane) {
    for (long long n = blockIdx.x * 32LL + lane; n < b.n_seqs; n += gridDim.x * 32LL) {
        Seq s;
        load_seq(b, int(n), s, true);
    }
}

// Cosine and sine of the angle a * 2^-63 * pi (a two's complement), within 7e-8 (2.4e-8 in the mean: an
// e4m3 page turns an error next to a rounding border into a whole step of e4m3, so
// the last bit is worth having).  The quadrant comes off in integers; the rest, at
// most pi / 4, is held as a sum p + e of two floats; then Taylor series, whose
// terms past the first add less than a third of it.
__device__ __forceinline__ float2 cos_sin(uint64_t a) {
    constexpr float kPi = 3.14159274f, kPiRest = -8.74227766e-8f;  // their sum is pi to 48 bits
    const int q = int((a + (uint64_t(1) << 61)) >> 62);
    const int64_t r = int64_t(a - (uint64_t(q) << 62));
    const float hi = float(r), u = hi * 0x1p-63f, lo = float(r - __float2ll_rn(hi)) * 0x1p-63f;
    const float p = __fmul_rn(u, kPi), e = fmaf(lo, kPi, fmaf(u, kPiRest, fmaf(u, kPi, -p))), z = p * p;
    const float s3 = fmaf(z, fmaf(z, fmaf(z, 1.0f / 362880, -1.0f / 5040), 1.0f / 120), -1.0f / 6) * z;
    const float sn = p + fmaf(p, s3, e * fmaf(z, -0.5f, 1.0f));
    const float c2 = fmaf(z, fmaf(z, fmaf(z, fmaf(z, -1.0f / 3628800, 1.0f / 40320), -1.0f / 720), 1.0f / 24), -0.5f);
    const float cn = 1.0f + fmaf(z, c2, -p * e);
    const float c = q & 1 ? sn : cn, s = q & 1 ? cn : sn;  // turned by a quarter
    return make_float2(q == 1 || q == 2 ? -c : c, q >= 2 ? -s : s);
}

// f / (2 pi) mod 1 in units of 2^-64, within one of them (for |f| up to 1e12): the product with 1 / (2 pi) as a sum of
// two doubles, the fractions of its halves taken exactly.  A position of 31 bits then turns by an angle that is off by
// at most 2^-33 turns, 8e-10 (with the quotient as one double: by 5e-7).
inline uint64_t turn_of(double f) {
    constexpr double kInvTwoPi = 0x1.45f306dc9c883p-3, kInvTwoPiRest = -0x1.6b01ec5417056p-57;
    const double hi = f * kInvTwoPi, lo = std::fma(f, kInvTwoPi, -hi) + f * kInvTwoPiRest;
    auto units = [](double t) {
        t -= std::rint(t);  // exact, in [-1/2, 1/2] (std::remainder, the same, takes a microsecond for 64 pairs)
        const uint64_t u = uint64_t(std::rint(std::fabs(t) * 0x1p64));
        return t < 0 ? 0 - u : u;
    };
    return units(hi) + units(lo);
}

}  // namespace kv
}  // namespace kda
