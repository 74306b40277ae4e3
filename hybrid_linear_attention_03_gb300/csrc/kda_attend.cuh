// kda_attend.cuh -- what the attention kernels share: how the keys of a call
// are shared out over the CTAs, the records of the shares and their layout in
// the workspace.
//
// An item is one row tile: the query heads of one cache head (the group, G of
// them) for TT consecutive tokens of one sequence, rows r = t * G + g.  Its
// keys are positions [0, ctx + last token + 1).  All items of a call, ordered
// by sequence, cache head and tile, form one line; an item is as long on it as
// it has keys, plus a constant: where there are more items than CTAs that of its
// start and output (in keys that take as long), else the shortest piece that a CTA
// is given, so that short items get a CTA each.  CTA c of C takes the c-th of C equal pieces of that line (a cut point
// inside an item rounded down to whole key steps).  So any
// mix of lengths loads every CTA alike, with no table built on the host and
// no launch per sequence.  An item cut by one or more cut points is computed
// in parts: every part leaves its unnormalised output, row maxima and row sums
// in the workspace, and the combine kernel joins them in order, so results do
// not depend on timing.
#pragma once

#include <mutex>

#include "kda_kv.cuh"

namespace kda {
namespace kv {

constexpr float kLog2e = 1.4426950408889634f;

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

struct alignas(16) Part {
    int32_t state;          // 0 none, 1 there, 2 there and the item's last
    int32_t row, rows, h;  // item: its first token's row, its rows, its cache head
};

struct AttendParams {
    BatchView b;
    const void *q;
    void *out;
    long long q_stride, out_stride;
    const void *pk, *pv;
    const uint8_t *sk, *sv;
    int32_t hq, hkv, group, dim;
    int32_t tile_tokens;  // TT
    int32_t key_step;     // keys per step; cut points are multiples of it
    int32_t item_cost;    // what an item costs beside its keys, key_step or more
    int32_t min_keys;     // a CTA's piece is at least this long, key_step or more (fewer CTAs take part in a small call)
    float scale_log2;     // scale * log2(e)
    Part *parts;          // [C][2]: the CTA's first part (of an item begun before) and its last
    float *part_data;     // [C][2][BM * (D + 2)]: out [BM][D], then row maxima [BM], then row sums [BM]
    uint32_t group_inv;   // ceil(2^16 / group)
    // r / group, exact for the rows of a tile: r < 256 and group <= 64 leave the error below 1 / group
    __device__ __forceinline__ int token_of(int r) const { return int(uint32_t(r) * group_inv >> 16); }
};

// Keys of tile i's last row: how far the item reaches.
__device__ __forceinline__ int tile_keys(int ctx, int T, int tt, int i) { return ctx + min(T, (i + 1) * tt); }

// Length on the line of the first m tiles of a sequence (m <= ceil(T / tt)),
// an item costing `cost` beside its keys.
__device__ __forceinline__ long long tile_prefix(int ctx, int T, int tt, int m, int cost) {
    const int full = min(m, T / tt);
    long long s = static_cast<long long>(full) * ctx + static_cast<long long>(tt) * full * (full + 1) / 2;
    if (m > full) s += ctx + T;
    return s + static_cast<long long>(cost) * m;
}

// a / b for a >= 0 and b > 0: most lines are shorter than 2^32.
__device__ __forceinline__ long long div_pos(long long a, long long b) {
    if ((a | b) >> 32 == 0) return static_cast<long long>(uint32_t(a) / uint32_t(b));
    return a / b;
}

struct Cursor {  // a place on the line: key `key` of item (n, h, tile)
    int n, h, tile, key;
};

// The whole warp finds this CTA's piece [from, to) of the line; false if it
// has none.  Lane i sums the sequences [i * per, (i + 1) * per), so the tables
// are read twice: once for the sums, once inside the piece's sequence.
// (P: the parameters of a kernel whose items are of this kind, with a batch view that load_seq reads.)
template <typename P>
__device__ __forceinline__ bool find_piece(const P &p, int cta, int n_cta, int lane, Cursor &from,
                                           Cursor &to) {
    const int N = p.b.n_seqs, per = (N + 31) / 32, tt = p.tile_tokens;
    const int n0 = min(lane * per, N), n1 = min(n0 + per, N);
    long long keys = 0, items = 0;  // of this lane's sequences, then of all lanes up to this one
    for (int n = n0; n < n1; ++n) {
        Seq s;
        if (load_seq(p.b, n, s, cta == 0) && s.T > 0) {
            const int tiles = (s.T + tt - 1) / tt;
            keys += tile_prefix(s.L - s.T, s.T, tt, tiles, 0) * p.hkv;
            items += static_cast<long long>(tiles) * p.hkv;
        }
    }
    const long long my_keys = keys, my_items = items;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long k = __shfl_up_sync(0xffffffffu, keys, o), i = __shfl_up_sync(0xffffffffu, items, o);
        if (lane >= o) keys += k, items += i;
    }
    const long long all_items = __shfl_sync(0xffffffffu, items, 31);
    const int cost = all_items > n_cta ? p.item_cost : p.min_keys;
    const long long sum = my_keys + cost * my_items, before = keys + cost * items - sum;
    const long long total = __shfl_sync(0xffffffffu, before + sum, 31);
    if (total == 0) return false;
    // A piece is never shorter than a key step: two cuts in one step would leave a CTA with nothing in the
    // middle of an item, whose parts are those of consecutive CTAs.
    const int active = int(min(static_cast<long long>(n_cta), max(div_pos(total, p.min_keys), 1LL)));
    if (cta >= active) return false;
    const long long share = div_pos(total, active);
    const int over = int(total - share * active);
    Cursor c[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const long long x = share * (cta + e) + over * (cta + e) / active;
        c[e] = Cursor{N, 0, 0, 0};
        if (x < total) {  // the lane whose sequences hold x walks them
            const unsigned owner = __ballot_sync(0xffffffffu, x >= before && x < before + sum);
            const int src = __ffs(owner) - 1;
            if (lane == src) {
                long long rest = x - before;
                for (int n = n0; n < n1; ++n) {
                    Seq s;
                    if (!load_seq(p.b, n, s, false) || s.T == 0) continue;
                    const int ctx = s.L - s.T, tiles = (s.T + tt - 1) / tt;
                    const long long head = tile_prefix(ctx, s.T, tt, tiles, cost);
                    if (rest >= head * p.hkv) {
                        rest -= head * p.hkv;
                        continue;
                    }
                    c[e].n = n;
                    c[e].h = int(div_pos(rest, head));
                    rest -= head * c[e].h;
                    int lo = 0, hi = tiles - 1;  // last tile whose prefix is at most rest
                    while (lo < hi) {
                        const int mid = (lo + hi + 1) / 2;
                        if (tile_prefix(ctx, s.T, tt, mid, cost) <= rest) lo = mid;
                        else hi = mid - 1;
                    }
                    c[e].tile = lo;
                    const int key = max(int(rest - tile_prefix(ctx, s.T, tt, lo, cost)) - cost, 0);
                    c[e].key = key / p.key_step * p.key_step;
                    break;
                }
            }
            c[e].n = __shfl_sync(0xffffffffu, c[e].n, src);
            c[e].h = __shfl_sync(0xffffffffu, c[e].h, src);
            c[e].tile = __shfl_sync(0xffffffffu, c[e].tile, src);
            c[e].key = __shfl_sync(0xffffffffu, c[e].key, src);
        }
    }
    from = c[0];
    to = c[1];
    return true;
}

// One item's share of a CTA's piece.
struct Item {
    int n, h, tile;
    int k0, k1, keys;  // this CTA's keys [k0, k1) of the item's [0, keys)
    int row0;          // row of the sequence's first token
    int ctx;           // position of that token
    int tok0, rows;    // the tile's first token and its rows
    __device__ __forceinline__ bool whole() const { return k0 == 0 && k1 == keys; }
    // where a part goes: the CTA's first part slot, or its last one for a part that begins its item
    __device__ __forceinline__ int slot() const { return k0 == 0 ? 1 : 0; }
    __device__ __forceinline__ Part part() const { return Part{k1 == keys ? 2 : 1, row0 + tok0, rows, h}; }
    // element offset of row r's channels in a row tensor
    __device__ __forceinline__ size_t at(int r, const AttendParams &p, long long stride, int D) const {
        const int t = p.token_of(r);
        return size_t(row0 + tok0 + t) * size_t(stride) + size_t(h * p.group + r - t * p.group) * size_t(D);
    }
};

// Walks a piece item by item; every role of a kernel runs its own copy.
struct ItemWalk {
    Cursor at, end;
    Seq sq;
    int tiles = -1;  // of sequence at.n; -1: not read yet
    __device__ __forceinline__ ItemWalk(const Cursor &a, const Cursor &z) : at(a), end(z) {}
    template <typename P> __device__ __forceinline__ bool next(const P &p, Item &it) {
        while (at.n < p.b.n_seqs && at.n <= end.n) {
            if (tiles < 0) tiles = load_seq(p.b, at.n, sq, false) ? (sq.T + p.tile_tokens - 1) / p.tile_tokens : 0;
            if (tiles == 0 || at.h >= p.hkv) {
                at = Cursor{at.n + 1, 0, 0, 0};
                tiles = -1;
                continue;
            }
            if (at.tile >= tiles) {
                at = Cursor{at.n, at.h + 1, 0, 0};
                continue;
            }
            const bool last = at.n == end.n && at.h == end.h && at.tile == end.tile;
            it.n = at.n, it.h = at.h, it.tile = at.tile;
            it.row0 = sq.row0, it.ctx = sq.L - sq.T;
            it.tok0 = at.tile * p.tile_tokens;
            it.rows = min(p.tile_tokens, sq.T - it.tok0) * p.group;
            it.keys = tile_keys(it.ctx, sq.T, p.tile_tokens, at.tile);
            it.k0 = at.key, it.k1 = last ? end.key : it.keys;
            if (last) at.n = p.b.n_seqs;  // done
            else ++at.tile, at.key = 0;
            if (it.k0 < it.k1) return true;
        }
        return false;
    }
};

// Workspace: the part records of every CTA, then their data, 256-aligned.
__host__ __device__ __forceinline__ size_t parts_bytes(int n_cta) {
    return (sizeof(Part) * 2 * size_t(n_cta) + 255) / 256 * 256;
}
inline size_t share_bytes(int n_cta, int bm, int D) {
    return parts_bytes(n_cta) + sizeof(float) * size_t(n_cta) * 2 * size_t(bm) * size_t(D + 2);
}

// Raises a kernel's shared memory limit, once per device.
template <auto kKernel> inline bool allow_smem(int bytes) {
    static std::once_flag once[64];
    static bool ok[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        cudaGetLastError();
        return false;
    }
    std::call_once(once[dev], [&] {
        ok[dev] = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess;
        if (!ok[dev]) cudaGetLastError();
    });
    return ok[dev];
}

// What a kernel of this family needs from the host: its row tile and its grid.
// A plan function says whether its kernel takes the call, on sizes and types alone.
struct AttendPlan {
    int bm;     // rows of a tile
    int n_cta;  // grid
};
bool few_plan(const kda_kv_cache *c, const kda_kv_batch *b, AttendPlan *plan);
kda_status few_launch(const kda_kv_cache *c, AttendParams &p, const AttendPlan &plan, cudaStream_t stream);
bool tile_plan(const kda_kv_cache *c, const kda_kv_batch *b, AttendPlan *plan);
kda_status tile_launch(const kda_kv_cache *c, AttendParams &p, const AttendPlan &plan, cudaStream_t stream);
bool lanes_plan(const kda_kv_cache *c, const kda_kv_batch *b, AttendPlan *plan);
kda_status lanes_launch(const kda_kv_cache *c, AttendParams &p, const AttendPlan &plan, cudaStream_t stream);
bool generic_plan(const kda_kv_cache *c, const kda_kv_batch *b, AttendPlan *plan);
kda_status generic_launch(const kda_kv_cache *c, AttendParams &p, const AttendPlan &plan, cudaStream_t stream);

}  // namespace kv
}  // namespace kda
