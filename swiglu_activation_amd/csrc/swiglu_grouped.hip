// Matrix products grouped by expert, for AMD MI355X (gfx950), with the C ABI
// in include/swiglu_gateup.h.
//
// What is computed: rows [ends[e-1], ends[e]) of the token matrix belong to
// expert e with its own weights W_e, and rows past ends[E-1] are spare:
//     mm      y[r]  = a[r] W_e^T                            W_e [n, k]
//     fc1     y[r]  = s_r silu(a[r] Wg_e^T) * (a[r] Wu_e^T) W_e = [Wg; Wu], [2n, k]
//     dgrad   da[r] = dy[r] W_e
//     wgrad   dW_e  = sum over e's rows of dy[r]^T a[r]
// Spare rows of y and da are set to zero, as is dW_e of an expert without rows.
// The sizes are read on the device: the host never waits for them. It launches
// enough workgroups for any split of the rows, and each finds its tile from
// the ends; those left over end at once.
//
// All four are products over one index of two operands, called here by the
// side of the output they make: F makes the output's contiguous (feature) index
// and T its row (token) index. An operand is either "row" laid (its rows run
// along the reduction: 16 bytes in memory are one lane's MFMA fragment) or
// "column" laid (its rows run along the output: fragments are read from LDS
// through the transposing read ds_read_b64_tr_b16):
//              F               T            reduced over
//     mm, fc1  W  row          a  row       k
//     dgrad    W  column       dy row       n
//     wgrad    a  column       dy column    e's rows
#include "swiglu_device.h"

namespace {

using namespace swiglu_impl;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef u32x4 u32x4_any __attribute__((aligned(2)));

enum Op { kMm, kFc1, kDgrad, kWgrad };

struct GroupedArgs {
    const uint16_t* f;       // operand F: weights, or (wgrad) the tokens a
    const uint16_t* t;       // operand T: tokens a or dy
    void* out;               // bf16, or fp32 for wgrad
    const float* scale;      // fc1: per row, or NULL
    const int32_t* ends;     // [experts]
    int64_t ldf, ldt, ldo;   // row strides (elements)
    int64_t f_stride;        // elements between experts' weights (not wgrad)
    int64_t o_stride;        // elements between experts' outputs (wgrad)
    int64_t scale_stride;
    int64_t rows;            // token rows, spare ones included
    int64_t experts;
    int64_t n_f;             // width of the output (features; wgrad: k)
    int64_t n_r;             // length of the reduction (not wgrad)
    int64_t n_t;             // wgrad: rows of one expert's output (n)
    int64_t up;              // fc1: rows from a gate row to its up row (n)
    bool large;              // wgrad: short groups, and an output larger than the caches
    bool stream;             // and it is written past them
};

__device__ __forceinline__ uint32_t lane_of(uint32_t v, int w) {
    return (uint32_t)__builtin_amdgcn_readlane((int)v, w);
}

// v from another lane of the wave, chosen by a DPP control; `none` where there is no
// such lane or its row of 16 is not in ROWS.
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ uint32_t from_lane(uint32_t none, uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)v, CTRL, ROWS, 0xf, false);
}
// The largest v of this lane and those before it (all lanes of the wave take part).
__device__ __forceinline__ uint32_t max_scan(uint32_t v) {
    auto with = [&](uint32_t o) { v = o > v ? o : v; };
    with(from_lane<0x111>(0, v));            // within rows of 16: 1, 2, 4 and 8 lanes before
    with(from_lane<0x112>(0, v));
    with(from_lane<0x114>(0, v));
    with(from_lane<0x118>(0, v));
    with(from_lane<0x142, 0xa>(0, v));       // a row's last lane to the next row (rows 1 and 3)
    with(from_lane<0x143, 0xc>(0, v));       // lane 31 to rows 2 and 3
    return v;
}

// Row range of expert e, or of the spare rows (e == P.experts). A group begins at
// the largest end before it (swiglu_host::group_end): no ends, whatever their values
// and order, lead outside the operands or make two groups share a row. The groups
// before expert `from` are known to end at row `begin`. All lanes of the wave take part.
__device__ __forceinline__ void expert_rows(const GroupedArgs& P, int64_t e, int64_t& lo, int64_t& hi,
                                            int64_t from = 0, int32_t begin = 0) {
    const int32_t rows = (int32_t)P.rows;
    if (from < e) {
        const int lane = threadIdx.x & 63;
        uint32_t m = (uint32_t)begin;
        for (int64_t b = from; b < e; b += 64) {
            const int64_t i = b + lane < e ? b + lane : e - 1;   // (the last one again)
            const uint32_t v = (uint32_t)swiglu_host::group_end(0, P.ends[i], rows);
            m = v > m ? v : m;
        }
        begin = (int32_t)lane_of(max_scan(m), 63);
    }
    lo = begin;
    hi = e == P.experts ? rows : swiglu_host::group_end(begin, P.ends[e], rows);
}

// The workgroup's place in the launch order of `total` tiles, or `total` if
// there is none for it. The hardware deals workgroups to the 8 XCDs in turn;
// each XCD is given a contiguous eighth of the order, so that the tiles which its
// own L2 serves at one time are neighbours that share operands.
constexpr uint32_t kXcds = 8;
__device__ __forceinline__ uint32_t place_of(uint32_t b, uint32_t total) {
    const uint32_t x = b % kXcds, i = b / kXcds, q = total / kXcds, r = total % kXcds;
    if (i >= q + (x < r ? 1 : 0)) return total;
    return x * q + (x < r ? x : r) + i;
}

// Order of the tiles of one expert: kGroupT row tiles of one feature tile, then
// the next feature tile. The 32 workgroups that run on an XCD then work on about
// 8 row tiles x 4 feature tiles: 12 tiles of operands for 32 of output.
constexpr uint32_t kGroupT = 8;
__device__ __forceinline__ void tile_in_expert(uint32_t in, uint32_t t_tiles, uint32_t f_tiles,
                                               uint32_t& tt, uint32_t& ft) {
    const uint32_t per_group = kGroupT * f_tiles;
    const uint32_t g = in / per_group, r = in % per_group;
    const uint32_t left = t_tiles - g * kGroupT, gs = left < kGroupT ? left : kGroupT;
    tt = g * kGroupT + r % gs;
    ft = r / gs;
}

// The row tiles of TILE rows: experts in order, each with its own rows cut in
// tiles, then (SPARE) the spare rows as one more (expert index P.experts). Every
// wave searches for itself, 64 experts at a time, one per lane.
template <int TILE, bool SPARE = true>
struct RowTiles {
    uint32_t l, h, mine, sum;            // lane's expert: rows, tiles, inclusive sum
    uint32_t total;                      // row tiles in all
    uint32_t top;                        // end of the last expert held in the lanes
    int64_t base;                        // first expert held in the lanes

    static __device__ __forceinline__ int64_t groups(const GroupedArgs& P) { return P.experts + SPARE; }
    // Experts b on, after those that the lanes hold (or from the first).
    __device__ __forceinline__ void scan(const GroupedArgs& P, int64_t b) {
        const int lane = threadIdx.x & 63;
        base = b;
        const uint32_t begin = b == 0 ? 0 : top;
        uint32_t v = 0;                                   // rows fit 31 bits
        if (b + lane < P.experts) v = (uint32_t)swiglu_host::group_end(0, P.ends[b + lane], (int32_t)P.rows);
        if (SPARE && b + lane == P.experts) v = (uint32_t)P.rows;
        v = max_scan(v);
        h = v > begin ? v : begin;
        l = from_lane<0x138>(begin, h);                   // the lane before
        top = lane_of(h, 63);
        mine = sum = (h - l + TILE - 1) / TILE;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const uint32_t o = __shfl_up(sum, d, 64);
            if (lane >= d) sum += o;
        }
    }
    __device__ __forceinline__ void init(const GroupedArgs& P) {
        scan(P, 0);
        total = lane_of(sum, 63);
        RowTiles later = *this;                           // (the first 64 stay in the lanes)
        for (int64_t b = 64; b < groups(P); b += 64) {
            later.scan(P, b);
            total += lane_of(later.sum, 63);
        }
    }
    // Tile `place` (below total * f_tiles) of the launch order.
    __device__ __forceinline__ void locate(const GroupedArgs& P, uint32_t place, uint32_t f_tiles,
                                           int64_t& expert, int64_t& lo, int64_t& hi, uint32_t& tt,
                                           uint32_t& ft) {
        const uint32_t slot = place / f_tiles;
        uint32_t before = 0;                              // tiles of earlier chunks
        expert = P.experts;
        lo = hi = 0;
        tt = ft = 0;
        for (int64_t b = 0; b < groups(P); b += 64) {
            if (b != base) scan(P, b);
            const uint64_t past = __ballot(before + sum > slot);
            if (past != 0) {
                const int w = __builtin_ctzll(past);
                const uint32_t tiles = lane_of(mine, w);
                const uint32_t first = before + lane_of(sum, w) - tiles;
                expert = b + w;
                lo = lane_of(l, w);
                hi = lane_of(h, w);
                tile_in_expert(place - first * f_tiles, tiles, f_tiles, tt, ft);
                return;
            }
            before += lane_of(sum, 63);
        }
    }
};

// The workgroup's tile, one each; false when there are fewer than workgroups.
template <int TILE>
__device__ __forceinline__ bool find_tile(const GroupedArgs& P, uint32_t f_tiles, int64_t& expert,
                                          int64_t& lo, int64_t& hi, uint32_t& tt, uint32_t& ft) {
    RowTiles<TILE> R;
    R.init(P);
    const uint32_t all = R.total * f_tiles, place = place_of(blockIdx.x, all);
    if (place == all) return false;
    R.locate(P, place, f_tiles, expert, lo, hi, tt, ft);
    return true;
}

// The same for wgrad, whose tiles do not depend on the ends.
__device__ __forceinline__ void wgrad_tile(uint32_t experts, uint32_t t_tiles, uint32_t f_tiles,
                                           int64_t& expert, uint32_t& tt, uint32_t& ft) {
    const uint32_t per = f_tiles * t_tiles, place = place_of(blockIdx.x, experts * per);
    expert = place / per;
    tile_in_expert(place % per, t_tiles, f_tiles, tt, ft);
}

// ---------------------------------------------------------------------------
// Few tiles: the reduction in parts
// ---------------------------------------------------------------------------
// When the output has fewer tiles than half of the CUs, the reduction of
// each is cut in parts, one workgroup each, that write fp32 sums to the
// workspace; a second launch adds a value's parts in order, rounds and stores.
// An output tile: rows [t0, t1) of the output, of which the first TT are made.
struct Job {
    int32_t expert, lo, t0, t1, f0;
    int32_t r0, len;         // the part of the reduction
    int32_t tt;              // 256 or 128; 0: none
};

constexpr int kRedTile = 64;                             // reduction indexes per step of the kernels
constexpr uint32_t kSplitJobs = 256;                     // workgroups, at most

// Parts of each tile's reduction of length len: as many as there are workgroups
// for, of at least 4 steps. Parts cost a second launch and their sums' way through
// memory, about as much as 12 steps of 0.85 us and, at 256 parts, 16 more
// (tiles of 128 x 256; 128 of them, k = 4096: 60 us whole, 52 in 2 parts; k = 1024: 19
// whole, 31 in 2 parts; 32 of them, k = 4096: 60 whole, 27 in 8 parts).
__host__ __device__ inline uint32_t split_parts(uint32_t tiles, int64_t len) {
    if (tiles == 0 || tiles > kSplitJobs / 2) return 1;
    const int64_t count = (len + kRedTile - 1) / kRedTile;
    int64_t s = kSplitJobs / tiles;
    if (s > count / 4) s = count / 4;
    if (s < 2) return 1;
    return count - (count + s - 1) / s >= 12 + s * tiles / 16 ? (uint32_t)s : 1;
}
// Part p of `parts`: its first reduction index and its length (0 if empty).
__device__ __forceinline__ void split_range(int32_t len, uint32_t parts, uint32_t p, int32_t& r0,
                                            int32_t& n) {
    const uint32_t tiles = ((uint32_t)len + kRedTile - 1) / kRedTile;
    const uint32_t a = (uint32_t)((uint64_t)tiles * p / parts), b = (uint32_t)((uint64_t)tiles * (p + 1) / parts);
    r0 = (int32_t)(a * kRedTile);
    const int64_t end = (int64_t)b * kRedTile < len ? (int64_t)b * kRedTile : len;
    n = end > r0 ? (int32_t)(end - r0) : 0;
}

// Tiles of TT rows x FF features (fc1: half gate, half up) in all, and the one
// at `place`.
template <Op OP, int TT, int FF>
struct SplitTiles {
    RowTiles<TT, false> R;
    uint32_t f_tiles, t_tiles, total;
    __device__ __forceinline__ void init(const GroupedArgs& P, uint32_t f) {
        f_tiles = f;
        if constexpr (OP == kWgrad) {
            t_tiles = (uint32_t)((P.n_t + TT - 1) / TT);
            total = (uint32_t)P.experts * f * t_tiles;
        } else {
            R.init(P);
            total = R.total * f;
        }
    }
    __device__ __forceinline__ Job get(const GroupedArgs& P, uint32_t place) {
        Job J{};
        int64_t expert, lo, hi;
        uint32_t tt, ft;
        if constexpr (OP == kWgrad) {
            expert = place / (f_tiles * t_tiles);
            tile_in_expert(place % (f_tiles * t_tiles), t_tiles, f_tiles, tt, ft);
            expert_rows(P, expert, lo, hi);
            J.lo = __builtin_amdgcn_readfirstlane((int32_t)lo);
            J.len = __builtin_amdgcn_readfirstlane((int32_t)(hi - lo));
            J.t0 = (int32_t)tt * TT;
            J.t1 = (int32_t)P.n_t;
        } else {
            R.locate(P, place, f_tiles, expert, lo, hi, tt, ft);
            J.lo = (int32_t)lo;
            J.len = (int32_t)P.n_r;
            J.t0 = (int32_t)lo + (int32_t)tt * TT;
            J.t1 = (int32_t)hi;
        }
        J.expert = (int32_t)expert;
        J.f0 = (int32_t)ft * (OP == kFc1 ? FF / 2 : FF);
        J.tt = TT;
        return J;
    }
};

// The first `count` of the 16 bytes' worth of elements in v, to p at any alignment.
template <typename OutT>
__device__ __forceinline__ void store_chunk(OutT* p, int64_t count, u32x4 v) {
    constexpr int kPer = 16 / (int)sizeof(OutT);
    if (count >= kPer) {
        *reinterpret_cast<u32x4_any*>(p) = v;
        return;
    }
    OutT e[kPer];
    __builtin_memcpy(e, &v, sizeof(v));
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        if (i < count) p[i] = e[i];
}

// Adds the parts: a thread makes 8 features of one row, a workgroup 2048 values of
// a tile.
constexpr int kJoinThreads = 256;
template <int TT, int FF> constexpr int kJoinGroups = TT * FF / 8 / kJoinThreads;
template <Op OP, typename OutT, int TT, int FF>
__global__ __launch_bounds__(kJoinThreads) void grouped_join_kernel(GroupedArgs P, uint32_t f_tiles,
                                                                    int64_t len, const float* ws) {
    constexpr int kPer = kJoinGroups<TT, FF>, kLanes = FF / 8;       // threads per row
    SplitTiles<OP, TT, FF> T;
    T.init(P, f_tiles);
    const uint32_t parts = split_parts(T.total, len), tile = blockIdx.x / kPer;
    if (parts == 1 || tile >= T.total) return;
    const Job J = T.get(P, tile);
    const int r = (int)(blockIdx.x % kPer) * (kJoinThreads / kLanes) + threadIdx.x / kLanes;
    const int c = threadIdx.x % kLanes * 8;
    const int32_t feats = (int32_t)P.n_f - J.f0;
    if (r >= J.t1 - J.t0 || c >= feats || (OP == kFc1 && c >= FF / 2)) return;
    const float* p = ws + (size_t)tile * parts * (TT * FF) + r * FF + c;
    float o[8] = {}, u[8] = {};
#pragma unroll 4
    for (uint32_t q = 0; q < parts; ++q, p += TT * FF) {
        if constexpr (OP == kWgrad) {
            int32_t r0, n;
            split_range(J.len, parts, q, r0, n);
            if (n == 0) continue;
        }
        auto add = [](const float* x, float (&v)[8]) {
            const u32x4 a = *reinterpret_cast<const u32x4*>(x), b = *reinterpret_cast<const u32x4*>(x + 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[e] += __uint_as_float(a[e]);
                v[4 + e] += __uint_as_float(b[e]);
            }
        };
        add(p, o);
        if constexpr (OP == kFc1) add(p + FF / 2, u);
    }
    if constexpr (OP == kFc1) {
        const float s = P.scale != nullptr ? P.scale[(int64_t)(J.t0 + r) * P.scale_stride] : 1.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float sig, osig, scl;
            sigmoid_pair<uint16_t, false>(o[e], sig, osig, scl);
            o[e] = s * ((o[e] * sig) * u[e]);
        }
    }
    OutT* out = static_cast<OutT*>(P.out) + (OP == kWgrad ? J.expert * P.o_stride : 0) +
                (int64_t)(J.t0 + r) * P.ldo + J.f0 + c;
    if constexpr (sizeof(OutT) == 4) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (c + 4 * h < feats)
                store_chunk(out + 4 * h, feats - c - 4 * h,
                            u32x4{__float_as_uint(o[4 * h]), __float_as_uint(o[4 * h + 1]),
                                  __float_as_uint(o[4 * h + 2]), __float_as_uint(o[4 * h + 3])});
    } else {
        uint32_t q[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            f32x2 pr = {o[2 * e], o[2 * e + 1]};
            q[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(pr, bf16x2));
        }
        store_chunk(out, feats - c, u32x4{q[0], q[1], q[2], q[3]});
    }
}

// ---------------------------------------------------------------------------
// General kernel: 128 x 128 tiles, any sizes and alignment
// ---------------------------------------------------------------------------
// 4 waves, each 64 x 64 (2 x 2 MFMA tiles of 32 x 32 x 16). The reduction is
// walked 64 at a time: the next tile's chunks are loaded to registers while the
// current one is multiplied, and go to LDS once every wave has read it. A
// chunk is 8 elements: rows that are not 16-byte aligned are loaded as
// unaligned vectors, and of a chunk that sticks out only what belongs to the row, with
// zeros after it, so that nothing outside the operands is read and no
// value of another row meets a product.
constexpr int kGenTile = 128, kGenK = 64, kGenThreads = 256;
constexpr int kGenChunks = kGenTile * kGenK / 8 / kGenThreads;      // per operand and thread: 4

// The first `count` elements at p, zeros after them. back: the 8 elements before
// p + count are the row's too; a chunk that sticks out is then those, shifted.
// (Lanes without any take neither branch; one element after the other costs a wave 8 loads in
// a row: dgrad, 664 rows, E = 26, n = 1699, k = 193: 54 us, and 49.)
__device__ __forceinline__ u32x4 load_chunk(const uint16_t* p, int32_t count, bool back) {
    u32x4 v = {};
    if (count >= 8) {
        v = *reinterpret_cast<const u32x4_any*>(p);
    } else if (count > 0) {
        if (back) {
            const u32x4 w = *reinterpret_cast<const u32x4_any*>(p - (8 - count));
            const int s = 16 * (8 - count);
            const uint64_t lo = (uint64_t)w[1] << 32 | w[0], hi = (uint64_t)w[3] << 32 | w[2];
            const uint64_t a = s >= 64 ? hi >> (s - 64) : lo >> s | hi << (64 - s), c = s >= 64 ? 0 : hi >> s;
            v = u32x4{(uint32_t)a, (uint32_t)(a >> 32), (uint32_t)c, (uint32_t)(c >> 32)};
        } else {
            uint16_t e[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) e[i] = i < count ? p[i] : (uint16_t)0;
            __builtin_memcpy(&v, e, sizeof(v));
        }
    }
    return v;
}

// 16-byte chunk c of LDS row r is kept in slot c ^ swizzle(r), so that the
// lanes that read together meet different banks. Row laid tiles: rows of 8
// chunks, a lane per row. Column laid tiles: rows of 16 chunks; a transposing
// read takes 4 rows x 64 bytes per 32 lanes, and the other 32 lanes the rows
// 8 below.
__device__ __forceinline__ int row_slot(int r, int c) { return c ^ ((r >> 1) & 7); }
__device__ __forceinline__ int col_slot(int r, int c) {
    return c ^ (((r & 3) << 2) | (((r >> 3) & 1) << 1));
}

template <bool COL>
__device__ __forceinline__ bf16x8 gen_frag(const uint16_t* lds, int out0, int step) {
    const int lane = threadIdx.x & 63;
    if constexpr (!COL) {
        const int r = out0 + lane % 32, c = 2 * step + lane / 32;
        return __builtin_bit_cast(bf16x8,
                                  *reinterpret_cast<const u32x4*>(lds + r * kGenK + row_slot(r, c) * 8));
    } else {
        const int r = 16 * step + 8 * (lane / 32) + (lane % 16) / 4;
        const int col = out0 + 16 * ((lane / 16) & 1) + 4 * (lane % 4);
        const int off = col_slot(r, col / 8) * 8 + col % 8;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds_s16x4*)(lds + r * kGenTile + off));
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds_s16x4*)(lds + (r + 4) * kGenTile + off));     // col_slot(r + 4) = col_slot(r)
        const __attribute__((ext_vector_type(8))) short v =
            __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        return __builtin_bit_cast(bf16x8, v);
    }
}

// One operand's tile: 128 of the output's index by 64 of the reduction.
template <bool COL>
struct GenSource {
    const uint16_t* p[kGenChunks];   // each chunk at reduction index 0
    int32_t count[kGenChunks];       // row laid: 1 if the row exists; column laid: columns left
    int64_t ld;
    bool back;                       // every row has 8 elements

    // all: elements of a row.
    template <typename RowPtr>
    __device__ __forceinline__ void init(RowPtr row_ptr, int64_t stride, int32_t width, int64_t all) {
        ld = stride;
        back = all >= 8;
#pragma unroll
        for (int i = 0; i < kGenChunks; ++i) {
            const int id = i * kGenThreads + threadIdx.x;
            if constexpr (!COL) {
                const int r = id / 8;
                bool valid;
                p[i] = row_ptr(r, valid) + (id % 8) * 8;
                count[i] = valid;
            } else {
                const int c = (id % 16) * 8;
                bool valid;
                p[i] = row_ptr(0, valid) + (int64_t)(id / 16) * ld + c;
                count[i] = width - c;
            }
        }
    }
    __device__ __forceinline__ void load(int32_t r0, int32_t len, u32x4 (&v)[kGenChunks]) const {
#pragma unroll
        for (int i = 0; i < kGenChunks; ++i) {
            const int id = i * kGenThreads + threadIdx.x;
            if constexpr (!COL)
                v[i] = load_chunk(p[i] + r0, count[i] ? len - r0 - (id % 8) * 8 : 0, back);
            else
                v[i] = load_chunk(p[i] + r0 * ld, r0 + id / 16 < len ? count[i] : 0, back);
        }
    }
    __device__ __forceinline__ void store(uint16_t* lds, const u32x4 (&v)[kGenChunks]) const {
#pragma unroll
        for (int i = 0; i < kGenChunks; ++i) {
            const int id = i * kGenThreads + threadIdx.x;
            uint16_t* d = COL ? lds + (id / 16) * kGenTile + col_slot(id / 16, id % 16) * 8
                              : lds + (id / 8) * kGenK + row_slot(id / 8, id % 8) * 8;
            *reinterpret_cast<u32x4*>(d) = v[i];
        }
    }
};

// SPLIT: a workgroup makes one part of a tile's reduction (plan: the length that
// parts are planned for) and writes its sums to ws.
template <Op OP, typename OutT, bool SPLIT>
__global__ __launch_bounds__(kGenThreads, 3) void grouped_general_kernel(GroupedArgs P, uint32_t f_tiles,
                                                                         int64_t plan, float* ws) {
    constexpr bool F_COL = OP == kDgrad || OP == kWgrad, T_COL = OP == kWgrad;
    constexpr int kTileF = OP == kFc1 ? kGenTile / 2 : kGenTile;     // output features per tile
    __shared__ __attribute__((aligned(16))) uint16_t lds[2 * kGenTile * kGenK];
    uint16_t *lds_f = lds, *lds_t = lds + kGenTile * kGenK;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;

    // The tile: output rows [t0, t1) and features [f0, ...), reduction [r0, r0 + len).
    int64_t expert, lo, hi, t0, t1;
    int32_t f0, r0 = 0, len;
    if constexpr (SPLIT) {
        SplitTiles<OP, kGenTile, kGenTile> T;
        T.init(P, f_tiles);
        const uint32_t parts = split_parts(T.total, plan);
        const uint32_t all = T.total * parts, place = place_of(blockIdx.x, all);
        // the spare rows' zeros, by workgroups in turn
        if constexpr (OP != kWgrad) {
            expert_rows(P, P.experts, lo, hi);
            for (int64_t r = lo + blockIdx.x; r < hi; r += gridDim.x)
                for (int64_t f = threadIdx.x; f < P.n_f; f += kGenThreads)
                    static_cast<OutT*>(P.out)[r * P.ldo + f] = OutT(0);
        }
        if (place == all) return;
        const uint32_t part = place / T.total, tile = place % T.total;
        const Job J = T.get(P, tile);
        split_range(J.len, parts, part, r0, len);
        if (len == 0 && parts > 1) return;               // (the sum skips such parts)
        expert = J.expert;
        lo = J.lo;
        t0 = J.t0;
        t1 = J.t1;
        f0 = J.f0;
        ws = parts > 1 ? ws + ((size_t)tile * parts + part) * (kGenTile * kGenTile) : nullptr;
    } else {
        uint32_t tt, ft;
        if constexpr (OP == kWgrad) {
            wgrad_tile((uint32_t)P.experts, (uint32_t)((P.n_t + kGenTile - 1) / kGenTile), f_tiles,
                       expert, tt, ft);
            expert_rows(P, expert, lo, hi);
            t0 = (int64_t)tt * kGenTile;
            t1 = P.n_t;
            len = (int32_t)(hi - lo);
        } else {
            if (!find_tile<kGenTile>(P, f_tiles, expert, lo, hi, tt, ft)) return;
            t0 = lo + (int64_t)tt * kGenTile;
            t1 = hi;
            len = expert == P.experts ? 0 : (int32_t)P.n_r;          // spare rows: zero
        }
        f0 = (int32_t)ft * kTileF;
    }

    f32x16 acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = f32x16{};
    const int wf = (wave % 2) * (OP == kFc1 ? 32 : 64), wt = (wave / 2) * 64;

    if (len > 0) {
        GenSource<F_COL> sf;
        GenSource<T_COL> st;
        if constexpr (OP == kWgrad) {
            sf.init([&](int, bool&) { return P.f + (lo + r0) * P.ldf + f0; }, P.ldf, (int32_t)P.n_f - f0, P.n_f);
            st.init([&](int, bool&) { return P.t + (lo + r0) * P.ldt + t0; }, P.ldt, (int32_t)(t1 - t0), P.n_t);
        } else {
            const uint16_t* w = P.f + expert * P.f_stride;
            if constexpr (OP == kDgrad)
                sf.init([&](int, bool&) { return w + r0 * P.ldf + f0; }, P.ldf, (int32_t)P.n_f - f0, P.n_f);
            else
                // fc1: 64 gate rows, then the 64 up rows of the same features
                sf.init([&](int r, bool& v) {
                    const int64_t row = f0 + (OP == kFc1 ? r % kTileF : r);
                    v = row < P.n_f;
                    return w + (v ? row + (OP == kFc1 && r >= kTileF ? P.up : 0) : 0) * P.ldf + r0;
                }, P.ldf, 0, r0 + len);
            st.init([&](int r, bool& v) {
                v = t0 + r < t1;
                return P.t + (v ? t0 + r : t0) * P.ldt + r0;
            }, P.ldt, 0, r0 + len);
        }
        u32x4 vf[kGenChunks], vt[kGenChunks];
        sf.load(0, len, vf);
        st.load(0, len, vt);
        for (int32_t r = 0;; r += kGenK) {
            sf.store(lds_f, vf);
            st.store(lds_t, vt);
            __syncthreads();
            const bool more = swiglu_host::more_steps(r, len, kGenK);
            if (more) {
                sf.load(r + kGenK, len, vf);
                st.load(r + kGenK, len, vt);
            }
#pragma unroll
            for (int s = 0; s < kGenK / 16; ++s) {
                bf16x8 ff[2], ft[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    ff[i] = gen_frag<F_COL>(lds_f, wf + (OP == kFc1 ? 64 : 32) * i, s);
                    ft[i] = gen_frag<T_COL>(lds_t, wt + 32 * i, s);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(ff[i], ft[j], acc[i][j], 0, 0, 0);
            }
            __syncthreads();
            if (!more) break;
        }
    }

    if constexpr (SPLIT) {
        if (ws != nullptr) {
            // fc1: gate features in columns 0 to 63, up features from 64
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int row = wt + 32 * j + lane % 32;
                        const int c = wf + (OP == kFc1 ? 64 : 32) * i + 8 * q + 4 * (lane / 32);
                        if (t0 + row < t1)
                            *reinterpret_cast<u32x4*>(ws + row * kGenTile + c) =
                                u32x4{__float_as_uint(acc[i][j][4 * q]), __float_as_uint(acc[i][j][4 * q + 1]),
                                      __float_as_uint(acc[i][j][4 * q + 2]), __float_as_uint(acc[i][j][4 * q + 3])};
                    }
            return;
        }
    }

    // Register e of a 32 x 32 tile holds feature (e % 4) + 8 (e / 4) +
    // 4 (lane / 32) and token lane % 32. Through the wave's own quarter of LDS, 32 rows of 128 bytes
    // at a time, so that every store writes whole rows of 128 bytes (fc1: 64).
    constexpr int kSize = (int)sizeof(OutT);
    constexpr int NI = OP == kFc1 ? 1 : 4 / kSize;       // feature tiles of 32 in 128 bytes
    constexpr int kRowBytes = NI * 32 * kSize, kPitch = 128 + 16;
    constexpr int kPerRow = kRowBytes / 16;              // lanes per row, 16 bytes each
    char* region = reinterpret_cast<char*>(lds) + wave * (2 * kGenTile * kGenK * 2 / 4);
    OutT* out = static_cast<OutT*>(P.out) + (OP == kWgrad ? expert * P.o_stride : 0);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int64_t row0 = t0 + wt + 32 * j;
        float s = 1.0f;
        if constexpr (OP == kFc1)
            if (P.scale != nullptr && len > 0 && row0 + lane % 32 < t1)
                s = P.scale[(row0 + lane % 32) * P.scale_stride];
#pragma unroll
        for (int i0 = 0; i0 < (OP == kFc1 ? 1 : 2); i0 += NI) {
#pragma unroll
            for (int i = i0; i < i0 + NI; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float v[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        v[r] = acc[i][j][4 * q + r];
                        if constexpr (OP == kFc1) {
                            float sig, osig, scl;
                            sigmoid_pair<uint16_t, false>(v[r], sig, osig, scl);
                            v[r] = len > 0 ? s * ((v[r] * sig) * acc[1][j][4 * q + r]) : 0.0f;
                        }
                    }
                    char* p = region + (lane % 32) * kPitch + (32 * (i - i0) + 8 * q + 4 * (lane / 32)) * kSize;
                    if constexpr (kSize == 4) {
                        *reinterpret_cast<u32x4*>(p) = u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]),
                                                             __float_as_uint(v[2]), __float_as_uint(v[3])};
                    } else {
                        uint32_t w[2];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            f32x2 pr = {v[2 * h], v[2 * h + 1]};
                            w[h] = __builtin_bit_cast(uint32_t, __builtin_convertvector(pr, bf16x2));
                        }
                        *reinterpret_cast<u32x2*>(p) = u32x2{w[0], w[1]};
                    }
                }
            const int c = lane % kPerRow;
            const int64_t f = f0 + wf + 32 * i0 + c * (16 / kSize);
#pragma unroll
            for (int it = 0; it < 32 * kPerRow / 64; ++it) {
                const int row = it * (64 / kPerRow) + lane / kPerRow;
                const u32x4 v = *reinterpret_cast<const u32x4*>(region + row * kPitch + c * 16);
                if (row0 + row < t1 && f < P.n_f)
                    store_chunk(out + (row0 + row) * P.ldo + f, P.n_f - f, v);
            }
        }
    }
}

}  // namespace

#include "swiglu_grouped_tile.h"
#include "swiglu_grouped_direct.h"

namespace {

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

constexpr int64_t kMaxTiles = (int64_t)1 << 24;          // output tiles of a launch

template <Op OP, typename OutT>
swiglu_status launch_tile(const GroupedArgs& P, hipStream_t stream) {
    constexpr int kTileF = OP == kFc1 ? 128 : 256;
    const int64_t f_tiles = (P.n_f + kTileF - 1) / kTileF;
    const int64_t slots = OP == kWgrad ? P.experts * ((P.n_t + 255) / 256)
                                       : swiglu_host::grouped_row_tiles(P.rows, P.experts, 128);
    if (slots > kMaxTiles / f_tiles) return SWIGLU_ERR_BAD_SHAPE;
    int dev = 0, cus = 0;
    if (hipGetDevice(&dev) != hipSuccess ||
        hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
        return SWIGLU_ERR_HIP;
    int64_t grid = cus / (int)kXcds * (int)kXcds;        // one workgroup fills a CU's LDS
    // An XCD's eighth of the tiles, all of them cut in halves, and one more (300 rows, E = 2, n = 512,
    // k = 4096: 41 us, and 77 with as many workgroups as tiles, whose halves then share one).
    const int64_t eighth = (slots * f_tiles + kXcds - 1) / kXcds;
    const int64_t most = OP == kWgrad ? eighth * kXcds : (2 * eighth + 1) * kXcds;
    grid = grid < kXcds ? kXcds : grid > most ? most : grid;
    uint32_t ft = (uint32_t)f_tiles;
    GroupedArgs Q = P;
    void* args[] = {&Q, &ft};
    if (hipLaunchKernel(reinterpret_cast<const void*>(&grouped_tile::grouped_tile_kernel<OP, OutT>),
                        dim3((uint32_t)grid), dim3(grouped_tile::kThreads), args, 0, stream) !=
        hipSuccess)
        return SWIGLU_ERR_HIP;
    return SWIGLU_OK;
}

// Rows of whole aligned 16-byte vectors, strides within the tile kernel's offsets.
bool whole_vectors(const void* p, int64_t ld, int64_t between, int64_t width, int64_t esz) {
    const int64_t v = 16 / esz;
    return (uintptr_t)p % 16 == 0 && ld % v == 0 && between % v == 0 && width % v == 0 &&
           ld <= grouped_tile::kMaxLd;
}

// (dgrad: whole vectors only)
template <Op OP, bool ANY>
swiglu_status launch_direct(const GroupedArgs& P, hipStream_t stream) {
    namespace gd = grouped_direct;
    static_assert(OP != kWgrad && !(OP == kDgrad && ANY), "what the direct kernels make");
    constexpr int kTileF = OP == kDgrad ? gd::kDF : gd::kF;
    const int64_t f_tiles = (P.n_f + kTileF - 1) / kTileF;
    const int64_t slots = swiglu_host::grouped_row_tiles(P.rows, P.experts, gd::kRows);
    uint32_t ft = (uint32_t)f_tiles;
    GroupedArgs Q = P;
    void* args[] = {&Q, &ft};
    const void* k;
    if constexpr (OP == kDgrad) k = reinterpret_cast<const void*>(&gd::grouped_direct_dgrad_kernel);
    else k = reinterpret_cast<const void*>(&gd::grouped_direct_kernel<OP, ANY>);
    if (hipLaunchKernel(k, dim3((uint32_t)(slots * f_tiles)), dim3(gd::kThreads), args, 0, stream) !=
        hipSuccess)
        return SWIGLU_ERR_HIP;
    return SWIGLU_OK;
}

// The split kernels' tiles: 128 x 256 (wgrad: 256 x 256), or 128 x 128 by the general one.
struct SplitShape {
    int rows, feats;
};
SplitShape split_shape(Op op, bool whole) {
    return {whole && op == kWgrad ? 256 : 128, whole ? 256 : 128};
}
// How many there are for any split of the rows (the spare rows are no tiles of theirs).
int64_t split_tiles(Op op, bool whole, int64_t rows, int64_t experts, int64_t n_f, int64_t n_t) {
    const SplitShape S = split_shape(op, whole);
    const int64_t tile_f = op == kFc1 ? S.feats / 2 : S.feats;
    const int64_t slots = op == kWgrad ? experts * ((n_t + S.rows - 1) / S.rows)
                                       : swiglu_host::grouped_row_tiles(rows, experts - 1, S.rows);
    return slots * ((n_f + tile_f - 1) / tile_f);
}

// Reduction length that the parts are planned for: wgrad's are the groups'
// sizes, of which the host knows the mean.
int64_t split_len(Op op, int64_t rows, int64_t experts, int64_t n_r) {
    return op == kWgrad ? (rows + experts - 1) / experts : n_r;
}

// Which kernel makes a product. The rows' split over the experts is on the
// device, so this goes by the sizes that the host has.
enum Path { kDirectPath, kSplitPath, kTilePath, kGeneralPath };

// Estimates in us, of which the smallest is taken. They were fitted to (and the
// comments give) the times of kernels that follow one another: direct, general, tiles. They
// are to rank the kernels, and are off by up to 1.6 times in places (fc1, 1014 rows, E = 24, n = 176,
// k = 2056: 23.5 for the direct kernel's 15; dgrad, 64 rows, E = 64, n = 1792, k = 4096: 291 for 188).
struct Estimate {
    double direct, general, tiles, split;
};
Estimate estimate(Op op, int64_t rows, int64_t experts, int64_t n_f, int64_t n_r) {
    const int64_t halves = op == kFc1 ? 2 : 1;
    const int64_t groups = rows < experts ? rows : experts;          // with rows, at most
    auto tiles = [&](int64_t t, int64_t f) {
        return (double)((groups + (rows - groups) / t) * ((n_f * halves + f - 1) / f));
    };
    const double steps = (double)((n_r + kRedTile - 1) / kRedTile);
    const double weights = (double)groups * (double)(n_f * halves) * (double)n_r * 2;
    const int64_t share = (rows + groups - 1) / groups;              // rows of a group; some have twice as many
    // Direct: what a workgroup reads, its features and its rows, at 45 bytes a ns and CU, and 1 us for each
    // workgroup of a CU but the first; or all weights at 6.2 TB/s.
    // fc1, 1014 rows, E = 24, n = 176, k = 2056: 15, 38, 31; 256, E = 64, n = 1792, k = 4096: 290, 362, 338;
    // 116, E = 60, n = 2568, k = 416: 58, 45, 46. mm, 1000 rows, E = 8, n = 512, k = 1024: 18, 20, 15;
    // 128, E = 8, n = 4096, k = 1792: 47, 32, 24; 64, E = 8, n = k = 4096: 72, 69, 48; 1602, E = 4,
    // n = 1176, k = 512: 32, 13, 12.
    const int64_t feats = op == kDgrad ? 32 : 16 * halves;
    const double per_cu = tiles(32, feats) / 256, turns = per_cu < 4 ? (double)(int)(per_cu + 0.999) : per_cu;
    const double reads = turns * (double)(feats + (share < 16 ? 2 * share : 32)) * (double)n_r * 2 / 45e3;
    // dgrad's workgroups fill a CU's LDS: 6.5 us more for each but the first (1 row, E = 2, n = 3816,
    // k = 1816: 8.6, 71, 41, and 14 split; 6, E = 6, n = 416, k = 3272: 17, 12, 11; 64, E = 64, n = 1792,
    // k = 4096: 188, 113, 103).
    const double own = reads + (turns - 1) * (op == kDgrad ? 6.5 : 1), all = weights / 6.2e6;
    const double direct = (op == kDgrad ? 3 : 4) + (own > all ? own : all);
    // General: 1.05 us a step in one round of 3 workgroups per CU. It starts and ends
    // faster than the tiles: dgrad, 2000 rows, E = 2, n = k = 256: 8.4 and 9.5; 546, E = 48,
    // n = 168, k = 216: 7.7 and 8.9; 6 rows, E = 6, n = 416, k = 3272 (7 steps): 12 and 11.
    const double general = steps <= 6 && tiles(128, 128) <= 768 ? 5 + 1.05 * steps : 1e30;
    // Tiles of 128 x 256: 0.55 us a step on half of the CUs, 0.65 of few rows, 0.85 of many, or all
    // weights at 5.6 TB/s; split, the parts' sums take their way through memory and a second launch
    // (mm, 256 rows, E = 1, n = 4096, k = 8192: 171 direct, 32 split, 72 whole).
    const double t = tiles(128, 256), parts = t <= kSplitJobs / 2 ? split_parts((uint32_t)t, n_r) : 1;
    const double step = t <= 128 ? 0.55 : share < 64 ? 0.65 : 0.85;
    const double read = weights / 5.6e6;
    const double busy = (t > 256 ? t / 256 : 1) * step * steps + t / 256 * 2;
    const double part = step * ((steps + parts - 1) / parts);
    const double whole = 6.5 + busy > 4 + read ? 6.5 + busy : 4 + read;
    const double split = parts > 1 ? 11 + 0.03 * parts * t + (part > read ? part : read) : 1e30;
    return {direct, general, whole, split};
}

// Whether the direct kernel's grid is one launch (fewer than 2^32 threads).
bool direct_fits(Op op, int64_t rows, int64_t experts, int64_t n_f) {
    namespace gd = grouped_direct;
    const int64_t feats = op == kDgrad ? gd::kDF : gd::kF;
    return swiglu_host::grouped_row_tiles(rows, experts, gd::kRows) <=
           (int64_t)(UINT32_MAX / gd::kThreads) / ((n_f + feats - 1) / feats);
}

Path path_of(Op op, bool whole, bool large, int64_t rows, int64_t experts, int64_t n_f, int64_t n_t,
             int64_t n_r) {
    // No product: the general kernel stores zeros (the others' epilogues a row's scale times zero, NaN
    // where that is not finite).
    if (experts == 0 || (op != kWgrad && n_r == 0)) return kGeneralPath;
    if (op == kWgrad) {
        // Short groups: 754 rows, E = 6, 328 x 176 into fp32: 9 general, 13 in tiles; 348, E = 43,
        // 2032 x 128 into fp32: 12 and 20; 33, E = 2, 7248 x 3800: 24 and 33; but 1000, E = 8,
        // 1024 x 4096: 32 and 24; 2000: 49 and 33. Gradients larger than the
        // caches stay with the tiles (1711, E = 124, 1256 x 464 into fp32: 71 and 58).
        const int64_t steps = (rows + experts * kRedTile - 1) / (experts * kRedTile);
        const int64_t tiles = experts * ((n_t + 127) / 128) * ((n_f + 127) / 128);
        const bool few = steps <= (tiles <= 768 ? 6 : 1);
        if (!whole || (few && !large)) return kGeneralPath;
        return split_tiles(op, whole, rows, experts, n_f, n_t) <= kSplitJobs / 2 ? kSplitPath : kTilePath;
    }
    const bool fits = direct_fits(op, rows, experts, n_f), products = op == kMm || op == kFc1;
    // Rows that are not whole vectors: groups of about 4 rows or fewer (fc1, 4 rows, E = 112, n = 131,
    // k = 3195: 21 direct, 59 general; 71, E = 15, n = 4057, k = 1321: 119 and 157; mm, 846, E = 8, n = 421,
    // k = 3291: 97 and 25), but for reductions of a wave's one piece with more workgroups than stay at once
    // (fc1, 133, E = 118, n = 3638, k = 375: 260 and 166; 46, E = 47, n = 5547, k = 184: 68 and 41; mm, 30,
    // E = 10, n = 3001, k = 501: 17 and 18). Where only the output's rows are not whole, the direct
    // kernel's loads are vectors all the same.
    if (!whole) {
        const int64_t groups = rows < experts ? rows : experts;
        const bool turnover = n_r <= 512 && groups * ((n_f + 15) / 16) > 4096;
        return products && fits && rows <= 16 + 4 * experts && !turnover ? kDirectPath : kGeneralPath;
    }
    const Estimate E = estimate(op, rows, experts, n_f, n_r);
    const double tiles = E.split < E.tiles ? E.split : E.tiles;
    if (fits && E.direct < E.general && E.direct < tiles) return kDirectPath;
    if (E.general < tiles) return kGeneralPath;
    return E.split < E.tiles ? kSplitPath : kTilePath;
}

// Bytes of partial sums, 0 where no reduction is split: the real number of tiles
// may be any up to the bound, so the largest over all of them.
size_t split_bytes(Op op, bool whole, int64_t rows, int64_t experts, int64_t n_f, int64_t n_t,
                   int64_t n_r) {
    const Path path = path_of(op, whole, false, rows, experts, n_f, n_t, n_r);
    if (experts == 0 || (whole ? path != kSplitPath : path != kGeneralPath)) return 0;
    const int64_t tiles = split_tiles(op, whole, rows, experts, n_f, n_t);
    const int64_t len = split_len(op, rows, experts, n_r);
    if (tiles > kSplitJobs / 2 || split_parts((uint32_t)tiles, len) == 1) return 0;
    // (fewer tiles than t give at most t times the parts that the length allows)
    const int64_t limit = (len + kRedTile - 1) / kRedTile / 4;
    int64_t most = 0;
    for (int64_t t = tiles; t > 0 && most < kSplitJobs && most < t * limit; --t) {
        const int64_t parts = t * split_parts((uint32_t)t, len);
        most = parts > most ? parts : most;
    }
    const SplitShape S = split_shape(op, whole);
    return (size_t)most * S.rows * S.feats * 4;
}

template <Op OP, typename OutT, bool WHOLE>
swiglu_status launch_split(const GroupedArgs& P, void* workspace, hipStream_t stream) {
    constexpr int TT = WHOLE && OP == kWgrad ? 256 : 128, FF = WHOLE ? 256 : 128;
    constexpr int kTileF = OP == kFc1 ? FF / 2 : FF;
    uint32_t ft = (uint32_t)((P.n_f + kTileF - 1) / kTileF);
    int64_t len = split_len(OP, P.rows, P.experts, P.n_r);
    GroupedArgs Q = P;
    float* ws = static_cast<float*>(workspace);
    void* args[] = {&Q, &ft, &len, &ws};
    const void* k;
    if constexpr (WHOLE) k = reinterpret_cast<const void*>(&grouped_tile::grouped_split_kernel<OP, OutT>);
    else k = reinterpret_cast<const void*>(&grouped_general_kernel<OP, OutT, true>);
    static_assert(grouped_tile::kThreads == kGenThreads, "one block size");
    if (hipLaunchKernel(k, dim3(kSplitJobs), dim3(kGenThreads), args, 0, stream) != hipSuccess)
        return SWIGLU_ERR_HIP;
    const uint32_t join = (uint32_t)split_tiles(OP, WHOLE, P.rows, P.experts, P.n_f, P.n_t) *
                          kJoinGroups<TT, FF>;
    if (hipLaunchKernel(reinterpret_cast<const void*>(&grouped_join_kernel<OP, OutT, TT, FF>), dim3(join),
                        dim3(kJoinThreads), args, 0, stream) != hipSuccess)
        return SWIGLU_ERR_HIP;
    return SWIGLU_OK;
}

template <Op OP, typename OutT>
swiglu_status launch_general(const GroupedArgs& P, hipStream_t stream);

template <Op OP, typename OutT>
swiglu_status launch(const GroupedArgs& P, void* workspace, size_t bytes, hipStream_t stream) {
    const int64_t wf = OP == kMm || OP == kFc1 ? P.n_r : P.n_f;
    const int64_t wt = OP == kWgrad ? P.n_t : P.n_r;
    const bool inputs = whole_vectors(P.f, P.ldf, OP == kWgrad ? 0 : P.f_stride, wf, 2) &&
                        whole_vectors(P.t, P.ldt, 0, wt, 2);
    const bool whole = inputs && whole_vectors(P.out, P.ldo, OP == kWgrad ? P.o_stride : 0, P.n_f, sizeof(OutT));
    // The size that the caller was told goes by the widths alone.
    const bool vectors = wf % 8 == 0 && wt % 8 == 0 && P.n_f % 8 == 0;
    const size_t told = split_bytes(OP, vectors, P.rows, P.experts, P.n_f, P.n_t, P.n_r);
    if (workspace != nullptr && (bytes < told || (uintptr_t)workspace % 16 != 0)) return SWIGLU_ERR_WORKSPACE;
    const size_t need = whole == vectors ? told
                                         : split_bytes(OP, whole, P.rows, P.experts, P.n_f, P.n_t, P.n_r);
    const bool split = workspace != nullptr && need > 0 && bytes >= need;
    const Path path = path_of(OP, whole, P.large, P.rows, P.experts, P.n_f, P.n_t, P.n_r);
    if constexpr (OP == kDgrad)
        if (path == kDirectPath) return launch_direct<OP, false>(P, stream);
    if constexpr (OP == kMm || OP == kFc1)
        if (path == kDirectPath)
            return inputs ? launch_direct<OP, false>(P, stream) : launch_direct<OP, true>(P, stream);
    if (split)
        return whole ? launch_split<OP, OutT, true>(P, workspace, stream)
                     : launch_split<OP, OutT, false>(P, workspace, stream);
    return path == kGeneralPath ? launch_general<OP, OutT>(P, stream) : launch_tile<OP, OutT>(P, stream);
}

template <Op OP, typename OutT>
swiglu_status launch_general(const GroupedArgs& P, hipStream_t stream) {
    constexpr int kTileF = OP == kFc1 ? kGenTile / 2 : kGenTile;
    const int64_t f_tiles = (P.n_f + kTileF - 1) / kTileF;
    // every split of the rows over the experts has at most this many row tiles
    int64_t slots;
    if (OP == kWgrad) slots = P.experts * ((P.n_t + kGenTile - 1) / kGenTile);
    else slots = swiglu_host::grouped_row_tiles(P.rows, P.experts, kGenTile);
    if (slots >= kMaxTiles / f_tiles) return SWIGLU_ERR_BAD_SHAPE;
    uint32_t ft = (uint32_t)f_tiles;
    GroupedArgs Q = P;
    int64_t plan = 0;
    float* ws = nullptr;
    void* args[] = {&Q, &ft, &plan, &ws};
    if (hipLaunchKernel(reinterpret_cast<const void*>(&grouped_general_kernel<OP, OutT, false>),
                        dim3((uint32_t)(slots * f_tiles)), dim3(kGenThreads), args, 0, stream) !=
        hipSuccess)
        return SWIGLU_ERR_HIP;
    return SWIGLU_OK;
}

constexpr int64_t kMaxSize = (int64_t)1 << 30;

swiglu_status check_sizes(int64_t rows, int64_t experts, int64_t n, int64_t k, swiglu_dtype dtype) {
    if (dtype != SWIGLU_DTYPE_BF16) return SWIGLU_ERR_BAD_DTYPE;
    if (rows < 0 || experts < 0 || n < 0 || k < 0) return SWIGLU_ERR_BAD_SHAPE;
    // ends are 32-bit row numbers
    if (rows > (int64_t)INT32_MAX || experts > kMaxSize || n > kMaxSize || k > kMaxSize)
        return SWIGLU_ERR_BAD_SHAPE;
    return SWIGLU_OK;
}

// [experts] matrices of [height, width] elements, `between` apart.
swiglu_status check_weights(int64_t experts, int64_t between, int64_t height, int64_t ld,
                            int64_t width, int64_t esz) {
    swiglu_status st = check_operand(height, ld, width, esz);
    if (st != SWIGLU_OK) return st;
    if (height == 0 || width == 0) return SWIGLU_OK;
    const int64_t span = (height - 1) * ld + width;
    if (experts > 1 && between < span) return SWIGLU_ERR_BAD_STRIDE;
    if (experts > 1 && (experts - 1) > (INT64_MAX / esz - span) / between) return SWIGLU_ERR_BAD_SHAPE;
    return SWIGLU_OK;
}

swiglu_host::Span span(const void* p, int64_t rows, int64_t ld, int64_t width, int64_t esz) {
    if (p == nullptr || rows <= 0 || width <= 0) return {0, 0};
    return swiglu_host::span_of(Operand{p, ld}, rows, width, esz);
}

swiglu_host::Span weights_span(const void* p, int64_t experts, int64_t between, int64_t height,
                               int64_t ld, int64_t width, int64_t esz) {
    if (p == nullptr || experts <= 0 || height <= 0 || width <= 0) return {0, 0};
    swiglu_host::Span s = span(p, height, ld, width, esz);
    s.hi += (uintptr_t)((experts - 1) * between * esz);
    return s;
}

// Shared by mm, fc1 and dgrad: T [rows, width_t] -> out [rows, width_o] through
// weights [experts][w_rows, w_cols].
template <Op OP>
swiglu_status run_rows(const void* t, int64_t ldt, int64_t width_t, const void* w, int64_t ldw,
                       int64_t between, int64_t w_rows, int64_t w_cols, const int32_t* ends,
                       const float* scale, int64_t scale_stride, void* out, int64_t ldo,
                       int64_t width_o, int64_t rows, int64_t experts, void* workspace,
                       size_t workspace_bytes, hipStream_t stream) {
    swiglu_status st;
    if ((st = check_operand(rows, ldt, width_t, 2)) != SWIGLU_OK) return st;
    if ((st = check_operand(rows, ldo, width_o, 2)) != SWIGLU_OK) return st;
    if ((st = check_weights(experts, between, w_rows, ldw, w_cols, 2)) != SWIGLU_OK) return st;
    if (scale != nullptr && (st = check_operand(rows, scale_stride, 1, 4)) != SWIGLU_OK) return st;
    if (rows == 0 || width_o == 0) return SWIGLU_OK;
    if (!out || (experts > 0 && !ends)) return SWIGLU_ERR_NULL_POINTER;
    if (experts > 0 && width_t > 0 && (!t || !w)) return SWIGLU_ERR_NULL_POINTER;
    const Operand oo{out, ldo}, ot{t, ldt};
    if (t != nullptr && views_overlap(oo, width_o, ot, width_t, rows, 2)) return SWIGLU_ERR_ALIASING;
    const swiglu_host::Span so = span(out, rows, ldo, width_o, 2);
    if (swiglu_host::spans_overlap(so, weights_span(w, experts, between, w_rows, ldw, w_cols, 2)) ||
        swiglu_host::spans_overlap(so, span(ends, 1, experts, experts, 4)) ||
        swiglu_host::spans_overlap(so, span(scale, rows, scale_stride, 1, 4)))
        return SWIGLU_ERR_ALIASING;
    for (const swiglu_host::Span& x :
         {so, span(t, rows, ldt, width_t, 2), weights_span(w, experts, between, w_rows, ldw, w_cols, 2),
          span(ends, 1, experts, experts, 4), span(scale, rows, scale_stride, 1, 4)})
        if (swiglu_host::spans_overlap(x, span(workspace, 1, 0, (int64_t)workspace_bytes, 1)))
            return SWIGLU_ERR_ALIASING;
    GroupedArgs P{};
    P.f = static_cast<const uint16_t*>(w);
    P.t = static_cast<const uint16_t*>(t);
    P.out = out;
    P.scale = scale;
    P.ends = ends;
    P.ldf = ldw;
    P.ldt = ldt;
    P.ldo = ldo;
    P.f_stride = between;
    P.scale_stride = scale_stride;
    P.rows = rows;
    P.experts = experts;
    P.n_f = width_o;
    P.n_r = width_t;
    P.up = width_o;
    return launch<OP, uint16_t>(P, workspace, workspace_bytes, stream);
}

}  // namespace

extern "C" {

__attribute__((visibility("default"))) size_t swiglu_grouped_workspace_size(
    swiglu_grouped_op op, int64_t rows, int64_t experts, int64_t n, int64_t k) {
    if (check_sizes(rows, experts, n, k, SWIGLU_DTYPE_BF16) != SWIGLU_OK) return 0;
    if (rows == 0 || n == 0 || k == 0) return 0;
    const bool whole = n % 8 == 0 && k % 8 == 0;
    switch (op) {
        case SWIGLU_GROUPED_MM: return split_bytes(kMm, whole, rows, experts, n, 0, k);
        case SWIGLU_GROUPED_FC1: return split_bytes(kFc1, whole, rows, experts, n, 0, k);
        case SWIGLU_GROUPED_MM_DGRAD: return split_bytes(kDgrad, whole, rows, experts, k, 0, n);
        case SWIGLU_GROUPED_MM_WGRAD: return split_bytes(kWgrad, whole, rows, experts, k, n, 0);
    }
    return 0;
}

__attribute__((visibility("default"))) swiglu_status swiglu_grouped_mm(
    const void* a, int64_t lda, const void* w, int64_t ldw, int64_t w_expert_stride,
    const int32_t* ends, void* y, int64_t ldy, int64_t rows, int64_t experts, int64_t n, int64_t k,
    swiglu_dtype dtype, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    const swiglu_status st = check_sizes(rows, experts, n, k, dtype);
    if (st != SWIGLU_OK) return st;
    return run_rows<kMm>(a, lda, k, w, ldw, w_expert_stride, n, k, ends, nullptr, 1, y, ldy, n, rows,
                         experts, workspace, workspace_bytes, stream);
}

__attribute__((visibility("default"))) swiglu_status swiglu_grouped_fc1(
    const void* a, int64_t lda, const void* w, int64_t ldw, int64_t w_expert_stride,
    const int32_t* ends, const float* scale, int64_t scale_stride, void* y, int64_t ldy,
    int64_t rows, int64_t experts, int64_t n, int64_t k, swiglu_dtype dtype, void* workspace,
    size_t workspace_bytes, hipStream_t stream) {
    const swiglu_status st = check_sizes(rows, experts, n, k, dtype);
    if (st != SWIGLU_OK) return st;
    return run_rows<kFc1>(a, lda, k, w, ldw, w_expert_stride, 2 * n, k, ends, scale, scale_stride, y,
                          ldy, n, rows, experts, workspace, workspace_bytes, stream);
}

__attribute__((visibility("default"))) swiglu_status swiglu_grouped_mm_dgrad(
    const void* dy, int64_t lddy, const void* w, int64_t ldw, int64_t w_expert_stride,
    const int32_t* ends, void* da, int64_t ldda, int64_t rows, int64_t experts, int64_t n, int64_t k,
    swiglu_dtype dtype, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    const swiglu_status st = check_sizes(rows, experts, n, k, dtype);
    if (st != SWIGLU_OK) return st;
    return run_rows<kDgrad>(dy, lddy, n, w, ldw, w_expert_stride, n, k, ends, nullptr, 1, da, ldda, k,
                            rows, experts, workspace, workspace_bytes, stream);
}

__attribute__((visibility("default"))) swiglu_status swiglu_grouped_mm_wgrad(
    const void* dy, int64_t lddy, const void* a, int64_t lda, const int32_t* ends, void* dw,
    int64_t lddw, int64_t dw_expert_stride, int64_t rows, int64_t experts, int64_t n, int64_t k,
    swiglu_dtype dtype, swiglu_dtype dw_dtype, void* workspace, size_t workspace_bytes,
    hipStream_t stream) {
    swiglu_status st = check_sizes(rows, experts, n, k, dtype);
    if (st != SWIGLU_OK) return st;
    if (dw_dtype != SWIGLU_DTYPE_BF16 && dw_dtype != SWIGLU_DTYPE_F32) return SWIGLU_ERR_BAD_DTYPE;
    const int64_t oesz = dw_dtype == SWIGLU_DTYPE_F32 ? 4 : 2;
    if ((st = check_operand(rows, lddy, n, 2)) != SWIGLU_OK) return st;
    if ((st = check_operand(rows, lda, k, 2)) != SWIGLU_OK) return st;
    if ((st = check_weights(experts, dw_expert_stride, n, lddw, k, oesz)) != SWIGLU_OK) return st;
    if (experts == 0 || n == 0 || k == 0) return SWIGLU_OK;
    if (!dw || !ends || (rows > 0 && (!dy || !a))) return SWIGLU_ERR_NULL_POINTER;
    const swiglu_host::Span so = weights_span(dw, experts, dw_expert_stride, n, lddw, k, oesz);
    if (swiglu_host::spans_overlap(so, span(dy, rows, lddy, n, 2)) ||
        swiglu_host::spans_overlap(so, span(a, rows, lda, k, 2)) ||
        swiglu_host::spans_overlap(so, span(ends, 1, experts, experts, 4)))
        return SWIGLU_ERR_ALIASING;
    for (const swiglu_host::Span& x : {so, span(dy, rows, lddy, n, 2), span(a, rows, lda, k, 2),
                                       span(ends, 1, experts, experts, 4)})
        if (swiglu_host::spans_overlap(x, span(workspace, 1, 0, (int64_t)workspace_bytes, 1)))
            return SWIGLU_ERR_ALIASING;
    GroupedArgs P{};
    P.f = static_cast<const uint16_t*>(a);
    P.t = static_cast<const uint16_t*>(dy);
    P.out = dw;
    P.ends = ends;
    P.ldf = lda;
    P.ldt = lddy;
    P.ldo = lddw;
    P.o_stride = dw_expert_stride;
    P.rows = rows;
    P.experts = experts;
    P.n_f = k;
    P.n_t = n;
    // Past 256 MiB, the size of the Infinity Cache, nothing of the gradients is
    // left there for a reader, and of short groups their stores are the time:
    // 940 MB from groups of 188 rows 228 us cached, 195 streamed; 537 MB from
    // groups of 2048 rows 852 and 868; 77 MB of token gradients 43 and 66.
    const bool lines = ((uintptr_t)dw | (uintptr_t)(lddw * oesz) | (uintptr_t)(dw_expert_stride * oesz)) % 128 == 0;
    P.large = experts > ((int64_t)256 << 20) / (n * k * oesz) && rows / experts < 1024;
    P.stream = P.large && lines;
    return dw_dtype == SWIGLU_DTYPE_F32 ? launch<kWgrad, float>(P, workspace, workspace_bytes, stream)
                                        : launch<kWgrad, uint16_t>(P, workspace, workspace_bytes, stream);
}

}  // extern "C"
