// The large-tile product of swiglu_grouped.hip, for operands whose rows are
// whole, aligned 16-byte vectors. Workgroups of 4 waves, one per CU, stay for the
// whole launch and make one output tile after the other: TT rows x 256 features
// (fc1: 128 gate and 128 up features) of an expert, TT = 256 or 128.
//
// Design (bf16 in, fp32 accumulate, MFMA 32x32x16):
//  * Each wave makes TT/2 rows x 128 features: 4 x (TT/64) MFMA tiles, for
//    TT = 256 all 256 accumulation registers of a lane. Features are the MFMA's row
//    operand, so a lane ends up with four consecutive features of one row.
//  * The reduction is walked in tiles of 64 through two rings of LDS stages, 2
//    of the T operand (TT x 64) and 3 of the F operand (256 x 64): 160 KiB in
//    all. Copies go from memory straight to LDS (buffer_load_dwordx4 lds). T is
//    copied one tile ahead, F two: the weights miss the L2 more often. Each stage
//    is an LDS array of its own (T: two, of half its rows) and the loop is unrolled over 6
//    tiles (the rings' common period), so every stage is named statically and no wait is put
//    in front of reads for copies that cannot alias them.
//  * A row laid operand's stage holds rows of 64 along the reduction, fragments
//    are 16-byte reads; a column laid one's holds 64 rows of the output's index
//    and fragments are two transposing 8-byte reads each. Chunks of 16 bytes are
//    permuted within their row by an XOR with bits of the row (chosen through
//    the global addresses: a copy writes LDS in lane order) so that lanes that
//    read together meet different banks.
//  * Rows, columns and reduction indexes past the end are given an offset past
//    the buffer descriptor's range: such lanes read zeros and touch no memory.
//    The descriptor's base moves along the reduction, so offsets are those
//    within one tile and fit 31 bits for any length.
//  * One k step of 16 is written out as its MFMAs with the next step's fragment
//    reads and the copies pinned between them; one barrier per tile.
//  * Between two tiles, the next one's first copies are started before the
//    finished one is rounded and stored, which goes through the one LDS stage
//    they leave free. As a workgroup per tile the launch, the search and the
//    first copies took 16 000 cycles of a tile's 162 000 (k = 4096).
#ifndef SWIGLU_GROUPED_TILE_H
#define SWIGLU_GROUPED_TILE_H

namespace grouped_tile {

using namespace swiglu_impl;

typedef __attribute__((address_space(3))) void lds_void;

constexpr int kThreads = 256, kWaves = 4;
constexpr int kK = 64;                               // reduction per stage
constexpr int kFRows = 256;                          // F rows (features) per tile
constexpr int kPeriod = 6;                           // lcm of the rings' 2 and 3 stages
constexpr uint32_t kOutside = 0x80000000u;           // an offset past every descriptor's range
constexpr int64_t kMaxLd = (int64_t)1 << 20;         // 256 rows x 4 bytes x ld stays within 2^30 + 2^10

// The LDS rings.
constexpr int kTRows = 256;                          // T rows of a stage (at most)
__shared__ __attribute__((aligned(16))) uint16_t gt_t0[kTRows * kK / 2];
__shared__ __attribute__((aligned(16))) uint16_t gt_t1[kTRows * kK / 2];
__shared__ __attribute__((aligned(16))) uint16_t gt_t2[kTRows * kK / 2];
__shared__ __attribute__((aligned(16))) uint16_t gt_t3[kTRows * kK / 2];
__shared__ __attribute__((aligned(16))) uint16_t gt_f0[kFRows * kK];
__shared__ __attribute__((aligned(16))) uint16_t gt_f1[kFRows * kK];
__shared__ __attribute__((aligned(16))) uint16_t gt_f2[kFRows * kK];

template <int S>
__device__ __forceinline__ uint16_t* half_t() {
    if constexpr (S == 0) return gt_t0;
    else if constexpr (S == 1) return gt_t1;
    else if constexpr (S == 2) return gt_t2;
    else return gt_t3;
}
template <int S>
__device__ __forceinline__ uint16_t* stage_f() {
    if constexpr (S == 0) return gt_f0;
    else if constexpr (S == 1) return gt_f1;
    else return gt_f2;
}

// Slot of 16-byte chunk c in LDS row r: rows of 8 chunks (row laid) or of
// ROWS / 8 (column laid, 4 rows x 64 bytes per 32 lanes of a transposing read).
__device__ __forceinline__ int row_slot(int r, int c) { return c ^ ((r >> 1) & 7); }
__device__ __forceinline__ int col_slot(int r, int c) {
    return c ^ (((r & 3) << 2) | (((r >> 3) & 1) << 1));
}

// s_waitcnt: at most N copies outstanding, and no LDS operation.
template <int N>
__device__ __forceinline__ void wait_copies_and_lds() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
}

__device__ __forceinline__ void ring_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// One operand of the tile: ROWS of the output's index by the reduction. SPLIT:
// the second half of the rows lies `up` bytes after the first (fc1's weights,
// whose up rows are too far from the gate rows for one range of offsets).
template <bool COL, int ROWS, bool SPLIT>
struct Source {
    static constexpr int kCopies = ROWS * kK * 2 / 1024 / kWaves;    // per wave and stage
    static constexpr int kLdsRow = COL ? ROWS : kK;                  // elements per LDS row
    static constexpr int kCopyRows = 512 / kLdsRow;                  // LDS rows per copy (1 KiB)
    const char* base;          // the tile's first element
    int64_t up;                // SPLIT
    int64_t step;              // bytes from one stage's tile to the next
    int last;                  // index of the last reduction tile
    int rem;                   // reduction indexes in it
    uint32_t off[kCopies];     // this lane's byte offset in each copy
    int first;                 // reduction index (within a tile) of this lane in copy 0

    // The memory row, counted from the half's first, of tile row r.
    static __device__ __forceinline__ int row_of(int r) { return SPLIT ? r % (ROWS / 2) : r; }
    // row(r): whether tile row r exists (row laid); width: columns left
    // (column laid).
    template <typename Row>
    __device__ __forceinline__ void init(const uint16_t* p, int64_t ld, int32_t len, int32_t width,
                                         Row row) {
        const int lane = threadIdx.x & 63;
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        base = reinterpret_cast<const char*>(p);
        step = COL ? kK * ld * 2 : kK * 2;
        last = (len - 1) / kK;
        rem = len - last * kK;
        constexpr int kPer = 64 / kCopyRows;                         // chunks per LDS row
        const int lr = lane / kPer, ls = lane % kPer;
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
            const int r = (i * kWaves + wave) * kCopyRows + lr;
            if constexpr (COL) {
                const int c = col_slot(r, ls) * 8;                   // an XOR: its own inverse
                off[i] = c < width ? (uint32_t)(r * (int32_t)ld * 2 + c * 2) : kOutside;
            } else {
                const int c = row_slot(r, ls) * 8;
                off[i] = row(r) ? (uint32_t)(row_of(r) * (int32_t)ld * 2 + c * 2) : kOutside;
            }
        }
        // row laid: a lane has the same chunk in all its copies (the rows of two
        // copies are a multiple of 16 apart)
        first = COL ? wave * kCopyRows + lr : row_slot(wave * kCopyRows + lr, ls) * 8;
    }

    // Starts copy i of reduction tile t to place `at` of stage memory lds. Past the last
    // tile every lane is outside: the copy is counted, and reads nothing.
    __device__ __forceinline__ void copy(int i, int t, uint16_t* lds) const { copy(i, t, lds, i); }
    __device__ __forceinline__ void copy(int i, int t, uint16_t* lds, int at) const {
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int left = t < last ? kK : t == last ? rem : 0;        // uniform
        uint32_t o = off[i];
        if constexpr (COL) o = first + i * kWaves * kCopyRows < left ? o : kOutside;
        else o = first < left ? o : kOutside;
        const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<char*>(base + (SPLIT && i >= kCopies / 2 ? up : 0) + t * step), 0,
            (int)kOutside, 0x00020000);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rsrc, (lds_void*)(lds + (at * kWaves + wave) * 512), 16, (int)o, 0, 0, 0);
    }
};

// Fragment addresses: element offsets in a stage. Row laid: tile rows lie
// 32 LDS rows apart, the four steps' chunks are permuted. Column laid: the steps lie 16
// LDS rows apart, the tiles' chunks are permuted.
template <bool COL, int ROWS>
struct FragBase {
    int off[4];
    __device__ __forceinline__ void init(int out0) {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if constexpr (!COL) {
                const int r = out0 + lane % 32;
                off[q] = r * kK + row_slot(r, 2 * q + lane / 32) * 8;
            } else {
                const int r = 8 * (lane / 32) + (lane % 16) / 4;
                const int c = out0 + 32 * q + 16 * ((lane / 16) & 1) + 4 * (lane % 4);
                off[q] = r * ROWS + col_slot(r, c / 8) * 8 + c % 8;
            }
        }
    }
    // Fragment of MFMA tile i (32 rows of the output's index; `at` elements
    // from the first for row laid operands) in k step s.
    __device__ __forceinline__ bf16x8 read(const uint16_t* lds, int i, int at, int s) const {
        if constexpr (!COL) {
            return __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(lds + at * kK + off[s]));
        } else {
            const uint16_t* p = lds + off[i] + 16 * s * ROWS;
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * ROWS));
            const __attribute__((ext_vector_type(8))) short v =
                __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
            return __builtin_bit_cast(bf16x8, v);
        }
    }
};

// ---------------------------------------------------------------------------
// Which tiles a workgroup makes (mm, fc1, dgrad). Every group's rows are cut in
// tiles of 256; a rest of at most 128 rows is a tile of 128. Each XCD takes a
// contiguous eighth of the large tiles and of the small ones, and its
// workgroups take them in turn, the large ones first. Small tiles go first to
// those whom the last round of the large ones left out, two each. If there are fewer and
// that round would keep at most half of the workgroups busy, its tiles are
// cut in halves (which read the weights twice: with enough small tiles that costs
// more than it gives).
// ---------------------------------------------------------------------------
struct Schedule {
    uint32_t f_tiles, per, j;              // feature tiles; workgroups per XCD; this one's place
    uint32_t full0, nf, half0, nh, keep;   // this XCD's tiles; keep: large ones not cut
    int64_t base;                          // first expert held in the lanes
    uint32_t top;                          // end of the last one
    uint32_t l, h, full, half, sfull, shalf;   // lane's expert: rows, tiles, inclusive sums

    // Experts b on, after those that the lanes hold (or from the first).
    __device__ __forceinline__ void scan(const GroupedArgs& P, int64_t b) {
        const int lane = threadIdx.x & 63;
        base = b;
        const uint32_t begin = b == 0 ? 0 : top;
        uint32_t v = 0;
        if (b + lane < P.experts) v = (uint32_t)swiglu_host::group_end(0, P.ends[b + lane], (int32_t)P.rows);
        v = max_scan(v);
        h = v > begin ? v : begin;
        l = from_lane<0x138>(begin, h);                  // the lane before
        top = lane_of(h, 63);
        const uint32_t rest = (h - l) % 256;
        half = rest > 0 && rest <= 128 ? 1 : 0;
        full = (h - l) / 256 + (rest > 128 ? 1 : 0);
        sfull = full;
        shalf = half;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const uint32_t a = __shfl_up(sfull, d, 64), c = __shfl_up(shalf, d, 64);
            if (lane >= d) {
                sfull += a;
                shalf += c;
            }
        }
    }
    static __device__ __forceinline__ void eighth(uint32_t total, uint32_t x, uint32_t& first,
                                                  uint32_t& n) {
        const uint32_t q = total / kXcds, r = total % kXcds;
        first = x * q + (x < r ? x : r);
        n = q + (x < r ? 1 : 0);
    }
    __device__ __forceinline__ void init(const GroupedArgs& P, uint32_t tiles) {
        f_tiles = tiles;
        per = gridDim.x / kXcds;
        j = blockIdx.x / kXcds;
        scan(P, 0);
        uint32_t fulls = lane_of(sfull, 63), halves = lane_of(shalf, 63);
        Schedule later = *this;                          // (the first 64 stay in the lanes)
        for (int64_t b = 64; b < P.experts; b += 64) {
            later.scan(P, b);
            fulls += lane_of(later.sfull, 63);
            halves += lane_of(later.shalf, 63);
        }
        eighth(fulls * f_tiles, blockIdx.x % kXcds, full0, nf);
        eighth(halves * f_tiles, blockIdx.x % kXcds, half0, nh);
        const uint32_t last = nf % per;
        keep = last <= per / 2 && nh < 2 * (per - last) ? nf - last : nf;
    }
    // Tile number idx of the large (or small) ones.
    __device__ __forceinline__ void locate(const GroupedArgs& P, bool large, uint32_t idx, Job& J) {
        const uint32_t slot = idx / f_tiles;
        uint32_t before = 0;
        for (int64_t b = 0; b < P.experts; b += 64) {
            if (b != base) scan(P, b);
            const uint32_t sum = large ? sfull : shalf;
            const uint64_t past = __ballot(before + sum > slot);
            if (past != 0) {
                const int w = __builtin_ctzll(past);
                const uint32_t tiles = lane_of(large ? full : half, w);
                const uint32_t in = idx - (before + lane_of(sum, w) - tiles) * f_tiles;
                uint32_t tt, ft;
                if (large) {
                    tile_in_expert(in, tiles, f_tiles, tt, ft);
                } else {
                    tt = lane_of(full, w);
                    ft = in;
                }
                J.expert = (int32_t)b + w;
                J.lo = (int32_t)lane_of(l, w);
                J.t0 = J.lo + (int32_t)tt * 256;
                J.t1 = (int32_t)lane_of(h, w);
                J.f0 = (int32_t)ft;                      // feature tile
                return;
            }
            before += lane_of(sum, 63);
        }
    }
    __device__ __forceinline__ Job get(const GroupedArgs& P, uint32_t i) {
        Job J{};
        const uint32_t mine = keep > j ? (keep - j - 1) / per + 1 : 0;
        if (i < mine) {
            locate(P, true, full0 + j + i * per, J);
            J.tt = 256;
            return J;
        }
        i -= mine;
        const uint32_t b = keep % per, out = b > 0 ? per - b : 0;   // left out of the last round
        uint32_t idx;
        if (b > 0 && j >= b) idx = i < 2 ? i * out + (j - b) : 2 * out + j + (i - 2) * per;
        else idx = 2 * out + j + i * per;
        if (idx < nh) {
            locate(P, false, half0 + idx, J);
        } else if (idx - nh < 2 * (nf - keep)) {
            locate(P, true, full0 + keep + (idx - nh) / 2, J);
            J.t0 += (idx - nh) % 2 * 128;
        } else {
            return J;
        }
        J.tt = 128;
        return J;
    }
};

// The operands of one tile.
template <Op OP>
struct Operands {
    static constexpr bool F_COL = OP == kDgrad || OP == kWgrad, T_COL = OP == kWgrad;
    typedef Source<F_COL, kFRows, OP == kFc1> SrcF;
    typedef Source<T_COL, kTRows, false> SrcT;
    SrcF sf;
    SrcT st;                                             // a tile of 128 uses the first half
    __device__ __forceinline__ void init(const GroupedArgs& P, const Job& J) {
        if constexpr (OP == kWgrad) {
            sf.init(P.f + (int64_t)(J.lo + J.r0) * P.ldf + J.f0, P.ldf, J.len, P.n_f - J.f0, [](int) { return true; });
            st.init(P.t + (int64_t)(J.lo + J.r0) * P.ldt + J.t0, P.ldt, J.len, J.t1 - J.t0, [](int) { return true; });
        } else {
            const uint16_t* w = P.f + J.expert * P.f_stride;
            if constexpr (OP == kDgrad) {
                sf.init(w + (int64_t)J.r0 * P.ldf + J.f0, P.ldf, J.len, P.n_f - J.f0, [](int) { return true; });
            } else {
                const int32_t left = (int32_t)P.n_f - J.f0;
                sf.init(w + (int64_t)J.f0 * P.ldf + J.r0, P.ldf, J.len, 0,
                        [&](int r) { return SrcF::row_of(r) < left; });
                if constexpr (OP == kFc1) sf.up = P.up * P.ldf * 2;
            }
            st.init(P.t + (int64_t)J.t0 * P.ldt + J.r0, P.ldt, J.len, 0,
                    [&](int r) { return r < J.t1 - J.t0; });
        }
    }
    // The copies that a tile's first slot expects: all of reduction tiles 0 and 1.
    template <int TT>
    __device__ __forceinline__ void fill() const {
        if constexpr (TT == 256) copy_t(0, half_t<0>(), half_t<1>());
        else copy_t(0, half_t<0>());
#pragma unroll
        for (int i = 0; i < SrcF::kCopies; ++i) sf.copy(i, 0, stage_f<0>());
        if constexpr (TT == 256) copy_t(1, half_t<2>(), half_t<3>());
        else copy_t(1, half_t<1>());
#pragma unroll
        for (int i = 0; i < SrcF::kCopies; ++i) sf.copy(i, 1, stage_f<1>());
    }
    // T's reduction tile t: 128 rows (the first half of the copies), or 256.
    __device__ __forceinline__ void copy_t(int t, uint16_t* a, uint16_t* b = nullptr) const {
        constexpr int kHalf = SrcT::kCopies / 2;
#pragma unroll
        for (int i = 0; i < kHalf; ++i) st.copy(i, t, a);
        if (b != nullptr)
#pragma unroll
            for (int i = 0; i < kHalf; ++i) st.copy(kHalf + i, t, b, i);
    }
};

template <Op OP, typename OutT, int TT>
struct Tile {
    // Stores of a wave for a tile of tt rows.
    static constexpr int Stores(int tt) { return tt / 16 * (OP == kFc1 ? 1 : (int)sizeof(OutT)); }
    static constexpr int kMT = TT / 64;                  // MFMA tiles per wave along the rows
    static constexpr int kMfma = 4 * kMT;                // per k step
    static constexpr int kReads = 4 + kMT;
    static constexpr int kCopiesT = TT / 32, kCopiesF = Operands<OP>::SrcF::kCopies;
    static constexpr int kHalfT = kCopiesT / 2, kHalfF = kCopiesF / 2;
    // Tiles of 256 fill two T arrays a slot; tiles of 128 one, so that T too is
    // copied two slots ahead (one ahead is 770 cycles before its use, less than the L2 takes
    // under load), and no slot's copies share an array with what is read meanwhile.
    static constexpr bool kPairs = TT == 128;
    static constexpr int kPeriodTT = kPairs ? 2 * kPeriod : kPeriod;
    static constexpr int kLeft = kPairs ? kCopiesT + kCopiesF : kCopiesF;   // copies of slot kt + 2 before the barrier
    // The MFMA after which a step's first copy goes, and the MFMAs between
    // two copies.
    static constexpr int kPos = kMT == 4 ? 9 : 4, kStride = kMT == 4 ? 2 : 1;

    struct Frags {
        bf16x8 f[4], t[kMT];
    };

    const Operands<OP>& src;
    FragBase<Operands<OP>::F_COL, kFRows> bf;
    FragBase<Operands<OP>::T_COL, kTRows> bt;
    f32x16 acc[4][kMT];

    __device__ __forceinline__ Tile(const Operands<OP>& s, int wf, int wt) : src(s) {
        bf.init(wf);
        bt.init(wt);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < kMT; ++j) acc[i][j] = f32x16{};
    }
    // Keeps the sums in the accumulation registers up to here: left to itself the
    // compiler moves them all to vector registers where paths meet, ahead of
    // their use, and spills what those held.
    __device__ __forceinline__ void pin() {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < kMT; ++j) asm volatile("" : "+a"(acc[i][j]));
    }
    // Row of the stage where the wave's MFMA tile i of F begins, counted from
    // its first: fc1 takes gate and up tiles in turn.
    static __device__ __forceinline__ constexpr int f_at(int i) {
        return OP == kFc1 ? 32 * (i / 2) + 128 * (i % 2) : 32 * i;
    }
    __device__ __forceinline__ bf16x8 read_f(const uint16_t* lds, int i, int s) const {
        return bf.read(lds, i, f_at(i), s);
    }
    // T's fragment of row tile j in k step s of the slot at place J. Of 256 rows an array
    // holds rows 0 to 127 or the others, and a wave takes two row tiles of each
    // (row_block); column laid, it holds the first or the last two k steps.
    template <int J>
    __device__ __forceinline__ bf16x8 read_t(int j, int s) const {
        if constexpr (kPairs) return bt.read(half_t<J % 4>(), j, 32 * j, s);
        else if constexpr (Operands<OP>::T_COL)
            return s < 2 ? bt.read(half_t<J % 2 * 2>(), j, 0, s) : bt.read(half_t<J % 2 * 2 + 1>(), j, 0, s - 2);
        else return j < 2 ? bt.read(half_t<J % 2 * 2>(), j, 32 * j, s)
                          : bt.read(half_t<J % 2 * 2 + 1>(), j, 32 * (j - 2), s);
    }

    // One k step: MFMA m, then at their places one fragment of the next step
    // (step S1 of the slot at place J, whose F stage is nf) and one copy, nothing moved across.
    template <int S1, int J, int NC, class CopyFn>
    __device__ __forceinline__ void step(const uint16_t* nf, const Frags& C, Frags& N, CopyFn copy) {
        static_assert(NC == 0 || kPos + (NC - 1) * kStride < kMfma, "every copy has an MFMA to follow");
        static_assert(kReads <= kMfma, "every read has an MFMA to follow");
#pragma unroll
        for (int m = 0; m < kMfma; ++m) {
            const int i = 2 * (m / (2 * kMT)) + (m & 1), j = (m / 2) % kMT;
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(C.f[i], C.t[j], acc[i][j], 0, 0, 0);
            if (m < kMT) N.t[m] = read_t<J>(m, S1);
            else if (m < kReads) N.f[m - kMT] = read_f(nf, m - kMT, S1);
            if (m >= kPos && (m - kPos) % kStride == 0 && (m - kPos) / kStride < NC)
                copy((m - kPos) / kStride);
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    // s_waitcnt for everything before the last N copies and stores.
    template <int N>
    static __device__ __forceinline__ void wait_before() {
        wait_copies_and_lds<(N < 63 ? N : 63)>();
    }
    // Reduction tile kt at place J of the period. Entering: A holds (or receives)
    // its first step's fragments; issued are the F copies up to tile kt + 1's and
    // the T copies up to (kPairs) all or the first half of tile kt + 1's.
    // Leaving: the same one tile on. FIRST: tile 0, all of whose and of tile 1's
    // copies came before the `stored` rows' stores of the tile before: those need
    // not have ended with it, which leaves them two slots' time.
    template <int J, bool FIRST = false>
    __device__ __forceinline__ void slot(int kt, Frags& A, Frags& B, int stored = 0) {
        constexpr int J1 = (J + 1) % kPeriodTT, J2 = (J + 2) % kPeriodTT;
        uint16_t *lf = stage_f<J % 3>(), *lf1 = stage_f<J1 % 3>(), *lf2 = stage_f<J2 % 3>();
        if constexpr (kPairs)
            step<1, J, kCopiesT>(lf, A, B, [&](int q) { src.st.copy(q, kt + 2, half_t<J2 % 4>()); });
        else if constexpr (FIRST)
            step<1, J, 0>(lf, A, B, [](int) {});
        else
            step<1, J, kHalfT>(lf, A, B, [&](int q) { src.st.copy(kHalfT + q, kt + 1, half_t<J1 % 2 * 2 + 1>(), q); });
        step<2, J, kHalfF>(lf, B, A, [&](int q) { src.sf.copy(q, kt + 2, lf2); });
        step<3, J, kHalfF>(lf, A, B, [&](int q) { src.sf.copy(kHalfF + q, kt + 2, lf2); });
        // tile kt + 1 is complete once only tile kt + 2's copies are left
        if (FIRST && stored == 256) wait_before<kLeft + Stores(256)>();
        else if (FIRST && stored == 128) wait_before<kLeft + Stores(128)>();
        else wait_before<kLeft>();
        ring_barrier();
        if constexpr (kPairs) step<0, J1, 0>(lf1, B, A, [](int) {});
        else step<0, J1, kHalfT>(lf1, B, A, [&](int q) { src.st.copy(q, kt + 2, half_t<J2 % 2 * 2>()); });
    }
    // Tiles kt + J - 1 on, at places J to the period's first.
    template <int J>
    __device__ __forceinline__ void period(int kt, Frags& A, Frags& B) {
        slot<J % kPeriodTT>(kt + J - 1, A, B);
        if constexpr (J < kPeriodTT) period<J + 1>(kt, A, B);
    }
    // (one branch after the other: nested ones cost the compiler its registers)
    template <int J>
    __device__ __forceinline__ void remainder(int kt, int rest, Frags& A, Frags& B) {
        if (rest >= J) slot<J>(kt + J - 1, A, B);
        if constexpr (J + 1 < kPeriodTT) remainder<J + 1>(kt, rest, A, B);
    }

    // All of the reduction, from the copies that fill() has started, and after
    // which exactly the stores of a tile of `stored` rows (0: none) were issued:
    // fewer would end a wait early. On return the stages are free.
    __device__ __forceinline__ void multiply(int stored) {
        constexpr int kTile1 = kCopiesT + kCopiesF;
        if (stored == 256) wait_before<kTile1 + Stores(256)>();
        else if (stored == 128) wait_before<kTile1 + Stores(128)>();
        else wait_before<kTile1>();
        ring_barrier();
        Frags A, B;
#pragma unroll
        for (int j = 0; j < kMT; ++j) A.t[j] = read_t<0>(j, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) A.f[i] = read_f(stage_f<0>(), i, 0);
        const int count = src.sf.last + 1;
        slot<0, true>(0, A, B, stored);
        int kt = 1;
        for (; kt + kPeriodTT <= count; kt += kPeriodTT) period<1>(kt, A, B);
        remainder<1>(kt, count - kt, A, B);
        wait_copies_and_lds<0>();                        // no copy may land in reused memory
        ring_barrier();
    }
};

// Writes BYTES of features (NI MFMA tiles of 32) of 32 of the wave's rows, from
// row 32 j and feature fw: value(i, e) is element e of the tile (feature tile i); register e
// holds feature (e % 4) + 8 (e / 4) + 4 (lane / 32) and row lane % 32. Staged through
// the wave's own part of the free LDS stage, so that every store writes BYTES of
// each of its rows: where rows are not whole 128-byte lines, runs of 256 bytes touch 5
// half lines for 4, runs of 128 3 for 2. 16-byte chunks are permuted within their row by
// an XOR with bits of the row. out: the wave's first row, of which `left` exist.
// Rows and features past the end are stored outside the descriptor's range,
// which drops them: the number of stores is always 32 BYTES / 1024 (the waits
// for the next tile's copies count them). stream: past the caches (nontemporal).
template <int BYTES, typename OutT, typename V>
__device__ __forceinline__ void epi_out(int wave, int j, int32_t left, int32_t fw, int32_t n_f, OutT* out,
                                        int32_t ld, bool stream, V value) {
    constexpr int kSize = (int)sizeof(OutT), NI = BYTES / (32 * kSize);
    constexpr int kPer = BYTES / 16, kAt = 64 / kPer;    // lanes per row, rows per store
    static_assert(kWaves * 32 * BYTES <= kFRows * kK * 2, "the waves' parts fit the stage");
    const int lane = threadIdx.x & 63;
    char* region = reinterpret_cast<char*>(stage_f<2>()) + wave * (32 * BYTES);
    const __amdgpu_buffer_rsrc_t rsrc =
        __builtin_amdgcn_make_buffer_rsrc(out, 0, (int)kOutside, 0x00020000);
    const int32_t f = fw + (lane % kPer) * (16 / kSize);
    const uint32_t at = f < n_f ? (uint32_t)(((lane / kPer) * ld + f) * kSize) : kOutside;
    const uint32_t step = (uint32_t)(kAt * ld * kSize);
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float v[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] = value(i, 4 * q + r);
            const int b = (32 * i + 8 * q + 4 * (lane / 32)) * kSize;             // byte of the row
            char* p = region + (lane % 32) * BYTES + (((b / 16) ^ (lane % kPer)) * 16 + b % 16);
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
    // back by rows: lane l takes 16 bytes of row kAt it + l / kPer
#pragma unroll
    for (int it = 0; it < 32 / kAt; ++it) {
        const int row = kAt * it + lane / kPer;
        const u32x4 v = *reinterpret_cast<const u32x4*>(
            region + row * BYTES + ((lane % kPer) ^ (row % kPer)) * 16);
        const uint32_t o = 32 * j + row < left && at != kOutside ? at + (32 / kAt * j + it) * step : kOutside;
        if (stream) __builtin_amdgcn_raw_buffer_store_b128(v, rsrc, (int)o, 0, 2);
        else __builtin_amdgcn_raw_buffer_store_b128(v, rsrc, (int)o, 0, 0);
    }
    __builtin_amdgcn_sched_barrier(0);                   // one block's registers at a time
}

// A wave's first row in the tile, and the block of 32 rows from there that its row
// tile j is: of 256 rows two blocks of the first 128 and two of the others (wgrad:
// four in a row).
template <Op OP>
__device__ __forceinline__ int wave_row(int wave) { return wave / 2 * (OP == kWgrad ? 128 : 64); }
template <Op OP>
__device__ __forceinline__ constexpr int row_block(int j) { return OP == kWgrad || j < 2 ? j : j + 2; }

// Rounds and stores the tile J of sums M (fc1: with its activation and the
// rows' scales s), all of a wave's features of 32 rows before the next rows: the
// lines that two runs share are then written soon after one another, and leave
// the L2 whole (98 fp32 gradients of 456 x 6104: 306 us, and 380 a run of all rows first).
template <Op OP, typename OutT, int TT, int NS>
__device__ __forceinline__ void store_tile(const GroupedArgs& P, const Job& J, const Tile<OP, OutT, TT>& M,
                                           const float (&s)[NS], int wave) {
    constexpr int kRows = TT / 2;                        // rows per wave
    const int wf = (wave % 2) * (OP == kFc1 ? 64 : 128), wt = wave_row<OP>(wave);
    const int32_t row = J.t0 + wt, left = J.t1 - row;
    OutT* out = static_cast<OutT*>(P.out) + (OP == kWgrad ? J.expert * P.o_stride : 0) +
                (int64_t)row * P.ldo;
#pragma unroll
    for (int j = 0; j < kRows / 32; ++j) {
        if constexpr (OP == kFc1) {
            epi_out<128, OutT>(wave, row_block<OP>(j), left, J.f0 + wf, (int32_t)P.n_f, out, (int32_t)P.ldo, false,
                               [&](int i, int e) {
                const float g = M.acc[2 * i][j][e];
                float sig, osig, scl;
                sigmoid_pair<uint16_t, false>(g, sig, osig, scl);
                return s[j] * ((g * sig) * M.acc[2 * i + 1][j][e]);
            });
        } else {
            constexpr int NI = 256 / (32 * (int)sizeof(OutT));
#pragma unroll
            for (int h = 0; h < 4 / NI; ++h)
                epi_out<256, OutT>(wave, row_block<OP>(j), left, J.f0 + wf + 32 * NI * h, (int32_t)P.n_f, out,
                                   (int32_t)P.ldo, OP == kWgrad && P.stream,
                                   [&](int i, int e) { return M.acc[NI * h + i][j][e]; });
        }
    }
}

// The scales of the wave's rows (this lane's in each block of 32).
template <Op OP, int NS>
__device__ __forceinline__ void load_scales(const GroupedArgs& P, const Job& J, int wt, float (&s)[NS]) {
    if constexpr (OP == kFc1) {
        const int lane = threadIdx.x & 63;
        const int32_t row = J.t0 + wt, left = J.t1 - row;
#pragma unroll
        for (int j = 0; j < NS; ++j) {
            const int r = 32 * row_block<OP>(j) + lane % 32;
            s[j] = P.scale != nullptr && r < left ? P.scale[(int64_t)(row + r) * P.scale_stride] : 1.0f;
        }
    }
}

// The spare rows' zeros, row by row.
template <typename OutT>
__device__ __forceinline__ void clear_spare(const GroupedArgs& P) {
    int64_t lo, hi;
    expert_rows(P, P.experts, lo, hi);
    const int64_t vecs = P.n_f * (int)sizeof(OutT) / 16;
    for (int64_t r = lo + blockIdx.x; r < hi; r += gridDim.x) {
        u32x4* p = reinterpret_cast<u32x4*>(static_cast<OutT*>(P.out) + r * P.ldo);
        for (int64_t v = threadIdx.x; v < vecs; v += kThreads) p[v] = u32x4{};
    }
}

template <Op OP, typename OutT>
struct Worker {
    const GroupedArgs& P;
    Schedule sched;
    Operands<OP> src;
    uint32_t i;                                          // number of the next job
    int stored;                                          // rows of the tile before (0: none)
    int32_t last, begin;                                 // wgrad: the last job's expert and its first row

    __device__ __forceinline__ Job next() {
        Job J{};
        if constexpr (OP == kWgrad) {
            const uint32_t per = sched.f_tiles * (uint32_t)((P.n_t + 255) / 256);
            // Experts differ in length: every XCD takes a part of each. The order
            // is dealt to the XCDs in runs of as many tiles as they have workgroups.
            const uint32_t place = (i * kXcds + blockIdx.x % kXcds) * sched.per + sched.j;
            if (place < (uint32_t)P.experts * per) {
                uint32_t tt, ft;
                J.expert = place / per;
                tile_in_expert(place % per, per / sched.f_tiles, sched.f_tiles, tt, ft);
                int64_t lo, hi;
                // (the order's experts do not decrease)
                expert_rows(P, J.expert, lo, hi, last, begin);
                J.lo = __builtin_amdgcn_readfirstlane((int32_t)lo);
                J.len = __builtin_amdgcn_readfirstlane((int32_t)(hi - lo));
                last = J.expert;
                begin = J.lo;
                J.t0 = (int32_t)tt * 256;
                J.t1 = (int32_t)P.n_t;
                J.f0 = (int32_t)ft;
                J.tt = 256;
            }
        } else {
            J = sched.get(P, i);
            J.len = (int32_t)P.n_r;
        }
        J.f0 *= OP == kFc1 ? kFRows / 2 : kFRows;
        ++i;
        return J;
    }
    __device__ __forceinline__ void start(const Job& J) {
        if (J.tt == 0 || J.len == 0) return;
        src.init(P, J);
        if (J.tt == 256) src.template fill<256>();
        else src.template fill<128>();
    }
    // Makes the tile J, whose copies have been started, starts the next one's
    // and stores J's results.
    template <int TT>
    __device__ __forceinline__ Job make(const Job& J) {
        constexpr int kRows = TT / 2;                    // rows per wave
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int wf = (wave % 2) * (OP == kFc1 ? 64 : 128), wt = wave_row<OP>(wave);
        Tile<OP, OutT, TT> M(src, wf, wt);
        if (J.len > 0) M.multiply(stored);
        M.pin();
        const Job N = next();
        float s[kRows / 32];
        load_scales<OP>(P, J, wt, s);
        start(N);
        M.pin();
        store_tile<OP, OutT, TT>(P, J, M, s, wave);
        stored = TT;
        return N;
    }
};

// The grid is a multiple of kXcds workgroups, at most one per CU.
template <Op OP, typename OutT>
__global__ __launch_bounds__(kThreads) void grouped_tile_kernel(GroupedArgs P, uint32_t f_tiles) {
    Worker<OP, OutT> W{P, {}, {}, 0, 0, 0, 0};
    if constexpr (OP == kWgrad) {
        W.sched.f_tiles = f_tiles;
        W.sched.per = gridDim.x / kXcds;
        W.sched.j = blockIdx.x / kXcds;
    } else {
        W.sched.init(P, f_tiles);
    }
    Job J = W.next();
    W.start(J);
    while (J.tt != 0) {
        if constexpr (OP == kWgrad) J = W.template make<256>(J);
        else J = J.tt == 256 ? W.template make<256>(J) : W.template make<128>(J);
    }
    if constexpr (OP != kWgrad) clear_spare<OutT>(P);
}

// ---------------------------------------------------------------------------
// Few tiles: the reduction in parts (see split_parts)
// ---------------------------------------------------------------------------
template <Op OP> constexpr int kSplitRows = OP == kWgrad ? 256 : 128;

// len: of the reduction that parts are planned for (wgrad: a group's mean).
template <Op OP, typename OutT>
__global__ __launch_bounds__(kThreads) void grouped_split_kernel(GroupedArgs P, uint32_t f_tiles,
                                                                 int64_t len, float* ws) {
    constexpr int TT = kSplitRows<OP>, kRows = TT / 2;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if constexpr (OP != kWgrad) clear_spare<OutT>(P);
    SplitTiles<OP, TT, kFRows> T;
    T.init(P, f_tiles);
    const uint32_t parts = split_parts(T.total, len);
    // tiles of one part are neighbours: they share operands in an XCD's L2
    const uint32_t all = T.total * parts, place = place_of(blockIdx.x, all);
    if (place == all) return;
    const uint32_t part = place / T.total, tile = place % T.total;
    Job J = T.get(P, tile);
    split_range(J.len, parts, part, J.r0, J.len);
    if (J.len == 0 && parts > 1) return;                 // (the sum skips such parts)
    Operands<OP> src;
    const int wf = (wave % 2) * (OP == kFc1 ? 64 : 128), wt = wave_row<OP>(wave);
    if (J.len > 0) {
        src.init(P, J);
        src.template fill<TT>();
    }
    Tile<OP, OutT, TT> M(src, wf, wt);
    if (J.len > 0) M.multiply(0);
    M.pin();
    if (parts == 1) {
        float s[kRows / 32];
        load_scales<OP>(P, J, wt, s);
        store_tile<OP, OutT, TT>(P, J, M, s, wave);
        return;
    }
    float* out = ws + ((size_t)tile * parts + part) * (TT * 256) + wt * 256;
    const int32_t left = J.t1 - J.t0 - wt, feats = (int32_t)P.n_f - J.f0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // fc1: gate features in columns 0 to 127, up features from 128
        const int c = OP == kFc1 ? wf + 32 * (i / 2) : wf + 32 * i, up = OP == kFc1 ? 128 * (i % 2) : 0;
#pragma unroll
        for (int j = 0; j < kRows / 32; ++j)
            epi_out<128, float>(wave, row_block<OP>(j), left, c + up, feats + up, out, 256, false,
                                [&](int, int e) { return M.acc[i][j][e]; });
    }
}

}  // namespace grouped_tile

#endif  // SWIGLU_GROUPED_TILE_H
