// The products of swiglu_grouped.hip for groups of a few rows (mm, fc1, dgrad), where
// the time is that of reading the weights once.
//
// Design of mm and fc1 (bf16 in, fp32 accumulate, MFMA 16x16x32):
//  * A workgroup of 8 waves makes 16 features (fc1: 16 gate and 16 up features) of
//    up to 32 rows, and the waves share its reduction: each takes every eighth
//    piece of 64 (whole 128-byte lines of 16 weight rows), so that even one token
//    has all CUs reading weights. The eight sums of a value are added in
//    order of the waves through LDS. (16 waves are no faster, not with one
//    workgroup per CU either: 12.5 and 12.0 us for two rows, n = 224, k = 5920. A CU reads
//    about 45 bytes a ns.)
//  * No weight is used by two waves, so fragments are loaded straight from
//    memory into registers, one piece ahead of the MFMAs.
//  * What lies outside (rows, features, the reduction's end) has an offset past
//    the buffer descriptor's range: it reads as zero and costs no traffic. Operands
//    whose rows are not whole, aligned 16-byte vectors (ANY) are loaded as unaligned
//    vectors through pointers (load_chunk).
#ifndef SWIGLU_GROUPED_DIRECT_H
#define SWIGLU_GROUPED_DIRECT_H

namespace grouped_direct {

using namespace swiglu_impl;

typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 512, kWaves = 8;
constexpr int kF = 16;                   // features of a tile
constexpr int kRows = 32;                // rows of a tile
constexpr int kPiece = 64;               // of the reduction
constexpr uint32_t kOutside = 0x80000000u;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const uint16_t* p) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(p), 0, (int)kOutside, 0x00020000);
}
__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0));
}

// Sums of 16 features and 16 MT rows in LDS: a row's values, gate and then up
// for fc1, and 4 more against bank conflicts.
template <Op OP> constexpr int kHalves = OP == kFc1 ? 2 : 1;
template <Op OP> constexpr int kPitch = kF * kHalves<OP> + 4;

// This wave's share of the reduction [0, len) of MT blocks of 16 rows.
template <Op OP, bool ANY, int MT>
__device__ __forceinline__ void make(const GroupedArgs& P, const uint16_t* w, const uint16_t* t,
                                     int32_t feats, int32_t rows, int32_t len, float* sums) {
    constexpr int H = kHalves<OP>;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i16 = lane % 16, g = lane / 16;
    // Offsets of this lane's loads at the reduction's start, kOutside for features and rows
    // that do not exist. ANY, whose strides have no bound that 32 bits would fit, goes by
    // pointers: its offsets are that mark or 0.
    const uint32_t of = i16 >= feats ? kOutside : ANY ? 0 : (uint32_t)(i16 * (int32_t)P.ldf * 2 + g * 16);
    uint32_t ot[MT];
#pragma unroll
    for (int j = 0; j < MT; ++j) {
        const int r = 16 * j + i16;
        ot[j] = r >= rows ? kOutside : ANY ? 0 : (uint32_t)(r * (int32_t)P.ldt * 2 + g * 16);
    }
    const __amdgpu_buffer_rsrc_t rt = buffer(t);
    __amdgpu_buffer_rsrc_t rf[H];
#pragma unroll
    for (int h = 0; h < H; ++h) rf[h] = buffer(w + h * P.up * P.ldf);
    f32x4 acc[H][MT];
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
        for (int j = 0; j < MT; ++j) acc[h][j] = f32x4{};

    struct Piece {
        u32x4 f[H][2], t[MT][2];
    };
    auto load = [&](int32_t k0, Piece& p) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int32_t k = k0 + 32 * s;
            const bool in = k + 8 * g < len;
#pragma unroll
            for (int h = 0; h < H; ++h) {
                if constexpr (ANY)
                    p.f[h][s] = load_chunk(w + (h * P.up + (of == kOutside ? 0 : i16)) * P.ldf + k + 8 * g,
                                           of == kOutside ? 0 : len - k - 8 * g, len >= 8);
                else
                    p.f[h][s] = load16(rf[h], in ? of + (uint32_t)k * 2 : kOutside);
            }
#pragma unroll
            for (int j = 0; j < MT; ++j) {
                if constexpr (ANY)
                    p.t[j][s] = load_chunk(t + (ot[j] == kOutside ? 0 : 16 * j + i16) * P.ldt + k + 8 * g,
                                           ot[j] == kOutside ? 0 : len - k - 8 * g, len >= 8);
                else
                    p.t[j][s] = load16(rt, in ? ot[j] + (uint32_t)k * 2 : kOutside);
            }
        }
    };
    auto multiply = [&](const Piece& p) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
                for (int j = 0; j < MT; ++j)
                    acc[h][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        __builtin_bit_cast(bf16x8, p.f[h][s]), __builtin_bit_cast(bf16x8, p.t[j][s]),
                        acc[h][j], 0, 0, 0);
    };
    // two pieces in turn, each loaded while the other is multiplied
    constexpr int32_t kStride = kWaves * kPiece;
    int32_t k0 = wave * kPiece;
    Piece a, b;
    if (k0 < len) load(k0, a);
    while (k0 < len) {
        if (k0 + kStride < len) load(k0 + kStride, b);
        multiply(a);
        k0 += kStride;
        if (k0 >= len) break;
        if (k0 + kStride < len) load(k0 + kStride, a);
        multiply(b);
        k0 += kStride;
    }
    // Register r of a 16 x 16 tile holds feature 4 (lane / 16) + r and row lane % 16.
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int h = 0; h < H; ++h)
            *reinterpret_cast<f32x4*>(sums + (wave * kRows + 16 * j + i16) * kPitch<OP> + kF * h + 4 * g) =
                acc[h][j];
}

template <Op OP, bool ANY>
__global__ __launch_bounds__(kThreads) void grouped_direct_kernel(GroupedArgs P, uint32_t f_tiles) {
    __shared__ __attribute__((aligned(16))) float sums[kWaves * kRows * kPitch<OP>];
    int64_t expert, lo, hi;
    uint32_t tt, ft;
    if (!find_tile<kRows>(P, f_tiles, expert, lo, hi, tt, ft)) return;
    const int64_t t0 = lo + (int64_t)tt * kRows;
    const int32_t f0 = (int32_t)ft * kF, feats = (int32_t)P.n_f - f0;
    const int32_t rows = (int32_t)(hi - t0);
    const bool spare = expert == P.experts;              // their results are zero
    if (!spare) {
        const uint16_t* w = P.f + expert * P.f_stride + (int64_t)f0 * P.ldf;
        const uint16_t* t = P.t + t0 * P.ldt;
        if (rows <= 16) make<OP, ANY, 1>(P, w, t, feats, rows, (int32_t)P.n_r, sums);
        else make<OP, ANY, 2>(P, w, t, feats, rows, (int32_t)P.n_r, sums);
    }
    __syncthreads();

    // Four features of one row per thread.
    const int r = threadIdx.x / 4, c = threadIdx.x % 4 * 4;
    if (r >= kRows || r >= rows || c >= feats) return;
    f32x4 o = {};
    if (!spare) {
        auto total = [&](int at) {
            const float* p = sums + r * kPitch<OP> + at;
            f32x4 v = *reinterpret_cast<const f32x4*>(p);
#pragma unroll
            for (int q = 1; q < kWaves; ++q)
                v += *reinterpret_cast<const f32x4*>(p + q * kRows * kPitch<OP>);
            return v;
        };
        o = total(c);
        if constexpr (OP == kFc1) {
            const f32x4 u = total(kF + c);
            const float s = P.scale != nullptr ? P.scale[(t0 + r) * P.scale_stride] : 1.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float sig, osig, scl;
                sigmoid_pair<uint16_t, false>(o[e], sig, osig, scl);
                o[e] = s * ((o[e] * sig) * u[e]);
            }
        }
    }
    uint32_t q[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        f32x2 pr = {o[2 * e], o[2 * e + 1]};
        q[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(pr, bf16x2));
    }
    uint16_t* out = static_cast<uint16_t*>(P.out) + (t0 + r) * P.ldo + f0 + c;
    if ((P.ldo | P.n_f) % 4 == 0 && (uintptr_t)P.out % 8 == 0) {     // (the same for all lanes)
        *reinterpret_cast<u32x2*>(out) = u32x2{q[0], q[1]};
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (c + e < feats) out[e] = (uint16_t)(q[e / 2] >> (16 * (e % 2)));
    }
}

// ---------------------------------------------------------------------------
// dgrad: da[r] = dy[r] W_e
// ---------------------------------------------------------------------------
// The weights' rows run along the output here, so their fragments come through
// LDS and its transposing read. A workgroup of 8 waves makes 32 features (64-byte
// pieces of the weights' rows; the workgroup that reads a line's other half is a neighbour on
// the same XCD) of up to 32 rows with MFMA 32x32x16. Each wave takes every eighth
// piece of 64 weight rows and has four stages of LDS of its own: it copies three
// pieces ahead, waits for its own copies only, and meets the others once, to add
// the sums. One k step's fragment is two reads of 4 contiguous rows, 256 bytes: no bank is met
// twice. Whole 16-byte vectors only.
constexpr int kDF = 32;                  // features of a tile
constexpr int kDStage = kPiece * kDF;    // elements of a wave's stage
constexpr int32_t kNever = 1 << 30;      // past every length left, and so are the 64 after it
constexpr int kDAhead = 3;               // pieces copied ahead, one stage less than there are
__shared__ __attribute__((aligned(16))) uint16_t gd_s0[kWaves * kDStage];
__shared__ __attribute__((aligned(16))) uint16_t gd_s1[kWaves * kDStage];
__shared__ __attribute__((aligned(16))) uint16_t gd_s2[kWaves * kDStage];
__shared__ __attribute__((aligned(16))) uint16_t gd_s3[kWaves * kDStage];

template <int S>
__device__ __forceinline__ uint16_t* dgrad_stage() {
    if constexpr (S == 0) return gd_s0;
    else if constexpr (S == 1) return gd_s1;
    else if constexpr (S == 2) return gd_s2;
    else return gd_s3;
}

struct DgradWave {
    static constexpr int kCopies = kDStage * 2 / 1024, kLoads = kPiece / 16;  // per piece
    const uint16_t *w, *t;               // the tile's first weight and first row
    int64_t ldf;
    int32_t len;
    int wave, lane;
    int at;                              // this lane's first element in a stage's fragment reads
    uint32_t ow, ot;                     // this lane's byte offsets in a piece's first copy and load,
    int32_t iw, it;                      // and its reduction indexes there (kNever: outside the operand)
    __amdgpu_buffer_rsrc_t rt;
    f32x16 acc;
    u32x4 v[4][kLoads];                  // the rows' fragments, by stage

    // Starts the copies and loads of piece p, outside the operands past the end.
    template <int S>
    __device__ __forceinline__ void start(int32_t p) {
        // (len is at most 2^30, and p at most 6 past its last piece)
        const int32_t r0 = (p * kWaves + wave) * kPiece, left = len - r0;
        const __amdgpu_buffer_rsrc_t rw = buffer(w + (int64_t)(left > 0 ? r0 : 0) * ldf);
#pragma unroll
        for (int c = 0; c < kCopies; ++c) {
            const uint32_t o = iw + 16 * c < left ? ow + (uint32_t)(16 * c * (int32_t)ldf * 2) : kOutside;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rw, (__attribute__((address_space(3))) void*)(dgrad_stage<S>() + (wave * kDStage + c * 512)), 16,
                (int)o, 0, 0, 0);
        }
#pragma unroll
        for (int s = 0; s < kLoads; ++s)
            v[S][s] = load16(rt, it + 16 * s < left ? ot + (uint32_t)((r0 + 16 * s) * 2) : kOutside);
        __builtin_amdgcn_sched_barrier(0);
    }
    template <int S>
    __device__ __forceinline__ void multiply() {
        // one offset from the array: through longer chains of them the compiler loses
        // which array is read, and waits for the copies to all
        const uint16_t* p = dgrad_stage<S>() + at;
#pragma unroll
        for (int s = 0; s < kLoads; ++s) {
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 16 * s * kDF));
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + (16 * s + 4) * kDF));
            const __attribute__((ext_vector_type(8))) short f =
                __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
            acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, f),
                                                          __builtin_bit_cast(bf16x8, v[S][s]), acc, 0, 0, 0);
        }
    }
    // s_waitcnt: all but the copies and loads of the last `pieces` started, and no
    // LDS read open.
    template <int PIECES>
    static __device__ __forceinline__ void wait() {
        constexpr int n = PIECES * (kCopies + kLoads);
        static_assert(n < 64, "vmcnt range");
        __builtin_amdgcn_s_waitcnt((n & 15) | ((n >> 4) << 14) | (7 << 4));
        asm volatile("" ::: "memory");
    }
    // Piece p in stage S: the copies of the third one after it go to the stage
    // whose reads the last piece's products have waited for.
    template <int S>
    __device__ __forceinline__ void piece(int32_t p) {
        start<(S + kDAhead) % 4>(p + kDAhead);
        wait<kDAhead>();
        multiply<S>();
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
};

__global__ __launch_bounds__(kThreads) void grouped_direct_dgrad_kernel(GroupedArgs P, uint32_t f_tiles) {
    int64_t expert, lo, hi;
    uint32_t tt, ft;
    if (!find_tile<kRows>(P, f_tiles, expert, lo, hi, tt, ft)) return;
    const int64_t t0 = lo + (int64_t)tt * kRows;
    const int32_t f0 = (int32_t)ft * kDF, feats = (int32_t)P.n_f - f0, rows = (int32_t)(hi - t0);
    const bool spare = expert == P.experts;              // their results are zero
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (!spare) {
        DgradWave D;
        D.w = P.f + expert * P.f_stride + f0;
        D.t = P.t + t0 * P.ldt;
        D.ldf = P.ldf;
        D.len = (int32_t)P.n_r;
        D.wave = wave;
        D.lane = lane;
        D.at = wave * kDStage + (8 * (lane / 32) + (lane % 16) / 4) * kDF + 16 * ((lane / 16) & 1) + 4 * (lane % 4);
        D.ow = (uint32_t)(lane / 4 * (int32_t)P.ldf * 2 + lane % 4 * 16);
        D.ot = (uint32_t)(lane % 32 * (int32_t)P.ldt * 2 + lane / 32 * 16);
        D.iw = lane % 4 * 8 < feats ? lane / 4 : kNever;
        D.it = lane % 32 < rows ? 8 * (lane / 32) : kNever;
        D.rt = buffer(D.t);
        D.acc = f32x16{};
        const int32_t pieces = (D.len + kWaves * kPiece - 1) / (kWaves * kPiece);
        D.start<0>(0);
        D.start<1>(1);
        D.start<2>(2);
        for (int32_t p = 0; p < pieces; p += 4) {        // (past the end: zeros)
            D.piece<0>(p);
            D.piece<1>(p + 1);
            D.piece<2>(p + 2);
            D.piece<3>(p + 3);
        }
        D.wait<0>();                                     // no copy may land in the sums
        // Register e holds feature (e % 4) + 8 (e / 4) + 4 (lane / 32) and row lane % 32. A wave's
        // sums take its own first stage; chunks of 4 are permuted within their row by an XOR.
        float* sums = reinterpret_cast<float*>(gd_s0) + wave * (kRows * kDF);
        const int r = lane % 32;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int c = 2 * q + lane / 32;
            *reinterpret_cast<f32x4*>(sums + r * kDF + (c ^ (r & 7)) * 4) =
                f32x4{D.acc[4 * q], D.acc[4 * q + 1], D.acc[4 * q + 2], D.acc[4 * q + 3]};
        }
    }
    __syncthreads();

    // Four features of one row per thread.
    const int r = threadIdx.x / 8, c = threadIdx.x % 8;
    if (r >= kRows || r >= rows || 4 * c >= feats) return;
    f32x4 o = {};
    if (!spare) {
        const float* p = reinterpret_cast<const float*>(gd_s0) + r * kDF + (c ^ (r & 7)) * 4;
        o = *reinterpret_cast<const f32x4*>(p);
#pragma unroll
        for (int q = 1; q < kWaves; ++q) o += *reinterpret_cast<const f32x4*>(p + q * kRows * kDF);
    }
    uint32_t q[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        f32x2 pr = {o[2 * e], o[2 * e + 1]};
        q[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(pr, bf16x2));
    }
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(P.out) + (t0 + r) * P.ldo + f0 + 4 * c) = u32x2{q[0], q[1]};
}

}  // namespace grouped_direct

#endif  // SWIGLU_GROUPED_DIRECT_H
