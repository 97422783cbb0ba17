// SwiGLU with its input kept in 8 bits for the backward pass, for AMD MI355X
// (gfx950), with the C ABI in include/swiglu_gateup.h.
//
// What is computed: the forward reads x = [g | u] of shape [rows, 2n] once and
// writes y = s silu(g) u together with x in 8 bits: every block of 32 columns
// of one half of a row becomes 32 e4m3 values q and one scale byte b with
// x ~ q 2^(b - 127). b is the smallest value >= 1 whose scale brings the
// block's largest finite magnitude to 448 (the largest e4m3 value) or below,
// so no value saturates and each within 2^-13 of the block's largest is kept to 4
// significant bits (smaller ones may fall in e4m3's subnormal range: steps of 2^-9
// scales). The backward reads q and b in x's place: per column 2 + 2/32 bytes instead
// of 4 (bf16) or 8 (fp32).
//
// Design. As in the plain SwiGLU kernels the op is a stream: every lane owns
// one 16-byte vector of x's gate half and the one of its up half. A block of 32
// columns is 4 lanes (bf16) or 8 (fp32), so its maximum takes two or three
// lane exchanges within a quad or half row (DPP, no LDS). The scale is found
// from the maximum's bits: with exponent field E and mantissa m, b = E - 8, or
// E - 7 where 1.m > 1.75 = 448 / 256. Multiplying by 2^(127 - b) is exact, so
// the hardware conversion's rounding (nearest even) is the only one.
#include "swiglu_device.h"

namespace {

using namespace swiglu_impl;

constexpr int kQBlock = 32;                 // columns that share a scale

// Lanes per row are counted in vectors of 16 bytes of x, whole blocks of 32
// columns: 4 lanes of 8 bf16 or 8 lanes of 4 fp32. A block's lanes are an
// aligned group of 4 or 8 lanes of one wave, in the flat grid too.
template <typename T> constexpr int kVec = 16 / (int)sizeof(T);
template <typename T> constexpr int kGroup = kQBlock / kVec<T>;

// Vectors at any element alignment: gfx950 loads and stores whole vectors
// from unaligned addresses, and an access that is aligned costs no more for
// being declared so.
template <int BYTES, int ALIGN> struct RawAt {
    typedef typename Raw<BYTES>::type type __attribute__((aligned(ALIGN)));
};

// VEC elements of T at p, of which the first `count` exist (the rest read as
// zero), widened to fp32.
template <typename T, int VEC>
__device__ __forceinline__ void load_part(const T* p, int count, float (&f)[VEC]) {
    typedef typename RawAt<VEC * sizeof(T), sizeof(T)>::type R;
    uint32_t w[VEC * sizeof(T) / 4];
    if (count >= VEC) {
        const typename Vec<T, VEC>::R r = __builtin_nontemporal_load(reinterpret_cast<const R*>(p));
        __builtin_memcpy(w, &r, sizeof(r));
    } else {
        T e[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) e[i] = i < count ? p[i] : T(0);
        __builtin_memcpy(w, e, sizeof(w));
    }
    if constexpr (sizeof(T) == 4) {
        __builtin_memcpy(f, w, sizeof(w));
    } else {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}

template <typename T, int VEC>
__device__ __forceinline__ void store_part(T* p, int count, const float (&f)[VEC]) {
    typedef typename RawAt<VEC * sizeof(T), sizeof(T)>::type R;
    typename Vec<T, VEC>::R r;
    if constexpr (sizeof(T) == 4) {
        __builtin_memcpy(&r, f, sizeof(r));
    } else {
        uint32_t w[VEC / 2];
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
            f32x2 pr = {f[2 * i], f[2 * i + 1]};
            w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(pr, bf16x2));
        }
        __builtin_memcpy(&r, w, sizeof(r));
    }
    if (count >= VEC) {
        __builtin_nontemporal_store(r, reinterpret_cast<R*>(p));
    } else {
        T e[VEC];
        __builtin_memcpy(e, &r, sizeof(r));
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (i < count) p[i] = e[i];
    }
}

// Largest value over the lane's block (aligned groups of 4 or 8 lanes).
template <int GROUP>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
    auto with = [&](uint32_t o) { v = o > v ? o : v; };
    with(__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xf, 0xf, true));      // lanes 1 0 3 2
    with(__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xf, 0xf, true));      // lanes 2 3 0 1
    if constexpr (GROUP == 8)
        with(__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xf, 0xf, true)); // mirrored in 8
    return v;
}

// The block's scale byte from the bits of its largest magnitudes. Infinities
// and NaN take no part in it (they are kept as NaN): they would leave no
// finite scale for the block's other values.
template <int VEC, int GROUP>
__device__ __forceinline__ uint32_t scale_byte(const float (&v)[VEC]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        const uint32_t a = __float_as_uint(v[i]) & 0x7fffffffu;
        m = a > m ? a : m;
    }
    m = group_max<GROUP>(m);
    if (m >= 0x7f800000u) {                 // rare; the block's lanes agree on it
        m = 0;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const uint32_t a = __float_as_uint(v[i]) & 0x7fffffffu;
            m = a < 0x7f800000u && a > m ? a : m;
        }
        m = group_max<GROUP>(m);
    }
    // 448 = 1.75 2^8: exponent field E takes b = E - 8, one more past 1.75
    const int b = (int)(m >> 23) - 8 + ((m & 0x7fffffu) > 0x600000u ? 1 : 0);
    return (uint32_t)(b < 1 ? 1 : b);
}

// Quantises the lane's VEC values with scale byte b and stores `count` of them.
template <int VEC>
__device__ __forceinline__ void store_q(uint8_t* p, int count, const float (&v)[VEC], uint32_t b) {
    const float inv = __uint_as_float((254u - b) << 23);       // 2^(127 - b); b is in [1, 247]
    uint32_t w[VEC / 4];
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) {
        int r = 0;
        r = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i] * inv, v[4 * i + 1] * inv, r, false);
        r = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2] * inv, v[4 * i + 3] * inv, r, true);
        w[i] = (uint32_t)r;
    }
    if (count >= VEC) {
        typedef typename RawAt<VEC, 1>::type R;
        typename Raw<VEC>::type r;
        __builtin_memcpy(&r, w, sizeof(r));
        __builtin_nontemporal_store(r, reinterpret_cast<R*>(p));
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (i < count) p[i] = (uint8_t)(w[i / 4] >> (8 * (i % 4)));
    }
}

// VEC values at p with scale byte b (0: 2^-127; 255, which the forward never
// writes, reads as NaN); past the fp32 range: its largest value.
template <int VEC>
__device__ __forceinline__ void load_q(const uint8_t* p, int count, uint32_t b, float (&v)[VEC]) {
    uint32_t w[VEC / 4];
    if (count >= VEC) {
        typedef typename RawAt<VEC, 1>::type R;
        const typename Raw<VEC>::type r = __builtin_nontemporal_load(reinterpret_cast<const R*>(p));
        __builtin_memcpy(w, &r, sizeof(r));
    } else {
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i) w[i] = 0;
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (i < count) w[i / 4] |= (uint32_t)p[i] << (8 * (i % 4));
    }
    uint32_t sb = b << 23;
    sb = b == 0 ? 0x00400000u : sb;
    sb = b == 255 ? 0x7fc00000u : sb;
    const float s = __uint_as_float(sb);
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) {
        const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false);
        const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
        v[4 * i] = lo.x * s;
        v[4 * i + 1] = lo.y * s;
        v[4 * i + 2] = hi.x * s;
        v[4 * i + 3] = hi.y * s;
    }
    if (b >= 247) {
        // A value within a rounding of 2^128 is kept as 2^128 itself (256 at
        // b = 247): it reads as the largest fp32 value, not as infinity,
        // which would make NaN of gradients that are finite.
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (__builtin_fabsf(v[i]) == __builtin_inff()) v[i] = __builtin_copysignf(__FLT_MAX__, v[i]);
    }
}

template <typename T, bool WIDE>
__global__ __launch_bounds__(kBlock) void ckpt8_fwd_kernel(
    const T* __restrict__ x, int64_t xs, const float* __restrict__ scale, int64_t ss,
    T* __restrict__ y, int64_t ys, uint8_t* __restrict__ q, int64_t qst, uint8_t* __restrict__ qs,
    int64_t qss, int64_t n, Geom G) {
    constexpr int VEC = kVec<T>, GROUP = kGroup<T>;
    int64_t row;
    uint32_t col;
    if (!locate<WIDE>(G, row, col)) return;           // whole blocks leave together
    const int64_t c = (int64_t)col * VEC;
    const int64_t left = n - c;
    const int count = left >= VEC ? VEC : left > 0 ? (int)left : 0;
    const T* xr = x + row * xs + c;
    float g[VEC], u[VEC], out[VEC];
    load_part<T, VEC>(xr, count, g);
    load_part<T, VEC>(xr + n, count, u);
    const float s = scale ? scale[row * ss] : 1.0f;
    const uint32_t bg = scale_byte<VEC, GROUP>(g), bu = scale_byte<VEC, GROUP>(u);
    uint8_t* qr = q + row * qst + c;
    store_q<VEC>(qr, count, g, bg);
    store_q<VEC>(qr + n, count, u, bu);
    if (col % GROUP == 0) {
        // single bytes of lines that other lanes complete: left to L2 to merge
        const int64_t nb = G.nv / GROUP, blk = col / GROUP;
        qs[row * qss + blk] = (uint8_t)bg;
        qs[row * qss + nb + blk] = (uint8_t)bu;
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        float sig, osig, scl;
        sigmoid_pair<T, false>(g[i], sig, osig, scl);
        out[i] = (s * ((g[i] * sig) * u[i])) * scl;
    }
    store_part<T, VEC>(y + row * ys + c, count, out);
}

struct BwdArgs {
    const void* dy;
    const uint8_t* q;
    const uint8_t* qs;
    const float* scale;      // NULL: 1
    void* dx;
    void* y;                 // NULL: not wanted
    float* ds;               // NULL: not wanted
    int64_t dys, qst, qss, ss, dxs, ys, dss;
    int64_t n;
};

// One vector of one row: writes dx (and y) and returns sum dy silu(g) u.
template <typename T>
__device__ __forceinline__ float bwd_vector(const BwdArgs& P, int64_t row, uint32_t col, uint32_t nv,
                                            float s) {
    constexpr int VEC = kVec<T>, GROUP = kGroup<T>;
    const int64_t c = (int64_t)col * VEC;
    const int64_t left = P.n - c;
    const int count = left >= VEC ? VEC : left > 0 ? (int)left : 0;
    const int64_t nb = nv / GROUP, blk = col / GROUP;
    const uint32_t bg = P.qs[row * P.qss + blk], bu = P.qs[row * P.qss + nb + blk];
    const uint8_t* qr = P.q + row * P.qst + c;
    float g[VEC], u[VEC], d[VEC], dg[VEC], du[VEC], yv[VEC];
    load_part<T, VEC>(static_cast<const T*>(P.dy) + row * P.dys + c, count, d);
    load_q<VEC>(qr, count, bg, g);
    load_q<VEC>(qr + P.n, count, bu, u);
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        float sig, osig, scl;
        sigmoid_pair<T, true>(g[i], sig, osig, scl);
        const float h = h_factor<T>(g[i], osig);
        const float silu = g[i] * sig;                         // times scl
        const float t = s * d[i];
        du[i] = (t * silu) * scl;
        dg[i] = ((t * u[i]) * (sig * h)) * scl;
        const float a = (silu * u[i]) * scl;
        yv[i] = s * a;
        if (i < count) dot = __builtin_fmaf(d[i], a, dot);
    }
    T* dxr = static_cast<T*>(P.dx) + row * P.dxs + c;
    store_part<T, VEC>(dxr, count, dg);
    store_part<T, VEC>(dxr + P.n, count, du);
    if (P.y != nullptr) store_part<T, VEC>(static_cast<T*>(P.y) + row * P.ys + c, count, yv);
    return dot;
}

// Without ds: a one-shot grid of vectors, as the forward.
template <typename T, bool WIDE>
__global__ __launch_bounds__(kBlock) void ckpt8_bwd_kernel(BwdArgs P, Geom G) {
    int64_t row;
    uint32_t col;
    if (!locate<WIDE>(G, row, col)) return;
    bwd_vector<T>(P, row, col, G.nv, P.scale ? P.scale[row * P.ss] : 1.0f);
}

// With ds the products of a row are added in a fixed order: a lane's, then the
// lanes' pairwise, then the waves' in order.
template <int TEAM>
__device__ __forceinline__ float team_sum(float sum, float* part) {
#pragma unroll
    for (int m = 1; m < (TEAM < 64 ? TEAM : 64); m *= 2) sum += __shfl_xor(sum, m, 64);
    if constexpr (TEAM > 64) {
        if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = sum;
        __syncthreads();
        const float* p = part + threadIdx.x / TEAM * (TEAM / 64);
        sum = p[0];
#pragma unroll
        for (int w = 1; w < TEAM / 64; ++w) sum += p[w];
    }
    return sum;
}

// Rows of at most TEAM vectors: one-shot, TEAM lanes a row. (A workgroup that walks
// a row keeps fewer loads in flight: 8192 x 32768 bf16 488 us walked, 427 in one
// shot with partial sums, 423 without ds; 4096 x 11003 fp32 201, 147 and 144.)
template <typename T, int TEAM>
__global__ __launch_bounds__(TEAM > kBlock ? TEAM : kBlock) void ckpt8_bwd_ds_kernel(BwdArgs P, Geom G) {
    constexpr int kThreads = TEAM > kBlock ? TEAM : kBlock, kRows = kThreads / TEAM;
    __shared__ float part[kThreads / 64];
    const uint32_t col = threadIdx.x % TEAM;
    const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / TEAM;
    float sum = 0.0f;
    if (row < G.rows && col < G.nv) sum = bwd_vector<T>(P, row, col, G.nv, P.scale[row * P.ss]);
    sum = team_sum<TEAM>(sum, part);
    if (row < G.rows && col == 0) P.ds[row * P.dss] = sum;
}

// Longer rows: a workgroup's 256 vectors give one partial sum of their row, which a
// second launch adds in order.
template <typename T>
__global__ __launch_bounds__(kBlock) void ckpt8_bwd_part_kernel(BwdArgs P, Geom G, float* parts) {
    __shared__ float part[kBlock / 64];
    int64_t row;
    uint32_t col;
    float sum = 0.0f;
    if (locate<true>(G, row, col)) sum = bwd_vector<T>(P, row, col, G.nv, P.scale[row * P.ss]);
    sum = team_sum<kBlock>(sum, part);
    if (threadIdx.x == 0) parts[(size_t)blockIdx.y * gridDim.x + blockIdx.x] = sum;
}

__global__ __launch_bounds__(kBlock) void ckpt8_ds_sum_kernel(const float* parts, uint32_t tiles,
                                                              int64_t rows, float* ds, int64_t dss) {
    const int64_t row = (int64_t)blockIdx.x * kBlock + threadIdx.x;
    if (row >= rows) return;
    const float* p = parts + row * tiles;
    float sum = p[0];
    for (uint32_t t = 1; t < tiles; ++t) sum += p[t];
    ds[row * dss] = sum;
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

// Vectors per row, whole blocks of 32 columns.
template <typename T>
Plan ckpt_plan(int64_t n) {
    return make_plan((n + kQBlock - 1) / kQBlock * kQBlock, kVec<T>);
}

struct Region {
    Operand o;               // in bytes
    int64_t rows, width;     // width in bytes
};

Region region(const void* p, int64_t stride, int64_t rows, int64_t width, int64_t esz) {
    return {Operand{p, stride * esz}, rows, width * esz};
}

bool apart(const Region& a, const Region& b) {
    if (a.o.p == nullptr || b.o.p == nullptr) return true;
    return !views_overlap(a.o, a.width, b.o, b.width, a.rows, 1);
}

int64_t esize(swiglu_dtype d) { return d == SWIGLU_DTYPE_F32 ? 4 : 2; }

swiglu_status check_common(int64_t rows, int64_t n, swiglu_dtype dtype, int64_t q_stride,
                           int64_t qs_stride, const void* scale, int64_t scale_stride) {
    swiglu_status st = check_shape(rows, n, dtype);
    if (st != SWIGLU_OK) return st;
    if ((st = check_operand(rows, q_stride, 2 * n, 1)) != SWIGLU_OK) return st;
    if ((st = check_operand(rows, qs_stride, 2 * ((n + kQBlock - 1) / kQBlock), 1)) != SWIGLU_OK)
        return st;
    if (scale != nullptr) return check_operand(rows, scale_stride, 1, 4);
    return SWIGLU_OK;
}

template <typename T>
swiglu_status fwd(const void* x, int64_t xs, const float* scale, int64_t ss, void* y, int64_t ys,
                  uint8_t* q, int64_t qst, uint8_t* qs, int64_t qss, int64_t rows, int64_t n,
                  hipStream_t stream) {
    const Plan P = ckpt_plan<T>(n);
    Geom G;
    G.nv = P.nv;
    G.inv_nv = 1.0 / (double)P.nv;
    for (int64_t r0 = 0; r0 < rows; r0 += P.rows_per_launch) {
        G.rows = rows - r0 < P.rows_per_launch ? rows - r0 : P.rows_per_launch;
        const dim3 grid = P.wide ? dim3(P.tiles, (uint32_t)G.rows)
                                 : dim3(swiglu_host::flat_blocks(G.rows, P.nv, kBlock), 1);
        auto k = P.wide ? &ckpt8_fwd_kernel<T, true> : &ckpt8_fwd_kernel<T, false>;
        const T* xp = static_cast<const T*>(x) + r0 * xs;
        T* yp = static_cast<T*>(y) + r0 * ys;
        const float* sp = scale ? scale + r0 * ss : nullptr;
        uint8_t* qp = q + r0 * qst;
        uint8_t* qsp = qs + r0 * qss;
        void* args[] = {&xp, &xs, &sp, &ss, &yp, &ys, &qp, &qst, &qsp, &qss, &n, &G};
        if (hipLaunchKernel(reinterpret_cast<const void*>(k), grid, dim3(kBlock), args, 0, stream) !=
            hipSuccess)
            return SWIGLU_ERR_HIP;
    }
    return SWIGLU_OK;
}

// Vectors of a row whose sum needs no partials. 512 lanes a row against partial sums:
// 16384 x 4096 bf16 111 us both; 1024 lanes, 16384 x 4096 fp32: 203 and 193.
constexpr uint32_t kMaxTeam = 512;

template <typename T>
size_t bwd_workspace(int64_t rows, int64_t n) {
    const Plan P = ckpt_plan<T>(n);
    return P.nv > kMaxTeam ? (size_t)rows * P.tiles * sizeof(float) : 0;
}

template <typename T, int TEAM>
const void* team_kernel(int& team) {
    team = TEAM;
    return reinterpret_cast<const void*>(&ckpt8_bwd_ds_kernel<T, TEAM>);
}

template <typename T>
swiglu_status bwd(const BwdArgs& A, int64_t rows, float* parts, hipStream_t stream) {
    const Plan P = ckpt_plan<T>(A.n);
    Geom G;
    G.nv = P.nv;
    G.inv_nv = 1.0 / (double)P.nv;
    const bool teams = A.ds != nullptr && P.nv <= kMaxTeam;
    int team = 0;
    const void* k;
    if (teams) {
        k = P.nv > 256   ? team_kernel<T, 512>(team)
            : P.nv > 128 ? team_kernel<T, 256>(team)
            : P.nv > 64  ? team_kernel<T, 128>(team)
            : P.nv > 32  ? team_kernel<T, 64>(team)
            : P.nv > 16  ? team_kernel<T, 32>(team)
                         : team_kernel<T, 16>(team);
    } else if (A.ds != nullptr) {
        k = reinterpret_cast<const void*>(&ckpt8_bwd_part_kernel<T>);
    } else {
        k = P.wide ? reinterpret_cast<const void*>(&ckpt8_bwd_kernel<T, true>)
                   : reinterpret_cast<const void*>(&ckpt8_bwd_kernel<T, false>);
    }
    const int threads = team > kBlock ? team : kBlock;
    const int64_t per = teams ? threads / team : 1;              // rows per workgroup
    const int64_t per_launch = teams ? per << 20 : P.rows_per_launch;
    for (int64_t r0 = 0; r0 < rows; r0 += per_launch) {
        G.rows = rows - r0 < per_launch ? rows - r0 : per_launch;
        BwdArgs B = A;
        B.dy = static_cast<const T*>(A.dy) + r0 * A.dys;
        B.q = A.q + r0 * A.qst;
        B.qs = A.qs + r0 * A.qss;
        B.scale = A.scale ? A.scale + r0 * A.ss : nullptr;
        B.dx = static_cast<T*>(A.dx) + r0 * A.dxs;
        B.y = A.y ? static_cast<T*>(A.y) + r0 * A.ys : nullptr;
        B.ds = A.ds ? A.ds + r0 * A.dss : nullptr;
        float* pr = parts ? parts + r0 * P.tiles : nullptr;
        const dim3 grid = teams    ? dim3((uint32_t)((G.rows + per - 1) / per), 1)
                          : P.wide ? dim3(P.tiles, (uint32_t)G.rows)
                                   : dim3(swiglu_host::flat_blocks(G.rows, P.nv, kBlock), 1);
        void* args[] = {&B, &G, &pr};                            // (only the partials' kernel takes pr)
        if (hipLaunchKernel(k, grid, dim3(threads), args, 0, stream) != hipSuccess) return SWIGLU_ERR_HIP;
        if (A.ds != nullptr && !teams) {
            uint32_t tiles = P.tiles;
            void* sum[] = {&pr, &tiles, &G.rows, &B.ds, &B.dss};
            if (hipLaunchKernel(reinterpret_cast<const void*>(&ckpt8_ds_sum_kernel),
                                dim3((uint32_t)((G.rows + kBlock - 1) / kBlock)), dim3(kBlock), sum, 0,
                                stream) != hipSuccess)
                return SWIGLU_ERR_HIP;
        }
    }
    return SWIGLU_OK;
}

}  // namespace

extern "C" {

__attribute__((visibility("default"))) swiglu_status swiglu_ckpt8_fwd(
    const void* x, int64_t x_row_stride, const float* scale, int64_t scale_stride, void* y,
    int64_t y_row_stride, void* q, int64_t q_row_stride, void* qs, int64_t qs_row_stride,
    int64_t rows, int64_t n, swiglu_dtype dtype, hipStream_t stream) {
    swiglu_status st = check_common(rows, n, dtype, q_row_stride, qs_row_stride, scale, scale_stride);
    if (st != SWIGLU_OK) return st;
    const int64_t esz = esize(dtype);
    if ((st = check_operand(rows, x_row_stride, 2 * n, esz)) != SWIGLU_OK) return st;
    if ((st = check_operand(rows, y_row_stride, n, esz)) != SWIGLU_OK) return st;
    if (rows == 0 || n == 0) return SWIGLU_OK;
    if (!x || !y || !q || !qs) return SWIGLU_ERR_NULL_POINTER;
    const int64_t nb = (n + kQBlock - 1) / kQBlock;
    const Region rx = region(x, x_row_stride, rows, 2 * n, esz), ry = region(y, y_row_stride, rows, n, esz);
    const Region rq = region(q, q_row_stride, rows, 2 * n, 1), rs = region(qs, qs_row_stride, rows, 2 * nb, 1);
    const Region sc = region(scale, scale_stride, rows, 1, 4);
    if (!apart(ry, rq) || !apart(ry, rs) || !apart(rq, rs)) return SWIGLU_ERR_ALIASING;
    for (const Region& out : {ry, rq, rs})
        if (!apart(out, rx) || !apart(out, sc)) return SWIGLU_ERR_ALIASING;
    uint8_t *qp = static_cast<uint8_t*>(q), *qsp = static_cast<uint8_t*>(qs);
    if (dtype == SWIGLU_DTYPE_BF16)
        return fwd<uint16_t>(x, x_row_stride, scale, scale_stride, y, y_row_stride, qp, q_row_stride,
                             qsp, qs_row_stride, rows, n, stream);
    return fwd<float>(x, x_row_stride, scale, scale_stride, y, y_row_stride, qp, q_row_stride, qsp,
                      qs_row_stride, rows, n, stream);
}

__attribute__((visibility("default"))) size_t swiglu_ckpt8_workspace_size(int64_t rows, int64_t n,
                                                                          swiglu_dtype dtype) {
    if (check_shape(rows, n, dtype) != SWIGLU_OK || rows == 0 || n == 0) return 0;
    return dtype == SWIGLU_DTYPE_BF16 ? bwd_workspace<uint16_t>(rows, n) : bwd_workspace<float>(rows, n);
}

__attribute__((visibility("default"))) swiglu_status swiglu_ckpt8_bwd(
    const void* dy, int64_t dy_row_stride, const void* q, int64_t q_row_stride, const void* qs,
    int64_t qs_row_stride, const float* scale, int64_t scale_stride, void* dx, int64_t dx_row_stride,
    void* y, int64_t y_row_stride, float* dscale, int64_t dscale_stride, void* workspace,
    size_t workspace_bytes, int64_t rows, int64_t n, swiglu_dtype dtype, hipStream_t stream) {
    swiglu_status st = check_common(rows, n, dtype, q_row_stride, qs_row_stride, scale, scale_stride);
    if (st != SWIGLU_OK) return st;
    const int64_t esz = esize(dtype);
    if ((st = check_operand(rows, dy_row_stride, n, esz)) != SWIGLU_OK) return st;
    if ((st = check_operand(rows, dx_row_stride, 2 * n, esz)) != SWIGLU_OK) return st;
    if (y != nullptr && (st = check_operand(rows, y_row_stride, n, esz)) != SWIGLU_OK) return st;
    if (dscale != nullptr && (st = check_operand(rows, dscale_stride, 1, 4)) != SWIGLU_OK) return st;
    if (dscale != nullptr && scale == nullptr) return SWIGLU_ERR_NULL_POINTER;
    if (rows == 0) return SWIGLU_OK;
    if (n == 0 && dscale == nullptr) return SWIGLU_OK;
    if (n > 0 && (!dy || !q || !qs || !dx)) return SWIGLU_ERR_NULL_POINTER;
    const int64_t nb = (n + kQBlock - 1) / kQBlock;
    const Region rdy = region(dy, dy_row_stride, rows, n, esz), rq = region(q, q_row_stride, rows, 2 * n, 1);
    const Region rs = region(qs, qs_row_stride, rows, 2 * nb, 1), sc = region(scale, scale_stride, rows, 1, 4);
    const Region rdx = region(dx, dx_row_stride, rows, 2 * n, esz), ry = region(y, y_row_stride, rows, n, esz);
    const Region rds = region(dscale, dscale_stride, rows, 1, 4);
    if (!apart(rdx, ry) || !apart(rdx, rds) || !apart(ry, rds)) return SWIGLU_ERR_ALIASING;
    for (const Region& out : {rdx, ry, rds})
        for (const Region& in : {rdy, rq, rs, sc})
            if (!apart(out, in)) return SWIGLU_ERR_ALIASING;
    const size_t need = dscale == nullptr ? 0 : swiglu_ckpt8_workspace_size(rows, n, dtype);
    if (need > 0) {
        if (workspace == nullptr || workspace_bytes < need || (uintptr_t)workspace % 16 != 0)
            return SWIGLU_ERR_WORKSPACE;
        const swiglu_host::Span ws{(uintptr_t)workspace, (uintptr_t)workspace + need};
        for (const Region& x : {rdy, rq, rs, sc, rdx, ry, rds})
            if (x.o.p != nullptr && swiglu_host::spans_overlap(ws, swiglu_host::span_of(x.o, x.rows, x.width, 1)))
                return SWIGLU_ERR_ALIASING;
    }
    const BwdArgs A{dy, static_cast<const uint8_t*>(q), static_cast<const uint8_t*>(qs), scale,
                    dx, y, dscale, dy_row_stride, q_row_stride, qs_row_stride, scale_stride,
                    dx_row_stride, y_row_stride, dscale_stride, n};
    float* parts = need > 0 ? static_cast<float*>(workspace) : nullptr;
    return dtype == SWIGLU_DTYPE_BF16 ? bwd<uint16_t>(A, rows, parts, stream)
                                      : bwd<float>(A, rows, parts, stream);
}

}  // extern "C"
