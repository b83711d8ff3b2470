// iqk_fp8.hip -- products in 8-bit floating point (e4m3) with a float32 scale
// for each block of 128: the quantization of activations, and
//
//   y[m, o] = sum_b sx[m, b] * sw[o / 128, b] * sum_{i in block b} qx[m, i] * qw[o, i]
//
// over dense rows (a shared expert) or over routed token-expert pairs.
//
// Quantization of one 1 x 128 block: a = max(max |x|, 2^-100), sx = a / 448,
// qx = e4m3(x * (448 / a)), each step rounded to nearest even (the reciprocal
// and the product to float32); 448 is the largest e4m3 value, and the floor
// keeps the reciprocal finite and an all-zero block zero.
//
// The inner sums run on the float16 matrix instructions: every e4m3 value is a
// float16 value, and those instructions sum the products exactly to float32
// rounding (5e-9 of a block's norm measured), where the 8-bit matrix
// instructions align the products of a step to the largest and drop what
// falls below it (1.7e-5 to 5e-5 measured: more than a float32 result may be
// off, less than a 16-bit result resolves).
#include "iqk_device.h"

namespace iqk {
namespace {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kBlock = 128;              // values per scale
constexpr float kE4m3Max = 448.f;
constexpr float kAmaxFloor = 0x1p-100f;

__device__ __forceinline__ uint16_t bf16_bits(float f) {
    const uint32_t u = __float_as_uint(f);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0x7FC0u;
    return (uint16_t)((u + 0x7FFFu + ((u >> 16) & 1u)) >> 16);
}
template <int DT>
__device__ __forceinline__ void store_y(void* y, int64_t i, float v) {
    if constexpr (DT == IQK_F32) ((float*)y)[i] = v;
    if constexpr (DT == IQK_F16) ((_Float16*)y)[i] = (_Float16)v;
    if constexpr (DT == IQK_BF16) ((uint16_t*)y)[i] = bf16_bits(v);
}

// 16 consecutive results, of which `left` are inside the row (`whole`: rows
// of y are multiples of 16 bytes long and aligned)
template <int DT>
__device__ __forceinline__ void store16(void* y, int64_t i, const float (&v)[16], bool whole, int left) {
    if (whole) {
        if constexpr (DT == IQK_F32) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *(float4*)((float*)y + i + 4 * q) = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
        } else {
            uint32_t w[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                if constexpr (DT == IQK_BF16) w[q] = bf16_bits(v[2 * q]) | ((uint32_t)bf16_bits(v[2 * q + 1]) << 16);
                else w[q] = __builtin_bit_cast(uint32_t, f16x2{(_Float16)v[2 * q], (_Float16)v[2 * q + 1]});
            }
            *(uint4*)((uint16_t*)y + i) = make_uint4(w[0], w[1], w[2], w[3]);
            *(uint4*)((uint16_t*)y + i + 8) = make_uint4(w[4], w[5], w[6], w[7]);
        }
    } else {
#pragma unroll
        for (int q = 0; q < 16; ++q)
            if (q < left) store_y<DT>(y, i + q, v[q]);
    }
}

// 8 consecutive activations as float32
template <int DT>
__device__ __forceinline__ void load8(const void* x, int64_t i, float (&v)[8]) {
    if constexpr (DT == IQK_F32) {
        const float4 a = *(const float4*)((const float*)x + i), b = *(const float4*)((const float*)x + i + 4);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
        const uint4 a = *(const uint4*)((const uint16_t*)x + i);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (DT == IQK_BF16) {
                v[2 * j] = __uint_as_float(w[j] << 16);
                v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
            } else {
                const f16x2 h = __builtin_bit_cast(f16x2, w[j]);
                v[2 * j] = (float)h[0];
                v[2 * j + 1] = (float)h[1];
            }
        }
    }
}

// e4m3 codes of 8 values already multiplied by 448 / a
__device__ __forceinline__ uint2 to_e4m3(const float (&v)[8]) {
    uint2 q;
    q.x = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
    q.x = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], q.x, true);
    q.y = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], 0, false);
    q.y = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], q.y, true);
    return q;
}

// float16 values of 8 e4m3 codes (exact; a NaN code gives NaN)
__device__ __forceinline__ f16x8 widen(uint32_t lo, uint32_t hi) {
    const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false);
    const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
    const f16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false);
    const f16x2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
    return f16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// ---------------------------------------------------------------------------
// quantization
// ---------------------------------------------------------------------------

constexpr int kQuantThreads = 256;  // 16 blocks of 128 values

// 16 lanes own one block, 8 consecutive values each (rows are multiples of 16
// values, so a lane's 8 are all inside a row or all past its end)
template <int DT>
__global__ __launch_bounds__(kQuantThreads) void fp8_quantize_kernel(Fp8QuantLaunch p) {
    const int64_t nb = (p.n + kBlock - 1) / kBlock;
    const int64_t i = (int64_t)blockIdx.x * (kQuantThreads / 16) + (threadIdx.x >> 4);
    const int sub = threadIdx.x & 15;
    if (i >= p.rows * nb) return;  // (whole rows of 16 lanes leave together)
    const int64_t row = i / nb, b = i - row * nb;
    const int64_t c = b * kBlock + 8 * sub;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (c < p.n) load8<DT>(p.x, row * p.n + c, v);
    float a = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) a = fmaxf(a, fabsf(v[j]));
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) a = fmaxf(a, __shfl_xor(a, d));
    a = fmaxf(a, kAmaxFloor);
    const float r = kE4m3Max / a;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= r;
    if (c < p.n) *(uint2*)(p.codes + row * p.n + c) = to_e4m3(v);
    if (sub == 0) p.scales[i] = a / kE4m3Max;
}

// ---------------------------------------------------------------------------
// product
// ---------------------------------------------------------------------------

// A workgroup owns 16 weight rows and up to 16 rows of x; its waves take the
// blocks of 128 of the depth in turn and add their partial sums through LDS
// in wave order.  Weights are the A operand and x the B operand of
// v_mfma_f32_16x16x32_f16: lane l holds row (l & 15) of both and, of each
// block, the 16 values at 16 * (l >> 4) and the 16 at 64 + 16 * (l >> 4) (any
// order of the depth will do that is the same in both).  A result lane holds
// four consecutive weight rows of one row of x.
constexpr int kWaves = 8;

struct ProductParams {
    const uint8_t* W;
    const float* sw;
    const uint8_t* x;
    const float* sx;
    int64_t M;
    int E, out, n, k, x_slots;
    const int32_t *ids, *offsets, *perm;
    void* y;
};

template <int YT, bool GROUPED>
__global__ __launch_bounds__(64 * kWaves) void fp8_rows_kernel(ProductParams p) {
    __shared__ float4 red[kWaves][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int li = lane & 15, g = lane >> 4;
    const int row0 = blockIdx.x * 16;
    const int nb = (p.n + kBlock - 1) / kBlock;
    int e = 0;
    int64_t begin = 0, count = p.M;
    if constexpr (GROUPED) {
        e = blockIdx.z;
        begin = p.offsets[e];
        count = p.offsets[e + 1] - begin;
    }
    const int nob = (p.out + kBlock - 1) / kBlock;
    const float* sw = p.sw + ((int64_t)e * nob + row0 / kBlock) * nb;
    const int wr = min(row0 + li, p.out - 1);  // rows past the end repeat the last, their results are dropped
    const uint8_t* wrow = p.W + ((int64_t)e * p.out + wr) * p.n;
    for (int64_t m0 = (int64_t)blockIdx.y * 16; m0 < count; m0 += (int64_t)gridDim.y * 16) {
        const int64_t m = min(m0 + li, count - 1);
        int64_t yrow = m, xr = m;
        if constexpr (GROUPED) {
            yrow = p.perm[begin + m];
            xr = p.x_slots == 1 ? yrow / p.k : yrow;
        }
        const uint8_t* xrow = p.x + xr * p.n;
        const float* sx = p.sx + xr * nb;
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
        for (int b = wave; b < nb; b += kWaves) {
            const int c0 = b * kBlock + 16 * g, c1 = c0 + 64;
            const uint4 z = make_uint4(0, 0, 0, 0);
            const uint4 w0 = c0 < p.n ? *(const uint4*)(wrow + c0) : z, w1 = c1 < p.n ? *(const uint4*)(wrow + c1) : z;
            const uint4 x0 = c0 < p.n ? *(const uint4*)(xrow + c0) : z, x1 = c1 < p.n ? *(const uint4*)(xrow + c1) : z;
            f32x4 d = {0.f, 0.f, 0.f, 0.f};
            d = __builtin_amdgcn_mfma_f32_16x16x32_f16(widen(w0.x, w0.y), widen(x0.x, x0.y), d, 0, 0, 0);
            d = __builtin_amdgcn_mfma_f32_16x16x32_f16(widen(w0.z, w0.w), widen(x0.z, x0.w), d, 0, 0, 0);
            d = __builtin_amdgcn_mfma_f32_16x16x32_f16(widen(w1.x, w1.y), widen(x1.x, x1.y), d, 0, 0, 0);
            d = __builtin_amdgcn_mfma_f32_16x16x32_f16(widen(w1.z, w1.w), widen(x1.z, x1.w), d, 0, 0, 0);
            const float f = sx[b] * sw[b];
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(d[i], f, acc[i]);
        }
        red[wave][lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
        __syncthreads();
        if (wave == 0) {
            float r[4] = {0.f, 0.f, 0.f, 0.f};
            for (int w = 0; w < kWaves; ++w) {
                const float4 v = red[w][lane];
                r[0] += v.x, r[1] += v.y, r[2] += v.z, r[3] += v.w;
            }
            if (m0 + li < count) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int o = row0 + 4 * g + i;
                    if (o < p.out) store_y<YT>(p.y, yrow * p.out + o, r[i]);
                }
            }
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// tiled product
// ---------------------------------------------------------------------------

typedef int i32x8 __attribute__((ext_vector_type(8)));

struct TileParams {
    const uint8_t* W;
    const float* sw;
    const uint8_t* x;
    const float* sx;
    int64_t M;
    int out, n, k, x_slots, E;
    const int32_t *offsets, *perm, *tiles;  // grouped: tiles[e] = 256- or 128-row tiles of x before expert e
    void* y;
};

// 16 bytes per lane from memory straight into LDS: lane l's go to dst + 16 l
// (an LDS address, the same in every lane).  Written as an instruction because the
// compiler takes every later LDS read to depend on the builtin's copy and
// waits for it at once; the kernel waits for its copies before the barrier
// that publishes them.  The instruction has no register result.
__device__ __forceinline__ void lds_copy16(const uint8_t* base, uint32_t off, uint32_t dst) {
    const uint32_t at = __builtin_amdgcn_readfirstlane(dst);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(at), "v"(off), "s"(base) : "memory");
}
__device__ __forceinline__ void lds_copy16(const uint8_t* src, uint32_t dst) {
    const uint32_t at = __builtin_amdgcn_readfirstlane(dst);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(at), "v"(src) : "memory");
}

// Waits for this wave's copies and LDS accesses, then for the other waves'.
__device__ __forceinline__ void publish() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// The 16-byte chunk of a 128-byte tile row is kept at slot chunk ^ key(row),
// so that eight neighbouring lanes of a fragment read eight slots.  A
// fragment's 16 lanes read weight rows 16 (l / 4) + l % 4 + const (keyed by
// the row's bits 0, 1 and 4) and x rows l + const (by its bits 0 to 2).
__device__ __forceinline__ int wkey(int r) { return (r & 3) | ((r >> 2) & 4); }
__device__ __forceinline__ int xkey(int r) { return r & 7; }

template <int TM, int TN, int WM, int WN, int YT, bool GROUPED>
__global__ __launch_bounds__(64 * (TM / WM) * (TN / WN)) void fp8_tile_kernel(TileParams p) {
    constexpr int kNW = (TM / WM) * (TN / WN);  // waves
    constexpr int kI = WN / 16, kJ = WM / 16;   // a wave's tiles of weight rows and of x rows
    constexpr int kRowsPerCopy = 8 * kNW;       // rows one copy instruction of all waves covers
    constexpr int kCW = TN / kRowsPerCopy, kCX = TM / kRowsPerCopy;
    __shared__ uint8_t sh[2][(TN + TM) * 128];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int li = lane & 15, g = lane >> 4;
    const int nb = (p.n + kBlock - 1) / kBlock;
    const int ntn = (p.out + TN - 1) / TN;

    // which tile: the tiles of one XCD (workgroups b with equal b % 8) are neighbours
    int e = 0;
    int64_t m0, count = p.M, begin = 0;
    int n0;
    {
        const int64_t tiles_m = GROUPED ? p.tiles[p.E] : (p.M + TM - 1) / TM;
        const int64_t total = tiles_m * ntn, per = (total + 7) / 8;
        const int64_t id = (int64_t)(blockIdx.x & 7) * per + (blockIdx.x >> 3);
        if ((int64_t)(blockIdx.x >> 3) >= per || id >= total) return;
        if constexpr (GROUPED) {
            const int t = (int)(id / ntn);
            n0 = (int)(id - (int64_t)t * ntn) * TN;
            // the expert of tile t: the last e with tiles[e] <= t, 64 candidates at a time
            int lo = 0, span = p.E;
            while (span > 1) {
                const int step = (span + 63) / 64;
                const int c = lo + lane * step;
                const uint64_t le = __ballot(c < lo + span && p.tiles[c < p.E ? c : p.E] <= t);
                const int last = 63 - __builtin_clzll(le);
                const int nlo = lo + last * step;
                span = min(step, lo + span - nlo);
                lo = nlo;
            }
            e = __builtin_amdgcn_readfirstlane(lo);
            begin = p.offsets[e];
            count = p.offsets[e + 1] - begin;
            m0 = (int64_t)(t - p.tiles[e]) * TM;
        } else {
            // bands of 8 tiles of x by all of the weights' tiles
            const int64_t band = id / (8 * ntn), in = id - band * 8 * ntn;
            const int64_t rows = min((int64_t)8, tiles_m - band * 8);
            m0 = (band * 8 + in % rows) * TM;
            n0 = (int)(in / rows) * TN;
        }
    }

    // copies: lane l of a copy moves slot l & 7 of row l >> 3 of its wave's
    // eight rows; rows past the end repeat the last, their results are dropped
    const int crow = wave * 8 + (lane >> 3);
    const int nob = (p.out + kBlock - 1) / kBlock;
    auto wchunk = [&](int c) { return 16 * ((lane & 7) ^ wkey(c * kRowsPerCopy + crow)); };
    auto xchunk = [&](int c) { return 16 * ((lane & 7) ^ xkey(c * kRowsPerCopy + crow)); };
    // row i of the tile's x rows, as a row of p.x, and as a row of y
    auto pair_of = [&](int i) { return p.perm[begin + min(m0 + i, count - 1)]; };
    auto row_of = [&](int i) -> int64_t {
        if constexpr (GROUPED) return p.x_slots == 1 ? pair_of(i) / p.k : pair_of(i);
        else return min(m0 + i, count - 1);
    };
    const uint8_t* wbase = p.W + ((int64_t)e * p.out + n0) * p.n;
    const uint8_t* xbase = GROUPED ? p.x : p.x + m0 * p.n;  // (dense: offsets inside the tile fit 32 bits)
    uint32_t woff[kCW], xoff[kCX];
    const uint8_t* xsrc[kCX];
#pragma unroll
    for (int c = 0; c < kCW; ++c)
        woff[c] = (uint32_t)(min(c * kRowsPerCopy + crow, p.out - 1 - n0) * p.n + wchunk(c));
#pragma unroll
    for (int c = 0; c < kCX; ++c) {
        if constexpr (GROUPED) xsrc[c] = p.x + row_of(c * kRowsPerCopy + crow) * p.n + xchunk(c);
        else xoff[c] = (uint32_t)((int)(row_of(c * kRowsPerCopy + crow) - m0) * p.n + xchunk(c));
    }
    auto copy_w = [&](int c, int k0, uint32_t d) { lds_copy16(wbase + k0, woff[c], d); };
    auto copy_x = [&](int c, int k0, uint32_t d) {
        if constexpr (GROUPED) lds_copy16(xsrc[c] + k0, d);
        else lds_copy16(xbase + k0, xoff[c], d);
    };
    const uint32_t sh0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)&sh[0][0];
    auto copy_block = [&](int b) {
        const int k0 = b * kBlock;
        const uint32_t at = (b & 1) * (TN + TM) * 128 + wave * 1024;
        if (k0 + kBlock <= p.n) {
#pragma unroll
            for (int c = 0; c < kCW; ++c) copy_w(c, k0, sh0 + at + c * kRowsPerCopy * 128);
#pragma unroll
            for (int c = 0; c < kCX; ++c) copy_x(c, k0, sh0 + at + (TN + c * kRowsPerCopy) * 128);
        } else {  // the partial last block: chunks past the depth are zero
#pragma unroll
            for (int c = 0; c < kCW; ++c) {
                const uint32_t d = at + c * kRowsPerCopy * 128;
                if (k0 + wchunk(c) < p.n) copy_w(c, k0, sh0 + d);
                else *(uint4*)(&sh[0][0] + d + lane * 16) = make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int c = 0; c < kCX; ++c) {
                const uint32_t d = at + (TN + c * kRowsPerCopy) * 128;
                if (k0 + xchunk(c) < p.n) copy_x(c, k0, sh0 + d);
                else *(uint4*)(&sh[0][0] + d + lane * 16) = make_uint4(0, 0, 0, 0);
            }
        }
    };

    const int wn = (wave % (TN / WN)) * WN, wm = (wave / (TN / WN)) * WM;  // this wave's part of the tile
    // scales: one per 128 weight rows (a wave's rows lie in one block), one per row of x
    const float* sw = p.sw + ((int64_t)e * nob + min((n0 + wn) / kBlock, nob - 1)) * nb;
    // (a vector load: a scalar load in flight would make every wait for an LDS read a wait for all of them)
    uint32_t swo = 0;
    asm("" : "+v"(swo));
    const float* sx = GROUPED ? p.sx : p.sx + m0 * nb;
    using Offset = std::conditional_t<GROUPED, int64_t, uint32_t>;
    Offset sxo[kJ];
#pragma unroll
    for (int j = 0; j < kJ; ++j) sxo[j] = (Offset)((row_of(wm + 16 * j + li) - (GROUPED ? 0 : m0)) * nb);

    f32x4 acc[kI][kJ];
#pragma unroll
    for (int i = 0; i < kI; ++i)
#pragma unroll
        for (int j = 0; j < kJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    // fragment rows: lane li of tile i reads weight row 64 (i / 4) + 16 (li / 4) + 4 (i % 4) + li % 4, so that a
    // result lane's four rows of four neighbouring tiles are 16 consecutive rows
    const int arow = wn + 16 * (li >> 2) + (li & 3);
    const int brow = wm + li;
    const int aoff = arow * 128 + 16 * (g ^ wkey(16 * (li >> 2) + (li & 3)));
    const int boff = (TN + brow) * 128 + 16 * (g ^ xkey(li));
    auto frag = [&](const uint8_t* s, int off) {
        const uint4 a = *(const uint4*)(s + off), b = *(const uint4*)(s + (off ^ 64));
        return i32x8{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
    };

    // Instruction t = i kJ + j of a block multiplies tile row i by x tile j.  Its product is added to the sums two
    // instructions later (kLag: it is done by then), and a tile row is read two rows before its first use.
    constexpr int kLag = 2, kRing = 4, kT = kI * kJ;
    static_assert(kT % kRing == 0, "a block's first products follow the last block's in the ring");
    float sxn[kJ], swn, f[kJ], fp[kJ];
    f32x4 d[kRing];
#pragma unroll
    for (int j = 0; j < kJ; ++j) fp[j] = 0.f;
#pragma unroll
    for (int t = 0; t < kRing; ++t) d[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto add = [&](int t, const float* w) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
            acc[t / kJ][t % kJ][q] = __builtin_fmaf(d[t % kRing][q], w[t % kJ], acc[t / kJ][t % kJ][q]);
    };
copy_block(0);
#pragma unroll
    for (int j = 0; j < kJ; ++j) sxn[j] = sx[sxo[j]];
    swn = sw[swo];
    publish();
    for (int b = 0; b < nb; ++b) {
        const uint8_t* cur = sh[b & 1];
#pragma unroll
        for (int j = 0; j < kJ; ++j) f[j] = sxn[j] * swn;
        if (b + 1 < nb) {
            copy_block(b + 1);
#pragma unroll
            for (int j = 0; j < kJ; ++j) sxn[j] = sx[sxo[j] + (b + 1)];
            swn = sw[swo + (b + 1)];
        }
        // (the key's bits are those of the row inside its 64: tile rows i and i + 4 are 64 rows apart, i and i + 1
        // four rows, which no key bit looks at)
        auto afrag = [&](int i) { return frag(cur, aoff + (i >> 2) * 8192 + (i & 3) * 512); };
        i32x8 af[3], bf[kJ];
        af[0] = afrag(0);
        bf[0] = frag(cur, boff);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 1; j < kJ; ++j) {
            bf[j] = frag(cur, boff + j * 2048);
            __builtin_amdgcn_sched_barrier(0);
        }
        af[1] = afrag(1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < kI; ++i) {
            if (i + 2 < kI) af[(i + 2) % 3] = afrag(i + 2);
#pragma unroll
            for (int j = 0; j < kJ; ++j) {
                const int t = i * kJ + j;
                const f32x4 r = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    af[i % 3], bf[j], f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0x7F7F7F7F, 0, 0x7F7F7F7F);
                __builtin_amdgcn_sched_barrier(0);
                if (t >= kLag) add(t - kLag, f);
                else add(kT - kLag + t, fp);
                d[t % kRing] = r;
                __builtin_amdgcn_sched_barrier(0);
            }
        }
#pragma unroll
        for (int j = 0; j < kJ; ++j) fp[j] = f[j];
        publish();
    }
#pragma unroll
    for (int t = kT - kLag; t < kT; ++t) add(t, fp);

    // result lane (li, g) holds, of x row 16 j + li, weight rows 64 (i / 4) + 16 g + 4 (i % 4) + q
    const bool whole = (p.out & 15) == 0 && ((uintptr_t)p.y & 15) == 0;
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
        const int i = wm + 16 * j + li;
        if (m0 + i >= count) continue;
        int64_t yrow = m0 + i;
        if constexpr (GROUPED) yrow = pair_of(i);
#pragma unroll
        for (int h = 0; h < kI / 4; ++h) {
            const int o = n0 + wn + 64 * h + 16 * g;
            if (o >= p.out) continue;
            float v[16];
#pragma unroll
            for (int q = 0; q < 16; ++q) v[q] = acc[4 * h + (q >> 2)][j][q & 3];
            store16<YT>(p.y, yrow * p.out + o, v, whole, p.out - o);
        }
    }
}

template <class F>
void by_y(int dt, F f) {
    if (dt == IQK_F32) f(std::integral_constant<int, IQK_F32>{});
    else if (dt == IQK_F16) f(std::integral_constant<int, IQK_F16>{});
    else f(std::integral_constant<int, IQK_BF16>{});
}

}  // namespace

hipError_t launch_fp8_quantize(const Fp8QuantLaunch& a, hipStream_t s) {
    const int64_t blocks128 = a.rows * ((a.n + kBlock - 1) / kBlock);
    const int64_t per = kQuantThreads / 16;
    const dim3 grid((unsigned)((blocks128 + per - 1) / per));
    by_y(a.x_dtype, [&](auto dt) {
        hipLaunchKernelGGL((fp8_quantize_kernel<decltype(dt)::value>), grid, dim3(kQuantThreads), 0, s, a);
    });
    return hipGetLastError();
}

hipError_t launch_fp8_product(const Fp8Launch& a, hipStream_t s) {
    ProductParams p{a.codes, a.scales, (const uint8_t*)a.x, a.x_scales, a.M, (int)a.E, (int)a.out, (int)a.n,
                    a.k, a.x_slots, a.ids, a.offsets, a.perm, a.y};
    if (!a.offsets && a.y_dtype != IQK_F32 && a.M > 32) {
        TileParams t{a.codes, a.scales, (const uint8_t*)a.x, a.x_scales, a.M, (int)a.out, (int)a.n, a.k, a.x_slots, 1,
                     nullptr, nullptr, nullptr, a.y};
        const int64_t big = ((a.M + 255) / 256) * ((a.out + 255) / 256);
        by_y(a.y_dtype, [&](auto yt) {
            constexpr int YT = decltype(yt)::value;
            if constexpr (YT != IQK_F32) {
                if (big >= 160) {
                    hipLaunchKernelGGL((fp8_tile_kernel<256, 256, 64, 128, YT, false>), dim3((unsigned)((big + 7) / 8 * 8)),
                                       dim3(512), 0, s, t);
                } else {
                    const int64_t tiles = ((a.M + 127) / 128) * ((a.out + 127) / 128);
                    hipLaunchKernelGGL((fp8_tile_kernel<128, 128, 64, 64, YT, false>), dim3((unsigned)((tiles + 7) / 8 * 8)),
                                       dim3(256), 0, s, t);
                }
            }
        });
        return hipGetLastError();
    }
    const unsigned gx = (unsigned)((a.out + 15) / 16);
    by_y(a.y_dtype, [&](auto yt) {
        constexpr int YT = decltype(yt)::value;
        if (a.offsets) {
            hipLaunchKernelGGL((fp8_rows_kernel<YT, true>), dim3(gx, 1, (unsigned)a.E), dim3(64 * kWaves), 0, s, p);
        } else {
            const unsigned gy = (unsigned)std::min<int64_t>((a.M + 15) / 16, 65535);
            hipLaunchKernelGGL((fp8_rows_kernel<YT, false>), dim3(gx, gy), dim3(64 * kWaves), 0, s, p);
        }
    });
    return hipGetLastError();
}

}  // namespace iqk
