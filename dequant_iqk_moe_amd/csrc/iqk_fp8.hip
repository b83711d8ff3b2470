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
