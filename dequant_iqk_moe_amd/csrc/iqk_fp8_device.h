// iqk_fp8_device.h -- device helpers of the 8-bit products: e4m3 conversions,
// loads of activations and stores of results.
//
//   y[m, o] = sum_b sx[m, b] * sw[o / 128, b] * sum_{i in block b} qx[m, i] * qw[o, i]
//
// Quantization of one 1 x 128 block: a = max(max |x|, 2^-100), sx = a / 448,
// qx = e4m3(x * (448 / a)), each step rounded to nearest even (the reciprocal
// and the product to float32); 448 is the largest e4m3 value, and the floor
// keeps the reciprocal finite and an all-zero block zero.
//
// Sums.  Every e4m3 value is a float16 value, and the float16 matrix
// instructions sum such products exactly to float32 rounding (5e-9 of a
// block's norm measured).  The 8-bit matrix instructions run at nearly twice
// their rate (4290 TFLOP/s against 2413), but cut each product of eight
// consecutive values toward zero to a multiple of 2^(E - 13), E the exponent
// of the largest of the eight: an error below 7 * 2^-13 = 8.6e-4 of that
// product (measured: 2.8e-4 of the sum of the products' magnitudes at worst,
// 1.7e-5 of the norm on normal operands, 8e-5 beside a loud channel).  That
// is below half a unit of bfloat16, 2^-9 and more of a value, and not below
// float16's 2^-12.  So float32 and float16 results are summed on the former
// everywhere, bfloat16 results on the latter where the matrix rate is what
// bounds the product.
#pragma once

#include <type_traits>

#include "iqk_device.h"
#include "iqk_layer.h"

namespace iqk {

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

// 8 consecutive results, of which `left` are inside the row.  Rows of y begin
// wherever their length puts them: vector stores take any address (333 x 4001
// results in tiles of 64: 1 us less than value by value, float32 3).
template <int DT>
__device__ __forceinline__ void store8(void* y, int64_t i, const float (&v)[8], int left) {
    if (left >= 8) {
        if constexpr (DT == IQK_F32) {
            __builtin_memcpy((float*)y + i, v, 32);
        } else {
            uint32_t w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if constexpr (DT == IQK_BF16) w[q] = bf16_bits(v[2 * q]) | ((uint32_t)bf16_bits(v[2 * q + 1]) << 16);
                else w[q] = __builtin_bit_cast(uint32_t, f16x2{(_Float16)v[2 * q], (_Float16)v[2 * q + 1]});
            }
            __builtin_memcpy((uint16_t*)y + i, w, 16);
        }
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q)
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


// max(largest |v| of the 16 lanes of a row, 2^-100): the block's amax, in
// every lane (rotations within the row of 16)
__device__ __forceinline__ float block_amax(const float (&v)[8]) {
    float a = kAmaxFloor;
#pragma unroll
    for (int j = 0; j < 8; ++j) a = fmaxf(a, fabsf(v[j]));
    auto ror = [](float x, auto ctrl) {
        return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), decltype(ctrl)::value, 0xF, 0xF, false));
    };
    a = fmaxf(a, ror(a, std::integral_constant<int, 0x128>{}));
    a = fmaxf(a, ror(a, std::integral_constant<int, 0x124>{}));
    a = fmaxf(a, ror(a, std::integral_constant<int, 0x122>{}));
    a = fmaxf(a, ror(a, std::integral_constant<int, 0x121>{}));
    return a;
}

// 16 bytes per lane from memory straight into LDS: lane l's go to dst + 16 l
// (an LDS address, the same in every lane).  Written as an instruction because the
// compiler takes every later LDS read to depend on the builtin's copy and
// waits for it at once; the kernel waits for its copies before the barrier
// that publishes them.  The instruction has no register result.  m0, which the
// copies write, is a register that the compiler gives to no value but sets for
// instructions of its own: named, it will not take an earlier setting to hold
// (its warning is about values kept in such registers).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void lds_copy16(const uint8_t* base, uint32_t off, uint32_t dst) {
    const uint32_t at = __builtin_amdgcn_readfirstlane(dst);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(at), "v"(off), "s"(base) : "memory", "m0");
}
__device__ __forceinline__ void lds_copy16(const uint8_t* src, uint32_t dst) {
    const uint32_t at = __builtin_amdgcn_readfirstlane(dst);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(at), "v"(src) : "memory", "m0");
}

// The same for 4 bytes per lane.
__device__ __forceinline__ void lds_copy4(const float* src, uint32_t dst) {
    const uint32_t at = __builtin_amdgcn_readfirstlane(dst);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(at), "v"(src) : "memory", "m0");
}

#pragma clang diagnostic pop

// Waits for this wave's LDS accesses and all but its last `LATER` memory
// accesses, then for the other waves'.
template <int LATER = 0>
__device__ __forceinline__ void publish() {
    static_assert(LATER < 64, "six bits of the wait's operand");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070 | (LATER & 15) | (LATER >> 4) << 14);  // vmcnt(LATER) lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// The 16-byte chunk c of a 128-byte row r in LDS is kept at slot c ^ key(r), so
// that eight neighbouring lanes of a fragment, which read chunk c of eight
// rows, read eight slots.  Rows of x: lane l reads row l + const.
__device__ __forceinline__ int xkey(int r) { return r & 7; }

// f(std::integral_constant<int, dtype>) for a float type of the C ABI
template <class F>
void by_float(int dt, F f) {
    if (dt == IQK_F32) f(std::integral_constant<int, IQK_F32>{});
    else if (dt == IQK_F16) f(std::integral_constant<int, IQK_F16>{});
    else f(std::integral_constant<int, IQK_BF16>{});
}

}  // namespace iqk
