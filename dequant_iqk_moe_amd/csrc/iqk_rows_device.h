// iqk_rows_device.h -- device helpers for kernels that pass over rows of any
// length: eight consecutive values of a row at any alignment, sums over a wave.
#pragma once

#include "iqk_fp8_device.h"

namespace iqk {

// Eight consecutive values as they lie in memory.
template <int DT>
struct Raw {
    uint32_t w[DT == IQK_F32 ? 8 : 4];
};

// Values i .. i + 7 of p, of which `left` are there; the others are zero.
// (Rows begin wherever their length puts them: loads take any address.)
template <int DT>
__device__ __forceinline__ Raw<DT> load_raw(const void* p, int64_t i, int left) {
    Raw<DT> r;
    constexpr int kSize = DT == IQK_F32 ? 4 : 2;
    if (left >= 8) {
        __builtin_memcpy(r.w, (const char*)p + i * kSize, 8 * kSize);
        return r;
    }
#pragma unroll
    for (int j = 0; j < 2 * kSize; ++j) r.w[j] = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (j >= left) continue;
        if constexpr (DT == IQK_F32) r.w[j] = ((const uint32_t*)p)[i + j];
        else r.w[j / 2] |= (uint32_t)((const uint16_t*)p)[i + j] << (j % 2 * 16);
    }
    return r;
}

template <int DT>
__device__ __forceinline__ void widen_raw(const Raw<DT>& r, float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if constexpr (DT == IQK_F32) v[j] = __uint_as_float(r.w[j]);
        else if constexpr (DT == IQK_BF16) v[j] = __uint_as_float(j % 2 ? r.w[j / 2] & 0xFFFF0000u : r.w[j / 2] << 16);
        else v[j] = half_to_float(j % 2 ? r.w[j / 2] >> 16 : r.w[j / 2] & 0xFFFFu);
    }
}

// Two values in 16 bits, rounded to nearest even (the hardware's conversions).
template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if constexpr (DT == IQK_F16) return __builtin_bit_cast(uint32_t, f16x2{(_Float16)a, (_Float16)b});
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
}

// min(left, 8) values of v to y + i (any address)
template <int DT>
__device__ __forceinline__ void store_some(void* y, int64_t i, const float (&v)[8], int left) {
    Raw<DT> r;
    if constexpr (DT == IQK_F32) {
#pragma unroll
        for (int j = 0; j < 8; ++j) r.w[j] = __float_as_uint(v[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) r.w[j] = pack2<DT>(v[2 * j], v[2 * j + 1]);
    }
    if (left >= 8) {
        __builtin_memcpy((char*)y + i * (DT == IQK_F32 ? 4 : 2), r.w, sizeof(r.w));
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (j >= left) continue;
        if constexpr (DT == IQK_F32) ((uint32_t*)y)[i + j] = r.w[j];
        else ((uint16_t*)y)[i + j] = (uint16_t)(r.w[j / 2] >> (j % 2 * 16));
    }
}

// x summed over the wave, in every lane: rotations within each 16 lanes, then
// the four sums in their order (the same result every time).
__device__ __forceinline__ float wave_sum(float x) {
    auto ror = [](float v, auto ctrl) {
        return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), decltype(ctrl)::value, 0xF, 0xF, false));
    };
    x += ror(x, std::integral_constant<int, 0x128>{});
    x += ror(x, std::integral_constant<int, 0x124>{});
    x += ror(x, std::integral_constant<int, 0x122>{});
    x += ror(x, std::integral_constant<int, 0x121>{});
    auto lane = [&](int l) { return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(x), l)); };
    return ((lane(0) + lane(16)) + lane(32)) + lane(48);
}

}  // namespace iqk
