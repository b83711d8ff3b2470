// iqk_layer.h -- launches of expert selection and the 8-bit products.  Nothing
// here is part of the C ABI.
#pragma once

#include "iqk_internal.h"

namespace iqk {

// Expert selection from router logits, and its gradient.
struct RouterLaunch {
    const void* logits;  // [T, E] of dtype
    int dtype;
    int64_t T;
    int E, k, scoring;
    const float* bias;  // [E] or null
    int n_group, topk_group, group_top, renorm;
    float scale;
    int32_t* ids;    // [T, k]
    float* weights;  // [T, k]
    bool wide = false, lane_groups = false;  // set by the launch
};

struct RouterGradLaunch {
    const void* logits;
    int dtype;
    const int32_t* ids;
    const float* d_weights;
    int64_t T;
    int E, k, scoring, renorm;
    float scale;
    void* d_logits;  // [T, E] of dtype
};

// Block quantization of activations to e4m3.
struct Fp8QuantLaunch {
    const void* x;  // [rows, n] of x_dtype
    int x_dtype;
    int64_t rows, n;
    uint8_t* codes;  // [rows, n]
    float* scales;   // [rows, ceil(n / 128)]
};

// Routed pairs grouped by expert for the 8-bit product (in no particular order
// inside an expert), with the number of `tile`-row tiles before each expert.
struct Fp8GroupLaunch {
    const int32_t* ids;  // [P]
    int64_t P;
    int E, tile;
    int32_t *counts, *offsets, *perm, *tiles, *hist;  // [E], [E + 1], [P], [E + 1], [slices, E]
    void* y;  // rows [P, out] of the call's result: NaN for pairs with an invalid id
    int out, y_half;
    int slices, nan_pairs;  // set by the launch
    int64_t slice, nans;
};

// The 8-bit product, dense (ids, offsets and perm null: M rows of x) or over
// routed pairs: per pair (ids) or grouped by expert (offsets, perm, tiles).
struct Fp8Launch {
    int64_t E, out, n;
    const uint8_t* codes;  // [E, out, n]
    const float* scales;   // [E, ceil(out / 128), ceil(n / 128)]
    const void* x;         // [rows, n] of x_dtype
    int x_dtype;
    const float* x_scales;  // [rows, ceil(n / 128)] for e4m3 x
    int64_t M;              // rows of y: tokens, or pairs
    int x_slots, k;
    const int32_t *ids, *offsets, *perm, *tiles;
    void* y;  // [M, out] of y_dtype
    int y_dtype;
    float* sums;  // dense, where the depth is split: fp8_sums_bytes()
};

// Whether a product's sums hold every product's bits whatever its path (see the sums' paragraph in iqk_fp8_device.h);
// bfloat16 results of many rows are summed on the 8-bit matrix instructions instead.
constexpr bool exact_sums(int y_dtype) { return y_dtype != IQK_BF16; }

hipError_t launch_router(const RouterLaunch& a, hipStream_t s);
hipError_t launch_router_grad(const RouterGradLaunch& a, hipStream_t s);
hipError_t launch_fp8_quantize(const Fp8QuantLaunch& a, hipStream_t s);
// slices of P pairs (the size of Fp8GroupLaunch::hist)
int fp8_group_slices(int64_t P);
// quantizes (unless q.x_dtype is e4m3) and groups
hipError_t launch_fp8_prep(Fp8GroupLaunch g, const Fp8QuantLaunch& q, hipStream_t s);
// whether launch_fp8_few takes `rows` rows of x of n values
bool fp8_few_fits(int64_t rows, int64_t n);
// few rows (or one pair per workgroup row), x of any type
hipError_t launch_fp8_few(const Fp8Launch& a, hipStream_t s);
// e4m3 x, up to 32 rows, in a pass over the weights
hipError_t launch_fp8_rows(const Fp8Launch& a, hipStream_t s);
// e4m3 x, many rows, by tiles of `rows` rows of x and `cols` weight rows, the
// depth in `parts` (each tile by a workgroup of its own per part)
struct Fp8Tile {
    int rows, cols, parts;
};
Fp8Tile fp8_grouped_tile(int64_t M, int64_t E, int64_t out, bool exact);
Fp8Tile fp8_dense_tile(int64_t M, int64_t out, int64_t n, bool exact);
// bytes of the parts' sums (0: not split), the same for every type of y
size_t fp8_sums_bytes(int64_t M, int64_t out, int64_t n);
hipError_t launch_fp8_tile(const Fp8Launch& a, const Fp8Tile& tile, hipStream_t s);

}  // namespace iqk
