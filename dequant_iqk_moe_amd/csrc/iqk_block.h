// iqk_block.h -- launches of the operators around the routed experts: rows
// sorted by expert and back, 8-bit integer products, block norms.  Nothing
// here is part of the C ABI.
#pragma once

#include "iqk_internal.h"

namespace iqk {

// Token rows in the order of their experts.
struct SortLaunch {
    const void* x;  // [T, n] of dtype
    int dtype;
    const int32_t* ids;  // [T, k]
    int64_t T;
    int k, E;
    int64_t n;
    int32_t* hist;  // [sort_slices(T, k), E + 1], where those are more than 0
    void* xs;       // [T * k, n]
    int32_t *offsets, *place;  // [E + 1], [T, k]
};

// Expert rows back to their tokens, and the gradient of that.
struct UnsortLaunch {
    const void* ys;  // [T * k, n] of ys_dtype
    int ys_dtype;
    const int32_t* place;  // [T, k]
    const float* weights;  // [T, k] or null
    int64_t T;
    int k;
    int64_t n;
    void* y;  // [T, n] of y_dtype
    int y_dtype;
};

struct UnsortGradLaunch {
    const void* dy;  // [T, n] of dy_dtype
    int dy_dtype;
    const void* ys;
    int ys_dtype;
    const int32_t* place;
    const float* weights;
    int64_t T;
    int k;
    int64_t n;
    void* d_ys;        // [T * k, n] of ys_dtype, or null
    float* d_weights;  // [T, k], or null
};

// Slices of its pairs that a large sort counts by themselves (0: none, it goes in one launch).
int sort_slices(int64_t T, int k);
hipError_t launch_sort(const SortLaunch& a, hipStream_t s);
hipError_t launch_unsort(const UnsortLaunch& a, hipStream_t s);
hipError_t launch_unsort_grad(const UnsortGradLaunch& a, hipStream_t s);

// Quantization of activations to 8-bit integers, and with it the tiles before
// each expert of a grouped product.
struct Int8QuantLaunch {
    const void* x;  // [rows, n] of x_dtype
    int x_dtype;
    int64_t rows, n;
    int8_t* codes;   // [rows, n]
    float* scales;   // [rows]
};
struct Int8Plan {
    const int32_t* offsets;  // [E + 1], or null: no plan
    int E, tile;             // rows of a tile
    int32_t* tiles;          // [E + 2]: tiles before expert e, before the rows of none, and in all
};

// The 8-bit integer product, dense (offsets null) or of rows sorted by expert.
struct Int8Launch {
    int64_t E, out, n;
    const int8_t* codes;  // [E, out, n]
    const float* scales;  // [E, out]
    const void* x;        // [M, n] of x_dtype
    int x_dtype;
    const float* x_scales;  // [M] for codes
    int64_t M;
    const int32_t *offsets, *tiles;
    void* y;  // [M, out] of y_dtype
    int y_dtype;
};
struct Int8Tile {
    int rows, cols;
};

// quantizes (unless q.x_dtype is IQK_INT8) and plans (if g.offsets is set)
hipError_t launch_int8_prep(const Int8QuantLaunch& q, const Int8Plan& g, hipStream_t s);
// whether launch_int8_few takes M rows of n values
bool int8_few_fits(int64_t M, int64_t n, bool grouped);
// few rows, x of any type
hipError_t launch_int8_few(const Int8Launch& a, hipStream_t s);
// whether launch_int8_rows takes M rows
bool int8_rows_fits(int64_t M, int64_t out);
// dense, x in codes, up to 32 rows
hipError_t launch_int8_rows(const Int8Launch& a, hipStream_t s);
// x in codes, by tiles
Int8Tile int8_tile(int64_t M, int64_t E, int64_t out, int64_t n, bool grouped);
hipError_t launch_int8_tile(const Int8Launch& a, const Int8Tile& tile, hipStream_t s);

// What the gradient of a block's norms is taken from and written to (any may be
// null but one of dr and dh).
struct NormGradOut {
    const void *dr, *dh;
    void *dx, *dy, *d_post, *d_gate, *d_next;
};

// Bytes of the teams' parts of `columns` parameters' gradients.
int64_t norm_sums_bytes(int64_t T, int64_t n, int columns);
hipError_t launch_norm(const iqk_block& b, void* r, void* h, hipStream_t s);
hipError_t launch_norm_grad(const iqk_block& b, const NormGradOut& o, float* sums, hipStream_t s);

}  // namespace iqk
