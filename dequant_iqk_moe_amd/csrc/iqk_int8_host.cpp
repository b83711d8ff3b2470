// iqk_int8_host.cpp -- C-ABI entry points of the 8-bit integer products.
// Argument validation and dispatch; see include/iqk.h for the contract of every
// call.
#include "iqk_block.h"
#include "iqk_status.h"

using iqk::fail;
using iqk::ok;

namespace {

int hip_fail(hipError_t e, const char* where) { return fail(IQK_E_HIP, "%s: %s", where, hipGetErrorString(e)); }

size_t round256(size_t b) { return (b + 255) / 256 * 256; }
bool is_float(int dt) { return dt == IQK_F32 || dt == IQK_F16 || dt == IQK_BF16; }
bool aligned(const void* p, size_t a) { return (uintptr_t)p % a == 0; }
size_t size_of(int dt) { return dt == IQK_F32 ? 4 : dt == IQK_INT8 ? 1 : 2; }
// whether two ranges of memory overlap
bool overlap(const void* a, size_t an, const void* b, size_t bn) {
    return (uintptr_t)a < (uintptr_t)b + bn && (uintptr_t)b < (uintptr_t)a + an;
}

constexpr int64_t kMaxRows = 1LL << 24;
constexpr int64_t kMaxDepth = 1LL << 16;  // (products of -128 by -128 sum to 2^30)
constexpr int64_t kMaxOut = 1LL << 20;
constexpr int64_t kMaxExperts = 2048;

int check_depth(int64_t n) {
    if (n <= 0 || n > kMaxDepth) return fail(IQK_E_ARG, "in = %lld outside [1, 2^16]", (long long)n);
    if (n % 16) return fail(IQK_E_SHAPE, "in = %lld must be a multiple of 16", (long long)n);
    return IQK_OK;
}

int check_shape(const iqk_int8_weights* w) {
    if (!w) return fail(IQK_E_ARG, "null weight descriptor");
    if (w->experts <= 0 || w->experts > kMaxExperts)
        return fail(IQK_E_ARG, "experts = %lld outside [1, 2048]", (long long)w->experts);
    if (w->out <= 0 || w->out > kMaxOut) return fail(IQK_E_ARG, "out = %lld outside [1, 2^20]", (long long)w->out);
    int rc = check_depth(w->in);
    if (rc) return rc;
    if (w->out * w->in > 0x7FFFFFFFLL) return fail(IQK_E_ARG, "out * in must be below 2^31");
    return IQK_OK;
}

int check_weights(const iqk_int8_weights* w) {
    int rc = check_shape(w);
    if (rc) return rc;
    if (!w->codes || !w->scales) return fail(IQK_E_ARG, "null codes or scales");
    if (!aligned(w->codes, 16) || !aligned(w->scales, 4))
        return fail(IQK_E_ARG, "codes must be 16-byte and scales 4-byte aligned");
    const size_t codes = (size_t)(w->experts * w->out * w->in), scales = (size_t)(w->experts * w->out);
    if (w->codes_bytes != codes) return fail(IQK_E_SIZE, "codes_bytes %zu != %zu", w->codes_bytes, codes);
    if (w->scales_count != scales) return fail(IQK_E_SIZE, "scales_count %zu != %zu", w->scales_count, scales);
    return IQK_OK;
}

int check_rows(int64_t rows) {
    if (rows < 0 || rows > kMaxRows) return fail(IQK_E_ARG, "rows = %lld outside [0, 2^24]", (long long)rows);
    return IQK_OK;
}

int check_x_type(int x_dtype) {
    if (!is_float(x_dtype) && x_dtype != IQK_INT8) return fail(IQK_E_ARG, "unknown x_dtype %d", x_dtype);
    return IQK_OK;
}

int check_io(const void* x, int x_dtype, const float* x_scales, const void* y, int y_dtype) {
    int rc = check_x_type(x_dtype);
    if (rc) return rc;
    if (!is_float(y_dtype)) return fail(IQK_E_ARG, "y must be IQK_F32, IQK_F16 or IQK_BF16");
    if (!x || !y) return fail(IQK_E_ARG, "null x or y");
    if (!aligned(x, 16)) return fail(IQK_E_ARG, "x must be 16-byte aligned");
    if (!aligned(y, size_of(y_dtype))) return fail(IQK_E_ARG, "y must be aligned to its type");
    if ((x_dtype == IQK_INT8) != (x_scales != nullptr))
        return fail(IQK_E_ARG, "x_scales goes with IQK_INT8 activations, and only with them");
    if (!aligned(x_scales, 4)) return fail(IQK_E_ARG, "x_scales must be 4-byte aligned");
    return IQK_OK;
}

// The plan (grouped), then the quantized x and its scales.
size_t plan_bytes(const iqk_int8_weights* w, bool grouped) { return grouped ? round256((size_t)(w->experts + 2) * 4) : 0; }
size_t workspace_bytes(const iqk_int8_weights* w, int64_t rows, int x_dtype, bool grouped) {
    if (rows == 0 || iqk::int8_few_fits(rows, w->in, grouped)) return 0;
    const size_t quantized = x_dtype == IQK_INT8 ? 0 : round256((size_t)(rows * w->in)) + round256((size_t)rows * 4);
    return plan_bytes(w, grouped) + quantized;
}

int product(const iqk_int8_weights* w, const void* x, int x_dtype, const float* x_scales, const int32_t* offsets, bool grouped,
            int64_t rows, void* workspace, size_t ws_bytes, void* y, int y_dtype, void* stream) {
    int rc = check_weights(w);
    if (!rc) rc = check_rows(rows);
    if (rc) return rc;
    if (rows == 0) return ok();
    rc = check_io(x, x_dtype, x_scales, y, y_dtype);
    if (rc) return rc;
    if (grouped && !offsets) return fail(IQK_E_ARG, "null offsets");
    if (!aligned(offsets, 4)) return fail(IQK_E_ARG, "offsets must be 4-byte aligned");
    const size_t need = workspace_bytes(w, rows, x_dtype, grouped);
    if (ws_bytes < need || (need && !workspace))
        return fail(IQK_E_SIZE, "workspace needs %zu bytes (got %zu)", need, workspace ? ws_bytes : 0);
    if (!aligned(workspace, 16)) return fail(IQK_E_ARG, "workspace must be 16-byte aligned");
    if (overlap(y, (size_t)(rows * w->out) * size_of(y_dtype), x, (size_t)(rows * w->in) * size_of(x_dtype)))
        return fail(IQK_E_ARG, "y must not overlap x");
    hipStream_t s = (hipStream_t)stream;
    iqk::Int8Launch L{w->experts, w->out, w->in, (const int8_t*)w->codes, w->scales, x, x_dtype, x_scales, rows,
                      grouped ? offsets : nullptr, nullptr, y, y_dtype};
    hipError_t e;
    if (iqk::int8_few_fits(rows, w->in, grouped)) {
        e = iqk::launch_int8_few(L, s);
    } else {
        const bool few = !grouped && iqk::int8_rows_fits(rows, w->out);
        const iqk::Int8Tile tile = iqk::int8_tile(rows, w->experts, w->out, w->in, grouped);
        uint8_t* at = (uint8_t*)workspace;
        iqk::Int8Plan plan{grouped ? offsets : nullptr, (int)w->experts, tile.rows, (int32_t*)at};
        at += plan_bytes(w, grouped);
        iqk::Int8QuantLaunch Q{x, x_dtype, rows, w->in, (int8_t*)at, (float*)(at + round256((size_t)(rows * w->in)))};
        e = iqk::launch_int8_prep(Q, plan, s);
        if (e != hipSuccess) return hip_fail(e, "quantize launch");
        if (x_dtype != IQK_INT8) {
            L.x = Q.codes;
            L.x_scales = Q.scales;
            L.x_dtype = IQK_INT8;
        }
        L.tiles = plan.tiles;
        e = few ? iqk::launch_int8_rows(L, s) : iqk::launch_int8_tile(L, tile, s);
    }
    if (e != hipSuccess) return hip_fail(e, "8-bit product launch");
    return ok();
}

}  // namespace

extern "C" {

int iqk_int8_quantize(const void* x, int x_dtype, int64_t rows, int64_t n, int8_t* codes, float* scales, void* stream) {
    int rc = check_rows(rows);
    if (!rc) rc = check_depth(n);
    if (rc) return rc;
    if (!is_float(x_dtype)) return fail(IQK_E_ARG, "x must be IQK_F32, IQK_F16 or IQK_BF16");
    if (rows == 0) return ok();
    if (!x || !codes || !scales) return fail(IQK_E_ARG, "null pointer");
    if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 4))
        return fail(IQK_E_ARG, "x and codes must be 16-byte and scales 4-byte aligned");
    if (overlap(codes, (size_t)(rows * n), x, (size_t)(rows * n) * size_of(x_dtype)))
        return fail(IQK_E_ARG, "codes must not overlap x");
    hipError_t e = iqk::launch_int8_prep(iqk::Int8QuantLaunch{x, x_dtype, rows, n, codes, scales}, iqk::Int8Plan{}, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "quantize launch");
    return ok();
}

int iqk_int8_linear_workspace(const iqk_int8_weights* w, int64_t M, int x_dtype, size_t* bytes) {
    if (!bytes) return fail(IQK_E_ARG, "null pointer");
    int rc = check_shape(w);
    if (!rc) rc = check_rows(M);
    if (!rc) rc = check_x_type(x_dtype);
    if (rc) return rc;
    *bytes = workspace_bytes(w, M, x_dtype, false);
    return ok();
}

int iqk_int8_linear(const iqk_int8_weights* w, const void* x, int x_dtype, const float* x_scales, int64_t M, void* workspace,
                    size_t ws_bytes, void* y, int y_dtype, void* stream) {
    if (w && w->experts > 1) return fail(IQK_E_ARG, "the dense product takes one expert's weights (got %lld)", (long long)w->experts);
    return product(w, x, x_dtype, x_scales, nullptr, false, M, workspace, ws_bytes, y, y_dtype, stream);
}

int iqk_int8_grouped_workspace(const iqk_int8_weights* w, int64_t rows, int x_dtype, size_t* bytes) {
    if (!bytes) return fail(IQK_E_ARG, "null pointer");
    int rc = check_shape(w);
    if (!rc) rc = check_rows(rows);
    if (!rc) rc = check_x_type(x_dtype);
    if (rc) return rc;
    *bytes = workspace_bytes(w, rows, x_dtype, true);
    return ok();
}

int iqk_int8_grouped(const iqk_int8_weights* w, const void* x, int x_dtype, const float* x_scales, const int32_t* offsets,
                     int64_t rows, void* workspace, size_t ws_bytes, void* y, int y_dtype, void* stream) {
    return product(w, x, x_dtype, x_scales, offsets, true, rows, workspace, ws_bytes, y, y_dtype, stream);
}

int iqk_int8_path(const iqk_int8_weights* w, int64_t rows, int grouped, int32_t* path) {
    if (!path) return fail(IQK_E_ARG, "null pointer");
    int rc = check_shape(w);
    if (!rc) rc = check_rows(rows);
    if (rc) return rc;
    if (rows == 0) return fail(IQK_E_ARG, "rows must lie in [1, 2^24]");
    if (grouped != 0 && grouped != 1) return fail(IQK_E_ARG, "grouped must be 0 or 1");
    if (!grouped && w->experts != 1) return fail(IQK_E_ARG, "the dense product takes one expert's weights");
    path[0] = path[1] = path[2] = 0;
    if (iqk::int8_few_fits(rows, w->in, grouped != 0)) return ok();
    path[0] = !grouped && iqk::int8_rows_fits(rows, w->out) ? 1 : 2;
    if (path[0] == 1) return ok();
    const iqk::Int8Tile t = iqk::int8_tile(rows, w->experts, w->out, w->in, grouped != 0);
    path[1] = t.rows;
    path[2] = t.cols;
    return ok();
}

}  // extern "C"
