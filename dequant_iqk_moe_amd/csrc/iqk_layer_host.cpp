// iqk_layer_host.cpp -- C-ABI entry points of what a MoE layer runs beside the
// IQ_K projections: expert selection from router logits and its gradient, and
// the 8-bit products.  Argument validation and dispatch; see include/iqk.h
// for the contract of every call.
#include <algorithm>
#include <cmath>

#include "iqk_layer.h"
#include "iqk_status.h"

using iqk::fail;
using iqk::ok;

namespace {

int hip_fail(hipError_t e, const char* where) { return fail(IQK_E_HIP, "%s: %s", where, hipGetErrorString(e)); }

size_t round256(size_t b) { return (b + 255) / 256 * 256; }
int64_t blocks128(int64_t n) { return (n + 127) / 128; }

bool is_float(int dt) { return dt == IQK_F32 || dt == IQK_F16 || dt == IQK_BF16; }
bool aligned(const void* p, size_t a) { return (uintptr_t)p % a == 0; }
size_t size_of(int dt) { return dt == IQK_F32 ? 4 : (dt == IQK_E4M3 ? 1 : 2); }

constexpr int64_t kMaxRows = 1LL << 24;  // rows or pairs of one call
constexpr int64_t kMaxSide = 1LL << 20;  // in and out of one expert
constexpr int64_t kMaxE = 16384;
constexpr int64_t kMaxValues = 1LL << 40;  // activations of one call

int check_router(const void* logits, int dtype, int64_t T, int64_t E, int k, int scoring, int renorm, float scale) {
    if (T < 0 || T > kMaxRows) return fail(IQK_E_ARG, "T = %lld outside [0, 2^24]", (long long)T);
    if (E <= 0 || E > 1024) return fail(IQK_E_ARG, "expert count %lld outside [1, 1024]", (long long)E);
    if (k <= 0 || k > 64 || k > E) return fail(IQK_E_ARG, "k = %d outside [1, min(64, E)]", k);
    if (!is_float(dtype)) return fail(IQK_E_ARG, "logits must be IQK_F32, IQK_F16 or IQK_BF16");
    if (scoring != IQK_SOFTMAX && scoring != IQK_SIGMOID) return fail(IQK_E_ARG, "unknown scoring %d", scoring);
    if (renorm != 0 && renorm != 1) return fail(IQK_E_ARG, "renorm must be 0 or 1");
    if (!std::isfinite(scale)) return fail(IQK_E_ARG, "scale must be finite");
    if (T > 0 && !logits) return fail(IQK_E_ARG, "null logits");
    if (!aligned(logits, size_of(dtype))) return fail(IQK_E_ARG, "logits must be aligned to their type");
    return IQK_OK;
}

int check_fp8_shape(const iqk_fp8_weights* w) {
    if (!w) return fail(IQK_E_ARG, "null weight descriptor");
    if (w->experts <= 0 || w->experts > kMaxE)
        return fail(IQK_E_ARG, "experts = %lld outside [1, 16384]", (long long)w->experts);
    if (w->out <= 0 || w->out > kMaxSide || w->in <= 0 || w->in > kMaxSide)
        return fail(IQK_E_ARG, "out and in must lie in [1, 2^20]");
    if (w->in % 16) return fail(IQK_E_SHAPE, "in = %lld must be a multiple of 16", (long long)w->in);
    if (w->out * w->in > 0x7FFFFFFFLL) return fail(IQK_E_ARG, "out * in must be below 2^31");
    return IQK_OK;
}

int check_fp8(const iqk_fp8_weights* w) {
    int rc = check_fp8_shape(w);
    if (rc) return rc;
    if (!w->codes || !w->scales) return fail(IQK_E_ARG, "null codes or scales");
    if (!aligned(w->codes, 16) || !aligned(w->scales, 4))
        return fail(IQK_E_ARG, "codes must be 16-byte and scales 4-byte aligned");
    const size_t codes = (size_t)(w->experts * w->out * w->in);
    const size_t scales = (size_t)(w->experts * blocks128(w->out) * blocks128(w->in));
    if (w->codes_bytes != codes) return fail(IQK_E_SIZE, "codes_bytes %zu != %zu", w->codes_bytes, codes);
    if (w->scales_count != scales) return fail(IQK_E_SIZE, "scales_count %zu != %zu", w->scales_count, scales);
    return IQK_OK;
}

// x, its scales and y of a product over `rows` rows of x
int check_fp8_io(const void* x, int x_dtype, const float* x_scales, const void* y, int y_dtype) {
    if (!is_float(x_dtype) && x_dtype != IQK_E4M3) return fail(IQK_E_ARG, "unknown x_dtype %d", x_dtype);
    if (!is_float(y_dtype)) return fail(IQK_E_ARG, "y must be IQK_F32, IQK_F16 or IQK_BF16");
    if (!x || !y) return fail(IQK_E_ARG, "null x or y");
    if (!aligned(x, 16)) return fail(IQK_E_ARG, "x must be 16-byte aligned");
    if (!aligned(y, size_of(y_dtype))) return fail(IQK_E_ARG, "y must be aligned to its type");
    if ((x_dtype == IQK_E4M3) != (x_scales != nullptr))
        return fail(IQK_E_ARG, "x_scales goes with IQK_E4M3 activations, and only with them");
    if (!aligned(x_scales, 4)) return fail(IQK_E_ARG, "x_scales must be 4-byte aligned");
    return IQK_OK;
}

int check_workspace(void* workspace, size_t have, size_t need) {
    if (have < need || (need && !workspace))
        return fail(IQK_E_SIZE, "workspace needs %zu bytes (got %zu)", need, workspace ? have : 0);
    if (!aligned(workspace, 16)) return fail(IQK_E_ARG, "workspace must be 16-byte aligned");
    return IQK_OK;
}

size_t quantized_bytes(int64_t rows, int64_t n) {
    return round256((size_t)(rows * n)) + round256((size_t)(rows * blocks128(n)) * 4);
}

// Rows of x up to which the dense product passes over the weights once
// without tiles.
constexpr int64_t kRowsPass = 32;
// Workspace of a tiled dense product's partial sums (0: none).
size_t dense_sums_bytes(int64_t M, int64_t out, int64_t n) {
    return M > kRowsPass ? round256(iqk::fp8_sums_bytes(M, out, n)) : 0;
}

// Whether the routed product takes each pair by itself: one launch without
// grouping, an expert's weights read once for each of its pairs.  Measured,
// each of its workgroups (16 weight rows) costs 3.3 ns of the card and its
// weights stream at 5.8 TB/s beside that; the grouped product reads the
// distinct experts at 5.2 TB/s after about 9 us for grouping (256 experts of
// 4096 x 4096, top-6: 1 token 25 us against 26, 2 tokens 47 against 45; 8
// experts, top-2: 4 tokens 28 against 35, 8 tokens 49 against 36; 256 experts
// of 1589 x 256, top-4: 4 tokens 12 against 17, 16 tokens 28 against 18).
bool pair_by_pair(int64_t P, int64_t E, int64_t out, int64_t n) {
    if (P > 4096 || !iqk::fp8_few_fits(1, n)) return false;
    const double us = 1e-6 * (double)(out * n);  // an expert's bytes at 1 TB/s
    const double pairs = (double)P * (3.3e-3 * (double)((out + 15) / 16) + us / 5.8);
    return pairs <= (double)std::min(P, E) * us / 5.2 + 9.0;
}

// Quantizes the rows of a product's x into `ws` and points L at the result.
hipError_t quantize_into(iqk::Fp8Launch* L, int64_t rows, uint8_t* ws, hipStream_t s) {
    iqk::Fp8QuantLaunch Q{L->x, L->x_dtype, rows, L->n, ws, (float*)(ws + round256((size_t)(rows * L->n)))};
    L->x = Q.codes;
    L->x_scales = Q.scales;
    L->x_dtype = IQK_E4M3;
    return iqk::launch_fp8_quantize(Q, s);
}

}  // namespace

extern "C" {

int iqk_router_topk(const void* logits, int dtype, int64_t T, int64_t E, int k, int scoring, const float* bias,
                    int n_group, int topk_group, int group_top, int renorm, float scale, int32_t* ids, float* weights,
                    void* stream) {
    int rc = check_router(logits, dtype, T, E, k, scoring, renorm, scale);
    if (rc) return rc;
    if (n_group < 1 || n_group > 64 || E % n_group)
        return fail(IQK_E_ARG, "n_group = %d must divide the %lld experts and be at most 64", n_group, (long long)E);
    if (topk_group < 1 || topk_group > n_group) return fail(IQK_E_ARG, "topk_group must lie in [1, n_group]");
    if (group_top != 1 && group_top != 2) return fail(IQK_E_ARG, "group_top must be 1 or 2");
    if (!aligned(bias, 4)) return fail(IQK_E_ARG, "bias must be 4-byte aligned");
    if (T == 0) return ok();
    if (!ids || !weights) return fail(IQK_E_ARG, "null ids or weights");
    iqk::RouterLaunch L{logits, dtype, T, (int)E, k, scoring, bias, n_group, topk_group, group_top, renorm, scale,
                        ids, weights};
    hipError_t e = iqk::launch_router(L, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "router launch");
    return ok();
}

int iqk_router_topk_grad(const void* logits, int dtype, const int32_t* ids, const float* d_weights, int64_t T,
                         int64_t E, int k, int scoring, int renorm, float scale, void* d_logits, void* stream) {
    int rc = check_router(logits, dtype, T, E, k, scoring, renorm, scale);
    if (rc) return rc;
    if (T == 0) return ok();
    if (!ids || !d_weights || !d_logits) return fail(IQK_E_ARG, "null ids, d_weights or d_logits");
    if (!aligned(d_logits, size_of(dtype))) return fail(IQK_E_ARG, "d_logits must be aligned to its type");
    iqk::RouterGradLaunch L{logits, dtype, ids, d_weights, T, (int)E, k, scoring, renorm, scale, d_logits};
    hipError_t e = iqk::launch_router_grad(L, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "router gradient launch");
    return ok();
}

int iqk_fp8_quantize(const void* x, int x_dtype, int64_t rows, int64_t n, uint8_t* codes, float* scales,
                     void* stream) {
    if (rows < 0 || rows > kMaxRows) return fail(IQK_E_ARG, "rows = %lld outside [0, 2^24]", (long long)rows);
    if (n <= 0 || n > kMaxSide) return fail(IQK_E_ARG, "n must lie in [1, 2^20]");
    if (n % 16) return fail(IQK_E_SHAPE, "n = %lld must be a multiple of 16", (long long)n);
    if (!is_float(x_dtype)) return fail(IQK_E_ARG, "x must be IQK_F32, IQK_F16 or IQK_BF16");
    if (rows * n > kMaxValues) return fail(IQK_E_ARG, "rows * n exceeds 2^40");
    if (rows == 0) return ok();
    if (!x || !codes || !scales) return fail(IQK_E_ARG, "null pointer");
    if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 4))
        return fail(IQK_E_ARG, "x and codes must be 16-byte and scales 4-byte aligned");
    iqk::Fp8QuantLaunch L{x, x_dtype, rows, n, codes, scales};
    hipError_t e = iqk::launch_fp8_quantize(L, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "quantize launch");
    return ok();
}

int iqk_fp8_linear_workspace(const iqk_fp8_weights* w, int64_t M, size_t* bytes) {
    if (!bytes) return fail(IQK_E_ARG, "null pointer");
    int rc = check_fp8_shape(w);
    if (rc) return rc;
    if (M < 0 || M > kMaxRows) return fail(IQK_E_ARG, "M = %lld outside [0, 2^24]", (long long)M);
    if (M * w->in > kMaxValues) return fail(IQK_E_ARG, "M * in exceeds 2^40");
    *bytes = iqk::fp8_few_fits(M, w->in) ? 0 : dense_sums_bytes(M, w->out, w->in) + quantized_bytes(M, w->in);
    return ok();
}

int iqk_fp8_linear(const iqk_fp8_weights* w, const void* x, int x_dtype, const float* x_scales, int64_t M,
                   void* workspace, size_t ws_bytes, void* y, int y_dtype, void* stream) {
    int rc = check_fp8(w);
    if (rc) return rc;
    if (w->experts != 1) return fail(IQK_E_ARG, "the dense product takes one expert's weights (got %lld)", (long long)w->experts);
    if (M < 0 || M > kMaxRows) return fail(IQK_E_ARG, "M = %lld outside [0, 2^24]", (long long)M);
    if (M * w->in > kMaxValues) return fail(IQK_E_ARG, "M * in exceeds 2^40");
    if (M == 0) return ok();
    rc = check_fp8_io(x, x_dtype, x_scales, y, y_dtype);
    if (rc) return rc;
    const bool quantize = x_dtype != IQK_E4M3;
    const bool few = iqk::fp8_few_fits(M, w->in);
    const size_t sums = few ? 0 : dense_sums_bytes(M, w->out, w->in);
    rc = check_workspace(workspace, ws_bytes, sums + (quantize && !few ? quantized_bytes(M, w->in) : 0));
    if (rc) return rc;
    hipStream_t s = (hipStream_t)stream;
    iqk::Fp8Launch L{1, w->out, w->in, (const uint8_t*)w->codes, w->scales, x, x_dtype, x_scales, M, 1, 1,
                     nullptr, nullptr, nullptr, nullptr, y, y_dtype, (float*)workspace};
    hipError_t e;
    if (few) {
        e = iqk::launch_fp8_few(L, s);
    } else {
        if (quantize && (e = quantize_into(&L, M, (uint8_t*)workspace + sums, s)) != hipSuccess)
            return hip_fail(e, "quantize launch");
        e = M <= kRowsPass ? iqk::launch_fp8_rows(L, s)
                           : iqk::launch_fp8_tile(L, iqk::fp8_dense_tile(M, w->out, w->in, iqk::exact_sums(y_dtype)), s);
    }
    if (e != hipSuccess) return hip_fail(e, "8-bit product launch");
    return ok();
}

int iqk_fp8_path(const iqk_fp8_weights* w, int64_t T, int k, int y_dtype, int32_t* path) {
    if (!path) return fail(IQK_E_ARG, "null pointer");
    int rc = check_fp8_shape(w);
    if (rc) return rc;
    if (k < 0 || T < 1 || T > kMaxRows / std::max(k, 1)) return fail(IQK_E_ARG, "T * max(k, 1) must lie in [1, 2^24]");
    if (k == 0 && w->experts != 1) return fail(IQK_E_ARG, "the dense product takes one expert's weights");
    if (!is_float(y_dtype)) return fail(IQK_E_ARG, "y must be IQK_F32, IQK_F16 or IQK_BF16");
    const bool exact = iqk::exact_sums(y_dtype);
    path[0] = path[1] = path[2] = path[3] = 0;
    if (k == 0 ? iqk::fp8_few_fits(T, w->in) : pair_by_pair(T * k, w->experts, w->out, w->in)) return ok();
    path[0] = k == 0 && T <= kRowsPass ? 1 : 2;
    if (path[0] == 1) return ok();
    const iqk::Fp8Tile t = k == 0 ? iqk::fp8_dense_tile(T, w->out, w->in, exact)
                                  : iqk::fp8_grouped_tile(T * k, w->experts, w->out, exact);
    path[1] = t.rows;
    path[2] = t.cols;
    path[3] = t.parts;
    return ok();
}

int iqk_moe_fp8_workspace(const iqk_fp8_weights* w, int64_t T, int k, int x_slots, size_t* bytes) {
    if (!bytes) return fail(IQK_E_ARG, "null pointer");
    int rc = check_fp8_shape(w);
    if (rc) return rc;
    if (T < 0 || k <= 0 || T > kMaxRows / k) return fail(IQK_E_ARG, "T * k must lie in [0, 2^24]");
    if (x_slots != 1 && x_slots != k) return fail(IQK_E_ARG, "x_slots must be 1 or k");
    if (T * x_slots * w->in > kMaxValues) return fail(IQK_E_ARG, "T * x_slots * in exceeds 2^40");
    const size_t E = (size_t)w->experts, P = (size_t)std::max<int64_t>(T * k, 1);
    if (pair_by_pair(T * k, w->experts, w->out, w->in)) {
        *bytes = 0;
        return ok();
    }
    *bytes = round256(E * 4) + 2 * round256((E + 1) * 4) + round256(P * 4) +
             round256((size_t)iqk::fp8_group_slices(P) * E * 4) + quantized_bytes(T * x_slots, w->in);
    return ok();
}

int iqk_moe_fp8(const iqk_fp8_weights* w, const void* x, int x_dtype, const float* x_scales, int x_slots,
                const int32_t* ids, int64_t T, int k, int sorted, void* workspace, size_t ws_bytes, void* y,
                int y_dtype, void* stream) {
    int rc = check_fp8(w);
    if (rc) return rc;
    size_t need = 0;
    rc = iqk_moe_fp8_workspace(w, T, k, x_slots, &need);
    if (rc) return rc;
    if (sorted != 0 && sorted != 1) return fail(IQK_E_ARG, "sorted must be 0 or 1");
    if (T == 0) return ok();
    rc = check_fp8_io(x, x_dtype, x_scales, y, y_dtype);
    if (rc) return rc;
    if (!ids) return fail(IQK_E_ARG, "null ids");
    if (x_dtype == IQK_E4M3 && need) need -= quantized_bytes(T * x_slots, w->in);
    rc = check_workspace(workspace, ws_bytes, need);
    if (rc) return rc;
    const int64_t E = w->experts, P = T * k;
    hipStream_t s = (hipStream_t)stream;
    iqk::Fp8Launch L{E, w->out, w->in, (const uint8_t*)w->codes, w->scales, x, x_dtype, x_scales, P, x_slots, k,
                     ids, nullptr, nullptr, nullptr, y, y_dtype, nullptr};
    hipError_t e;
    if (pair_by_pair(P, E, w->out, w->in)) {
        e = iqk::launch_fp8_few(L, s);
        if (e != hipSuccess) return hip_fail(e, "8-bit product launch");
        return ok();
    }
    uint8_t* ws = (uint8_t*)workspace;
    auto take = [&](size_t bytes) {
        uint8_t* at = ws;
        ws += round256(bytes);
        return at;
    };
    const iqk::Fp8Tile tile = iqk::fp8_grouped_tile(P, E, w->out, iqk::exact_sums(y_dtype));
    iqk::Fp8GroupLaunch G{};
    G.ids = ids;
    G.P = P;
    G.E = (int)E;
    G.tile = tile.rows;
    G.counts = (int32_t*)take((size_t)E * 4);
    G.offsets = (int32_t*)take((size_t)(E + 1) * 4);
    G.tiles = (int32_t*)take((size_t)(E + 1) * 4);
    G.perm = (int32_t*)take((size_t)P * 4);
    G.hist = (int32_t*)take((size_t)iqk::fp8_group_slices(P) * E * 4);
    G.y = y;
    G.out = (int)w->out;
    G.y_half = y_dtype != IQK_F32;
    iqk::Fp8QuantLaunch Q{x, x_dtype, T * x_slots, w->in, ws, (float*)(ws + round256((size_t)(T * x_slots * w->in)))};
    e = iqk::launch_fp8_prep(G, Q, s);
    if (e != hipSuccess) return hip_fail(e, "grouping launch");
    if (x_dtype != IQK_E4M3) {
        L.x = Q.codes;
        L.x_scales = Q.scales;
        L.x_dtype = IQK_E4M3;
    }
    L.ids = nullptr;
    L.offsets = G.offsets;
    L.perm = G.perm;
    L.tiles = G.tiles;
    e = iqk::launch_fp8_tile(L, tile, s);
    if (e != hipSuccess) return hip_fail(e, "8-bit grouped product launch");
    return ok();
}

}  // extern "C"
