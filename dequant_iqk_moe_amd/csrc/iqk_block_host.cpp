// iqk_block_host.cpp -- C-ABI entry points of the operators around the routed
// experts: rows sorted by expert and back, block norms.  Argument validation;
// see include/iqk.h for the contract of every call.
#include <cmath>

#include "iqk_block.h"
#include "iqk_status.h"

using iqk::fail;
using iqk::ok;

namespace {

int hip_fail(hipError_t e, const char* where) { return fail(IQK_E_HIP, "%s: %s", where, hipGetErrorString(e)); }

bool is_float(int dt) { return dt == IQK_F32 || dt == IQK_F16 || dt == IQK_BF16; }
bool aligned(const void* p, size_t a) { return (uintptr_t)p % a == 0; }
size_t size_of(int dt) { return dt == IQK_F32 ? 4 : 2; }
bool typed(const void* p, int dt) { return aligned(p, size_of(dt)); }
// whether two ranges of memory overlap (null: none)
bool overlap(const void* a, size_t an, const void* b, size_t bn) {
    return a && b && (uintptr_t)a < (uintptr_t)b + bn && (uintptr_t)b < (uintptr_t)a + an;
}

constexpr int64_t kMaxRows = 1LL << 24;
constexpr int64_t kMaxWidth = 1LL << 20;
constexpr int64_t kMaxExperts = 2048;
constexpr int64_t kMaxNorm = 8192;

int check_pairs(int64_t T, int k) {
    if (k < 1 || k > 64) return fail(IQK_E_ARG, "k = %d outside [1, 64]", k);
    if (T < 0 || T > kMaxRows / k) return fail(IQK_E_ARG, "T * k must lie in [0, 2^24]");
    return IQK_OK;
}

int check_width(int64_t n) {
    if (n < 1 || n > kMaxWidth) return fail(IQK_E_ARG, "n = %lld outside [1, 2^20]", (long long)n);
    return IQK_OK;
}

int check_experts(int64_t E) {
    if (E < 1 || E > kMaxExperts) return fail(IQK_E_ARG, "expert count %lld outside [1, 2048]", (long long)E);
    return IQK_OK;
}

size_t sort_bytes(int64_t T, int k, int64_t E) { return (size_t)iqk::sort_slices(T, k) * (size_t)(E + 1) * 4; }

int check_block(const iqk_block* b) {
    if (!b) return fail(IQK_E_ARG, "null block descriptor");
    if (b->T < 0 || b->T > kMaxRows) return fail(IQK_E_ARG, "T = %lld outside [0, 2^24]", (long long)b->T);
    if (b->n < 1 || b->n > kMaxNorm) return fail(IQK_E_ARG, "n = %lld outside [1, 8192]", (long long)b->n);
    if (!is_float(b->dtype)) return fail(IQK_E_ARG, "x must be IQK_F32, IQK_F16 or IQK_BF16");
    if (!std::isfinite(b->alpha) || !std::isfinite(b->beta)) return fail(IQK_E_ARG, "alpha and beta must be finite");
    if (!(b->eps > 0) || !std::isfinite(b->eps)) return fail(IQK_E_ARG, "eps must be positive and finite");
    if (b->gate_kind < IQK_GATE_NONE || b->gate_kind > IQK_GATE_ELEMENT) return fail(IQK_E_ARG, "unknown gate_kind %d", b->gate_kind);
    if ((b->gate_kind != IQK_GATE_NONE) != (b->gate != nullptr)) {
        // (a gate of no tokens has no memory)
        if (b->T > 0 || b->gate) return fail(IQK_E_ARG, "gate goes with a gate_kind, and only with one");
    }
    if ((b->post_weight || b->next_weight) && !is_float(b->weight_dtype))
        return fail(IQK_E_ARG, "weights must be IQK_F32, IQK_F16 or IQK_BF16");
    if (b->gate && !is_float(b->gate_dtype)) return fail(IQK_E_ARG, "gate must be IQK_F32, IQK_F16 or IQK_BF16");
    if (b->T > 0 && !b->x) return fail(IQK_E_ARG, "null x");
    if (b->y) {
        if (b->y_dtype != b->dtype && b->y_dtype != IQK_F32) return fail(IQK_E_ARG, "y must be of x's type or IQK_F32");
    } else if (b->T > 0) {
        if (b->post_weight || b->gate) return fail(IQK_E_ARG, "post_weight and gate need y");
        if (!b->next_weight) return fail(IQK_E_ARG, "a call without y needs next_weight");
        if (b->alpha != 1.f) return fail(IQK_E_ARG, "alpha must be 1 without y");
    }
    if (!typed(b->x, b->dtype) || (b->y && !typed(b->y, b->y_dtype)) || (b->gate && !typed(b->gate, b->gate_dtype)) ||
        (b->post_weight && !typed(b->post_weight, b->weight_dtype)) || (b->next_weight && !typed(b->next_weight, b->weight_dtype)))
        return fail(IQK_E_ARG, "x, y, weights and gate must be aligned to their types");
    return IQK_OK;
}

}  // namespace

extern "C" {

int iqk_moe_sort_workspace(int64_t T, int k, int64_t E, size_t* bytes) {
    if (!bytes) return fail(IQK_E_ARG, "null pointer");
    int rc = check_pairs(T, k);
    if (!rc) rc = check_experts(E);
    if (rc) return rc;
    *bytes = sort_bytes(T, k, E);
    return ok();
}

int iqk_moe_sort(const void* x, int dtype, const int32_t* ids, int64_t T, int k, int64_t E, int64_t n, void* workspace,
                 size_t ws_bytes, void* xs, int32_t* offsets, int32_t* place, void* stream) {
    int rc = check_pairs(T, k);
    if (!rc) rc = check_experts(E);
    if (!rc) rc = check_width(n);
    if (rc) return rc;
    if (!is_float(dtype)) return fail(IQK_E_ARG, "x must be IQK_F32, IQK_F16 or IQK_BF16");
    if (!offsets) return fail(IQK_E_ARG, "null offsets");
    if (T > 0 && (!x || !ids || !xs || !place)) return fail(IQK_E_ARG, "null x, ids, xs or place");
    if (!typed(x, dtype) || !typed(xs, dtype)) return fail(IQK_E_ARG, "x and xs must be aligned to their type");
    if (!aligned(ids, 4) || !aligned(offsets, 4) || !aligned(place, 4))
        return fail(IQK_E_ARG, "ids, offsets and place must be 4-byte aligned");
    const size_t need = sort_bytes(T, k, E);
    if (ws_bytes < need || (need && !workspace))
        return fail(IQK_E_SIZE, "workspace needs %zu bytes (got %zu)", need, workspace ? ws_bytes : 0);
    if (!aligned(workspace, 4)) return fail(IQK_E_ARG, "workspace must be 4-byte aligned");
    const size_t rows = (size_t)(T * n) * size_of(dtype), pairs = (size_t)(T * k) * 4;
    if (overlap(xs, rows * k, x, rows) || overlap(place, pairs, ids, pairs))
        return fail(IQK_E_ARG, "xs must not overlap x, nor place ids");
    iqk::SortLaunch L{x, dtype, ids, T, k, (int)E, n, (int32_t*)workspace, xs, offsets, place};
    hipError_t e = iqk::launch_sort(L, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "sort launch");
    return ok();
}

int iqk_moe_unsort(const void* ys, int ys_dtype, const int32_t* place, const float* weights, int64_t T, int k, int64_t n,
                   void* y, int y_dtype, void* stream) {
    int rc = check_pairs(T, k);
    if (!rc) rc = check_width(n);
    if (rc) return rc;
    if (!is_float(ys_dtype) || !is_float(y_dtype)) return fail(IQK_E_ARG, "ys and y must be IQK_F32, IQK_F16 or IQK_BF16");
    if (T == 0) return ok();
    if (!ys || !place || !y) return fail(IQK_E_ARG, "null ys, place or y");
    if (!typed(ys, ys_dtype) || !typed(y, y_dtype)) return fail(IQK_E_ARG, "ys and y must be aligned to their types");
    if (!aligned(place, 4) || !aligned(weights, 4)) return fail(IQK_E_ARG, "place and weights must be 4-byte aligned");
    iqk::UnsortLaunch L{ys, ys_dtype, place, weights, T, k, n, y, y_dtype};
    hipError_t e = iqk::launch_unsort(L, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "unsort launch");
    return ok();
}

int iqk_moe_unsort_grad(const void* dy, int dy_dtype, const void* ys, int ys_dtype, const int32_t* place, const float* weights,
                        int64_t T, int k, int64_t n, void* d_ys, float* d_weights, void* stream) {
    int rc = check_pairs(T, k);
    if (!rc) rc = check_width(n);
    if (rc) return rc;
    if (!is_float(ys_dtype) || !is_float(dy_dtype)) return fail(IQK_E_ARG, "ys and dy must be IQK_F32, IQK_F16 or IQK_BF16");
    if (T == 0) return ok();
    if (!d_ys && !d_weights) return fail(IQK_E_ARG, "neither d_ys nor d_weights");
    if (!dy || !place || (d_weights && !ys)) return fail(IQK_E_ARG, "null dy, place or ys");
    if (!typed(dy, dy_dtype) || !typed(ys, ys_dtype) || !typed(d_ys, ys_dtype))
        return fail(IQK_E_ARG, "dy, ys and d_ys must be aligned to their types");
    if (!aligned(place, 4) || !aligned(weights, 4) || !aligned(d_weights, 4))
        return fail(IQK_E_ARG, "place, weights and d_weights must be 4-byte aligned");
    iqk::UnsortGradLaunch L{dy, dy_dtype, ys, ys_dtype, place, weights, T, k, n, d_ys, d_weights};
    hipError_t e = iqk::launch_unsort_grad(L, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "unsort gradient launch");
    return ok();
}

int iqk_block_norm(const iqk_block* b, void* r, void* h, void* stream) {
    int rc = check_block(b);
    if (rc) return rc;
    if (b->T == 0) return ok();
    if ((r != nullptr) != (b->y != nullptr)) return fail(IQK_E_ARG, "r goes with y, and only with it");
    if ((h != nullptr) != (b->next_weight != nullptr)) return fail(IQK_E_ARG, "h goes with next_weight, and only with it");
    if (r == h) return fail(IQK_E_ARG, "r and h must differ");
    if (!typed(r, b->dtype) || !typed(h, b->dtype)) return fail(IQK_E_ARG, "r and h must be aligned to their type");
    const size_t values = (size_t)(b->T * b->n), bytes = values * size_of(b->dtype), y_bytes = values * size_of(b->y_dtype);
    for (const void* p : {r, h}) {
        // (row by row a result may take its input's place; moved by part of a row, or in a type of another size, it would
        // lie over rows that another workgroup has yet to read)
        if ((p != b->x && overlap(p, bytes, b->x, bytes)) || ((p != b->y || b->y_dtype != b->dtype) && overlap(p, bytes, b->y, y_bytes)))
            return fail(IQK_E_ARG, "r and h may be x, or y of x's type, but not overlap them otherwise");
    }
    if (overlap(r, bytes, h, bytes)) return fail(IQK_E_ARG, "r and h must not overlap");
    hipError_t e = iqk::launch_norm(*b, r, h, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "norm launch");
    return ok();
}

int iqk_block_norm_grad_workspace(const iqk_block* b, size_t* bytes) {
    if (!bytes) return fail(IQK_E_ARG, "null pointer");
    if (!b) return fail(IQK_E_ARG, "null block descriptor");
    if (b->T < 0 || b->T > kMaxRows) return fail(IQK_E_ARG, "T = %lld outside [0, 2^24]", (long long)b->T);
    if (b->n < 1 || b->n > kMaxNorm) return fail(IQK_E_ARG, "n = %lld outside [1, 8192]", (long long)b->n);
    const int columns = (b->post_weight != nullptr) + (b->next_weight != nullptr) + (b->gate_kind == IQK_GATE_CHANNEL);
    *bytes = (size_t)iqk::norm_sums_bytes(b->T, b->n, columns);
    return ok();
}

int iqk_block_norm_grad(const iqk_block* b, const void* dr, const void* dh, void* dx, void* dy, void* d_post, void* d_gate,
                        void* d_next, void* workspace, size_t ws_bytes, void* stream) {
    int rc = check_block(b);
    if (rc) return rc;
    if (dh && !b->next_weight) return fail(IQK_E_ARG, "dh needs next_weight");
    if (b->T > 0 && !dr && !dh) return fail(IQK_E_ARG, "neither dr nor dh");
    if ((b->T > 0 && dy && !b->y) || (d_post && !b->post_weight) || (d_next && !b->next_weight) ||
        (d_gate && b->gate_kind == IQK_GATE_NONE))
        return fail(IQK_E_ARG, "a gradient of an input that is null");
    if (!typed(dr, b->dtype) || !typed(dh, b->dtype) || !typed(dx, b->dtype) || (dy && !typed(dy, b->y_dtype)) ||
        (d_post && !typed(d_post, b->weight_dtype)) || (d_next && !typed(d_next, b->weight_dtype)) ||
        (d_gate && !typed(d_gate, b->gate_dtype)))
        return fail(IQK_E_ARG, "gradients must be aligned to their types");
    const bool channel = b->gate_kind == IQK_GATE_CHANNEL && d_gate;
    const int columns = (d_post != nullptr) + (d_next != nullptr) + channel;
    const size_t need = (size_t)iqk::norm_sums_bytes(b->T, b->n, columns);
    if (ws_bytes < need || (need && !workspace))
        return fail(IQK_E_SIZE, "workspace needs %zu bytes (got %zu)", need, workspace ? ws_bytes : 0);
    if (!aligned(workspace, 16)) return fail(IQK_E_ARG, "workspace must be 16-byte aligned");
    if (b->T == 0 && columns == 0) return ok();
    iqk::NormGradOut o{dr, dh, dx, dy, d_post, d_gate, d_next};
    hipError_t e = iqk::launch_norm_grad(*b, o, (float*)workspace, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "norm gradient launch");
    return ok();
}

}  // extern "C"
