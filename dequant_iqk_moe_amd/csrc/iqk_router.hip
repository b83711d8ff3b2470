// iqk_router.hip -- expert selection from router logits, and its gradient.
//
// The "Surface" section of the "mlx-iqk" package description takes the
// routing (indices, and the weights that sum the k slots) as inputs of the
// switch-linear call; these kernels make them from a router's logits.
//
//   s_e = 1 / (1 + exp(-l_e))  or  exp(l_e - max l) / sum exp(l - max l)
//   c_e = s_e + b_e with a bias, else l_e (both scores grow with the logit, so
//         choosing by the logit chooses the same experts and never ties two
//         logits that differ)
//   groups of E / G consecutive experts: a group counts its best c, or the sum
//         of its best two (of the scores where there is no bias); the best
//         `topk_group` groups stay, equal groups in favour of the lowest
//   ids = the k largest c of the groups that stay, equal c in favour of the
//         lowest id; w_j = scale * s_j / D, D = the sum of the chosen s or 1
//
// One wave owns one token: expert v * 64 + lane is register v of a lane, so
// the row is loaded and the gradient stored 64 consecutive values at a time,
// and a selection step is one wave-wide maximum (DPP) and one ballot per
// register, whose first set bit is the lowest id.  No LDS, no barrier.  All
// arithmetic is float32.
#include "iqk_internal.h"

namespace iqk {
namespace {

constexpr int kRouterWaves = 4;  // waves (tokens) per workgroup

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

// Maximum and sum over the 64 lanes of a wave, the result in every lane.  The
// first four steps rotate within rows of 16 lanes, the last two broadcast a
// row's last lane to the rows after it; lane 63 then holds the result.
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ float dpp_or(float v, float otherwise) {
    return __uint_as_float(__builtin_amdgcn_update_dpp(__float_as_uint(otherwise), __float_as_uint(v), CTRL, ROW_MASK,
                                                       0xF, false));
}
__device__ __forceinline__ float wave_max(float v) {
    v = fmaxf(v, dpp_or<0x128, 0xF>(v, v));  // row_ror:8
    v = fmaxf(v, dpp_or<0x124, 0xF>(v, v));  // row_ror:4
    v = fmaxf(v, dpp_or<0x122, 0xF>(v, v));  // row_ror:2
    v = fmaxf(v, dpp_or<0x121, 0xF>(v, v));  // row_ror:1
    v = fmaxf(v, dpp_or<0x142, 0xA>(v, v));  // row_bcast:15 into rows 1 and 3
    v = fmaxf(v, dpp_or<0x143, 0xC>(v, v));  // row_bcast:31 into rows 2 and 3
    return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 63));
}
__device__ __forceinline__ float wave_sum(float v) {
    v += dpp_or<0x128, 0xF>(v, 0.f);
    v += dpp_or<0x124, 0xF>(v, 0.f);
    v += dpp_or<0x122, 0xF>(v, 0.f);
    v += dpp_or<0x121, 0xF>(v, 0.f);
    v += dpp_or<0x142, 0xA>(v, 0.f);
    v += dpp_or<0x143, 0xC>(v, 0.f);
    return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 63));
}
__device__ __forceinline__ float lane_value(float v, int lane) {
    return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), lane));
}

template <int DT>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
    if constexpr (DT == IQK_F32) return ((const float*)p)[i];
    if constexpr (DT == IQK_F16) return (float)((const _Float16*)p)[i];
    return __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16);
}
template <int DT>
__device__ __forceinline__ void store_logit(void* p, int64_t i, float v) {
    if constexpr (DT == IQK_F32) ((float*)p)[i] = v;
    if constexpr (DT == IQK_F16) ((_Float16*)p)[i] = (_Float16)v;
    if constexpr (DT == IQK_BF16) {
        const uint32_t u = __float_as_uint(v);
        ((uint16_t*)p)[i] = (u & 0x7FFFFFFFu) > 0x7F800000u ? 0x7FC0u : (uint16_t)((u + 0x7FFFu + ((u >> 16) & 1u)) >> 16);
    }
}

__device__ __forceinline__ float sigmoid(float l) { return 1.0f / (1.0f + expf(-l)); }

// Largest of the V registers of all lanes and where it first stands.  `m` is
// -inf when nothing is left.
template <int V>
__device__ __forceinline__ float wave_best(const float (&c)[V], int* reg, int* lane) {
    float m = c[0];
#pragma unroll
    for (int v = 1; v < V; ++v) m = fmaxf(m, c[v]);
    m = wave_max(m);
    *reg = V;
    *lane = 0;
#pragma unroll
    for (int v = V - 1; v >= 0; --v) {
        const uint64_t b = __ballot(c[v] == m);
        if (b) {
            *reg = v;
            *lane = __builtin_ctzll(b);
        }
    }
    return m;
}

template <int V, int DT>
__global__ __launch_bounds__(64 * kRouterWaves) void router_kernel(RouterLaunch p) {
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * kRouterWaves + (threadIdx.x >> 6);
    if (t >= p.T) return;
    const int E = p.E;
    float l[V], s[V], c[V];
    bool bad = false;  // a NaN, or an infinite logit under softmax
    float top = neg_inf();
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = v * 64 + lane;
        l[v] = e < E ? load_logit<DT>(p.logits, t * E + e) : neg_inf();
        c[v] = p.bias && e < E ? p.bias[e] : 0.f;
        bad |= l[v] != l[v] || c[v] != c[v] || (p.scoring == IQK_SOFTMAX && l[v] == __builtin_inff());
        top = fmaxf(top, l[v]);
    }
    if (__ballot(bad)) {
        if (lane < p.k) {
            p.ids[t * p.k + lane] = -1;
            p.weights[t * p.k + lane] = __builtin_nanf("");
        }
        return;
    }
    float total = 1.f;
    if (p.scoring == IQK_SOFTMAX) {
        top = wave_max(top);
        float sum = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            s[v] = l[v] == neg_inf() ? 0.f : expf(l[v] - top);
            sum += s[v];
        }
        total = wave_sum(sum);
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) s[v] = sigmoid(l[v]);
    }
    // what the choice goes by; an expert whose logit or bias is -inf is out (c = -inf)
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const float sv = p.scoring == IQK_SOFTMAX ? s[v] / total : s[v];
        c[v] = p.bias && l[v] != neg_inf() ? sv + c[v] : l[v];
    }
    if (p.n_group > 1) {
        // a group's worth in lane g, -inf where none of its experts is in
        const int per = E / p.n_group;
        float worth = neg_inf();
        for (int g = 0; g < p.n_group; ++g) {
            float a[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int e = v * 64 + lane;
                const bool in = e >= g * per && e < (g + 1) * per && c[v] != neg_inf();
                a[v] = !in ? neg_inf() : (p.group_top == 2 && !p.bias ? s[v] : c[v]);
            }
            int reg, ln;
            float w = wave_best<V>(a, &reg, &ln);
            if (p.group_top == 2) {
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (v == reg && lane == ln) a[v] = neg_inf();
                const float second = wave_best<V>(a, &reg, &ln);
                if (second != neg_inf()) w += second;
            }
            if (lane == g) worth = w;
        }
        // the groups that stay, as a mask of group numbers
        uint64_t stay = 0;
        for (int i = 0; i < p.topk_group; ++i) {
            const float m = wave_max(worth);
            if (m == neg_inf()) break;
            const int g = __builtin_ctzll(__ballot(worth == m));
            stay |= 1ull << g;
            if (lane == g) worth = neg_inf();
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = v * 64 + lane;
            if (e >= E || !((stay >> (e / per)) & 1)) c[v] = neg_inf();
        }
    }
    // the k best; slot j's id, score and logit in lane j
    int id = -1;
    float score = 0.f, logit = neg_inf();
    int found = 0;
    for (; found < p.k; ++found) {
        int reg, ln;
        if (wave_best<V>(c, &reg, &ln) == neg_inf()) break;
        float sv = 0.f, lv = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (v == reg) {
                sv = lane_value(s[v], ln);
                lv = lane_value(l[v], ln);
                if (lane == ln) c[v] = neg_inf();
            }
        }
        if (lane == found) {
            id = reg * 64 + ln;
            score = sv;
            logit = lv;
        }
    }
    const bool filled = lane < found;
    float w = 0.f;
    if (p.scoring == IQK_SOFTMAX && p.renorm) {
        // exp(l - the largest chosen logit): the row's other experts cancel
        const float best = wave_max(logit);
        const float e = filled ? expf(logit - best) : 0.f;
        w = e / wave_sum(e);
    } else if (p.renorm) {
        const float d = wave_sum(filled ? score : 0.f);
        w = d > 0.f ? score / d : 0.f;
    } else {
        w = score / total;
    }
    // slots that no expert is left for repeat the first one at weight zero
    const int first = __builtin_amdgcn_readlane(id, 0);
    if (lane < p.k) {
        p.ids[t * p.k + lane] = filled ? id : first;
        p.weights[t * p.k + lane] = filled ? w * p.scale : 0.f;
    }
}

// Gradient with respect to the logits.  With g_j = scale * dL/dw_j and
//   renorm:    ds_j = (g_j - sum_m g_m s_m / D) / D,   D = sum_m s_m
//   otherwise: ds_j = g_j
// sigmoid: dl = ds * s (1 - s) at the chosen experts, zero elsewhere; softmax
// without renorm: dl_e = p_e (ds_e - sum_j ds_j p_j) for every expert, with
// renorm the second term is zero and w is the softmax of the chosen logits
// alone: dl_j = w_j (g_j - sum_m g_m w_m).  Only softmax without renorm reads
// the whole row of logits; the others read the chosen ones.
template <int V, int DT>
__global__ __launch_bounds__(64 * kRouterWaves) void router_grad_kernel(RouterGradLaunch p) {
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * kRouterWaves + (threadIdx.x >> 6);
    if (t >= p.T) return;
    const int E = p.E;
    // slot j in lane j; a slot outside [0, E), and one that repeats the first
    // (a slot the selection could not fill), takes no part
    int id = lane < p.k ? p.ids[t * p.k + lane] : -1;
    const int first = __builtin_amdgcn_readlane(id, 0);
    if (id < 0 || id >= E || (lane > 0 && id == first)) id = -1;
    const bool in = id >= 0;
    const float g = in ? p.d_weights[t * p.k + lane] * p.scale : 0.f;
    const float l = in ? load_logit<DT>(p.logits, t * E + id) : neg_inf();
    float o[V];
    float d = 0.f;  // this slot's gradient, at its expert
    if (p.scoring == IQK_SOFTMAX && !p.renorm) {
        float x[V];
        float top = neg_inf();
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = v * 64 + lane;
            x[v] = e < E ? load_logit<DT>(p.logits, t * E + e) : neg_inf();
            top = fmaxf(top, x[v]);
        }
        top = wave_max(top);
        float sum = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            x[v] = x[v] == neg_inf() ? 0.f : expf(x[v] - top);
            sum += x[v];
        }
        const float total = wave_sum(sum);
        const float pr = in && l != neg_inf() ? expf(l - top) / total : 0.f;
        const float dot = wave_sum(g * pr);
        d = pr * (g - dot);
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] = x[v] == 0.f ? 0.f : -(x[v] / total) * dot;
    } else {
        if (p.scoring == IQK_SOFTMAX) {
            const float top = wave_max(l);
            const float e = in && l != neg_inf() ? expf(l - top) : 0.f;
            const float sum = wave_sum(e);
            const float w = sum > 0.f ? e / sum : 0.f;
            d = w * (g - wave_sum(g * w));
        } else {
            // s = 1 / (1 + exp(-l)), s (1 - s) = q / (1 + q)^2 with q = exp(-|l|)
            const float q = expf(-fabsf(l));
            const float slope = in ? q / ((1.f + q) * (1.f + q)) : 0.f;
            float ds = g;
            if (p.renorm) {
                const float s = in ? sigmoid(l) : 0.f;
                const float D = wave_sum(s);
                const float dot = wave_sum(g * s);
                ds = D > 0.f ? (g - dot / D) / D : 0.f;
            }
            d = ds * slope;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] = 0.f;
    }
    for (int j = 0; j < p.k; ++j) {
        const int e = __builtin_amdgcn_readlane(id, j);
        const float dv = lane_value(d, j);
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (e == v * 64 + lane) o[v] = dv;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = v * 64 + lane;
        if (e < E) store_logit<DT>(p.d_logits, t * E + e, o[v]);
    }
}

// Registers per lane for E experts: 1, 2, 4, 8 or 16 (E <= 1024).
template <class F>
void by_width(int E, F f) {
    if (E <= 64) f(std::integral_constant<int, 1>{});
    else if (E <= 128) f(std::integral_constant<int, 2>{});
    else if (E <= 256) f(std::integral_constant<int, 4>{});
    else if (E <= 512) f(std::integral_constant<int, 8>{});
    else f(std::integral_constant<int, 16>{});
}
template <class F>
void by_dtype(int dt, F f) {
    if (dt == IQK_F32) f(std::integral_constant<int, IQK_F32>{});
    else if (dt == IQK_F16) f(std::integral_constant<int, IQK_F16>{});
    else f(std::integral_constant<int, IQK_BF16>{});
}

}  // namespace

hipError_t launch_router(const RouterLaunch& a, hipStream_t s) {
    const unsigned blocks = (unsigned)((a.T + kRouterWaves - 1) / kRouterWaves);
    by_width(a.E, [&](auto v) {
        by_dtype(a.dtype, [&](auto dt) {
            hipLaunchKernelGGL((router_kernel<decltype(v)::value, decltype(dt)::value>), dim3(blocks),
                               dim3(64 * kRouterWaves), 0, s, a);
        });
    });
    return hipGetLastError();
}

hipError_t launch_router_grad(const RouterGradLaunch& a, hipStream_t s) {
    const unsigned blocks = (unsigned)((a.T + kRouterWaves - 1) / kRouterWaves);
    by_width(a.E, [&](auto v) {
        by_dtype(a.dtype, [&](auto dt) {
            hipLaunchKernelGGL((router_grad_kernel<decltype(v)::value, decltype(dt)::value>), dim3(blocks),
                               dim3(64 * kRouterWaves), 0, s, a);
        });
    });
    return hipGetLastError();
}

}  // namespace iqk
