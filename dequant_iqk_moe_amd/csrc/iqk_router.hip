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
// A row of L lanes owns one token, L = 64 (few tokens: the shortest chain) or 16
// (many: four tokens per wave, whose instructions then do four tokens' work).
// Lane i of it holds the V consecutive experts from i V, so its loads are wide,
// the lowest id among equals is the lowest lane's, and a group is a number of
// whole lanes.  Each lane keeps its own best; a selection step is a maximum
// over the row (DPP), one ballot, and a new best in the lane that won.  Scores
// are computed only for the experts whose score something needs: a choice by
// logits with weights divided by their sum needs those of the chosen alone.
// No LDS, no barrier; all arithmetic is float32.  Bound: vector instructions,
// not bytes: 16384 tokens of 256 bfloat16 logits, k = 6, take 9.6 us where
// their 9 MB would take 1.9, and issue 4.05e6 of them, 74 % of the SIMDs' busy
// cycles by the counters; one token 5.7 us, a launch and a chain of k maxima.
#include "iqk_layer.h"

namespace iqk {
namespace {

constexpr int kRouterWaves = 4;          // waves per workgroup
constexpr int64_t kManyTokens = 8192;    // tokens from which rows of 16 lanes are taken

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

// Maximum and sum over a row of L = 16 or 64 lanes, the result in every lane.
// Four rotations within rows of 16 lanes; for 64, two broadcasts of a row's
// last lane to the rows after it, after which lane 63 holds the result.
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ float dpp_or(float v, float otherwise) {
    return __uint_as_float(__builtin_amdgcn_update_dpp(__float_as_uint(otherwise), __float_as_uint(v), CTRL, ROW_MASK,
                                                       0xF, false));
}
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return dpp_or<CTRL, 0xF>(v, v);
}
constexpr int kRor1 = 0x121, kRor2 = 0x122, kRor4 = 0x124, kRor8 = 0x128, kBcast15 = 0x142, kBcast31 = 0x143;
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;  // quad permutes, mirrors of 8 and 16
__device__ __forceinline__ float lane_value(float v, int lane) {
    return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), lane));
}
template <int L>
__device__ __forceinline__ float row_max(float v) {
    v = fmaxf(v, dpp<kRor8>(v));
    v = fmaxf(v, dpp<kRor4>(v));
    v = fmaxf(v, dpp<kRor2>(v));
    v = fmaxf(v, dpp<kRor1>(v));
    if constexpr (L == 64) {
        v = fmaxf(v, dpp_or<kBcast15, 0xA>(v, v));
        v = fmaxf(v, dpp_or<kBcast31, 0xC>(v, v));
        v = lane_value(v, 63);
    }
    return v;
}
template <int L>
__device__ __forceinline__ float row_sum(float v) {
    v += dpp<kRor8>(v);
    v += dpp<kRor4>(v);
    v += dpp<kRor2>(v);
    v += dpp<kRor1>(v);
    if constexpr (L == 64) {
        v += dpp_or<kBcast15, 0xA>(v, 0.f);
        v += dpp_or<kBcast31, 0xC>(v, 0.f);
        v = lane_value(v, 63);
    }
    return v;
}
// The ballot bits of this lane's row, from bit 0.
template <int L>
__device__ __forceinline__ uint64_t row_bits(uint64_t ballot, int lane) {
    if constexpr (L == 64) return ballot;
    else return (uint32_t)(ballot >> (lane & 48)) & 0xFFFFu;
}
__device__ __forceinline__ float wave_max(float v) { return row_max<64>(v); }
__device__ __forceinline__ float wave_sum(float v) { return row_sum<64>(v); }

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

// V consecutive logits from element i, of which `left` are inside the row;
// the others read -inf.  `wide`: rows are multiples of 16 bytes, so aligned
// words of at most 16 bytes are all inside or all outside.
template <int V, int DT>
__device__ __forceinline__ void load_logits(const void* p, int64_t i, int left, bool wide, float (&l)[V]) {
    constexpr int kSize = DT == IQK_F32 ? 4 : 2;
    constexpr int kWord = V * kSize < 16 ? V * kSize : 16, kPer = kWord / kSize;
#pragma unroll
    for (int v = 0; v < V; ++v) l[v] = neg_inf();
    if constexpr (kWord >= 4) {
        if (wide) {
#pragma unroll
            for (int c = 0; c < V; c += kPer) {
                if (c >= left) continue;
                uint32_t w[kWord / 4];
                __builtin_memcpy(w, __builtin_assume_aligned((const char*)p + (i + c) * kSize, kWord), kWord);
#pragma unroll
                for (int u = 0; u < kPer; ++u) {
                    if constexpr (DT == IQK_F32) l[c + u] = __uint_as_float(w[u]);
                    if constexpr (DT == IQK_BF16) l[c + u] = __uint_as_float(u & 1 ? w[u / 2] & 0xFFFF0000u : w[u / 2] << 16);
                    if constexpr (DT == IQK_F16) l[c + u] = (float)__builtin_bit_cast(_Float16, (uint16_t)(w[u / 2] >> (16 * (u & 1))));
                }
            }
            return;
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (v < left) l[v] = load_logit<DT>(p, i + v);
}

// The lane's best value and where it first stands.
template <int V>
__device__ __forceinline__ float lane_best(const float (&c)[V], int* at) {
    float m = c[0];
    int i = 0;
#pragma unroll
    for (int v = 1; v < V; ++v) {
        const bool more = c[v] > m;
        m = more ? c[v] : m;
        i = more ? v : i;
    }
    *at = i;
    return m;
}

template <int L, int V, int DT>
__global__ __launch_bounds__(64 * kRouterWaves) void router_kernel(RouterLaunch p) {
    const int lane = threadIdx.x & 63, sub = lane & (L - 1);
    const int64_t row = ((int64_t)blockIdx.x * (64 * kRouterWaves) + threadIdx.x) / L;
    const bool there = row < p.T;  // (a wave's rows past the last work on a copy of it and write nothing)
    const int64_t t = there ? row : p.T - 1;
    const int E = p.E, e0 = sub * V, left = E - e0;
    const bool softmax = p.scoring == IQK_SOFTMAX;
    float l[V], s[V], c[V];
    load_logits<V, DT>(p.logits, t * E + e0, left, p.wide, l);
    bool bad = false;  // a NaN, or an infinite logit under softmax
    float top = neg_inf();
#pragma unroll
    for (int v = 0; v < V; ++v) {
        bad |= l[v] != l[v] || (softmax && l[v] == __builtin_inff());
        top = fmaxf(top, l[v]);
        c[v] = l[v];
    }
    // scores of all experts, where the choice or the weights need them
    const bool two = p.n_group > 1 && p.group_top == 2;
    // A group's worth of two: half of their sum where a bias takes part, which orders groups alike (halving is exact)
    // and does not leave float32 with biases at its ends, so that only a group without an expert is worth -inf.
    const float part = p.bias ? 0.5f : 1.f;
    float total = 1.f;
    if (p.bias || two || (softmax && !p.renorm)) {
        if (softmax) {
            top = row_max<L>(top);
            float sum = 0.f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                s[v] = l[v] == neg_inf() ? 0.f : expf(l[v] - top);
                sum += s[v];
            }
            total = row_sum<L>(sum);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) s[v] = sigmoid(l[v]);
        }
    }
    // what the choice goes by; an expert whose logit or bias is -inf is out (c = -inf)
    if (p.bias) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float b = v < left ? p.bias[e0 + v] : 0.f;
            bad |= b != b;
            c[v] = l[v] != neg_inf() ? (softmax ? s[v] / total : s[v]) + b : l[v];
        }
    }
    if (p.n_group > 1) {
        const int per = E / p.n_group;
        if (p.lane_groups) {  // a group is 1, 2, 4, 8 or 16 whole lanes
            const int lanes = per / V;
            float a = neg_inf(), b = neg_inf();  // the lane's best two
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float w = two && !p.bias && c[v] != neg_inf() ? s[v] : c[v];
                b = fmaxf(b, fminf(a, w));
                a = fmaxf(a, w);
            }
            auto merge = [&](float oa, float ob) {
                b = fmaxf(fminf(a, oa), fmaxf(b, ob));
                a = fmaxf(a, oa);
            };
            if (lanes > 1) merge(dpp<kXor1>(a), dpp<kXor1>(b));
            if (lanes > 2) merge(dpp<kXor2>(a), dpp<kXor2>(b));
            if (lanes > 4) merge(dpp<kHalfMirror>(a), dpp<kHalfMirror>(b));
            if (lanes > 8) merge(dpp<kMirror>(a), dpp<kMirror>(b));
            float worth = a;
            if (two) worth = part * a + (b != neg_inf() ? part * b : 0.f);
            if (left <= 0) worth = neg_inf();
            bool stays = false;
            for (int i = 0; i < p.topk_group; ++i) {
                const float m = row_max<L>(worth);
                const uint64_t best = row_bits<L>(__ballot(worth == m), lane);
                const int first = __builtin_ctzll(best | (1ull << 63));
                if (m != neg_inf() && sub / lanes == first / lanes) {
                    stays = true;
                    worth = neg_inf();
                }
            }
#pragma unroll
            for (int v = 0; v < V; ++v) c[v] = stays ? c[v] : neg_inf();
        } else if constexpr (L == 64) {
            // a group's worth in lane g, -inf where none of its experts is in
            float worth = neg_inf();
            for (int g = 0; g < p.n_group; ++g) {
                float a[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const bool in = e0 + v >= g * per && e0 + v < (g + 1) * per && c[v] != neg_inf();
                    a[v] = !in ? neg_inf() : (two && !p.bias ? s[v] : c[v]);
                }
                int at;
                float best = lane_best<V>(a, &at);
                float w = row_max<64>(best);
                if (two) {
                    const int first = __builtin_ctzll(__ballot(best == w));
                    if (lane == first) {
#pragma unroll
                        for (int v = 0; v < V; ++v) a[v] = v == at ? neg_inf() : a[v];
                        best = lane_best<V>(a, &at);
                    }
                    const float second = row_max<64>(best);
                    w = part * w + (second != neg_inf() ? part * second : 0.f);
                }
                if (lane == g) worth = w;
            }
            uint64_t stay = 0;  // the groups that stay, as a mask of group numbers
            for (int i = 0; i < p.topk_group; ++i) {
                const float m = row_max<64>(worth);
                if (m == neg_inf()) break;
                const int g = __builtin_ctzll(__ballot(worth == m));
                stay |= 1ull << g;
                if (lane == g) worth = neg_inf();
            }
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (v >= left || !((stay >> ((e0 + v) / per)) & 1)) c[v] = neg_inf();
        }
    }
    // the k best: slot j's id goes out from the lane that holds the expert, its score (or logit) to lane j
    const bool whole_row_bad = row_bits<L>(__ballot(bad), lane) != 0;
    int at;
    float best = lane_best<V>(c, &at);
    float value = 0.f, first_id = -1.f;
    int found = 0;
    int32_t* ids = p.ids + t * p.k;
    for (int j = 0; j < p.k; ++j) {
        const float m = row_max<L>(best);
        const bool any = m != neg_inf();
        if (!__ballot(any)) break;
        const uint64_t bits = row_bits<L>(__ballot(any && best == m), lane);
        const bool won = any && sub == __builtin_ctzll(bits | (1ull << 63));
        float got = m;  // the choice went by logits: the winner's logit
        if (p.bias) {
            float mine = neg_inf();  // its score
#pragma unroll
            for (int v = 0; v < V; ++v) mine = won && v == at ? s[v] : mine;
            got = row_max<L>(mine);
        }
        if (j == 0) first_id = row_max<L>(won ? (float)(e0 + at) : -1.f);
        if (won) {
            if (there && !whole_row_bad) ids[j] = e0 + at;
#pragma unroll
            for (int v = 0; v < V; ++v) c[v] = v == at ? neg_inf() : c[v];
            best = lane_best<V>(c, &at);
        }
        found += any;
        value = any && sub == j ? got : value;
    }
    const bool filled = sub < found;
    float w = 0.f;
    if (p.bias) {  // value is a score (softmax: before its division by the total)
        const float d = p.renorm ? row_sum<L>(filled ? value : 0.f) : total;
        w = d > 0.f ? value / d : 0.f;
    } else if (softmax) {  // value is a logit; renorm: the row's other experts cancel
        const float most = p.renorm ? row_max<L>(filled ? value : neg_inf()) : top;
        const float x = filled ? expf(value - most) : 0.f;
        w = x / (p.renorm ? row_sum<L>(x) : total);
    } else {
        const float x = filled ? sigmoid(value) : 0.f;
        const float d = p.renorm ? row_sum<L>(x) : 1.f;
        w = d > 0.f ? x / d : 0.f;
    }
    // slots that no expert is left for repeat the first one at weight zero
    for (int j = sub; j < p.k && there; j += L) {
        if (whole_row_bad) {
            ids[j] = -1;
            p.weights[t * p.k + j] = __builtin_nanf("");
        } else {
            if (j >= found) ids[j] = (int)first_id;
            p.weights[t * p.k + j] = j < found ? w * p.scale : 0.f;
        }
    }
}

// Gradient with respect to the logits.  With g_j = scale * dL/dw_j and
//   renorm:    ds_j = (g_j - sum_m g_m s_m / D) / D,   D = sum_m s_m
//   otherwise: ds_j = g_j
// sigmoid: dl = ds * s (1 - s) at the chosen experts (with renorm as w_j (1 - s_j)
// (g_j - sum_m g_m w_m), w_m = s_m / D), zero elsewhere; softmax
// without renorm: dl_e = p_e (ds_e - sum_j ds_j p_j) for every expert, with
// renorm the second term is zero and w is the softmax of the chosen logits
// alone: dl_j = w_j (g_j - sum_m g_m w_m).  Only softmax without renorm reads
// the whole row of logits; the others read the chosen ones.  One wave owns one
// token, lane e % 64 the logit e, so rows are read and written whole and the
// sums stay in the wave.  512 tokens of 256 float32 logits: 3.6 us, a launch;
// 8191 of 160 bfloat16 logits: 6.4 us for 5 MB (1.2 us at a copy's rate), bound
// by vector instructions (2.4e6, 74 % of the SIMDs' busy cycles).
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
        for (int v = 0; v < V; ++v) o[v] = x[v] == 0.f || !__ballot(in) ? 0.f : -(x[v] / total) * dot;
    } else {
        if (p.scoring == IQK_SOFTMAX) {
            const float top = wave_max(l);
            const float e = in && l != neg_inf() ? expf(l - top) : 0.f;
            const float sum = wave_sum(e);
            const float w = sum > 0.f ? e / sum : 0.f;
            d = w * (g - wave_sum(g * w));
        } else {
            if (p.renorm) {
                // dl_j = w_j (1 - s_j) (g_j - sum_m g_m w_m) with w_j = s_j / D: no factor leaves float32 where D is
                // tiny (a 1 / D by itself would); 1 - s_j = 1 / (1 + exp(l_j))
                const float s = in ? sigmoid(l) : 0.f;
                const float D = wave_sum(s);
                const float w = D > 0.f ? s / D : 0.f;
                const float dot = wave_sum(g * w);
                d = in ? w * sigmoid(-l) * (g - dot) : 0.f;
            } else {
                // s = 1 / (1 + exp(-l)), s (1 - s) = q / (1 + q)^2 with q = exp(-|l|)
                const float q = expf(-fabsf(l));
                d = in ? g * (q / ((1.f + q) * (1.f + q))) : 0.f;
            }
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
    RouterLaunch p = a;
    const int size = a.dtype == IQK_F32 ? 4 : 2;
    p.wide = (int64_t)a.E * size % 16 == 0 && (uintptr_t)a.logits % 16 == 0;
    const int per = a.E / a.n_group;
    by_width(a.E, [&](auto v64) {
        constexpr int V64 = decltype(v64)::value, V16 = 4 * V64;  // experts per lane of 64 and of 16
        // whether a group is 2^i <= 16 whole lanes
        auto whole = [&](int V) { return per % V == 0 && per / V <= 16 && (per / V & (per / V - 1)) == 0; };
        // Rows of 16 lanes: four tokens for little more than one's instructions, in a chain a few times as long, so
        // they win where tokens far outnumber the card's 8192 resident waves (256 experts, softmax, k = 6: 4096
        // tokens 6.9 us against 5.3 with rows of 64, 16384 tokens 8.8 against 12.5 a queued call; 512 experts gain nothing).
        const bool many = a.T >= kManyTokens && V16 <= 16 && a.k <= 16 && (a.n_group == 1 || whole(V16));
        p.lane_groups = a.n_group > 1 && whole(many ? V16 : V64);
        by_dtype(a.dtype, [&](auto dt) {
            constexpr int DT = decltype(dt)::value;
            const int64_t lanes = a.T * (many ? 16 : 64);
            const dim3 grid((unsigned)((lanes + 64 * kRouterWaves - 1) / (64 * kRouterWaves))), block(64 * kRouterWaves);
            if constexpr (V16 <= 16) {
                if (many) hipLaunchKernelGGL((router_kernel<16, V16, DT>), grid, block, 0, s, p);
            }
            if (!many) hipLaunchKernelGGL((router_kernel<64, V64, DT>), grid, block, 0, s, p);
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
