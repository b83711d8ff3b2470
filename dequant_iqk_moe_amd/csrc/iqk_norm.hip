// iqk_norm.hip -- the norm behind a block, its gate, the scaled residual and the
// norm before the next block in one pass over the rows, and their gradient.
//
//   u = y s(y) wp            s(v) = (mean v^2 + eps)^-1/2   (u = y without wp)
//   r = alpha x + beta g u
//   h = r s(r) wn            from r before its rounding
//
// Gradient, from dr and dh, with s = s(y), q = s(r):
//   D    = dr + q wn dh - r q^3 / n sum(wn dh r)
//   dx   = alpha D           d_wn = sum_t dh r q
//   dg   = beta D u          (summed over tokens or over the row with g's kind)
//   v    = beta g D wp       d_wp = sum_t beta g D y s
//   dy   = s v - y s^3 / n sum(v y)     (beta g D without wp)
// r is computed again from x and y, so it is not rounded there either, and is
// not read beside them.
//
// Bound: bytes.  A team (a wave, or a workgroup) holds a row in registers as it
// lies in memory; sums go through float32, lanes and waves in a fixed order.
#include <algorithm>

#include "iqk_block.h"
#include "iqk_rows_device.h"

namespace iqk {
namespace {

struct NormParams {
    const void *x, *y, *wp, *g, *wn;
    int w_dtype, g_dtype, g_kind;
    int64_t T;
    int n;
    float alpha, beta, eps;
    void *r, *h;
    const void *dr, *dh;
    void *dx, *dy, *dg;  // dg: a gate of tokens or elements
    float* sums;         // [teams, columns, n]: this team's part of d_wp, d_wn and a channel gate's gradient
    int has_dwp, has_dwn, has_dgc, columns;
};

// Teams of one wave share a workgroup, larger ones are one.
template <int TEAM>
struct Team {
    static constexpr int kWaves = TEAM / 64, kThreads = TEAM == 64 ? 256 : TEAM, kTeams = kThreads / TEAM;
};

// Sums of N values over a team, the same in every lane.  `turn`: sums that
// follow each other take other memory, so that one barrier does for each.
template <int TEAM, int N>
__device__ __forceinline__ void team_sum(float (&v)[N], float (*lds)[2], int turn) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
    if constexpr (TEAM > 64) {
        constexpr int W = TEAM / 64;
        float(*at)[2] = lds + turn * W;
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) at[threadIdx.x >> 6][i] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float t = at[0][i];
#pragma unroll
            for (int w = 1; w < W; ++w) t += at[w][i];
            v[i] = t;
        }
    }
}

__device__ __forceinline__ float inv_rms(float squares, const NormParams& p) {
    return 1.f / sqrtf(squares / (float)p.n + p.eps);
}

// The gate's values at chunk c of row t (1 without a gate).
template <int V>
__device__ __forceinline__ void gate_at(const NormParams& p, int64_t t, int c, int left, float (&g)[V]) {
    if (p.g_kind == IQK_GATE_NONE || left <= 0) {
#pragma unroll
        for (int j = 0; j < V; ++j) g[j] = 1.f;
    } else if (p.g_kind == IQK_GATE_TOKEN) {
        float one[4];
        load_any(p.g, p.g_dtype, t, 1, one);
#pragma unroll
        for (int j = 0; j < V; ++j) g[j] = one[0];
    } else {
        load_any(p.g, p.g_dtype, p.g_kind == IQK_GATE_ELEMENT ? t * p.n + c : c, left, g);
    }
}

// r's values from x's and y's, and u's
template <int V>
__device__ __forceinline__ void mix(const NormParams& p, const float (&x)[V], const float (&y)[V], const float (&wp)[V], float s,
                                    const float (&g)[V], float (&u)[V], float (&r)[V]) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
        u[j] = p.wp ? y[j] * s * wp[j] : y[j];
        r[j] = __builtin_fmaf(p.beta * g[j], u[j], p.alpha * x[j]);
    }
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------

template <int XT, int YT, int TEAM, int NV>
__global__ __launch_bounds__(Team<TEAM>::kThreads) void norm_kernel(NormParams p) {
    using Tm = Team<TEAM>;
    __shared__ float lds[2 * Tm::kWaves][2];
    const int tid = threadIdx.x % TEAM;
    const int64_t t = (blockIdx.y * (int64_t)gridDim.x + blockIdx.x) * Tm::kTeams + threadIdx.x / TEAM;
    if (t >= p.T) return;  // (whole teams: no barrier misses a wave)
    Raw<XT> x[NV];
    Raw<YT> y[NV];
    auto chunk = [&](int i) { return (i * TEAM + tid) * 8; };
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = chunk(i);
        if (p.y) y[i] = load_raw<YT>(p.y, t * p.n + c, p.n - c);
        x[i] = load_raw<XT>(p.x, t * p.n + c, p.n - c);
    }
    float s[1] = {0.f};
    if (p.wp) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float v[8];
            widen_raw(y[i], v);
#pragma unroll
            for (int j = 0; j < 8; ++j) s[0] = __builtin_fmaf(v[j], v[j], s[0]);
        }
        team_sum<TEAM, 1>(s, lds, 0);
        s[0] = inv_rms(s[0], p);
    }
    float r[NV][8], q[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = chunk(i), left = p.n - c;
        widen_raw(x[i], r[i]);
        if (p.y) {
            float g[8], wp[8], u[8], yv[8], xv[8];
            gate_at(p, t, c, left, g);
            if (p.wp) load_any(p.wp, p.w_dtype, c, left, wp);
            widen_raw(y[i], yv);
#pragma unroll
            for (int j = 0; j < 8; ++j) xv[j] = r[i][j];
            mix(p, xv, yv, wp, s[0], g, u, r[i]);
            store_some<XT>(p.r, t * p.n + c, r[i], left);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) q[0] = __builtin_fmaf(r[i][j], r[i][j], q[0]);
    }
    if (!p.h) return;
    team_sum<TEAM, 1>(q, lds, 1);
    q[0] = inv_rms(q[0], p);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = chunk(i), left = p.n - c;
        float w[8];
        load_any(p.wn, p.w_dtype, c, left, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] *= r[i][j] * q[0];
        store_some<XT>(p.h, t * p.n + c, w, left);
    }
}

// ---------------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------------

template <int XT, int YT, int NV>
struct GradRow {
    Raw<XT> x[NV], dr[NV], dh[NV];
    Raw<YT> y[NV];
};

// What the compiler knows of a row's values ends here: it would keep every
// pass's float32 values for the next instead of widening them again (200
// registers where 128 do).
template <class R>
__device__ __forceinline__ void forget(R& r) {
#pragma unroll
    for (auto& w : r.w) asm volatile("" : "+v"(w));
}

// A team takes every teams-th row, so its threads meet the same columns in each:
// its parts of the parameters' gradients stay in registers, and another launch
// joins the teams' parts in their order.  So do the parameters' values.
// HOLD: the row stays in registers; else each pass reads it again, from the L2.
// AHEAD: the next row is asked for while this one is taken.
template <int XT, int YT, int TEAM, int NV, bool HOLD, bool AHEAD>
__global__ __launch_bounds__(Team<TEAM>::kThreads) void norm_grad_kernel(NormParams p) {
    using Tm = Team<TEAM>;
    __shared__ float lds[6 * Tm::kWaves][2];  // (a row's sums and the next one's take turns)
    const int tid = threadIdx.x % TEAM;
    const int64_t team = (int64_t)blockIdx.x * Tm::kTeams + threadIdx.x / TEAM, teams = (int64_t)gridDim.x * Tm::kTeams;
    const int64_t n = p.n;
    auto chunk = [&](int i) { return (i * TEAM + tid) * 8; };
    float wp[NV][8], wn[NV][8], gc[NV][8];  // (ones where there are none)
    float awp[NV][8], awn[NV][8], agc[NV][8];  // sums of their gradients
    auto params = [&](int i) {
        const int c = chunk(i), left = p.n - c;
#pragma unroll
        for (int j = 0; j < 8; ++j) wp[i][j] = wn[i][j] = gc[i][j] = 1.f;
        if (p.wp) load_any(p.wp, p.w_dtype, c, left, wp[i]);
        if (p.wn) load_any(p.wn, p.w_dtype, c, left, wn[i]);
        if (p.g_kind == IQK_GATE_CHANNEL) load_any(p.g, p.g_dtype, c, left, gc[i]);
    };
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int j = 0; j < 8; ++j) awp[i][j] = awn[i][j] = agc[i][j] = 0.f;
        params(i);
    }
    using Row = GradRow<XT, YT, NV>;
    auto load = [&](Row& a, int64_t t, int i) {
        const int c = chunk(i), left = p.n - c;
        const int64_t at = t * n + c;
        a.x[i] = load_raw<XT>(p.x, at, left);
        if (p.y) a.y[i] = load_raw<YT>(p.y, at, left);
        if (p.dr) a.dr[i] = load_raw<XT>(p.dr, at, left);
        if (p.dh) a.dh[i] = load_raw<XT>(p.dh, at, left);
    };
    Row cur, ahead;
    for (Row* a : {&cur, &ahead}) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            for (auto& w : a->y[i].w) w = 0;
            for (auto& w : a->dr[i].w) w = 0;
            for (auto& w : a->dh[i].w) w = 0;
        }
    }
    if (AHEAD && team < p.T) {
#pragma unroll
        for (int i = 0; i < NV; ++i) load(ahead, team, i);
    }
    int odd = 0;
    for (int64_t t = team; t < p.T; t += teams, odd = 3 - odd) {
        if constexpr (AHEAD) {
            cur = ahead;
            if (t + teams < p.T) {
#pragma unroll
                for (int i = 0; i < NV; ++i) load(ahead, t + teams, i);
            }
        } else if constexpr (HOLD) {
#pragma unroll
            for (int i = 0; i < NV; ++i) load(cur, t, i);
        }
        float gt[4] = {1.f, 0.f, 0.f, 0.f};
        if (p.g_kind == IQK_GATE_TOKEN) load_any(p.g, p.g_dtype, t, 1, gt);
        // a chunk's gate and u, and r, widened anew in every pass
        auto gate = [&](int i, float (&g)[8]) {
            if (p.g_kind == IQK_GATE_ELEMENT) {
                load_any(p.g, p.g_dtype, t * n + chunk(i), p.n - chunk(i), g);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) g[j] = gc[i][j] * gt[0];
            }
        };
        auto open = [&](int i, float s, const float (&g)[8], float (&u)[8], float (&r)[8]) {
            float y[8];
            forget(cur.y[i]);
            forget(cur.x[i]);
            widen_raw(cur.y[i], y);
            widen_raw(cur.x[i], r);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                u[j] = p.wp ? y[j] * s * wp[i][j] : y[j];
                r[j] = __builtin_fmaf(p.beta * g[j], u[j], p.alpha * r[j]);
            }
        };
        float s[1] = {0.f};
        if (p.wp) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if constexpr (!HOLD) load(cur, t, i);
                float v[8];
                widen_raw(cur.y[i], v);
#pragma unroll
                for (int j = 0; j < 8; ++j) s[0] = __builtin_fmaf(v[j], v[j], s[0]);
            }
            team_sum<TEAM, 1>(s, lds, odd);
            s[0] = inv_rms(s[0], p);
        }
        float two[2] = {0.f, 0.f};  // r^2, wn dh r
        if (p.dh) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if constexpr (!HOLD) load(cur, t, i);
                float g[8], u[8], r[8], dh[8];
                gate(i, g);
                open(i, s[0], g, u, r);
                widen_raw(cur.dh[i], dh);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    two[0] = __builtin_fmaf(r[j], r[j], two[0]);
                    two[1] = __builtin_fmaf(r[j], wn[i][j] * dh[j], two[1]);
                }
            }
            team_sum<TEAM, 2>(two, lds, odd + 1);
        }
        // (without dh its values are zero, and so is back)
        const float q = inv_rms(two[0], p), back = q * q * q / (float)p.n * two[1];
        // D, and beta D
        auto grown = [&](int i, const float (&r)[8], float (&d)[8], bool first) {
            float dr[8], dh[8];
            forget(cur.dr[i]);
            forget(cur.dh[i]);
            widen_raw(cur.dr[i], dr);
            widen_raw(cur.dh[i], dh);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                d[j] = dr[j] + (q * (wn[i][j] * dh[j]) - back * r[j]);
                if (first) awn[i][j] = __builtin_fmaf(dh[j], r[j] * q, awn[i][j]);
            }
        };
        float end[2] = {0.f, 0.f};  // v y, beta D u
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = chunk(i), left = p.n - c;
            if constexpr (!HOLD) load(cur, t, i);
            float g[8], u[8], r[8], d[8];
            gate(i, g);
            open(i, s[0], g, u, r);
            grown(i, r, d, true);
            if (p.dx) {
#pragma unroll
                for (int j = 0; j < 8; ++j) r[j] = p.alpha * d[j];
                store_some<XT>(p.dx, t * n + c, r, left);
            }
            if (!p.y) continue;
            float y[8];
            widen_raw(cur.y[i], y);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                d[j] *= p.beta;
                r[j] = d[j] * u[j];
                end[1] += r[j];
                agc[i][j] += r[j];
                const float v = d[j] * g[j];
                awp[i][j] = __builtin_fmaf(v, y[j] * s[0], awp[i][j]);
                end[0] = __builtin_fmaf(v * wp[i][j], y[j], end[0]);
            }
            if (p.dg && p.g_kind == IQK_GATE_ELEMENT && left > 0) store_any(p.dg, p.g_dtype, t * n + c, r, left);
        }
        const bool token = p.dg && p.g_kind == IQK_GATE_TOKEN;
        if (p.wp || token) team_sum<TEAM, 2>(end, lds, odd + 2);
        if (token && tid == 0) {
            const float one[4] = {end[1], 0.f, 0.f, 0.f};
            store_any(p.dg, p.g_dtype, t, one, 1);
        }
        if (!p.dy) continue;
        const float off = p.wp ? s[0] * s[0] * s[0] / (float)p.n * end[0] : 0.f, by = p.wp ? s[0] : 1.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if constexpr (!HOLD) load(cur, t, i);
            float g[8], u[8], r[8], d[8], y[8];
            gate(i, g);
            open(i, s[0], g, u, r);
            grown(i, r, d, false);
            widen_raw(cur.y[i], y);
#pragma unroll
            for (int j = 0; j < 8; ++j) d[j] = by * (p.beta * d[j] * g[j] * wp[i][j]) - off * y[j];
            store_some<YT>(p.dy, t * n + chunk(i), d, p.n - chunk(i));
        }
    }
    float* sums = p.sums + team * p.columns * n;
    auto put = [&](int has, const float (&a)[NV][8]) {
        if (!has) return;
#pragma unroll
        for (int i = 0; i < NV; ++i) store_some<IQK_F32>(sums, chunk(i), a[i], p.n - chunk(i));
        sums += n;
    };
    put(p.has_dwp, awp);
    put(p.has_dwn, awn);
    put(p.has_dgc, agc);
}

// Sums of the teams' parts, column by column: 64 columns by 16 runs of teams,
// whose sums are added in their order.
constexpr int kRuns = 16;

struct NormJoin {
    const float* sums;
    int64_t teams, width;  // width: columns of all arrays together
    int n;
    void* out[3];
    int dtype[3];
};

__global__ __launch_bounds__(64 * kRuns) void norm_join_kernel(NormJoin p) {
    __shared__ float lds[kRuns][64];
    const int lane = threadIdx.x & 63, run = threadIdx.x >> 6;
    const int64_t c = (int64_t)blockIdx.x * 64 + lane;
    const int64_t per = (p.teams + kRuns - 1) / kRuns, end = min((run + 1) * per, p.teams);
    float v = 0.f;
    if (c < p.width) {
#pragma unroll 8
        for (int64_t t = run * per; t < end; ++t) v += p.sums[t * p.width + c];
    }
    lds[run][lane] = v;
    __syncthreads();
    if (run != 0 || c >= p.width) return;
#pragma unroll
    for (int i = 1; i < kRuns; ++i) v += lds[i][lane];
    const int which = (int)(c / p.n);
    const int64_t at = c - (int64_t)which * p.n;
    if (p.dtype[which] == IQK_F32) store_y<IQK_F32>(p.out[which], at, v);
    else if (p.dtype[which] == IQK_F16) store_y<IQK_F16>(p.out[which], at, v);
    else store_y<IQK_BF16>(p.out[which], at, v);
}

NormParams params_of(const iqk_block& b) {
    NormParams p{};
    p.x = b.x;
    p.y = b.y;
    p.wp = b.post_weight;
    p.g = b.gate;
    p.wn = b.next_weight;
    p.w_dtype = b.weight_dtype;
    p.g_dtype = b.gate_dtype;
    p.g_kind = b.gate_kind;
    p.T = b.T;
    p.n = (int)b.n;
    p.alpha = b.alpha;
    p.beta = b.beta;
    p.eps = b.eps;
    return p;
}

// f(x's type, y's type)
template <class F>
void by_types(const iqk_block& b, F f) {
    by_float(b.dtype, [&](auto xt) {
        constexpr int XT = decltype(xt)::value;
        if (XT != IQK_F32 && b.y && b.y_dtype == IQK_F32) f(xt, std::integral_constant<int, IQK_F32>{});
        else f(xt, xt);
    });
}

template <int V>
using Int = std::integral_constant<int, V>;

// f(threads of a team, chunks of a thread) for rows of n values
template <class F>
void by_row(int64_t n, F f) {
    if (n <= 512) f(Int<64>{}, Int<1>{});
    else if (n <= 1024) f(Int<64>{}, Int<2>{});
    else if (n <= 2048) f(Int<256>{}, Int<1>{});
    else if (n <= 4096) f(Int<256>{}, Int<2>{});
    else f(Int<512>{}, Int<2>{});
}

// The gradient, whose parts of the parameters' gradients take three registers a
// value: eight values of a thread as far as 512 threads reach, which is as many
// as have the 200 registers that it needs.
template <class F>
void by_grad_row(int64_t n, F f) {
    if (n <= 512) f(Int<64>{}, Int<1>{});
    else if (n <= 1024) f(Int<128>{}, Int<1>{});
    else if (n <= 2048) f(Int<256>{}, Int<1>{});
    else if (n <= 4096) f(Int<512>{}, Int<1>{});
    else f(Int<512>{}, Int<2>{});
}

int team_size(int64_t n) {
    int team = 0;
    by_grad_row(n, [&](auto t, auto) { team = decltype(t)::value; });
    return team;
}

// Teams of the gradient: the 512 threads that a CU holds of it.
int64_t grad_teams(int64_t T, int64_t n) {
    const int team = team_size(n), per = team == 64 ? 4 : 1;
    const int64_t most = 256 * 512 / team;
    return (std::min(std::max<int64_t>(T, 1), most) + per - 1) / per * per;
}

// A grid of `groups` workgroups; a launch of more than 2^32 threads goes out as a plane.
dim3 grid_of(int64_t groups) {
    constexpr int64_t kMost = 1 << 20;
    return groups <= kMost ? dim3((unsigned)groups) : dim3((unsigned)kMost, (unsigned)((groups + kMost - 1) / kMost));
}

}  // namespace

int64_t norm_sums_bytes(int64_t T, int64_t n, int columns) { return grad_teams(T, n) * columns * n * 4; }

hipError_t launch_norm(const iqk_block& b, void* r, void* h, hipStream_t s) {
    NormParams p = params_of(b);
    p.r = r;
    p.h = h;
    by_types(b, [&](auto xt, auto yt) {
        by_row(b.n, [&](auto team, auto nv) {
            constexpr int TEAM = decltype(team)::value;
            using Tm = Team<TEAM>;
            hipLaunchKernelGGL((norm_kernel<decltype(xt)::value, decltype(yt)::value, TEAM, decltype(nv)::value>),
                               grid_of((p.T + Tm::kTeams - 1) / Tm::kTeams), dim3(Tm::kThreads), 0, s, p);
        });
    });
    return hipGetLastError();
}

hipError_t launch_norm_grad(const iqk_block& b, const NormGradOut& o, float* sums, hipStream_t s) {
    NormParams p = params_of(b);
    p.dr = o.dr;
    p.dh = o.dh;
    p.dx = o.dx;
    p.dy = o.dy;
    p.dg = b.gate_kind == IQK_GATE_CHANNEL ? nullptr : o.d_gate;
    p.sums = sums;
    p.has_dwp = o.d_post != nullptr;
    p.has_dwn = o.d_next != nullptr;
    p.has_dgc = b.gate_kind == IQK_GATE_CHANNEL && o.d_gate;
    p.columns = p.has_dwp + p.has_dwn + p.has_dgc;
    const int64_t teams = grad_teams(p.T, p.n);
    by_types(b, [&](auto xt, auto yt) {
        by_grad_row(b.n, [&](auto team, auto nv) {
            constexpr int TEAM = decltype(team)::value, XT = decltype(xt)::value, YT = decltype(yt)::value;
            constexpr int NV = decltype(nv)::value;
            using Tm = Team<TEAM>;
            constexpr bool HOLD = NV == 1, AHEAD = HOLD && XT != IQK_F32;
            hipLaunchKernelGGL((norm_grad_kernel<XT, YT, TEAM, NV, HOLD, AHEAD>),
                               dim3((unsigned)(teams / Tm::kTeams)), dim3(Tm::kThreads), 0, s, p);
        });
    });
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.columns == 0) return e;
    NormJoin j{};
    j.sums = sums;
    j.teams = teams;
    j.width = (int64_t)p.columns * p.n;
    j.n = p.n;
    int at = 0;
    auto put = [&](int has, void* out, int dtype) {
        if (!has) return;
        j.out[at] = out;
        j.dtype[at++] = dtype;
    };
    put(p.has_dwp, o.d_post, b.weight_dtype);
    put(p.has_dwn, o.d_next, b.weight_dtype);
    put(p.has_dgc, o.d_gate, b.gate_dtype);
    hipLaunchKernelGGL(norm_join_kernel, dim3((unsigned)((j.width + 63) / 64)), dim3(64 * kRuns), 0, s, j);
    return hipGetLastError();
}

}  // namespace iqk
