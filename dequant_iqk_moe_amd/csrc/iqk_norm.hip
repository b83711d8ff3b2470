// iqk_norm.hip -- the norm behind a block, its gate, the scaled residual and the
// norm before the next block in one pass over the rows, and their gradient.
//
//   u = y s(y) wp            s(v) = (mean v^2 + eps)^-1/2   (u = y without wp)
//   r = alpha x + beta g u
//   h = r s(r) wn            from r before its rounding
//
// Gradient, from dr and dh, with s = s(y), q = s(r):
//   D    = dr + q (wn dh - r q m), m = q / n sum(wn dh r)
//   dx   = alpha D           d_wn = sum_t dh r q
//   dg   = beta D u          (summed over tokens or over the row with g's kind)
//   v    = beta g D wp       d_wp = sum_t beta g D y s
//   dy   = s (v - y s / n sum(v y s))   (beta g D without wp)
// Each factor of s or q meets a row's values by itself: a cube of them leaves
// float32 from rows of 1e12 on, and beside zeros and an eps below 1e-25.
// r is computed again from x and y, so it is not rounded there either, and is
// not read beside them.
//
// Bound: bytes.  A team (a wave, or a workgroup) holds a row in registers as it
// lies in memory, so each row is read once; sums go through float32, lanes and
// waves in a fixed order.  8192 x 4096 bfloat16: 52 us (268 MB, 5.2 TB/s; a large
// copy runs at 4.8); the gradient of 4095 rows 52 us, of which 46 the rows (201 MB,
// 4.4 TB/s, and 25 MB of parts of the parameters' gradients) and 5 their join.
// Chunks of eight values are read where every row begins at a multiple of 16 bytes,
// single values elsewhere: either way a chunk is in its row or past it, where a
// buffer's loads give zeros and its stores are dropped, so no path has a branch for
// the end of a row.
#include <algorithm>
#include <cmath>

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

// V values of a row as they lie in memory.
template <int DT, int V>
struct Piece {
    static constexpr int kWords = V == 1 ? 1 : (DT == IQK_F32 ? V : V / 2);
    uint32_t w[kWords];
};
template <int DT>
constexpr int kSizeOf = DT == IQK_F32 ? 4 : 2;

__device__ __forceinline__ int size_of(int dtype) { return dtype == IQK_F32 ? 4 : 2; }

// Row t (the same in every lane) of n values
__device__ __forceinline__ Rsrc row_of(const void* p, int64_t t, int n, int size) {
    return make_rsrc((const char*)p + t * n * size, p ? (uint32_t)(n * size) : 0u);
}

// the V values from value c on
template <int DT, int V>
__device__ __forceinline__ Piece<DT, V> load_piece(Rsrc r, int c) {
    Piece<DT, V> p;
    const uint32_t off = (uint32_t)c * kSizeOf<DT>;
    if constexpr (V == 1) {
        p.w[0] = DT == IQK_F32 ? ld32(r, off) : ld16(r, off);
    } else {
#pragma unroll
        for (int i = 0; i < Piece<DT, V>::kWords; i += 4) {
            const uint4 u = ld128(r, off + 4 * i);
            p.w[i] = u.x, p.w[i + 1] = u.y, p.w[i + 2] = u.z, p.w[i + 3] = u.w;
        }
    }
    return p;
}
template <int DT, int V>
__device__ __forceinline__ void widen_piece(const Piece<DT, V>& p, float (&v)[V]) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
        if constexpr (DT == IQK_F32) v[j] = __uint_as_float(p.w[j]);
        else if constexpr (DT == IQK_BF16) v[j] = __uint_as_float(j % 2 ? p.w[j / 2] & 0xFFFF0000u : p.w[j / 2] << 16);
        else v[j] = half_to_float(j % 2 ? p.w[j / 2] >> 16 : p.w[j / 2] & 0xFFFFu);
    }
}
template <int DT, int V>
__device__ __forceinline__ void store_piece(Rsrc r, int c, const float (&v)[V]) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    const uint32_t off = (uint32_t)c * kSizeOf<DT>;
    if constexpr (V == 1) {
        if constexpr (DT == IQK_F32) __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[0]), r, off, 0, 0);
        else __builtin_amdgcn_raw_buffer_store_b16((uint16_t)pack2<DT>(v[0], v[0]), r, off, 0, 0);
    } else if constexpr (DT == IQK_F32) {
#pragma unroll
        for (int i = 0; i < V; i += 4)
            __builtin_amdgcn_raw_buffer_store_b128(u32x4{__float_as_uint(v[i]), __float_as_uint(v[i + 1]), __float_as_uint(v[i + 2]), __float_as_uint(v[i + 3])},
                                                   r, off + 4 * i, 0, 0);
    } else {
        __builtin_amdgcn_raw_buffer_store_b128(u32x4{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]), pack2<DT>(v[4], v[5]), pack2<DT>(v[6], v[7])},
                                               r, off, 0, 0);
    }
}
// The same for a type known at run time only (the same in every lane).
template <int V>
__device__ __forceinline__ void load_typed(Rsrc r, int dtype, int c, float (&v)[V]) {
    if (dtype == IQK_F32) widen_piece(load_piece<IQK_F32, V>(r, c), v);
    else if (dtype == IQK_BF16) widen_piece(load_piece<IQK_BF16, V>(r, c), v);
    else widen_piece(load_piece<IQK_F16, V>(r, c), v);
}
template <int V>
__device__ __forceinline__ void store_typed(Rsrc r, int dtype, int c, const float (&v)[V]) {
    if (dtype == IQK_F32) store_piece<IQK_F32>(r, c, v);
    else if (dtype == IQK_BF16) store_piece<IQK_BF16>(r, c, v);
    else store_piece<IQK_F16>(r, c, v);
}
// The value of a gate of tokens at row t
__device__ __forceinline__ float token_gate(const NormParams& p, int64_t t) {
    float one[1];
    load_typed(row_of(p.g, t, 1, size_of(p.g_dtype)), p.g_dtype, 0, one);
    return one[0];
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------

template <int XT, int YT, int TEAM, int V, int NV>
__global__ __launch_bounds__(Team<TEAM>::kThreads) void norm_kernel(NormParams p) {
    using Tm = Team<TEAM>;
    __shared__ float lds[2 * Tm::kWaves][2];
    const int tid = threadIdx.x % TEAM;
    const int64_t t = (blockIdx.y * (int64_t)gridDim.x + blockIdx.x) * Tm::kTeams + __builtin_amdgcn_readfirstlane(threadIdx.x / TEAM);
    if (t >= p.T) return;  // (whole teams: no barrier misses a wave)
    Piece<XT, V> x[NV];
    Piece<YT, V> y[NV];
    auto chunk = [&](int i) { return (i * TEAM + tid) * V; };
    const Rsrc xr = row_of(p.x, t, p.n, kSizeOf<XT>), yr = row_of(p.y, t, p.n, kSizeOf<YT>);
#pragma unroll
    for (int i = 0; i < NV; ++i) y[i] = load_piece<YT, V>(yr, chunk(i));  // (zeros without y)
#pragma unroll
    for (int i = 0; i < NV; ++i) x[i] = load_piece<XT, V>(xr, chunk(i));
    float s[1] = {0.f};
    if (p.wp) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float v[V];
            widen_piece(y[i], v);
#pragma unroll
            for (int j = 0; j < V; ++j) s[0] = __builtin_fmaf(v[j], v[j], s[0]);
        }
        team_sum<TEAM, 1>(s, lds, 0);
        s[0] = inv_rms(s[0], p);
    }
    const Rsrc wpr = row_of(p.wp, 0, p.n, size_of(p.w_dtype)), wnr = row_of(p.wn, 0, p.n, size_of(p.w_dtype));
    const Rsrc gr = row_of(p.g, p.g_kind == IQK_GATE_ELEMENT ? t : 0, p.n, size_of(p.g_dtype));
    const Rsrc rr = row_of(p.r, t, p.n, kSizeOf<XT>), hr = row_of(p.h, t, p.n, kSizeOf<XT>);
    const float beta = p.g_kind == IQK_GATE_TOKEN ? p.beta * token_gate(p, t) : p.beta;
    float r[NV][V], q[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = chunk(i);
        widen_piece(x[i], r[i]);
        if (p.y) {
            float u[V], w[V];
            widen_piece(y[i], u);
            if (p.wp) {
                load_typed(wpr, p.w_dtype, c, w);
#pragma unroll
                for (int j = 0; j < V; ++j) u[j] = u[j] * s[0] * w[j];
            }
            if (p.g_kind == IQK_GATE_CHANNEL || p.g_kind == IQK_GATE_ELEMENT) {
                load_typed(gr, p.g_dtype, c, w);
#pragma unroll
                for (int j = 0; j < V; ++j) r[i][j] = __builtin_fmaf(beta * w[j], u[j], p.alpha * r[i][j]);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) r[i][j] = __builtin_fmaf(beta, u[j], p.alpha * r[i][j]);
            }
            store_piece<XT>(rr, c, r[i]);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) q[0] = __builtin_fmaf(r[i][j], r[i][j], q[0]);
    }
    if (!p.h) return;
    team_sum<TEAM, 1>(q, lds, 1);
    q[0] = inv_rms(q[0], p);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float w[V];
        load_typed(wnr, p.w_dtype, chunk(i), w);
#pragma unroll
        for (int j = 0; j < V; ++j) w[j] *= r[i][j] * q[0];
        store_piece<XT>(hr, chunk(i), w);
    }
}

// ---------------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------------

// What the compiler knows of a row's values ends here: it would keep a pass's
// float32 values for the next one instead of widening them again.
template <class R>
__device__ __forceinline__ void forget(R& r) {
#pragma unroll
    for (auto& w : r.w) asm volatile("" : "+v"(w));
}

// A team takes every teams-th row, so its threads meet the same columns in each:
// the parameters' values and its parts of their gradients stay in registers, and
// another launch joins the teams' parts in their order.  What is not there is taken
// as what changes nothing (weights and gates one, y, dr and dh zero), so that every
// form is one straight path.
template <int XT, int YT, int TEAM, int V, int NV>
__global__ __launch_bounds__(Team<TEAM>::kThreads) __attribute__((amdgpu_waves_per_eu(V == 8 && NV == 1 && YT != IQK_F32 ? 4 : 2))) void
norm_grad_kernel(NormParams p) {
    using Tm = Team<TEAM>;
    __shared__ float lds[6 * Tm::kWaves][2];  // (a row's sums and the next one's take turns)
    const int tid = threadIdx.x % TEAM;
    const int64_t team = (int64_t)blockIdx.x * Tm::kTeams + __builtin_amdgcn_readfirstlane(threadIdx.x / TEAM);
    const int64_t teams = (int64_t)gridDim.x * Tm::kTeams;
    auto chunk = [&](int i) { return (i * TEAM + tid) * V; };
    struct Params {
        float wp[V], wn[V], bg[V];  // bg: of beta and the gate what all rows share
    };
    auto load_params = [&](int i) {
        Params a;
#pragma unroll
        for (int j = 0; j < V; ++j) a.wp[j] = a.wn[j] = a.bg[j] = 1.f;
        if (p.wp) load_typed(row_of(p.wp, 0, p.n, size_of(p.w_dtype)), p.w_dtype, chunk(i), a.wp);
        if (p.wn && p.dh) load_typed(row_of(p.wn, 0, p.n, size_of(p.w_dtype)), p.w_dtype, chunk(i), a.wn);  // (no part without dh)
        if (p.g_kind == IQK_GATE_CHANNEL) load_typed(row_of(p.g, 0, p.n, size_of(p.g_dtype)), p.g_dtype, chunk(i), a.bg);
#pragma unroll
        for (int j = 0; j < V; ++j) a.bg[j] *= p.g_kind == IQK_GATE_ELEMENT ? 1.f : p.beta;
        return a;
    };
    // (sixteen single values leave no registers for them)
    constexpr bool KEEP = V > 1 || NV <= 8;
    Params kept[KEEP ? NV : 1];
    auto params = [&](int i) { return KEEP ? kept[KEEP ? i : 0] : load_params(i); };
    // Sums over the rows: of what is wn's gradient, and of b D y s, b being what is a row's own of beta and the gate,
    // which is d_wp but for bg, and dg of a gate of channels (b = 1) but for beta and wp.
    float awp[NV][V], awn[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (KEEP) kept[KEEP ? i : 0] = load_params(i);
#pragma unroll
        for (int j = 0; j < V; ++j) awp[i][j] = awn[i][j] = 0.f;
    }
    int odd = 0;
    for (int64_t t = team; t < p.T; t += teams, odd = 3 - odd) {
        struct Row {
            Piece<XT, V> x[NV], dr[NV], dh[NV];
            Piece<YT, V> y[NV];
        } row;
        const Rsrc xr = row_of(p.x, t, p.n, kSizeOf<XT>), yr = row_of(p.y, t, p.n, kSizeOf<YT>);
        const Rsrc drr = row_of(p.dr, t, p.n, kSizeOf<XT>), dhr = row_of(p.dh, t, p.n, kSizeOf<XT>);
#pragma unroll
        for (int i = 0; i < NV; ++i) row.y[i] = load_piece<YT, V>(yr, chunk(i));  // (zeros without them)
#pragma unroll
        for (int i = 0; i < NV; ++i) row.x[i] = load_piece<XT, V>(xr, chunk(i));
#pragma unroll
        for (int i = 0; i < NV; ++i) row.dh[i] = load_piece<XT, V>(dhr, chunk(i));
#pragma unroll
        for (int i = 0; i < NV; ++i) row.dr[i] = load_piece<XT, V>(drr, chunk(i));
        const float gt = p.g_kind == IQK_GATE_TOKEN ? token_gate(p, t) : 1.f;
        const Rsrc gr = row_of(p.g, t, p.n, size_of(p.g_dtype)), dgr = row_of(p.dg, t, p.n, size_of(p.g_dtype));
        // b at a chunk
        auto gate = [&](int i, float (&b)[V]) {
            if (p.g_kind == IQK_GATE_ELEMENT) {
                load_typed(gr, p.g_dtype, chunk(i), b);
#pragma unroll
                for (int j = 0; j < V; ++j) b[j] *= p.beta;
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) b[j] = gt;
            }
        };
        float s[1] = {0.f};
        if (p.wp) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float v[V];
                widen_piece(row.y[i], v);
#pragma unroll
                for (int j = 0; j < V; ++j) s[0] = __builtin_fmaf(v[j], v[j], s[0]);
            }
            team_sum<TEAM, 1>(s, lds, odd);
            s[0] = inv_rms(s[0], p);
        } else {
            s[0] = 1.f;
        }
        float r[NV][V], two[2] = {0.f, 0.f};  // r^2, wn dh r
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float b[V], y[V], dh[V];
            const Params a = params(i);
            gate(i, b);
            forget(row.y[i]);
            widen_piece(row.y[i], y);
            widen_piece(row.x[i], r[i]);
            widen_piece(row.dh[i], dh);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                r[i][j] = __builtin_fmaf(a.bg[j] * b[j], y[j] * s[0] * a.wp[j], p.alpha * r[i][j]);
                two[0] = __builtin_fmaf(r[i][j], r[i][j], two[0]);
                two[1] = __builtin_fmaf(r[i][j], a.wn[j] * dh[j], two[1]);
            }
        }
        float q = 0.f, mean = 0.f;  // m of the formula
        if (p.dh) {
            team_sum<TEAM, 2>(two, lds, odd + 1);
            q = inv_rms(two[0], p);
            mean = two[1] * q / (float)p.n;
        } else {  // D is dr, whatever r
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j) r[i][j] = 0.f;
        }
        const Rsrc dxr = row_of(p.dx, t, p.n, kSizeOf<XT>);
        float end[2] = {0.f, 0.f};  // v y s, D u
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float b[V], y[V], dr[V], dh[V], d[V];
            const Params a = params(i);
            gate(i, b);
            forget(row.y[i]);
            forget(row.dh[i]);
            widen_piece(row.y[i], y);
            widen_piece(row.dr[i], dr);
            widen_piece(row.dh[i], dh);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float rq = r[i][j] * q;
                d[j] = __builtin_fmaf(q, a.wn[j] * dh[j] - rq * mean, dr[j]);
                awn[i][j] = __builtin_fmaf(dh[j], rq, awn[i][j]);
                dr[j] = p.alpha * d[j];
            }
            store_piece<XT>(dxr, chunk(i), dr);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float ys = y[j] * s[0], du = d[j] * (ys * a.wp[j]), bd = b[j] * d[j];
                end[1] += du;
                awp[i][j] = __builtin_fmaf(bd, ys, awp[i][j]);
                r[i][j] = bd * a.bg[j] * a.wp[j];  // (v of the formula, where r was)
                end[0] = __builtin_fmaf(r[i][j], ys, end[0]);
                d[j] = p.beta * du;
            }
            if (p.dg && p.g_kind == IQK_GATE_ELEMENT) store_typed(dgr, p.g_dtype, chunk(i), d);
        }
        const bool token = p.dg && p.g_kind == IQK_GATE_TOKEN;
        if (p.wp || token) team_sum<TEAM, 2>(end, lds, odd + 2);
        if (token && tid == 0) {
            const float one[1] = {p.beta * end[1]};
            store_typed(row_of(p.dg, t, 1, size_of(p.g_dtype)), p.g_dtype, 0, one);
        }
        if (!p.dy) continue;
        const float off = end[0] / (float)p.n;
        const Rsrc dyr = row_of(p.dy, t, p.n, kSizeOf<YT>);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (p.wp) {  // (else it is v, whatever y)
                float y[V];
                forget(row.y[i]);
                widen_piece(row.y[i], y);
#pragma unroll
                for (int j = 0; j < V; ++j) r[i][j] = s[0] * (r[i][j] - y[j] * s[0] * off);
            }
            store_piece<YT>(dyr, chunk(i), r[i]);
        }
    }
    float* sums = p.sums + team * p.columns * p.n;
    auto put = [&](int has, auto value) {
        if (!has) return;
        const Rsrc to = row_of(sums, 0, p.n, 4);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Params a = params(i);
            float o[V];
#pragma unroll
            for (int j = 0; j < V; ++j) o[j] = value(a, i, j);
            store_piece<IQK_F32>(to, chunk(i), o);
        }
        sums += p.n;
    };
    put(p.has_dwp, [&](const Params& a, int i, int j) { return a.bg[j] * awp[i][j]; });
    put(p.has_dwn, [&](const Params&, int i, int j) { return awn[i][j]; });
    put(p.has_dgc, [&](const Params& a, int i, int j) { return p.beta * a.wp[j] * awp[i][j]; });
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

// f(threads of a team, values of a chunk, chunks of a thread) for rows of n values.
// Eight values a thread to 2048, sixteen beyond (bfloat16, with 8, 16 and 32 of them:
// 16384 x 512 14.2, 16.6 and 21.6 us; 16384 x 1024 27.9, 28.7 and 32.2; 2048 x 2048 7.6,
// 7.5 and 8.3; 2048 x 4096 14.6, 13.2 and 14.1; 2048 x 8192 31.1, 28.5 and 29.0; 256 x
// 2048 3.6, 4.3 and 5.7; 256 x 4096 4.0, 4.7 and 6.1).  The rows' number has no part in
// it, so a row's results are the same alone and among others.  Where one of the call's
// rows or parameters begins at no multiple of 16 bytes, or n is no multiple of 8, a
// thread has other values of the row, whose sums then go in another order.
template <class F>
void by_row(int64_t n, bool wide, F f) {
    auto go = [&](auto team, auto values) {
        constexpr int N = decltype(values)::value;  // of a thread
        if (wide) f(team, Int<8>{}, Int<N / 8>{});
        else f(team, Int<1>{}, values);
    };
    if (n <= 512) go(Int<64>{}, Int<8>{});
    else if (n <= 1024) go(Int<128>{}, Int<8>{});
    else if (n <= 2048) go(Int<256>{}, Int<8>{});
    else if (n <= 4096) go(Int<256>{}, Int<16>{});
    else go(Int<512>{}, Int<16>{});
}

// The gradient, whose parts of the parameters' gradients and their values take five
// registers a value: eight values of a thread as far as 512 threads reach, in 108 to
// 117 registers, so that a CU holds two teams of 4096 values (rows of 4095 x 4096 46
// us; 60 with branches for a row's end and 256 threads of sixteen values).  In single
// values they take 127 to 153, and a CU holds one team of 512 threads (4095 x 4095 77 us).
template <class F>
void by_grad_row(int64_t n, bool wide, F f) {
    auto go = [&](auto team, auto values) {
        constexpr int N = decltype(values)::value;
        if (wide) f(team, Int<8>{}, Int<N / 8>{});
        else f(team, Int<1>{}, values);
    };
    if (n <= 512) go(Int<64>{}, Int<8>{});
    else if (n <= 1024) go(Int<128>{}, Int<8>{});
    else if (n <= 2048) go(Int<256>{}, Int<8>{});
    else if (n <= 4096) go(Int<512>{}, Int<8>{});
    else go(Int<512>{}, Int<16>{});
}

int team_size(int64_t n) {
    int team = 0;
    by_grad_row(n, true, [&](auto t, auto, auto) { team = decltype(t)::value; });
    return team;
}

// Whether chunks of eight values lie at multiples of 16 bytes in all that a call reads
// or writes by rows: its inputs, and `more`.  (A gate of tokens is read one value at a
// time.)
bool wide_rows(const iqk_block& b, std::initializer_list<const void*> more) {
    bool wide = b.n % 8 == 0;
    auto take = [&](const void* p) { wide = wide && (uintptr_t)p % 16 == 0; };
    for (const void* p : {b.x, b.y, b.post_weight, b.next_weight}) take(p);
    if (b.gate_kind != IQK_GATE_TOKEN) take(b.gate);
    for (const void* p : more) take(p);
    return wide;
}

// Teams of the gradient, at most the threads that the card's CUs hold of it in chunks of eight values: 1024 of a CU up
// to n = 4096 (up to 128 registers), 512 beyond.  Single values, which take more, go by the same number (it gives the
// workspace's size, in which addresses have no part): a CU holds fewer of those teams at a time.  A team's time grows
// with its rows and the join's with the teams, so the sum is least where rows grow with the root of T, and with powers
// of two, which leave the CUs equal shares: 4095 x 512 takes 29 us with a team for each row, 19.5 with one for two rows,
// 16.2 for four, 18.5 for eight; 300 rows 8.9, 8.5, 11.1, 15.4; 8192 rows 28, 28, 22 and 22, and 24.5 with six.
int64_t grad_teams(int64_t T, int64_t n) {
    const int team = team_size(n), per = team == 64 ? 4 : 1;
    const int64_t most = 256 * (n <= 4096 ? 1024 : 512) / team;
    const int64_t rows = (int64_t)std::exp2(std::max(0.0, std::round(std::log2(std::sqrt((double)T) / 12))));
    const int64_t teams = std::max<int64_t>(1, (T + rows - 1) / rows);
    return (std::min(teams, most) + per - 1) / per * per;
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
        by_row(b.n, wide_rows(b, {r, h}), [&](auto team, auto v, auto nv) {
            constexpr int TEAM = decltype(team)::value;
            using Tm = Team<TEAM>;
            hipLaunchKernelGGL((norm_kernel<decltype(xt)::value, decltype(yt)::value, TEAM, decltype(v)::value, decltype(nv)::value>),
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
        // (the gradients of a gate of channels or tokens are written one value at a time)
        const bool wide = wide_rows(b, {o.dr, o.dh, o.dx, o.dy, b.gate_kind == IQK_GATE_ELEMENT ? o.d_gate : nullptr, sums});
        by_grad_row(b.n, wide, [&](auto team, auto v, auto nv) {
            constexpr int TEAM = decltype(team)::value;
            using Tm = Team<TEAM>;
            hipLaunchKernelGGL((norm_grad_kernel<decltype(xt)::value, decltype(yt)::value, TEAM, decltype(v)::value, decltype(nv)::value>),
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
