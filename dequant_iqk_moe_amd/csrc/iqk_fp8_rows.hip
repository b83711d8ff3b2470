// iqk_fp8_rows.hip -- the 8-bit product for few rows: weights straight from
// memory into matrix operands.
//
// Weights are the A operand and x the B operand of v_mfma_f32_16x16x32_f16
// (both widened to float16 in registers): lane l holds row l & 15 of both and,
// of each block of 128, the 16 values at 16 * (l >> 4) and the 16 at
// 64 + 16 * (l >> 4) (any order of the depth will do that is the same in
// both).  A result lane holds four consecutive weight rows of one row of x.
// The waves of a workgroup take the blocks of the depth in turn, so that
// together they read consecutive bytes of each weight row, and add their sums
// through LDS in wave order: the same result every time.
//
// Bound: bytes of the weights, and a launch's start.  A widened weight costs
// half a vector instruction and an eighth of a matrix instruction's lane slot,
// well below what memory delivers.  One row of x by 4096 x 4096 weights: 5.6
// us (3.0 TB/s of 16.8 MB); one token at six experts of that size: 22 us (4.5
// TB/s; a plain read of as many bytes 17.7 us).
#include "iqk_fp8_device.h"

namespace iqk {
namespace {

// The 32 bytes of block b that a lane holds of one row; bytes past the depth
// read zero (offsets past the resource's records).
struct Frag {
    uint4 lo, hi;
};
// (The default cache policy: the two loads ask for halves of the same 128-byte
// lines, which a non-temporal line does not always outlive.  Six experts of
// 4096 x 4096: 23.7 us against 26.4.)
__device__ __forceinline__ Frag load_frag(Rsrc r, uint32_t row_off, int b, int g, int n) {
    const int c0 = b * kBlock + 16 * g, c1 = c0 + 64;
    return Frag{ld128(r, c0 < n ? row_off + c0 : kOob), ld128(r, c1 < n ? row_off + c1 : kOob)};
}
struct Wide {
    f16x8 v[4];
};
__device__ __forceinline__ Wide widen_frag(const Frag& f) {
    return Wide{{widen(f.lo.x, f.lo.y), widen(f.lo.z, f.lo.w), widen(f.hi.x, f.hi.y), widen(f.hi.z, f.hi.w)}};
}
__device__ __forceinline__ f32x4 block_product(const Wide& w, const Wide& x) {
    f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) d = __builtin_amdgcn_mfma_f32_16x16x32_f16(w.v[i], x.v[i], d, 0, 0, 0);
    return d;
}
__device__ __forceinline__ void add_scaled(f32x4& acc, const f32x4& d, float f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(d[i], f, acc[i]);
}

struct RowsParams {
    const uint8_t* W;
    const float* sw;
    const void* x;
    const float* sx;
    int64_t M;
    int E, out, n, k, x_slots;
    const int32_t* ids;
    void* y;
};

// ---------------------------------------------------------------------------
// up to 16 rows of x, quantized by every workgroup for itself
// ---------------------------------------------------------------------------

// A workgroup owns 16 weight rows and all M rows of x (PAIRS: one routed pair,
// whose expert's rows it reads).  It requests its first weights, then
// quantizes x into LDS while they are on their way: a launch of its own for
// that costs more than the few values each workgroup repeats.
constexpr int kFewWaves = 8;
constexpr int kFewAhead = 4;           // blocks of the depth a wave requests together
constexpr int kFewBytes = 33 * 1024;   // most codes of x a workgroup keeps: eight rows of 4096 (there 9.7 us against 10.9
                                       // with a launch for quantizing; one row 6.3 against 10.8)

// row stride of the codes in LDS: 16 bytes over the depth, so that the rows a
// fragment reads together start on different banks
__host__ __device__ constexpr int few_stride(int n) { return (n + kBlock - 1) / kBlock * kBlock + 16; }

template <int XT, int YT, bool PAIRS>
__global__ __launch_bounds__(64 * kFewWaves) void fp8_few_kernel(RowsParams p) {
    extern __shared__ __align__(16) uint8_t few_lds[];
    __shared__ float4 red[kFewWaves][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int li = lane & 15, g = lane >> 4;
    const int row0 = blockIdx.x * 16;
    const int n = p.n, nb = (n + kBlock - 1) / kBlock, stride = few_stride(n);
    const int rows = PAIRS ? 1 : (int)p.M;
    int e = 0;
    int64_t x0 = 0, y0 = 0;  // first row of x and of y
    if constexpr (PAIRS) {
        const int64_t pr = blockIdx.y;
        e = p.ids[pr];
        x0 = p.x_slots == 1 ? pr / p.k : pr;
        y0 = pr;
        if (e < 0 || e >= p.E) {
            const int o = row0 + (int)threadIdx.x;
            if (threadIdx.x < 16 && o < p.out) store_y<YT>(p.y, y0 * p.out + o, __builtin_nanf(""));
            return;
        }
    }
    const int left = min(16, p.out - row0);
    const Rsrc wr = make_rsrc(p.W + ((int64_t)e * p.out + row0) * n, (uint32_t)left * (uint32_t)n);
    const uint32_t woff = (uint32_t)li * (uint32_t)n;  // (rows past the last are out of range and read zero)
    // x: codes [rows][stride], then scales [rows][nb]; 16 lanes own a block of it.  A wave's memory accesses come
    // back in order, so the first values of x are asked for before the first weights, and quantized while those
    // are on their way.
    float* sxl = (float*)(few_lds + (size_t)rows * stride);
    constexpr int kPer = 64 * kFewWaves / 16;
    struct Values {
        float v[8];
        uint2 q;
        float s;
    };
    auto load_x = [&](int i) {
        Values r{};
        const int row = min(i / nb, rows - 1), b = i - i / nb * nb, c = b * kBlock + 8 * (threadIdx.x & 15);
        if constexpr (XT == IQK_E4M3) {
            if (c < n) r.q = *(const uint2*)((const uint8_t*)p.x + (x0 + row) * n + c);
            r.s = p.sx[(x0 + row) * nb + b];
        } else {
            if (c < n) load8<XT>(p.x, (x0 + row) * n + c, r.v);
        }
        return r;
    };
    auto keep_x = [&](int i, Values& r) {
        if (i >= rows * nb) return;
        if constexpr (XT != IQK_E4M3) {
            const float a = block_amax(r.v), f = kE4m3Max / a;
#pragma unroll
            for (int j = 0; j < 8; ++j) r.v[j] *= f;
            r.q = to_e4m3(r.v);
            r.s = a / kE4m3Max;
        }
        const int row = i / nb, b = i - row * nb;
        *(uint2*)(few_lds + row * stride + b * kBlock + 8 * (threadIdx.x & 15)) = r.q;
        if ((threadIdx.x & 15) == 0) sxl[i] = r.s;
    };
    const int i0 = threadIdx.x >> 4;
    Values first = load_x(i0);
    __builtin_amdgcn_sched_barrier(0);
    Frag w[2][kFewAhead];
#pragma unroll
    for (int i = 0; i < kFewAhead; ++i) w[0][i] = load_frag(wr, woff, wave + i * kFewWaves, g, n);
    __builtin_amdgcn_sched_barrier(0);
    keep_x(i0, first);
    for (int i = i0 + kPer; i < rows * nb; i += kPer) {
        Values r = load_x(i);
        keep_x(i, r);
    }
    __syncthreads();

    const int xr = min(li, rows - 1);
    const uint8_t* xl = few_lds + xr * stride + 16 * g;
    const float* sx = sxl + xr * nb;
    const int nob = (p.out + kBlock - 1) / kBlock;
    const float* sw = p.sw + ((int64_t)e * nob + row0 / kBlock) * nb;
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    auto step = [&](int b0, const Frag (&cur)[kFewAhead], Frag (&next)[kFewAhead]) {
        if (b0 + kFewAhead * kFewWaves < nb) {
#pragma unroll
            for (int i = 0; i < kFewAhead; ++i)
                next[i] = load_frag(wr, woff, b0 + (kFewAhead + i) * kFewWaves, g, n);
        }
#pragma unroll
        for (int i = 0; i < kFewAhead; ++i) {
            const int b = b0 + i * kFewWaves;
            if (b >= nb) break;
            const Frag xf{*(const uint4*)(xl + b * kBlock), *(const uint4*)(xl + b * kBlock + 64)};
            add_scaled(acc, block_product(widen_frag(cur[i]), widen_frag(xf)), sx[b] * sw[b]);
        }
    };
    for (int b0 = wave; b0 < nb; b0 += 2 * kFewAhead * kFewWaves) {
        step(b0, w[0], w[1]);
        if (b0 + kFewAhead * kFewWaves < nb) step(b0 + kFewAhead * kFewWaves, w[1], w[0]);
    }
    red[wave][lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    __syncthreads();
    // one thread per result: value q of lane l is weight row 4 (l / 16) + q of row l % 16 of x
    const int i = threadIdx.x;
    if (i < 256) {
        const int r = i >> 4, o = i & 15;
        if (r < rows && o < left) {
            float v = 0.f;
#pragma unroll
            for (int u = 0; u < kFewWaves; ++u) v += ((const float*)&red[u][16 * (o >> 2) + r])[o & 3];
            store_y<YT>(p.y, (y0 + r) * p.out + row0 + o, v);
        }
    }
}

// ---------------------------------------------------------------------------
// up to 16 NT rows of x, quantized before, in one pass over the weights
// ---------------------------------------------------------------------------

// A workgroup owns 16 weight rows; it holds the sums of the rows of x and
// requests the next block's weights and x while it multiplies the last ones.
// (One weight tile per workgroup and the depth split over its waves: the dense
// product of few rows has no other way to occupy the card.)  Bound: bytes of
// the weights and a launch's start, and x, which every workgroup reads again: 17
// rows by 4096 x 4096 8.6 us, 32 rows 11.0 (1.5 TB/s of weights).
constexpr int kRowsWaves = 4;

template <int NT, int YT>
__global__ __launch_bounds__(64 * kRowsWaves, 4) void fp8_rows_kernel(RowsParams p) {
    __shared__ float4 red[kRowsWaves][NT][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int li = lane & 15, g = lane >> 4;
    const int n = p.n, nb = (n + kBlock - 1) / kBlock;
    const int row0 = blockIdx.x * 16;
    const int left = min(16, p.out - row0);
    const Rsrc wr = make_rsrc(p.W + (int64_t)row0 * n, (uint32_t)left * (uint32_t)n);  // (rows past the last read zero)
    const uint32_t woff = (uint32_t)li * (uint32_t)n;
    const float* sw = p.sw + (int64_t)(row0 / kBlock) * nb;
    const uint8_t* xr[NT];
    const float* sx[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int64_t r = min((int64_t)16 * t + li, p.M - 1);  // rows past the last repeat it, their results are dropped
        xr[t] = (const uint8_t*)p.x + r * n;
        sx[t] = p.sx + r * nb;
    }
    f32x4 acc[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    struct Stage {
        Frag w, x[NT];
        float f[NT];
    } st[2];
    // (blocks past the last, which the loop requests and multiplies like any other, have zero weights)
    auto request = [&](int b, Stage& s) {
        const int c0 = b * kBlock + 16 * g, c1 = c0 + 64;
        const uint32_t o0 = c0 < n ? woff + c0 : kOob, o1 = c1 < n ? woff + c1 : kOob;
        s.w = Frag{ld128(wr, o0), ld128(wr, o1)};
        // a chunk of x past the depth meets zero weights; its row's first bytes are read instead of the next
        // row's, which could be NaN
        const int x0 = c0 < n ? c0 : 0, x1 = c1 < n ? c1 : 0, sb = min(b, nb - 1);
        const float fw = sw[sb];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            s.x[t].lo = *(const uint4*)(xr[t] + x0);
            s.x[t].hi = *(const uint4*)(xr[t] + x1);
            s.f[t] = sx[t][sb] * fw;
        }
    };
    auto multiply = [&](const Stage& s) {
        const Wide w = widen_frag(s.w);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            add_scaled(acc[t], block_product(w, widen_frag(s.x[t])), s.f[t]);
            __builtin_amdgcn_sched_barrier(0);  // (else all tiles are widened at once, and registers run out)
        }
    };
    request(wave, st[0]);
    for (int b = wave; b < nb; b += 2 * kRowsWaves) {
        request(b + kRowsWaves, st[1]);
        multiply(st[0]);
        request(b + 2 * kRowsWaves, st[0]);
        multiply(st[1]);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) red[wave][t][lane] = make_float4(acc[t][0], acc[t][1], acc[t][2], acc[t][3]);
    __syncthreads();
    // four neighbouring threads write the 16 results of one row of x
    for (int u = threadIdx.x; u < 16 * NT * 4; u += 64 * kRowsWaves) {
        const int q = u & 3, r = u >> 2, o = 4 * q;
        if (r >= p.M || o >= left) continue;
        float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kRowsWaves; ++w) {
            const float4 a = red[w][r >> 4][16 * q + (r & 15)];
            v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
        }
        const int64_t at = (int64_t)r * p.out + row0 + o;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (o + j < left) store_y<YT>(p.y, at + j, v[j]);
    }
}

RowsParams rows_params(const Fp8Launch& a) {
    return RowsParams{a.codes, a.scales, a.x, a.x_scales, a.M, (int)a.E, (int)a.out, (int)a.n, a.k, a.x_slots,
                      a.ids, a.y};
}

template <int NT, int YT>
void rows_launch(const RowsParams& p, hipStream_t s) {
    hipLaunchKernelGGL((fp8_rows_kernel<NT, YT>), dim3((unsigned)((p.out + 15) / 16)), dim3(64 * kRowsWaves), 0, s, p);
}

}  // namespace

bool fp8_few_fits(int64_t rows, int64_t n) { return rows <= 16 && rows * few_stride((int)n) <= kFewBytes; }

hipError_t launch_fp8_few(const Fp8Launch& a, hipStream_t s) {
    const RowsParams p = rows_params(a);
    const bool pairs = a.ids != nullptr;
    const int64_t rows = pairs ? 1 : a.M;
    const unsigned lds = (unsigned)(rows * few_stride((int)a.n) + rows * ((a.n + kBlock - 1) / kBlock) * 4);
    const dim3 grid((unsigned)((a.out + 15) / 16), pairs ? (unsigned)a.M : 1u);
    by_float(a.y_dtype, [&](auto yt) {
        auto go = [&](auto xt) {
            constexpr int XT = decltype(xt)::value, YT = decltype(yt)::value;
            if (pairs) hipLaunchKernelGGL((fp8_few_kernel<XT, YT, true>), grid, dim3(64 * kFewWaves), lds, s, p);
            else hipLaunchKernelGGL((fp8_few_kernel<XT, YT, false>), grid, dim3(64 * kFewWaves), lds, s, p);
        };
        if (a.x_dtype == IQK_E4M3) go(std::integral_constant<int, IQK_E4M3>{});
        else by_float(a.x_dtype, go);
    });
    return hipGetLastError();
}

hipError_t launch_fp8_rows(const Fp8Launch& a, hipStream_t s) {
    if (a.M > 32) return hipErrorInvalidValue;
    const RowsParams p = rows_params(a);
    by_float(a.y_dtype, [&](auto yt) {
        constexpr int YT = decltype(yt)::value;
        if (a.M <= 16) rows_launch<1, YT>(p, s);
        else rows_launch<2, YT>(p, s);
    });
    return hipGetLastError();
}

}  // namespace iqk
