// iqk_int8_rows.hip -- quantization of activations to 8-bit integers, and the
// product of few rows: weights straight from memory into matrix operands.
//
//   y[m, o] = (sum_i qx[m, i] qw[o, i]) * (sx[m] sw[o])
//   a = max(max |x[m]|, 2^-100), sx[m] = a / 127, qx[m, i] = round(x[m, i] * (127 / a))
//
// The reciprocal and the product are rounded to float32 and the codes to nearest
// even, so codes are the definition's bit for bit; sums are exact in 32 bits (2^14
// a product, at most 2^16 of them).
#include <algorithm>

#include "iqk_block.h"
#include "iqk_rows_device.h"

namespace iqk {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr float kMaxCode = 127.f;

// The largest |v| seen, as the bits of a non-negative number (a NaN's are above infinity's): 16-bit values two at a
// time, in their own type, until lifted to float32.
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
template <int DT>
__device__ __forceinline__ uint32_t most_bits(uint32_t m, const Raw<DT>& r) {
#pragma unroll
    for (int i = 0; i < (DT == IQK_F32 ? 8 : 4); ++i) {
        if constexpr (DT == IQK_F32) m = max(m, r.w[i] & 0x7FFFFFFFu);
        else
            m = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, m), __builtin_bit_cast(u16x2, r.w[i] & 0x7FFF7FFFu)));
    }
    return m;
}
template <int DT>
__device__ __forceinline__ uint32_t lift_bits(uint32_t m) {
    if constexpr (DT == IQK_F32) return m;
    const uint32_t both = max(m & 0xFFFFu, m >> 16);
    return DT == IQK_BF16 ? both << 16 : __float_as_uint(half_to_float(both));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
    auto ror = [](uint32_t v, auto ctrl) {
        return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, decltype(ctrl)::value, 0xF, 0xF, false);
    };
    x = max(x, ror(x, std::integral_constant<int, 0x128>{}));
    x = max(x, ror(x, std::integral_constant<int, 0x124>{}));
    x = max(x, ror(x, std::integral_constant<int, 0x122>{}));
    x = max(x, ror(x, std::integral_constant<int, 0x121>{}));
    auto lane = [&](int l) { return (uint32_t)__builtin_amdgcn_readlane((int)x, l); };
    return max(max(lane(0), lane(16)), max(lane(32), lane(48)));
}

// A row's scale and the factor that makes its codes, from its largest value's bits.
struct RowScale {
    float scale, factor;
};
__device__ __forceinline__ RowScale row_scale(uint32_t bits) {
    if (bits >= 0x7F800000u) return {__builtin_nanf(""), 0.f};
    const float a = fmaxf(__uint_as_float(bits), kAmaxFloor);
    return {a / kMaxCode, kMaxCode / a};
}

// Codes of 8 values (zeros in a row whose scale is NaN).  A product of at most 2^7
// added to 1.5 * 2^23 is rounded to a whole number, to nearest even, whose lowest
// byte is the code: with the bytes picked out by permutes and 16-bit maxima half the
// instructions of conversions (24576 bfloat16 rows of 4096 48.2 us with those, 46.1 so).
__device__ __forceinline__ uint2 to_int8(const float (&v)[8], float factor) {
#pragma clang fp contract(off)  // (the product is rounded by itself)
    uint32_t q[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t c[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            c[j] = __float_as_uint(v[4 * h + j] * factor + 12582912.f);
        }
        q[h] = __builtin_amdgcn_perm(c[1], c[0], 0x0C0C0400u) | __builtin_amdgcn_perm(c[3], c[2], 0x04000C0Cu);
        q[h] = factor == 0.f ? 0u : q[h];
    }
    return make_uint2(q[0], q[1]);
}

// ---------------------------------------------------------------------------
// quantization
// ---------------------------------------------------------------------------

constexpr int kThreads = 256;

struct PrepParams {
    const void* x;
    int64_t rows;
    int n;
    int8_t* codes;
    float* scales;
    int64_t quant_groups;  // workgroups that quantize; one more makes the plan
    int E, tile;
    const int32_t* offsets;
    int32_t* tiles;
};

// Tiles before each expert, by one workgroup: ceil(rows / tile) of each, summed.
__device__ __forceinline__ void make_plan(const PrepParams& p) {
    __shared__ int32_t sums[kThreads / 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    auto begin = [&](int e) { return e == 0 ? 0 : (int)min(max((int64_t)p.offsets[e], (int64_t)0), p.rows); };
    int before = 0;
    for (int base = 0; base <= p.E; base += kThreads) {
        const int e = base + threadIdx.x;
        int mine = 0;
        if (e <= p.E) {
            const int count = (e < p.E ? begin(e + 1) : (int)p.rows) - begin(e);
            mine = count > 0 ? (count + p.tile - 1) / p.tile : 0;
        }
        int upto = mine;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int o = __shfl_up(upto, d);
            if (lane >= d) upto += o;
        }
        if (lane == 63) sums[wave] = upto;
        __syncthreads();
        upto += before;
        for (int w = 0; w < kThreads / 64; ++w) {
            if (w < wave) upto += sums[w];
            before += sums[w];
        }
        if (e <= p.E) p.tiles[e + 1] = upto;
        if (e == 0) p.tiles[0] = 0;
        __syncthreads();
    }
}

// A team of 64 or 256 threads takes a row; rows of up to 32 values a thread stay in
// registers between the largest value and the codes, longer ones are read again.
// Bound: bytes (bfloat16 rows of 4096: 8192 in 17 us, 5.9 TB/s; 24576 in 46, 6.5).
constexpr int kChunks = 4;

template <int XT, int TEAM, bool HOLD>
__global__ __launch_bounds__(kThreads) void int8_prep_kernel(PrepParams p) {
    const int64_t group = blockIdx.y * (int64_t)gridDim.x + blockIdx.x;
    if (group >= p.quant_groups) {
        if (group == p.quant_groups && p.offsets) make_plan(p);
        return;
    }
    __shared__ uint32_t most[kThreads / 64];
    const int tid = threadIdx.x % TEAM;
    const int64_t row = group * (kThreads / TEAM) + threadIdx.x / TEAM;
    if (row >= p.rows) return;  // (whole teams)
    const int64_t at = row * p.n;
    const int chunks = HOLD ? kChunks : (p.n / 8 + TEAM - 1) / TEAM;
    auto load = [&](int i) {
        const int c = (i * TEAM + tid) * 8;
        return load_raw<XT>(p.x, at + c, c < p.n ? 8 : 0);
    };
    Raw<XT> held[HOLD ? kChunks : 1];
    uint32_t bits = 0;
    if constexpr (HOLD) {
#pragma unroll
        for (int i = 0; i < kChunks; ++i) held[i] = load(i);
    }
#pragma unroll kChunks
    for (int i = 0; i < chunks; ++i) {
        bits = most_bits<XT>(bits, HOLD ? held[HOLD ? i : 0] : load(i));
    }
    bits = wave_max(lift_bits<XT>(bits));
    if constexpr (TEAM > 64) {
        if ((threadIdx.x & 63) == 0) most[threadIdx.x >> 6] = bits;
        __syncthreads();
        bits = max(max(most[0], most[1]), max(most[2], most[3]));
    }
    const RowScale s = row_scale(bits);
#pragma unroll kChunks
    for (int i = 0; i < chunks; ++i) {
        const int c = (i * TEAM + tid) * 8;
        if (c >= p.n) break;
        float v[8];
        widen_raw(HOLD ? held[HOLD ? i : 0] : load(i), v);
        *(uint2*)(p.codes + at + c) = to_int8(v, s.factor);
    }
    if (tid == 0) p.scales[row] = s.scale;
}

// ---------------------------------------------------------------------------
// few rows
// ---------------------------------------------------------------------------

// A workgroup owns 16 weight rows and up to 16 rows of x, which it quantizes into
// LDS while its first weights are on their way: a launch of its own for that costs
// more than the values each workgroup repeats.  Its waves take the blocks of 128 of
// the depth in turn, so that together they read consecutive bytes of each weight
// row, and add their sums through LDS.  Weights are the A operand and x the B
// operand of v_mfma_i32_16x16x64_i8: lane l holds row l & 15 of both and, of each
// block, the 16 values at 16 * (l >> 4) and the 16 at 64 + 16 * (l >> 4).
// Grouped: workgroup column s starts at row s, and takes part if an expert's rows
// begin there, or its next ones that do not fit a workgroup.
// Bound: bytes of the weights, and a launch's start (one row by 4096 x 4096: 5.1 us
// in the kernel, 3.3 TB/s, of which 3.5 us is what the smallest kernel takes).
constexpr int kFewWaves = 8, kFewThreads = 64 * kFewWaves;
constexpr int kFewAhead = 4;          // blocks of the depth a wave requests together
constexpr int kFewBytes = 33 * 1024;  // most codes of x a workgroup keeps
constexpr int64_t kFewGrouped = 32;   // rows of a grouped product up to which each may start a workgroup
constexpr int kFewDense = 4;          // of a dense one (out = in = 4096: 4 rows 8.1 us against 9.1 with a launch for quantizing
                                      // and int8_rows_kernel, 8 rows 11.0 against 9.5)
constexpr int kFewRows = 16;
constexpr int kDepth = 128;           // of a block

// row stride of the codes in LDS: 16 bytes over the depth, so that the rows a
// fragment reads together start on different banks
__host__ __device__ constexpr int few_stride(int64_t n) { return (int)((n + kDepth - 1) / kDepth * kDepth + 16); }
__host__ __device__ constexpr int few_rows(int64_t n) { return std::min(kFewRows, kFewBytes / few_stride(n)); }

struct FewParams {
    const int8_t* W;
    const float* sw;
    const void* x;
    const float* sx;
    int M, E, out, n;
    const int32_t* offsets;
    void* y;
};

template <int XT, int YT, bool GROUPED>
__global__ __launch_bounds__(kFewThreads) void int8_few_kernel(FewParams p) {
    extern __shared__ __align__(16) int8_t few_lds[];
    __shared__ int red[kFewWaves][64][4];
    __shared__ uint32_t most[kFewRows][kFewWaves];
    __shared__ float sxl[kFewRows];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int li = lane & 15, g = lane >> 4;
    const int row0 = blockIdx.x * 16;
    const int n = p.n, stride = few_stride(n);
    int e = 0, x0 = 0, rows = p.M;
    if constexpr (GROUPED) {
        const int s = blockIdx.y;
        auto begin = [&](int i) { return i == 0 ? 0 : min(max(p.offsets[i], 0), p.M); };
        // the last expert that begins at or before row s: 64 candidates at a time
        int lo = 0, span = p.E + 1;
        while (span > 1) {
            const int step = (span + 63) / 64, c = lo + lane * step;
            const uint64_t le = __ballot(c < lo + span && begin(min(c, p.E)) <= s);
            const int nlo = lo + (63 - __builtin_clzll(le)) * step;
            span = min(step, lo + span - nlo);
            lo = nlo;
        }
        e = __builtin_amdgcn_readfirstlane(lo);
        x0 = s;
        if (e == p.E) {  // a row of no expert
            const int o = row0 + (int)threadIdx.x;
            if (threadIdx.x < 16 && o < p.out) store_y<YT>(p.y, (int64_t)x0 * p.out + o, 0.f);
            return;
        }
        const int most_rows = few_rows(n);
        if ((s - begin(e)) % most_rows) return;
        rows = max(1, min(most_rows, begin(e + 1) - s));  // (1 at least whatever the offsets)
    }
    const int left = min(16, p.out - row0);
    const Rsrc wr = make_rsrc(p.W + ((int64_t)e * p.out + row0) * n, (uint32_t)left * (uint32_t)n);
    const uint32_t woff = (uint32_t)li * (uint32_t)n;  // (rows past the last are out of range and read zero)
    struct Frag {
        i32x4 lo, hi;
    };
    auto load_w = [&](int b) {
        const int c0 = b * kDepth + 16 * g, c1 = c0 + 64;
        const uint4 u = ld128(wr, c0 < n ? woff + c0 : kOob), v = ld128(wr, c1 < n ? woff + c1 : kOob);
        return Frag{{(int)u.x, (int)u.y, (int)u.z, (int)u.w}, {(int)v.x, (int)v.y, (int)v.z, (int)v.w}};
    };
    // x: item i of a thread is 8 values of row i / per.  A wave's memory accesses come back in order, so the first
    // values of x are asked for before the first weights and kept until their row's scale is known; further ones
    // are read again then.
    const int per = (n / 8 + kFewThreads - 1) / kFewThreads, items = rows * per;
    constexpr int kHeld = 2;
    auto load_x = [&](int i) {
        const int row = i / per, c = ((i - row * per) * kFewThreads + (int)threadIdx.x) * 8;
        return load_raw<XT>(p.x, (int64_t)(x0 + row) * n + c, c < n ? 8 : 0);
    };
    Frag w[2][kFewAhead];
    const int nb = (n + kDepth - 1) / kDepth;
    auto first_weights = [&]() {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < kFewAhead; ++i) w[0][i] = load_w(wave + i * kFewWaves);
        __builtin_amdgcn_sched_barrier(0);
    };
    if constexpr (XT == IQK_INT8) {
        // codes: 16 bytes a thread
        first_weights();
        const int chunks = n / 16;
        for (int i = threadIdx.x; i < rows * chunks; i += kFewThreads) {
            const int row = i / chunks, c = (i - row * chunks) * 16;
            *(uint4*)(few_lds + row * stride + c) = *(const uint4*)((const int8_t*)p.x + (int64_t)(x0 + row) * n + c);
        }
        if ((int)threadIdx.x < rows) sxl[threadIdx.x] = p.sx[x0 + threadIdx.x];
    } else {
        Raw<XT> held[kHeld];
#pragma unroll
        for (int i = 0; i < kHeld; ++i) held[i] = load_x(min(i, items - 1));
        first_weights();
        uint32_t bits = 0;
        auto take = [&](int i, const Raw<XT>& r) {
            bits = most_bits<XT>(bits, r);
            if ((i + 1) % per == 0) {
                bits = wave_max(lift_bits<XT>(bits));
                if (lane == 0) most[i / per][wave] = bits;
                bits = 0;
            }
        };
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
            if (i < items) take(i, held[i]);
        for (int i = kHeld; i < items; ++i) take(i, load_x(i));
        __syncthreads();
        auto keep = [&](int i, const Raw<XT>& r) {
            const int row = i / per, c = ((i - row * per) * kFewThreads + (int)threadIdx.x) * 8;
            uint32_t b = most[row][0];
#pragma unroll
            for (int u = 1; u < kFewWaves; ++u) b = max(b, most[row][u]);
            const RowScale s = row_scale(b);
            float v[8];
            widen_raw(r, v);
            if (c < n) *(uint2*)(few_lds + row * stride + c) = to_int8(v, s.factor);
            if (c == 0) sxl[row] = s.scale;
        };
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
            if (i < items) keep(i, held[i]);
        for (int i = kHeld; i < items; ++i) keep(i, load_x(i));
    }
    __syncthreads();

    const int8_t* xl = few_lds + min(li, rows - 1) * stride + 16 * g;
    i32x4 acc = {0, 0, 0, 0};
    // (codes past the depth in LDS are whatever they are: they meet zero weights)
    auto step = [&](int b0, const Frag (&cur)[kFewAhead], Frag (&next)[kFewAhead]) {
        if (b0 + kFewAhead * kFewWaves < nb) {
#pragma unroll
            for (int i = 0; i < kFewAhead; ++i) next[i] = load_w(b0 + (kFewAhead + i) * kFewWaves);
        }
#pragma unroll
        for (int i = 0; i < kFewAhead; ++i) {
            const int b = b0 + i * kFewWaves;
            if (b >= nb) break;
            const i32x4 lo = *(const i32x4*)(xl + b * kDepth), hi = *(const i32x4*)(xl + b * kDepth + 64);
            acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(cur[i].lo, lo, acc, 0, 0, 0);
            acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(cur[i].hi, hi, acc, 0, 0, 0);
        }
    };
    for (int b0 = wave; b0 < nb; b0 += 2 * kFewAhead * kFewWaves) {
        step(b0, w[0], w[1]);
        if (b0 + kFewAhead * kFewWaves < nb) step(b0 + kFewAhead * kFewWaves, w[1], w[0]);
    }
    *(i32x4*)red[wave][lane] = acc;
    __syncthreads();
    // one thread per result: value q of lane l is weight row 4 (l / 16) + q of row l % 16 of x
    const int i = threadIdx.x;
    if (i < 256) {
        const int r = i >> 4, o = i & 15;
        if (r < rows && o < left) {
            int v = 0;
#pragma unroll
            for (int u = 0; u < kFewWaves; ++u) v += red[u][16 * (o >> 2) + r][o & 3];
            float f = (float)v * (sxl[r] * p.sw[(int64_t)e * p.out + row0 + o]);
            if constexpr (YT == IQK_F16) asm("" : "+v"(f));  // (fused with the conversion the product would round once)
            store_y<YT>(p.y, (int64_t)(x0 + r) * p.out + row0 + o, f);
        }
    }
}

// ---------------------------------------------------------------------------
// up to 16 NT rows of x in codes, dense
// ---------------------------------------------------------------------------

// As above, with x's fragments straight from memory (the L2, after the first
// workgroups): each is used by one wave of the workgroup.  The next blocks are asked
// for while the last ones are multiplied.
// Bound: the fragments of x, which every 16 weight rows read again (17 rows by 4096
// x 4096 with their quantization 10.9 us, 32 rows 11).
template <int NT, int YT>
__global__ __launch_bounds__(kFewThreads) void int8_rows_kernel(FewParams p) {
    __shared__ int red[kFewWaves][NT][64][4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int li = lane & 15, g = lane >> 4;
    const int n = p.n, nb = (n + kDepth - 1) / kDepth;
    const int row0 = blockIdx.x * 16, left = min(16, p.out - row0);
    const Rsrc wr = make_rsrc(p.W + (int64_t)row0 * n, (uint32_t)left * (uint32_t)n);  // (rows past the last read zero)
    const uint32_t woff = (uint32_t)li * (uint32_t)n;
    const int8_t* xr[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) xr[t] = (const int8_t*)p.x + (int64_t)min(16 * t + li, p.M - 1) * n;  // (rows past the last repeat it)
    struct Stage {
        i32x4 w[2], x[NT][2];
    } st[2];
    // (blocks past the last have zero weights; a chunk of x past the depth is its row's first)
    auto request = [&](int b, Stage& s) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c = b * kDepth + 16 * g + 64 * h;
            const uint4 u = ld128(wr, c < n ? woff + c : kOob);
            s.w[h] = i32x4{(int)u.x, (int)u.y, (int)u.z, (int)u.w};
#pragma unroll
            for (int t = 0; t < NT; ++t) s.x[t][h] = *(const i32x4*)(xr[t] + (c < n ? c : 0));
        }
    };
    i32x4 acc[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t] = i32x4{0, 0, 0, 0};
    auto multiply = [&](const Stage& s) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(s.w[h], s.x[t][h], acc[t], 0, 0, 0);
    };
    request(wave, st[0]);
    for (int b = wave; b < nb; b += 2 * kFewWaves) {
        request(b + kFewWaves, st[1]);
        multiply(st[0]);
        request(b + 2 * kFewWaves, st[0]);
        multiply(st[1]);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) *(i32x4*)red[wave][t][lane] = acc[t];
    __syncthreads();
    // sixteen neighbouring threads write the results of one row of x
    for (int i = threadIdx.x; i < 256 * NT; i += kFewThreads) {
        const int r = i >> 4, o = i & 15;
        if (r >= p.M || o >= left) continue;
        int v = 0;
#pragma unroll
        for (int u = 0; u < kFewWaves; ++u) v += red[u][r >> 4][16 * (o >> 2) + (r & 15)][o & 3];
        float f = (float)v * (p.sx[r] * p.sw[row0 + o]);
        if constexpr (YT == IQK_F16) asm("" : "+v"(f));
        store_y<YT>(p.y, (int64_t)r * p.out + row0 + o, f);
    }
}

}  // namespace

bool int8_few_fits(int64_t M, int64_t n, bool grouped) {
    return grouped ? M <= kFewGrouped && few_rows(n) >= 1 : M <= std::min(kFewDense, few_rows(n));
}

// Every 16 weight rows read x again, which tiles of 128 do less often: out = 4096, in = 4096, 17 rows 10.9 us with the
// quantization against 15.0 in tiles of 16 x 128, 33 rows (four fragments of x a weight) 14.9 against 15.0; out = 8192,
// 32 rows 17.8 against 17.4; out = 16384, in = 2048, 17 rows 14.4 against 12.7.
bool int8_rows_fits(int64_t M, int64_t out) { return M <= 32 && out <= 8192; }

hipError_t launch_int8_prep(const Int8QuantLaunch& q, const Int8Plan& g, hipStream_t s) {
    const bool quantize = q.x_dtype != IQK_INT8;
    const int team = q.n <= 64 * 8 * kChunks ? 64 : 256;
    const int64_t per = kThreads / team;
    PrepParams p{q.x, q.rows, (int)q.n, q.codes, q.scales, quantize ? (q.rows + per - 1) / per : 0, g.E, g.tile, g.offsets, g.tiles};
    const int64_t groups = p.quant_groups + (g.offsets ? 1 : 0);
    if (groups == 0) return hipSuccess;
    constexpr int64_t kMost = 1 << 22;  // (a launch has less than 2^32 threads in a row of its grid)
    const dim3 grid((unsigned)std::min(groups, kMost), (unsigned)((groups + kMost - 1) / kMost));
    by_float(quantize ? q.x_dtype : IQK_F32, [&](auto xt) {
        constexpr int XT = decltype(xt)::value;
        if (team == 64) hipLaunchKernelGGL((int8_prep_kernel<XT, 64, true>), grid, dim3(kThreads), 0, s, p);
        else if (q.n <= 256 * 8 * kChunks) hipLaunchKernelGGL((int8_prep_kernel<XT, 256, true>), grid, dim3(kThreads), 0, s, p);
        else hipLaunchKernelGGL((int8_prep_kernel<XT, 256, false>), grid, dim3(kThreads), 0, s, p);
    });
    return hipGetLastError();
}

hipError_t launch_int8_few(const Int8Launch& a, hipStream_t s) {
    const FewParams p{a.codes, a.scales, a.x, a.x_scales, (int)a.M, (int)a.E, (int)a.out, (int)a.n, a.offsets, a.y};
    const bool grouped = a.offsets != nullptr;
    const int rows = (int)std::min<int64_t>(a.M, few_rows(a.n));
    const unsigned lds = (unsigned)(rows * few_stride(a.n));
    const dim3 grid((unsigned)((a.out + 15) / 16), grouped ? (unsigned)a.M : 1u);
    by_float(a.y_dtype, [&](auto yt) {
        auto go = [&](auto xt) {
            constexpr int XT = decltype(xt)::value, YT = decltype(yt)::value;
            if (grouped) hipLaunchKernelGGL((int8_few_kernel<XT, YT, true>), grid, dim3(kFewThreads), lds, s, p);
            else hipLaunchKernelGGL((int8_few_kernel<XT, YT, false>), grid, dim3(kFewThreads), lds, s, p);
        };
        if (a.x_dtype == IQK_INT8) go(std::integral_constant<int, IQK_INT8>{});
        else by_float(a.x_dtype, go);
    });
    return hipGetLastError();
}

hipError_t launch_int8_rows(const Int8Launch& a, hipStream_t s) {
    if (a.M > 32) return hipErrorInvalidValue;
    const FewParams p{a.codes, a.scales, a.x, a.x_scales, (int)a.M, 1, (int)a.out, (int)a.n, nullptr, a.y};
    const dim3 grid((unsigned)((a.out + 15) / 16)), block(kFewThreads);
    by_float(a.y_dtype, [&](auto yt) {
        constexpr int YT = decltype(yt)::value;
        if (a.M <= 16) hipLaunchKernelGGL((int8_rows_kernel<1, YT>), grid, block, 0, s, p);
        else hipLaunchKernelGGL((int8_rows_kernel<2, YT>), grid, block, 0, s, p);
    });
    return hipGetLastError();
}

}  // namespace iqk
