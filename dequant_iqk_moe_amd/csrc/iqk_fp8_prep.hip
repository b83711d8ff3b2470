// iqk_fp8_prep.hip -- what an 8-bit product needs before it: quantized
// activations and, for routed pairs, the pairs grouped by expert.
//
// The grouping here is not iqk_route's: the product of a pair does not depend
// on its place in its expert's group, so pairs take places as they come (LDS
// atomics) instead of in order, and the ranking that a stable order costs
// goes.  One launch quantizes, groups and writes the NaN rows of pairs that no
// expert here takes, each by workgroups of its own (3072 pairs of 256 experts
// and 3072 x 2048 values: 7.3 us; iqk_route alone takes 9.5 in the kernel
// trace).  Above 8192 pairs several workgroups count and a second launch places
// (24576 pairs and 4096 x 4096 values: 12.8 + 8.1 us).
#include <algorithm>

#include "iqk_fp8_device.h"

namespace iqk {
namespace {

constexpr int kPrepThreads = 1024;
constexpr int kPrepWaves = kPrepThreads / 64;
constexpr int kPrepBlocks = kPrepThreads / 16;  // blocks of 128 values per workgroup
constexpr int kGroupE = 1024;                   // experts one workgroup counts, one per thread

// A launch's x extent holds fewer than 2^32 threads, so many workgroups take
// rows of 2^20 of a plane.
dim3 plane(int64_t groups) {
    const int64_t x = std::min<int64_t>(groups, 1 << 20);
    return dim3((unsigned)x, (unsigned)((groups + x - 1) / x));
}
__device__ __forceinline__ int64_t plane_index() { return (int64_t)blockIdx.y * gridDim.x + blockIdx.x; }

// 16 lanes own one block of 128, 8 consecutive values each (rows are multiples
// of 16 values, so a lane's 8 are all inside a row or all past its end).  Bound
// by bytes: 8192 x 4096 bfloat16 (102 MB read and written) in 18.5 us = 5.5
// TB/s, where a 4 GiB copy runs at 4.75.
template <int DT>
__device__ __forceinline__ void quantize_blocks(const Fp8QuantLaunch& p, int64_t block, int threads) {
    const int64_t nb = (p.n + kBlock - 1) / kBlock;
    const int64_t i = block * (threads / 16) + (threadIdx.x >> 4);
    const int sub = threadIdx.x & 15;
    if (i >= p.rows * nb) return;  // (whole groups of 16 lanes leave together)
    const int64_t row = i / nb, b = i - row * nb;
    const int64_t c = b * kBlock + 8 * sub;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (c < p.n) load8<DT>(p.x, row * p.n + c, v);
    const float a = block_amax(v);
    const float r = kE4m3Max / a;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= r;
    if (c < p.n) *(uint2*)(p.codes + row * p.n + c) = to_e4m3(v);
    if (sub == 0) p.scales[i] = a / kE4m3Max;
}

template <int DT>
__global__ __launch_bounds__(256) void fp8_quantize_kernel(Fp8QuantLaunch p) {
    quantize_blocks<DT>(p, plane_index(), 256);
}

// Inclusive sum over the workgroup of one value per thread.
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t* part) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint64_t o = __shfl_up(v, d);
        if (lane >= d) v += o;
    }
    if (lane == 63) part[wave] = v;
    __syncthreads();
    uint64_t before = 0;
    for (int w = 0; w < wave; ++w) before += part[w];
    __syncthreads();
    return v + before;
}

// Rows of y for pairs whose id lies outside [0, E) become NaN: a wave looks at
// p.nan_pairs of them.  By workgroups of their own: written by those that group,
// the rows of 24576 pairs of 2048 bfloat16 values, 7 of 8 outside as on a device
// that holds an eighth of the experts, made the product 820 us long; it takes 200
// so, and 300 with every id inside.
__device__ __forceinline__ void nan_rows(const Fp8GroupLaunch& p, int64_t first) {
    const int lane = threadIdx.x & 63;
    const int64_t q = first + lane;
    const int e = lane < p.nan_pairs && q < p.P ? p.ids[q] : 0;
    uint64_t bad = __ballot(e < 0 || e >= p.E);
    const int size = p.y_half ? 2 : 4, bytes = p.out * size;
    const uint32_t nan = p.y_half ? 0x7FFF7FFFu : 0x7FC00000u;  // (0x7FFF: in float16 and in bfloat16)
    const uint4 four = {nan, nan, nan, nan};
    while (bad) {
        char* row = (char*)p.y + (first + __builtin_ctzll(bad)) * (int64_t)bytes;
        bad &= bad - 1;
        for (int i = 16 * lane; i + 16 <= bytes; i += 16 * 64) __builtin_memcpy(row + i, &four, 16);  // (any address)
        const int i = (bytes & ~15) + size * lane;
        if (i < bytes) __builtin_memcpy(row + i, &nan, size == 2 ? 2 : 4);
    }
}

// Counts of a slice's pairs per expert.
__device__ __forceinline__ void count_slice(const Fp8GroupLaunch& p, int64_t p0, int64_t p1, int32_t* cnt) {
    for (int e = threadIdx.x; e < p.E; e += kPrepThreads) cnt[e] = 0;
    __syncthreads();
    for (int64_t q = p0 + threadIdx.x; q < p1; q += kPrepThreads) {
        const int e = p.ids[q];
        if (e >= 0 && e < p.E) atomicAdd(&cnt[e], 1);
    }
    __syncthreads();
}

// Offsets, tile counts and the places of slice h's pairs, from the counts of
// all slices (`before` = the pairs of this thread's expert in earlier slices,
// `total` = in all).  Slice 0 writes the arrays that all share.
__device__ __forceinline__ void place_slice(const Fp8GroupLaunch& p, int h, int64_t p0, int64_t p1, int32_t before,
                                            int32_t total, int32_t* cur, uint64_t* part) {
    const int e = threadIdx.x;
    const uint64_t mine = (uint32_t)total | ((uint64_t)((total + p.tile - 1) / p.tile) << 32);
    const uint64_t sum = block_scan(e < p.E ? mine : 0, part) - (e < p.E ? mine : 0);
    if (e < p.E) cur[e] = (int32_t)(uint32_t)sum + before;
    if (h == 0 && e <= p.E && e < kPrepThreads) {
        p.offsets[e] = (int32_t)(uint32_t)sum;
        p.tiles[e] = (int32_t)(sum >> 32);
    }
    if (h == 0 && p.E == kPrepThreads && e == kPrepThreads - 1) {
        p.offsets[e + 1] = (int32_t)(uint32_t)(sum + mine);
        p.tiles[e + 1] = (int32_t)((sum + mine) >> 32);
    }
    __syncthreads();
    for (int64_t q = p0 + threadIdx.x; q < p1; q += kPrepThreads) {
        const int id = p.ids[q];
        if (id >= 0 && id < p.E) p.perm[atomicAdd(&cur[id], 1)] = (int32_t)q;
    }
}

// Workgroups below p.slices group (one slice: count and place; more: count, the
// next kernel places), the next p.nans write NaN rows, the others quantize.
template <int DT>
__global__ __launch_bounds__(kPrepThreads) void fp8_prep_kernel(Fp8GroupLaunch p, Fp8QuantLaunch q) {
    __shared__ int32_t cnt[kGroupE];
    __shared__ uint64_t part[kPrepWaves];
    int64_t group = plane_index();
    if (group < p.slices) {
        const int h = (int)group;
        const int64_t p0 = h * p.slice, p1 = min(p0 + p.slice, p.P);
        count_slice(p, p0, p1, cnt);
        if (p.slices == 1) {
            const int32_t total = (int)threadIdx.x < p.E ? cnt[threadIdx.x] : 0;
            place_slice(p, 0, p0, p1, 0, total, cnt, part);
        } else {
            for (int e = threadIdx.x; e < p.E; e += kPrepThreads) p.hist[(int64_t)h * p.E + e] = cnt[e];
        }
        return;
    }
    group -= p.slices;
    if (group < p.nans) return nan_rows(p, (group * kPrepWaves + (threadIdx.x >> 6)) * p.nan_pairs);
    if constexpr (DT != IQK_E4M3) quantize_blocks<DT>(q, group - p.nans, kPrepThreads);
}

__global__ __launch_bounds__(kPrepThreads) void fp8_place_kernel(Fp8GroupLaunch p) {
    __shared__ int32_t cur[kGroupE];
    __shared__ uint64_t part[kPrepWaves];
    const int h = blockIdx.x, e = threadIdx.x;
    int32_t before = 0, total = 0;
    if (e < p.E) {
        for (int i = 0; i < p.slices; ++i) {
            const int32_t c = p.hist[(int64_t)i * p.E + e];
            before += i < h ? c : 0;
            total += c;
        }
    }
    const int64_t p0 = h * p.slice, p1 = min(p0 + p.slice, p.P);
    place_slice(p, h, p0, p1, before, total, cur, part);
}

// For more experts than one workgroup counts: the NaN rows that iqk_route's
// grouping leaves out, and tile counts from its offsets.
__global__ __launch_bounds__(kPrepThreads) void fp8_nan_kernel(Fp8GroupLaunch p) {
    nan_rows(p, ((int64_t)blockIdx.x * kPrepWaves + (threadIdx.x >> 6)) * p.nan_pairs);
}

__global__ __launch_bounds__(kPrepThreads) void fp8_tiles_kernel(Fp8GroupLaunch p) {
    __shared__ uint64_t part[kPrepWaves];
    uint64_t base = 0;
    for (int e0 = 0; e0 < p.E; e0 += kPrepThreads) {
        const int e = e0 + threadIdx.x;
        const uint64_t c = e < p.E ? (p.offsets[e + 1] - p.offsets[e] + p.tile - 1) / p.tile : 0;
        const uint64_t sum = block_scan(c, part);
        if (e < p.E) p.tiles[e] = (int32_t)(base + sum - c);
        __shared__ uint64_t all;
        if (threadIdx.x == kPrepThreads - 1) all = sum;
        __syncthreads();
        base += all;
        __syncthreads();
    }
    if (threadIdx.x == 0) p.tiles[p.E] = (int32_t)base;
}

}  // namespace

hipError_t launch_fp8_quantize(const Fp8QuantLaunch& a, hipStream_t s) {
    const int64_t blocks128 = a.rows * ((a.n + kBlock - 1) / kBlock);
    by_float(a.x_dtype, [&](auto dt) {
        hipLaunchKernelGGL((fp8_quantize_kernel<decltype(dt)::value>), plane((blocks128 + 15) / 16), dim3(256), 0, s, a);
    });
    return hipGetLastError();
}

int fp8_group_slices(int64_t P) {
    // one workgroup up to 8192 pairs, then slices of as many, 64 at most
    return (int)std::min<int64_t>(64, (P + 8191) / 8192);
}

hipError_t launch_fp8_prep(Fp8GroupLaunch g, const Fp8QuantLaunch& q, hipStream_t s) {
    const bool quantize = q.x_dtype != IQK_E4M3;
    const int64_t blocks128 = quantize ? q.rows * ((q.n + kBlock - 1) / kBlock) : 0;
    const int64_t qb = (blocks128 + kPrepBlocks - 1) / kPrepBlocks;
    // Eight pairs a wave spread few pairs' rows over the card (3072 pairs of 4096 float32 values, none inside: 28 us
    // against 67 with 32 a wave); of many pairs, that many waves hold up the quantization behind them (24576: 19 us
    // for this launch with 8 a wave, 13 with 32, as without any).
    g.nan_pairs = g.P <= 8192 ? 8 : 32;
    g.nans = (g.P + kPrepWaves * g.nan_pairs - 1) / (kPrepWaves * g.nan_pairs);
    if (g.E > kGroupE) {
        hipError_t e = launch_route(RouteLaunch{g.ids, g.P, g.E, 0, g.counts, g.offsets, g.perm}, s);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(fp8_nan_kernel, dim3((unsigned)g.nans), dim3(kPrepThreads), 0, s, g);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        hipLaunchKernelGGL(fp8_tiles_kernel, dim3(1), dim3(kPrepThreads), 0, s, g);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        return quantize ? launch_fp8_quantize(q, s) : hipSuccess;
    }
    g.slices = fp8_group_slices(g.P);
    g.slice = (g.P + g.slices - 1) / g.slices;
    const dim3 grid = plane(g.slices + qb + g.nans);
    if (quantize) {
        by_float(q.x_dtype, [&](auto dt) {
            hipLaunchKernelGGL((fp8_prep_kernel<decltype(dt)::value>), grid, dim3(kPrepThreads), 0, s, g, q);
        });
    } else {
        hipLaunchKernelGGL((fp8_prep_kernel<IQK_E4M3>), grid, dim3(kPrepThreads), 0, s, g, q);
    }
    if (g.slices > 1) {
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(fp8_place_kernel, dim3((unsigned)g.slices), dim3(kPrepThreads), 0, s, g);
    }
    return hipGetLastError();
}

}  // namespace iqk
