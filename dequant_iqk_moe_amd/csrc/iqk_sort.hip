// iqk_sort.hip -- token rows in the order of their experts, back again with
// the router's weights, and the gradient of that.
//
//   xs[row(t, j)] = x[t],  y[t] = sum_j w[t, j] ys[row(t, j)],
//   d_ys[row(t, j)] = w[t, j] dy[t],  d_w[t, j] = <dy[t], ys[row(t, j)]>
//
// where row(t, j) is the place of pair t k + j in a stable sort by expert, the
// pairs whose id is outside [0, E) last.  place[t, j] = row(t, j), and
// -1 - row(t, j) for those, whose rows count as zeros.
//
// Bound: bytes.  All row kernels go token by token, so a token's own row is
// read or written once for its k expert rows, in pieces of 16 bytes a lane; its
// places are read before any row.  Measured, bfloat16 rows of 4096 (a large copy
// runs at 4.8 TB/s): 8192 tokens of 6 slots sorted in 105 us, 85 of them the
// copy (5.5 TB/s); 500 tokens of float32 rows unsorted in 10 us (5 TB/s); the
// gradient of 4096 tokens in 92 us, 85 in the kernel (5.1 TB/s).
#include <algorithm>

#include "iqk_block.h"
#include "iqk_rows_device.h"

namespace iqk {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kKeys = 8;  // keys that a pass over the ids counts at once

struct SortParams {
    const uint8_t* x;
    const int32_t* ids;
    int64_t T, P;
    int k, E;
    int64_t row;  // bytes
    int32_t* hist;
    int slices;
    int64_t slice;
    uint8_t* xs;
    int32_t *offsets, *place;
};

// The expert of pair p, E for an id outside [0, E).
__device__ __forceinline__ int expert_of(const SortParams& p, int64_t pair) {
    const int e = p.ids[pair];
    return (unsigned)e < (unsigned)p.E ? e : p.E;
}

// Copies part `part` of `parts` of token t's row to the rows of its slots from j0 on,
// kKeys of them (zeros where they have no expert); at(j) is place[t, j].
template <class At>
__device__ __forceinline__ void copy_slots(const SortParams& p, int64_t t, int j0, int part, int parts, At at) {
    const int64_t chunks = p.row / 16;
    const uint8_t* src = p.x + t * p.row;
    int32_t to[kKeys];  // (all before the first store)
#pragma unroll
    for (int j = 0; j < kKeys; ++j) to[j] = at(min(j0 + j, p.k - 1));
    auto row = [&](int j) { return p.xs + (int64_t)(to[j] < 0 ? -1 - to[j] : to[j]) * p.row; };
    for (int64_t c = (int64_t)part * kThreads + threadIdx.x; c < chunks; c += (int64_t)parts * kThreads) {
        uint4 v;
        __builtin_memcpy(&v, src + 16 * c, 16);
#pragma unroll
        for (int j = 0; j < kKeys; ++j) {
            if (j0 + j >= p.k) continue;
            const uint4 z = to[j] < 0 ? make_uint4(0, 0, 0, 0) : v;
            __builtin_memcpy(row(j) + 16 * c, &z, 16);
        }
    }
    // what no 16 bytes hold, two at a time
    const int64_t tail = 16 * chunks + 2 * threadIdx.x;
    if (part == parts - 1 && tail < p.row) {
        const uint16_t v = *(const uint16_t*)(src + tail);
#pragma unroll
        for (int j = 0; j < kKeys; ++j)
            if (j0 + j < p.k) *(uint16_t*)(row(j) + tail) = to[j] < 0 ? 0 : v;
    }
}

// ---------------------------------------------------------------------------
// few pairs: one launch
// ---------------------------------------------------------------------------

// The place of pair p is the number of pairs q with (expert, q) below its own, and
// offsets[e] the number below (e, 0).  A workgroup counts up to kKeys of these, the
// pairs of a token or offsets: P^2 / 64 comparisons of a wave in all, on the whole
// card, and no pass that waits for another.  Each is a compare, a bit count and an
// addition, the latter two on the scalar unit that a CU's waves share.
constexpr int64_t kDirect = 8192;         // pairs that a key holds the index of
constexpr int kShift = 13;                // (its lower bits; the expert is above)
constexpr int64_t kDirectWork = 8 << 20;  // comparisons of a lane with kKeys keys up to which the ids go this way
constexpr int kBatch = 2;                 // ids of a thread that are asked for together (768 x 8 pairs: one 16.0 us, two 9.9, four
                                          // 13.6, whose comparisons wait for scalar registers)

__global__ __launch_bounds__(kThreads) void sort_direct_kernel(SortParams p) {
    __shared__ int32_t part[kWaves][kKeys];
    __shared__ int32_t at[kKeys];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int groups = (p.k + kKeys - 1) / kKeys, rows = (int)p.T * groups;  // workgroups that have rows
    const bool pairs = (int)blockIdx.x < rows;
    if (!pairs && blockIdx.y > 0) return;
    const int t = blockIdx.x / groups, j0 = ((int)blockIdx.x - t * groups) * kKeys, e0 = ((int)blockIdx.x - rows) * kKeys;
    const int count = pairs ? min(kKeys, p.k - j0) : min(kKeys, p.E + 1 - e0), p0 = t * p.k + j0;
    uint32_t key[kKeys];
    int below[kKeys];
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
        uint32_t v = 0;
        if (i < count) v = pairs ? (uint32_t)expert_of(p, p0 + i) << kShift | (uint32_t)(p0 + i) : (uint32_t)(e0 + i) << kShift;
        key[i] = __builtin_amdgcn_readfirstlane(v);
        below[i] = 0;
    }
    const int P = (int)p.P;
    for (int q0 = wave * 64; q0 < P; q0 += kBatch * kThreads) {
        uint32_t v[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int q = q0 + b * kThreads + lane;
            const uint32_t e = (uint32_t)expert_of(p, min(q, P - 1));
            v[b] = q < P ? e << kShift | (uint32_t)q : 0xFFFFFFFFu;
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
#pragma unroll
            for (int i = 0; i < kKeys; ++i) below[i] += __builtin_popcountll(__ballot(v[b] < key[i]));
    }
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < kKeys; ++i) part[wave][i] = below[i];
    }
    __syncthreads();
    if ((int)threadIdx.x < count) {
        const int u = threadIdx.x;
        int32_t v = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) v += part[w][u];
        if (pairs) {
            if (expert_of(p, p0 + u) == p.E) v = -1 - v;
            at[u] = v;
            if (blockIdx.y == 0) p.place[p0 + u] = v;
        } else {
            p.offsets[e0 + u] = v;
        }
    }
    __syncthreads();
    if (pairs) copy_slots(p, t, j0, blockIdx.y, gridDim.y, [&](int j) { return __builtin_amdgcn_readfirstlane(at[j - j0]); });
}

// ---------------------------------------------------------------------------
// many pairs: slices are counted, then placed, then the rows are copied
// ---------------------------------------------------------------------------

// A thousand pairs a slice: the counts of 48 slices (49152 pairs, 256 experts) are
// summed in 2 of the placing kernel's 7.7 us, which ranks 256 pairs a wave; slices
// of 512 rank half as many and sum twice as many counts, in the same time.
constexpr int64_t kSlices = 128, kSlicePairs = 1024;

__global__ __launch_bounds__(kThreads) void sort_count_kernel(SortParams p) {
    extern __shared__ int32_t counts[];
    for (int e = threadIdx.x; e <= p.E; e += kThreads) counts[e] = 0;
    __syncthreads();
    const int64_t q1 = min(((int64_t)blockIdx.x + 1) * p.slice, p.P);
    for (int64_t q = (int64_t)blockIdx.x * p.slice + threadIdx.x; q < q1; q += kThreads) atomicAdd(&counts[expert_of(p, q)], 1);
    __syncthreads();
    for (int e = threadIdx.x; e <= p.E; e += kThreads) p.hist[(int64_t)blockIdx.x * (p.E + 1) + e] = counts[e];
}

// A slice's pairs take the places behind those of lower experts and of the same
// expert in earlier slices, in order: the slice is cut into a run for each wave,
// whose counts are made first (of pairs, so their order does not matter), and a
// wave ranks 64 pairs at a time by the lanes before them with the same expert.
__global__ __launch_bounds__(kThreads) void sort_place_kernel(SortParams p) {
    extern __shared__ int32_t next[];  // [kWaves][E + 1]
    __shared__ int32_t sums[kWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int stride = p.E + 1;
    for (int i = threadIdx.x; i < kWaves * stride; i += kThreads) next[i] = 0;
    __syncthreads();
    const int64_t q0 = (int64_t)blockIdx.x * p.slice, run = (p.slice / kWaves + 63) / 64 * 64;
    const int64_t end = min(q0 + p.slice, p.P), r0 = min(q0 + wave * run, end), r1 = wave == kWaves - 1 ? end : min(r0 + run, end);
    for (int64_t q = r0 + lane; q < r1; q += 64) atomicAdd(&next[wave * stride + expert_of(p, q)], 1);
    __syncthreads();
    int before = 0;  // pairs of the experts below those of this pass
    constexpr int kEach = 2, kTogether = 16;  // experts of a thread, slices asked for at once: a batch costs a memory latency
    for (int base = 0; base < stride; base += kEach * kThreads) {
        int total[kEach] = {}, earlier[kEach] = {};
        for (int s0 = 0; s0 < p.slices; s0 += kTogether) {
            int v[kTogether][kEach];
#pragma unroll
            for (int i = 0; i < kTogether; ++i)
#pragma unroll
                for (int u = 0; u < kEach; ++u)
                    v[i][u] = p.hist[(uint32_t)(min(s0 + i, p.slices - 1) * stride + min(base + u * kThreads + (int)threadIdx.x, p.E))];
#pragma unroll
            for (int i = 0; i < kTogether; ++i)
#pragma unroll
                for (int u = 0; u < kEach; ++u) {
                    total[u] += s0 + i < p.slices ? v[i][u] : 0;
                    earlier[u] += s0 + i < (int)blockIdx.x ? v[i][u] : 0;
                }
        }
#pragma unroll
        for (int u = 0; u < kEach; ++u) {
            const int e = base + u * kThreads + threadIdx.x;
            const int mine = e < stride ? total[u] : 0;
            int upto = mine;  // inclusive sum over the wave
#pragma unroll
            for (int d = 1; d < 64; d *= 2) {
                const int o = __shfl_up(upto, d);
                if (lane >= d) upto += o;
            }
            if (lane == 63) sums[wave] = upto;
            __syncthreads();
            int at = before + upto - mine;
            for (int w = 0; w < kWaves; ++w) {
                if (w < wave) at += sums[w];
                before += sums[w];
            }
            if (e < stride) {
                if (blockIdx.x == 0) p.offsets[e] = at;
                at += earlier[u];
                for (int w = 0; w < kWaves; ++w) {
                    const int v = next[w * stride + e];
                    next[w * stride + e] = at;
                    at += v;
                }
            }
            __syncthreads();
        }
    }
    const int bits = 32 - __builtin_clz(p.E);  // an expert index, E among them
    for (int64_t q = r0; q < r1; q += 64) {
        const bool there = q + lane < r1;
        const int e = there ? expert_of(p, q + lane) : -1;
        uint64_t same = __ballot(there);
        for (int b = 0; b < bits; ++b) {
            const uint64_t set = __ballot(e >> b & 1);
            same &= e >> b & 1 ? set : ~set;
        }
        if (there) {
            const uint64_t before_me = same & ((1ull << lane) - 1);
            const int32_t row = next[wave * stride + e] + __builtin_popcountll(before_me);
            p.place[q + lane] = e == p.E ? -1 - row : row;
            __builtin_amdgcn_wave_barrier();
            if (same >> lane == 1) next[wave * stride + e] = row + 1;  // the last of its expert
        }
        __builtin_amdgcn_wave_barrier();
    }
}

__global__ __launch_bounds__(kThreads) void sort_copy_kernel(SortParams p) {
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        const int32_t* place = p.place + t * p.k;
        for (int j0 = 0; j0 < p.k; j0 += kKeys) copy_slots(p, t, j0, blockIdx.y, gridDim.y, [&](int j) { return place[j]; });
    }
}

// ---------------------------------------------------------------------------
// back to the tokens
// ---------------------------------------------------------------------------

struct UnsortParams {
    const void* ys;
    const int32_t* place;
    const float* w;
    int64_t T, P, n;
    int k;
    void* y;
    const void* dy;
    void* d_ys;
    float* d_w;
};

// Rows of at least eight values are taken in chunks of eight, the last of which
// ends with the row: what it shares with the one before is made twice, with the same
// bits.  So no load has a branch for the row's end, and all of a token's rows are
// asked for together (gradient of 4096 x 6 rows of 4096: 109 us with the branches,
// 85 without; 1025 x 8 rows of 2047 float32 values back 16 and 13).  Shorter rows
// are one chunk.
struct Chunk {
    int64_t c;       // its first value
    int left, twice;  // its values, and how many of them are the one before's too
};
template <bool LONG>
__device__ __forceinline__ Chunk chunk_at(int64_t c, int64_t n) {
    if constexpr (LONG) {
        const int64_t at = min(c, n - 8);
        return {at, 8, (int)(c - at)};
    }
    return {c, (int)(n - c), 0};
}

// kAhead of a token's slots: their places and weights, read before any row.
constexpr int kAhead = kKeys;
struct Slots {
    int32_t row[kAhead];
    float w[kAhead];
};
__device__ __forceinline__ Slots load_slots(const UnsortParams& p, int64_t t, int j0) {
    Slots s;
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
        const int64_t at = t * p.k + min(j0 + j, p.k - 1);
        s.row[j] = p.place[at];
        s.w[j] = p.w ? p.w[at] : 1.f;
    }
    return s;
}
__device__ __forceinline__ bool known(const UnsortParams& p, int32_t row) { return (uint32_t)row < (uint64_t)p.P; }
// A row of ys to read for a pair: its own, or row 0, which is then not used.
__device__ __forceinline__ int64_t row_to_read(const UnsortParams& p, int32_t row) { return known(p, row) ? row : 0; }

// Slots are added in their order, each product rounded by itself, as iqk_combine
// does: the two agree bit for bit.
template <int ST, int YT, bool LONG>
__global__ __launch_bounds__(kThreads) void unsort_kernel(UnsortParams p) {
    const int64_t c0 = ((int64_t)blockIdx.y * kThreads + threadIdx.x) * 8;
    if (c0 >= p.n) return;
    const Chunk c = chunk_at<LONG>(c0, p.n);
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int j0 = 0; j0 < p.k; j0 += kAhead) {
            const Slots s = load_slots(p, t, j0);
            Raw<ST> r[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                if (j0 + j < p.k) r[j] = load_raw<ST>(p.ys, row_to_read(p, s.row[j]) * p.n + c.c, LONG ? 8 : c.left);
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                if (j0 + j >= p.k) continue;
                float v[8];
                widen_raw(r[j], v);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float m = __fmul_rn(s.w[j], known(p, s.row[j]) ? v[i] : 0.f);
                    acc[i] = j0 + j == 0 ? m : __fadd_rn(acc[i], m);
                }
            }
        }
        store_some<YT>(p.y, t * p.n + c.c, acc, LONG ? 8 : c.left);
    }
}

// A workgroup owns a token: dy's chunks are read once for all of its pairs (of
// up to kAhead; further ones read them again), whose dot products are summed over
// lanes and waves in a fixed order.
template <int ST, int YT, bool LONG>
__global__ __launch_bounds__(kThreads) void unsort_grad_kernel(UnsortParams p) {
    __shared__ float part[kWaves][kAhead];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        for (int j0 = 0; j0 < p.k; j0 += kAhead) {
            const Slots s = load_slots(p, t, j0);
            const int slots = min(kAhead, p.k - j0);
            float dot[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) dot[j] = 0.f;
            for (int64_t c0 = (int64_t)threadIdx.x * 8; c0 < p.n; c0 += kThreads * 8) {
                const Chunk c = chunk_at<LONG>(c0, p.n);
                const int left = LONG ? 8 : c.left;
                float d[8];
                const Raw<YT> dr = load_raw<YT>(p.dy, t * p.n + c.c, left);
                Raw<ST> r[kAhead];
                if (p.d_w) {
#pragma unroll
                    for (int j = 0; j < kAhead; ++j)
                        if (j < slots) r[j] = load_raw<ST>(p.ys, row_to_read(p, s.row[j]) * p.n + c.c, left);
                }
                widen_raw(dr, d);
                if (p.d_ys) {
#pragma unroll
                    for (int j = 0; j < kAhead; ++j) {
                        if (j >= slots) continue;
                        const int64_t row = s.row[j], to = row < 0 ? -1 - row : row;
                        if (to >= p.P) continue;
                        float v[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[i] = row < 0 ? 0.f : s.w[j] * d[i];
                        store_some<ST>(p.d_ys, to * p.n + c.c, v, left);
                    }
                }
                if (p.d_w) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) d[i] = LONG && i < c.twice ? 0.f : d[i];
#pragma unroll
                    for (int j = 0; j < kAhead; ++j) {
                        if (j >= slots) continue;
                        float v[8];
                        widen_raw(r[j], v);
#pragma unroll
                        for (int i = 0; i < 8; ++i) dot[j] = __builtin_fmaf(d[i], LONG && i < c.twice ? 0.f : v[i], dot[j]);
                    }
                }
            }
            if (!p.d_w) continue;
#pragma unroll
            for (int j = 0; j < kAhead; ++j) dot[j] = wave_sum(dot[j]);
            if (lane == 0) {
#pragma unroll
                for (int j = 0; j < kAhead; ++j) part[wave][j] = dot[j];
            }
            __syncthreads();
            if ((int)threadIdx.x < slots) {
                float v = 0.f;
#pragma unroll
                for (int w = 0; w < kWaves; ++w) v += part[w][threadIdx.x];
                p.d_w[t * p.k + j0 + threadIdx.x] = known(p, p.place[t * p.k + j0 + threadIdx.x]) ? v : 0.f;
            }
            __syncthreads();
        }
    }
}

int64_t size_of(int dtype) { return dtype == IQK_F32 ? 4 : 2; }

// Workgroups that share a token's row of `chunks` pieces of 16 bytes or 8 values:
// each thread has one piece where tokens are few, more where they fill the card.
unsigned row_parts(int64_t T, int64_t chunks) {
    const int64_t most = std::max<int64_t>(1, (chunks + kThreads - 1) / kThreads);
    return (unsigned)std::max<int64_t>(1, std::min(most, 2048 / std::max<int64_t>(T, 1)));
}

// Tokens that workgroups of their own start on; they step on by as many.
unsigned token_groups(int64_t T) { return (unsigned)std::min<int64_t>(T, 1 << 22); }

}  // namespace

// Three launches take 12.5 us and the rows' bytes, whatever the pairs are: one is as fast at 1000 tokens of 8 slots (12.2).
int sort_slices(int64_t T, int k) {
    const int64_t P = T * k;
    if (P <= kDirect && T * ((k + kKeys - 1) / kKeys) * P <= kDirectWork) return 0;
    return (int)std::min(kSlices, (P + kSlicePairs - 1) / kSlicePairs);
}

hipError_t launch_sort(const SortLaunch& a, hipStream_t s) {
    SortParams p{};
    p.x = (const uint8_t*)a.x;
    p.ids = a.ids;
    p.T = a.T;
    p.P = a.T * a.k;
    p.k = a.k;
    p.E = a.E;
    p.row = a.n * size_of(a.dtype);
    p.hist = a.hist;
    p.xs = (uint8_t*)a.xs;
    p.offsets = a.offsets;
    p.place = a.place;
    p.slices = sort_slices(a.T, a.k);
    const int64_t chunks = p.row / 16;
    if (p.slices == 0) {
        const int64_t groups = a.T * ((a.k + kKeys - 1) / kKeys);
        const dim3 grid((unsigned)(groups + (a.E + kKeys) / kKeys), row_parts(groups, chunks));
        hipLaunchKernelGGL(sort_direct_kernel, grid, dim3(kThreads), 0, s, p);
        return hipGetLastError();
    }
    p.slice = (p.P + p.slices - 1) / p.slices;
    const unsigned lds = (unsigned)(a.E + 1) * 4;
    hipLaunchKernelGGL(sort_count_kernel, dim3((unsigned)p.slices), dim3(kThreads), lds, s, p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(sort_place_kernel, dim3((unsigned)p.slices), dim3(kThreads), kWaves * lds, s, p);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(sort_copy_kernel, dim3(token_groups(a.T), row_parts(a.T, chunks)), dim3(kThreads), 0, s, p);
    return hipGetLastError();
}

hipError_t launch_unsort(const UnsortLaunch& a, hipStream_t s) {
    UnsortParams p{};
    p.ys = a.ys;
    p.place = a.place;
    p.w = a.weights;
    p.T = a.T;
    p.P = a.T * a.k;
    p.n = a.n;
    p.k = a.k;
    p.y = a.y;
    const dim3 grid(token_groups(a.T), (unsigned)((a.n + 8 * kThreads - 1) / (8 * kThreads)));
    by_float(a.ys_dtype, [&](auto st) {
        by_float(a.y_dtype, [&](auto yt) {
            constexpr int ST = decltype(st)::value, YT = decltype(yt)::value;
            if (p.n >= 8) hipLaunchKernelGGL((unsort_kernel<ST, YT, true>), grid, dim3(kThreads), 0, s, p);
            else hipLaunchKernelGGL((unsort_kernel<ST, YT, false>), grid, dim3(kThreads), 0, s, p);
        });
    });
    return hipGetLastError();
}

hipError_t launch_unsort_grad(const UnsortGradLaunch& a, hipStream_t s) {
    UnsortParams p{};
    p.ys = a.ys;
    p.place = a.place;
    p.w = a.weights;
    p.T = a.T;
    p.P = a.T * a.k;
    p.n = a.n;
    p.k = a.k;
    p.dy = a.dy;
    p.d_ys = a.d_ys;
    p.d_w = a.d_weights;
    by_float(a.ys_dtype, [&](auto st) {
        by_float(a.dy_dtype, [&](auto yt) {
            constexpr int ST = decltype(st)::value, YT = decltype(yt)::value;
            if (p.n >= 8) hipLaunchKernelGGL((unsort_grad_kernel<ST, YT, true>), dim3(token_groups(a.T)), dim3(kThreads), 0, s, p);
            else hipLaunchKernelGGL((unsort_grad_kernel<ST, YT, false>), dim3(token_groups(a.T)), dim3(kThreads), 0, s, p);
        });
    });
    return hipGetLastError();
}

}  // namespace iqk
