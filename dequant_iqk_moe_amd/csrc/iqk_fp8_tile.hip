// iqk_fp8_tile.hip -- the 8-bit product tile by tile.
//
// A workgroup owns TM rows of x by TN weight rows.  Each block of 128 of the
// depth goes from memory straight into LDS, S - 1 blocks ahead, as 128 bytes
// per row with their 16-byte chunks permuted (xkey, wkey) so that a fragment's
// reads meet no bank twice (no conflicts by the counters); the block's scales
// go along.  Every block's products start at zero and are added to the float32
// sums with the product of the two scales, so a matrix instruction's
// accumulator is never carried from one block to the next.
//
// EXACT (float32 and float16 results) widens the fragments to float16 in
// registers and uses v_mfma_f32_16x16x32_f16; otherwise one
// v_mfma_scale_f32_16x16x128_f8f6f4 (both scales 2^0) takes a whole block.
//
// Measured, with bfloat16 results: 8192 x 4096 x 4096 in 127 us = 2.16 PFLOP/s
// (137 us behind the quantization of activations with loud channels), matrix
// pipes busy 52 % of the launch's CU cycles by the counters, where the same
// instructions with the four multiply-adds each needs, and nothing else, run at
// 3.1 to 3.9 PFLOP/s.  A block of 256 x 256 tiles takes 3540 cycles of a CU for
// 2048 of its matrix pipes (58 %; the rest of the launch is its start and end):
// about 450 until a block's first fragments are there, 250 at its barrier, and
// two waves per SIMD that share its pipe at 40 cycles per instruction of 32.
// More stages do not fit its LDS, and smaller tiles, which would leave room for
// them, move more bytes per product (128 x 256 in three stages 166 us).  float32
// results: 300 us = 0.92 PFLOP/s; float16: 265.
//
// Few rows per expert: bytes of the weights.  The copies need no registers, so
// as many are in flight as the LDS holds, and each is whole 128-byte lines,
// where fragments loaded by their lanes ask for halves of 16 lines at a time
// (256 experts of 4096 x 2048, 12 rows each: 410 us = 5.3 TB/s of weights;
// with fragments loaded by their lanes 430 to 460).  What is left to the 6.4
// TB/s of a plain read is the start of each workgroup and the results' stores.
#include <algorithm>
#include <cmath>

#include "iqk_fp8_device.h"

namespace iqk {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

struct TileParams {
    const uint8_t* W;
    const float* sw;
    const uint8_t* x;
    const float* sx;
    int64_t M;
    int out, n, k, x_slots, E;
    int run;  // weight tiles a workgroup takes one after the other
    int parts;  // SPLIT: of the depth, part i into the i-th array of sums at y
    const int32_t *offsets, *perm, *tiles;  // grouped: tiles[e] = TM-row tiles of x before expert e
    void* y;
};

// What copies past the depth read.
__device__ const uint4 g_zero = {0, 0, 0, 0};

// Key of a tile's weight rows: a fragment's 16 lanes read rows 8 (l / 4) + l % 4
// + const, so bits 0, 1 and 3 of the row tell eight neighbouring lanes apart.
__device__ __forceinline__ int wkey(int r) { return (r & 3) | ((r >> 1) & 4); }

template <int TM, int TN, int WM, int WN, int S>
struct TileShape {
    static constexpr int kWaves = (TM / WM) * (TN / WN);
    static constexpr int kI = WN / 16, kJ = WM / 16;     // a wave's tiles of weight rows and of rows of x
    static constexpr int kG = 2;                         // tiles whose rows are dealt out four at a time
    static_assert(kI % kG == 0, "whole groups of tiles");
    static constexpr int kRowsPerCopy = 8 * kWaves;      // rows one copy instruction of all waves covers
    static constexpr int kCW = TN / kRowsPerCopy;
    static constexpr int kCX = (TM + kRowsPerCopy - 1) / kRowsPerCopy;
    static constexpr int kCopies = kCW + kCX + 1;        // memory instructions of a wave per block
    static constexpr int kX = TN * 128, kScales = kX + kCX * kRowsPerCopy * 128;  // offsets in a stage
    static constexpr int kStage = kScales + kWaves * 256;
    static_assert(TM + (TN + 127) / 128 <= 64 * kWaves, "one scale per lane");
    static_assert(S * kStage <= 160 * 1024, "LDS");
};

template <int TM, int TN, int WM, int WN, int S, int YT, bool GROUPED, bool EXACT, bool PART, bool SPLIT>
__global__ __launch_bounds__(64 * (TM / WM) * (TN / WN)) void fp8_tile_kernel(TileParams p) {
    using Sh = TileShape<TM, TN, WM, WN, S>;
    constexpr int kI = Sh::kI, kJ = Sh::kJ, kG = Sh::kG;
    __shared__ __align__(16) uint8_t sh[S * Sh::kStage];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int li = lane & 15, g = lane >> 4;
    const int nb = (p.n + kBlock - 1) / kBlock, nob = (p.out + kBlock - 1) / kBlock;
    const int ntn = (p.out + TN - 1) / TN, runs = (ntn + p.run - 1) / p.run;

    // the blocks of the depth this workgroup takes
    const int b0 = SPLIT ? (int)blockIdx.y * nb / p.parts : 0, b1 = SPLIT ? ((int)blockIdx.y + 1) * nb / p.parts : nb;

    // which tile of x and run of weight tiles: those of one XCD (workgroups b with equal b % 8) are neighbours
    int e = 0, n0;
    int64_t m0, count = p.M, begin = 0;
    {
        const int64_t tiles_m = GROUPED ? p.tiles[p.E] : (p.M + TM - 1) / TM;
        const int64_t total = tiles_m * runs, per = (total + 7) / 8;
        const int64_t id = (int64_t)(blockIdx.x & 7) * per + (blockIdx.x >> 3);
        if ((int64_t)(blockIdx.x >> 3) >= per || id >= total) return;
        if constexpr (GROUPED) {
            const int t = (int)(id / runs);
            n0 = (int)(id - (int64_t)t * runs) * p.run * TN;
            // the expert of tile t: the last e with tiles[e] <= t, 64 candidates at a time
            int lo = 0, span = p.E;
            while (span > 1) {
                const int step = (span + 63) / 64;
                const int c = lo + lane * step;
                const uint64_t le = __ballot(c < lo + span && p.tiles[min(c, p.E)] <= t);
                const int nlo = lo + (63 - __builtin_clzll(le)) * step;
                span = min(step, lo + span - nlo);
                lo = nlo;
            }
            e = __builtin_amdgcn_readfirstlane(lo);
            begin = p.offsets[e];
            count = p.offsets[e + 1] - begin;
            m0 = (int64_t)(t - p.tiles[e]) * TM;
        } else {
            // bands of 8 tiles of x by all of the weights' runs
            const int64_t band = id / (8 * runs), in = id - band * 8 * runs;
            const int64_t rows = min((int64_t)8, tiles_m - band * 8);
            m0 = (band * 8 + in % rows) * TM;
            n0 = (int)(in / rows) * p.run * TN;
        }
    }

    // row i of the tile's rows of x, as a row of p.x; rows past the last
    // repeat it, their results are dropped
    auto pair_of = [&](int i) { return p.perm[begin + min(m0 + i, count - 1)]; };
    auto row_of = [&](int i) -> int64_t {
        if constexpr (GROUPED) return p.x_slots == 1 ? pair_of(i) / p.k : pair_of(i);
        else return min(m0 + i, count - 1);
    };

    // copies: lane l of a copy moves slot l & 7 of row l >> 3 of its wave's eight rows
    const int crow = wave * 8 + (lane >> 3);
    static_assert(Sh::kRowsPerCopy % 32 == 0, "a lane's chunk is the same in all of its copies");
    const int wch = 16 * ((lane & 7) ^ wkey(crow)), xch = 16 * ((lane & 7) ^ xkey(crow));
    const uint8_t* xbase = GROUPED ? p.x : p.x + m0 * p.n;  // (dense: offsets inside the tile fit 32 bits)
    uint32_t woff[Sh::kCW], xoff[Sh::kCX];                  // (grouped: xoff is the row of x, multiplied out at each copy)
#pragma unroll
    for (int c = 0; c < Sh::kCX; ++c) {
        const int64_t row = row_of(min(c * Sh::kRowsPerCopy + crow, TM - 1));
        xoff[c] = GROUPED ? (uint32_t)row : (uint32_t)((int)(row - m0) * p.n + xch);
    }
    auto xsrc = [&](int c, int k0) {
        if constexpr (GROUPED) return xbase + ((uint64_t)xoff[c] * (uint32_t)p.n + (uint32_t)(k0 + xch));
        else return xbase + k0 + xoff[c];
    };
    // scales: of row u of x in lane u < TM of the workgroup, then of the tile's blocks of 128 weight rows
    const int su = wave * 64 + lane;
    const float* sptr = p.sx + row_of(min(su, TM - 1)) * nb;
    // the next block to copy: block cb of the weight tile at row cn
    const int nend = min(n0 + p.run * TN, p.out);
    int cb = b0, cn = n0;
    const uint8_t* wbase;
    auto weight_tile = [&]() {
        wbase = p.W + ((int64_t)e * p.out + cn) * p.n;
#pragma unroll
        for (int c = 0; c < Sh::kCW; ++c)
            woff[c] = (uint32_t)(min(c * Sh::kRowsPerCopy + crow, p.out - 1 - cn) * p.n + wch);
        if (su >= TM)
            sptr = p.sw + ((int64_t)e * nob + min(cn / kBlock + min(su - TM, (TN + 127) / 128 - 1), nob - 1)) * nb;
    };
    weight_tile();
    const uint32_t sh0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)sh;
    // Copy c of the kCopies that bring the next block into a stage: weight rows, rows of x, scales.  PART: the depth's
    // last block is partial, and chunks past the depth are zero.  (Once the last block is on its way the last tile's
    // first one is copied again, which nothing reads: every step takes as many instructions, and the waits count them.)
    auto copy = [&](int c, int slot) {
        const int k0 = cb * kBlock;
        const uint32_t at = sh0 + slot * Sh::kStage + wave * 1024;
        if (c < Sh::kCW) {
            const uint32_t d = at + c * Sh::kRowsPerCopy * 128;
            if constexpr (PART) lds_copy16(k0 + wch < p.n ? wbase + k0 + woff[c] : (const uint8_t*)&g_zero, d);
            else lds_copy16(wbase + k0, woff[c], d);
        } else if (c < Sh::kCW + Sh::kCX) {
            const int i = c - Sh::kCW;
            const uint32_t d = at + Sh::kX + i * Sh::kRowsPerCopy * 128;
            if constexpr (PART) lds_copy16(k0 + xch < p.n ? xsrc(i, k0) : (const uint8_t*)&g_zero, d);
            else if constexpr (GROUPED) lds_copy16(xsrc(i, k0), d);
            else lds_copy16(xbase + k0, xoff[i], d);
        } else {
            lds_copy4(sptr + cb, sh0 + slot * Sh::kStage + Sh::kScales + wave * 256);
        }
    };
    auto advance = [&]() {
        if (++cb < b1) return;
        cb = b0;
        if (cn + TN < nend) {
            cn += TN;
            weight_tile();
        }
    };
    // A wave that has copies to issue waits until the memory pipeline takes them, which is slower than it issues them
    // (all at the head of a block: half of the waves 2800 cycles of a block's 4800), so they go out between the
    // tile rows' products: kPer at each of the first rows.  Waves of one or two tile rows have too few products to
    // put between them and issue them first (64 x 64 tiles, 4096 deep: 13.7 us that way, 14.7 the other).
    constexpr bool kFirst = kI <= 2;
    constexpr int kPer = (4 * Sh::kCopies + 3 * kI - 1) / (3 * kI);

    const int wn = (wave % (TN / WN)) * WN, wm = (wave / (TN / WN)) * WM;  // this wave's part of the tile
    const bool busy = m0 + wm < count;                                     // whether any of its rows of x is there
    f32x4 acc[kI][kJ];
#pragma unroll
    for (int i = 0; i < kI; ++i)
#pragma unroll
        for (int j = 0; j < kJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    // lane li of tile i reads weight row 32 (i / 2) + 8 (li / 4) + 4 (i % 2) + li % 4, so that a result lane's four
    // rows of two neighbouring tiles are eight consecutive rows, and the four lanes of a row of x store 32 at a time
    // (whole 64-byte pieces of 16-bit results)
    const int afirst = 4 * kG * (li >> 2) + (li & 3);
    const int aoff = (wn + afirst) * 128 + 16 * (g ^ wkey(afirst));
    const int boff = Sh::kX + (wm + li) * 128 + 16 * (g ^ xkey(li));
    const int soff = Sh::kScales + 4 * (wm + li), swoff = Sh::kScales + 4 * (TM + wn / kBlock);
    auto frag = [&](const uint8_t* s, int off) {
        const uint4 a = *(const uint4*)(s + off), b = *(const uint4*)(s + (off ^ 64));
        return i32x8{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
    };

    // result lane (li, g) holds, of row 16 j + li of x, weight rows 32 h + 8 g + 4 i + q of its wave's
    auto store_tile = [&]() {
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
            const int i = wm + 16 * j + li;
            if (m0 + i >= count) continue;
            int64_t yrow = m0 + i;
            if constexpr (SPLIT) yrow += blockIdx.y * p.M;
            if constexpr (GROUPED) yrow = pair_of(i);
#pragma unroll
            for (int h = 0; h < kI / kG; ++h) {
                const int o = n0 + wn + 32 * h + 8 * g;
                if (o >= p.out) continue;
                float v[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    v[q] = acc[2 * h + (q >> 2)][j][q & 3];
                    // (the tile's last products are added right before: fused with the conversion to f16 they would
                    // round once, where the others round twice, and a row's bits would depend on its place)
                    if constexpr (YT == IQK_F16) asm("" : "+v"(v[q]));
                }
                store8<YT>(p.y, yrow * p.out + o, v, p.out - o);
            }
        }
    };

    // Instruction t = i kJ + j of a block multiplies tile row i by x tile j.  Its product is added to the sums two
    // instructions later (kLag: it is done by then), and a tile row is read kAhead rows before its first use.
    constexpr int kAhead = kI < 4 ? 1 : ((GROUPED || PART) && TM * TN > 128 * 128 ? 1 : 2);  // (two would spill there)
    constexpr int kLag = 2, kT = kI * kJ, kRing = kT < 4 ? kT : 4;
    static_assert(EXACT || kT % kRing == 0, "a block's first products follow the last block's in the ring");
    float f[kJ], fp[kJ];
    f32x4 d[kRing];
#pragma unroll
    for (int j = 0; j < kJ; ++j) fp[j] = 0.f;
#pragma unroll
    for (int t = 0; t < kRing; ++t) d[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto add = [&](int t, const float* w) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
            acc[t / kJ][t % kJ][q] = __builtin_fmaf(d[t % kRing][q], w[t % kJ], acc[t / kJ][t % kJ][q]);
    };

    constexpr int kBehind = (S - 2) * Sh::kCopies;  // copies that may still be on their way when a block is published
    const int steps = (b1 - b0) * ((nend - n0 + TN - 1) / TN);
#pragma unroll
    for (int b = 0; b < S - 1; ++b) {
#pragma unroll
        for (int c = 0; c < Sh::kCopies; ++c) copy(c, b);
        advance();
    }
    publish<kBehind>();
    int slot = 0, b = 0;  // b: block of the tile that is being multiplied
    for (int step = 0; step < steps; ++step) {
        const uint8_t* cur = sh + slot * Sh::kStage;
        const int into = slot == 0 ? S - 1 : slot - 1;
        auto copy_some = [&](int i) {
#pragma unroll
            for (int c = i * kPer; c < (i + 1) * kPer; ++c)
                if (!kFirst && c < Sh::kCopies) copy(c, into);
        };
        if (kFirst || !busy) {
#pragma unroll
            for (int c = 0; c < Sh::kCopies; ++c) copy(c, into);
        }
        if (busy) {
            // (pairs of tiles are 32 rows apart, a pair's tiles four rows, which no bit of the key looks at)
            auto afrag = [&](int i) { return frag(cur, aoff + (i >> 1) * 4096 + (i & 1) * 512); };
            i32x8 af[kAhead + 1], bf[kJ];
            af[0] = afrag(0);
            bf[0] = frag(cur, boff);
            const float fw = *(const float*)(cur + swoff);
#pragma unroll
            for (int j = 0; j < kJ; ++j) f[j] = *(const float*)(cur + soff + 64 * j);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int j = 1; j < kJ; ++j) {
                bf[j] = frag(cur, boff + j * 2048);
                __builtin_amdgcn_sched_barrier(0);
            }
            if constexpr (kAhead > 1) af[1] = afrag(1);
#pragma unroll
            for (int j = 0; j < kJ; ++j) f[j] *= fw;
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (EXACT) {
                f16x8 xw[kJ][4];
#pragma unroll
                for (int j = 0; j < kJ; ++j)
#pragma unroll
                    for (int h = 0; h < 4; ++h) xw[j][h] = widen(bf[j][2 * h], bf[j][2 * h + 1]);
#pragma unroll
                for (int i = 0; i < kI; ++i) {
                    if (i + kAhead < kI) af[(i + kAhead) % (kAhead + 1)] = afrag(i + kAhead);
                    copy_some(i);
                    f16x8 ww[4];
#pragma unroll
                    for (int h = 0; h < 4; ++h) ww[h] = widen(af[i % (kAhead + 1)][2 * h], af[i % (kAhead + 1)][2 * h + 1]);
                    f32x4 r[kJ];
#pragma unroll
                    for (int j = 0; j < kJ; ++j) r[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int h = 0; h < 4; ++h)
#pragma unroll
                        for (int j = 0; j < kJ; ++j) r[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ww[h], xw[j][h], r[j], 0, 0, 0);
#pragma unroll
                    for (int j = 0; j < kJ; ++j)
#pragma unroll
                        for (int q = 0; q < 4; ++q) acc[i][j][q] = __builtin_fmaf(r[j][q], f[j], acc[i][j][q]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < kI; ++i) {
                    if (i + kAhead < kI) af[(i + kAhead) % (kAhead + 1)] = afrag(i + kAhead);
#pragma unroll
                    for (int j = 0; j < kJ; ++j) {
                        const int t = i * kJ + j;
                        const f32x4 r = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                            af[i % (kAhead + 1)], bf[j], f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0x7F7F7F7F, 0, 0x7F7F7F7F);
                        __builtin_amdgcn_sched_barrier(0);
                        if (j == 0) copy_some(i);
                        if (t >= kLag) add(t - kLag, f);
                        else add(kT - kLag + t, fp);
                        d[t % kRing] = r;
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
#pragma unroll
                for (int j = 0; j < kJ; ++j) fp[j] = f[j];
            }
        }
        advance();
        publish<kBehind>();
        slot = slot == S - 1 ? 0 : slot + 1;
        if (++b == b1 - b0) {  // (after the wait, so that the stores are on their way while the next block is multiplied)
            if constexpr (!EXACT) {
#pragma unroll
                for (int t = kT - kLag; t < kT; ++t) add(t, fp);
#pragma unroll
                for (int t = 0; t < kRing; ++t) d[t] = f32x4{0.f, 0.f, 0.f, 0.f};
                // (the next tile's first sums add 0 * fp, which is not zero where a scale of this tile is infinite)
#pragma unroll
                for (int j = 0; j < kJ; ++j) fp[j] = 0.f;
            }
            store_tile();
#pragma unroll
            for (int i = 0; i < kI; ++i)
#pragma unroll
                for (int j = 0; j < kJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
            b = 0;
            n0 += TN;
        }
    }
    // no copy may land in the LDS of the workgroup that gets it next
    __builtin_amdgcn_s_waitcnt(0x0070);
}

constexpr int64_t kMaxRun = 2;

// Joins the parts' sums in their order: the same result every time.
constexpr int kJoinThreads = 256;
template <int YT>
__global__ __launch_bounds__(kJoinThreads) void fp8_join_kernel(const float* sums, int parts, int64_t count, void* y) {
    const int64_t i = (int64_t)blockIdx.x * kJoinThreads + threadIdx.x;
    if (i >= count) return;
    float v = sums[i];
    for (int part = 1; part < parts; ++part) v += sums[part * count + i];
    store_y<YT>(y, i, v);
}

template <int YT>
hipError_t split_launch(const Fp8Launch& a, int parts, hipStream_t s) {
    using Sh = TileShape<64, 64, 16, 32, 4>;
    constexpr bool EXACT = exact_sums(YT);
    const TileParams p{a.codes, a.scales, (const uint8_t*)a.x, a.x_scales, a.M, (int)a.out, (int)a.n, a.k, a.x_slots,
                       (int)a.E, 1, parts, nullptr, nullptr, nullptr, a.sums};
    const int64_t tiles = (a.M + 63) / 64 * ((a.out + 63) / 64), count = a.M * a.out;
    const dim3 grid((unsigned)((tiles + 7) / 8 * 8), (unsigned)parts), block(64 * Sh::kWaves);
    if (a.n % kBlock)
        hipLaunchKernelGGL((fp8_tile_kernel<64, 64, 16, 32, 4, IQK_F32, false, EXACT, true, true>), grid, block, 0, s, p);
    else
        hipLaunchKernelGGL((fp8_tile_kernel<64, 64, 16, 32, 4, IQK_F32, false, EXACT, false, true>), grid, block, 0, s, p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((fp8_join_kernel<YT>), dim3((unsigned)((count + kJoinThreads - 1) / kJoinThreads)),
                       dim3(kJoinThreads), 0, s, a.sums, parts, count, a.y);
    return hipGetLastError();
}

// TM x TN tiles by waves of WM x WN, S stages
template <int TM, int TN, int WM, int WN, int S, bool EXACT, int YT, bool GROUPED>
hipError_t tile_launch(const Fp8Launch& a, hipStream_t s) {
    using Sh = TileShape<TM, TN, WM, WN, S>;
    const int64_t ntn = (a.out + TN - 1) / TN;
    const int64_t tiles = (a.M + TM - 1) / TM + (GROUPED ? std::min<int64_t>(a.E, a.M) : 0);  // (partial last tiles)
    // A workgroup's first blocks arrive a memory latency after it starts and its results leave while nothing else
    // of it runs, so it takes two weight tiles in a run where the runs fill the card as evenly as tiles do (8192 x
    // 4096 x 4096: 133 us against 139; 256 experts of 4096 x 2048 with 12 rows each: 425 against 442; four and eight
    // were no faster: their last turn is emptier).  Large groups differ too much in size for that: 350 against 337.
    constexpr int64_t kResident = 256 * std::min(2, 160 * 1024 / (S * Sh::kStage));
    auto turns = [&](int64_t run) { return (tiles * ((ntn + run - 1) / run) + kResident - 1) / kResident * run; };
    int64_t run = 1;
    while ((TM <= 64 || !GROUPED) && run < kMaxRun && 2 * run <= ntn && turns(2 * run) * 16 <= turns(1) * 17) run *= 2;
    const TileParams p{a.codes, a.scales, (const uint8_t*)a.x, a.x_scales, a.M, (int)a.out, (int)a.n, a.k, a.x_slots,
                       (int)a.E, (int)run, 1, a.offsets, a.perm, a.tiles, a.y};
    const int64_t total = tiles * ((ntn + run - 1) / run);
    if (total >= (int64_t)(UINT32_MAX / (64 * Sh::kWaves))) return hipErrorInvalidConfiguration;
    const dim3 grid((unsigned)((total + 7) / 8 * 8)), block(64 * Sh::kWaves);
    if (a.n % kBlock) hipLaunchKernelGGL((fp8_tile_kernel<TM, TN, WM, WN, S, YT, GROUPED, EXACT, true, false>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((fp8_tile_kernel<TM, TN, WM, WN, S, YT, GROUPED, EXACT, false, false>), grid, block, 0, s, p);
    return hipGetLastError();
}

template <int YT>
hipError_t grouped_launch(const Fp8Launch& a, const Fp8Tile& t, hipStream_t s) {
    constexpr bool EXACT = exact_sums(YT);
    // few rows per expert: the weights stream through, exact sums cost nothing there
    if (t.rows == 16) return tile_launch<16, 128, 16, 32, 4, true, YT, true>(a, s);
    if (t.rows == 32) return tile_launch<32, 128, 32, 32, 3, true, YT, true>(a, s);
    if (t.rows == 64) return tile_launch<64, 128, 32, 64, 2, true, YT, true>(a, s);
    if constexpr (!EXACT) {
        if (t.rows == 256) return tile_launch<256, 256, 64, 128, 2, false, YT, true>(a, s);
    }
    if (t.cols == 128) return tile_launch<128, 128, 64, 64, 2, EXACT, YT, true>(a, s);
    return tile_launch<128, 256, 64, 64, 3, EXACT, YT, true>(a, s);
}

template <int YT>
hipError_t dense_launch(const Fp8Launch& a, const Fp8Tile& t, hipStream_t s) {
    constexpr bool EXACT = exact_sums(YT);
    if (t.parts > 1) return split_launch<YT>(a, t.parts, s);
    if (t.rows == 64) return tile_launch<64, 64, 16, 32, 4, EXACT, YT, false>(a, s);
    if constexpr (!EXACT) {
        if (t.rows == 256) return tile_launch<256, 256, 64, 128, 2, false, YT, false>(a, s);
    }
    return tile_launch<128, 128, 64, 64, 2, EXACT, YT, false>(a, s);
}

// Rows of x in a tile of the grouped product.
int grouped_rows(int64_t M, int64_t E, int64_t out, bool exact) {
    auto count = [&](int64_t t) { return (M + t - 1) / t * ((out + t - 1) / t); };
    const double rows_per_expert = (double)M / (double)E;
    // A block of a small tile takes its time however few there are, less the smaller it is: where workgroups of 16
    // or of 32 rows about have a CU each, they are taken (8 experts of 1024 x 4096, 37 rows each: tiles of 16, 32
    // and 64 rows 24, 28 and 37 us; 16 of 1024 x 2048, 50 rows each: 32 rows 23, 64 rows 27, 128 rows 32).
    const double experts = std::min((double)M, (double)M / rows_per_expert);
    auto groups = [&](int64_t t) { return ((double)(M / t) + experts / 2) * (double)((out + 127) / 128); };
    if (groups(16) <= 192) return 16;
    if (groups(32) <= 288) return 32;
    // Else the rows a tile holds are what most experts have (their counts spread like a square root; 64 experts of
    // 4096 x 2048, 24 rows each: tiles of 32 rows 127 us, of 64 rows 145; 128 of 2048 x 2048, 26 rows: the same).
    const double spread = std::sqrt(rows_per_expert);
    if (rows_per_expert + 2 * spread <= 16) return 16;
    if (rows_per_expert + spread <= 32) return 32;
    if (rows_per_expert + 2 * spread <= 64) return 64;
    // 64 experts of 2048 x 4096, 384 rows each: 256-row tiles 333 us, 128-row ones 380; 96 rows each: 294 and 271
    return !exact && rows_per_expert >= 192 && count(256) >= 160 ? 256 : 128;
}

// Side of a tile of the dense product.  256 x 256 tiles move half the bytes per product that 128 x 128 ones do, and
// those half of what 64 x 64 do; the largest is taken that gives most of the 256 CUs a tile.
int dense_side(int64_t M, int64_t out, bool exact) {
    auto count = [&](int64_t t) { return (M + t - 1) / t * ((out + t - 1) / t); };
    if (!exact && count(256) >= 160) return 256;
    return count(128) >= 160 ? 128 : 64;
}

// Parts of the depth of the dense product that workgroups of their own take.
// A block of 64 x 64 tiles takes about 0.4 us however few tiles there are, so a long depth is split while each part
// of each tile has a CU to itself (with two parts per CU 2017 x 117 x 5136 takes 25 us instead of 23) and four blocks,
// where that saves more than 10 us: the launch that joins the sums costs about 3 us of the card and as much of the
// host.  141 x 261 x 7920, float32: 19.5 us against 43; 308 x 1099 x 6880: 25 against 32; 64 x 4096 x 4096, not split:
// 17 against 20.
int depth_parts(int64_t M, int64_t out, int64_t n) {
    if (dense_side(M, out, true) != 64) return 1;  // (the same whatever y's type: where it is 64, it is for all)
    const int64_t tiles = (M + 63) / 64 * ((out + 63) / 64), nb = (n + kBlock - 1) / kBlock;
    const int64_t parts = std::min<int64_t>({256 / tiles, nb / 4, 16});
    return parts > 1 && 0.4 * (double)(nb - (nb + parts - 1) / parts) > 10.0 ? (int)parts : 1;
}

}  // namespace

Fp8Tile fp8_grouped_tile(int64_t M, int64_t E, int64_t out, bool exact) {
    const int tm = grouped_rows(M, E, out, exact);
    if (tm < 128) return Fp8Tile{tm, 128, 1};
    if (tm == 256) return Fp8Tile{256, 256, 1};
    // A CU holds one workgroup of 128 x 256 tiles or two of 128 x 128 ones, which take as long together.  The
    // small ones are taken where each has a CU to itself, or where they fit at once and the others do not (16
    // experts of 310 x 2960, 1000 rows each: 62 us against 81; float32 results of 312 x 1456, 433 rows: 34
    // against 42; else 171 against 165 for 64 experts of 2048 x 4096, 96 rows each).
    const int64_t rows = M / 128 + std::min(E, M) / 2;
    const int64_t small = rows * ((out + 127) / 128), large = rows * ((out + 255) / 256);
    return Fp8Tile{128, small <= 256 || (large > 256 && small <= 512) ? 128 : 256, 1};
}

Fp8Tile fp8_dense_tile(int64_t M, int64_t out, int64_t n, bool exact) {
    const int side = dense_side(M, out, exact);
    return Fp8Tile{side, side, depth_parts(M, out, n)};
}

size_t fp8_sums_bytes(int64_t M, int64_t out, int64_t n) {
    const int parts = depth_parts(M, out, n);
    return parts > 1 ? (size_t)(parts * M * out) * 4 : 0;
}

hipError_t launch_fp8_tile(const Fp8Launch& a, const Fp8Tile& tile, hipStream_t s) {
    hipError_t e = hipSuccess;
    by_float(a.y_dtype, [&](auto yt) {
        constexpr int YT = decltype(yt)::value;
        e = a.offsets ? grouped_launch<YT>(a, tile, s) : dense_launch<YT>(a, tile, s);
    });
    return e;
}

}  // namespace iqk
