// iqk_int8_tile.hip -- the 8-bit integer product tile by tile, dense or over rows
// sorted by expert.
//
// A workgroup owns TM rows of x by TN weight rows.  Each block of 128 of the depth
// goes from memory straight into LDS, S - 1 blocks ahead, as 128 bytes per row with
// their 16-byte chunks permuted (xkey, wkey) so that a fragment's reads meet no bank
// twice.  The sums are int32 and exact, so they stay in the matrix instructions'
// accumulators over the whole depth, and the scales are applied once at the end.
#include <algorithm>
#include <cmath>

#include "iqk_block.h"
#include "iqk_fp8_device.h"

namespace iqk {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

struct TileParams {
    const uint8_t* W;
    const float* sw;
    const uint8_t* x;
    const float* sx;
    int64_t M;
    int out, n, E;
    int run;  // weight tiles a workgroup takes one after the other
    const int32_t *offsets, *tiles;
    void* y;
};

// What copies past the depth read.
__device__ const uint4 g_zero = {0, 0, 0, 0};

// Key of a tile's weight rows: eight neighbouring lanes of a fragment read rows that
// differ in bits 0, 1 and 3.
__device__ __forceinline__ int wkey(int r) { return (r & 3) | ((r >> 1) & 4); }

// Matrix instructions of side MF (32: depth 32, 16: depth 64) and their accumulators.
template <int MF>
struct Mfma;
template <>
struct Mfma<32> {
    using Acc = i32x16;
    static constexpr int kDepth = 32;
    static __device__ __forceinline__ Acc run(i32x4 a, i32x4 b, Acc c) { return __builtin_amdgcn_mfma_i32_32x32x32_i8(a, b, c, 0, 0, 0); }
};
template <>
struct Mfma<16> {
    using Acc = i32x4;
    static constexpr int kDepth = 64;
    static __device__ __forceinline__ Acc run(i32x4 a, i32x4 b, Acc c) { return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0); }
};

template <int TM, int TN, int WM, int WN, int S, int MF>
struct TileShape {
    static constexpr int kWaves = (TM / WM) * (TN / WN);
    static constexpr int kI = WN / MF, kJ = WM / MF;  // a wave's tiles of weight rows and of rows of x
    static_assert(MF == 32 || kI % 2 == 0, "tiles of 16 weight rows come in pairs");
    static constexpr int kSteps = kBlock / Mfma<MF>::kDepth;  // instructions' depths in a block
    static constexpr int kRowsPerCopy = 8 * kWaves;           // rows one copy instruction of all waves covers
    static constexpr int kCW = TN / kRowsPerCopy;
    static constexpr int kCX = (TM + kRowsPerCopy - 1) / kRowsPerCopy;
    static constexpr int kCopies = kCW + kCX;  // memory instructions of a wave per block
    static constexpr int kX = TN * 128;        // offset of x's rows in a stage
    static constexpr int kStage = kX + kCX * kRowsPerCopy * 128;
    static_assert(S * kStage <= 160 * 1024, "LDS");
};

template <int TM, int TN, int WM, int WN, int S, int MF, int YT, bool GROUPED, bool PART>
__global__ __launch_bounds__(64 * (TM / WM) * (TN / WN)) void int8_tile_kernel(TileParams p) {
    using Sh = TileShape<TM, TN, WM, WN, S, MF>;
    using Mf = Mfma<MF>;
    constexpr int kI = Sh::kI, kJ = Sh::kJ, kSteps = Sh::kSteps;
    __shared__ __align__(16) uint8_t sh[S * Sh::kStage];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int nb = (p.n + kBlock - 1) / kBlock;
    const int ntn = (p.out + TN - 1) / TN, runs = (ntn + p.run - 1) / p.run;

    // which tile of x and run of weight tiles: those of one XCD (workgroups b with equal b % 8) are neighbours
    int e = 0, n0;
    int64_t m0, count = p.M, begin = 0;
    {
        const int64_t tiles_m = GROUPED ? p.tiles[p.E + 1] : (p.M + TM - 1) / TM;
        const int64_t total = tiles_m * runs, per = (total + 7) / 8;
        const int64_t id = (int64_t)(blockIdx.x & 7) * per + (blockIdx.x >> 3);
        if ((int64_t)(blockIdx.x >> 3) >= per || id >= total) return;
        if constexpr (GROUPED) {
            const int t = (int)(id / runs);
            n0 = (int)(id - (int64_t)t * runs) * p.run * TN;
            // the expert of tile t (E: rows of none): the last e with tiles[e] <= t, 64 candidates at a time
            int lo = 0, span = p.E + 1;
            while (span > 1) {
                const int step = (span + 63) / 64;
                const int c = lo + lane * step;
                const uint64_t le = __ballot(c < lo + span && p.tiles[min(c, p.E + 1)] <= t);
                const int nlo = lo + (63 - __builtin_clzll(le)) * step;
                span = min(step, lo + span - nlo);
                lo = nlo;
            }
            e = __builtin_amdgcn_readfirstlane(lo);
            auto at = [&](int i) { return i == 0 ? 0 : (int64_t)min(max((int64_t)p.offsets[i], (int64_t)0), p.M); };
            begin = at(e);
            count = (e < p.E ? at(e + 1) : p.M) - begin;
            m0 = (int64_t)(t - p.tiles[e]) * TM;
        } else {
            // bands of 8 tiles of x by all of the weights' runs
            const int64_t band = id / (8 * runs), in = id - band * 8 * runs;
            const int64_t rows = min((int64_t)8, tiles_m - band * 8);
            m0 = (band * 8 + in % rows) * TM;
            n0 = (int)(in / rows) * p.run * TN;
        }
    }
    const int nend = min(n0 + p.run * TN, p.out);
    const int rows = (int)min((int64_t)TM, count - m0);  // of x that are there
    if constexpr (GROUPED) {
        if (e == p.E) {
            for (int i = wave; i < rows; i += Sh::kWaves)
                for (int o = n0 + lane; o < nend; o += 64) store_y<YT>(p.y, (begin + m0 + i) * p.out + o, 0.f);
            return;
        }
    }

    // copies: lane l of a copy moves slot l & 7 of row l >> 3 of its wave's eight rows; rows past the last repeat
    // it, their results are dropped
    const int crow = wave * 8 + (lane >> 3);
    static_assert(Sh::kRowsPerCopy % 16 == 0, "a lane's chunk is the same in all of its copies");
    const int wch = 16 * ((lane & 7) ^ wkey(crow)), xch = 16 * ((lane & 7) ^ xkey(crow));
    const uint8_t* xbase = p.x + (begin + m0) * p.n;
    uint32_t woff[Sh::kCW], xoff[Sh::kCX];
#pragma unroll
    for (int c = 0; c < Sh::kCX; ++c) xoff[c] = (uint32_t)(min(c * Sh::kRowsPerCopy + crow, rows - 1) * p.n + xch);
    // the next block to copy: block cb of the weight tile at row cn
    int cb = 0, cn = n0;
    const uint8_t* wbase;
    auto weight_tile = [&]() {
        wbase = p.W + ((int64_t)e * p.out + cn) * p.n;
#pragma unroll
        for (int c = 0; c < Sh::kCW; ++c) woff[c] = (uint32_t)(min(c * Sh::kRowsPerCopy + crow, p.out - 1 - cn) * p.n + wch);
    };
    weight_tile();
    const uint32_t sh0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)sh;
    // Copy c of the kCopies that bring the next block into a stage: weight rows, rows of x.  PART: the depth's last
    // block is partial, and chunks past the depth are zero.  (Once the last block is on its way the last tile's first
    // one is copied again, which nothing reads: every step takes as many instructions, and the waits count them.)
    auto copy = [&](int c, int slot) {
        const int k0 = cb * kBlock;
        const uint32_t at = sh0 + slot * Sh::kStage + wave * 1024;
        if (c < Sh::kCW) {
            const uint32_t d = at + c * Sh::kRowsPerCopy * 128;
            if constexpr (PART) lds_copy16(k0 + wch < p.n ? wbase + k0 + woff[c] : (const uint8_t*)&g_zero, d);
            else lds_copy16(wbase + k0, woff[c], d);
        } else {
            const int i = c - Sh::kCW;
            const uint32_t d = at + Sh::kX + i * Sh::kRowsPerCopy * 128;
            if constexpr (PART) lds_copy16(k0 + xch < p.n ? xbase + k0 + xoff[i] : (const uint8_t*)&g_zero, d);
            else lds_copy16(xbase + k0, xoff[i], d);
        }
    };
    auto advance = [&]() {
        if (++cb < nb) return;
        cb = 0;
        if (cn + TN < nend) {
            cn += TN;
            weight_tile();
        }
    };

    const int wn = (wave % (TN / WN)) * WN, wm = (wave / (TN / WN)) * WM;  // this wave's part of the tile
    const bool busy = wm < rows;                                           // whether any of its rows of x is there
    typename Mf::Acc acc[kI][kJ];
    auto clear = [&]() {
#pragma unroll
        for (int i = 0; i < kI; ++i)
#pragma unroll
            for (int j = 0; j < kJ; ++j) acc[i][j] = typename Mf::Acc{};
    };
    clear();

    // Weight rows are dealt to a fragment's lanes so that a result lane's values are eight consecutive outputs: of a
    // 32-row tile, lane l reads row 16 (l / 16) + 8 (l / 4 % 2) + 4 (l / 8 % 2) + l % 4; of a pair of 16-row tiles,
    // row 8 (l / 4) + l % 4, and 4 more in the second.
    const int l = lane & (MF - 1), g = lane / MF;
    const int afirst = MF == 32 ? 16 * (l >> 4) + 8 * ((l >> 2) & 1) + 4 * ((l >> 3) & 1) + (l & 3) : 8 * (l >> 2) + (l & 3);
    const int aoff = (wn + afirst) * 128 + 16 * (g ^ wkey(afirst));
    const int boff = Sh::kX + (wm + l) * 128 + 16 * (g ^ xkey(l));
    // fragments of weight tile i and x tile j at depth step k of the stage at s
    auto afrag = [&](const uint8_t* s, int i, int k) {
        const int tile = MF == 32 ? i * 4096 : (i >> 1) * 4096 + (i & 1) * 512;
        return *(const i32x4*)(s + (aoff ^ (k * Mf::kDepth)) + tile);
    };
    auto bfrag = [&](const uint8_t* s, int j, int k) { return *(const i32x4*)(s + (boff ^ (k * Mf::kDepth)) + j * MF * 128); };

    // the results of the weight tile at row n0
    auto store_tile = [&]() {
        float sx[kJ];
#pragma unroll
        for (int j = 0; j < kJ; ++j) sx[j] = p.sx[begin + m0 + min(wm + MF * j + l, rows - 1)];
        constexpr int kPieces = MF == 32 ? kI * 2 : kI / 2;
#pragma unroll
        for (int h = 0; h < kPieces; ++h) {
            const int o = n0 + wn + (MF == 32 ? 16 * h : 32 * h) + 8 * g;
            float sw[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) sw[q] = p.sw[(int64_t)e * p.out + min(o + q, p.out - 1)];
#pragma unroll
            for (int j = 0; j < kJ; ++j) {
                const int i = wm + MF * j + l;
                float v[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const int a = MF == 32 ? acc[h >> 1][j][8 * (h & 1) + q] : acc[2 * h + (q >> 2)][j][q & 3];
                    v[q] = (float)a * (sx[j] * sw[q]);
                    // (fused with the conversion to f16 the product would round once, where the definition's rounds twice)
                    if constexpr (YT == IQK_F16) asm("" : "+v"(v[q]));
                }
                if (i < rows && o < p.out) store8<YT>(p.y, (begin + m0 + i) * p.out + o, v, p.out - o);
            }
        }
    };

    constexpr int kBehind = (S - 2) * Sh::kCopies;  // copies that may still be on their way when a block is published
    const int steps = nb * ((nend - n0 + TN - 1) / TN);
#pragma unroll
    for (int b = 0; b < S - 1; ++b) {
#pragma unroll
        for (int c = 0; c < Sh::kCopies; ++c) copy(c, b);
        advance();
    }
    publish<kBehind>();
    // Fragments of a depth step are read while the step before it is multiplied; the block's last step is multiplied
    // behind the barrier that publishes the next block, with that block's first fragments read beside it.
    i32x4 af[2][kI], bf[2][kJ];
#pragma unroll
    for (int i = 0; i < kI; ++i) af[0][i] = afrag(sh, i, 0);
#pragma unroll
    for (int j = 0; j < kJ; ++j) bf[0][j] = bfrag(sh, j, 0);
    static_assert(kSteps % 2 == 0, "a block ends on the fragments it began with");
    constexpr int kT = kI * kJ, kReads = kI + kJ;
    int slot = 0, b = 0;  // b: block of the tile that is being multiplied
    for (int step = 0; step < steps; ++step) {
        const uint8_t* cur = sh + slot * Sh::kStage;
        const int into = slot == 0 ? S - 1 : slot - 1;
        slot = slot == S - 1 ? 0 : slot + 1;
        const uint8_t* next = sh + slot * Sh::kStage;
        constexpr int kSlots = (kSteps - 1) * kT;  // products before the block's last depth step
        constexpr int kPer = (Sh::kCopies + kSlots - 1) / kSlots;
        if (!busy) {
#pragma unroll
            for (int c = 0; c < Sh::kCopies; ++c) copy(c, into);
            advance();
            publish<kBehind>();
        } else {
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
                const bool last = k == kSteps - 1;
                if (last) {
                    advance();
                    publish<kBehind>();
                }
                // fragment r of the next depth step
                auto read = [&](int r) {
                    const uint8_t* s = last ? next : cur;
                    const int kk = last ? 0 : k + 1;
                    if (r < kJ) bf[(k + 1) & 1][r] = bfrag(s, r, kk);
                    else af[(k + 1) & 1][r - kJ] = afrag(s, r - kJ, kk);
                };
                constexpr int kReadPer = (kReads + kT - 1) / kT;
#pragma unroll
                for (int t = 0; t < kT; ++t) {
                    acc[t / kJ][t % kJ] = Mf::run(af[k & 1][t / kJ], bf[k & 1][t % kJ], acc[t / kJ][t % kJ]);
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int r = t * kReadPer; r < (t + 1) * kReadPer; ++r)
                        if (r < kReads) read(r);
                    if (!last) {
#pragma unroll
                        for (int c = (k * kT + t) * kPer; c < (k * kT + t + 1) * kPer; ++c)
                            if (c < Sh::kCopies) copy(c, into);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
        if (++b == nb) {
            if (busy) store_tile();
            clear();
            b = 0;
            n0 += TN;
        }
    }
    // no copy may land in the LDS of the workgroup that gets it next
    __builtin_amdgcn_s_waitcnt(0x0070);
}

constexpr int64_t kMaxRun = 2;

// TM x TN tiles by waves of WM x WN, S stages
template <int TM, int TN, int WM, int WN, int S, int MF, int YT, bool GROUPED>
hipError_t tile_launch(const Int8Launch& a, hipStream_t s) {
    using Sh = TileShape<TM, TN, WM, WN, S, MF>;
    const int64_t ntn = (a.out + TN - 1) / TN;
    const int64_t tiles = (a.M + TM - 1) / TM + (GROUPED ? std::min<int64_t>(a.E + 1, a.M) : 0);  // (partial last tiles)
    constexpr int64_t kResident = 256 * std::min(2, 160 * 1024 / (S * Sh::kStage));
    auto turns = [&](int64_t run) { return (tiles * ((ntn + run - 1) / run) + kResident - 1) / kResident * run; };
    int64_t run = 1;
    while ((TM <= 64 || !GROUPED) && run < kMaxRun && 2 * run <= ntn && turns(2 * run) * 16 <= turns(1) * 17) run *= 2;
    const TileParams p{(const uint8_t*)a.codes, a.scales, (const uint8_t*)a.x, a.x_scales, a.M, (int)a.out, (int)a.n, (int)a.E,
                       (int)run, a.offsets, a.tiles, a.y};
    const int64_t total = tiles * ((ntn + run - 1) / run);
    if (total >= (int64_t)(UINT32_MAX / (64 * Sh::kWaves))) return hipErrorInvalidConfiguration;
    const dim3 grid((unsigned)((total + 7) / 8 * 8)), block(64 * Sh::kWaves);
    if (a.n % kBlock) hipLaunchKernelGGL((int8_tile_kernel<TM, TN, WM, WN, S, MF, YT, GROUPED, true>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((int8_tile_kernel<TM, TN, WM, WN, S, MF, YT, GROUPED, false>), grid, block, 0, s, p);
    return hipGetLastError();
}

}  // namespace

Int8Tile int8_tile(int64_t M, int64_t E, int64_t out, bool grouped) {
    auto count = [&](int64_t t) { return (M + t - 1) / t * ((out + t - 1) / t); };
    if (!grouped) return count(256) >= 160 ? Int8Tile{256, 256} : (count(128) >= 160 ? Int8Tile{128, 128} : Int8Tile{64, 64});
    const double per = (double)M / (double)E, spread = std::sqrt(per);
    if (per + 2 * spread <= 16) return {16, 128};
    if (per + spread <= 32) return {32, 128};
    if (per + 2 * spread <= 64) return {64, 128};
    return per >= 192 && count(256) >= 160 ? Int8Tile{256, 256} : Int8Tile{128, 128};
}

hipError_t launch_int8_tile(const Int8Launch& a, const Int8Tile& t, hipStream_t s) {
    hipError_t e = hipSuccess;
    by_float(a.y_dtype, [&](auto yt) {
        constexpr int YT = decltype(yt)::value;
        if (a.offsets) {
            if (t.rows == 16) e = tile_launch<16, 128, 16, 32, 4, 16, YT, true>(a, s);
            else if (t.rows == 32) e = tile_launch<32, 128, 32, 32, 3, 16, YT, true>(a, s);
            else if (t.rows == 64) e = tile_launch<64, 128, 32, 64, 2, 32, YT, true>(a, s);
            else if (t.rows == 128) e = tile_launch<128, 128, 64, 64, 2, 32, YT, true>(a, s);
            else e = tile_launch<256, 256, 64, 128, 2, 32, YT, true>(a, s);
        } else {
            if (t.rows == 64) e = tile_launch<64, 64, 32, 32, 4, 32, YT, false>(a, s);
            else if (t.rows == 128) e = tile_launch<128, 128, 64, 64, 2, 32, YT, false>(a, s);
            else e = tile_launch<256, 256, 64, 128, 2, 32, YT, false>(a, s);
        }
    });
    return e;
}

}  // namespace iqk
