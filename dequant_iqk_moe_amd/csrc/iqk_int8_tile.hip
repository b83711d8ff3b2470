// iqk_int8_tile.hip -- the 8-bit integer product tile by tile, dense or over rows
// sorted by expert.
//
// A workgroup owns TM rows of x by TN weight rows.  Each block of 128 of the depth
// goes from memory straight into LDS, S - 1 blocks ahead.  The sums are int32 and
// exact, so they stay in the matrix instructions' accumulators over the whole depth,
// and the scales are applied once at the end.
//
// Bound: the matrix instructions run at 3.2 POP/s by themselves on such values (their
// power; 4.4 on zeros), and a tile of 256 x 256 needs 64 KiB from the L2 for each 16.8
// MOP.  8192 x 4096 x 4096 takes 127 us (2.16 POP/s beside copies at 8.5 TB/s; 2.10
// POP/s in a library's product without scales): without copies 85, without the
// results' stores 113, with codes of zero 115.  Smaller tiles copy more for a product:
// 128 x 256 need 48 KiB for 8.4 MOP, and 24576 rows by 64 experts of 2048 x 4096 take
// 276 us (1.5 POP/s, 8 % of the products on rows that are not there).
// Two stages of a tile of 256 x 256 are 128 KiB of LDS, so a CU has one: eight waves,
// two a SIMD, whose sums are 128 of their 256 registers.
#include <algorithm>
#include <cmath>

#include "iqk_block.h"
#include "iqk_rows_device.h"

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

// 16 bytes per lane from a buffer straight into LDS (zeros where the offset is past
// its records): lane l's go to dst + 16 l.  An instruction of its own, with m0 named,
// for lds_copy16's reasons.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void lds_copy16(u32x4 rsrc, uint32_t off, uint32_t dst) {
    const uint32_t at = __builtin_amdgcn_readfirstlane(dst);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(at), "v"(off), "s"(rsrc) : "memory", "m0");
}
#pragma clang diagnostic pop
__device__ __forceinline__ u32x4 tile_rsrc(const uint8_t* base, uint32_t bytes) {
    const uint64_t a = (uint64_t)(uintptr_t)base;
    auto uniform = [](uint32_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)v); };
    return u32x4{uniform((uint32_t)a), uniform((uint32_t)(a >> 32)), uniform(bytes), (uint32_t)kRsrcWord3};
}

// The 16-byte chunk c of a row in LDS is kept at slot c ^ key(row).  The 64 lanes of a
// 16-byte read go in four turns of 256 bytes, lanes {0-3, 12-15, 20-27} of each 32
// together and the others together (read off the conflict counter), so the sixteen of
// a turn have to differ in their place modulo 256.  A fragment of 32 rows reads one
// chunk of rows l, or of weight rows that are the same two sets, whose lowest bit
// tells halves of the 256 apart.  Fragments of 16 rows read four chunks: rows l, and
// weight rows that differ in bits 0, 1 and 3.
template <int MF>
__device__ __forceinline__ int xkey_of(int r) { return MF == 32 ? (r >> 1) & 7 : xkey(r); }
template <int MF>
__device__ __forceinline__ int wkey_of(int r) { return MF == 32 ? (r >> 1) & 7 : (r & 3) | ((r >> 1) & 4); }

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
    static_assert(WN % 32 == 0, "tiles of 16 weight rows come in pairs");
    static constexpr int kSteps = kBlock / Mfma<MF>::kDepth;  // instructions' depths in a block
    static constexpr int kRowsPerCopy = 8 * kWaves;           // rows one copy instruction of all waves covers
    static constexpr int kCW = TN / kRowsPerCopy;
    static constexpr int kCX = (TM + kRowsPerCopy - 1) / kRowsPerCopy;
    static constexpr int kCopies = kCW + kCX;  // memory instructions of a wave per block
    static constexpr int kX = TN * kBlock;         // offset of x's rows in a stage
    static constexpr int kStage = kX + kCX * kRowsPerCopy * kBlock;
    static constexpr int kLds = S * kStage;
    static_assert(kLds <= 160 * 1024, "LDS");
    static constexpr int kResident = 2 * kLds <= 160 * 1024 ? 2 : 1;  // workgroups of a CU
};

template <int TM, int TN, int WM, int WN, int S, int MF, int YT, bool GROUPED, bool PART>
__global__ __launch_bounds__(64 * (TM / WM) * (TN / WN), (TileShape<TM, TN, WM, WN, S, MF>::kResident)) void int8_tile_kernel(TileParams p) {
    using Sh = TileShape<TM, TN, WM, WN, S, MF>;
    using Mf = Mfma<MF>;
    constexpr int kSteps = Sh::kSteps;
    __shared__ __align__(16) uint8_t sh[Sh::kLds];
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

    // copies: eight lanes move the slots of a row; rows past the last are past the buffer's records
    const int crow = wave * 8 + (lane >> 3), cslot = lane & 7;
    static_assert(Sh::kRowsPerCopy % 16 == 0, "a lane's chunk is the same in all of its copies");
    const int wch = 16 * (cslot ^ wkey_of<MF>(crow)), xch = 16 * (cslot ^ xkey_of<MF>(crow));
    const uint32_t woff = (uint32_t)(crow * p.n + wch), xoff = (uint32_t)(crow * p.n + xch);
    const uint32_t apart = (uint32_t)(Sh::kRowsPerCopy * p.n);  // of a lane's rows in two copies
    const uint8_t* xbase = p.x + (begin + m0) * p.n;
    const uint32_t xbytes = (uint32_t)(rows * p.n);
    // the next block to copy: block cb of the weight tile at row cn
    int cb = 0, cn = n0;
    const uint8_t* wbase;
    uint32_t wbytes;
    auto weight_tile = [&]() {
        wbase = p.W + ((int64_t)e * p.out + cn) * p.n;
        wbytes = (uint32_t)(min(TN, p.out - cn) * p.n);
    };
    weight_tile();
    const uint32_t sh0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)sh;
    // Copy c of the kCopies that bring the next block into a stage: weight rows, rows of x.  PART: the depth's last
    // block is partial, and chunks past the depth are zero.  (Once the last block is on its way the last tile's first
    // one is copied again, which nothing reads: every step takes as many instructions, and the waits count them.)
    auto copy = [&](int c, int slot) {
        const uint32_t k0 = cb * kBlock, at = sh0 + slot * Sh::kStage + wave * 1024;
        if (c < Sh::kCW) {
            const uint32_t off = PART && (int)k0 + wch >= p.n ? kOob : woff;
            lds_copy16(tile_rsrc(wbase + k0, wbytes - k0), off + c * apart, at + c * Sh::kRowsPerCopy * kBlock);
        } else {
            const int i = c - Sh::kCW;
            const uint32_t off = PART && (int)k0 + xch >= p.n ? kOob : xoff;
            lds_copy16(tile_rsrc(xbase + k0, xbytes - k0), off + i * apart, at + Sh::kX + i * Sh::kRowsPerCopy * kBlock);
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

    // Weight rows are dealt to a fragment's lanes so that a result lane's values are eight consecutive outputs: of a
    // 32-row tile, lane l reads row 16 (l / 16) + 8 (l / 4 % 2) + 4 (l / 8 % 2) + l % 4; of a pair of 16-row tiles,
    // row 8 (l / 4) + l % 4, and 4 more in the second.
    const int l = lane & (MF - 1), g = lane / MF;
    const int afirst = MF == 32 ? 16 * (l >> 4) + 8 * ((l >> 2) & 1) + 4 * ((l >> 3) & 1) + (l & 3) : 8 * (l >> 2) + (l & 3);

    constexpr int kBehind = (S - 2) * Sh::kCopies;  // copies that may still be on their way when a block is published
    const int steps = nb * ((nend - n0 + TN - 1) / TN);
#pragma unroll
    for (int b = 0; b < S - 1; ++b) {
#pragma unroll
        for (int c = 0; c < Sh::kCopies; ++c) copy(c, b);
        advance();
    }
    publish<kBehind>();

    // the tiles by this wave: kI tiles of weight rows from wn on and kJ of x from wm on
    auto multiply = [&](const int wn, const int wm) {
        constexpr int kI = WN / MF, kJ = WM / MF;
        int slot = 0;
        if (wm >= rows) {  // none of its rows of x is there: it copies for the others
            for (int step = 0; step < steps; ++step) {
                const int into = slot == 0 ? S - 1 : slot - 1;
                slot = slot == S - 1 ? 0 : slot + 1;
#pragma unroll
                for (int c = 0; c < Sh::kCopies; ++c) copy(c, into);
                advance();
                publish<kBehind>();
            }
            return;
        }
        typename Mf::Acc acc[kI][kJ];
        const int aoff = (wn + afirst) * kBlock + 16 * (g ^ wkey_of<MF>(afirst));
        const int boff = Sh::kX + (wm + l) * kBlock + 16 * (g ^ xkey_of<MF>(l));
        // fragments of weight tile i and x tile j at depth step k of the stage at s
        auto afrag = [&](const uint8_t* s, int i, int k) {
            const int tile = (MF == 32 ? i * 32 : (i >> 1) * 32 + (i & 1) * 4) * kBlock;
            return *(const i32x4*)(s + (aoff ^ (k * Mf::kDepth)) + tile);
        };
        auto bfrag = [&](const uint8_t* s, int j, int k) { return *(const i32x4*)(s + (boff ^ (k * Mf::kDepth)) + j * MF * kBlock); };

        // value q of the eight of piece h (of 16 outputs, or of 32 of two tiles of 16 rows) in x tile j
        auto value = [&](int h, int j, int q, float scale) {
            const int a = MF == 32 ? acc[h >> 1][j][8 * (h & 1) + q] : acc[2 * h + (q >> 2)][j][q & 3];
            float v = (float)a * scale;
            // (fused with the conversion to f16 the product would round once, where the definition's rounds twice)
            if constexpr (YT == IQK_F16) asm("" : "+v"(v));
            return v;
        };
        constexpr int kPieces = MF == 32 ? kI * 2 : kI / 2, kPiece = MF == 32 ? 16 : 32;  // outputs
        // the results of the weight tile at row n0
        auto store_tile = [&]() {
            // (addresses are made here: kept over the loop they would not leave enough registers)
            int lane_ = lane;
            asm volatile("" : "+v"(lane_));
            const int l = lane_ & (MF - 1), g = lane_ / MF;
            float sx[kJ];
#pragma unroll
            for (int j = 0; j < kJ; ++j) sx[j] = p.sx[begin + m0 + min(wm + MF * j + l, rows - 1)];
            float sw[kPieces][8];  // (zeros past the last output)
            const Rsrc sr = make_rsrc(p.sw + (int64_t)e * p.out, (uint32_t)p.out * 4);
#pragma unroll
            for (int h = 0; h < kPieces; ++h)
#pragma unroll
                for (int q = 0; q < 8; ++q) sw[h][q] = __uint_as_float(ld32(sr, (uint32_t)(n0 + wn + 8 * g) * 4 + (kPiece * h + q) * 4));
#pragma unroll
            for (int h = 0; h < kPieces; ++h) {
                const int o = n0 + wn + kPiece * h + 8 * g;
#pragma unroll
                for (int j = 0; j < kJ; ++j) {
                    const int i = wm + MF * j + l;
                    float v[8];
#pragma unroll
                    for (int q = 0; q < 8; ++q) v[q] = value(h, j, q, sx[j] * sw[h][q]);
                    if (i < rows && o < p.out) store_some<YT>(p.y, (begin + m0 + i) * p.out + o, v, p.out - o);
                }
                __builtin_amdgcn_sched_barrier(0);  // (else all of the tile's values are wanted at once)
            }
        };

        // Fragments of a depth step are read while the step before it is multiplied; the block's last step is multiplied
        // behind the barrier that publishes the next block, with that block's first fragments read beside it.
        // (A tile's first ones are read at its start, so that none is held while the last tile's results leave.)
        i32x4 af[2][kI], bf[2][kJ];
        static_assert(kSteps % 2 == 0, "a block ends on the fragments it began with");
        constexpr int kT = kI * kJ, kReads = kI + kJ;
        // Products before the block's last depth step, and those of them that copies go behind: where there are enough, the
        // ones that no read goes behind (a wave issues an instruction in four cycles, and a product takes 32).
        constexpr int kReadPer = (kReads + kT - 1) / kT, kReadSlots = (kReads + kReadPer - 1) / kReadPer;
        constexpr int kSlots = (kSteps - 1) * kT;
        constexpr bool kApart = (kSteps - 1) * (kT - kReadSlots) >= Sh::kCopies;
        constexpr int kPer = kApart ? 1 : (Sh::kCopies + kSlots - 1) / kSlots;
        for (; n0 < nend; n0 += TN) {
#pragma unroll
            for (int i = 0; i < kI; ++i)
#pragma unroll
                for (int j = 0; j < kJ; ++j) acc[i][j] = typename Mf::Acc{};
#pragma unroll
            for (int i = 0; i < kI; ++i) af[0][i] = afrag(sh + slot * Sh::kStage, i, 0);
#pragma unroll
            for (int j = 0; j < kJ; ++j) bf[0][j] = bfrag(sh + slot * Sh::kStage, j, 0);
            int b = nb;
            do {
                const uint8_t* cur = sh + slot * Sh::kStage;
                const int into = slot == 0 ? S - 1 : slot - 1;
                slot = slot == S - 1 ? 0 : slot + 1;
                const uint8_t* next = sh + slot * Sh::kStage;
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
#pragma unroll
                    for (int t = 0; t < kT; ++t) {
                        acc[t / kJ][t % kJ] = Mf::run(af[k & 1][t / kJ], bf[k & 1][t % kJ], acc[t / kJ][t % kJ]);
                        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                        for (int r = t * kReadPer; r < (t + 1) * kReadPer; ++r)
                            if (r < kReads) read(r);
                        if (!last && (!kApart || t >= kReadSlots)) {
                            const int at = kApart ? k * (kT - kReadSlots) + t - kReadSlots : k * kT + t;
#pragma unroll
                            for (int c = at * kPer; c < (at + 1) * kPer; ++c)
                                if (c < Sh::kCopies) copy(c, into);
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
            } while (--b > 0);
            store_tile();
        }
    };
    multiply((wave % (TN / WN)) * WN, (wave / (TN / WN)) * WM);
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
    constexpr int64_t kResident = 256 * Sh::kResident;
    auto turns = [&](int64_t run) { return (tiles * ((ntn + run - 1) / run) + kResident - 1) / kResident * run; };
    int64_t run = 1;
    while (!GROUPED && run < kMaxRun && 2 * run <= ntn && turns(2 * run) * 16 <= turns(1) * 17) run *= 2;
    const TileParams p{(const uint8_t*)a.codes, a.scales, (const uint8_t*)a.x, a.x_scales, a.M, (int)a.out, (int)a.n, (int)a.E,
                       (int)run, a.offsets, a.tiles, a.y};
    const int64_t total = tiles * ((ntn + run - 1) / run);
    if (total >= (int64_t)(UINT32_MAX / (64 * Sh::kWaves))) return hipErrorInvalidConfiguration;
    const dim3 grid((unsigned)((total + 7) / 8 * 8)), block(64 * Sh::kWaves);
    if (a.n % kBlock) hipLaunchKernelGGL((int8_tile_kernel<TM, TN, WM, WN, S, MF, YT, GROUPED, true>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((int8_tile_kernel<TM, TN, WM, WN, S, MF, YT, GROUPED, false>), grid, block, 0, s, p);
    return hipGetLastError();
}

// Tiles, and what one takes where each CU has one: microseconds before its first block and behind its last, and for
// each block of 128 of the depth (measured, bfloat16 results: 1024 x 4096 x 4096 in tiles of 128 x 128 26 us, 2048 rows
// in 128 x 256 38, 8192 in 256 x 256 129; 8 experts of 1024 x 4096 with 37 rows each in tiles of 16, 32 and 64 rows 15,
// 18 and 19).  Where two tiles share a CU they take about twice as long.
struct Kind {
    int rows, cols;
    double fixed, block;
    bool shared;
};
constexpr Kind kKinds[] = {{16, 128, 4, 0.34, true},  {32, 128, 4, 0.43, true},  {64, 128, 4, 0.48, true},
                           {128, 128, 5, 0.62, false}, {128, 256, 8, 0.85, false}, {256, 256, 15, 1.45, false}};

}  // namespace

// The kind whose rounds over the 256 CUs take the shortest by that, or as long as the weights from memory; the one of
// the fewest rows of those within 5 % of it.  (Experts' last tiles are half full in the mean.)
Int8Tile int8_tile(int64_t M, int64_t E, int64_t out, int64_t n, bool grouped) {
    const double blocks = (double)((n + 127) / 128), used = grouped ? (double)std::min(M, E) : 0.0;
    const double bytes = std::max(used, 1.0) * (double)(out * n) / 5.3e6;
    auto us = [&](const Kind& k) {
        const double rows = grouped ? (double)M / k.rows + used / 2 : (double)((M + k.rows - 1) / k.rows);
        const double rounds = rows * (double)((out + k.cols - 1) / k.cols) / 256;
        return std::max(bytes, (k.shared ? std::max(rounds, 1.0) : std::ceil(rounds)) * (k.fixed + k.block * blocks));
    };
    double best = us(kKinds[0]);
    for (const Kind& k : kKinds) best = std::min(best, us(k));
    for (const Kind& k : kKinds)
        if (us(k) <= 1.05 * best) return Int8Tile{k.rows, k.cols};
    return Int8Tile{256, 256};
}

hipError_t launch_int8_tile(const Int8Launch& a, const Int8Tile& t, hipStream_t s) {
    hipError_t e = hipSuccess;
    by_float(a.y_dtype, [&](auto yt) {
        auto go = [&](auto grouped) {
            constexpr int YT = decltype(yt)::value;
            constexpr bool G = decltype(grouped)::value;
            if (t.rows == 16) e = tile_launch<16, 128, 16, 32, 4, 16, YT, G>(a, s);
            else if (t.rows == 32) e = tile_launch<32, 128, 32, 32, 3, 16, YT, G>(a, s);
            else if (t.rows == 64) e = tile_launch<64, 128, 32, 64, 3, 32, YT, G>(a, s);
            else if (t.cols == 128) e = tile_launch<128, 128, 64, 64, 4, 32, YT, G>(a, s);
            else if (t.rows == 128) e = tile_launch<128, 256, 64, 64, 3, 32, YT, G>(a, s);
            else e = tile_launch<256, 256, 64, 128, 2, 32, YT, G>(a, s);
        };
        if (a.offsets) go(std::true_type{});
        else go(std::false_type{});
    });
    return e;
}

}  // namespace iqk
