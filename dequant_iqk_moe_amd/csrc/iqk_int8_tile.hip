// iqk_int8_tile.hip -- the 8-bit integer product tile by tile, dense or over rows
// sorted by expert.
//
// A workgroup owns TM rows of x by TN weight rows.  Each block of BK of the depth goes
// from memory straight into LDS, S - 1 blocks ahead.  The sums are int32 and exact, so they stay in the matrix instructions'
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
    bool whole;  // y's rows begin at multiples of 16 bytes
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

// The 16-byte chunk c of a row in LDS is kept at slot c ^ key(row), so that eight
// neighbouring lanes of a fragment, which read chunk c of eight rows, meet 128 bytes
// no two of which are in one bank.  Rows of x: lane l reads row l + const.  Weight
// rows: eight lanes' rows differ in bits 0, 1 and 3.  Two rows of 64 bytes share the
// 128, which their lowest bit tells apart.
template <int BK>
__device__ __forceinline__ int xkey_of(int r) { return BK == 128 ? r & 7 : (r >> 1) & 3; }
template <int BK>
__device__ __forceinline__ int wkey_of(int r) { return BK == 128 ? (r & 3) | ((r >> 1) & 4) : ((r >> 1) & 1) | ((r >> 2) & 2); }

// Two results as 16-bit values, rounded to nearest even (the hardware's conversions).
template <int YT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if constexpr (YT == IQK_F16) return __builtin_bit_cast(uint32_t, f16x2{(_Float16)a, (_Float16)b});
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
}

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

template <int TM, int TN, int WM, int WN, int BK, int S, int MF>
struct TileShape {
    static constexpr int kWaves = (TM / WM) * (TN / WN);
    static_assert(MF == 32 || WN % 32 == 0, "tiles of 16 weight rows come in pairs");
    // a tile of x with at most half of its rows there is one row of waves, each with fewer weight rows
    static constexpr bool kHalves = TM == 256 && WM == 128;
    static constexpr int kSteps = BK / Mfma<MF>::kDepth;         // instructions' depths in a block
    static constexpr int kLanes = BK / 16;                       // lanes of a copy that share a row
    static constexpr int kRowsPerCopy = 64 / kLanes * kWaves;    // rows one copy instruction of all waves covers
    static constexpr int kCW = TN / kRowsPerCopy;
    static constexpr int kCX = (TM + kRowsPerCopy - 1) / kRowsPerCopy;
    static constexpr int kCopies = kCW + kCX;  // memory instructions of a wave per block
    static constexpr int kX = TN * BK;         // offset of x's rows in a stage
    static constexpr int kStage = kX + kCX * kRowsPerCopy * BK;
    // Results of large tiles go through LDS, 8 KiB of a wave at a time, and leave in whole rows of it.
    static constexpr bool kStaged = kHalves;
    static constexpr int kOut = 8192, kLds = S * kStage + (kStaged ? kWaves * kOut : 0);
    static_assert(kLds <= 160 * 1024, "LDS");
    static constexpr int kResident = 2 * kLds <= 160 * 1024 ? 2 : 1;  // workgroups of a CU
};

template <int TM, int TN, int WM, int WN, int BK, int S, int MF, int YT, bool GROUPED, bool PART>
__global__ __launch_bounds__(64 * (TM / WM) * (TN / WN), (TileShape<TM, TN, WM, WN, BK, S, MF>::kResident)) void int8_tile_kernel(TileParams p) {
    using Sh = TileShape<TM, TN, WM, WN, BK, S, MF>;
    using Mf = Mfma<MF>;
    constexpr int kSteps = Sh::kSteps;
    __shared__ __align__(16) uint8_t sh[Sh::kLds];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int nb = (p.n + BK - 1) / BK;
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

    // copies: kLanes lanes move the slots of a row; rows past the last are past the buffer's records
    const int crow = (wave * 64 + lane) / Sh::kLanes, cslot = lane % Sh::kLanes;
    static_assert(Sh::kRowsPerCopy % 16 == 0, "a lane's chunk is the same in all of its copies");
    const int wch = 16 * (cslot ^ wkey_of<BK>(crow)), xch = 16 * (cslot ^ xkey_of<BK>(crow));
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
        const uint32_t k0 = cb * BK, at = sh0 + slot * Sh::kStage + wave * 1024;
        if (c < Sh::kCW) {
            const uint32_t off = PART && (int)k0 + wch >= p.n ? kOob : woff;
            lds_copy16(tile_rsrc(wbase + k0, wbytes - k0), off + c * apart, at + c * Sh::kRowsPerCopy * BK);
        } else {
            const int i = c - Sh::kCW;
            const uint32_t off = PART && (int)k0 + xch >= p.n ? kOob : xoff;
            lds_copy16(tile_rsrc(xbase + k0, xbytes - k0), off + i * apart, at + Sh::kX + i * Sh::kRowsPerCopy * BK);
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
    auto multiply = [&](auto ki, auto kj, const int wn, const int wm) {
        constexpr int kI = decltype(ki)::value, kJ = decltype(kj)::value;
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
        const int aoff = (wn + afirst) * BK + 16 * (g ^ wkey_of<BK>(afirst));
        const int boff = Sh::kX + (wm + l) * BK + 16 * (g ^ xkey_of<BK>(l));
        // fragments of weight tile i and x tile j at depth step k of the stage at s
        auto afrag = [&](const uint8_t* s, int i, int k) {
            const int tile = (MF == 32 ? i * 32 : (i >> 1) * 32 + (i & 1) * 4) * BK;
            return *(const i32x4*)(s + (aoff ^ (k * Mf::kDepth)) + tile);
        };
        auto bfrag = [&](const uint8_t* s, int j, int k) { return *(const i32x4*)(s + (boff ^ (k * Mf::kDepth)) + j * MF * BK); };

        // value q of the eight of piece h (of 16 outputs, or of 32 of two tiles of 16 rows) in x tile j
        auto value = [&](int h, int j, int q, float scale) {
            int a = MF == 32 ? acc[h >> 1][j][8 * (h & 1) + q] : acc[2 * h + (q >> 2)][j][q & 3];
            // (a large tile's sums fill the accumulation registers, and the compiler would move all of them at once)
            if constexpr (Sh::kStaged) {
                const int in = a;
                asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(a) : "a"(in));
            }
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
            if constexpr (!Sh::kStaged) {
#pragma unroll
                for (int h = 0; h < kPieces; ++h) {
                    const int o = n0 + wn + kPiece * h + 8 * g;
#pragma unroll
                    for (int j = 0; j < kJ; ++j) {
                        const int i = wm + MF * j + l;
                        float v[8];
#pragma unroll
                        for (int q = 0; q < 8; ++q) v[q] = value(h, j, q, sx[j] * sw[h][q]);
                        if (i < rows && o < p.out) store8<YT>(p.y, (begin + m0 + i) * p.out + o, v, p.out - o);
                    }
                    __builtin_amdgcn_sched_barrier(0);  // (else all of the tile's values are wanted at once)
                }
            } else {
                // (the reads below are not the compiler's: the last products' results are waited for here)
                __builtin_amdgcn_sched_barrier(0);
                asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
                // 32 rows of x by kCols outputs, 16 bytes at slot c ^ (row & 15 or less) of a row; lanes then take
                // neighbouring chunks of a row
                constexpr int kSize = YT == IQK_F32 ? 4 : 2, kAll = kI * 32, kCols = kAll * kSize > 256 ? 256 / kSize : kAll;
                constexpr int kChunks = kCols * kSize / 16, kPer = 16 / kSize;  // chunks of a row, values of a chunk
                uint8_t* mine = sh + S * Sh::kStage + wave * Sh::kOut;
                const Rsrc yr = make_rsrc((uint8_t*)p.y + (begin + m0) * p.out * kSize, (uint32_t)rows * (uint32_t)p.out * kSize);
#pragma unroll
                for (int c0 = 0; c0 < kAll; c0 += kCols) {
#pragma unroll
                    for (int j = 0; j < kJ; ++j) {
#pragma unroll
                        for (int h = c0 / 16; h < (c0 + kCols) / 16; ++h) {
                            float v[8];
#pragma unroll
                            for (int q = 0; q < 8; ++q) v[q] = value(h, j, q, sx[j] * sw[h][q]);
                            const int chunk = ((16 * h - c0) + 8 * g) / kPer;
                            auto slot = [&](int c) { return (uint4*)(mine + l * kChunks * 16 + 16 * (c ^ (l & (kChunks - 1)))); };
                            if constexpr (YT == IQK_F32) {
                                *(float4*)slot(chunk) = make_float4(v[0], v[1], v[2], v[3]);
                                *(float4*)slot(chunk + 1) = make_float4(v[4], v[5], v[6], v[7]);
                            } else {
                                uint4 w;
                                w.x = pack2<YT>(v[0], v[1]), w.y = pack2<YT>(v[2], v[3]), w.z = pack2<YT>(v[4], v[5]), w.w = pack2<YT>(v[6], v[7]);
                                *slot(chunk) = w;
                            }
                            __builtin_amdgcn_sched_barrier(0);
                        }
                        auto piece = [&](int u) { return *(const uint4*)(mine + u / kChunks * kChunks * 16 + 16 * (u % kChunks ^ (u / kChunks & (kChunks - 1)))); };
                        if (p.whole) {  // (rows past the last are past the records, outputs are made so)
                            constexpr int kTurns = 32 * kChunks / 64;
                            uint4 w[kTurns];
#pragma unroll
                            for (int u = 0; u < kTurns; ++u) w[u] = piece(u * 64 + lane_);
#pragma unroll
                            for (int u = 0; u < kTurns; ++u) {
                                const int at = u * 64 + lane_, o = n0 + wn + c0 + at % kChunks * kPer;
                                const uint32_t to = (uint32_t)((wm + 32 * j + at / kChunks) * p.out + o) * kSize;
                                __builtin_amdgcn_raw_buffer_store_b128(u32x4{w[u].x, w[u].y, w[u].z, w[u].w}, yr, o < p.out ? to : kOob, 0, 0);
                            }
                        } else {
#pragma unroll 1
                            for (int u = lane_; u < 32 * kChunks; u += 64) {
                                const int i = wm + 32 * j + u / kChunks, o = n0 + wn + c0 + u % kChunks * kPer;
                                if (i >= rows || o >= p.out) continue;
                                const uint4 w = piece(u);
                                const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                                for (int q = 0; q < kPer; ++q) {
                                    if (o + q >= p.out) continue;
                                    const int64_t at = (begin + m0 + i) * p.out + o + q;
                                    if constexpr (YT == IQK_F32) ((uint32_t*)p.y)[at] = a[q];
                                    else ((uint16_t*)p.y)[at] = (uint16_t)(a[q / 2] >> (16 * (q & 1)));
                                }
                            }
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
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
    constexpr int kI = WN / MF, kJ = WM / MF;
    const int wn = (wave % (TN / WN)) * WN, wm = (wave / (TN / WN)) * WM;
    if (Sh::kHalves && rows <= TM / 2) {
        constexpr int kRows = TM / WM;
        multiply(std::integral_constant<int, Sh::kHalves ? kI / kRows : kI>{}, std::integral_constant<int, kJ>{}, wave * (WN / kRows), 0);
    } else {
        multiply(std::integral_constant<int, kI>{}, std::integral_constant<int, kJ>{}, wn, wm);
    }
    // no copy may land in the LDS of the workgroup that gets it next
    __builtin_amdgcn_s_waitcnt(0x0070);
}

constexpr int64_t kMaxRun = 2;

// TM x TN tiles by waves of WM x WN, S stages
template <int TM, int TN, int WM, int WN, int BK, int S, int MF, int YT, bool GROUPED>
hipError_t tile_launch(const Int8Launch& a, hipStream_t s) {
    using Sh = TileShape<TM, TN, WM, WN, BK, S, MF>;
    const int64_t ntn = (a.out + TN - 1) / TN;
    const int64_t tiles = (a.M + TM - 1) / TM + (GROUPED ? std::min<int64_t>(a.E + 1, a.M) : 0);  // (partial last tiles)
    constexpr int64_t kResident = 256 * Sh::kResident;
    auto turns = [&](int64_t run) { return (tiles * ((ntn + run - 1) / run) + kResident - 1) / kResident * run; };
    int64_t run = 1;
    while ((TM <= 64 || !GROUPED) && run < kMaxRun && 2 * run <= ntn && turns(2 * run) * 16 <= turns(1) * 17) run *= 2;
    const TileParams p{(const uint8_t*)a.codes, a.scales, (const uint8_t*)a.x, a.x_scales, a.M, (int)a.out, (int)a.n, (int)a.E,
                       (int)run, a.offsets, a.tiles, a.y, a.out % (a.y_dtype == IQK_F32 ? 4 : 8) == 0 && (uintptr_t)a.y % 16 == 0};
    const int64_t total = tiles * ((ntn + run - 1) / run);
    if (total >= (int64_t)(UINT32_MAX / (64 * Sh::kWaves))) return hipErrorInvalidConfiguration;
    const dim3 grid((unsigned)((total + 7) / 8 * 8)), block(64 * Sh::kWaves);
    if (a.n % BK) hipLaunchKernelGGL((int8_tile_kernel<TM, TN, WM, WN, BK, S, MF, YT, GROUPED, true>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((int8_tile_kernel<TM, TN, WM, WN, BK, S, MF, YT, GROUPED, false>), grid, block, 0, s, p);
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
            if (t.rows == 16) e = tile_launch<16, 128, 16, 32, 128, 4, 16, YT, true>(a, s);
            else if (t.rows == 32) e = tile_launch<32, 128, 32, 32, 128, 3, 16, YT, true>(a, s);
            else if (t.rows == 64) e = tile_launch<64, 128, 32, 64, 128, 2, 32, YT, true>(a, s);
            else if (t.rows == 128) e = tile_launch<128, 128, 64, 64, 128, 2, 32, YT, true>(a, s);
            else e = tile_launch<256, 256, 128, 128, 64, 4, 32, YT, true>(a, s);
        } else {
            if (t.rows == 64) e = tile_launch<64, 64, 32, 32, 128, 4, 32, YT, false>(a, s);
            else if (t.rows == 128) e = tile_launch<128, 128, 64, 64, 128, 2, 32, YT, false>(a, s);
            else e = tile_launch<256, 256, 128, 128, 64, 4, 32, YT, false>(a, s);
        }
    });
    return e;
}

}  // namespace iqk
