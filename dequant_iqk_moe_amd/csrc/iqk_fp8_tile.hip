// iqk_fp8_tile.hip -- the 8-bit product for many rows, tile by tile.
#include <algorithm>

#include "iqk_fp8_device.h"

namespace iqk {
namespace {

// ---------------------------------------------------------------------------
// tiled product
// ---------------------------------------------------------------------------

typedef int i32x8 __attribute__((ext_vector_type(8)));

struct TileParams {
    const uint8_t* W;
    const float* sw;
    const uint8_t* x;
    const float* sx;
    int64_t M;
    int out, n, k, x_slots, E;
    const int32_t *offsets, *perm, *tiles;  // grouped: tiles[e] = 256- or 128-row tiles of x before expert e
    void* y;
};

// 16 bytes per lane from memory straight into LDS: lane l's go to dst + 16 l
// (an LDS address, the same in every lane).  Written as an instruction because the
// compiler takes every later LDS read to depend on the builtin's copy and
// waits for it at once; the kernel waits for its copies before the barrier
// that publishes them.  The instruction has no register result.
__device__ __forceinline__ void lds_copy16(const uint8_t* base, uint32_t off, uint32_t dst) {
    const uint32_t at = __builtin_amdgcn_readfirstlane(dst);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(at), "v"(off), "s"(base) : "memory");
}
__device__ __forceinline__ void lds_copy16(const uint8_t* src, uint32_t dst) {
    const uint32_t at = __builtin_amdgcn_readfirstlane(dst);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(at), "v"(src) : "memory");
}

// Waits for this wave's copies and LDS accesses, then for the other waves'.
__device__ __forceinline__ void publish() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// The 16-byte chunk of a 128-byte tile row is kept at slot chunk ^ key(row),
// so that eight neighbouring lanes of a fragment read eight slots.  A
// fragment's 16 lanes read weight rows 16 (l / 4) + l % 4 + const (keyed by
// the row's bits 0, 1 and 4) and x rows l + const (by its bits 0 to 2).
__device__ __forceinline__ int wkey(int r) { return (r & 3) | ((r >> 2) & 4); }
__device__ __forceinline__ int xkey(int r) { return r & 7; }

template <int TM, int TN, int WM, int WN, int YT, bool GROUPED, bool EXACT>
__global__ __launch_bounds__(64 * (TM / WM) * (TN / WN)) void fp8_tile_kernel(TileParams p) {
    constexpr int kNW = (TM / WM) * (TN / WN);  // waves
    constexpr int kI = WN / 16, kJ = WM / 16;   // a wave's tiles of weight rows and of x rows
    constexpr int kRowsPerCopy = 8 * kNW;       // rows one copy instruction of all waves covers
    constexpr int kCW = TN / kRowsPerCopy, kCX = TM / kRowsPerCopy;
    __shared__ uint8_t sh[2][(TN + TM) * 128];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int li = lane & 15, g = lane >> 4;
    const int nb = (p.n + kBlock - 1) / kBlock;
    const int ntn = (p.out + TN - 1) / TN;

    // which tile: the tiles of one XCD (workgroups b with equal b % 8) are neighbours
    int e = 0;
    int64_t m0, count = p.M, begin = 0;
    int n0;
    {
        const int64_t tiles_m = GROUPED ? p.tiles[p.E] : (p.M + TM - 1) / TM;
        const int64_t total = tiles_m * ntn, per = (total + 7) / 8;
        const int64_t id = (int64_t)(blockIdx.x & 7) * per + (blockIdx.x >> 3);
        if ((int64_t)(blockIdx.x >> 3) >= per || id >= total) return;
        if constexpr (GROUPED) {
            const int t = (int)(id / ntn);
            n0 = (int)(id - (int64_t)t * ntn) * TN;
            // the expert of tile t: the last e with tiles[e] <= t, 64 candidates at a time
            int lo = 0, span = p.E;
            while (span > 1) {
                const int step = (span + 63) / 64;
                const int c = lo + lane * step;
                const uint64_t le = __ballot(c < lo + span && p.tiles[c < p.E ? c : p.E] <= t);
                const int last = 63 - __builtin_clzll(le);
                const int nlo = lo + last * step;
                span = min(step, lo + span - nlo);
                lo = nlo;
            }
            e = __builtin_amdgcn_readfirstlane(lo);
            begin = p.offsets[e];
            count = p.offsets[e + 1] - begin;
            m0 = (int64_t)(t - p.tiles[e]) * TM;
        } else {
            // bands of 8 tiles of x by all of the weights' tiles
            const int64_t band = id / (8 * ntn), in = id - band * 8 * ntn;
            const int64_t rows = min((int64_t)8, tiles_m - band * 8);
            m0 = (band * 8 + in % rows) * TM;
            n0 = (int)(in / rows) * TN;
        }
    }

    // copies: lane l of a copy moves slot l & 7 of row l >> 3 of its wave's
    // eight rows; rows past the end repeat the last, their results are dropped
    const int crow = wave * 8 + (lane >> 3);
    const int nob = (p.out + kBlock - 1) / kBlock;
    static_assert(kRowsPerCopy % 32 == 0, "a lane's chunk is the same in all of its copies");
    const int wch = 16 * ((lane & 7) ^ wkey(crow)), xch = 16 * ((lane & 7) ^ xkey(crow));
    // row i of the tile's x rows, as a row of p.x, and as a row of y
    auto pair_of = [&](int i) { return p.perm[begin + min(m0 + i, count - 1)]; };
    auto row_of = [&](int i) -> int64_t {
        if constexpr (GROUPED) return p.x_slots == 1 ? pair_of(i) / p.k : pair_of(i);
        else return min(m0 + i, count - 1);
    };
    const uint8_t* wbase = p.W + ((int64_t)e * p.out + n0) * p.n;
    const uint8_t* xbase = GROUPED ? p.x : p.x + m0 * p.n;  // (dense: offsets inside the tile fit 32 bits)
    uint32_t woff[kCW], xoff[kCX];  // (grouped: xoff is the row of x, multiplied out at each copy)
#pragma unroll
    for (int c = 0; c < kCW; ++c)
        woff[c] = (uint32_t)(min(c * kRowsPerCopy + crow, p.out - 1 - n0) * p.n + wch);
#pragma unroll
    for (int c = 0; c < kCX; ++c) {
        const int64_t row = row_of(c * kRowsPerCopy + crow);
        xoff[c] = GROUPED ? (uint32_t)row : (uint32_t)((int)(row - m0) * p.n + xch);
    }
    auto copy_w = [&](int c, int k0, uint32_t d) { lds_copy16(wbase + k0, woff[c], d); };
    auto copy_x = [&](int c, int k0, uint32_t d) {
        if constexpr (GROUPED) lds_copy16(xbase + ((uint64_t)xoff[c] * (uint32_t)p.n + (uint32_t)(k0 + xch)), d);
        else lds_copy16(xbase + k0, xoff[c], d);
    };
    const uint32_t sh0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)&sh[0][0];
    auto copy_block = [&](int b) {
        const int k0 = b * kBlock;
        const uint32_t at = (b & 1) * (TN + TM) * 128 + wave * 1024;
        if (k0 + kBlock <= p.n) {
#pragma unroll
            for (int c = 0; c < kCW; ++c) copy_w(c, k0, sh0 + at + c * kRowsPerCopy * 128);
#pragma unroll
            for (int c = 0; c < kCX; ++c) copy_x(c, k0, sh0 + at + (TN + c * kRowsPerCopy) * 128);
        } else {  // the partial last block: chunks past the depth are zero
#pragma unroll
            for (int c = 0; c < kCW; ++c) {
                const uint32_t d = at + c * kRowsPerCopy * 128;
                if (k0 + wch < p.n) copy_w(c, k0, sh0 + d);
                else *(uint4*)(&sh[0][0] + d + lane * 16) = make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int c = 0; c < kCX; ++c) {
                const uint32_t d = at + (TN + c * kRowsPerCopy) * 128;
                if (k0 + xch < p.n) copy_x(c, k0, sh0 + d);
                else *(uint4*)(&sh[0][0] + d + lane * 16) = make_uint4(0, 0, 0, 0);
            }
        }
    };

    const int wn = (wave % (TN / WN)) * WN, wm = (wave / (TN / WN)) * WM;  // this wave's part of the tile
    // scales: one per 128 weight rows (a wave's rows lie in one block), one per row of x
    const float* sw = p.sw + ((int64_t)e * nob + min((n0 + wn) / kBlock, nob - 1)) * nb;
    // (a vector load: a scalar load in flight would make every wait for an LDS read a wait for all of them)
    uint32_t swo = 0;
    asm("" : "+v"(swo));
    const float* sx = GROUPED ? p.sx : p.sx + m0 * nb;
    uint32_t sxo[kJ];  // (grouped: the row of x)
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
        const int64_t row = row_of(wm + 16 * j + li);
        sxo[j] = GROUPED ? (uint32_t)row : (uint32_t)((row - m0) * nb);
    }
    auto x_scale = [&](int j, int b) {
        if constexpr (GROUPED) return sx[(uint64_t)sxo[j] * (uint32_t)nb + (uint32_t)b];
        else return sx[sxo[j] + (uint32_t)b];
    };

    f32x4 acc[kI][kJ];
#pragma unroll
    for (int i = 0; i < kI; ++i)
#pragma unroll
        for (int j = 0; j < kJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    // fragment rows: lane li of tile i reads weight row 64 (i / 4) + 16 (li / 4) + 4 (i % 4) + li % 4, so that a
    // result lane's four rows of four neighbouring tiles are 16 consecutive rows
    const int arow = wn + 16 * (li >> 2) + (li & 3);
    const int brow = wm + li;
    const int aoff = arow * 128 + 16 * (g ^ wkey(16 * (li >> 2) + (li & 3)));
    const int boff = (TN + brow) * 128 + 16 * (g ^ xkey(li));
    auto frag = [&](const uint8_t* s, int off) {
        const uint4 a = *(const uint4*)(s + off), b = *(const uint4*)(s + (off ^ 64));
        return i32x8{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
    };

    // Instruction t = i kJ + j of a block multiplies tile row i by x tile j.  Its product is added to the sums two
    // instructions later (kLag: it is done by then), and a tile row is read kAhead rows before its first use.
    constexpr int kAhead = GROUPED && TM * TN > 128 * 128 ? 1 : 2;  // (two would spill where rows are gathered)
    constexpr int kLag = 2, kRing = 4, kT = kI * kJ;
    static_assert(kT % kRing == 0, "a block's first products follow the last block's in the ring");
    float sxn[kJ], swn, f[kJ], fp[kJ];
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
copy_block(0);
#pragma unroll
    for (int j = 0; j < kJ; ++j) sxn[j] = x_scale(j, 0);
    swn = sw[swo];
    publish();
    for (int b = 0; b < nb; ++b) {
        const uint8_t* cur = sh[b & 1];
#pragma unroll
        for (int j = 0; j < kJ; ++j) f[j] = sxn[j] * swn;
        if (b + 1 < nb) {
            copy_block(b + 1);
#pragma unroll
            for (int j = 0; j < kJ; ++j) sxn[j] = x_scale(j, b + 1);
            swn = sw[swo + (b + 1)];
        }
        // (the key's bits are those of the row inside its 64: tile rows i and i + 4 are 64 rows apart, i and i + 1
        // four rows, which no key bit looks at)
        auto afrag = [&](int i) { return frag(cur, aoff + (i >> 2) * 8192 + (i & 3) * 512); };
        i32x8 af[kAhead + 1], bf[kJ];
        af[0] = afrag(0);
        bf[0] = frag(cur, boff);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 1; j < kJ; ++j) {
            bf[j] = frag(cur, boff + j * 2048);
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (kAhead > 1) af[1] = afrag(1);
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
                    if (t >= kLag) add(t - kLag, f);
                    else add(kT - kLag + t, fp);
                    d[t % kRing] = r;
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < kJ; ++j) fp[j] = f[j];
        publish();
    }
    if constexpr (!EXACT) {
#pragma unroll
        for (int t = kT - kLag; t < kT; ++t) add(t, fp);
    }

    // result lane (li, g) holds, of x row 16 j + li, weight rows 64 (i / 4) + 16 g + 4 (i % 4) + q
    const bool whole = (p.out & 15) == 0 && ((uintptr_t)p.y & 15) == 0;
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
        const int i = wm + 16 * j + li;
        if (m0 + i >= count) continue;
        int64_t yrow = m0 + i;
        if constexpr (GROUPED) yrow = pair_of(i);
#pragma unroll
        for (int h = 0; h < kI / 4; ++h) {
            const int o = n0 + wn + 64 * h + 16 * g;
            if (o >= p.out) continue;
            float v[16];
#pragma unroll
            for (int q = 0; q < 16; ++q) v[q] = acc[4 * h + (q >> 2)][j][q & 3];
            store16<YT>(p.y, yrow * p.out + o, v, whole, p.out - o);
        }
    }
}

// TM x TN tiles by waves of WM x WN
template <int TM, int TN, int WM, int WN, bool EXACT>
void tile_launch(const Fp8Launch& a, hipStream_t s) {
    const TileParams p{a.codes, a.scales, (const uint8_t*)a.x, a.x_scales, a.M, (int)a.out, (int)a.n, a.k, a.x_slots,
                       (int)a.E, a.offsets, a.perm, a.tiles, a.y};
    // (grouped: each expert's last tile may be partial)
    const int64_t tiles = (a.M + TM - 1) / TM + (a.offsets ? std::min<int64_t>(a.E, a.M) : 0);
    const int64_t total = tiles * ((a.out + TN - 1) / TN);
    const dim3 grid((unsigned)((total + 7) / 8 * 8)), block(64 * (TM / WM) * (TN / WN));
    by_float(a.y_dtype, [&](auto yt) {
        constexpr int YT = decltype(yt)::value;
        if constexpr ((YT == IQK_F32) == EXACT) {
            if (a.offsets) hipLaunchKernelGGL((fp8_tile_kernel<TM, TN, WM, WN, YT, true, EXACT>), grid, block, 0, s, p);
            else hipLaunchKernelGGL((fp8_tile_kernel<TM, TN, WM, WN, YT, false, EXACT>), grid, block, 0, s, p);
        }
    });
}

}  // namespace

int fp8_tile_rows(int64_t rows_per_expert, int64_t M, int64_t out, bool exact) {
    if (exact) return 128;
    // 256 x 256 tiles move half the bytes per product that 128 x 128 ones do;
    // they are taken where they fill most of the 256 CUs and most of themselves
    const bool fill = (M + 255) / 256 * ((out + 255) / 256) >= 160;
    return fill && rows_per_expert >= 192 ? 256 : 128;
}

hipError_t launch_fp8_tile(const Fp8Launch& a, int tile, hipStream_t s) {
    if (a.y_dtype == IQK_F32) tile_launch<128, 128, 64, 64, true>(a, s);
    else if (tile == 256) tile_launch<256, 256, 64, 128, false>(a, s);
    else tile_launch<128, 128, 64, 64, false>(a, s);
    return hipGetLastError();
}

}  // namespace iqk
