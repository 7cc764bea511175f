// tiles.h -- device parts shared by the kernels over weights in 16-row tiles
// (the layouts of dg_repack_q4_0_tiles and dg_repack_q8_0_tiles; gemv_tiles.hip
// describes them and the matrix-core arithmetic): the formats, one group's
// loads, its products, and a tile's sums.  Device code only.
#pragma once

#include "glu.h"
#include "mfma_formats.h"

namespace dg {
namespace {   // each source that includes this has its own

using namespace q4;
using namespace mfma;

constexpr int kGroupBlocks = 8;      // blocks per group of a tile
constexpr int kGroupSlots = 18;      // 16-byte slots of one column's Q8_1 blocks per group (8 x 36 / 16)
constexpr uint32_t kHiNib = 0xF0F0F0F0u;

// Tiled weight formats.  A group (16 rows x 8 blocks) is kCodeLoads KiB of
// codes in lane order, then 256 bytes of scales (16 per row); a lane loads
// kCodeLoads + 1 16-byte vectors per group.  bops gives the lane's B operand
// dwords of block i for its low k-slots (activation code dword g) and high
// k-slots (dword 4 + g); kUnscale divides out the factor the integer operands
// and the scale products (4 d8 d4) carry.
struct TilesQ4_0 {
    static constexpr int kCodeLoads = 2;
    static constexpr int kGroupBytes = 2304;     // 16 rows x 8 blocks x 18 bytes
    static constexpr float kUnscale = 1.0f / 64.0f;   // 16 (q - 8) codes, 4 d8 d4
    __device__ __forceinline__ static void bops(const u32x4* w, int i, uint32_t& lo, uint32_t& hi) {
        const u32x4 v = w[i >> 2];
        const uint32_t c = (i & 3) == 0 ? v.x : (i & 3) == 1 ? v.y : (i & 3) == 2 ? v.z : v.w;
        lo = (c << 4) & kHiNib;   // signed nibbles (codes q XOR 8) in the high half of each byte: 16 (q - 8)
        hi = c & kHiNib;
    }
};
struct TilesQ8_0 {
    static constexpr int kCodeLoads = 4;
    static constexpr int kGroupBytes = 4352;     // 16 rows x 8 blocks x 34 bytes
    static constexpr float kUnscale = 1.0f / 4.0f;    // codes as they are, 4 d8 d4
    __device__ __forceinline__ static void bops(const u32x4* w, int i, uint32_t& lo, uint32_t& hi) {
        const u32x4 v = w[i >> 1];
        lo = (i & 1) ? v.z : v.x;
        hi = (i & 1) ? v.w : v.y;
    }
};

// One group of a lane's weights: kCodeLoads 16-byte loads of codes (its B
// operands) and one of its row's eight scales.
template <class TF>
__device__ __forceinline__ void load_group(const uint8_t* __restrict__ g0, int lane, int rn,
                                           u32x4 (&w)[TF::kCodeLoads + 1]) {
#pragma unroll
    for (int c = 0; c < TF::kCodeLoads; ++c)
        w[c] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(g0 + c * 1024 + lane * 16));
    w[TF::kCodeLoads] =
        __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(g0 + TF::kCodeLoads * 1024 + rn * 16));
}

// Column tiles of a launch with MP padded columns: a full tile of 16 columns
// (MP >= 16) and a pair tile of 8 columns from c0 = MP - 8 (MP = 8 or 24).
// The pair tile computes two blocks per matrix-core instruction: a
// v_mfma_i32_16x16x64_i8 (as fast as the 32-deep one on gfx950) whose 64
// k-slots hold both blocks, A rows 0..7 carrying the 8 columns' codes of the
// first block (zeros in the second block's k-slots, read from a zero column
// in LDS) and rows 8..15 those of the second: output row m' is the block sum
// of column c0 + m' % 8 and block i + m' / 8.  Per output that is half the
// instructions of a 16-column tile with eight columns unused.
template <int MP>
struct TileSet {
    static constexpr int kFull = MP >= 16 ? 1 : 0;
    static constexpr int kPair = (MP == 8 || MP == 24) ? 1 : 0;
    // f32x4 accumulators per lane: the full tile's even and odd blocks apart
    // (so that every column is summed in the same order as the pair tile's:
    // even blocks, odd blocks, then the two sums), then the pair tile's
    static constexpr int kNA = 2 * kFull + kPair;
    static constexpr int kPairAcc = 2 * kFull;
    static constexpr int kC0 = MP - 8;          // first column of the pair tile
};

// Per-lane LDS byte offsets of the A operands within the column copy.
struct ALanes {
    uint32_t full;   // the full tile: column rn
    uint32_t p01;    // pair tile, first block's k-slots: column c0 + rn (rn < 8), else the zero column
    uint32_t p23;    // pair tile, second block's k-slots: column c0 + rn - 8 (rn >= 8), else the zero column
    uint32_t ps;     // pair tile, d8: this row's column, one block further for rn >= 8
    uint32_t sel;    // byte selector: that d8 into the low (rn < 8) or high half of a dword
};

// One group of 8 blocks: operands, matrix-core products, fp32 scaling into
// acc, which gathers 1 / TF::kUnscale times the sums (divided out at the
// store):
//  * B (weights), Q4_0: the tiled codes are signed nibbles (q - 8), so
//    masking the high nibbles of a code dword, and of the dword shifted left
//    by 4, gives 16 (q - 8) as int8 for the lane's 8 k-slots: one MFMA per
//    block (per two blocks in the pair tile) gives 16 times the exact block
//    sums (|16 S| < 2^20), with no offset term; Q8_0: the codes as loaded;
//  * the scale products come from one v_mfma_f32_16x16x16_f16 per block (per
//    two blocks in the pair tile) in which B is the lane's raw pair of scale
//    dwords (the d4 of four blocks, one per k-slot, repeated in all four lane
//    groups) and A carries each output row's d8 at the k-slot of its block
//    in every lane group, zeros elsewhere: each output is 4 d8 d4, exact in
//    fp32 (binary16 products are exact, and so are sums of four equal ones).
// blk is the group's first block within the LDS copy of the columns.
template <class TF, int MP>
__device__ __forceinline__ void tiles_group(const u32x4 (&w)[TF::kCodeLoads + 1], const uint8_t* lds,
                                            const ALanes& al, uint32_t blk, int g,
                                            f32x4 (&acc)[TileSet<MP>::kNA]) {
    using TS = TileSet<MP>;
    const u32x4 sv = w[TF::kCodeLoads];
    const f16x4 d4q[2] = {__builtin_bit_cast(f16x4, u32x2{sv.x, sv.y}),    // blocks 0..3
                          __builtin_bit_cast(f16x4, u32x2{sv.z, sv.w})};   // blocks 4..7
    uint32_t blo[8], bhi[8];   // B operand dwords of the lane's low and high k-slots
#pragma unroll
    for (int i = 0; i < kGroupBlocks; ++i) TF::bops(w, i, blo[i], bhi[i]);
    if constexpr (TS::kFull) {
#pragma unroll
        for (int i = 0; i < kGroupBlocks; ++i) {
            const uint32_t* ab = reinterpret_cast<const uint32_t*>(lds + al.full + (blk + i) * kQ81Bytes);
            const long aop = (long)((uint64_t)ab[1 + g] | ((uint64_t)ab[5 + g] << 32));
            const long bop = (long)((uint64_t)blo[i] | ((uint64_t)bhi[i] << 32));
            const uint32_t h = (i & 1) ? ab[0] << 16 : ab[0] & 0xFFFFu;   // d8, in the half of k-slot i % 4
            const f16x4 a8 = __builtin_bit_cast(f16x4, (i & 2) ? u32x2{0u, h} : u32x2{h, 0u});
            const i32x4 dsum = __builtin_amdgcn_mfma_i32_16x16x32_i8(aop, bop, i32x4{0, 0, 0, 0}, 0, 0, 0);
            const f32x4 sc = __builtin_amdgcn_mfma_f32_16x16x16f16(a8, d4q[i >> 2], f32x4{0.0f, 0.0f, 0.0f, 0.0f},
                                                                   0, 0, 0);
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[i & 1][r] = fmaf((float)dsum[r], sc[r], acc[i & 1][r]);
        }
    }
    if constexpr (TS::kPair) {
#pragma unroll
        for (int i = 0; i < kGroupBlocks; i += 2) {
            const uint32_t* x01 = reinterpret_cast<const uint32_t*>(lds + al.p01 + (blk + i) * kQ81Bytes);
            const uint32_t* x23 = reinterpret_cast<const uint32_t*>(lds + al.p23 + (blk + i + 1) * kQ81Bytes);
            const i32x4 aop = {(int)x01[1 + g], (int)x01[5 + g], (int)x23[1 + g], (int)x23[5 + g]};
            const i32x4 bop = {(int)blo[i], (int)bhi[i], (int)blo[i + 1], (int)bhi[i + 1]};
            const uint32_t d8 = *reinterpret_cast<const uint32_t*>(lds + al.ps + (blk + i) * kQ81Bytes);
            const uint32_t h = __builtin_amdgcn_perm(0u, d8, al.sel);   // k-slot i % 4 + (row >= 8)
            const f16x4 a8 = __builtin_bit_cast(f16x4, (i & 2) ? u32x2{0u, h} : u32x2{h, 0u});
            const i32x4 dsum = __builtin_amdgcn_mfma_i32_16x16x64_i8(aop, bop, i32x4{0, 0, 0, 0}, 0, 0, 0);
            const f32x4 sc = __builtin_amdgcn_mfma_f32_16x16x16f16(a8, d4q[i >> 2], f32x4{0.0f, 0.0f, 0.0f, 0.0f},
                                                                   0, 0, 0);
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[TS::kPairAcc][r] = fmaf((float)dsum[r], sc[r], acc[TS::kPairAcc][r]);
        }
    }
}

// Marks a group's registers as written here (an empty asm): arithmetic on
// them cannot move above this point, and its loads are waited for here.
template <int L>
__device__ __forceinline__ void bind_group(u32x4 (&w)[L]) {
    static_assert(L == 3 || L == 5, "three or five loads per group");
    if constexpr (L == 3) asm volatile("" : "+v"(w[0]), "+v"(w[1]), "+v"(w[2])::"memory");
    else asm volatile("" : "+v"(w[0]), "+v"(w[1]), "+v"(w[2]), "+v"(w[3]), "+v"(w[4])::"memory");
}

// A tile's outputs (unscaled) held by a lane, made by all 64 lanes.  The full
// tile adds its even- and odd-block sums; the pair tile's sit in lane groups g
// and g + 2 (output rows m' and m' + 8).
template <class TF, int MP>
struct TileOut {
    using TS = TileSet<MP>;
    float full[TS::kFull ? 4 : 1], pair[TS::kPair ? 4 : 1];
    __device__ __forceinline__ explicit TileOut(const f32x4 (&acc)[TS::kNA]) {
        if constexpr (TS::kFull) {
#pragma unroll
            for (int r = 0; r < 4; ++r) full[r] = (acc[0][r] + acc[1][r]) * TF::kUnscale;
        }
        if constexpr (TS::kPair) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                pair[r] = (acc[TS::kPairAcc][r] + __shfl_xor(acc[TS::kPairAcc][r], 32)) * TF::kUnscale;
        }
    }
    __device__ __forceinline__ void gate(int act, const TileOut& up) {
        if constexpr (TS::kFull) {
#pragma unroll
            for (int r = 0; r < 4; ++r) full[r] = glu(act, full[r], up.full[r]);
        }
        if constexpr (TS::kPair) {
#pragma unroll
            for (int r = 0; r < 4; ++r) pair[r] = glu(act, pair[r], up.pair[r]);
        }
    }
    __device__ __forceinline__ void store(float* __restrict__ Y, int N, int M, int t, int g, int rn) const {
        const int n = t * 16 + rn;
        if (n >= N) return;
        if constexpr (TS::kFull) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int m = g * 4 + r;
                if (m < M) Y[(size_t)m * N + n] = full[r];
            }
        }
        if constexpr (TS::kPair) {
            if (g < 2) {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int m = TS::kC0 + g * 4 + r;
                    if (m < M) Y[(size_t)m * N + n] = pair[r];
                }
            }
        }
    }
};

}  // namespace
}  // namespace dg
