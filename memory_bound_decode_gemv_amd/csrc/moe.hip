// moe.hip -- routed experts: the router's choice per token, and the gated
// feed-forward layer of a few tokens through the experts they were routed to,
// over Q4_0 or Q8_0 weights in 16-row tiles.
//
//   H[m][j] = Q8_1( act(Wg[e] X[m]) (Wu[e] X[m]) ),  e = ids[m][j]
//   Y[m]    = sum_j w[m][j] (Wd[e] H[m][j])
//
// Three launches: the gated products of every (expert, 32 rows) into Q8_1
// columns, the down products of every (expert, row group) into one fp32 column
// per slot (a slot is a token's j-th expert, p = m k + j), and the slots'
// weighted sum in the order of j.
//
// A workgroup finds its own work: it reads the ids (at most 4096), and what
// matches its expert are its columns.  Where there are no more slots than
// experts, workgroups stand for slots and those whose expert has an earlier
// slot leave; otherwise they stand for experts.  No list is built beforehand, so
// no launch is spent on one.
#include <algorithm>
#include <type_traits>

#include "dg_internal.h"
#include "q81_rules.h"
#include "tiles.h"

namespace dg {
namespace {

using namespace tiles;

constexpr int kMaxSlots = 4096;
constexpr int kTileColumns = 16;

// ---------------------------------------------------------------------------
// The router: one wave per token, NV experts per lane (e = lane + 64 i).
//
// An expert's rank is a whole number that orders as its binary32 logit (softmax
// without a bias) or its binary64 score does; 0 is none, which no finite number
// and no infinity but the lowest maps to.  Each of the k choices is a maximum over
// the wave, then the lowest place that holds it.  Scores of softmax ranked by
// their logits are made for the chosen alone, in the lanes that store them; the
// softmax's sum is left out where the weights are divided by their own.
// ---------------------------------------------------------------------------
struct RouteArgs {
    const float* bias;
    int32_t* ids;
    float* weights;
    int64_t M, ld, first;
    int E, k, renorm;
    float scale;
};

constexpr int kRouteRows = 4;   // waves of a workgroup

__device__ __forceinline__ uint32_t rank_bits(float v) {   // -0 as +0
    const uint32_t u = __builtin_bit_cast(uint32_t, v + 0.0f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ uint64_t rank_bits(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v + 0.0);
    return u ^ ((uint64_t)((int64_t)u >> 63) | ((uint64_t)1 << 63));
}
__device__ __forceinline__ float from_rank(uint32_t r) {
    return __builtin_bit_cast(float, r ^ ((r >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {   // lanes without a source give 0
    v = max(v, dpp_mov_u32<kDppRowShr1, 0xF>(v));
    v = max(v, dpp_mov_u32<kDppRowShr2, 0xF>(v));
    v = max(v, dpp_mov_u32<kDppRowShr4, 0xF>(v));
    v = max(v, dpp_mov_u32<kDppRowShr8, 0xF>(v));
    v = max(v, dpp_mov_u32<kDppRowBcast15, 0xA>(v));
    v = max(v, dpp_mov_u32<kDppRowBcast31, 0xC>(v));
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ uint64_t wave_max(uint64_t v) {   // high words, then the low ones beside the highest
    const uint32_t hi = wave_max((uint32_t)(v >> 32));
    const uint32_t lo = wave_max((uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
    return ((uint64_t)hi << 32) | lo;
}

template <int CTRL, int ROW_MASK>
__device__ __forceinline__ double dpp_add_f64(double v) {   // lanes without a source add 0
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = dpp_mov_u32<CTRL, ROW_MASK>((uint32_t)u);
    const uint32_t hi = dpp_mov_u32<CTRL, ROW_MASK>((uint32_t)(u >> 32));
    return v + __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ double readlane_f64(double v, int lane) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, lane);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ double wave_sum_f64(double v) {
    v = dpp_add_f64<kDppRowShr1, 0xF>(v);
    v = dpp_add_f64<kDppRowShr2, 0xF>(v);
    v = dpp_add_f64<kDppRowShr4, 0xF>(v);
    v = dpp_add_f64<kDppRowShr8, 0xF>(v);
    v = dpp_add_f64<kDppRowBcast15, 0xA>(v);
    v = dpp_add_f64<kDppRowBcast31, 0xC>(v);
    return readlane_f64(v, 63);
}

// exp(v - top), 1 at the top itself (which may be infinite).
__device__ __forceinline__ double softmax_term(float v, float top) {
    return v == top ? 1.0 : exp((double)v - (double)top);
}

// BY_LOGIT: softmax without a bias.  SOFTMAX: softmax with one, else sigmoid.
template <class T, int NV, bool BY_LOGIT, bool SOFTMAX>
__global__ void __launch_bounds__(64 * kRouteRows) k_moe_route(const T* __restrict__ x, RouteArgs a) {
    using Rank = typename std::conditional<BY_LOGIT, uint32_t, uint64_t>::type;
    constexpr float kNone = -__builtin_huge_valf();
    const int lane = lane_id();
    const int64_t m = a.first + (int64_t)blockIdx.x * kRouteRows + wave_in_block();
    if (m >= a.M) return;
    float v[NV], bias[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = lane + 64 * i;
        v[i] = e < a.E ? (float)x[m * a.ld + e] : kNone;
        bias[i] = !BY_LOGIT && a.bias && e < a.E ? a.bias[e] : 0.0f;
    }
    Rank key[NV];
    double s[BY_LOGIT ? 1 : NV];
    float top = 0.0f;
    double sum = 1.0;
    if constexpr (BY_LOGIT || SOFTMAX) {
        uint32_t r = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) r = max(r, v[i] > kNone ? rank_bits(v[i]) : 0u);
        r = wave_max(r);
        top = r ? from_rank(r) : 0.0f;
        if (SOFTMAX || !a.renorm) {   // wave-uniform
            sum = 0.0;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const double t = v[i] > kNone ? softmax_term(v[i], top) : 0.0;
                if constexpr (SOFTMAX) s[i] = t;
                sum += t;
            }
            sum = wave_sum_f64(sum);
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if constexpr (BY_LOGIT) {
            key[i] = v[i] > kNone ? rank_bits(v[i]) : 0;
        } else {
            if constexpr (SOFTMAX) s[i] = s[i] / sum;
            else s[i] = 1.0 / (1.0 + exp(-(double)v[i]));
            const double by = s[i] + (double)bias[i];
            key[i] = v[i] > kNone && by > -__builtin_huge_val() ? rank_bits(by) : 0;
        }
    }
    // lane j holds the j-th choice
    int chosen = -1;
    double mine = 0.0;
    float logit = 0.0f;
    for (int j = 0; j < a.k; ++j) {
        Rank best = key[0];
#pragma unroll
        for (int i = 1; i < NV; ++i) best = key[i] > best ? key[i] : best;
        best = wave_max(best);
        if (best == 0) break;   // nothing is left
        bool found = false;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const uint64_t at = __ballot(key[i] == best);
            if (found || at == 0) continue;   // wave-uniform
            found = true;
            const int l = __builtin_ctzll(at);
            if (lane == j) chosen = 64 * i + l;
            if constexpr (!BY_LOGIT) {
                const double t = readlane_f64(s[i], l);
                if (lane == j) mine = t;
            }
            if (lane == l) key[i] = 0;
        }
        if constexpr (BY_LOGIT)
            if (lane == j) logit = from_rank(best);
    }
    if constexpr (BY_LOGIT) mine = chosen >= 0 ? softmax_term(logit, top) / sum : 0.0;
    if (a.renorm) {
        const double total = wave_sum_f64(mine);
        mine = total > 0.0 ? mine / total : 0.0;
    }
    if (lane < a.k) {
        a.ids[m * a.k + lane] = chosen;
        a.weights[m * a.k + lane] = (float)(mine * (double)a.scale);
    }
}

// ---------------------------------------------------------------------------
// The experts' products.
// ---------------------------------------------------------------------------
struct MoeArgs {
    const int32_t* ids;
    int P, E, k;
    int by_slot;      // workgroups stand for slots, not experts
    int rows, K;      // rows of one expert's matrix, columns
    int groups;       // row groups of one expert
    int64_t first;    // the first workgroup of this launch
    int lds_cols;     // LDS bytes for the columns of a pass
};

// The slots routed to the workgroup's expert, in order, into list (by wave 0);
// their number.  Zero where the workgroup has nothing to do.  Every wave comes
// to the same result.
__device__ __forceinline__ int claim(const MoeArgs& a, int item, uint16_t* list, int& e, int lane, int wave) {
    e = a.by_slot ? a.ids[item] : item;
    if (e < 0 || e >= a.E) return 0;
    int cnt = 0;
    for (int p0 = 0; p0 < a.P; p0 += kWave) {
        const int p = p0 + lane;
        const bool hit = p < a.P && a.ids[p] == e;
        const uint64_t mask = __ballot(hit);
        if (a.by_slot && cnt == 0 && mask != 0 && p0 + __builtin_ctzll(mask) < item) return 0;   // an earlier slot's
        if (wave == 0 && hit) list[cnt + __popcll(mask & (((uint64_t)1 << lane) - 1))] = (uint16_t)p;
        cnt += __popcll(mask);
    }
    return cnt;
}

// The tile sums of this wave (its part of K: kw of KW) over M columns of X,
// staged in LDS in passes.  Lane i holds the number of column i; the copies take
// it from there by a shuffle, because the compiler waits for every copy into LDS
// that is under way before it reads LDS.
template <class TF, int MP, int W, int KW, int D>
__device__ __forceinline__ void tile_sums(f32x4 (&acc)[TileSet<MP>::kNA], const uint8_t* tile, const uint8_t* X,
                                          int column, int S, int M, uint8_t* lds, int lds_cols, int lane, int wave,
                                          int kw) {
    using TS = TileSet<MP>;
    constexpr int L = TF::kCodeLoads + 1;
    constexpr int kGroupBytes = TF::kGroupBytes;
    const int g = lane >> 4, rn = lane & 15;
    // groups of a pass: whole rounds of every wave where the row does not fit at once
    int spp = ((lds_cols - 1024) / (16 * (M + 1)) - 1) / kGroupSlots;
    if (spp < S) {
        constexpr int kRound = KW * D;
        const int passes = (S + spp - 1) / spp;
        const int even = (S + passes - 1) / passes;
        const int round = (even + kRound - 1) / kRound * kRound;
        spp = round <= spp ? round : even;
    } else {
        spp = S;
    }
    const int cs_slots = kGroupSlots * spp + 1;
    const uint32_t magic = 0xFFFFFFFFu / (uint32_t)cs_slots + 1u;   // ceil(2^32 / stride): the stride is odd
    const int copies = (M * cs_slots + kWave - 1) / kWave;
    ALanes al;
    {
        const uint32_t stride = (uint32_t)cs_slots * 16u;
        const uint32_t zero = (uint32_t)copies * 1024u;
        al.full = (uint32_t)(rn < M ? rn : M - 1) * stride;
        const int c = TS::kC0 + (rn & 7);
        const uint32_t pc = (uint32_t)(c < M ? c : M - 1) * stride;
        const bool hi = rn >= 8;
        al.p01 = hi ? zero : pc;
        al.p23 = hi ? pc : zero;
        al.ps = pc + (hi ? (uint32_t)kQ81Bytes : 0u);
        al.sel = hi ? 0x01000C0Cu : 0x0C0C0100u;
    }
    if constexpr (TS::kPair) {
        u32x4* const z = reinterpret_cast<u32x4*>(lds + copies * 1024);
        for (int e = wave * kWave + lane; e < cs_slots; e += W * kWave) z[e] = u32x4{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int a = 0; a < TS::kNA; ++a) acc[a] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    for (int p0 = 0; p0 < S; p0 += spp) {
        const int np = min(spp, S - p0);
        // Wave kw takes the groups kw, kw + KW, ... of the whole row, so that its
        // order of sums does not depend on where passes end, and so not on M.
        const int w0 = ((kw - p0) % KW + KW) % KW;   // its first group of the pass
        const int cnt = max(0, (np - w0 + KW - 1) / KW);
        const uint8_t* const wbase = tile + (size_t)(p0 + (cnt > 0 ? w0 : 0)) * kGroupBytes;
        const int last = cnt > 0 ? cnt - 1 : 0;
        constexpr int kStep = KW * kGroupBytes;
        if (p0 > 0) lds_barrier();   // every wave is done with the columns of the pass before
        {
            const int used = np * kGroupSlots;
            const uint8_t* const xr = X + (size_t)p0 * kGroupBlocks * kQ81Bytes;
            for (int j = wave; j < copies; j += W) {
                const uint32_t q = (uint32_t)(j * kWave + lane);
                const uint32_t m = __umulhi(q, magic);
                const uint32_t c = q - m * (uint32_t)cs_slots;
                const bool ok = m < (uint32_t)M && c < (uint32_t)used;
                const size_t at = (size_t)__shfl(column, ok ? (int)m : 0) * ((size_t)S * kGroupSlots * 16);
                const uint8_t* src = xr + at + (ok ? (size_t)c * 16 : 0);
                __builtin_amdgcn_global_load_lds(src, (lds_void_t*)(lds + j * 1024), 16, 0, 0);
            }
        }
        __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0): the copies only
        lds_barrier();                        // every other wave's copies have landed too
        u32x4 wb[D][L];
#pragma unroll
        for (int d = 0; d < D; ++d)
            load_group<TF>(wbase + (size_t)(d < cnt ? d : last) * kStep, lane, rn, wb[d]);
        const int rounds = (cnt + D - 1) / D;
        for (int rd = 0; rd + 1 < rounds; ++rd) {
#pragma unroll
            for (int d = 0; d < D; ++d) {
                const int i = rd * D + d;
                tiles_group<TF, MP>(wb[d], lds, al, (uint32_t)(w0 + i * KW) * kGroupBlocks, g, acc);
                const int nx = i + D;
                load_group<TF>(wbase + (size_t)(nx < cnt ? nx : last) * kStep, lane, rn, wb[d]);
                bind_group(wb[(d + 1) % D]);
            }
        }
        if (rounds > 0) {
#pragma unroll
            for (int d = 0; d < D; ++d) {
                const int i = (rounds - 1) * D + d;
                if (d > 0) bind_group(wb[d]);
                if (i < cnt) tiles_group<TF, MP>(wb[d], lds, al, (uint32_t)(w0 + i * KW) * kGroupBlocks, g, acc);
            }
        }
    }
    lds_barrier();   // every wave is done with the columns
}

// The KW parts of each tile, added in the order 0..KW-1 by the waves with kw = 0.
template <int NA, int KW>
__device__ __forceinline__ void join_parts(f32x4 (&acc)[NA], f32x4* red, int lane, int wave, int kw) {
    if constexpr (KW > 1) {
        if (kw > 0) {
#pragma unroll
            for (int a = 0; a < NA; ++a) red[(wave * NA + a) * kWave + lane] = acc[a];
        }
        lds_barrier();
        if (kw == 0) {
            for (int k2 = 1; k2 < KW; ++k2)
#pragma unroll
                for (int a = 0; a < NA; ++a) {
                    const f32x4 v = red[((wave + k2) * NA + a) * kWave + lane];
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[a][r] += v[r];
                }
        }
    }
}

// f(column, value) for each output of a lane's tile row.
template <class TF, int MP, class F>
__device__ __forceinline__ void each_output(const TileOut<TF, MP>& o, int M, int g, F f) {
    if constexpr (TileSet<MP>::kFull) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (g * 4 + r < M) f(g * 4 + r, o.full[r]);
    } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (g < 2 && g * 4 + r < M) f(g * 4 + r, o.pair[r]);
    }
}

// Gate and up products of 32 rows of one expert and M of its columns, then
// their Q8_1 blocks.
template <class TF, int MP, int KW, int D>
__device__ __forceinline__ void glu_columns(const MoeArgs& a, const uint8_t* Wg, const uint8_t* Wu,
                                            const uint8_t* Xq, uint8_t* Hq, int act, int e, int grp, int M,
                                            const uint16_t* list, uint8_t* lds, int lane, int wave) {
    constexpr int RT = 4, W = RT * KW, NA = TileSet<MP>::kNA;
    const int rt = wave / KW, kw = wave - rt * KW;
    const bool up = rt & 1;
    const int S = a.K >> 8;
    const size_t t = (size_t)e * (a.rows >> 4) + (size_t)grp * 2 + (rt >> 1);
    const uint8_t* const tile = (up ? Wu : Wg) + t * S * TF::kGroupBytes;
    f32x4 acc[NA];
    const int slot = list[min(lane, M - 1)];
    tile_sums<TF, MP, W, KW, D>(acc, tile, Xq, (int)((unsigned)slot / (unsigned)a.k), S, M, lds, a.lds_cols, lane, wave,
                                kw);
    f32x4* const red = reinterpret_cast<f32x4*>(lds);
    join_parts<NA, KW>(acc, red, lane, wave, kw);
    if (kw == 0 && up) {
#pragma unroll
        for (int i = 0; i < NA; ++i) red[(wave * NA + i) * kWave + lane] = acc[i];
    }
    lds_barrier();
    float* const h = reinterpret_cast<float*>(lds + W * NA * 1024);   // [column][32 rows]
    if (kw == 0 && !up) {
        f32x4 us[NA];
#pragma unroll
        for (int i = 0; i < NA; ++i) us[i] = red[((wave + KW) * NA + i) * kWave + lane];
        TileOut<TF, MP> out(acc);
        out.gate(act, TileOut<TF, MP>(us));
        each_output<TF, MP>(out, M, lane >> 4, [&](int m, float v) { h[m * 32 + (rt >> 1) * 16 + (lane & 15)] = v; });
    }
    lds_barrier();
    // one Q8_1 block per half wave
    for (int v = wave * kWave + lane; v < M * 32; v += W * kWave) {
        const int m = v >> 5, j = v & 31;
        const float f = h[v];
        float amax = fabsf(f);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) amax = fmaxf(amax, __shfl_xor(amax, d));
        const float d8 = q81_scale(amax);
        const int c = q81_code(f, d8);
        int sum = c;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) sum += __shfl_xor(sum, d);
        uint32_t w = (uint32_t)(uint8_t)(int8_t)c << (8 * (j & 3));
        w |= __shfl_xor(w, 1);
        w |= __shfl_xor(w, 2);
        uint32_t* const block =
            reinterpret_cast<uint32_t*>(Hq + ((size_t)list[m] * (a.rows >> 5) + (size_t)grp) * kQ81Bytes);
        if ((j & 3) == 0) block[1 + (j >> 2)] = w;
        if (j == 0) block[0] = q81_header(d8, sum);
    }
}

template <class TF, int KW, int D>
__global__ void __launch_bounds__(64 * 4 * KW)
k_moe_glu(const uint8_t* __restrict__ Wg, const uint8_t* __restrict__ Wu, const uint8_t* __restrict__ Xq,
          uint8_t* __restrict__ Hq, int act, MoeArgs a) {
    extern __shared__ u32x4 moe_lds[];
    uint8_t* const lds = reinterpret_cast<uint8_t*>(moe_lds);
    uint16_t* const list = reinterpret_cast<uint16_t*>(lds + a.lds_cols);
    const int lane = lane_id(), wave = wave_in_block();
    const int64_t b = a.first + blockIdx.x;
    const int item = (int)(b / a.groups);
    int e;
    const int cnt = claim(a, item, list, e, lane, wave);
    if (cnt == 0) return;   // workgroup-uniform, before any barrier
    const int grp = (int)(b - (int64_t)item * a.groups);
    lds_barrier();          // the list is written
    for (int c0 = 0; c0 < cnt; c0 += kTileColumns) {
        const int M = min(kTileColumns, cnt - c0);
        if (c0 > 0) lds_barrier();
        if (M <= 8) glu_columns<TF, 8, KW, D>(a, Wg, Wu, Xq, Hq, act, e, grp, M, list + c0, lds, lane, wave);
        else glu_columns<TF, 16, KW, D>(a, Wg, Wu, Xq, Hq, act, e, grp, M, list + c0, lds, lane, wave);
    }
}

template <class TF, int MP, int RT, int KW, int D>
__device__ __forceinline__ void down_columns(const MoeArgs& a, const uint8_t* Wd, const uint8_t* Hq, float* part,
                                             int e, int grp, int M, const uint16_t* list, uint8_t* lds, int lane,
                                             int wave) {
    constexpr int W = RT * KW, NA = TileSet<MP>::kNA;
    const int rt = wave / KW, kw = wave - rt * KW;
    const int S = a.K >> 8;
    const int t = grp * RT + rt;
    const uint8_t* const tile = Wd + ((size_t)e * (a.rows >> 4) + t) * S * TF::kGroupBytes;
    f32x4 acc[NA];
    tile_sums<TF, MP, W, KW, D>(acc, tile, Hq, list[min(lane, M - 1)], S, M, lds, a.lds_cols, lane, wave, kw);
    join_parts<NA, KW>(acc, reinterpret_cast<f32x4*>(lds), lane, wave, kw);
    if (kw == 0) {
        const TileOut<TF, MP> out(acc);
        const int n = t * 16 + (lane & 15);
        each_output<TF, MP>(out, M, lane >> 4, [&](int m, float v) { part[(size_t)list[m] * a.rows + n] = v; });
    }
}

template <class TF, int RT, int KW, int D>
__global__ void __launch_bounds__(64 * RT * KW)
k_moe_down(const uint8_t* __restrict__ Wd, const uint8_t* __restrict__ Hq, float* __restrict__ part, MoeArgs a) {
    extern __shared__ u32x4 moe_lds[];
    uint8_t* const lds = reinterpret_cast<uint8_t*>(moe_lds);
    uint16_t* const list = reinterpret_cast<uint16_t*>(lds + a.lds_cols);
    const int lane = lane_id(), wave = wave_in_block();
    const int64_t b = a.first + blockIdx.x;
    const int item = (int)(b / a.groups);
    int e;
    const int cnt = claim(a, item, list, e, lane, wave);
    if (cnt == 0) return;   // workgroup-uniform, before any barrier
    const int grp = (int)(b - (int64_t)item * a.groups);
    lds_barrier();          // the list is written
    for (int c0 = 0; c0 < cnt; c0 += kTileColumns) {
        const int M = min(kTileColumns, cnt - c0);
        if (c0 > 0) lds_barrier();
        if (M <= 8) down_columns<TF, 8, RT, KW, D>(a, Wd, Hq, part, e, grp, M, list + c0, lds, lane, wave);
        else down_columns<TF, 16, RT, KW, D>(a, Wd, Hq, part, e, grp, M, list + c0, lds, lane, wave);
    }
}

// Y[m][n] = sum_j w[m][j] part[m k + j][n], in the order of j; four n a thread.
template <class T>
__global__ void __launch_bounds__(256)
k_moe_sum(const float* __restrict__ part, const int32_t* __restrict__ ids, const float* __restrict__ weights,
          T* __restrict__ Y, int K, int E, int k) {
#pragma clang fp contract(off)
    const int n = (int)(blockIdx.x * blockDim.x + threadIdx.x) * 4;
    const int m = blockIdx.y;
    if (n >= K) return;
    float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int j = 0; j < k; ++j) {
        const int p = m * k + j;
        const int e = ids[p];
        if (e < 0 || e >= E) continue;
        const float w = weights[p];
        const float4 v = *reinterpret_cast<const float4*>(part + (size_t)p * K + n);
        y[0] += w * v.x;
        y[1] += w * v.y;
        y[2] += w * v.z;
        y[3] += w * v.w;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) Y[(size_t)m * K + n + i] = (T)bind_f32(y[i]);
}

template <class T, int NV>
void route_launch(const MoeRoute& r, const RouteArgs& a, int64_t rows, hipStream_t s) {
    const bool softmax = r.score == DG_ROUTE_SOFTMAX;
    const auto kernel = softmax && !r.bias ? k_moe_route<T, NV, true, false>
                        : softmax          ? k_moe_route<T, NV, false, true>
                                           : k_moe_route<T, NV, false, false>;
    hipLaunchKernelGGL(kernel, dim3((unsigned)((rows + kRouteRows - 1) / kRouteRows)), dim3(64 * kRouteRows), 0, s,
                       (const T*)r.x, a);
}

template <class T>
hipError_t route_dtype(const MoeRoute& r, hipStream_t s) {
    RouteArgs a{r.bias, r.ids, r.weights, r.M, r.ld, 0, (int)r.E, r.k, r.renorm, r.scale};
    hipError_t e = hipSuccess;
    for (; a.first < r.M && e == hipSuccess; a.first += kMaxGroupsPerLaunch * kRouteRows) {
        const int64_t rows = std::min<int64_t>(r.M - a.first, kMaxGroupsPerLaunch * kRouteRows);
        if (r.E <= 64) route_launch<T, 1>(r, a, rows, s);
        else if (r.E <= 128) route_launch<T, 2>(r, a, rows, s);
        else if (r.E <= 256) route_launch<T, 4>(r, a, rows, s);
        else if (r.E <= 512) route_launch<T, 8>(r, a, rows, s);
        else route_launch<T, 16>(r, a, rows, s);
        e = hipGetLastError();
    }
    return e;
}

// One kernel over (items, row groups), in launches of what one takes.
template <class F>
hipError_t over_groups(int64_t items, MoeArgs& a, F launch) {
    const int64_t all = items * a.groups;
    hipError_t e = hipSuccess;
    for (a.first = 0; a.first < all && e == hipSuccess; a.first += kMaxGroupsPerLaunch) {
        launch((unsigned)std::min<int64_t>(all - a.first, kMaxGroupsPerLaunch));
        e = hipGetLastError();
    }
    return e;
}

template <class TF>
hipError_t moe_layer(const MoeLayer& q, hipStream_t s) {
    const int P = (int)(q.M * q.k);
    uint8_t* const Hq = (uint8_t*)q.ws;
    float* const part = (float*)(Hq + (size_t)P * (q.N / 32) * kQ81Bytes);
    MoeArgs a{};
    a.ids = q.ids;
    a.P = P;
    a.E = (int)q.E;
    a.k = q.k;
    a.by_slot = P <= q.E;
    const int64_t items = std::min<int64_t>(P, q.E);
    a.lds_cols = 64 * 1024;
    const size_t lds = a.lds_cols + (size_t)P * 2;

    constexpr int KW = 2, D = 2;
    a.rows = (int)q.N;
    a.K = (int)q.K;
    a.groups = (int)(q.N / 32);
    hipError_t e = over_groups(items, a, [&](unsigned grid) {
        hipLaunchKernelGGL((k_moe_glu<TF, KW, D>), dim3(grid), dim3(64 * 4 * KW), lds, s, (const uint8_t*)q.Wg,
                           (const uint8_t*)q.Wu, (const uint8_t*)q.Xq, Hq, q.act, a);
    });
    if (e != hipSuccess) return e;
    a.rows = (int)q.K;
    a.K = (int)q.N;
    constexpr int RT = 4;
    a.groups = (int)(q.K / 16 / RT);
    e = over_groups(items, a, [&](unsigned grid) {
        hipLaunchKernelGGL((k_moe_down<TF, RT, KW, D>), dim3(grid), dim3(64 * RT * KW), lds, s, (const uint8_t*)q.Wd,
                           Hq, part, a);
    });
    return e;
}

template <class T>
hipError_t moe_sum(const MoeLayer& q, hipStream_t s) {
    const int P = (int)(q.M * q.k);
    const float* const part = (const float*)((const uint8_t*)q.ws + (size_t)P * (q.N / 32) * kQ81Bytes);
    hipLaunchKernelGGL((k_moe_sum<T>), dim3((unsigned)((q.K / 4 + 255) / 256), (unsigned)q.M), dim3(256), 0, s, part,
                       q.ids, q.weights, (T*)q.Y, (int)q.K, (int)q.E, q.k);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_moe_route(const MoeRoute& r, hipStream_t s) {
    if (r.dtype == DG_DTYPE_F32) return route_dtype<float>(r, s);
    if (r.dtype == DG_DTYPE_F16) return route_dtype<_Float16>(r, s);
    return route_dtype<__bf16>(r, s);
}

size_t moe_workspace_bytes(int64_t N, int64_t K, int64_t M, int k) {
    return (size_t)(M * k) * ((size_t)(N / 32) * kQ81Bytes + (size_t)K * 4);
}

hipError_t launch_moe(const MoeLayer& layer, hipStream_t s) {
    MoeLayer q = layer;
    if (q.N == 0) q.k = 0;   // empty products: sums of no slots
    hipError_t e = q.k == 0 ? hipSuccess : q.q8 ? moe_layer<TilesQ8_0>(q, s) : moe_layer<TilesQ4_0>(q, s);
    if (e != hipSuccess) return e;
    if (q.ydtype == DG_DTYPE_F32) return moe_sum<float>(q, s);
    if (q.ydtype == DG_DTYPE_F16) return moe_sum<_Float16>(q, s);
    return moe_sum<__bf16>(q, s);
}

}  // namespace dg
