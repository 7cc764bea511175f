// moe.hip -- routed experts: the router's choice per token, and the gated
// feed-forward layer of a few tokens through the experts they were routed to,
// over Q4_0 or Q8_0 weights in 16-row tiles.
//
//   H[m][j] = Q8_1( act(Wg[e] X[m]) (Wu[e] X[m]) ),  e = ids[m][j]
//   Y[m]    = sum_j w[m][j] (Wd[e] H[m][j])
//
// Three launches: the gated products of every (expert, 32 or 64 rows) into Q8_1
// columns, the down products of every (expert, row group) into one fp32 column
// per slot (a slot is a token's j-th expert, p = m k + j), and the slots'
// weighted sum in the order of j; for a few tokens the last two are one.
//
// The weights of the chosen experts are nearly all that is read, so large experts
// are bound by HBM: 32 tokens through 2 of 8 Q8_0 experts of 14336 x 4096 (1.5 GB)
// 150 + 76 + 4 us, 6.7 TB/s; one token through Q4_0 ones 24.2 + 16.5, 5.4 and 4.0
// TB/s, the down products held up by the copies of the hidden columns before them
// (k_moe_down_tokens).  Small experts are bound by the dependent steps of each launch:
// one token through 8 of 128 of 768 x 2048 8.6 + 5.1 us for 21 MB, in which a wave has
// two of its row's eight weight groups in flight, so four round trips to memory beside
// those of the ids, and two of three in the down products.  Between them 24 tokens
// through 6 of 64 of 1536 x 2048 35 + 19 + 4, 5.4 TB/s.  Many tokens: a workgroup looks
// through all slots, 128 a round trip, before its first weights, and an expert's weights
// are read again for every 16 of its tokens (200 tokens through 8 of 128 of 768 x 2048
// 132 us, 340 MB).
//
// A workgroup finds its own work: it reads the ids (at most 4096), and what
// matches its expert are its columns.  Where there are no more slots than
// experts, workgroups stand for slots and those whose expert has an earlier
// slot leave; otherwise they stand for experts.  No list is built beforehand, so
// no launch is spent on one.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "dg_batch.h"
#include "q81_rules.h"
#include "tiles.h"

namespace dg {
namespace {

// At most 128 registers a wave: 16 waves to a CU.  Left alone the compiler takes a
// few more for some shapes, and half the waves no longer fit (24 tokens through 64
// experts of 1536 x 2048: 98 us against 79); held to 96 it spills (32 tokens
// through 8 of 14336 x 4096, Q8_0: 250 against 230).
#define MOE_WAVES __attribute__((amdgpu_waves_per_eu(4, 8)))
constexpr int kTileColumns = 16;

// ---------------------------------------------------------------------------
// The router: one wave per token, NV experts per lane (e = lane + 64 i).
//
// An expert's rank is a whole number that orders as its binary32 logit (softmax
// without a bias) or its binary64 score does; 0 is none, which no finite number
// and no infinity but the lowest maps to.  Each of the k choices is a maximum over
// the wave, then the lowest place that holds it.  Scores of softmax ranked by
// their logits are made for the chosen alone, in the lanes that store them; the
// softmax's sum is left out where the weights are divided by their own.  One token
// of 64 experts, k 6: 2.6 us, the launch and the choices one after another; 4096 of
// 256, k 8, with a sigmoid and a bias 8.1, of which some 600 vector instructions a
// wave are issued in half the busy cycles.  The rest is waiting, for the lane moves of
// the choices (two whole maxima for a 64-bit rank) and for the loads: as compiled, a
// 16-bit logit, and a logit with its bias, is waited for before the next is asked for
// (NV trips, 2 NV for 16 bits with a bias); only binary32 logits of softmax without a
// bias are on their way together.  Ranks sorted in each lane first, so that a
// choice looks at one a lane: 8.6, and 78 against 11 for 1024 experts.
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
    int run, runs;    // row groups of a workgroup, workgroups of an expert
    int64_t first;    // the first workgroup of this launch
    int lds_cols;     // LDS bytes for the columns of a pass
    int lds_sums;     // and for the sums and hidden values that meet there
};

// The slots routed to the workgroup's expert, in order, into list (by wave 0);
// their number.  Zero where the workgroup has nothing to do.  Every wave comes
// to the same result.
__device__ __forceinline__ int claim(const MoeArgs& a, int item, uint16_t* list, int& e, int lane, int wave) {
    // Runs of 64 slots on their way together.  1, 2 and 4: 200 tokens through 8 of 128 experts 138.4, 132.6,
    // 129.9 us, 24 through 6 of 64 56.8, 56.7, 56.6, one through 2 of 8 40.6, 40.8, 41.0.
    constexpr int U = 2;
    int id[U];
    auto load = [&](int p0) {
#pragma unroll
        for (int u = 0; u < U; ++u) id[u] = a.ids[min(p0 + u * kWave + lane, a.P - 1)];
    };
    load(0);
    e = a.by_slot ? a.ids[item] : item;
    if (e < 0 || e >= a.E) return 0;
    int cnt = 0;
    for (int p0 = 0;;) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int p = p0 + u * kWave + lane;
            const bool hit = p < a.P && id[u] == e;
            const uint64_t mask = __ballot(hit);
            if (a.by_slot && cnt == 0 && mask != 0 && p0 + u * kWave + __builtin_ctzll(mask) < item) return 0;   // an earlier slot's
            if (wave == 0 && hit) list[cnt + __popcll(mask & (((uint64_t)1 << lane) - 1))] = (uint16_t)p;
            cnt += __popcll(mask);
        }
        p0 += U * kWave;
        if (p0 >= a.P) return cnt;
        load(p0);
    }
}

// Where a lane's A operands lie: M columns in LDS from `column` on, `stride`
// bytes apart, a column of zeros at `zero`.  Columns past M: the last again, their
// results dropped.
template <int MP>
__device__ __forceinline__ ALanes a_lanes(uint32_t column, uint32_t stride, uint32_t zero, int M, int rn) {
    ALanes al;
    al.full = column + (uint32_t)min(rn, M - 1) * stride;
    const uint32_t pc = column + (uint32_t)min(TileSet<MP>::kC0 + (rn & 7), M - 1) * stride;
    const bool hi = rn >= 8;
    al.p01 = hi ? zero : pc;
    al.p23 = hi ? pc : zero;
    al.ps = pc + (hi ? (uint32_t)kQ81Bytes : 0u);
    al.sel = hi ? 0x01000C0Cu : 0x0C0C0100u;
    return al;
}

// A wave's groups of a tile, `step` bytes apart, D of them in flight.
template <class TF, int D>
struct Stream {
    u32x4 wb[D][TF::kCodeLoads + 1];
    const uint8_t* base;
    int cnt, last, step;
    __device__ __forceinline__ void load(int d, int i, int lane) {
        load_group<TF>(base + (size_t)(i < cnt ? i : last) * step, lane, lane & 15, wb[d]);
    }
    __device__ __forceinline__ Stream(const uint8_t* b, int n, int st, int lane)
        : cnt(n), last(n > 0 ? n - 1 : 0), step(st) {
        start(b, lane);
    }
    __device__ __forceinline__ void start(const uint8_t* b, int lane) {
        base = b;
#pragma unroll
        for (int d = 0; d < D; ++d) load(d, d, lane);
    }
    // The products, group i against the blocks (first + i every) * 8 of the columns in LDS.
    template <int MP>
    __device__ __forceinline__ void products(f32x4 (&acc)[TileSet<MP>::kNA], const uint8_t* lds, const ALanes& al,
                                             int first, int every, int lane) {
        const int g = lane >> 4;
        const int rounds = (cnt + D - 1) / D;
        for (int rd = 0; rd + 1 < rounds; ++rd) {
#pragma unroll
            for (int d = 0; d < D; ++d) {
                const int i = rd * D + d;
                tiles_group<TF, MP>(wb[d], lds, al, (uint32_t)(first + i * every) * kGroupBlocks, g, acc);
                load(d, i + D, lane);
                bind_group(wb[(d + 1) % D]);
            }
        }
        if (rounds > 0) {
#pragma unroll
            for (int d = 0; d < D; ++d) {
                const int i = (rounds - 1) * D + d;
                if (d > 0) bind_group(wb[d]);
                if (i < cnt) tiles_group<TF, MP>(wb[d], lds, al, (uint32_t)(first + i * every) * kGroupBlocks, g, acc);
            }
        }
    }
};

template <int NA>
__device__ __forceinline__ void clear(f32x4 (&acc)[NA]) {
#pragma unroll
    for (int a = 0; a < NA; ++a) acc[a] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
}

// The sums of this wave (its part of K: kw of KW) of `run` tiles, one after the
// other, over M columns of X that are staged in LDS: once where whole rows fit, in
// passes over K for every tile where not.  tile(r): the r-th tile's address;
// out(r, acc): what is done with its sums (not in the columns' LDS).
//
// Lane i holds the number of column i; the copies take it from there by a
// shuffle, because the compiler waits for every copy into LDS that is under way
// before it reads LDS.
template <class TF, int MP, bool RUNS, int W, int KW, int D, class Tile, class Out>
__device__ __forceinline__ void each_tile(int run, Tile tile, const uint8_t* X, int column, int S, int M, uint8_t* lds,
                                          int lds_cols, int lane, int wave, int kw, Out out) {
    using TS = TileSet<MP>;
    constexpr int kGroupBytes = TF::kGroupBytes;
    int spp = ((lds_cols - 1024) / (16 * (M + 1)) - 1) / kGroupSlots;   // groups of a pass
    if (spp < S) {   // whole rounds of every wave
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
    const ALanes al = a_lanes<MP>(0, (uint32_t)cs_slots * 16u, (uint32_t)copies * 1024u, M, lane & 15);
    if constexpr (TS::kPair) {
        u32x4* const z = reinterpret_cast<u32x4*>(lds + copies * 1024);
        for (int e = wave * kWave + lane; e < cs_slots; e += W * kWave) z[e] = u32x4{0u, 0u, 0u, 0u};
    }
    auto stage = [&](int p0, int np) {
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
        __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0)
        lds_barrier();                        // every other wave's copies have landed too
    };
    f32x4 acc[TS::kNA];
    // A tile's first weights go out before the copies, which then take no round
    // trip of their own, or before the epilogue of the tile before it.
    if (RUNS && spp == S) {
        const int cnt = max(0, (S - kw + KW - 1) / KW);
        const int first = cnt > 0 ? kw * kGroupBytes : 0;
        Stream<TF, D> weights(tile(0) + first, cnt, KW * kGroupBytes, lane);
        stage(0, S);
        for (int r = 0; r < run; ++r) {
            clear(acc);
            weights.template products<MP>(acc, lds, al, kw, KW, lane);
            if (r + 1 < run) weights.start(tile(r + 1) + first, lane);
            out(r, acc);
        }
        return;
    }
    for (int r = 0; r < (RUNS ? run : 1); ++r) {
        clear(acc);
        for (int p0 = 0; p0 < S; p0 += spp) {
            const int np = min(spp, S - p0);
            // Wave kw takes the groups kw, kw + KW, ... of the whole row, so that its
            // order of sums does not depend on where passes end, and so not on M.
            const int w0 = ((kw - p0) % KW + KW) % KW;   // its first group of the pass
            const int cnt = max(0, (np - w0 + KW - 1) / KW);
            Stream<TF, D> weights(tile(r) + (size_t)(p0 + (cnt > 0 ? w0 : 0)) * kGroupBytes, cnt, KW * kGroupBytes, lane);
            if (r + p0 > 0) lds_barrier();   // every wave is done with the columns of the pass before
            stage(p0, np);
            weights.template products<MP>(acc, lds, al, w0, KW, lane);
        }
        out(r, acc);
    }
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

// Gate and up products of `run` groups of 8 RT rows of one expert and M of its
// columns, then their Q8_1 blocks.  Waves: one for each of the RT tiles, the gate's
// and the up matrix's in turn, with the whole K.
template <class TF, int MP, bool RUNS, int RT, int D>
__device__ __forceinline__ void glu_columns(const MoeArgs& a, const uint8_t* Wg, const uint8_t* Wu,
                                            const uint8_t* Xq, uint8_t* Hq, int act, int e, int grp, int run, int M,
                                            const uint16_t* list, uint8_t* lds, int lane, int wave) {
    static_assert(RT % 4 == 0, "whole Q8_1 blocks");
    constexpr int NA = TileSet<MP>::kNA, kRows = RT * 8;
    const bool up = wave & 1;
    const int S = a.K >> 8;
    const uint8_t* const tiles = (up ? Wu : Wg) +
                                 ((size_t)e * (a.rows >> 4) + (size_t)grp * (RT / 2) + (wave >> 1)) * S * TF::kGroupBytes;
    f32x4* const red = reinterpret_cast<f32x4*>(lds + a.lds_cols);            // the up sums
    float* const h = reinterpret_cast<float*>(lds + a.lds_cols + RT / 2 * NA * 1024);   // [column][rows]
    const int slot = list[min(lane, M - 1)];
    each_tile<TF, MP, RUNS, RT, 1, D>(
        run, [&](int r) { return tiles + (size_t)r * (RT / 2) * S * TF::kGroupBytes; }, Xq,
        (int)((unsigned)slot / (unsigned)a.k), S, M, lds, a.lds_cols, lane, wave, 0, [&](int r, f32x4(&acc)[NA]) {
            f32x4* const mine = red + (wave >> 1) * NA * kWave + lane;
            if (up) {
#pragma unroll
                for (int i = 0; i < NA; ++i) mine[i * kWave] = acc[i];
            }
            lds_barrier();
            if (!up) {
                f32x4 us[NA];
#pragma unroll
                for (int i = 0; i < NA; ++i) us[i] = mine[i * kWave];
                TileOut<TF, MP> o(acc);
                o.gate(act, TileOut<TF, MP>(us));
                each_output<TF, MP>(o, M, lane >> 4,
                                    [&](int m, float v) { h[m * kRows + (wave >> 1) * 16 + (lane & 15)] = v; });
            }
            lds_barrier();
            // one Q8_1 block per half wave
            for (int v = wave * kWave + lane; v < M * kRows; v += RT * kWave) {
                const int m = v / kRows, b = v % kRows >> 5, j = v & 31;
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
                uint32_t* const block = reinterpret_cast<uint32_t*>(
                    Hq + ((size_t)list[m] * (a.rows >> 5) + (size_t)(grp + r) * (RT / 4) + b) * kQ81Bytes);
                if ((j & 3) == 0) block[1 + (j >> 2)] = w;
                if (j == 0) block[0] = q81_header(d8, sum);
            }
        });
}

// The down products of `run` groups of RT row tiles of one expert and M of its
// columns, each in KW parts of K, into the slots' partial columns.
template <class TF, int MP, bool RUNS, int RT, int KW, int D>
__device__ __forceinline__ void down_columns(const MoeArgs& a, const uint8_t* Wd, const uint8_t* Hq, float* part,
                                             int e, int grp, int run, int M, const uint16_t* list, uint8_t* lds,
                                             int lane, int wave) {
    static_assert(!RUNS || KW == 1, "parts that meet in LDS leave it after one row group");
    constexpr int W = RT * KW, NA = TileSet<MP>::kNA;
    const int rt = wave / KW, kw = wave - rt * KW;
    const int S = a.K >> 8;
    const int t = grp * RT + rt;
    const uint8_t* const tiles = Wd + ((size_t)e * (a.rows >> 4) + t) * S * TF::kGroupBytes;
    each_tile<TF, MP, RUNS, W, KW, D>(
        run, [&](int r) { return tiles + (size_t)r * RT * S * TF::kGroupBytes; }, Hq, list[min(lane, M - 1)], S, M, lds,
        a.lds_cols, lane, wave, kw, [&](int r, f32x4(&acc)[NA]) {
            join_parts<NA, KW>(acc, reinterpret_cast<f32x4*>(lds + a.lds_cols), lane, wave, kw);
            if (kw > 0) return;
            const TileOut<TF, MP> o(acc);
            const int n = (t + r * RT) * 16 + (lane & 15);
            each_output<TF, MP>(o, M, lane >> 4, [&](int m, float v) { part[(size_t)list[m] * a.rows + n] = v; });
        });
}

// What both kernels do: find the workgroup's expert and columns, and take them
// 16 (8) at a time.  f(mp, e, first row group, row groups, M, list)
template <bool MANY, class F>
__device__ __forceinline__ void each_columns(const MoeArgs& a, uint8_t* lds, F f) {
    uint16_t* const list = reinterpret_cast<uint16_t*>(lds + a.lds_cols + a.lds_sums);
    const int64_t b = a.first + blockIdx.x;
    const int item = (int)(b / a.runs);
    int e;
    const int cnt = claim(a, item, list, e, lane_id(), wave_in_block());
    if (cnt == 0) return;   // workgroup-uniform, before any barrier
    const int grp = (int)(b - (int64_t)item * a.runs) * a.run;
    const int run = min(a.run, a.groups - grp);
    lds_barrier();          // the list is written
    constexpr int kTile = MANY ? 16 : 8;
    for (int c0 = 0; c0 < cnt; c0 += kTile) {
        const int M = min(kTile, cnt - c0);
        if (c0 > 0) lds_barrier();   // the columns and sums before are done with
        if (!MANY || M <= 8) f(std::integral_constant<int, 8>(), e, grp, run, M, list + c0);
        else if constexpr (MANY) f(std::integral_constant<int, 16>(), e, grp, run, M, list + c0);
    }
}

template <class TF, bool MANY, bool RUNS, int RT, int D>
__global__ void __launch_bounds__(64 * RT) MOE_WAVES
k_moe_glu(const uint8_t* __restrict__ Wg, const uint8_t* __restrict__ Wu, const uint8_t* __restrict__ Xq,
          uint8_t* __restrict__ Hq, int act, MoeArgs a) {
    extern __shared__ u32x4 moe_lds[];
    uint8_t* const lds = reinterpret_cast<uint8_t*>(moe_lds);
    each_columns<MANY>(a, lds, [&](auto mp, int e, int grp, int run, int M, const uint16_t* list) {
        glu_columns<TF, mp.value, RUNS, RT, D>(a, Wg, Wu, Xq, Hq, act, e, grp, run, M, list, lds, lane_id(), wave_in_block());
    });
}

template <class TF, bool MANY, bool RUNS, int RT, int KW, int D>
__global__ void __launch_bounds__(64 * RT * KW) MOE_WAVES
k_moe_down(const uint8_t* __restrict__ Wd, const uint8_t* __restrict__ Hq, float* __restrict__ part, MoeArgs a) {
    extern __shared__ u32x4 moe_lds[];
    uint8_t* const lds = reinterpret_cast<uint8_t*>(moe_lds);
    each_columns<MANY>(a, lds, [&](auto mp, int e, int grp, int run, int M, const uint16_t* list) {
        down_columns<TF, mp.value, RUNS, RT, KW, D>(a, Wd, Hq, part, e, grp, run, M, list, lds, lane_id(), wave_in_block());
    });
}

__device__ __forceinline__ void store_y(void* Y, int ydtype, size_t i, float v) {
    if (ydtype == DG_DTYPE_F32) ((float*)Y)[i] = v;
    else if (ydtype == DG_DTYPE_F16) ((_Float16*)Y)[i] = (_Float16)bind_f32(v);
    else ((__bf16*)Y)[i] = (__bf16)bind_f32(v);
}

// The down products and their weighted sum for one token at a time: a workgroup
// has RT row tiles of one token, a wave (j, rt, kw) its j-th expert's products
// with that expert's hidden column, so nothing is left to a third launch.  Each
// token reads its experts' weights for itself.  The order of every sum is that of
// k_moe_down and k_moe_sum.  The columns go into LDS 16 bytes a lane and turn, each turn
// behind its slot's id and its own load, and the first of these waits is one for the
// weights sent ahead too: 12 turns of 256 threads for two columns of 14336 (16.5 us for
// 66 MB).  Waves: k RT KW.
template <class TF, int RT, int KW, int D>
__global__ void __launch_bounds__(1024) MOE_WAVES
k_moe_down_tokens(const uint8_t* __restrict__ Wd, const uint8_t* __restrict__ Hq, const float* __restrict__ weights,
                  void* __restrict__ Y, int ydtype, MoeArgs a) {
#pragma clang fp contract(off)
    constexpr int NA = TileSet<8>::kNA;
    extern __shared__ u32x4 moe_lds[];
    uint8_t* const lds = reinterpret_cast<uint8_t*>(moe_lds);
    const int lane = lane_id(), wave = wave_in_block();
    const int j = wave / (RT * KW), rt = wave / KW % RT, kw = wave % KW;
    const int64_t b = a.first + blockIdx.x;
    const int m = (int)(b / a.groups);
    const int t = (int)(b - (int64_t)m * a.groups) * RT + rt;
    const int p = m * a.k + j;
    const int e = a.ids[p];
    const bool live = e >= 0 && e < a.E;   // wave-uniform
    const int S = a.K >> 8;
    const uint32_t stride = (uint32_t)(kGroupSlots * S) * 16u;
    const uint32_t zero = (uint32_t)a.k * stride;
    const int cnt = live ? (S - kw + KW - 1) / KW : 0;
    const uint8_t* const tile = Wd + ((size_t)(live ? e : 0) * (a.rows >> 4) + t) * S * TF::kGroupBytes;
    Stream<TF, D> stream(tile + (cnt > 0 ? kw : 0) * TF::kGroupBytes, cnt, KW * TF::kGroupBytes, lane);
    // the k hidden columns lie one after the other; a slot without an expert has none
    const int waves = a.k * RT * KW, slots = kGroupSlots * S;
    u32x4* const cols = moe_lds;
    for (int i = wave * kWave + lane; i < (a.k + 1) * slots; i += waves * kWave) {
        const int c = i / slots;
        const bool has = c < a.k && (uint32_t)a.ids[m * a.k + min(c, a.k - 1)] < (uint32_t)a.E;
        cols[i] = has ? reinterpret_cast<const u32x4*>(Hq + (size_t)m * a.k * stride)[i] : u32x4{0u, 0u, 0u, 0u};
    }
    lds_barrier();
    const ALanes al = a_lanes<8>((uint32_t)j * stride, 0, zero, 1, lane & 15);
    f32x4 acc[NA];
#pragma unroll
    for (int i = 0; i < NA; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    stream.template products<8>(acc, lds, al, kw, KW, lane);
    lds_barrier();   // every wave is done with the columns
    join_parts<NA, KW>(acc, reinterpret_cast<f32x4*>(lds), lane, wave, kw);
    lds_barrier();
    float* const sums = reinterpret_cast<float*>(lds);   // [j][RT * 16]
    if (kw == 0) {
        const TileOut<TF, 8> out(acc);
        if (lane < 16) sums[(j * RT + rt) * 16 + lane] = out.pair[0];
    }
    lds_barrier();
    const int n = wave * kWave + lane;
    if (n < RT * 16) {
        float y = 0.0f;
        for (int i = 0; i < a.k; ++i) {
            const int ei = a.ids[m * a.k + i];
            if (ei < 0 || ei >= a.E) continue;
            y += weights[m * a.k + i] * sums[i * RT * 16 + n];
        }
        store_y(Y, ydtype, (size_t)m * a.rows + (size_t)(t - rt) * 16 + n, y);
    }
}

constexpr int kSumSlots = 8, kSumThreads = 64;

// Y[m][n] = sum_j w[m][j] part[m k + j][n], in the order of j; four n a thread, kSumSlots
// slots' values on their way together (what a slot without an expert holds is not used).
template <class T>
__global__ void __launch_bounds__(kSumThreads)
k_moe_sum(const float* __restrict__ part, const int32_t* __restrict__ ids, const float* __restrict__ weights,
          T* __restrict__ Y, int K, int E, int k) {
#pragma clang fp contract(off)
    const int n = (int)(blockIdx.x * blockDim.x + threadIdx.x) * 4;
    const int m = blockIdx.y;
    if (n >= K) return;
    f32x4 y = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int j0 = 0; j0 < k; j0 += kSumSlots) {
        f32x4 v[kSumSlots];
#pragma unroll
        for (int j = 0; j < kSumSlots; ++j)
            v[j] = *reinterpret_cast<const f32x4*>(part + (size_t)(m * k + min(j0 + j, k - 1)) * K + n);
#pragma unroll
        for (int j = 0; j < kSumSlots; ++j) {
            const int p = m * k + min(j0 + j, k - 1);
            const bool has = j0 + j < k && (uint32_t)ids[p] < (uint32_t)E;   // wave-uniform
            const float w = weights[p];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float next = y[i] + w * v[j][i];
                y[i] = has ? next : y[i];
            }
        }
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

// One kernel over (items, workgroups of each), in launches of what one takes.
template <class F>
hipError_t over_groups(int64_t items, MoeArgs& a, F launch) {
    const int64_t all = items * a.runs;
    hipError_t e = hipSuccess;
    for (a.first = 0; a.first < all && e == hipSuccess; a.first += kMaxGroupsPerLaunch) {
        launch((unsigned)std::min<int64_t>(all - a.first, kMaxGroupsPerLaunch));
        e = hipGetLastError();
    }
    return e;
}

// LDS for the columns of a pass: the whole rows of as many columns as an expert
// has on the mean, twice over, where that leaves room for two workgroups on a CU.
int lds_for_columns(const MoeLayer& q, const MoeArgs& a) {
    const int64_t experts = std::min<int64_t>(a.P, q.E);
    const int64_t cols = std::min<int64_t>(std::min<int64_t>(kTileColumns, q.M), 2 * ((a.P + experts - 1) / experts));
    const int64_t want = (cols + 1) * (kGroupSlots * (a.K / 256) + 1) * 16 + 1024;
    const int64_t room = 80 * 1024 - 256 - a.lds_sums - (a.P * 2 + 15) / 16 * 16;
    return (int)std::max<int64_t>(8192, std::min<int64_t>(want, room) / 16 * 16);
}

// Experts that the tokens reach, chosen evenly.
double live_experts(const MoeLayer& q) {
    return (double)q.E * (1.0 - std::pow(1.0 - std::min(1.0, (double)q.k / (double)q.E), (double)q.M));
}

// Row groups of a workgroup.  Over Q4_0 rows of up to 2048 a workgroup's start and
// end weigh as much as its weights, so it takes as many row groups as make the best
// use of the workgroups that are resident together: in units of one row group's
// weights, `start` before each workgroup's first, and a third of a round for the
// uneven end of more than one round.  One row group each and as modelled: 24 tokens
// through 6 of 64 experts of 1536 x 2048 60.3 and 58.0 us, 16 53.1 and 52.6, 32 63.2 and
// 63.7; 24 through 8 of 128 of 768 x 2048 58.5 and 56.0, 32 62.5 and 59.7, 200 138 and 132;
// 8 through 8 of 64 of 1280 x 2048 42.2 and 40.6.  It is wrong at 16 through 8 of 128,
// 49.2 and 54.3.  Longer rows and two parts of K: no difference, so their kernels have no
// such loop.
template <class TF, int KW>
constexpr bool kRuns = std::is_same<TF, TilesQ4_0>::value && KW == 1;

void set_runs(const MoeLayer& q, MoeArgs& a, int waves, bool runs) {
    a.run = 1;
    if (runs && a.K <= 2048) {
        const double live = live_experts(q), resident = device_cu_count() * 16.0 / waves, start = 0.75;
        double best = 0;
        for (int r = 1; r <= std::min(8, a.groups); ++r) {
            const double rounds = live * ((a.groups + r - 1) / r) / resident;
            const double t = (r + start) * (rounds <= 1.0 ? 1.0 : rounds + 0.35);
            if (r == 1 || t < best) best = t, a.run = r;
        }
    }
    a.runs = (a.groups + a.run - 1) / a.run;
}

template <class TF, bool MANY, int RT, int D>
hipError_t moe_glu(const MoeLayer& q, MoeArgs a, int64_t items, uint8_t* Hq, hipStream_t s) {
    a.rows = (int)q.N;
    a.K = (int)q.K;
    a.groups = (int)(q.N / (8 * RT));
    a.lds_sums = RT / 2 * (MANY ? 2 : 1) * 1024 + (MANY ? 16 : 8) * 8 * RT * 4;
    a.lds_cols = lds_for_columns(q, a);
    constexpr bool kLoop = kRuns<TF, 1> && RT == 4;   // eight waves: rows that are too long for it
    set_runs(q, a, RT, kLoop);
    return over_groups(items, a, [&](unsigned grid) {
        const auto kernel = a.run > 1 ? k_moe_glu<TF, MANY, kLoop, RT, D> : k_moe_glu<TF, MANY, false, RT, D>;
        hipLaunchKernelGGL(kernel, dim3(grid), dim3(64 * RT), a.lds_cols + a.lds_sums + (size_t)a.P * 2, s,
                           (const uint8_t*)q.Wg, (const uint8_t*)q.Wu, (const uint8_t*)q.Xq, Hq, q.act, a);
    });
}

template <class TF, bool MANY, int RT, int KW, int D>
hipError_t moe_down(const MoeLayer& q, MoeArgs a, int64_t items, const uint8_t* Hq, float* part, hipStream_t s) {
    a.rows = (int)q.K;
    a.K = (int)q.N;
    a.groups = (int)(q.K / 16 / RT);
    a.lds_sums = KW > 1 ? RT * KW * (MANY ? 2 : 1) * 1024 : 0;
    a.lds_cols = lds_for_columns(q, a);
    set_runs(q, a, RT * KW, kRuns<TF, KW>);
    return over_groups(items, a, [&](unsigned grid) {
        const auto kernel = a.run > 1 ? k_moe_down<TF, MANY, kRuns<TF, KW>, RT, KW, D> : k_moe_down<TF, MANY, false, RT, KW, D>;
        hipLaunchKernelGGL(kernel, dim3(grid), dim3(64 * RT * KW), a.lds_cols + a.lds_sums + (size_t)a.P * 2, s,
                           (const uint8_t*)q.Wd, Hq, part, a);
    });
}

template <class TF, int RT, int KW, int D>
hipError_t moe_down_tokens(const MoeLayer& q, MoeArgs a, const uint8_t* Hq, hipStream_t s) {
    a.rows = (int)q.K;
    a.K = (int)q.N;
    a.groups = a.runs = (int)(q.K / 16 / RT);
    a.run = 1;
    const int waves = q.k * RT * KW;
    const size_t lds = std::max<size_t>((size_t)(q.k + 1) * kGroupSlots * (a.K / 256) * 16, (size_t)waves * 1024);
    return over_groups(q.M, a, [&](unsigned grid) {
        hipLaunchKernelGGL((k_moe_down_tokens<TF, RT, KW, D>), dim3(grid), dim3(64 * waves), lds, s,
                           (const uint8_t*)q.Wd, Hq, q.weights, q.Y, q.ydtype, a);
    });
}

// Parts of K per row tile of the down products.  It fixes the order of their
// sums, so it goes by the row's length alone.  With 2, 4 and 8 parts of 14336: one
// token through 2 of 8 Q4_0 experts 40.6, 39.3, 38.5 us, 16 tokens 123, 125, 135, 32
// through Q8_0 ones 228, 234, 249.  With 1 and 2 parts of 1536 (64 experts, k 6): one
// token 16.3, 15.6, 24 tokens 58, 63; of 768 (128 experts, k 8): 14.1, 14.3, 60, 66 (16).
int down_parts(const MoeLayer& q) { return q.N >= 4096 ? 2 : 1; }

// Whether k_moe_down_tokens takes the layer: the weights that tokens of one expert
// read again (with experts chosen evenly) cost less than the third launch.  Without
// and with it, by the bytes that are read again: 8 experts of 14336 x 4096, one token
// (none) 43.0 and 40.6 us, three (45e6) 78.8 and 83.0; 64 of 1536 x 2048, k 6, eight
// tokens (23e6) 44.5 and 41.4, twelve (48e6) 51.6 and 52.2; 128 Q8_0 ones of 768 x
// 2048, k 8, one token 19 and 16.3, twelve (45e6) 65.8 and 70.3.
bool by_token(const MoeLayer& q) {
    const double again = ((double)(q.M * q.k) - live_experts(q)) * (double)q.N * (double)q.K * (q.q8 ? 34.0 / 32 : 18.0 / 32);
    return again <= 24e6 && q.k * down_parts(q) <= 16 && (size_t)(q.k + 1) * kGroupSlots * (q.N / 256) * 16 <= 80 * 1024;
}

template <class TF, int KW, int D>
hipError_t moe_down_tokens_kw(const MoeLayer& q, const MoeArgs& a, const uint8_t* Hq, hipStream_t s) {
    const int64_t tiles = q.M * (q.K / 16);
    if (q.k * KW * 4 <= 8 && tiles >= 1024) return moe_down_tokens<TF, 4, KW, D>(q, a, Hq, s);
    if (q.k * KW * 2 <= 8 && tiles >= 512) return moe_down_tokens<TF, 2, KW, D>(q, a, Hq, s);
    return moe_down_tokens<TF, 1, KW, D>(q, a, Hq, s);
}

template <class TF, bool MANY>
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
    // Eight waves a workgroup share an expert's columns; four leave more workgroups, and shorter
    // ones, where the row is short.  Eight and four: 32 tokens through 8 Q8_0 experts of 14336 x
    // 4096 229 and 235 us, one through Q4_0 ones 40.6 and 41.6; 8 tokens through 8 of 128 of 768 x
    // 2048 35.0 and 33.0, 4 through 6 of 64 of 1536 x 2048 30.4 and 29.4, 24 57.7 and 58.5.
    const bool eight = q.K > 2048 && items * (q.N / 64) >= 256;
    const hipError_t e = eight ? moe_glu<TF, MANY, 8, 2>(q, a, items, Hq, s) : moe_glu<TF, MANY, 4, 2>(q, a, items, Hq, s);
    if (e != hipSuccess) return e;
    const bool two = down_parts(q) == 2;
    if (by_token(q)) return two ? moe_down_tokens_kw<TF, 2, 4>(q, a, Hq, s) : moe_down_tokens_kw<TF, 1, 2>(q, a, Hq, s);
    return two ? moe_down<TF, MANY, 4, 2, 2>(q, a, items, Hq, part, s) : moe_down<TF, MANY, 4, 1, 2>(q, a, items, Hq, part, s);
}

// MANY: an expert can have more than 8 columns.
template <class TF>
hipError_t moe_format(const MoeLayer& q, hipStream_t s) {
    return q.M > 8 ? moe_layer<TF, true>(q, s) : moe_layer<TF, false>(q, s);
}

template <class T>
hipError_t moe_sum(const MoeLayer& q, hipStream_t s) {
    const int P = (int)(q.M * q.k);
    const float* const part = (const float*)((const uint8_t*)q.ws + (size_t)P * (q.N / 32) * kQ81Bytes);
    hipLaunchKernelGGL((k_moe_sum<T>), dim3((unsigned)((q.K / 4 + kSumThreads - 1) / kSumThreads), (unsigned)q.M), dim3(kSumThreads), 0, s, part,
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
    hipError_t e = q.k == 0 ? hipSuccess : q.q8 ? moe_format<TilesQ8_0>(q, s) : moe_format<TilesQ4_0>(q, s);
    if (e != hipSuccess || (q.k > 0 && by_token(q))) return e;
    if (q.ydtype == DG_DTYPE_F32) return moe_sum<float>(q, s);
    if (q.ydtype == DG_DTYPE_F16) return moe_sum<_Float16>(q, s);
    return moe_sum<__bf16>(q, s);
}

}  // namespace dg
