// lora.hip -- low-rank adapters of many requests beside a shared projection:
//
//   h[m][r] = sum_k A[a][r][k] x[m][k],  Y[m][n] = base[m][n] + scale[a] sum_r B[a][n][r] h[m][r],  a = adapter[m]
//
// Two launches: h (a wave per row and rank), then Y (a lane eight ranks of an output,
// LG lanes an output).  A workgroup of Y stands for an adapter and a window of rows,
// or for a row where a window has fewer rows than there are adapters (it leaves if
// an earlier row has its adapter).  It finds its rows by reading the window's
// adapters, and takes them four at a time, so that B is read once for four rows.
// Few rows of few ranks and columns are one launch.
//
// Everything is widened to binary32 and multiplied and added there.  The order of a
// row's sums goes by K and R alone, so neither the other rows nor their adapters
// change it.  Matrix cores with 16 rows of one adapter a product were slower wherever
// an adapter has few rows, which is what a batch of requests has, and faster past some
// hundred rows of high rank: 64 x 4096 x 4096, R 16, one adapter 21 us against 7.5;
// 24 x 14336 x 4096 of binary32, R 64, 8 adapters 20 against 10.6; 200 x 28669 x 8192,
// R 32, 64 adapters 49 against 49.5; 2048 x 4096 x 4096, R 64, 4 adapters 56 against 111.
// Their sums are in another order, so a rule between the two would make a row's
// results depend on the number of rows; they are not used.
//
// What bounds it: few rows, the latency of dependent loads (the adapter, the runs of A
// and x, B behind their sums; dot_rows says how many trips a run is); many rows of many
// adapters, memory for Y (35 us of the 200 rows above, which move 191 MB) and loads waited
// for one pair at a time for h (14); many rows of one adapter, the vector operations.
#include <algorithm>
#include <type_traits>

#include "dg_batch.h"
#include "q4_common.h"

namespace dg {
namespace {

using q4::lds_barrier;

typedef float f32x4 __attribute__((ext_vector_type(4)));

struct LoraF32 {
    using raw = float;
    __device__ __forceinline__ static float widen(raw v) { return v; }
};
struct LoraF16 {
    using raw = _Float16;
    __device__ __forceinline__ static float widen(raw v) { return (float)v; }
};
struct LoraBF16 {
    using raw = __bf16;
    __device__ __forceinline__ static float widen(raw v) { return (float)v; }
};

// Eight consecutive elements as they lie in memory.  Loads here have no branch
// around them: the compiler waits for a load where the branch that holds it ends.
template <class E>
union Eight {
    static constexpr int kVecs = sizeof(typename E::raw) / 2;
    u32x4 q[kVecs];
    typename E::raw e[8];
    __device__ __forceinline__ void load(const typename E::raw* p) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) q[i] = reinterpret_cast<const u32x4*>(p)[i];
    }
};

constexpr int kMaxWindow = 256;    // rows that are looked through together
constexpr int kRows = 4;           // rows of one adapter that are taken together

struct LoraArgs {
    const int32_t *adapter, *ranks;
    const float* scale;
    int64_t M, N, ld;
    int K, R, L;
    int window;          // rows that are looked through together
    int by_row;          // workgroups stand for rows of the window, not adapters (the first: none)
    int block;           // outputs of a workgroup
    int64_t window0, block0;   // the launch's first
};

__device__ __forceinline__ int rank_of(const LoraArgs& a, int ad) {
    return a.ranks ? min(max(a.ranks[ad], 0), a.R) : a.R;
}
__device__ __forceinline__ int valid(const LoraArgs& a, int ad) { return (uint32_t)ad < (uint32_t)a.L ? ad : -1; }

// The workgroup's adapter (-1: none) of the window from row w0 on.  False: a row past
// the last.
__device__ __forceinline__ bool adapter_of(const LoraArgs& a, int64_t w0, int item, int& ad) {
    if (a.by_row && w0 + item >= a.M) return false;
    ad = a.by_row ? valid(a, a.adapter[w0 + item]) : item - 1;
    return true;
}

// The window's rows with the adapter, as places in the window, into list (by wave
// 0); their number, 0 where the adapter is that of a row before `item` and
// workgroups stand for rows.  Every wave comes to the same result.
__device__ __forceinline__ int rows_of(const LoraArgs& a, int64_t w0, int item, int ad, uint8_t* list, int lane, int wave) {
    const int n = (int)min((int64_t)a.window, a.M - w0);
    int id[kMaxWindow / kWave];
#pragma unroll
    for (int j = 0; j < kMaxWindow / kWave; ++j) id[j] = a.adapter[w0 + min(j * kWave + lane, n - 1)];
    int cnt = 0, first = kMaxWindow;
#pragma unroll
    for (int j = 0; j < kMaxWindow / kWave; ++j) {
        const bool same = j * kWave + lane < n && valid(a, id[j]) == ad;
        const uint64_t mask = __ballot(same);
        first = mask != 0 && cnt == 0 ? j * kWave + __builtin_ctzll(mask) : first;
        if (wave == 0 && same) list[cnt + __popcll(mask & (((uint64_t)1 << lane) - 1))] = (uint8_t)(j * kWave + lane);
        cnt += __popcll(mask);
    }
    return a.by_row && first < item ? 0 : cnt;
}

constexpr int kDotWaves = 4;

// The dots of a row of x with TR ranks' rows of A, in every lane.  A lane has every
// 64th run of eight columns, U of them a turn, and adds them in their order.  How many of
// a turn's loads are in flight is the compiler's choice: all or nearly all of them for
// binary32 rows and for binary16 by binary16; of bfloat16 by bfloat16 it waits for each
// run's two loads before it asks for the next (eight round trips a turn), and so for
// most runs of the mixed 16-bit pairs.
template <class EX, class EW, int TR>
__device__ __forceinline__ void dot_rows(const typename EX::raw* xr, const typename EW::raw* const (&Ar)[TR], int K,
                                         int lane, float (&sum)[TR]) {
    constexpr int U = sizeof(typename EX::raw) == 2 && TR == 1 ? 8 : 4;
#pragma unroll
    for (int t = 0; t < TR; ++t) sum[t] = 0.0f;
    for (int s = 0; s < K; s += U * 512) {
        Eight<EW> w[TR][U];
        Eight<EX> v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = min(s + u * 512 + lane * 8, K - 8);
#pragma unroll
            for (int t = 0; t < TR; ++t) w[t][u].load(Ar[t] + k);
            v[u].load(xr + k);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool some = s + u * 512 + lane * 8 < K;
#pragma unroll
            for (int e = 0; e < 8; ++e)
#pragma unroll
                for (int t = 0; t < TR; ++t) {
                    const float next = fmaf(EW::widen(w[t][u].e[e]), EX::widen(v[u].e[e]), sum[t]);
                    sum[t] = some ? next : sum[t];
                }
        }
    }
#pragma unroll
    for (int t = 0; t < TR; ++t) sum[t] = wave_sum_f32(sum[t]);
}

// h of one row and kDotWaves ranks, one a wave: x and A come from L2 but for their first
// readers, and what bounds it is the round trips of its loads (dot_rows; 200 bfloat16 rows
// of 8192 columns and 32 ranks make 16 in each of 6400 waves, 13.9 us).  With the loads
// as they are, two or four ranks a wave, for fewer reads of x, were
// no faster (24 rows of binary32, K 4096, R 64, with B: 10.6 us with one, 11.5 with two,
// 13.9 with four; 200 of bfloat16, K 8192, R 32: 54, 56, 56), nor were four rows of one
// adapter a wave (13 us, 64 us).  Grid: (runs of ranks, rows).
template <class EX, class EW>
__global__ void __launch_bounds__(64 * kDotWaves)
k_lora_dots(const typename EX::raw* __restrict__ x, const typename EW::raw* __restrict__ A, float* __restrict__ h,
            LoraArgs a) {
    const int lane = lane_id(), r = blockIdx.x * kDotWaves + q4::wave_in_block();
    const int64_t m = a.window0 + blockIdx.y;
    const int ad = valid(a, a.adapter[m]);
    if (ad < 0 || r >= rank_of(a, ad)) return;
    const typename EW::raw* const Ar[1] = {A + ((size_t)ad * a.R + r) * a.K};
    float sum[1];
    dot_rows<EX, EW, 1>(x + m * a.ld, Ar, a.K, lane, sum);
    if (lane == 0) h[m * a.R + r] = sum[0];
}

// The value of lane i's partner at a level of the sum over 2 D lanes: up to four, the
// mirrored lane of its 2 D, so that partners lie in opposite halves; then lane i ^ D.
template <int D>
__device__ __forceinline__ float partner(float v) {
    if constexpr (D == 1) return dpp_mov_f32<0xB1, 0xF>(v);         // quad_perm 1 0 3 2
    else if constexpr (D == 2) return dpp_mov_f32<0x1B, 0xF>(v);    // quad_perm 3 2 1 0
    else if constexpr (D == 4) return dpp_mov_f32<0x141, 0xF>(v);   // row_half_mirror
    else if constexpr (D == 8) return dpp_mov_f32<0x128, 0xF>(v);   // row_ror 8
    else return __shfl_xor(v, D);
}

// Of V values a lane, the sums over V lanes, each lane its own: half the values go to
// the partner at each level, down to v[0], the sum of value number lane % V.
template <int V>
__device__ __forceinline__ void scatter_sums(float (&v)[8], int lane) {
    if constexpr (V > 1) {
        constexpr int D = V / 2;
        const bool hi = lane & D;
#pragma unroll
        for (int j = 0; j < D; ++j) v[j] = (hi ? v[j + D] : v[j]) + partner<D>(hi ? v[j] : v[j + D]);
        scatter_sums<D>(v, lane);
    }
}

// Y of cnt <= TM rows for the workgroup's outputs; h[t]: eight ranks from 8 (lane %
// LG) on of row t.  A wave takes a strip of V * 64 / LG outputs at a time, V =
// min(LG, 8): value j of a lane is the part of output 64 / LG j + lane / LG of the
// strip that its eight ranks give.
template <class EW, int LG, int TM>
__device__ __forceinline__ void expand_rows(const typename EW::raw* Bn, const float* const (&base)[TM], float* const (&Y)[TM],
                                            const float (&h)[TM][8], int cnt, bool has_base, int len, int R, int rank,
                                            float scale, int lane, int wave, int waves) {
    constexpr int V = LG < 8 ? LG : 8, kOut = kWave / LG, kStrip = V * kOut;
    const int slice = lane % LG, out = lane / LG;
    const int mine = lane % V * kOut + out;   // the output of a strip that the lane stores, where slice < V
    for (int n = wave * kStrip; n < len; n += waves * kStrip) {
        Eight<EW> w[V];
        float add[TM];
#pragma unroll
        for (int j = 0; j < V; ++j)
            w[j].load(Bn + (size_t)min(n + j * kOut + out, len - 1) * R + min(8 * slice, R - 8));
#pragma unroll
        for (int t = 0; t < TM; ++t) add[t] = base[t][min(n + mine, len - 1)];
        if (rank < 8 * LG) {   // ranks past the adapter's: nothing, whatever is there
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) w[j].e[e] = 8 * slice + e < rank ? w[j].e[e] : (typename EW::raw)0.0f;
        }
#pragma unroll
        for (int t = 0; t < TM; ++t) {
            if (t >= cnt) continue;   // workgroup-uniform
            float v[8];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                v[j] = EW::widen(w[j].e[0]) * h[t][0];
#pragma unroll
                for (int e = 1; e < 8; ++e) v[j] = fmaf(EW::widen(w[j].e[e]), h[t][e], v[j]);
            }
            scatter_sums<V>(v, lane);
            if constexpr (LG > 8) v[0] += partner<8>(v[0]);
            if constexpr (LG > 16) v[0] += partner<16>(v[0]);
            if constexpr (LG > 32) v[0] += partner<32>(v[0]);
            const float y = (has_base ? add[t] : 0.0f) + scale * v[0];
            if (slice < V && n + mine < len) Y[t][n + mine] = y;
        }
    }
}

constexpr int kExpandWaves = 4;

// Y of a window's rows of one adapter for `block` outputs.  Grid: (blocks of outputs,
// adapters or rows, windows).  base: Y itself where there is none (!has_base).
template <class EW, int LG>
__global__ void __launch_bounds__(64 * kExpandWaves)
k_lora_expand(const typename EW::raw* __restrict__ B, const float* __restrict__ h, const float* base, float* Y,
              int has_base, LoraArgs a) {
    __shared__ uint8_t list[kMaxWindow];
    const int lane = lane_id(), wave = q4::wave_in_block(), item = blockIdx.y;
    const int64_t w0 = (a.window0 + blockIdx.z) * a.window;
    int ad;
    if (!adapter_of(a, w0, item, ad) || (ad < 0 && has_base && base == Y)) return;
    const int rank = ad < 0 ? 0 : rank_of(a, ad);
    const int64_t n0 = (a.block0 + blockIdx.x) * a.block;
    const int len = (int)min((int64_t)a.block, a.N - n0);
    const int all = rows_of(a, w0, item, ad, list, lane, wave);
    if (all == 0) return;   // workgroup-uniform, before any barrier
    lds_barrier();
    if (ad < 0) {   // rows without an adapter
        constexpr int V = 4;
        for (int r = wave; r < all; r += 2 * kExpandWaves) {   // two a wave, the last again
            int64_t o[2] = {(w0 + list[r]) * a.N + n0, (w0 + list[min(r + kExpandWaves, all - 1)]) * a.N + n0};
            for (int n = lane; n < len; n += V * kWave) {
                float v[2][V];
#pragma unroll
                for (int j = 0; j < V; ++j)
#pragma unroll
                    for (int k = 0; k < 2; ++k) v[k][j] = base[o[k] + min(n + j * kWave, len - 1)];
#pragma unroll
                for (int j = 0; j < V; ++j)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        if (n + j * kWave < len) Y[o[k] + n + j * kWave] = has_base ? v[k][j] : 0.0f;
            }
        }
        return;
    }
    const float scale = a.scale ? a.scale[ad] : 1.0f;
    const typename EW::raw* const Bn = B + ((size_t)ad * a.N + n0) * a.R;
    auto take = [&](auto rows, int c0) {
        constexpr int TM = decltype(rows)::value;
        const float* br[TM];
        float *yr[TM], v[TM][8];
        const int r0 = 8 * (lane % LG);
#pragma unroll
        for (int t = 0; t < TM; ++t) {   // fewer rows than TM: the last again
            const int64_t row = w0 + list[min(c0 + t, all - 1)];
            br[t] = base + row * a.N + n0;
            yr[t] = Y + row * a.N + n0;
            const f32x4* const p = reinterpret_cast<const f32x4*>(h + row * a.R + min(r0, a.R - 8));
            const f32x4 lo = p[0], hi = p[1];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[t][e] = r0 + e < rank && a.K > 0 ? (e < 4 ? lo[e] : hi[e - 4]) : 0.0f;
        }
        expand_rows<EW, LG, TM>(Bn, br, yr, v, min(TM, all - c0), has_base, len, a.R, rank, scale, lane, wave, kExpandWaves);
    };
    int c0 = 0;
    for (; c0 + 1 < all; c0 += kRows) take(std::integral_constant<int, kRows>(), c0);
    if (c0 < all) take(std::integral_constant<int, 1>(), c0);
}

constexpr int kOneWaves = 16;
constexpr int kOneBlock = 1024;   // outputs of a workgroup

// Whether one launch does the whole call: every workgroup of a row makes its h for
// itself, so A has to be little, and the workgroups few.  Microseconds on the GPU in one
// and two launches (the host's second launch, about 3, comes on top), bfloat16, rows x
// outputs x columns, rank: 1 x 4096 x 4096, 8: 3.9, 5.9; 16: 4.9, 6.0; 32: 6.4, 6.0; 4 x
// 4096 x 8192, 8: 5.5, 8.0; 16 x 4096 x 2048, 32: 4.9, 7.6; 1 x 4096 x 1024, 64 (with four
// ranks a wave, one after the other) 12.0, 6.0; 8 x 14336 x 4096 (112 workgroups), 16: 6.1,
// 6.4; 32: 8.1, 6.7.  Binary32 rows of x, 4 x 4096 x 8192, 8: 5.4, 6.6; 16: 8.2, 6.6.
bool one_launch(const LoraRows& q) {
    constexpr int64_t kMostGroups = 128, kMostReads = int64_t(1) << 23;
    const int64_t most = q.dtype == DG_DTYPE_F32 ? 65536 : 131072, one = q.R * q.K;
    if (one == 0 || one > most || q.R > 2 * kOneWaves || q.M > kMostGroups) return false;
    const int64_t groups = q.M * ((q.N + kOneBlock - 1) / kOneBlock);
    return groups <= kMostGroups && groups * one <= kMostReads;
}

// The sums are those of the two launches.  Grid: (blocks of outputs, rows).
template <class EX, class EW, int LG>
__global__ void __launch_bounds__(64 * kOneWaves)
k_lora_one(const typename EX::raw* __restrict__ x, const typename EW::raw* __restrict__ A,
           const typename EW::raw* __restrict__ B, const float* base, float* Y, int has_base, LoraArgs a) {
    __shared__ float hs[8 * LG];
    const int lane = lane_id(), wave = q4::wave_in_block();
    const int64_t m = blockIdx.y, n0 = (int64_t)blockIdx.x * kOneBlock;
    const int len = (int)min((int64_t)kOneBlock, a.N - n0);
    const int ad = valid(a, a.adapter[m]);
    const float* const br[1] = {base + m * a.N + n0};
    float* const yr[1] = {Y + m * a.N + n0};
    if (ad < 0) {
        if (has_base && base == Y) return;
        for (int n = threadIdx.x; n < len; n += 64 * kOneWaves) yr[0][n] = has_base ? br[0][n] : 0.0f;
        return;
    }
    const int rank = rank_of(a, ad);
    constexpr int TR = LG <= 2 ? 1 : 2;   // ranks of a wave
    static_assert(8 * LG <= TR * kOneWaves, "every rank");
    if (wave < rank) {
        const typename EW::raw* Ar[TR];
        float sum[TR];
#pragma unroll
        for (int t = 0; t < TR; ++t) {   // a rank that there is not: the first again
            const int r = wave + t * kOneWaves;
            Ar[t] = A + ((size_t)ad * a.R + (r < rank ? r : wave)) * a.K;
        }
        dot_rows<EX, EW, TR>(x + m * a.ld, Ar, a.K, lane, sum);
#pragma unroll
        for (int t = 0; t < TR; ++t)
            if (lane == 0 && wave + t * kOneWaves < rank) hs[wave + t * kOneWaves] = sum[t];
    }
    lds_barrier();
    float h[1][8];
#pragma unroll
    for (int e = 0; e < 8; ++e) h[0][e] = 8 * (lane % LG) + e < rank ? hs[8 * (lane % LG) + e] : 0.0f;
    expand_rows<EW, LG, 1>(B + ((size_t)ad * a.N + n0) * a.R, br, yr, h, 1, has_base, len, a.R, rank,
                           a.scale ? a.scale[ad] : 1.0f, lane, wave, kOneWaves);
}

template <class EX, class EW>
hipError_t lora_one(const LoraRows& q, const LoraArgs& a, hipStream_t s) {
    const auto kernel = q.R <= 8 ? k_lora_one<EX, EW, 1> : q.R <= 16 ? k_lora_one<EX, EW, 2> : k_lora_one<EX, EW, 4>;
    hipLaunchKernelGGL(kernel, dim3((unsigned)((q.N + kOneBlock - 1) / kOneBlock), (unsigned)q.M), dim3(64 * kOneWaves),
                       0, s, (const typename EX::raw*)q.x, (const typename EW::raw*)q.A, (const typename EW::raw*)q.B,
                       q.base ? q.base : q.Y, q.Y, q.base != nullptr, a);
    return hipGetLastError();
}

// launch(grid, arguments) over blocks, items and windows, in launches of what one takes.
template <class F>
hipError_t over_windows(int64_t blocks, int items, int64_t windows, LoraArgs a, F launch) {
    hipError_t e = hipSuccess;
    const int64_t xs = std::min<int64_t>(blocks, std::max<int64_t>(1, kMaxGroupsPerLaunch / items));
    const int64_t zs = std::min<int64_t>(32768, std::max<int64_t>(1, kMaxGroupsPerLaunch / (items * xs)));
    for (a.window0 = 0; a.window0 < windows; a.window0 += zs)
        for (a.block0 = 0; a.block0 < blocks && e == hipSuccess; a.block0 += xs) {
            launch(dim3((unsigned)std::min(xs, blocks - a.block0), (unsigned)items,
                        (unsigned)std::min(zs, windows - a.window0)), a);
            e = hipGetLastError();
        }
    return e;
}

template <class EW>
hipError_t lora_expand(const LoraRows& q, const LoraArgs& a, int items, int64_t windows, hipStream_t s) {
    const auto kernel = q.R <= 8     ? k_lora_expand<EW, 1>
                        : q.R <= 16  ? k_lora_expand<EW, 2>
                        : q.R <= 32  ? k_lora_expand<EW, 4>
                        : q.R <= 64  ? k_lora_expand<EW, 8>
                        : q.R <= 128 ? k_lora_expand<EW, 16>
                        : q.R <= 256 ? k_lora_expand<EW, 32>
                                     : k_lora_expand<EW, 64>;
    return over_windows((q.N + a.block - 1) / a.block, items, windows, a, [&](dim3 grid, const LoraArgs& v) {
        hipLaunchKernelGGL(kernel, grid, dim3(64 * kExpandWaves), 0, s, (const typename EW::raw*)q.B, (const float*)q.ws,
                           q.base ? q.base : q.Y, q.Y, q.base != nullptr, v);
    });
}

template <class EX, class EW>
hipError_t lora(const LoraRows& q, hipStream_t s) {
    LoraArgs a{};
    a.adapter = q.adapter;
    a.ranks = q.ranks;
    a.scale = q.scale;
    a.M = q.M;
    a.N = q.N;
    a.ld = q.ld;
    a.K = (int)q.K;
    a.R = (int)q.R;
    a.L = (int)q.L;
    if (one_launch(q)) return lora_one<EX, EW>(q, a, s);
    hipError_t e = hipSuccess;
    if (q.K > 0 && q.L > 0) {
        constexpr int64_t kMost = 16384;   // rows of a launch, of up to 128 workgroups
        const unsigned runs = (unsigned)((q.R + kDotWaves - 1) / kDotWaves);
        for (LoraArgs v = a; v.window0 < q.M && e == hipSuccess; v.window0 += kMost) {
            hipLaunchKernelGGL((k_lora_dots<EX, EW>), dim3(runs, (unsigned)std::min(kMost, q.M - v.window0)),
                               dim3(64 * kDotWaves), 0, s, (const typename EX::raw*)q.x,
                               (const typename EW::raw*)q.A, (float*)q.ws, v);
            e = hipGetLastError();
        }
    }
    if (e != hipSuccess) return e;
    a.window = (int)std::min<int64_t>(kMaxWindow, std::max<int64_t>(kRows, kRows * q.L));   // kRows of an adapter on the mean
    const int64_t windows = (q.M + a.window - 1) / a.window, rows = std::min<int64_t>(q.M, a.window);
    a.by_row = rows < q.L + 1;
    const int items = (int)std::min<int64_t>(rows, q.L + 1);
    // Long blocks read h and the adapters less often, short ones fill the machine: 200 x 28669
    // x 8192, R 32, 64 adapters 49.5 us with 512 or 256, 54 with 1024, 66 with 2048; 200 x
    // 14336 x 4096, R 16, 4 adapters 17.8 with 512, 19.1 with 256; 96 x 8192 x 1024, R 64, 16
    // adapters (272 workgroups of 1024) 15.0 with 256, 16.9 with 512.
    a.block = 512;
    if (windows * items * ((q.N + a.block - 1) / a.block) < 1024) a.block = 256;
    return lora_expand<EW>(q, a, items, windows, s);
}

template <class EX>
hipError_t lora_x(const LoraRows& q, hipStream_t s) {
    return q.wdtype == DG_DTYPE_F16 ? lora<EX, LoraF16>(q, s) : lora<EX, LoraBF16>(q, s);
}

}  // namespace

size_t lora_workspace_bytes(int64_t M, int64_t K, int64_t R) {
    (void)K;
    return (size_t)M * (size_t)R * 4;
}

hipError_t launch_lora_rows(const LoraRows& q, hipStream_t s) {
    if (q.dtype == DG_DTYPE_F32) return lora_x<LoraF32>(q, s);
    if (q.dtype == DG_DTYPE_F16) return lora_x<LoraF16>(q, s);
    return lora_x<LoraBF16>(q, s);
}

}  // namespace dg
