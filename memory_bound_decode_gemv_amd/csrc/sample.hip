// sample.hip -- one token per row from given random numbers: temperature,
// top-k, top-p and min-p over float32, binary16 or bfloat16 logits.
//
// Weights.  w_i = exp((x_i - m) / T) with m the row's maximum, in binary64,
// held as the integer W_i = round(2^F w_i), F = min(51, 62 - ceil(log2 C)):
// every sum of them fits 62 bits and is exact, so it does not depend on the
// order of summation, on the split of a row over workgroups or on the order
// in which atomics arrive, and the same call gives the same token on any
// launch shape.  A token with W_i = 0 (below 2^-(F+1) of the likeliest) has no
// part in anything.
//
// Rank order is value descending, index ascending, which is the descending
// order of the 64-bit keys of the argmax (value image, then inverted index).
// top-k and top-p each keep a prefix of that order, so what they keep together
// is { key >= threshold } for one threshold key; min-p compares w_i itself.
// The token is the first kept index whose running sum of W exceeds u times
// the kept total.
//
// Rows of up to kCand elements: one workgroup and one launch, the row's keys
// in LDS.  Longer rows, four launches:
//   max     every chunk's largest key and smallest finite value;
//   hist    (rows with top-k or top-p) counts and masses of kBins equal steps
//           of m - x over the part of the row's range that has weight: steps
//           of the value itself, not of its bits, so that a bell of logits
//           spreads over the bins;
//   gather  every workgroup reads the bins and finds the ones that the
//           borders fall into; sums what lies above them for sure, per
//           sub-chunk, and lists the keys of the border bins;
//   pick    one workgroup per row resolves the borders within the listed keys,
//           adds the kept ones to the sub-chunk sums, and finds the sub-chunk and
//           in it the element that u falls into.  Up to 64 keys: every key against
//           every other, in one wave; up to 1024: sorted, one per thread; more: a
//           radix descent over the key bits that differ.
// A row whose border bins hold more than kCand elements is resolved by the same
// descent reading the row, several times and from one workgroup, instead of the
// list.  That is slow: 128256 equal logits with top-p take 560 us.  It happens to
// many equal values, and to flat rows of which a token is masked with a finite
// number, which stretches the bins over the whole range that has weight: 128000
// logits of deviation 0.5 at temperature 1, top-p 0.9, take 25 us, and 408 with
// one of them at the lowest value; 262144 of deviation 1, 28 and 915 (128000 of
// deviation 1: 26 and 27).  Tokens masked with -infinity have no part in the bins.
//
// One row of 128256 float32 logits takes 18 us, four dependent launches of 3 to
// 6 us (16 with one to five tokens allowed, 11 without top-k and top-p, 6.4 if
// greedy); 256 rows of 128000 with top-p alone 123 us, bound by instruction issue
// (the vector unit is busy for 82 to 86 % of hist and gather, which compute
// every weight anew: 43.5 and 57.6 us) after a first pass at 5.9 TB/s (22 us).
// 64 rows of 128256 bfloat16 logits with mixed filters take 43 us; the pick sorts
// their lists in 9.2 us, where the descent took 13.1.  Rows of 4096 take 6.5 us
// without top-k and top-p and 18 to 22 with them, in which the one workgroup's
// descent has up to eight steps of several barriers each.
#include "argkey.h"
#include "dg_device.h"
#include "dg_internal.h"
#include "sample_bins.h"

// Every kernel computes an element's weight and bin anew; they have to agree
// to the bit, so no kernel may contract what another does not.
#pragma clang fp contract(off)

namespace dg {
namespace {

constexpr int kCand = 4096;          // keys that the pick kernel holds in LDS
constexpr int kChunkList = 2048;     // of them that one workgroup of the gather kernel lists
constexpr int kSubMin = 2048;        // elements of a sub-chunk, at least
constexpr int kMaxSubs = 1024;       // sub-chunks of a row, at most
constexpr int kChunkThreads = 256;
constexpr int kPickThreads = 1024;
static_assert(kPickThreads == kMaxSubs, "a thread of the pick kernel per sub-chunk");
constexpr int kTargetGroups = 1024;
constexpr int kBatchRows = 512;      // rows whose workspace exists at once
constexpr double kLog2e = 1.4426950408889634;

typedef unsigned long long u64;

template <class T>
struct Logit {
    __device__ __forceinline__ static float load(const T* p) { return (float)*p; }
};

constexpr int kPer = 8;   // elements per thread of the chunk kernels: kChunkThreads of them fill a shortest sub-chunk
constexpr int kTogether = 4;   // of them whose weights are computed side by side
static_assert(kPer * kChunkThreads == kSubMin, "one load step per shortest sub-chunk");

// This thread's kPer elements of the kSubMin from c0 on (those at C and past
// it as -infinity, which has no weight): consecutive ones in one or two
// 16-byte loads where the row is 16-byte aligned, else a coalesced stride
// apart.  element(i, vec) is the offset of the i-th from c0.  Binary32 loads stay
// in flight past load(), so that a step is loaded ahead of its use.  16-bit ones
// do not: they are widened in the branch that loads them and waited for there,
// eight times in rows that are not 16-byte aligned.
template <class T>
struct Share {
    float v[kPer];
    __device__ __forceinline__ static int element(int i, bool vec) {
        return vec ? (int)threadIdx.x * kPer + i : i * kChunkThreads + (int)threadIdx.x;
    }
    __device__ __forceinline__ void load(const T* __restrict__ row, int64_t c0, int64_t C, bool vec) {
        constexpr int kVecs = kPer * sizeof(T) / 16;
        if (vec && c0 + element(kPer - 1, true) < C) {
            union {
                u32x4 q[kVecs];
                T e[kPer];
            } b;
            const u32x4* p = reinterpret_cast<const u32x4*>(row + c0 + element(0, true));
#pragma unroll
            for (int i = 0; i < kVecs; ++i) b.q[i] = p[i];
#pragma unroll
            for (int i = 0; i < kPer; ++i) v[i] = (float)b.e[i];
        } else {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int64_t c = c0 + element(i, vec);
                v[i] = c < C ? Logit<T>::load(row + c) : -INFINITY;
            }
        }
    }
};

struct SampleArgs {
    const float *u, *temperature, *top_p, *min_p;
    const int32_t* top_k;
    int64_t* idx;
    int C;
    int64_t ld;
    int F;          // fraction bits of the integer weights
    int sub;        // elements per sub-chunk
    int nsub;
    int G;          // chunks per row
    int subs_per_chunk;
    bool vec;       // rows are 16-byte aligned
};

__device__ __forceinline__ float key_value(u64 key) {
    const uint32_t img = (uint32_t)(key >> 32);
    return __builtin_bit_cast(float, (img & 0x80000000u) ? img ^ 0x80000000u : ~img);
}

// One row's parameters and what follows from its extremes.
struct Row {
    float m;          // maximum
    float scale;      // bins per unit of m - x
    double c;         // log2(e) / T
    double min_p;     // 0: off
    double p;         // >= 1: off
    double u;
    int64_t known;    // the token, when no draw is needed; else -2
    int k;            // 0: off
    int F;
    float far;        // elements whose m - x exceeds this have w < min_p

    // w as a binary64 number in [0, 1]
    __device__ __forceinline__ double weight(float x) const {
        double w[1];
        weights(&x, w);
        return w[0];
    }
    // The weights of N elements, side by side so that their chains of dependent
    // operations overlap.  w = 2^t, t = (x - m) log2(e) / T; t = n + f with n an
    // integer and |f| <= 1/2, and 2^f by the polynomial of degree 10 that
    // interpolates it at the Chebyshev nodes of [-1/2, 1/2] (within 3.2e-16,
    // and 1 at 0).  n is the low word of t + 1.5 2^52 and goes into the exponent
    // by an integer addition: every operation but the first is a full-rate
    // binary64 one.  t below -200, or not a number, counts as -200, far below
    // any weight that counts; an infinite m, which cannot be subtracted, is the
    // largest binary64 number instead.
    template <int N>
    __device__ __forceinline__ void weights(const float* x, double (&w)[N]) const {
        constexpr double kLargest = 1.7976931348623157e308, kRound = 6755399441055744.0;
        const double top = fmin((double)m, kLargest);
        double f[N];
        uint32_t n[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const double t = fmax((fmin((double)x[i], kLargest) - top) * c, -200.0);
            const double z = t + kRound;
            n[i] = (uint32_t)__builtin_bit_cast(u64, z);
            f[i] = t - (z - kRound);
            w[i] = 7.072585949269223e-09;
        }
#define DG_TERM(C)                                          \
    _Pragma("unroll") for (int i = 0; i < N; ++i) w[i] = fma(w[i], f[i], C);
        DG_TERM(1.0208690299958306e-07)
        DG_TERM(1.321544258792169e-06)
        DG_TERM(1.5252657260200837e-05)
        DG_TERM(0.0001540353044173605)
        DG_TERM(0.0013333558230164974)
        DG_TERM(0.009618129107606888)
        DG_TERM(0.05550410866444772)
        DG_TERM(0.24022650695910097)
        DG_TERM(0.69314718055995)
        DG_TERM(1.0)
#undef DG_TERM
#pragma unroll
        for (int i = 0; i < N; ++i) {
            // the high word plus n << 20, as one operation (the compiler widens the
            // addition to 64 bits), and bound here, or it moves each chain into the
            // branch of its first use, one after the other (the gather of 256 rows
            // of 128000: 97 us against 81)
            const u64 v = __builtin_bit_cast(u64, w[i]);
            uint32_t hi = (uint32_t)(v >> 32);
            if constexpr (N > 1) asm volatile("v_lshl_add_u32 %0, %1, 20, %0" : "+v"(hi) : "v"(n[i]));
            else hi += n[i] << 20;
            w[i] = __builtin_bit_cast(double, (u64)hi << 32 | (uint32_t)v);
        }
    }
    // round(2^F w) by the binary64 addition 2^52 + 2^F w (F <= 51)
    __device__ __forceinline__ u64 fixed(double w) const {
        const double v = fma(w, (double)(1ull << F), 4503599627370496.0);
        return __builtin_bit_cast(u64, v) & 0x000FFFFFFFFFFFFFull;
    }
    __device__ __forceinline__ float below(float x) const { return bin_distance(m, x); }
    __device__ __forceinline__ float place(float d) const { return bin_place(d, scale); }
    __device__ __forceinline__ int bin(float x) const { return (int)place(below(x)); }
};

// What the bins say about the borders of top-k and top-p.
struct Borders {
    int sure;              // bins below this are kept whole
    int kbin;              // the bin of the k-th token, or kBins when top-k is off
    int p0, p1;            // bins p0..p1 may hold top-p's border (p0 > p1: top-p is off)
    uint32_t krank;        // its rank within kbin, from 1
    u64 kmass;             // mass above kbin
    u64 pmass;             // mass above p0
    u64 total;             // mass of all bins (0 without top-p)
};

__device__ __forceinline__ bool border_bin(const Borders& b, int i) { return i == b.kbin || (i >= b.p0 && i <= b.p1); }

// The workspace of one row.
struct RowSpace {
    Row row;                 // from the gather kernel to the pick kernel
    Borders borders;
    u64 key[kMaxSubs];       // per chunk: largest key
    uint32_t low[kMaxSubs];  // per chunk: inverted image of its smallest value above -infinity (0 if none)
    u64 mass[kBins];
    uint32_t count[kBins];
    uint32_t ncand;
    uint32_t pad;
    u64 sum[kMaxSubs];       // per sub-chunk: kept for sure
    u64 cand[kCand];
};

// A row's parameters as the caller gave them.
struct Params {
    float T, p, min_p, u;
    int k;
};

__device__ __forceinline__ Params load_params(const SampleArgs& a, int64_t r) {
    Params t;
    t.T = a.temperature ? a.temperature[r] : 1.0f;
    t.p = a.top_p ? a.top_p[r] : 1.0f;
    t.min_p = a.min_p ? a.min_p[r] : 0.0f;
    t.u = a.u[r];
    t.k = a.top_k ? a.top_k[r] : 0;
    return t;
}

__device__ __forceinline__ Row make_row(const SampleArgs& a, const Params& t, u64 top, float low) {
    Row q;
    q.m = key_value(top);
    q.known = -2;
    if ((uint32_t)(top >> 32) == 0xFFFFFFFFu || !(t.T > 0.0f)) q.known = (int64_t)key_index(top);   // a NaN, or greedy
    else if (q.m == -INFINITY) q.known = -1;                                                       // nothing to draw from
    q.k = t.k > 0 && t.k < a.C ? t.k : 0;
    q.p = t.p < 1.0f ? (t.p > 0.0f ? t.p : 0.0f) : 1.0f;
    q.min_p = t.min_p > 0.0f ? (t.min_p < 1.0f ? t.min_p : 1.0f) : 0.0f;
    q.u = t.u > 0.0f ? (t.u < 1.0f ? t.u : 1.0f) : 0.0f;
    q.F = a.F;
    q.c = kLog2e / (double)t.T;
    constexpr float kLn2 = 0.69314718f;
    q.scale = bin_scale(q.m, low, (float)(a.F + 1) * kLn2 * t.T);
    if (q.m == INFINITY) q.c = 1.0;   // m - x is 0 or infinite, at any temperature
    // -log2(min_p) / c, and more than its roundings
    q.far = q.min_p > 0.0 ? (1.001f * -log2f((float)q.min_p) + 1e-5f) * kLn2 * t.T : INFINITY;
    return q;
}

__device__ __forceinline__ uint32_t umax32(uint32_t a, uint32_t b) { return a > b ? a : b; }

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
    v = umax32(v, dpp_mov_u32<kDppRowShr1, 0xF>(v));
    v = umax32(v, dpp_mov_u32<kDppRowShr2, 0xF>(v));
    v = umax32(v, dpp_mov_u32<kDppRowShr4, 0xF>(v));
    v = umax32(v, dpp_mov_u32<kDppRowShr8, 0xF>(v));
    v = umax32(v, dpp_mov_u32<kDppRowBcast15, 0xA>(v));
    v = umax32(v, dpp_mov_u32<kDppRowBcast31, 0xC>(v));
    return (uint32_t)__builtin_amdgcn_readlane((int)v, kWave - 1);
}

__device__ __forceinline__ uint32_t wave_scan_u32(uint32_t v) {   // inclusive sums
    v += dpp_mov_u32<kDppRowShr1, 0xF>(v);
    v += dpp_mov_u32<kDppRowShr2, 0xF>(v);
    v += dpp_mov_u32<kDppRowShr4, 0xF>(v);
    v += dpp_mov_u32<kDppRowShr8, 0xF>(v);
    v += dpp_mov_u32<kDppRowBcast15, 0xA>(v);
    v += dpp_mov_u32<kDppRowBcast31, 0xC>(v);
    return v;
}

constexpr int kQuadXor1 = 0xB1;         // DPP quad_perm [1,0,3,2]
constexpr int kQuadXor2 = 0x4E;         // DPP quad_perm [2,3,0,1]
constexpr int kQuadXor3 = 0x1B;         // DPP quad_perm [3,2,1,0]
constexpr int kHalfRowMirror = 0x141;   // DPP: lane ^ 7
constexpr int kRowRotate8 = 0x128;      // DPP row_ror 8: lane ^ 8

// Inclusive sums over the wave, on DPP moves (lanes without a source receive 0).
__device__ __forceinline__ u64 wave_scan_u64(u64 v) {
    v += dpp_key<kDppRowShr1, 0xF>(v);
    v += dpp_key<kDppRowShr2, 0xF>(v);
    v += dpp_key<kDppRowShr4, 0xF>(v);
    v += dpp_key<kDppRowShr8, 0xF>(v);
    v += dpp_key<kDppRowBcast15, 0xA>(v);
    v += dpp_key<kDppRowBcast31, 0xC>(v);
    return v;
}

__device__ __forceinline__ u64 wave_or_u64(u64 v) {   // in lane 63
    v |= dpp_key<kDppRowShr1, 0xF>(v);
    v |= dpp_key<kDppRowShr2, 0xF>(v);
    v |= dpp_key<kDppRowShr4, 0xF>(v);
    v |= dpp_key<kDppRowShr8, 0xF>(v);
    v |= dpp_key<kDppRowBcast15, 0xA>(v);
    v |= dpp_key<kDppRowBcast31, 0xC>(v);
    return v;
}

// A lane's value in every lane (the lane is the same in all of them).
__device__ __forceinline__ u64 lane_u64(u64 v, int src) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, src);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), src);
    return ((u64)hi << 32) | lo;
}

__device__ __forceinline__ u64 wave_sum_u64(u64 v) { return lane_u64(wave_scan_u64(v), kWave - 1); }

// Inclusive sums over the workgroup in thread order; *total = the whole sum.
template <int THREADS>
__device__ __forceinline__ u64 block_scan_u64(u64 v, u64* total) {
    constexpr int kWaves = THREADS / kWave;
    __shared__ u64 part[kWaves];
    const int wave = threadIdx.x / kWave;
    v = wave_scan_u64(v);
    __syncthreads();   // the array's last use is over
    if (lane_id() == kWave - 1) part[wave] = v;
    __syncthreads();
    u64 before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        if (w < wave) before += part[w];
        all += part[w];
    }
    *total = all;
    return before + v;
}

// A row's extremes from its chunks (every wave by itself).
__device__ __forceinline__ void row_extremes(const RowSpace* ws, int G, u64* top, float* low) {
    u64 t = 0;
    uint32_t l = 0;
    for (int g = lane_id(); g < G; g += kWave) {
        t = umax64(t, ws->key[g]);
        l = umax32(l, ws->low[g]);
    }
    *top = wave_max_u64(t);
    l = wave_max_u32(l);
    *low = l ? key_value((u64)~l << 32) : INFINITY;
}

// The largest and the smallest of three, as one instruction each (fmaxf and
// fminf of loaded values take one more to quieten NaNs).
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
    float r;
    asm("v_min3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}

// ---- max ----------------------------------------------------------------------
template <class T>
__global__ void __launch_bounds__(kChunkThreads)
k_sample_max(const T* __restrict__ x, RowSpace* __restrict__ spaces, SampleArgs a) {
    const int g = blockIdx.x;
    const int64_t r = blockIdx.y;
    RowSpace* ws = spaces + r;
    const T* row = x + r * a.ld;
    const int64_t c0 = (int64_t)g * a.subs_per_chunk * a.sub;
    const int64_t c1 = c0 + (int64_t)a.subs_per_chunk * a.sub < a.C ? c0 + (int64_t)a.subs_per_chunk * a.sub : a.C;
    Share<T> ahead;
    ahead.load(row, c0, a.C, a.vec);
    uint32_t best = 0u, low = 0u;
    u64 key = 0;
    if (c0 + kSubMin >= c1) {   // one load step: every element's key at once
        uint32_t bidx = 0xFFFFFFFFu;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {   // a thread's elements in increasing order
            const uint32_t img = order_image(ahead.v[i]);
            if (img > best) { best = img; bidx = (uint32_t)(c0 + Share<T>::element(i, a.vec)); }
            if (ahead.v[i] > -INFINITY) low = umax32(low, ~img);
        }
        key = pack_key(best, bidx);
    } else {
        // Per step only the largest image and the smallest value: by the counters
        // 9 vector instructions an element in place of 20, conversions and the
        // rest of the launch included (256 rows of 128000 float32); 64 rows of
        // 128256 bfloat16 take 6.4 us in place of 8.4.  The place within the step is looked up once, by the lanes that
        // hold the wave's maximum, at the cost of another round trip (one step:
        // 3.6 us for 3.1).
        int64_t at = c0;            // the step of `best`
        float least = INFINITY;     // above -infinity
        for (int64_t c = c0; c < c1; c += kSubMin) {
            const Share<T> e = ahead;
            if (c + kSubMin < c1) ahead.load(row, c + kSubMin, a.C, a.vec);
            float most = e.v[0], min8 = e.v[0];
            bool nan = e.v[0] != e.v[0];
#pragma unroll
            for (int i = 1; i < kPer; i += 2) {
                const float second = e.v[i + 1 < kPer ? i + 1 : i];
                most = max3(most, e.v[i], second);
                min8 = min3(min8, e.v[i], second);
                nan |= __builtin_isunordered(e.v[i], second);
            }
            const uint32_t img = nan ? 0xFFFFFFFFu : order_image(most);
            if (img > best) { best = img; at = c; }
            if (min8 == -INFINITY) {
                min8 = INFINITY;
#pragma unroll
                for (int i = 0; i < kPer; ++i)
                    if (e.v[i] > -INFINITY) min8 = fminf(min8, e.v[i]);
            }
            least = fminf(least, min8);
        }
        low = least < INFINITY ? ~order_image(least) : 0u;
        if (best == wave_max_u32(best)) {
            Share<T> e;
            e.load(row, at, a.C, a.vec);
#pragma unroll
            for (int i = kPer - 1; i >= 0; --i)   // the first of the step's
                if (order_image(e.v[i]) == best) key = pack_key(best, (uint32_t)(at + Share<T>::element(i, a.vec)));
        }
    }
    key = wave_max_u64(key);
    low = wave_max_u32(low);
    __shared__ u64 keys[kChunkThreads / kWave];
    __shared__ uint32_t lows[kChunkThreads / kWave];
    if (lane_id() == 0) {
        keys[threadIdx.x / kWave] = key;
        lows[threadIdx.x / kWave] = low;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int w = 1; w < kChunkThreads / kWave; ++w) {
            key = umax64(key, keys[w]);
            low = umax32(low, lows[w]);
        }
        ws->key[g] = key;
        ws->low[g] = low;
    }
    // the row's bins and list, cleared for the next launches
    for (int i = g * kChunkThreads + threadIdx.x; i < kBins; i += a.G * kChunkThreads) {
        ws->mass[i] = 0;
        ws->count[i] = 0;
    }
    if (g == 0 && threadIdx.x == 0) ws->ncand = 0;
}

// ---- hist ---------------------------------------------------------------------
template <class T>
__global__ void __launch_bounds__(kChunkThreads)
k_sample_hist(const T* __restrict__ x, RowSpace* __restrict__ spaces, SampleArgs a) {
    __shared__ u64 mass[kBins];
    __shared__ uint32_t count[kBins];
    const int g = blockIdx.x;
    const int64_t r = blockIdx.y;
    RowSpace* ws = spaces + r;
    const T* row = x + r * a.ld;
    const int64_t c0 = (int64_t)g * a.subs_per_chunk * a.sub;
    const int64_t c1 = c0 + (int64_t)a.subs_per_chunk * a.sub < a.C ? c0 + (int64_t)a.subs_per_chunk * a.sub : a.C;
    Share<T> ahead;
    const Params given = load_params(a, r);
    ahead.load(row, c0, a.C, a.vec);   // binary32: in flight while the row's extremes arrive
    u64 top;
    float low;
    row_extremes(ws, a.G, &top, &low);
    const Row q = make_row(a, given, top, low);
    if (q.known != -2 || (q.k == 0 && q.p >= 1.0)) return;   // workgroup-uniform: nothing to select
    for (int i = threadIdx.x; i < kBins; i += kChunkThreads) {
        mass[i] = 0;
        count[i] = 0;
    }
    __syncthreads();
    // top-k needs the counts, top-p the masses.  Counting alone takes no
    // weights: elements without weight are in the last bin, behind all others,
    // and it does not matter whether they are counted.
    const bool by_mass = q.p < 1.0, by_count = q.k > 0;
    for (int64_t c = c0; c < c1; c += kSubMin) {
        const Share<T> e = ahead;
        if (c + kSubMin < c1) ahead.load(row, c + kSubMin, a.C, a.vec);
#pragma unroll
        for (int h = 0; h < kPer; h += kTogether) {
            if (by_mass) {
                double w[kTogether];
                q.weights(e.v + h, w);
#pragma unroll
                for (int i = 0; i < kTogether; ++i) {
                    const u64 W = q.fixed(w[i]);
                    if (W) {
                        const int b = q.bin(e.v[h + i]);
                        atomicAdd(&mass[b], W);
                        if (by_count) atomicAdd(&count[b], 1u);
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < kTogether; ++i)
                    if (e.v[h + i] > -INFINITY) atomicAdd(&count[q.bin(e.v[h + i])], 1u);
            }
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kBins; i += kChunkThreads) {
        if (mass[i]) atomicAdd(&ws->mass[i], mass[i]);
        if (count[i]) atomicAdd(&ws->count[i], count[i]);
    }
}

// ---- borders ------------------------------------------------------------------
// The shortest prefix has mass >= this: ceil(p * total), at least 1.
__device__ __forceinline__ u64 p_target(double p, u64 total) {
    const u64 t = (u64)ceil(p * (double)total);
    return t < 1 ? 1 : (t > total ? total : t);
}

constexpr int kLaneBins = kBins / kWave;

// The bins of a lane of the first wave (the others load nothing).
struct LaneBins {
    u64 mass[kLaneBins];
    uint32_t count[kLaneBins];
    __device__ __forceinline__ void load(const RowSpace* ws) {
        if (threadIdx.x < kWave) {
#pragma unroll
            for (int i = 0; i < kLaneBins; ++i) {
                mass[i] = ws->mass[threadIdx.x * kLaneBins + i];
                count[i] = ws->count[threadIdx.x * kLaneBins + i];
            }
        }
    }
};

// Every thread of the workgroup calls this; the first wave scans the bins,
// eight per lane.
__device__ __forceinline__ Borders find_borders(const LaneBins& bins_of, const Row& q) {
    __shared__ Borders out;
    if (threadIdx.x < kWave) {
        const int lane = threadIdx.x;
        const u64(&mass)[kLaneBins] = bins_of.mass;
        const uint32_t(&count)[kLaneBins] = bins_of.count;
        Borders b;
        b.total = 0;
        b.kbin = kBins;
        b.krank = 0;
        b.kmass = 0;
        b.p0 = 1;
        b.p1 = 0;
        b.pmass = 0;
        u64 m_in = 0, m_to = 0;
        if (q.p < 1.0) {
#pragma unroll
            for (int i = 0; i < kLaneBins; ++i) m_in += mass[i];
            m_to = wave_scan_u64(m_in);
            b.total = lane_u64(m_to, kWave - 1);
        }
        u64 m_low = b.total, m_high = b.total;   // the mass that top-p is a share of, at least and at most
        if (q.k) {
            uint32_t c_in = 0;
#pragma unroll
            for (int i = 0; i < kLaneBins; ++i) c_in += count[i];
            const uint32_t c_to = wave_scan_u32(c_in);
            if ((uint32_t)q.k < (uint32_t)__builtin_amdgcn_readlane((int)c_to, kWave - 1)) {
                // the lane and the bin in which the count reaches k
                uint32_t c = c_to - c_in, rank = 0;
                u64 m = m_to - m_in, above = 0, upto = 0;
                int bin = kBins;
#pragma unroll
                for (int i = 0; i < kLaneBins; ++i) {
                    if (c < (uint32_t)q.k && c + count[i] >= (uint32_t)q.k) {
                        bin = lane * kLaneBins + i;
                        rank = (uint32_t)q.k - c;
                        above = m;
                        upto = m + mass[i];
                    }
                    c += count[i];
                    m += mass[i];
                }
                const int src = __ffsll((unsigned long long)__ballot(bin != kBins)) - 1;   // exactly one lane
                b.kbin = __builtin_amdgcn_readlane(bin, src);
                b.krank = (uint32_t)__builtin_amdgcn_readlane((int)rank, src);
                if (q.p < 1.0) {
                    b.kmass = lane_u64(above, src);
                    m_low = b.kmass;
                    m_high = lane_u64(upto, src);
                }
            }
        }
        if (q.p < 1.0) {
            const u64 t[2] = {m_low ? p_target(q.p, m_low) : 1ull, p_target(q.p, m_high)};
            int bins[2];
            u64 aboves[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                u64 m = m_to - m_in, above = 0;
                int bin = kBins;
#pragma unroll
                for (int i = 0; i < kLaneBins; ++i) {
                    if (m < t[j] && m + mass[i] >= t[j]) {
                        bin = lane * kLaneBins + i;
                        above = m;
                    }
                    m += mass[i];
                }
                const int src = __ffsll((unsigned long long)__ballot(bin != kBins)) - 1;
                bins[j] = __builtin_amdgcn_readlane(bin, src);
                aboves[j] = lane_u64(above, src);
            }
            b.p0 = bins[0];
            b.p1 = bins[1];
            b.pmass = aboves[0];
        }
        b.sure = q.p < 1.0 ? b.p0 : b.kbin;
        if (lane == 0) out = b;
    }
    __syncthreads();
    return out;
}

__device__ __forceinline__ Borders no_borders() {
    Borders b;
    b.sure = kBins;
    b.kbin = kBins;
    b.p0 = 1;
    b.p1 = 0;
    b.krank = 0;
    b.kmass = b.pmass = b.total = 0;
    return b;
}

// ---- gather -------------------------------------------------------------------
template <class T>
__global__ void __launch_bounds__(kChunkThreads)
k_sample_gather(const T* __restrict__ x, RowSpace* __restrict__ spaces, SampleArgs a) {
    __shared__ uint32_t list[kChunkList];   // offsets from the chunk's first element
    __shared__ u64 sums[kMaxSubs];   // of the chunk's sub-chunks
    __shared__ uint32_t n_list, base;
    const int g = blockIdx.x;
    const int64_t r = blockIdx.y;
    RowSpace* ws = spaces + r;
    const T* row = x + r * a.ld;
    const int s0 = g * a.subs_per_chunk;
    const int subs = a.nsub - s0 < a.subs_per_chunk ? a.nsub - s0 : a.subs_per_chunk;
    const int64_t c0 = (int64_t)s0 * a.sub;
    const int64_t c1 = c0 + (int64_t)subs * a.sub < a.C ? c0 + (int64_t)subs * a.sub : a.C;
    const Params given = load_params(a, r);
    LaneBins bins;
    bins.load(ws);
    Share<T> ahead;
    ahead.load(row, c0, a.C, a.vec);   // binary32: in flight while the row's extremes and bins arrive
    u64 top;
    float low;
    row_extremes(ws, a.G, &top, &low);
    const Row q = make_row(a, given, top, low);
    const bool drawn = q.known == -2;
    const Borders b = drawn && (q.k || q.p < 1.0) ? find_borders(bins, q) : no_borders();
    if (g == 0 && threadIdx.x == 0) {
        ws->row = q;
        ws->borders = b;
    }
    if (!drawn) return;   // workgroup-uniform
    // border bins lie in sure .. last (p1 <= kbin)
    const bool borders = b.kbin < kBins || b.p0 <= b.p1;
    const int last = b.kbin < kBins ? b.kbin : b.p1;
    const float sure = (float)b.sure, past = (float)(last + 1);   // without borders the listed bits are not used
    const bool sift = (b.p0 <= b.p1 && b.kbin < kBins && b.kbin > b.p1 + 1) || last == kBins - 1;
    if (threadIdx.x == 0) n_list = 0;
    for (int i = threadIdx.x; i < subs; i += kChunkThreads) sums[i] = 0;
    __syncthreads();
    const int steps = a.sub / kSubMin;   // load steps of a sub-chunk
    int step = 0, sub = 0;
    u64 sum = 0;
    for (int64_t c = c0; c < c1; c += kSubMin) {
        const Share<T> e = ahead;
        if (c + kSubMin < c1) ahead.load(row, c + kSubMin, a.C, a.vec);
        uint32_t listed = 0;   // of this thread's elements, a bit each
#pragma unroll
        for (int h = 0; h < kPer; h += kTogether) {
            bool whole[kTogether], some = false;   // kept for sure unless min-p drops it
#pragma unroll
            for (int i = 0; i < kTogether; ++i) {
                const float d = q.below(e.v[h + i]);
                const float at = q.place(d);   // below n exactly where the bin is
                whole[i] = at < sure && d <= q.far;
                some |= whole[i];
                listed |= at >= sure && at < past ? 1u << (h + i) : 0u;
            }
            if (!__any(some)) continue;   // most steps of a wave, where few tokens are kept
            double w[kTogether];
            q.weights(e.v + h, w);
#pragma unroll
            for (int i = 0; i < kTogether; ++i) {
                u64 W = q.fixed(w[i]);
                asm volatile("" : "+v"(W));   // or a branch around each
                sum += whole[i] && w[i] >= q.min_p ? W : 0ull;
            }
        }
        if (borders && __any(listed != 0)) {
            if (sift) {   // bins between top-p's and top-k's, or elements without weight
                uint32_t kept = 0;
#pragma unroll
                for (int i = 0; i < kPer; ++i)
                    if ((listed >> i & 1) && border_bin(b, q.bin(e.v[i])) && q.fixed(q.weight(e.v[i]))) kept |= 1u << i;
                listed = kept;
            }
            // places in the list: the wave's from one atomic, a lane's after those of the lanes before it
            const uint32_t mine = (uint32_t)__popc(listed);
            const uint32_t upto = wave_scan_u32(mine);
            uint32_t at = 0;
            if (lane_id() == kWave - 1) at = atomicAdd(&n_list, upto);
            at = (uint32_t)__builtin_amdgcn_readlane((int)at, kWave - 1) + upto - mine;
            for (; listed; listed &= listed - 1, ++at)
                if (at < (uint32_t)kChunkList)
                    list[at] = (uint32_t)(c - c0) + (uint32_t)Share<T>::element(__ffs((int)listed) - 1, a.vec);
        }
        if (++step == steps || c + kSubMin >= c1) {
            sum = wave_sum_u64(sum);
            if (lane_id() == 0 && sum) atomicAdd(&sums[sub], sum);
            sum = 0;
            step = 0;
            ++sub;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < subs; i += kChunkThreads) ws->sum[s0 + i] = sums[i];
    if (!borders) return;   // workgroup-uniform
    __syncthreads();
    // more than kChunkList here, or kCand in all: the pick reads the row
    if (threadIdx.x == 0)
        base = n_list ? atomicAdd(&ws->ncand, n_list <= (uint32_t)kChunkList ? n_list : (uint32_t)kCand + 1u) : 0u;
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < n_list && i < (uint32_t)kChunkList && base + i < (uint32_t)kCand;
         i += kChunkThreads) {
        const int64_t c = c0 + list[i];
        ws->cand[base + i] = pack_key(order_image(Logit<T>::load(row + c)), (uint32_t)c);
    }
}

// ---- pick ---------------------------------------------------------------------
struct PickShared {
    u64 key[kCand];
    u64 W[kCand];        // the keys' weights
    u64 mass[256];
    uint32_t count[256];
    u64 sum[kMaxSubs];
    u64 prefix, left, some_set, some_clear, found_key;
    uint32_t hits;
    int64_t found;
    __device__ __forceinline__ void put(int i, u64 k, const Row& q) {
        key[i] = k;
        W[i] = q.fixed(q.weight(key_value(k)));
    }
    // A kept key's weight to its sub-chunk.
    __device__ __forceinline__ void keep(u64 k, u64 w, int sub_size) {
        atomicAdd(&sum[min(key_index(k) / (uint32_t)sub_size, (uint32_t)kMaxSubs - 1)], w);
    }
};

// Calls f(key, W) for this thread's share of the border elements: those of
// the list in LDS, or (row != nullptr) those of the row that lie in a border
// bin.
template <class T, class Fn>
__device__ __forceinline__ void each_listed(const PickShared& s, int n, const T* row, const Row& q, const Borders& b,
                                            int C, Fn f) {
    if (row) {
        for (int64_t c = threadIdx.x; c < C; c += kPickThreads) {
            const float v = Logit<T>::load(row + c);
            const u64 W = q.fixed(q.weight(v));
            if (W && border_bin(b, q.bin(v))) f(pack_key(order_image(v), (uint32_t)c), W);
        }
    } else {
        for (int i = threadIdx.x; i < n; i += kPickThreads) f(s.key[i], s.W[i]);
    }
}

// The largest key t such that the border elements with keys of at least t
// that `take` accepts number (BY_MASS: weigh) at least `want`; 0 when all of
// them together do not.  `want` >= 1.  A descent over the key's digits of up
// to eight bits below the bits that all accepted keys share, until one key is
// left; every thread returns the same key.
template <bool BY_MASS, class T, class Take>
__device__ __forceinline__ u64 select_key(PickShared& s, int n, const T* row, const Row& q, const Borders& b, int C,
                                          u64 want, Take take) {
    __syncthreads();
    if (threadIdx.x == 0) s.some_set = s.some_clear = 0;
    __syncthreads();
    u64 set = 0, clear = 0;
    each_listed(s, n, row, q, b, C, [&](u64 key, u64) {
        if (take(key)) {
            set |= key;
            clear |= ~key;
        }
    });
    set = wave_or_u64(set);
    clear = wave_or_u64(clear);
    if (lane_id() == kWave - 1 && (set | clear)) {
        atomicOr(&s.some_set, set);
        atomicOr(&s.some_clear, clear);
    }
    __syncthreads();
    if ((s.some_set | s.some_clear) == 0) return 0;   // none accepted
    const u64 diff = s.some_set & s.some_clear;
    int shift = diff ? 64 - __clzll((long long)diff) : 0;   // bits shift.. are shared
    u64 prefix = shift < 64 ? s.some_set >> shift << shift : 0;
    while (shift > 0) {
        const int bits = shift < 8 ? shift : 8;
        const int next = shift - bits;
        const u64 mask = shift < 64 ? ~0ull << shift : 0ull;
        __syncthreads();
        if (threadIdx.x < 256) {
            if (BY_MASS) s.mass[threadIdx.x] = 0;
            s.count[threadIdx.x] = 0;
        }
        __syncthreads();
        each_listed(s, n, row, q, b, C, [&](u64 key, u64 W) {
            if (take(key) && (key & mask) == prefix) {
                const int d = (int)((key >> next) & 255u) & ((1 << bits) - 1);
                if (BY_MASS) atomicAdd(&s.mass[d], W);
                atomicAdd(&s.count[d], 1u);
            }
        });
        __syncthreads();
        if (threadIdx.x < kWave) {   // digits from the top, four per lane
            const int lane = threadIdx.x;
            u64 v[4], in = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int d = 255 - (lane * 4 + i);
                v[i] = BY_MASS ? s.mass[d] : (u64)s.count[d];
                in += v[i];
            }
            u64 at = wave_scan_u64(in) - in;
            int digit = -1;
            u64 above = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (digit < 0 && at < want && at + v[i] >= want) {
                    digit = 255 - (lane * 4 + i);
                    above = at;
                }
                at += v[i];
            }
            const u64 hit = __ballot(digit >= 0);
            if (hit == 0) {
                if (lane == 0) s.hits = 0;
            } else {
                const int src = __ffsll((unsigned long long)hit) - 1;
                const int dg = __builtin_amdgcn_readlane(digit, src);
                const u64 ab = lane_u64(above, src);
                if (lane == 0) {
                    s.hits = s.count[dg];
                    s.prefix = prefix | ((u64)dg << next);
                    s.left = want - ab;
                }
            }
        }
        __syncthreads();
        const uint32_t hits = s.hits;
        if (hits == 0) return 0;   // fewer than wanted (only at the first digit)
        prefix = s.prefix;
        want = s.left;
        shift = next;
        if (hits == 1 && shift > 0) {   // one key has this prefix: the rest of its bits
            const u64 found = ~0ull << shift;
            each_listed(s, n, row, q, b, C, [&](u64 key, u64) {
                if (take(key) && (key & found) == prefix) s.found_key = key;
            });
            __syncthreads();
            return s.found_key;
        }
    }
    return prefix;
}

// The element of c0..c1 at which the kept weight passes u times the kept total
// (`before` is what is kept ahead of c0; whole: the range is the row and its
// own sum the total).
template <class T>
__device__ __forceinline__ void find_element(const T* row, const Row& q, const SampleArgs& a, u64 threshold, int64_t c0,
                                             int64_t c1, u64 before, u64 kept, bool whole, int64_t r) {
    const int64_t per = (c1 - c0 + kPickThreads - 1) / kPickThreads;   // consecutive elements per thread
    auto kept_weight = [&](int64_t c) -> u64 {
        const float v = Logit<T>::load(row + c);
        if (q.below(v) > q.far) return 0ull;
        const double w = q.weight(v);
        return w >= q.min_p && pack_key(order_image(v), (uint32_t)c) >= threshold ? q.fixed(w) : 0ull;
    };
    const int64_t a0 = c0 + per * threadIdx.x;
    const int64_t a1 = a0 + per < c1 ? a0 + per : c1;
    u64 mine = 0;
    for (int64_t c = a0; c < a1; ++c) mine += kept_weight(c);
    u64 all;
    const u64 upto = block_scan_u64<kPickThreads>(mine, &all);
    if (whole) kept = all;
    u64 t = (u64)(q.u * (double)kept);
    if (t >= kept) t = kept - 1;
    if (before + upto > t && before + upto - mine <= t) {   // exactly one thread
        u64 at = before + upto - mine;
        for (int64_t c = a0; c < a1; ++c) {
            at += kept_weight(c);
            if (at > t) {
                a.idx[r] = c;
                break;
            }
        }
    }
}

// The token, from the kept mass of every sub-chunk in s.sum.
template <class T>
__device__ __forceinline__ void draw_from_sums(PickShared& s, const T* row, const Row& q, const SampleArgs& a,
                                               u64 threshold, int64_t r) {
    u64 kept;
    const u64 mine = (int)threadIdx.x < a.nsub ? s.sum[threadIdx.x] : 0ull;
    const u64 upto = block_scan_u64<kPickThreads>(mine, &kept);
    u64 t = (u64)(q.u * (double)kept);
    if (t >= kept) t = kept - 1;
    if (upto > t && upto - mine <= t) {   // exactly one thread
        s.found = threadIdx.x;
        s.left = upto - mine;
    }
    __syncthreads();
    const int64_t c0 = s.found * a.sub;
    const int64_t c1 = c0 + a.sub < a.C ? c0 + a.sub : a.C;
    find_element<T>(row, q, a, threshold, c0, c1, s.left, kept, false, r);
}

// Resolves a row whose border elements are in s.key[0..n) or in `row`, and
// writes its token.  whole: the list is the whole row (nothing was summed).
template <class T>
__device__ __forceinline__ void pick_token(PickShared& s, int n, bool from_row, const T* row, const Row& q,
                                           const Borders& b, const SampleArgs& a, bool whole, int64_t r) {
    const T* scan = from_row ? row : nullptr;
    const int C = a.C;
    u64 threshold = 0;
    u64 kkey = 0;
    u64 total = b.total;
    if (b.kbin < kBins) {
        const int kbin = b.kbin;
        auto in_kbin = [&](u64 key) { return q.bin(key_value(key)) == kbin; };
        kkey = select_key<false>(s, n, scan, q, b, C, (u64)b.krank, in_kbin);
        threshold = kkey;
        if (q.p < 1.0) {   // the mass that top-k keeps
            u64 part = 0;
            each_listed(s, n, scan, q, b, C, [&](u64 key, u64 W) {
                if (in_kbin(key) && key >= kkey) part += W;
            });
            u64 all;
            block_scan_u64<kPickThreads>(part, &all);
            total = b.kmass + all;
        }
    }
    if (q.p < 1.0) {
        const int p0 = b.p0, p1 = b.p1;
        const u64 target = p_target(q.p, total);
        auto in_reach = [&](u64 key) {
            const int i = q.bin(key_value(key));
            return i >= p0 && i <= p1 && key >= kkey;
        };
        const u64 pkey = select_key<true>(s, n, scan, q, b, C, target > b.pmass ? target - b.pmass : 1ull, in_reach);
        if (pkey > threshold) threshold = pkey;
    }

    if (whole) {
        find_element<T>(row, q, a, threshold, 0, C, 0, 0, true, r);
        return;
    }
    __syncthreads();
    if (from_row) {
        // a wave's 64 consecutive elements lie in one sub-chunk
        for (int64_t base = (int64_t)(threadIdx.x / kWave) * kWave; base < C; base += kPickThreads) {
            const int64_t c = base + lane_id();
            u64 add = 0;
            if (c < C) {
                const float v = Logit<T>::load(row + c);
                const double w = q.weight(v);
                const u64 W = q.fixed(w);
                if (W && w >= q.min_p && border_bin(b, q.bin(v)) && q.bin(v) >= b.sure &&
                    pack_key(order_image(v), (uint32_t)c) >= threshold)
                    add = W;
            }
            add = wave_sum_u64(add);
            if (add && lane_id() == 0) atomicAdd(&s.sum[base / a.sub], add);
        }
    } else {
        for (int i = threadIdx.x; i < n; i += kPickThreads) {
            const u64 key = s.key[i];
            if (key >= threshold && q.weight(key_value(key)) >= q.min_p) s.keep(key, s.W[i], a.sub);
        }
    }
    __syncthreads();
    draw_from_sums<T>(s, row, q, a, threshold, r);
}

// The words of lane ^ 16 or lane ^ 32: the two copies trade their odd rows (or
// upper half) for even rows (lower half), which leaves every lane's partner in
// one of them.
template <int D>
__device__ __forceinline__ uint32_t swap_rows(uint32_t v) {
    static_assert(D == 16 || D == 32, "rows or halves");
    const auto p = D == 16 ? __builtin_amdgcn_permlane16_swap(v, v, false, false)
                           : __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return lane_id() & D ? p[0] : p[1];
}

template <int D>
__device__ __forceinline__ u64 lane_xor(u64 v) {   // the value of lane ^ D
    if constexpr (D == 1) return dpp_key<kQuadXor1, 0xF>(v);
    else if constexpr (D == 2) return dpp_key<kQuadXor2, 0xF>(v);
    else if constexpr (D == 4) return dpp_key<kQuadXor3, 0xF>(dpp_key<kHalfRowMirror, 0xF>(v));   // ^ 7, then ^ 3
    else if constexpr (D == 8) return dpp_key<kRowRotate8, 0xF>(v);
    else return (u64)swap_rows<D>((uint32_t)(v >> 32)) << 32 | swap_rows<D>((uint32_t)v);
}

// Sorts a key per thread of the first P (a power of two, from 64 to
// kPickThreads), largest first: a bitonic network, its exchanges within a wave
// on lane moves and those between waves through s.key, of which two halves take
// turns so that one barrier separates them.
__device__ __forceinline__ u64 sort_keys(PickShared& s, u64 key, int P) {
    const int tid = threadIdx.x;
    const bool in = tid < P;   // wave-uniform
    int half = 0;
    for (int k = 2; k <= P; k <<= 1) {   // sorted runs of k, every other one in ascending order
        const bool falling = (tid & k) == 0;
        auto exchange = [&](u64 other, int d) {
            if ((other > key) == (((tid & d) == 0) == falling)) key = other;
        };
        for (int d = k >> 1; d >= kWave; d >>= 1) {
            s.key[half + tid] = key;
            __syncthreads();
            exchange(s.key[half + (tid ^ d)], d);
            half ^= kPickThreads;
        }
        if (in) {
            if (k > 32) exchange(lane_xor<32>(key), 32);
            if (k > 16) exchange(lane_xor<16>(key), 16);
            if (k > 8) exchange(lane_xor<8>(key), 8);
            if (k > 4) exchange(lane_xor<4>(key), 4);
            if (k > 2) exchange(lane_xor<2>(key), 2);
            exchange(lane_xor<1>(key), 1);
        }
    }
    return key;
}

// As pick_token, for a list of at most a key per thread (this thread's: `key`,
// 0 past n): sorted, so that the border of top-k is a place and that of top-p a
// running sum.  Entered with s.hits = 0 and s.found_key = ~0.
template <class T>
__device__ __forceinline__ void pick_sorted(PickShared& s, int n, u64 key, const T* row, const Row& q, const Borders& b,
                                            const SampleArgs& a, int64_t r) {
    int P = kWave;
    while (P < n) P <<= 1;
    key = sort_keys(s, key, P);
    const int place = threadIdx.x;
    const bool have = place < n;
    double w = 0.0;
    u64 W = 0;
    int bin = kBins;
    if (have) {
        const float v = key_value(key);
        w = q.weight(v);
        W = q.fixed(w);
        bin = q.bin(v);
    }
    // listed keys of bins ahead of kbin, and the mass of those of p0..p1 ahead of this one
    const u64 ahead = __ballot(have && bin < b.kbin);
    if (lane_id() == 0 && ahead) atomicAdd(&s.hits, (uint32_t)__popcll(ahead));
    const bool in_p = have && bin >= b.p0 && bin <= b.p1;
    u64 all;
    const u64 mass = block_scan_u64<kPickThreads>(in_p ? W : 0ull, &all) - (in_p ? W : 0ull);
    bool keep = have && (bin != b.kbin || (uint32_t)place - s.hits < b.krank);
    if (q.p < 1.0) {
        u64 total = b.total;
        if (b.kbin < kBins) {   // the mass that top-k keeps
            block_scan_u64<kPickThreads>(keep && bin == b.kbin ? W : 0ull, &all);
            total = b.kmass + all;
        }
        keep = keep && in_p && b.pmass + mass < p_target(q.p, total);
    }
    const u64 kept = __ballot(keep);
    if (kept) {   // wave-uniform; the wave's smallest kept key is its last
        const u64 least = lane_u64(key, 63 - __clzll((long long)kept));
        if (lane_id() == 0) atomicMin(&s.found_key, least);
    }
    if (keep && w >= q.min_p) s.keep(key, W, a.sub);
    __syncthreads();
    draw_from_sums<T>(s, row, q, a, n ? s.found_key : 0ull, r);
}

template <class T>
__global__ void __launch_bounds__(kPickThreads)
k_sample_pick(const T* __restrict__ x, RowSpace* __restrict__ spaces, SampleArgs a) {
    __shared__ PickShared s;
    const int64_t r = blockIdx.x;
    RowSpace* ws = spaces + r;
    const u64 first = ws->cand[threadIdx.x];   // most lists are no longer; used only if so many are listed
    const u64 sum = (int)threadIdx.x < a.nsub ? ws->sum[threadIdx.x] : 0ull;
    const uint32_t listed = ws->ncand;
    const Row q = ws->row;
    const Borders b = ws->borders;
    if (q.known != -2) {   // workgroup-uniform
        if (threadIdx.x == 0) a.idx[r] = q.known;
        return;
    }
    if (listed <= (uint32_t)kWave && a.nsub <= kWave) {
        // A short list and few sub-chunks, one of each per lane: the first wave
        // settles the borders by comparing every listed key with every other.
        if (threadIdx.x < kWave) {
            const int lane = threadIdx.x;
            const int n = (int)listed;
            const bool have = lane < n;
            const u64 key = have ? first : 0ull;
            const float v = key_value(key);
            const double w = have ? q.weight(v) : 0.0;
            const u64 W = have ? q.fixed(w) : 0ull;
            const int bin = have ? q.bin(v) : kBins;
            const u64 in_k = __ballot(have && bin == b.kbin);
            const u64 in_p = __ballot(have && bin >= b.p0 && bin <= b.p1);
            uint32_t ahead = 0;   // keys of kbin before this one
            u64 mass = 0;         // mass of the keys of p0..p1 before this one
            for (int j = 0; j < n; ++j) {
                const u64 Wj = lane_u64(W, j);   // with every lane active: lane j's own comparison is false
                const bool before = lane_u64(key, j) > key;
                ahead += before && (in_k >> j & 1) ? 1u : 0u;
                mass += before && (in_p >> j & 1) ? Wj : 0ull;
            }
            bool keep = have && (bin != b.kbin || ahead < b.krank);
            if (q.p < 1.0) {
                u64 total = b.total;
                if (b.kbin < kBins) total = b.kmass + wave_sum_u64(keep && bin == b.kbin ? W : 0ull);
                keep = keep && (in_p >> lane & 1) && b.pmass + mass < p_target(q.p, total);
            }
            // the smallest kept key (0, all of them, where nothing is listed)
            const u64 threshold = n ? ~wave_max_u64(keep ? ~key : 0ull) : 0ull;
            s.sum[lane] = sum;
            if (keep && w >= q.min_p) atomicAdd(&s.sum[min(key_index(key) / (uint32_t)a.sub, (uint32_t)kWave - 1)], W);
            // other lanes' additions, too: without the clobber the compiler reads
            // back only in lanes that added something themselves
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            const u64 mine = s.sum[lane];
            const u64 upto = wave_scan_u64(mine);
            const u64 kept = lane_u64(upto, kWave - 1);
            u64 t = (u64)(q.u * (double)kept);
            if (t >= kept) t = kept - 1;
            const u64 hit = __ballot(upto > t);   // the first sub-chunk to pass u
            const int src = hit ? __ffsll((unsigned long long)hit) - 1 : 0;
            if (lane == 0) {
                s.prefix = threshold;
                s.some_set = kept;
                s.left = lane_u64(upto, src) - lane_u64(mine, src);
                s.found = src;
            }
        }
        __syncthreads();
        const int64_t c0 = s.found * a.sub;
        const int64_t c1 = c0 + a.sub < a.C ? c0 + a.sub : a.C;
        find_element<T>(x + r * a.ld, q, a, s.prefix, c0, c1, s.left, s.some_set, false, r);
        return;
    }
    const bool from_row = listed > (uint32_t)kCand;
    const int n = from_row ? 0 : (int)listed;
    const bool sorted = listed <= (uint32_t)kPickThreads;
    if (!sorted)
        for (int i = threadIdx.x; i < n; i += kPickThreads) s.put(i, i < kPickThreads ? first : ws->cand[i], q);
    s.sum[threadIdx.x] = sum;
    if (threadIdx.x == 0) {
        s.found = s.left = 0;
        s.hits = 0;
        s.found_key = ~0ull;
    }
    __syncthreads();
    if (sorted) {
        pick_sorted<T>(s, n, (int)threadIdx.x < n ? first : 0ull, x + r * a.ld, q, b, a, r);
        return;
    }
    pick_token<T>(s, n, from_row, x + r * a.ld, q, b, a, false, r);
}

// A row of at most kCand elements: every element is listed, in one bin.
template <class T>
__global__ void __launch_bounds__(kPickThreads)
k_sample_row(const T* __restrict__ x, SampleArgs a) {
    __shared__ PickShared s;
    __shared__ u64 keys[kPickThreads / kWave];
    const int64_t r = blockIdx.x;
    const T* row = x + r * a.ld;
    u64 top = 0;
    for (int c = threadIdx.x; c < a.C; c += kPickThreads) {
        const u64 key = pack_key(order_image(Logit<T>::load(row + c)), (uint32_t)c);
        s.key[c] = key;
        top = umax64(top, key);
    }
    top = wave_max_u64(top);
    if (lane_id() == 0) keys[threadIdx.x / kWave] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kPickThreads / kWave; ++w) top = umax64(top, keys[w]);
    Row q = make_row(a, load_params(a, r), top, 0.0f);
    if (q.known != -2) {   // workgroup-uniform
        if (threadIdx.x == 0) a.idx[r] = q.known;
        return;
    }
    q.scale = 0.0f;
    Borders b = no_borders();
    if (q.k) {
        b.kbin = 0;
        b.krank = (uint32_t)q.k;
    }
    if (q.p < 1.0) {
        b.p0 = 0;
        b.p1 = 0;
        u64 mass = 0;
        for (int c = threadIdx.x; c < a.C; c += kPickThreads) {   // this thread's own keys
            s.put(c, s.key[c], q);
            mass += s.W[c];
        }
        block_scan_u64<kPickThreads>(mass, &b.total);
    }
    pick_token<T>(s, a.C, false, row, q, b, a, true, r);
}

// ---- host ---------------------------------------------------------------------
// The arguments for rows r0 .. r0 + R - 1.
SampleArgs plan_rows(const SampleRows& p, int64_t r0, int64_t R) {
    const int64_t C = p.C;
    SampleArgs a{};
    a.u = p.u + r0;
    a.temperature = p.temperature ? p.temperature + r0 : nullptr;
    a.top_k = p.top_k ? p.top_k + r0 : nullptr;
    a.top_p = p.top_p ? p.top_p + r0 : nullptr;
    a.min_p = p.min_p ? p.min_p + r0 : nullptr;
    a.idx = p.idx + r0;
    a.ld = p.ld;
    a.C = (int)C;
    const int size = p.dtype == DG_DTYPE_F32 ? 4 : 2;
    a.vec = (uintptr_t)p.x % 16 == 0 && p.ld * size % 16 == 0;
    int bits = 0;
    while (((int64_t)1 << bits) < C) ++bits;
    a.F = 62 - bits < 51 ? 62 - bits : 51;
    int64_t sub = (C + kMaxSubs - 1) / kMaxSubs;
    sub = (sub + kSubMin - 1) / kSubMin * kSubMin;
    a.sub = (int)sub;
    a.nsub = (int)((C + sub - 1) / sub);
    int64_t G = (kTargetGroups + R - 1) / R;
    if (G > a.nsub) G = a.nsub;
    a.subs_per_chunk = (int)((a.nsub + G - 1) / G);
    a.G = (a.nsub + a.subs_per_chunk - 1) / a.subs_per_chunk;
    return a;
}

template <class T>
hipError_t launch_sample(const SampleRows& p, hipStream_t s) {
    const T* x = (const T*)p.x;
    if (p.C <= kCand) {
        for (int64_t r0 = 0; r0 < p.R; r0 += kMaxGroupsPerLaunch) {
            const int64_t rn = p.R - r0 < kMaxGroupsPerLaunch ? p.R - r0 : kMaxGroupsPerLaunch;
            hipLaunchKernelGGL((k_sample_row<T>), dim3((unsigned)rn), dim3(kPickThreads), 0, s, x + r0 * p.ld,
                               plan_rows(p, r0, rn));
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
        return hipSuccess;
    }
    RowSpace* ws = (RowSpace*)p.ws;
    for (int64_t r0 = 0; r0 < p.R; r0 += kBatchRows) {
        const int64_t rn = p.R - r0 < kBatchRows ? p.R - r0 : kBatchRows;
        const SampleArgs a = plan_rows(p, r0, rn);
        const T* xr = x + r0 * p.ld;
        const dim3 chunks((unsigned)a.G, (unsigned)rn);
        hipLaunchKernelGGL((k_sample_max<T>), chunks, dim3(kChunkThreads), 0, s, xr, ws, a);
        if (p.top_k || p.top_p)
            hipLaunchKernelGGL((k_sample_hist<T>), chunks, dim3(kChunkThreads), 0, s, xr, ws, a);
        hipLaunchKernelGGL((k_sample_gather<T>), chunks, dim3(kChunkThreads), 0, s, xr, ws, a);
        hipLaunchKernelGGL((k_sample_pick<T>), dim3((unsigned)rn), dim3(kPickThreads), 0, s, xr, ws, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

size_t sample_workspace_bytes(int64_t R, int64_t C) {
    if (R <= 0 || C <= kCand) return 0;
    return (size_t)(R < kBatchRows ? R : kBatchRows) * sizeof(RowSpace);
}

hipError_t launch_sample_rows(const SampleRows& p, hipStream_t s) {
    switch (p.dtype) {
        case DG_DTYPE_F32: return launch_sample<float>(p, s);
        case DG_DTYPE_F16: return launch_sample<_Float16>(p, s);
        case DG_DTYPE_BF16: return launch_sample<__bf16>(p, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace dg
