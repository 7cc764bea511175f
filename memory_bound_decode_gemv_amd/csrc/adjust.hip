// adjust.hip -- penalties for repeated tokens, biases and grammar masks on rows
// of logits, in one pass over the row.
//
//   v = x[c];  in the history: v > 0 ? v / rep : v rep;  n times in the output: (v - freq n) - pres;
//   v + bias;  -infinity where the mask has no bit
//
// A workgroup takes a chunk of one row's vocabulary, up to 64 KiB of logits in
// its registers.  It counts the row's history into a table in LDS, one word per
// token of the chunk: the low bits the number of times it is in the output, the
// top bit whether it is in the prompt.  LDS additions of whole numbers: the
// counts do not depend on their order.  Words of 16 bits, two to a dword, where
// no count can reach the top bit (T <= 32767) and a logit fits, else of 32.
//
// Every chunk of a row reads the whole history, so chunks are as large as leaves
// enough workgroups.  Few tokens of a chunk are in a history, but few waves have
// none: with the arithmetic at the elements nearly every wave ran it.  So the
// first to count a token lists it, the listed tokens are worked off side by side,
// and the result takes the place of the token's count; a bit per token says
// where.  One wave goes through the row's biases from the end, 64 at a time, and
// marks which entries are the last of their token, and those tokens, which are
// worked off by the entries.
//
// The first tokens and, of a chunk without a mask or a partial group, all logits are
// on their way before the first wait; a group's word of the mask, and each logit of a
// row's last, partial group, is waited for by itself.  What bounds it are the steps that
// follow one another (tokens, table, list, results, stores; three barriers), the stores
// of unchanged logits behind the counts: one row of 128256 binary32 logits 4.5 us, 64 of
// bfloat16 with histories of 4096 to 8192 12.9, in place too (34 MB, 2.6 TB/s; the vector
// unit active in a quarter of the busy cycles).
#include <algorithm>

#include "dg_batch.h"
#include "q4_common.h"

#pragma clang fp contract(off)

namespace dg {
namespace {

using q4::lds_barrier;

constexpr int kThreads = 1024;
constexpr int kScan = 2;             // 16-byte loads of tokens in flight per thread

typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));   // rows of 16-bit values at any place

struct AdjustArgs {
    dg_adjustments a;
    int64_t ld, ldy, first;
    int C, chunks;
};

__device__ __forceinline__ int clampi(int v, int hi) { return min(max(v, 0), hi); }

template <class E> struct Bits;
template <> struct Bits<float> { using type = uint32_t; };
template <> struct Bits<_Float16> { using type = uint16_t; };
template <> struct Bits<__bf16> { using type = uint16_t; };

// The table of words W (16 bits, two to a dword, or 32).
template <class W>
struct Table {
    static constexpr bool kWide = sizeof(W) == 4;
    static constexpr uint32_t kPrompt = kWide ? 0x80000000u : 0x8000u;
    // Counts token t; true for the first time it comes.
    __device__ __forceinline__ static bool add(W* table, uint32_t t, bool prompt) {
        uint32_t* const w = reinterpret_cast<uint32_t*>(table) + (kWide ? t : t >> 1);
        const uint32_t s = kWide ? 0 : 16 * (t & 1);
        const uint32_t old = prompt ? atomicOr(w, kPrompt << s) : atomicAdd(w, 1u << s);
        return kWide ? old == 0 : ((old >> s) & 0xFFFFu) == 0;
    }
};

// E: the logits' type; W: the table's words, no narrower; G: 16-byte groups per
// thread.
template <class E, class W, int G>
__global__ void __launch_bounds__(kThreads) k_adjust(const E* x, E* y, AdjustArgs p) {
    constexpr int V = 16 / sizeof(E);          // elements of a group
    constexpr int kChunk = kThreads * V * G;   // tokens of a workgroup
    using Raw = typename Bits<E>::type;
    static_assert(sizeof(W) >= sizeof(Raw), "a result in the place of a count");
    extern __shared__ u32x4 adjust_lds[];
    __shared__ uint32_t listed;
    const dg_adjustments& a = p.a;
    W* const table = reinterpret_cast<W*>(adjust_lds);
    uint32_t* const changed = reinterpret_cast<uint32_t*>(table + kChunk);   // a bit per token
    uint64_t* const last = reinterpret_cast<uint64_t*>(changed + kChunk / 32);   // a bit per entry of the bias list
    uint16_t* const list = reinterpret_cast<uint16_t*>(last + (a.bias ? (a.B + 63) / 64 : 0));
    const int tid = threadIdx.x;
    const int64_t b = p.first + blockIdx.x;
    const int64_t r = b / p.chunks;
    const int c0 = (int)(b - r * p.chunks) * kChunk;
    const int n = min(kChunk, p.C - c0);
    const E* const xr = x + r * p.ld + c0;
    E* const yr = y + r * p.ldy + c0;

    // Asked for before anything is worked off: the first tokens (of the T that a row
    // may have, before its length is known), the biased tokens, the logits and the
    // mask.  As compiled, a word of the mask and a logit of a partial group are each
    // waited for where they are read.
    const int T = a.tokens ? (int)a.T : 0;
    const int32_t* const tok = a.tokens + r * a.ldt;
    u32x4 t[kScan];
    auto load_tokens = [&](int i0) {   // four at a time, never past the row's end
#pragma unroll
        for (int s = 0; s < kScan; ++s)
            t[s] = *reinterpret_cast<const u32x4_a4*>(tok + min(i0 + s * kThreads * 4, T - 4));
    };
    if (T >= 4) load_tokens(tid * 4);
    else if (tid < T) t[0].x = (uint32_t)tok[tid];
    const int B = a.bias ? (int)a.B : 0;
    const bool bias_wave = tid >= kThreads - kWave;
    uint32_t bias_id = ~0u;
    if (bias_wave && lane_id() < B) bias_id = (uint32_t)a.bias_ids[r * a.B + lane_id()];

    union Group {
        u32x4 v;
        E e[V];
        Raw raw[V];
    } q[G];
    uint32_t allowed[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const int i = (g * kThreads + tid) * V;
        if (i + V <= n) {
            q[g].v = *reinterpret_cast<const u32x4_a2*>(xr + i);
        } else {
            q[g].v = u32x4{0, 0, 0, 0};
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (i + e < n) q[g].e[e] = xr[i + e];
        }
        allowed[g] = ~0u;
        if (a.mask && i < n) allowed[g] = a.mask[r * a.ldm + ((c0 + i) >> 5)] >> ((c0 + i) & 31);
    }

    const int len = a.tokens ? clampi(a.lens ? a.lens[r] : T, T) : 0;
    const int prompt = a.prompt_lens ? clampi(a.prompt_lens[r], len) : 0;
    const int biases = a.bias ? clampi(a.bias_lens ? a.bias_lens[r] : B, B) : 0;
    const bool some = len > 0 || biases > 0;   // workgroup-uniform
    if (some) {
        constexpr int kZero = (int)(kChunk * sizeof(W) + kChunk / 8) / 16;   // the table and the bits
        for (int i = tid; i < kZero; i += kThreads) adjust_lds[i] = u32x4{0, 0, 0, 0};
        if (tid == 0) listed = 0;
        lds_barrier();
        auto take = [&](uint32_t c, bool in_prompt) {
            if (c < (uint32_t)n && Table<W>::add(table, c, in_prompt)) list[atomicAdd(&listed, 1u)] = (uint16_t)c;
        };
        if (T >= 4) {
            for (int i0 = tid * 4; i0 < len; i0 += kThreads * 4 * kScan) {
                if (i0 != tid * 4) load_tokens(i0);
#pragma unroll
                for (int s = 0; s < kScan; ++s) {
                    const int i = i0 + s * kThreads * 4;
                    if (i >= len) continue;
                    if (__all(i + 4 <= len)) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) take(t[s][e] - (uint32_t)c0, i + e < prompt);
                    } else {   // the last four of the row may overlap others: a thread counts from its own first on
                        const int at = min(i, T - 4);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            take(at + e >= i && at + e < len ? t[s][e] - (uint32_t)c0 : ~0u, at + e < prompt);
                    }
                }
            }
        } else if (tid < len) {
            take(t[0].x - (uint32_t)c0, tid < prompt);
        }
        if (biases > 0 && bias_wave) {
            for (int k = (biases - 1) / kWave; k >= 0; --k) {
                const int i = k * kWave + lane_id();
                if (k > 0) bias_id = i < biases ? (uint32_t)a.bias_ids[r * a.B + i] : ~0u;
                else if (biases > kWave) bias_id = (uint32_t)a.bias_ids[r * a.B + i];
                const uint32_t c = i < biases ? bias_id - (uint32_t)c0 : ~0u;
                const uint32_t bit = 1u << (c & 31);
                const uint64_t inside = __ballot(c < (uint32_t)n);
                const bool set = c < (uint32_t)n && (atomicOr(changed + (c >> 5), bit) & bit);
                bool mine = c < (uint32_t)n;
                for (uint64_t m = __ballot(set); m != 0;) {   // tokens that came before, in these 64 or behind them
                    const uint32_t cl = (uint32_t)__builtin_amdgcn_readlane((int)c, __builtin_ctzll(m));
                    const uint64_t same = __ballot(c == cl) & inside;
                    const bool here = (same & ~__ballot(set)) != 0;   // one of these marked it: the last one counts
                    if (c == cl) mine = here && lane_id() == 63 - __builtin_clzll(same);
                    m &= ~same;
                }
                const uint64_t m = __ballot(mine);
                if (lane_id() == 0) last[k] = m;
            }
        }
        lds_barrier();
        float rep = a.repetition ? a.repetition[r] : 1.0f;
        if (!(rep > 0.0f)) rep = 1.0f;
        const float freq = a.frequency ? a.frequency[r] : 0.0f;
        const float pres = a.presence ? a.presence[r] : 0.0f;
        auto penalties = [&](float v, uint32_t k) {   // k: the token's count
            if (k == 0) return v;
            v = rep == 1.0f ? v : v > 0.0f ? v / rep : v * rep;
            const uint32_t out = k & (Table<W>::kPrompt - 1);
            return out == 0 ? v : (v - freq * (float)out) - pres;
        };
        auto result = [&](int c, float v) {
            const E e = (E)bind_f32(v);
            table[c] = (W)__builtin_bit_cast(Raw, e);
        };
        for (int i = tid; i < biases; i += kThreads) {
            if (!((last[i >> 6] >> (i & 63)) & 1u)) continue;
            const int c = a.bias_ids[r * a.B + i] - c0;
            result(c, penalties((float)xr[c], table[c]) + a.bias[r * a.B + i]);
        }
        const int m = len > 0 ? (int)listed : 0;
        for (int j = tid; j < m; j += kThreads) {
            const int c = list[j];
            const float v = (float)xr[c];
            const uint32_t bit = 1u << (c & 31);
            if (!(atomicOr(changed + (c >> 5), bit) & bit)) result(c, penalties(v, table[c]));   // else a biased one
        }
        lds_barrier();
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const int i = (g * kThreads + tid) * V;
        if (i >= n) continue;
        if (some) {
            const uint32_t bits = changed[i >> 5] >> (i & 31);
            if (bits & ((1u << V) - 1)) {
#pragma unroll
                for (int e = 0; e < V; ++e)
                    if ((bits >> e) & 1u) q[g].raw[e] = (Raw)table[i + e];
            }
        }
        if (a.mask) {
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (!((allowed[g] >> e) & 1u)) q[g].e[e] = (E)-__builtin_huge_valf();
        }
        if (i + V <= n) {
            *reinterpret_cast<u32x4_a2*>(yr + i) = q[g].v;
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (i + e < n) yr[i + e] = q[g].e[e];
        }
    }
}

template <class E, class W, int G>
struct Config {
    static constexpr int kChunk = kThreads * (16 / (int)sizeof(E)) * G;
    // The table, the bits, the biases' marks and the list: tokens of a history, at most a chunk's.
    static constexpr size_t bytes(bool table, int64_t biases, int64_t tokens) {
        return (table ? kChunk * sizeof(W) + kChunk / 8 : 0) + (size_t)(biases + 63) / 64 * 8 +
               (size_t)std::min<int64_t>(tokens, kChunk) * 2;
    }
    static_assert(bytes(true, 65535, kChunk) <= 160 * 1024 - 256, "every call fits");
    static size_t lds(const AdjustRows& q) {
        return bytes(q.a.tokens || q.a.bias, q.a.bias ? q.a.B : 0, q.a.tokens ? q.a.T : 0);
    }
    static hipError_t launch(const AdjustRows& q, hipStream_t s) {
        AdjustArgs p{q.a, q.ld, q.ldy, 0, (int)q.C, (int)((q.C + kChunk - 1) / kChunk)};
        const int64_t all = q.R * p.chunks;
        hipError_t e = hipSuccess;
        for (; p.first < all && e == hipSuccess; p.first += kMaxGroupsPerLaunch) {
            hipLaunchKernelGGL((k_adjust<E, W, G>), dim3((unsigned)std::min<int64_t>(all - p.first, kMaxGroupsPerLaunch)),
                               dim3(kThreads), lds(q), s, (const E*)q.x, (E*)q.y, p);
            e = hipGetLastError();
        }
        return e;
    }
};

// Chunks of four 16-byte groups a thread from 1024 single-group chunks on, of two
// from 512, else of one (us in graphs, GPU alone, 1 / 2 / 4 groups): 64 rows of
// 128256 bfloat16 with histories of 4096 to 8192 tokens 16.9 / 13.4 / 12.9; 200 of
// 32003 binary16 with 500 to 1000 tokens and a mask 13.8 / 11.0 / 11.7; one of
// 128256 binary32 4.5 / 5.0 / 5.8.  Four groups of 16-bit logits and 32-bit words
// (T > 32767) would need 196 KiB of LDS for the table and the list: two.  T counts here
// and for the words, not the lengths, which the host does not know: the 64 rows above
// 12.7 with T = 8192 and 32767, 16.8 with 65536; the 200 11.3, 12.5 and 16.0 with 1000,
// 32767 and 65536.
template <class E, class W>
hipError_t adjust_words(const AdjustRows& q, hipStream_t s) {
    const int64_t groups = q.R * ((q.C + Config<E, W, 1>::kChunk - 1) / Config<E, W, 1>::kChunk);
    if constexpr (sizeof(E) == sizeof(W))
        if (groups >= 1024) return Config<E, W, 4>::launch(q, s);
    if (groups >= 512) return Config<E, W, 2>::launch(q, s);
    return Config<E, W, 1>::launch(q, s);
}

template <class E>
hipError_t adjust(const AdjustRows& q, hipStream_t s) {
    if constexpr (sizeof(E) == 2)
        if (!q.a.tokens || q.a.T <= 32767) return adjust_words<E, uint16_t>(q, s);
    return adjust_words<E, uint32_t>(q, s);
}

}  // namespace

hipError_t launch_adjust_rows(const AdjustRows& q, hipStream_t s) {
    if (q.dtype == DG_DTYPE_F32) return adjust<float>(q, s);
    if (q.dtype == DG_DTYPE_F16) return adjust<_Float16>(q, s);
    return adjust<__bf16>(q, s);
}

}  // namespace dg
