// adjust.hip -- penalties for repeated tokens, biases and grammar masks on rows
// of logits, in one pass over the row.
//
//   v = x[c];  in the history: v > 0 ? v / rep : v rep;  n times in the output: (v - freq n) - pres;
//   v + bias;  -infinity where the mask has no bit
//
// A workgroup takes a chunk of one row's vocabulary.  It counts the row's
// history into a table in LDS, one 32-bit word per token of the chunk: the low 31
// bits the number of times it is in the output, the top bit whether it is in
// the prompt.  LDS additions of whole numbers: the counts do not depend on their
// order.  A second table holds 1 + the last place of the token in the bias list.
#include <algorithm>

#include "dg_device.h"
#include "dg_internal.h"

#pragma clang fp contract(off)

namespace dg {
namespace {

constexpr int kChunk = 8192;     // tokens of a workgroup
constexpr int kThreads = 512;

struct AdjustArgs {
    dg_adjustments a;
    int64_t ld, ldy, first;
    int C, chunks;
};

__device__ __forceinline__ int clampi(int v, int hi) { return min(max(v, 0), hi); }

template <class T>
__global__ void __launch_bounds__(kThreads) k_adjust(const T* x, T* y, AdjustArgs p) {
    __shared__ uint32_t count[kChunk];
    __shared__ uint32_t place[kChunk];
    const int64_t b = p.first + blockIdx.x;
    const int64_t r = b / p.chunks;
    const int c0 = (int)(b - r * p.chunks) * kChunk;
    const int n = min(kChunk, p.C - c0);
    const dg_adjustments& a = p.a;
    const int len = a.tokens ? clampi(a.lens ? a.lens[r] : (int)a.T, (int)a.T) : 0;
    const int prompt = a.prompt_lens ? clampi(a.prompt_lens[r], len) : 0;
    const int biases = a.bias ? clampi(a.bias_lens ? a.bias_lens[r] : (int)a.B, (int)a.B) : 0;
    if (len > 0)
        for (int i = threadIdx.x; i < n; i += kThreads) count[i] = 0;
    if (biases > 0)
        for (int i = threadIdx.x; i < n; i += kThreads) place[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < len; i += kThreads) {
        const uint32_t t = (uint32_t)(a.tokens[r * a.ldt + i] - c0);
        if (t < (uint32_t)n) {
            if (i < prompt) atomicOr(&count[t], 0x80000000u);
            else atomicAdd(&count[t], 1u);
        }
    }
    for (int i = threadIdx.x; i < biases; i += kThreads) {
        const uint32_t t = (uint32_t)(a.bias_ids[r * a.B + i] - c0);
        if (t < (uint32_t)n) atomicMax(&place[t], (uint32_t)i + 1u);
    }
    __syncthreads();
    float rep = a.repetition ? a.repetition[r] : 1.0f;
    if (!(rep > 0.0f)) rep = 1.0f;
    const float freq = a.frequency ? a.frequency[r] : 0.0f;
    const float pres = a.presence ? a.presence[r] : 0.0f;
    for (int i = threadIdx.x; i < n; i += kThreads) {
        float v = (float)x[r * p.ld + c0 + i];
        if (len > 0) {
            const uint32_t k = count[i];
            if (k != 0 && rep != 1.0f) v = v > 0.0f ? v / rep : v * rep;
            const uint32_t out = k & 0x7FFFFFFFu;
            if (out != 0) v = bind_f32(v - bind_f32(freq * (float)out)) - pres;
        }
        if (biases > 0) {
            const uint32_t at = place[i];
            if (at != 0) v = v + a.bias[r * a.B + (at - 1)];
        }
        if (a.mask && !((a.mask[r * a.ldm + ((c0 + i) >> 5)] >> ((c0 + i) & 31)) & 1u)) v = -__builtin_huge_valf();
        y[r * p.ldy + c0 + i] = (T)bind_f32(v);
    }
}

template <class T>
hipError_t adjust(const AdjustRows& q, hipStream_t s) {
    AdjustArgs p{q.a, q.ld, q.ldy, 0, (int)q.C, (int)((q.C + kChunk - 1) / kChunk)};
    const int64_t all = q.R * p.chunks;
    hipError_t e = hipSuccess;
    for (; p.first < all && e == hipSuccess; p.first += kMaxGroupsPerLaunch) {
        hipLaunchKernelGGL((k_adjust<T>), dim3((unsigned)std::min<int64_t>(all - p.first, kMaxGroupsPerLaunch)),
                           dim3(kThreads), 0, s, (const T*)q.x, (T*)q.y, p);
        e = hipGetLastError();
    }
    return e;
}

}  // namespace

hipError_t launch_adjust_rows(const AdjustRows& q, hipStream_t s) {
    if (q.dtype == DG_DTYPE_F32) return adjust<float>(q, s);
    if (q.dtype == DG_DTYPE_F16) return adjust<_Float16>(q, s);
    return adjust<__bf16>(q, s);
}

}  // namespace dg
