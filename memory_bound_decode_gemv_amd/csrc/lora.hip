// lora.hip -- low-rank adapters of many requests beside a shared projection:
//
//   h[m][r] = sum_k A[a][r][k] x[m][k],  Y[m][n] = base[m][n] + scale[a] sum_r B[a][n][r] h[m][r],  a = adapter[m]
//
// Two launches: h (one wave per row and rank) into the workspace, then Y (one
// thread per output).
#include <algorithm>

#include "dg_device.h"
#include "dg_internal.h"

namespace dg {
namespace {

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

template <class E>
__device__ __forceinline__ void load8(const typename E::raw* p, float (&v)[8]) {
    constexpr int kVecs = sizeof(typename E::raw) / 2;
    union {
        u32x4 q[kVecs];
        typename E::raw e[8];
    } b;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) b.q[i] = reinterpret_cast<const u32x4*>(p)[i];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = E::widen(b.e[i]);
}

struct LoraArgs {
    const int32_t *adapter, *ranks;
    const float* scale;
    int64_t N, ld, first;
    int K, R, L;
    int parts;   // workgroups per row
};

__device__ __forceinline__ int rank_of(const LoraArgs& a, int ad) {
    return a.ranks ? min(max(a.ranks[ad], 0), a.R) : a.R;
}

constexpr int kShrinkWaves = 4;

template <class EX, class EW>
__global__ void __launch_bounds__(64 * kShrinkWaves)
k_lora_shrink(const typename EX::raw* __restrict__ x, const typename EW::raw* __restrict__ A, float* __restrict__ h,
              LoraArgs a) {
    const int64_t b = a.first + blockIdx.x;
    const int64_t m = b / a.parts;
    const int r = (int)(b - m * a.parts) * kShrinkWaves + __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int ad = a.adapter[m];
    if (ad < 0 || ad >= a.L || r >= rank_of(a, ad)) return;
    const typename EX::raw* const xr = x + m * a.ld;
    const typename EW::raw* const Ar = A + ((size_t)ad * a.R + r) * a.K;
    float sum = 0.0f;
    for (int k = lane_id() * 8; k < a.K; k += 512) {
        float w[8], v[8];
        load8<EW>(Ar + k, w);
        load8<EX>(xr + k, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fmaf(w[i], v[i], sum);
    }
    sum = wave_sum_f32(sum);
    if (lane_id() == 0) h[m * a.R + r] = sum;
}

constexpr int kExpandThreads = 256;

template <class EW>
__global__ void __launch_bounds__(kExpandThreads)
k_lora_expand(const typename EW::raw* __restrict__ B, const float* __restrict__ h, const float* base, float* Y,
              LoraArgs a) {
    const int64_t b = a.first + blockIdx.x;
    const int64_t m = b / a.parts;
    const int64_t n = (b - m * a.parts) * kExpandThreads + threadIdx.x;
    if (n >= a.N) return;
    const int ad = a.adapter[m];
    float y = base ? base[m * a.N + n] : 0.0f;
    if (ad >= 0 && ad < a.L) {
        const int rank = rank_of(a, ad);
        const typename EW::raw* const Br = B + ((size_t)ad * a.N + n) * a.R;
        const float* const hr = h + m * a.R;
        float sum = 0.0f;
        int r = 0;
        for (; r + 8 <= rank; r += 8) {
            float w[8];
            load8<EW>(Br + r, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = fmaf(w[i], hr[r + i], sum);
        }
        for (; r < rank; ++r) sum = fmaf(EW::widen(Br[r]), hr[r], sum);
        y += (a.scale ? a.scale[ad] : 1.0f) * sum;
    }
    Y[m * a.N + n] = y;
}

template <class F>
hipError_t over_rows(int64_t M, LoraArgs& a, F launch) {
    const int64_t all = M * a.parts;
    hipError_t e = hipSuccess;
    for (a.first = 0; a.first < all && e == hipSuccess; a.first += kMaxGroupsPerLaunch) {
        launch((unsigned)std::min<int64_t>(all - a.first, kMaxGroupsPerLaunch));
        e = hipGetLastError();
    }
    return e;
}

template <class EX, class EW>
hipError_t lora(const LoraRows& q, hipStream_t s) {
    LoraArgs a{q.adapter, q.ranks, q.scale, q.N, q.ld, 0, (int)q.K, (int)q.R, (int)q.L, 0};
    a.parts = (int)(q.R / kShrinkWaves);
    hipError_t e = over_rows(q.M, a, [&](unsigned grid) {
        hipLaunchKernelGGL((k_lora_shrink<EX, EW>), dim3(grid), dim3(64 * kShrinkWaves), 0, s,
                           (const typename EX::raw*)q.x, (const typename EW::raw*)q.A, (float*)q.ws, a);
    });
    if (e != hipSuccess) return e;
    a.parts = (int)((q.N + kExpandThreads - 1) / kExpandThreads);
    return over_rows(q.M, a, [&](unsigned grid) {
        hipLaunchKernelGGL((k_lora_expand<EW>), dim3(grid), dim3(kExpandThreads), 0, s, (const typename EW::raw*)q.B,
                           (const float*)q.ws, q.base, q.Y, a);
    });
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
