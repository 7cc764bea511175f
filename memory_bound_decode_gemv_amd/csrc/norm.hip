// norm.hip -- RMS norm of rows with the residual's addition, into Q8_1 columns
// (the operand of every quantised GEMV here) or into float rows.
//
//   h = T(x + res)                       binary32 sum, rounded to the storage type T (h = x without res)
//   r = binary32(1 / sqrt(sum_k h_k^2 / K + eps))
//   y = (h r) w                          two binary32 products, then the Q8_1 rules or the output type
//
// The sum, the root and the quotient are binary64 and are rounded once, to r:
// the square of a binary32 value is exact in binary64 and the sum's own error
// is about 2^-53 sqrt(K), so r is the same binary32 value for any order of
// summation except within that distance of a rounding border (about one row
// in 10^8).  A binary32 sum would move r by an ulp with the split of the row,
// and an ulp of r moves the codes of activations next to a rounding border:
// the Q8_1 bytes would depend on the launch.
//
// Every binary32 result that is rounded on to a 16-bit type is bound to a
// register (bind_f32): the compiler would otherwise round some of the exact
// sums and products once, straight to binary16 (v_fma_mixlo_f16).
//
// One workgroup per row, eight consecutive elements per thread and group (16
// bytes of a 16-bit type, two 16-byte loads of binary32), so the four
// neighbouring threads of a quad hold one 32-element Q8_1 block and its
// largest magnitude and code sum are two quad steps each.  The row stays in
// registers between the sum and the product: x and res are read once, h and
// the output written once.  All the threads a row can use, up to 1024: 2048 rows
// of 8192 bfloat16 elements take 22.0 us (6.1 TB/s of the 134 MB that they read
// and write) with 1024 or 512 threads a row, 24.8 with 256 and 31.2 with 64; one
// row of 4096 binary32 elements takes 3.5 us, 4.4 with 256.  The weights' loads
// stand before the sum and the sum is reduced on DPP: with shuffles and a later
// load the two took 24.5 and 3.7.
//
// What bounds short calls: the launch (1.7 us) and round trips to memory one
// after another.  Loads of binary32 operands are in flight together.  A group of
// a 16-bit operand is widened within the branch that loads it, so the compiler
// waits for it there: x, then res, then 16-bit weights are three round trips (24
// rows of 8192 bfloat16 into Q8_1: 4.6 us, on 24 of 256 CUs), and a 16-bit row
// that is not 16-byte aligned is eight per operand.  Into Q8_1 eight exact
// divisions a thread come on top.  Rows longer than the registers of a workgroup
// hold (kMaxGroups groups per thread) are read a second time.
#include "dg_device.h"
#include "dg_internal.h"
#include "q81_rules.h"

#pragma clang fp contract(off)

namespace dg {
namespace {

constexpr int kGroup = 8;          // elements per thread and group
constexpr int kMaxThreads = 1024;
constexpr int kMaxGroups = 4;      // groups a thread keeps in registers

struct NormF32 {
    using raw = float;
    static constexpr int kVecs = 2;   // 16-byte vectors per group
    __device__ __forceinline__ static float widen(raw v) { return v; }
    __device__ __forceinline__ static raw narrow(float v) { return v; }
};
struct NormF16 {
    using raw = _Float16;
    static constexpr int kVecs = 1;
    __device__ __forceinline__ static float widen(raw v) { return (float)v; }
    __device__ __forceinline__ static raw narrow(float v) { return (raw)v; }
};
struct NormBF16 {
    using raw = __bf16;
    static constexpr int kVecs = 1;
    __device__ __forceinline__ static float widen(raw v) { return (float)v; }
    __device__ __forceinline__ static raw narrow(float v) { return (raw)v; }
};

template <class E>
union GroupBits {
    u32x4 v[E::kVecs];
    typename E::raw e[kGroup];
};

// Elements k0 .. k0 + 7 of a row, those past K as zeros.  `vec`: the row is
// 16-byte aligned, so a whole group is one or two vector loads.
template <class E>
__device__ __forceinline__ void load_group8(const typename E::raw* row, int k0, int K, bool vec, float (&v)[kGroup]) {
    if (vec && k0 + kGroup <= K) {
        GroupBits<E> b;
#pragma unroll
        for (int i = 0; i < E::kVecs; ++i) b.v[i] = reinterpret_cast<const u32x4*>(row + k0)[i];
#pragma unroll
        for (int i = 0; i < kGroup; ++i) v[i] = E::widen(b.e[i]);
    } else {
#pragma unroll
        for (int i = 0; i < kGroup; ++i) v[i] = k0 + i < K ? E::widen(row[k0 + i]) : 0.0f;
    }
}

template <class E>
__device__ __forceinline__ void store_group8(typename E::raw* row, int k0, int K, bool vec, const float (&v)[kGroup]) {
    if (vec && k0 + kGroup <= K) {
        GroupBits<E> b;
#pragma unroll
        for (int i = 0; i < kGroup; ++i) b.e[i] = E::narrow(v[i]);
#pragma unroll
        for (int i = 0; i < E::kVecs; ++i) reinterpret_cast<u32x4*>(row + k0)[i] = b.v[i];
    } else {
#pragma unroll
        for (int i = 0; i < kGroup; ++i)
            if (k0 + i < K) row[k0 + i] = E::narrow(v[i]);
    }
}

__device__ __forceinline__ void load_weights8(const void* w, int wdtype, int k0, int K, bool vec,
                                              float (&v)[kGroup]) {
    if (wdtype == DG_DTYPE_F32) load_group8<NormF32>((const float*)w, k0, K, vec, v);
    else if (wdtype == DG_DTYPE_F16) load_group8<NormF16>((const _Float16*)w, k0, K, vec, v);
    else load_group8<NormBF16>((const __bf16*)w, k0, K, vec, v);
}

template <int CTRL, int ROW_MASK>
__device__ __forceinline__ double dpp_add_f64(double v) {   // lanes without a source add 0
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = dpp_mov_u32<CTRL, ROW_MASK>((uint32_t)u);
    const uint32_t hi = dpp_mov_u32<CTRL, ROW_MASK>((uint32_t)(u >> 32));
    return v + __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

__device__ __forceinline__ double lane_f64(double v, int src) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, src);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), src);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// Sum over the workgroup (at most 16 waves) in a fixed order, in every thread:
// DPP within a wave, one LDS exchange, DPP over the waves' sums.
__device__ __forceinline__ double block_sum_f64(double v) {
    __shared__ double part[kMaxThreads / kWave];
    v = dpp_add_f64<kDppRowShr1, 0xF>(v);
    v = dpp_add_f64<kDppRowShr2, 0xF>(v);
    v = dpp_add_f64<kDppRowShr4, 0xF>(v);
    v = dpp_add_f64<kDppRowShr8, 0xF>(v);
    v = dpp_add_f64<kDppRowBcast15, 0xA>(v);
    v = dpp_add_f64<kDppRowBcast31, 0xC>(v);
    const int lane = lane_id();
    if (lane == kWave - 1) part[threadIdx.x / kWave] = v;
    __syncthreads();
    double s = lane < (int)blockDim.x / kWave ? part[lane & 15] : 0.0;
    s = dpp_add_f64<kDppRowShr1, 0xF>(s);
    s = dpp_add_f64<kDppRowShr2, 0xF>(s);
    s = dpp_add_f64<kDppRowShr4, 0xF>(s);
    s = dpp_add_f64<kDppRowShr8, 0xF>(s);
    return lane_f64(s, 15);
}

constexpr int kQuadXor1 = 0xB1;   // DPP quad_perm [1,0,3,2]
constexpr int kQuadXor2 = 0x4E;   // DPP quad_perm [2,3,0,1]

// The quad's 32 values as one Q8_1 block, two code dwords per thread.  Quads
// are whole (K % 32 == 0): every lane of a quad is here or none.
__device__ __forceinline__ void store_q81(uint8_t* col, int k0, const float (&y)[kGroup]) {
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < kGroup; ++i) amax = fmaxf(amax, fabsf(y[i]));
    amax = fmaxf(amax, dpp_mov_f32<kQuadXor1, 0xF>(amax));
    amax = fmaxf(amax, dpp_mov_f32<kQuadXor2, 0xF>(amax));
    const float d = q81_scale(amax);
    uint32_t words[2] = {0u, 0u};
    int sum = 0;
#pragma unroll
    for (int i = 0; i < kGroup; ++i) {
        const int c = q81_code(y[i], d);
        sum += c;
        words[i >> 2] |= (uint32_t)(uint8_t)(int8_t)c << (8 * (i & 3));
    }
    sum += (int)dpp_mov_u32<kQuadXor1, 0xF>((uint32_t)sum);
    sum += (int)dpp_mov_u32<kQuadXor2, 0xF>((uint32_t)sum);
    const int j = (k0 / kGroup) & 3;
    uint32_t* blk = reinterpret_cast<uint32_t*>(col + (size_t)(k0 / 32) * 36);
    if (j == 0) blk[0] = q81_header(d, sum);
    blk[1 + 2 * j] = words[0];
    blk[2 + 2 * j] = words[1];
}

constexpr int kOutQ81 = kRmsNormQ81;   // beside the DG_DTYPE_* output types

template <int OUT>
__device__ __forceinline__ void store_out(void* out, int64_t row, int64_t ldy, int K, int k0, bool vec,
                                          const float (&y)[kGroup]) {
    if constexpr (OUT == kOutQ81) store_q81((uint8_t*)out + row * (K / 32) * 36, k0, y);
    else if constexpr (OUT == DG_DTYPE_F32) store_group8<NormF32>((float*)out + row * ldy, k0, K, vec, y);
    else if constexpr (OUT == DG_DTYPE_F16) store_group8<NormF16>((_Float16*)out + row * ldy, k0, K, vec, y);
    else store_group8<NormBF16>((__bf16*)out + row * ldy, k0, K, vec, y);
}

// G > 0: the row's groups stay in registers (K <= 8 G threads).  G = 0: they
// are read again for the products (h where it was stored, since h may be x or
// res itself).  x, res and h carry no __restrict__: h may be either of them.
template <class E, int OUT, int G>
__global__ void __launch_bounds__(kMaxThreads)
k_rmsnorm(const typename E::raw* x, const typename E::raw* res, typename E::raw* h, const void* __restrict__ w,
          int wdtype, void* __restrict__ out, int K, int64_t ld, int64_t ldy, float eps, double inv_k, int vec) {
    const int64_t row = blockIdx.x;
    const typename E::raw* xr = x + row * ld;
    const typename E::raw* rr = res ? res + row * ld : nullptr;
    typename E::raw* hr = h ? h + row * ld : nullptr;
    const bool vrow = vec & 1, vw = vec & 2, vy = vec & 4;
    const int step = (int)blockDim.x * kGroup;
    const int k_first = (int)threadIdx.x * kGroup;

    auto load_h = [&](int k0, float (&v)[kGroup]) {
        load_group8<E>(xr, k0, K, vrow, v);
        if (rr) {
            float a[kGroup];
            load_group8<E>(rr, k0, K, vrow, a);
#pragma unroll
            for (int i = 0; i < kGroup; ++i) v[i] = E::widen(E::narrow(bind_f32(v[i] + a[i])));
        }
    };
    auto finish = [&](int k0, const float (&v)[kGroup], const float (&wv)[kGroup], float r) {
        float y[kGroup];
#pragma unroll
        for (int i = 0; i < kGroup; ++i) y[i] = bind_f32((v[i] * r) * wv[i]);
        store_out<OUT>(out, row, ldy, K, k0, vy, y);
    };

    auto scale = [&](double ss) { return (float)(1.0 / sqrt(block_sum_f64(ss) * inv_k + (double)eps)); };

    double ss = 0.0;
    if constexpr (G > 0) {
        float v[G][kGroup], wv[G][kGroup];
#pragma unroll
        for (int g = 0; g < G; ++g)
            if (k_first + g * step < K) load_h(k_first + g * step, v[g]);
#pragma unroll
        for (int g = 0; g < G; ++g)   // binary32 weights stay in flight during the sum
            if (k_first + g * step < K) load_weights8(w, wdtype, k_first + g * step, K, vw, wv[g]);
#pragma unroll
        for (int g = 0; g < G; ++g)
            if (k_first + g * step < K) {
                if (hr) store_group8<E>(hr, k_first + g * step, K, vrow, v[g]);
#pragma unroll
                for (int i = 0; i < kGroup; ++i) ss += (double)v[g][i] * (double)v[g][i];
            }
        const float r = scale(ss);
#pragma unroll
        for (int g = 0; g < G; ++g)
            if (k_first + g * step < K) finish(k_first + g * step, v[g], wv[g], r);
    } else {
        for (int k0 = k_first; k0 < K; k0 += step) {
            float v[kGroup];
            load_h(k0, v);
            if (hr) store_group8<E>(hr, k0, K, vrow, v);
#pragma unroll
            for (int i = 0; i < kGroup; ++i) ss += (double)v[i] * (double)v[i];
        }
        const float r = scale(ss);
        for (int k0 = k_first; k0 < K; k0 += step) {
            float v[kGroup], wv[kGroup];
            if (hr) load_group8<E>(hr, k0, K, vrow, v);
            else load_h(k0, v);
            load_weights8(w, wdtype, k0, K, vw, wv);
            finish(k0, v, wv, r);
        }
    }
}

bool aligned16(const void* p) { return (uintptr_t)p % 16 == 0; }

template <class E, int OUT>
hipError_t launch_norm_out(const RmsNorm& a, hipStream_t s) {
    using raw = typename E::raw;
    const int K = (int)a.K;
    const int groups = (K + kGroup - 1) / kGroup;
    int threads = (groups + kWave - 1) / kWave * kWave;
    if (threads > kMaxThreads) threads = kMaxThreads;
    const int per = (groups + threads - 1) / threads;   // groups per thread
    const int ysize = OUT == DG_DTYPE_F32 ? 4 : 2;
    int vec = 0;
    if (aligned16(a.x) && aligned16(a.res) && aligned16(a.h) && a.ld * (int64_t)sizeof(raw) % 16 == 0) vec |= 1;
    if (aligned16(a.w)) vec |= 2;
    if (aligned16(a.out) && a.ldy * ysize % 16 == 0) vec |= 4;
    for (int64_t r0 = 0; r0 < a.M; r0 += kMaxGroupsPerLaunch) {
        const unsigned rows = (unsigned)(a.M - r0 < kMaxGroupsPerLaunch ? a.M - r0 : kMaxGroupsPerLaunch);
        const raw* x = (const raw*)a.x + r0 * a.ld;
        const raw* res = a.res ? (const raw*)a.res + r0 * a.ld : nullptr;
        raw* h = a.h ? (raw*)a.h + r0 * a.ld : nullptr;
        void* out = (uint8_t*)a.out + r0 * (OUT == kOutQ81 ? (int64_t)(K / 32) * 36 : a.ldy * ysize);
#define DG_NORM(GG)                                                                                               \
    hipLaunchKernelGGL((k_rmsnorm<E, OUT, GG>), dim3(rows), dim3(threads), 0, s, x, res, h, a.w, a.wdtype, out, K, \
                       a.ld, a.ldy, a.eps, 1.0 / (double)K, vec)
        if (per <= 1) DG_NORM(1);
        else if (per <= 2) DG_NORM(2);
        else if (per <= kMaxGroups) DG_NORM(kMaxGroups);
        else DG_NORM(0);
#undef DG_NORM
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <class E>
hipError_t launch_norm_in(const RmsNorm& a, hipStream_t s) {
    switch (a.out_kind) {
        case kOutQ81: return launch_norm_out<E, kOutQ81>(a, s);
        case DG_DTYPE_F32: return launch_norm_out<E, DG_DTYPE_F32>(a, s);
        case DG_DTYPE_F16: return launch_norm_out<E, DG_DTYPE_F16>(a, s);
        case DG_DTYPE_BF16: return launch_norm_out<E, DG_DTYPE_BF16>(a, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_rmsnorm(const RmsNorm& a, hipStream_t s) {
    switch (a.dtype) {
        case DG_DTYPE_F32: return launch_norm_in<NormF32>(a, s);
        case DG_DTYPE_F16: return launch_norm_in<NormF16>(a, s);
        case DG_DTYPE_BF16: return launch_norm_in<NormBF16>(a, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace dg
