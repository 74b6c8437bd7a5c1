// What the kernels of the 4-bit projections share: the parameters, the way
// from 4-bit words to bf16 operands, and the launch.
#pragma once
#include <atomic>

#include "naju_common.cuh"
#include "naju_kernels.h"

namespace naju {

struct W4Params {
    const void* x;
    const uint4* wq;
    const __nv_bfloat16* scales;
    const float* bias;
    const void* residual;
    void* y;
    int64_t m, n_in, n_out, nb, ng;  // nb: 128-input blocks of a row, ng: groups of a row
    int split;                       // blocks (or warps) that share the inputs of their rows
};

// (a & mask) | bits in one instruction: with both constants as immediates the
// compiler takes two, and the logic unit is what bounds the unpacking.
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t mask, uint32_t bits) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(a), "r"(mask), "r"(bits));
    return r;
}
// A constant that stays in a register.
__device__ __forceinline__ uint32_t held(uint32_t v) {
    uint32_t r;
    asm volatile("mov.b32 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// Nibbles i and i + 4 of a word (inputs 2 i, 2 i + 1) as two bf16 of
// (q - 8) / 1024: or-ing q into the bits of 128 gives 128 + q, exactly.  The
// factor keeps a group's sum (at most 128 * 8 values of x) in range for every
// finite x; the sums are multiplied by 1024 once, at the end.
struct PairBits {
    uint32_t mask, bits;
    __device__ __forceinline__ PairBits() : mask(held(0x000f000fu)), bits(held(0x43004300u)) {}
};
__device__ __forceinline__ uint32_t unpack_pair(uint32_t w, int i, const PairBits& k) {
    const uint32_t t = and_or(w >> (4 * i), k.mask, k.bits);
    const __nv_bfloat162 r =
        __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&t), __float2bfloat162_rn(1.f / 1024.f),
                __float2bfloat162_rn(-136.f / 1024.f));
    return *reinterpret_cast<const uint32_t*>(&r);
}

// Finishes four sums of one row of x (outputs o .. o + 3): the factor, bias and
// residual, one rounding.
template <typename T>
__device__ __forceinline__ void w4_finish(const W4Params& p, int64_t m, int64_t o, float4 s) {
    float v[4] = {s.x * 1024.f, s.y * 1024.f, s.z * 1024.f, s.w * 1024.f};
    const int n = (int)min64(4, p.n_out - o);
    if (p.bias) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) v[i] += p.bias[o + i];
    }
    const T* res = static_cast<const T*>(p.residual);
    T* y = static_cast<T*>(p.y) + m * p.n_out + o;
    if (p.n_out % 4 == 0) {  // rows start on four elements
        struct alignas(4 * sizeof(T)) Four {
            T e[4];
        } r;
        if (res) {
            r = *reinterpret_cast<const Four*>(res + m * p.n_out + o);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] += to_f(r.e[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) r.e[i] = from_f<T>(v[i]);
        *reinterpret_cast<Four*>(y) = r;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i < n) {
                if (res) v[i] += to_f(res[m * p.n_out + o + i]);
                y[i] = from_f<T>(v[i]);
            }
        }
    }
}
__device__ __forceinline__ float4 operator+(float4 a, float4 b) {
    return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}

// Launches clusters of `split` blocks.  `ready`: the devices on which this
// kernel's attributes are set.
template <typename... Args>
inline cudaError_t w4_launch(void (*kern)(Args...), dim3 grid, int threads, int smem, int split,
                             std::atomic<uint64_t>& ready, cudaStream_t st, const Args&... args) {
    cudaError_t e = smem_once(reinterpret_cast<const void*>(kern), smem, ready);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)split;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

cudaError_t launch_w4_tc(const W4Params& p, int group, int sms, cudaStream_t st);

}  // namespace naju
