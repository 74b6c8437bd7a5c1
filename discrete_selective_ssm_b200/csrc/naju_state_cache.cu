// 8-bit cache of decode states: store (quantise into pool slots) and load
// (dequantise into batch places).  sm_100a, memory-bound.
//
// A row of N state values has scale = fp32(max|x| / 127) and
// q = round(x / scale), both quotients exact before their one rounding (to
// nearest, ties to even).
// A warp takes 32 / Q whole rows per instruction, Q = N / 4 lanes a row, four
// values (16 bytes of fp32, 4 bytes of int8) a lane, and kBatch such
// instructions in flight, so every access covers whole contiguous rows.
// Bound by HBM: 256 x 2048 x 64 (168 MB moved) stored in 37 us, loaded in 33 us
// (4.6 and 5.1 TB/s); four instructions in flight 52 us.
#include "naju_common.cuh"
#include "naju_kernels.h"

namespace naju {

constexpr int kBatch = 8;
constexpr int kCacheThreads = 256;

// round(x / s) and the scale, exactly.
//
// x / s for s in the normal range: t = x (1 / s) + 1.5 2^23, in one rounding,
// holds round(x / s) in its low bits (two's complement) unless the quotient
// lies within the product's error of a middle between two integers.  Those are
// rare (|remainder| above 0.4999 quanta: one value in five thousand) and go
// through quant_exact: the remainder x - q s of a guess q within one is exact
// in fp32 (a multiple of the smaller of x's and s's last places, and at most
// about s), so comparing it with s / 2 settles the last step.  (The conversion
// instructions run at an eighth of the adder's rate; the sum above costs none.)
constexpr float kMagic = 12582912.f;  // 1.5 2^23

// m / 127 rounded to fp32, for every finite m >= 0: the remainder m - 127 p of
// the product p = m fp32(1 / 127) is exact, and what it adds to p is rounded once
// (equal to the quotient for all 2^31 - 2^23 such m; the product alone is one
// place off for one in 22).
__device__ __forceinline__ float over_127(float m) {
    const float p = m * (1.f / 127.f);
    return fmaf(fmaf(-127.f, p, m), 1.f / 127.f, p);
}

__device__ __noinline__ int quant_exact(float x, float s) {
    // below the normal range both sides are scaled up by 2^24, exactly
    if (s < 1.17549435e-38f) {
        x *= 16777216.f;
        s *= 16777216.f;
    }
    float q = rintf(__fdiv_rn(x, s));
    const float r = fmaf(-q, s, x);
    const float over = fabsf(r) + fabsf(r) - s;
    // past the middle: one further; on it: the even one of the two
    if (over > 0.f || (over == 0.f && ((int)q & 1))) q += copysignf(1.f, r);
    return (int)fminf(fmaxf(q, -127.f), 127.f);
}

// Rows are numbered place * d + channel.
template <int N>
__global__ void __launch_bounds__(kCacheThreads)
state_store_kernel(int64_t n, int64_t d, int64_t n_slots, const float* __restrict__ state,
                   const int* __restrict__ slots, int8_t* __restrict__ pool_q,
                   float* __restrict__ pool_scale) {
    constexpr int Q = N / 4, RPI = 32 / Q;  // lanes per row, rows per instruction
    const int64_t place = blockIdx.y;
    const int lane = threadIdx.x & 31, ql = lane % Q;
    const int64_t warp = (int64_t)blockIdx.x * (kCacheThreads / 32) + (threadIdx.x >> 5);
    const int64_t c0 = warp * RPI * kBatch + lane / Q;
    float4 x[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
        const int64_t c = c0 + k * RPI;
        x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c < d) x[k] = __ldcs(reinterpret_cast<const float4*>(state + (place * d + c) * N) + ql);
    }
    // meanwhile: a slot named again by a later place is that place's to store
    const int slot = slots[place];
    bool skip = slot < 0 || slot >= n_slots;
    for (int64_t i = place + 1 + threadIdx.x; i < n && !skip; i += kCacheThreads)
        skip = slots[i] == slot;
    if (__syncthreads_or(skip)) return;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
        const int64_t c = c0 + k * RPI;
        const float4 v = x[k];
        const float e[4] = {v.x, v.y, v.z, v.w};
        // the largest magnitude as bits: infinities and NaN sort above the rest
        unsigned m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max(m, __float_as_uint(e[i]) & 0x7fffffffu);
#pragma unroll
        for (int o = 1; o < Q; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float s = m < 0x7f800000u ? over_127(__uint_as_float(m)) : NAN;
        uint32_t q = 0;
        if (s > 0.f) {
            const float inv = rcpa_(s);
            uint32_t t[4];
            float far = s < 1.17549435e-38f ? 1.f : 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float f = fmaf(e[i], inv, kMagic);
                t[i] = __float_as_uint(f);
                far = fmaxf(far, fabsf(fmaf(e[i], inv, kMagic - f)));
            }
            if (far > 0.4999f) {
#pragma unroll
                for (int i = 0; i < 4; ++i) t[i] = (uint32_t)quant_exact(e[i], s);
            }
            q = __byte_perm(__byte_perm(t[0], t[1], 0x0040), __byte_perm(t[2], t[3], 0x0040),
                            0x5410);
        }
        if (c < d) {
            const int64_t row = (int64_t)slot * d + c;
            reinterpret_cast<uint32_t*>(pool_q + row * N)[ql] = q;
            if (ql == 0) pool_scale[row] = s;
        }
    }
}

template <int N>
__global__ void __launch_bounds__(kCacheThreads)
state_load_kernel(int64_t d, int64_t n_slots, const int8_t* __restrict__ pool_q,
                  const float* __restrict__ pool_scale, const int* __restrict__ slots,
                  float* __restrict__ state) {
    constexpr int Q = N / 4, RPI = 32 / Q;
    const int64_t place = blockIdx.y;
    const int slot = slots[place];
    const bool live = slot >= 0 && slot < n_slots;
    const int lane = threadIdx.x & 31, ql = lane % Q;
    const int64_t warp = (int64_t)blockIdx.x * (kCacheThreads / 32) + (threadIdx.x >> 5);
    const int64_t c0 = warp * RPI * kBatch + lane / Q;
    uint32_t q[kBatch];
    float s[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
        const int64_t c = c0 + k * RPI;
        q[k] = 0;
        s[k] = 0.f;
        if (live && c < d) {
            const int64_t row = (int64_t)slot * d + c;
            q[k] = __ldg(reinterpret_cast<const uint32_t*>(pool_q + row * N) + ql);
            s[k] = __ldg(pool_scale + row);
        }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
        const int64_t c = c0 + k * RPI;
        // a byte as a float: q + 128 in the low bits of 2^23
        const uint32_t u = q[k] ^ 0x80808080u;
        float f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f[i] = s[k] * (__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440 | i)) - 8388736.f);
        if (c < d)
            reinterpret_cast<float4*>(state + (place * d + c) * N)[ql] =
                make_float4(f[0], f[1], f[2], f[3]);
    }
}

template <int N>
static dim3 cache_grid(int64_t n, int64_t d) {
    const int64_t per_block = (kCacheThreads / 32) * (32 / (N / 4)) * kBatch;
    return dim3((unsigned)((d + per_block - 1) / per_block), (unsigned)n);
}

cudaError_t launch_state_store(int64_t n, int64_t d, int64_t N, int64_t n_slots,
                               const float* state, const int* slots, int8_t* pool_q,
                               float* pool_scale, cudaStream_t st) {
#define NAJU_STORE(NN)                                                         \
    state_store_kernel<NN><<<cache_grid<NN>(n, d), kCacheThreads, 0, st>>>(    \
        n, d, n_slots, state, slots, pool_q, pool_scale)
    switch (N) {
        case 16: NAJU_STORE(16); break;
        case 32: NAJU_STORE(32); break;
        case 64: NAJU_STORE(64); break;
        case 128: NAJU_STORE(128); break;
        default: return cudaErrorInvalidValue;
    }
#undef NAJU_STORE
    return cudaGetLastError();
}

cudaError_t launch_state_load(int64_t n, int64_t d, int64_t N, int64_t n_slots,
                              const int8_t* pool_q, const float* pool_scale, const int* slots,
                              float* state, cudaStream_t st) {
#define NAJU_LOAD(NN)                                                          \
    state_load_kernel<NN><<<cache_grid<NN>(n, d), kCacheThreads, 0, st>>>(     \
        d, n_slots, pool_q, pool_scale, slots, state)
    switch (N) {
        case 16: NAJU_LOAD(16); break;
        case 32: NAJU_LOAD(32); break;
        case 64: NAJU_LOAD(64); break;
        case 128: NAJU_LOAD(128); break;
        default: return cudaErrorInvalidValue;
    }
#undef NAJU_LOAD
    return cudaGetLastError();
}

}  // namespace naju
