// 8-bit cache of decode states: store (quantise into pool slots) and load
// (dequantise into batch places).  sm_100a, memory-bound.
//
// A row of N state values has scale = fp32(max|x| / 127) and
// q = round(x / scale), the exact quotient rounded to nearest, ties to even.
// A warp takes 32 / Q whole rows per instruction, Q = N / 4 lanes a row, four
// values (16 bytes of fp32, 4 bytes of int8) a lane, and kBatch such
// instructions in flight, so every access covers whole contiguous rows.
#include "naju_common.cuh"
#include "naju_kernels.h"

namespace naju {

constexpr int kBatch = 4;
constexpr int kCacheThreads = 256;

// round(x / s), exactly, for 2^-126 <= s and |x| up to a few hundred s:
// x * (1 / s) lands within one of it, and the remainder x - q s of that guess
// is exact in fp32 (a multiple of the smaller of x's and s's last places, and
// at most about s), so comparing it with s / 2 settles the last step.
__device__ __forceinline__ float quant1(float x, float s, float inv) {
    float q = rintf(x * inv);
    const float r = fmaf(-q, s, x);
    const float over = fabsf(r) + fabsf(r) - s;
    // past the middle: one further; on it: the even one of the two
    if (over > 0.f || (over == 0.f && ((int)q & 1))) q += copysignf(1.f, r);
    return fminf(fmaxf(q, -127.f), 127.f);
}

// Rows are numbered place * d + channel.
template <int N>
__global__ void __launch_bounds__(kCacheThreads)
state_store_kernel(int64_t n, int64_t d, int64_t n_slots, const float* __restrict__ state,
                   const int* __restrict__ slots, int8_t* __restrict__ pool_q,
                   float* __restrict__ pool_scale) {
    constexpr int Q = N / 4, RPI = 32 / Q;  // lanes per row, rows per instruction
    __shared__ int s_slot;
    const int64_t place = blockIdx.y;
    // a slot named again by a later place is that place's to store
    if (threadIdx.x == 0) s_slot = 1;
    __syncthreads();
    const int slot = slots[place];
    bool again = slot < 0 || slot >= n_slots;
    for (int64_t i = place + 1 + threadIdx.x; i < n && !again; i += kCacheThreads)
        again = slots[i] == slot;
    if (again) s_slot = 0;
    __syncthreads();
    if (!s_slot) return;
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
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
        const int64_t c = c0 + k * RPI;
        const float4 v = x[k];
        float m = fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
        // (fmaxf drops a NaN: an infinity stands for whatever is not finite)
        if (!(fabsf(v.x) < INFINITY && fabsf(v.y) < INFINITY && fabsf(v.z) < INFINITY &&
              fabsf(v.w) < INFINITY))
            m = INFINITY;
#pragma unroll
        for (int o = 1; o < Q; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float s = m < INFINITY ? __fdiv_rn(m, 127.f) : NAN;
        char4 q = make_char4(0, 0, 0, 0);
        if (s > 0.f) {
            // below the normal range both sides are scaled up by 2^24, exactly
            const float up = s < 1.17549435e-38f ? 16777216.f : 1.f, t = s * up;
            const float inv = __fdiv_rn(1.f, t);
            q = make_char4(
                (signed char)quant1(v.x * up, t, inv), (signed char)quant1(v.y * up, t, inv),
                (signed char)quant1(v.z * up, t, inv), (signed char)quant1(v.w * up, t, inv));
        }
        if (c < d) {
            const int64_t row = (int64_t)slot * d + c;
            reinterpret_cast<char4*>(pool_q + row * N)[ql] = q;
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
    char4 q[kBatch];
    float s[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
        const int64_t c = c0 + k * RPI;
        q[k] = make_char4(0, 0, 0, 0);
        s[k] = 0.f;
        if (live && c < d) {
            const int64_t row = (int64_t)slot * d + c;
            q[k] = __ldg(reinterpret_cast<const char4*>(pool_q + row * N) + ql);
            s[k] = __ldg(pool_scale + row);
        }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
        const int64_t c = c0 + k * RPI;
        if (c < d)
            reinterpret_cast<float4*>(state + (place * d + c) * N)[ql] =
                make_float4(s[k] * q[k].x, s[k] * q[k].y, s[k] * q[k].z, s[k] * q[k].w);
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
