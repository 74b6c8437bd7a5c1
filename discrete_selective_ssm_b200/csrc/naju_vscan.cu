// Vector-state scan: forward and decode step.
#include "naju_kernels.h"
#include "naju_vscan.cuh"

namespace naju {

template <typename Tin, typename Tout, bool HASB, bool HASZ, bool VEC>
__global__ void __launch_bounds__(256) vscan_fwd_kernel(VscanParams p) {
    constexpr int CP = VRow<Tin>::CP, W = 32 * CP;
    __shared__ float2 sagg[kVWarps][W];
    __shared__ float sE[W];
    __shared__ int s_item;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int64_t item = blockIdx.x;
    if (p.nk > 1) {
        if (tid == 0) s_item = atomicAdd(p.ticket, 1);
        __syncthreads();
        item = s_item;
    } else if (item == 0 && tid == 0) {
        *p.status = 0;
    }
    const int64_t k = item / p.units, u = item % p.units;
    const int64_t bb = u / p.ntiles, c0 = (u % p.ntiles) * W;
    const int64_t t0 = k * kVTok + warp * kVRun;
    const int64_t base = (bb * p.L + t0) * p.d;
    const int n = (int)max64(0, min64(kVRun, p.L - t0));

    uint32_t rh[kVRun], ra[kVRun], rb[kVRun], rz[kVRun];
#pragma unroll
    for (int q = 0; q < kVRun; ++q) {
        const int64_t o = base + q * p.d;
        if (q < n) {
            ra[q] = vload<Tin, VEC>(static_cast<const Tin*>(p.a) + o, c0, lane, p.d);
            rh[q] = vload<Tin, VEC>(static_cast<const Tin*>(p.h) + o, c0, lane, p.d);
            if (HASB) rb[q] = vload<Tin, VEC>(static_cast<const Tin*>(p.b) + o, c0, lane, p.d);
            if (HASZ) rz[q] = vload<Tin, VEC>(static_cast<const Tin*>(p.z) + o, c0, lane, p.d);
        }
    }
    // gates; this warp's (P, X) from a zero state
    float f[kVRun][CP], v[kVRun][CP], P[CP], X[CP];
#pragma unroll
    for (int j = 0; j < CP; ++j) P[j] = 1.f, X[j] = 0.f;
#pragma unroll
    for (int q = 0; q < kVRun; ++q) {
        if (q < n) {
            float a[CP], h[CP], b[CP];
            VRow<Tin>::unpack(ra[q], a);
            VRow<Tin>::unpack(rh[q], h);
            if (HASB) VRow<Tin>::unpack(rb[q], b);
#pragma unroll
            for (int j = 0; j < CP; ++j) {
                float fc;
                gate2(a[j], f[q][j], fc);
                v[q][j] = (HASB ? sigm(b[j]) : fc) * h[j];
                P[j] *= f[q][j];
                X[j] = fmaf(f[q][j], X[j], v[q][j]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < CP; ++j) sagg[warp][vchan<CP, VEC>(lane, j)] = make_float2(P[j], X[j]);
    __syncthreads();

    // warp 0: the item's entering state, and the one that leaves it
    if (warp == 0) {
        float PC[CP], XC[CP], E[CP];
        int64_t ch[CP];
#pragma unroll
        for (int j = 0; j < CP; ++j) {
            ch[j] = vchan<CP, VEC>(lane, j);
            PC[j] = 1.f, XC[j] = 0.f;
#pragma unroll
            for (int w = 0; w < kVWarps; ++w) {
                const float2 g = sagg[w][ch[j]];
                PC[j] *= g.x;
                XC[j] = fmaf(g.x, XC[j], g.y);
            }
        }
        int* flag = p.flags + u * p.nk + k;
        float* ck = p.ckpt + u * p.nk * W;
        const bool last = k + 1 == p.nk;
        if (k == 0) {
#pragma unroll
            for (int j = 0; j < CP; ++j) {
                E[j] = p.x0 && c0 + ch[j] < p.d ? p.x0[bb * p.d + c0 + ch[j]] : 0.f;
                ck[ch[j]] = E[j];
            }
        } else {
            float2* ag = p.agg + u * p.nk * W;
            if (!last) {
#pragma unroll
                for (int j = 0; j < CP; ++j) __stcg(ag + k * W + ch[j], make_float2(PC[j], XC[j]));
                vpublish(flag, kVAgg, lane);
            }
            const int dist = vlook(flag - 1, -1, k, lane, p.status, p.wait_limit);
            __syncwarp();
#pragma unroll
            for (int j = 0; j < CP; ++j) {
                E[j] = dist ? __ldcg(ck + (k - dist + 1) * W + ch[j]) : 0.f;
                for (int i = dist - 1; i >= 1; --i) {
                    const float2 g = __ldcg(ag + (k - i) * W + ch[j]);
                    E[j] = fmaf(g.x, E[j], g.y);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < CP; ++j) {
            sE[ch[j]] = E[j];
            const float out = fmaf(PC[j], E[j], XC[j]);
            if (!last)
                __stcg(ck + (k + 1) * W + ch[j], out);
            else if (p.x_final && c0 + ch[j] < p.d)
                p.x_final[bb * p.d + c0 + ch[j]] = out;
        }
        if (!last && !(p.fault_skip_publish && k == 0)) vpublish(flag, kVIncl, lane);
    }
    __syncthreads();

    // every warp: its entering state, then its tokens
    float x[CP];
#pragma unroll
    for (int j = 0; j < CP; ++j) {
        const int ch = vchan<CP, VEC>(lane, j);
        x[j] = sE[ch];
        for (int w = 0; w < warp; ++w) {
            const float2 g = sagg[w][ch];
            x[j] = fmaf(g.x, x[j], g.y);
        }
    }
    Tout* y = static_cast<Tout*>(p.y) + base;
#pragma unroll
    for (int q = 0; q < kVRun; ++q) {
        if (q < n) {
            float o[CP], z[CP];
            if (HASZ) VRow<Tin>::unpack(rz[q], z);
#pragma unroll
            for (int j = 0; j < CP; ++j) {
                x[j] = fmaf(f[q][j], x[j], v[q][j]);
                o[j] = HASZ ? x[j] * (z[j] * sigm(z[j])) : x[j];
            }
            vstore<Tout, CP, VEC>(y + q * p.d, c0, lane, p.d, o);
        }
    }
}

template <typename Tin, typename Tout, bool VEC>
static cudaError_t fwd_t(const VscanParams& p, cudaStream_t st) {
    const unsigned grid = (unsigned)(p.units * p.nk);
    if (p.b)
        p.z ? vscan_fwd_kernel<Tin, Tout, true, true, VEC><<<grid, 256, 0, st>>>(p)
            : vscan_fwd_kernel<Tin, Tout, true, false, VEC><<<grid, 256, 0, st>>>(p);
    else
        p.z ? vscan_fwd_kernel<Tin, Tout, false, true, VEC><<<grid, 256, 0, st>>>(p)
            : vscan_fwd_kernel<Tin, Tout, false, false, VEC><<<grid, 256, 0, st>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_vscan_fwd(const VscanParams& p, int dtype, int out_dtype, cudaStream_t st) {
    typedef __nv_bfloat16 bf;
    if (dtype == NAJU_F32) return fwd_t<float, float, true>(p, st);
    const bool vec = p.d % 2 == 0;
    if (out_dtype == NAJU_BF16) return vec ? fwd_t<bf, bf, true>(p, st) : fwd_t<bf, bf, false>(p, st);
    return vec ? fwd_t<bf, float, true>(p, st) : fwd_t<bf, float, false>(p, st);
}

int vscan_tile(int dtype) { return dtype == NAJU_F32 ? 32 : 64; }
int vscan_tokens() { return kVTok; }

// ------------------------------------------------------------ decode step
// Elementwise over batch * d_inner: 8 consecutive values per thread (16-byte
// accesses), the last ones of a size that is no multiple of 8 one by one.
template <typename T>
__global__ void __launch_bounds__(128)
vscan_step_kernel(int64_t n, const T* __restrict__ h, const T* __restrict__ a,
                  const T* __restrict__ b, const T* __restrict__ z, float* __restrict__ state,
                  T* __restrict__ y) {
    const int64_t e0 = ((int64_t)blockIdx.x * 128 + threadIdx.x) * 8;
    if (e0 >= n) return;
    float hv[8], av[8], bv[8], zv[8], x[8];
    const int m = (int)min64(8, n - e0);
    if (m == 8) {
        load8(h + e0, hv);
        load8(a + e0, av);
        if (b) load8(b + e0, bv);
        if (z) load8(z + e0, zv);
        load8(state + e0, x);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const bool ok = k < m;
            hv[k] = ok ? to_f(h[e0 + k]) : 0.f;
            av[k] = ok ? to_f(a[e0 + k]) : 0.f;
            bv[k] = ok && b ? to_f(b[e0 + k]) : 0.f;
            zv[k] = ok && z ? to_f(z[e0 + k]) : 0.f;
            x[k] = ok ? state[e0 + k] : 0.f;
        }
    }
    float o[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        float f, fc;
        gate2(av[k], f, fc);
        x[k] = fmaf(f, x[k], (b ? sigm(bv[k]) : fc) * hv[k]);
        o[k] = z ? x[k] * (zv[k] * sigm(zv[k])) : x[k];
    }
    if (m == 8) {
        store8(state + e0, x);
        store8(y + e0, o);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (k < m) {
                state[e0 + k] = x[k];
                y[e0 + k] = from_f<T>(o[k]);
            }
        }
    }
}

cudaError_t launch_vscan_step(int64_t n, const void* h, const void* a, const void* b,
                              const void* z, float* state, void* y, int dtype, cudaStream_t st) {
    const unsigned grid = (unsigned)((n + 1023) / 1024);
    if (dtype == NAJU_F32) {
        typedef float T;
        vscan_step_kernel<T><<<grid, 128, 0, st>>>(
            n, static_cast<const T*>(h), static_cast<const T*>(a), static_cast<const T*>(b),
            static_cast<const T*>(z), state, static_cast<T*>(y));
    } else {
        typedef __nv_bfloat16 T;
        vscan_step_kernel<T><<<grid, 128, 0, st>>>(
            n, static_cast<const T*>(h), static_cast<const T*>(a), static_cast<const T*>(b),
            static_cast<const T*>(z), state, static_cast<T*>(y));
    }
    return cudaGetLastError();
}

}  // namespace naju
