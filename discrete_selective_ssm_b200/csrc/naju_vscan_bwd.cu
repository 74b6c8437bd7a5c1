// Vector-state scan: backward.
//
// With dx_t = dy_t SiLU(z_t) the adjoint is g_t = dx_t + r_{t+1}, where
// r_t = f_t g_t is what a token hands to the one before it (r_L = dx_final,
// r_0 = dx0).  A run of tokens acts on r as r -> P r + R with the forward's
// own P, so the runs compose like the forward's, in the other direction.  The
// gradients also need x_{t-1}: each item recomputes its states from the
// forward's checkpoint of its first token (one fp32 value per kVTok tokens)
// instead of reading stored states.
#include "naju_kernels.h"
#include "naju_vscan.cuh"

namespace naju {

template <typename Tin, typename Tout, bool HASB, bool HASZ, bool VEC>
__global__ void __launch_bounds__(256) vscan_bwd_kernel(VscanParams p) {
    constexpr int CP = VRow<Tin>::CP, W = 32 * CP;
    __shared__ float2 sagg[kVWarps][W];  // (P, X) of each warp's tokens
    __shared__ float srev[kVWarps][W];   // R of each warp's tokens
    __shared__ float sE[W], sA[W];
    __shared__ int s_item;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int64_t item = blockIdx.x;
    if (p.nk > 1) {
        if (tid == 0) s_item = atomicAdd(p.ticket, 1);
        __syncthreads();
        item = s_item;
    }
    const int64_t k = p.nk - 1 - item / p.units, u = item % p.units;
    const int64_t bb = u / p.ntiles, c0 = (u % p.ntiles) * W;
    const int64_t t0 = k * kVTok + warp * kVRun;
    const int64_t base = (bb * p.L + t0) * p.d;
    const int n = (int)max64(0, min64(kVRun, p.L - t0));

    uint32_t rh[kVRun], ra[kVRun], rb[kVRun], rz[kVRun], rd[kVRun];
#pragma unroll
    for (int q = 0; q < kVRun; ++q) {
        const int64_t o = base + q * p.d;
        if (q < n) {
            ra[q] = vload<Tin, VEC>(static_cast<const Tin*>(p.a) + o, c0, lane, p.d);
            rh[q] = vload<Tin, VEC>(static_cast<const Tin*>(p.h) + o, c0, lane, p.d);
            rd[q] = vload<Tin, VEC>(static_cast<const Tin*>(p.dy) + o, c0, lane, p.d);
            if (HASB) rb[q] = vload<Tin, VEC>(static_cast<const Tin*>(p.b) + o, c0, lane, p.d);
            if (HASZ) rz[q] = vload<Tin, VEC>(static_cast<const Tin*>(p.z) + o, c0, lane, p.d);
        }
    }
    float E0[CP];  // warp 0: the item's entering state
    if (warp == 0) {
#pragma unroll
        for (int j = 0; j < CP; ++j)
            E0[j] = p.ckpt[(u * p.nk + k) * W + vchan<CP, VEC>(lane, j)];
    }
    // Kept per token: both gates packed, sigmoid(z).
    float ga[kVRun][CP], gb[kVRun][CP], sz[kVRun][CP], P[CP], X[CP], R[CP];
#pragma unroll
    for (int j = 0; j < CP; ++j) P[j] = 1.f, X[j] = 0.f, R[j] = 0.f;
#pragma unroll
    for (int q = 0; q < kVRun; ++q) {
        if (q < n) {
            float a[CP], h[CP], b[CP], z[CP];
            VRow<Tin>::unpack(ra[q], a);
            VRow<Tin>::unpack(rh[q], h);
            if (HASB) VRow<Tin>::unpack(rb[q], b);
            if (HASZ) VRow<Tin>::unpack(rz[q], z);
#pragma unroll
            for (int j = 0; j < CP; ++j) {
                float f, fc, i, ic;
                ga[q][j] = gate_pack(a[j]);
                gate_of(ga[q][j], f, fc);
                if (HASB) {
                    gb[q][j] = gate_pack(b[j]);
                    gate_of(gb[q][j], i, ic);
                } else {
                    i = fc;
                }
                if (HASZ) sz[q][j] = sigm(z[j]);
                P[j] *= f;
                X[j] = fmaf(f, X[j], i * h[j]);
            }
        }
    }
#pragma unroll
    for (int q = kVRun - 1; q >= 0; --q) {
        if (q < n) {
            float dy[CP], z[CP];
            VRow<Tin>::unpack(rd[q], dy);
            if (HASZ) VRow<Tin>::unpack(rz[q], z);
#pragma unroll
            for (int j = 0; j < CP; ++j) {
                float f, fc;
                gate_of(ga[q][j], f, fc);
                const float dx = HASZ ? dy[j] * (z[j] * sz[q][j]) : dy[j];
                R[j] = f * (dx + R[j]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < CP; ++j) {
        const int ch = vchan<CP, VEC>(lane, j);
        sagg[warp][ch] = make_float2(P[j], X[j]);
        srev[warp][ch] = R[j];
    }
    __syncthreads();

    if (warp == 0) {
        float PC[CP], RC[CP], A[CP];
        int64_t ch[CP];
#pragma unroll
        for (int j = 0; j < CP; ++j) {
            ch[j] = vchan<CP, VEC>(lane, j);
            PC[j] = 1.f, RC[j] = 0.f;
#pragma unroll
            for (int w = kVWarps - 1; w >= 0; --w) {
                const float g = sagg[w][ch[j]].x;
                PC[j] *= g;
                RC[j] = fmaf(g, RC[j], srev[w][ch[j]]);
            }
        }
        int* flag = p.flags + u * p.nk + k;
        float* adj = p.adj + u * p.nk * W;  // r leaving item k, at k
        if (k + 1 == p.nk) {
#pragma unroll
            for (int j = 0; j < CP; ++j)
                A[j] = p.dx_final && c0 + ch[j] < p.d ? p.dx_final[bb * p.d + c0 + ch[j]] : 0.f;
        } else {
            float2* ag = p.agg + u * p.nk * W;
            if (k > 0) {
#pragma unroll
                for (int j = 0; j < CP; ++j) __stcg(ag + k * W + ch[j], make_float2(PC[j], RC[j]));
                vpublish(flag, kVAgg, lane);
            }
            const int dist = vlook(flag + 1, 1, p.nk - 1 - k, lane, p.status, p.wait_limit);
            __syncwarp();
#pragma unroll
            for (int j = 0; j < CP; ++j) {
                A[j] = dist ? __ldcg(adj + (k + dist) * W + ch[j]) : 0.f;
                for (int i = dist - 1; i >= 1; --i) {
                    const float2 g = __ldcg(ag + (k + i) * W + ch[j]);
                    A[j] = fmaf(g.x, A[j], g.y);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < CP; ++j) {
            sE[ch[j]] = E0[j];
            sA[ch[j]] = A[j];
            const float out = fmaf(PC[j], A[j], RC[j]);
            if (k > 0)
                __stcg(adj + k * W + ch[j], out);
            else if (p.dx0 && c0 + ch[j] < p.d)
                p.dx0[bb * p.d + c0 + ch[j]] = out;
        }
        if (k > 0 && !(p.fault_skip_publish && k + 1 == p.nk)) vpublish(flag, kVIncl, lane);
    }
    __syncthreads();

    float x[CP], r[CP], xs[kVRun + 1][CP];
#pragma unroll
    for (int j = 0; j < CP; ++j) {
        const int ch = vchan<CP, VEC>(lane, j);
        x[j] = sE[ch];
        for (int w = 0; w < warp; ++w) {
            const float2 g = sagg[w][ch];
            x[j] = fmaf(g.x, x[j], g.y);
        }
        r[j] = sA[ch];
        for (int w = kVWarps - 1; w > warp; --w) r[j] = fmaf(sagg[w][ch].x, r[j], srev[w][ch]);
        xs[0][j] = x[j];
    }
#pragma unroll
    for (int q = 0; q < kVRun; ++q) {
        if (q < n) {
            float h[CP];
            VRow<Tin>::unpack(rh[q], h);
#pragma unroll
            for (int j = 0; j < CP; ++j) {
                float f, fc, i, ic;
                gate_of(ga[q][j], f, fc);
                if (HASB) gate_of(gb[q][j], i, ic);
                xs[q + 1][j] = fmaf(f, xs[q][j], (HASB ? i : fc) * h[j]);
            }
        }
    }
#pragma unroll
    for (int q = kVRun - 1; q >= 0; --q) {
        if (q < n) {
            float dy[CP], h[CP], z[CP], oh[CP], oa[CP], ob[CP], oz[CP];
            VRow<Tin>::unpack(rd[q], dy);
            VRow<Tin>::unpack(rh[q], h);
            if (HASZ) VRow<Tin>::unpack(rz[q], z);
#pragma unroll
            for (int j = 0; j < CP; ++j) {
                float f, fc, i, ic;
                gate_of(ga[q][j], f, fc);
                float dx = dy[j];
                if (HASZ) {
                    const float s = sz[q][j], zs = z[j] * s;
                    // SiLU'(z) = s + z s (1 - s)
                    oz[j] = dy[j] * xs[q + 1][j] * fmaf(zs, 1.f - s, s);
                    dx *= zs;
                }
                const float g = dx + r[j];
                r[j] = f * g;
                oa[j] = (r[j] * fc) * (HASB ? xs[q][j] : xs[q][j] - h[j]);
                if (HASB) {
                    gate_of(gb[q][j], i, ic);
                    oh[j] = g * i;
                    ob[j] = oh[j] * (h[j] * ic);
                } else {
                    oh[j] = g * fc;
                }
            }
            const int64_t o = base + q * p.d;
            vstore<Tout, CP, VEC>(static_cast<Tout*>(p.dh) + o, c0, lane, p.d, oh);
            vstore<Tout, CP, VEC>(static_cast<Tout*>(p.da) + o, c0, lane, p.d, oa);
            if (HASB) vstore<Tout, CP, VEC>(static_cast<Tout*>(p.db) + o, c0, lane, p.d, ob);
            if (HASZ) vstore<Tout, CP, VEC>(static_cast<Tout*>(p.dz) + o, c0, lane, p.d, oz);
        }
    }
}

template <typename Tin, typename Tout, bool VEC>
static cudaError_t bwd_t(const VscanParams& p, cudaStream_t st) {
    const unsigned grid = (unsigned)(p.units * p.nk);
    if (p.b)
        p.z ? vscan_bwd_kernel<Tin, Tout, true, true, VEC><<<grid, 256, 0, st>>>(p)
            : vscan_bwd_kernel<Tin, Tout, true, false, VEC><<<grid, 256, 0, st>>>(p);
    else
        p.z ? vscan_bwd_kernel<Tin, Tout, false, true, VEC><<<grid, 256, 0, st>>>(p)
            : vscan_bwd_kernel<Tin, Tout, false, false, VEC><<<grid, 256, 0, st>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_vscan_bwd(const VscanParams& p, int dtype, int out_dtype, cudaStream_t st) {
    typedef __nv_bfloat16 bf;
    if (dtype == NAJU_F32) return bwd_t<float, float, true>(p, st);
    const bool vec = p.d % 2 == 0;
    if (out_dtype == NAJU_BF16) return vec ? bwd_t<bf, bf, true>(p, st) : bwd_t<bf, bf, false>(p, st);
    return vec ? bwd_t<bf, float, true>(p, st) : bwd_t<bf, float, false>(p, st);
}

}  // namespace naju
