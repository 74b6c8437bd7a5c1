// Vector-state scan: forward and decode step.
#include "naju_kernels.h"
#include "naju_vscan.cuh"

namespace naju {

struct VscanMaps {
    CUtensorMap h, a, b, z;
};

// TMA: the item's rows come as one box of kVTokF rows x 128 bytes per tensor
// (rows past the sequence and channels past the width read as zero);
// otherwise every thread loads its own values.
template <typename Tin, typename Tout, bool HASB, bool HASZ, bool TMA, bool VEC>
__global__ void __launch_bounds__(kVThreads, 3)
vscan_fwd_kernel(const __grid_constant__ VscanParams p, const __grid_constant__ VscanMaps maps) {
    constexpr int CP = VRow<Tin>::CP, W = 32 * CP, RUN = kVRunF;
    constexpr int kBox = kVTokF * 128;                // bytes of one tensor's box
    constexpr int kNT = 2 + (HASB ? 1 : 0) + (HASZ ? 1 : 0);
    typedef Vf<CP> V;
    extern __shared__ __align__(128) unsigned char stage[];  // h, a, [b], [z]
    __shared__ VPair<CP> sagg[2][kVWarps][32];  // each warp's (P, X), by round parity
    __shared__ V sE[2][32];                     // the item's entering state
    __shared__ VExchange<CP> ex;
    __shared__ __align__(8) uint64_t full, empty;  // the stage is filled; has been read
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t cs = p.cluster, rank = cluster_rank();
    const unsigned u = blockIdx.x / cs;
    const int64_t bb = u / p.ntiles;
    const int c0 = (int)(u % p.ntiles) * W;
    const int nk = (int)p.nk, rounds = (nk + (int)cs - 1) / (int)cs;

    const auto fetch = [&](int k) {
        const int x = (int)(u % p.ntiles) * 64, t = k * kVTokF;
        tma::expect_tx(&full, kNT * kBox);
        tma::load_3d(stage, &maps.h, x, t, (int)bb, &full);
        tma::load_3d(stage + kBox, &maps.a, x, t, (int)bb, &full);
        if (HASB) tma::load_3d(stage + 2 * kBox, &maps.b, x, t, (int)bb, &full);
        if (HASZ) tma::load_3d(stage + (kNT - 1) * kBox, &maps.z, x, t, (int)bb, &full);
    };
    if (tid == 32 * kVWarps) {
        ex.init();
        mbar_init(&full, 1);
        mbar_init(&empty, kVWarps);
        mbar_init_release();
        if (TMA) {
            fence_proxy_async();
            if ((int)rank < nk) fetch(rank);
        }
    }
    __syncwarp();
    if (cs > 1)
        cluster_sync();  // every block's mbarriers exist before anything is sent to them
    else
        __syncthreads();

    if (warp == kVWarps) {  // ------------------------------------- scout
        const bool first = blockIdx.x == 0 && lane == 0;
        const StatusWord was = first ? status_begin(p) : 0;
        V E;
        const int64_t row = bb * p.d + c0;
        const int left = (int)min64(W, p.d - c0);
#pragma unroll
        for (int j = 0; j < CP; ++j) {
            const int ch = vchan<CP, VEC>(lane, j);
            E[j] = p.x0 && ch < left ? p.x0[row + ch] : 0.f;
        }
        bool alive = true;
        for (int i = 0; i < rounds; ++i) {
            const int par = i & 1, k = i * (int)cs + (int)rank;
            if (cs == 1) sE[par][lane] = E;  // known before the item is
            if (TMA && k + (int)cs < nk) {
                if (lane == 0) {
                    if (!mbar_wait(&empty, par, kTmaPolls))
                        status_timeout<true>(p);
                    fetch(k + cs);
                }
                __syncwarp();
            }
            named_bar(1, kVThreads);         // the warps' (P, X) are there
            VPair<CP> c = {vset<CP>(1.f), vset<CP>(0.f)};
#pragma unroll
            for (int w = 0; w < kVWarps; ++w) {
                const VPair<CP> g = sagg[par][w][lane];
                c.P = c.P * g.P;
                c.X = vfma(g.P, c.X, g.X);
            }
            // (a block whose wait ran out sends nothing from then on)
            if (cs > 1 && alive && !(p.fault_skip_publish && i == 0 && rank == 0))
                ex.send(i, rank, cs, lane, c);
            V mine = E;
            if (cs > 1) {
                mine = ex.template fold<true>(i, rank, cs, lane, E, alive, p);
                sE[par][lane] = mine;
                named_arrive(2, kVThreads);
            } else {
                E = vfma(c.P, E, c.X);
            }
            if (k < nk) {
                float* ck = p.ckpt + ((int64_t)u * p.nck + (int64_t)k * (kVTokF / kVTokB)) * W;
#pragma unroll
                for (int j = 0; j < CP; ++j) ck[vchan<CP, VEC>(lane, j)] = mine[j];
            }
        }
        if (rank == 0 && p.x_final) {
#pragma unroll
            for (int j = 0; j < CP; ++j) {
                const int ch = vchan<CP, VEC>(lane, j);
                if (ch < left) p.x_final[row + ch] = E[j];
            }
        }
        if (first) status_keep(p, was);
    } else {  // ------------------------------------------- compute warps
        const int cl = c0 + vchan<CP, VEC>(lane, 0);
        const int left = (int)p.d - cl;
        const uint32_t stride = (uint32_t)p.d * sizeof(Tout);
        const uint32_t off0 = ((uint32_t)(warp * RUN) * (uint32_t)p.d + cl) * sizeof(Tout);
        for (int i = 0; i < rounds; ++i) {
            const int par = i & 1, k = i * (int)cs + (int)rank;
            const int64_t tile = (bb * p.L + (int64_t)k * kVTokF) * p.d;  // uniform
            // this warp's tokens (<= 0: none)
            const int n = k < nk ? (int)min64(RUN, p.L - k * kVTokF - warp * RUN) : 0;
            V f[RUN], v[RUN], P = vset<CP>(1.f), X = vset<CP>(0.f);
            uint32_t rz[RUN];
            if (n > 0) {
                uint32_t rh[RUN], ra[RUN], rb[RUN];
                if (TMA) {
                    if (!mbar_wait(&full, par, kTmaPolls))
                        status_timeout<true>(p);
                    const unsigned char* at = stage + warp * RUN * 128 + lane * 4;
                    const auto get = [&](int which, int q) {
                        return *reinterpret_cast<const uint32_t*>(at + which * kBox + q * 128);
                    };
#pragma unroll
                    for (int q = 0; q < RUN; ++q) {
                        rh[q] = get(0, q);
                        ra[q] = get(1, q);
                        if (HASB) rb[q] = get(2, q);
                        if (HASZ) rz[q] = get(kNT - 1, q);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&empty);  // the next tiles may come in
                } else {
#pragma unroll
                    for (int q = 0; q < RUN; ++q) {
                        rh[q] = ra[q] = rb[q] = rz[q] = 0;
                        if (q < n) {
                            const int64_t o = tile + (int64_t)(warp * RUN + q) * p.d;
                            ra[q] = vload<Tin, VEC>(static_cast<const Tin*>(p.a) + o, c0, lane, p.d);
                            rh[q] = vload<Tin, VEC>(static_cast<const Tin*>(p.h) + o, c0, lane, p.d);
                            if (HASB)
                                rb[q] = vload<Tin, VEC>(static_cast<const Tin*>(p.b) + o, c0, lane,
                                                        p.d);
                            if (HASZ)
                                rz[q] = vload<Tin, VEC>(static_cast<const Tin*>(p.z) + o, c0, lane,
                                                        p.d);
                        }
                    }
                }
                // gates; this warp's (P, X) from a zero state
#pragma unroll
                for (int q = 0; q < RUN; ++q) {
                    V r, s;
                    if (HASB) {
                        V r2, s2;
                        gate_rs2<Tin>(ra[q], rb[q], r, s, r2, s2);
                        v[q] = gate_sel<Tin>(rb[q], r2, s2);
                    } else {
                        gate_rs<Tin>(ra[q], r, s);
                        v[q] = gate_sel<Tin>(ra[q], s, r);
                    }
                    f[q] = gate_sel<Tin>(ra[q], r, s);
                    v[q] = v[q] * VRow<Tin>::unpack(rh[q]);
                }
                if (n < RUN) {  // past the sequence: the identity
#pragma unroll
                    for (int q = 0; q < RUN; ++q)
                        if (q >= n) f[q] = vset<CP>(1.f), v[q] = vset<CP>(0.f);
                }
#pragma unroll
                for (int q = 0; q < RUN; ++q) {
                    P = P * f[q];
                    X = vfma(f[q], X, v[q]);
                }
            } else if (TMA && lane == 0) {
                mbar_arrive(&empty);  // (a warp past the sequence's end)
            }
            sagg[par][warp][lane] = {P, X};
            named_bar(1, kVThreads);
            // the warps before this one, while the exchange goes on
            VPair<CP> c = {vset<CP>(1.f), vset<CP>(0.f)};
            for (int w = 0; w < warp; ++w) {
                const VPair<CP> g = sagg[par][w][lane];
                c.P = c.P * g.P;
                c.X = vfma(g.P, c.X, g.X);
            }
            if (cs > 1) named_bar(2, kVThreads);
            if (n <= 0) continue;
            V x = vfma(c.P, sE[par][lane], c.X);  // this warp's entering state
            if (warp > 0 && warp * RUN % kVTokB == 0) {  // a checkpoint inside the item
                float* ck = p.ckpt + ((int64_t)u * p.nck + (int64_t)k * (kVTokF / kVTokB) +
                                      warp * RUN / kVTokB) * W;
#pragma unroll
                for (int j = 0; j < CP; ++j) ck[vchan<CP, VEC>(lane, j)] = x[j];
            }
            char* y = reinterpret_cast<char*>(static_cast<Tout*>(p.y) + tile);
            const auto token = [&](int q) {
                x = vfma(f[q], x, v[q]);
                V o = x;
                if (HASZ) {
                    const V z = VRow<Tin>::unpack(rz[q]);
                    o = x * (z * vsigm<CP>(z));
                }
                vstore<Tout, CP, VEC>(reinterpret_cast<Tout*>(y + (off0 + q * stride)), left, o);
            };
            if (n == RUN) {
#pragma unroll
                for (int q = 0; q < RUN; ++q) token(q);
            } else {
#pragma unroll
                for (int q = 0; q < RUN; ++q)
                    if (q < n) token(q);
            }
        }
    }
    // no block leaves while another may still send to it
    if (cs > 1) {
        __syncwarp();
        cluster_sync();
    }
}

template <typename Tin, typename Tout, bool HASB, bool HASZ, bool TMA, bool VEC>
static cudaError_t fwd_k(const VscanParams& p, const VscanMaps& maps, cudaStream_t st) {
    const int smem = TMA ? (2 + HASB + HASZ) * kVTokF * 128 : 0;
    static std::atomic<uint64_t> ready{0};
    return vscan_launch(vscan_fwd_kernel<Tin, Tout, HASB, HASZ, TMA, VEC>, p, maps, smem, ready,
                        st);
}

template <typename Tin, typename Tout, bool TMA, bool VEC>
static cudaError_t fwd_t(const VscanParams& p, const VscanMaps& m, cudaStream_t st) {
    if (p.b)
        return p.z ? fwd_k<Tin, Tout, true, true, TMA, VEC>(p, m, st)
                   : fwd_k<Tin, Tout, true, false, TMA, VEC>(p, m, st);
    return p.z ? fwd_k<Tin, Tout, false, true, TMA, VEC>(p, m, st)
               : fwd_k<Tin, Tout, false, false, TMA, VEC>(p, m, st);
}

// Rows as 2-byte elements (TMA moves bits; an fp32 value is two of them).
bool vscan_map(CUtensorMap* map, const void* base, int64_t Bt, int64_t L, int64_t d, int dtype,
               int rows) {
    return tma_encode_bf16_3d(map, base, Bt, L, dtype == NAJU_F32 ? 2 * d : d, rows, 64);
}

// Whether rows start on TMA's 16 bytes.
bool vscan_tma(int64_t d, int dtype) { return d * (dtype == NAJU_F32 ? 4 : 2) % 16 == 0; }

cudaError_t launch_vscan_fwd(const VscanParams& p, int dtype, int out_dtype, cudaStream_t st) {
    typedef __nv_bfloat16 bf;
    const int64_t Bt = p.units / p.ntiles;
    VscanMaps m{};
    if (vscan_tma(p.d, dtype)) {
        const auto enc = [&](CUtensorMap* map, const void* base) {
            return !base || vscan_map(map, base, Bt, p.L, p.d, dtype, kVTokF);
        };
        if (!(enc(&m.h, p.h) && enc(&m.a, p.a) && enc(&m.b, p.b) && enc(&m.z, p.z)))
            return cudaErrorInvalidValue;
        if (dtype == NAJU_F32) return fwd_t<float, float, true, true>(p, m, st);
        return out_dtype == NAJU_BF16 ? fwd_t<bf, bf, true, true>(p, m, st)
                                      : fwd_t<bf, float, true, true>(p, m, st);
    }
    if (dtype == NAJU_F32) return fwd_t<float, float, false, true>(p, m, st);
    if (p.d % 2 == 0)
        return out_dtype == NAJU_BF16 ? fwd_t<bf, bf, false, true>(p, m, st)
                                      : fwd_t<bf, float, false, true>(p, m, st);
    return out_dtype == NAJU_BF16 ? fwd_t<bf, bf, false, false>(p, m, st)
                                  : fwd_t<bf, float, false, false>(p, m, st);
}

int vscan_tile(int dtype) { return dtype == NAJU_F32 ? 32 : 64; }
int vscan_tokens() { return kVTokF; }
int vscan_tokens_bwd() { return kVTokB; }

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
        const uint32_t bits = __float_as_uint(av[k]);
        Vf<1> r, s;
        gate_rs<float>(bits, r, s);
        const float f = gate_sel<float>(bits, r, s).x, fc = gate_sel<float>(bits, s, r).x;
        x[k] = fmaf(f, x[k], (b ? sigmoidx_(bv[k]) : fc) * hv[k]);
        o[k] = z ? x[k] * (zv[k] * sigmoidx_(zv[k])) : x[k];
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
