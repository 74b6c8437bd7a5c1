// Vector-state scan: backward.
//
// With dx_t = dy_t SiLU(z_t) the adjoint is g_t = dx_t + r_{t+1}, where
// r_t = f_t g_t is what a token hands to the one before it (r_L = dx_final,
// r_0 = dx0).  A run of tokens acts on r as r -> P r + R with the forward's
// own P, so the runs compose like the forward's, in the other direction:
//   dh = g i,  db = g h i (1 - i),  da = g f (1 - f) x_{t-1}  (coupled:
//   x_{t-1} - h in its place),  dz = dy SiLU'(z) x.
// The states are recomputed from the forward's checkpoints (one fp32 value per
// 32 tokens and channel), which costs one multiply-add a token and saves
// reading them.
#include "naju_kernels.h"
#include "naju_vscan.cuh"

namespace naju {

struct VscanBwdMaps {
    CUtensorMap h, a, b, z, dy;
};

template <typename Tin, typename Tout, bool HASB, bool HASZ, bool TMA, bool VEC>
__global__ void __launch_bounds__(kVThreads, 2)
vscan_bwd_kernel(const __grid_constant__ VscanParams p,
                 const __grid_constant__ VscanBwdMaps maps) {
    constexpr int CP = VRow<Tin>::CP, W = 32 * CP, RUN = kVRunB;
    constexpr int kBox = kVTokB * 128;
    constexpr int kNT = 3 + (HASB ? 1 : 0) + (HASZ ? 1 : 0);
    typedef Vf<CP> V;
    extern __shared__ __align__(128) unsigned char stage[];  // h, a, dy, [b], [z]
    __shared__ VPair<CP> sagg[2][kVWarps][32];  // each warp's (P, X), by round parity
    __shared__ V srev[2][kVWarps][32];          // and R
    __shared__ V sE[2][32], sA[2][32];          // the item's entering state and adjoint
    __shared__ VExchange<CP> ex;
    __shared__ __align__(8) uint64_t full, empty;  // the stage is filled; has been read
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t cs = p.cluster, rank = cluster_rank();
    const unsigned u = blockIdx.x / cs;
    const int64_t bb = u / p.ntiles;
    const int c0 = (int)(u % p.ntiles) * W;
    // items in the order in which they are walked: o = 0 is the last one
    const int nk = (int)p.nk, rounds = (nk + (int)cs - 1) / (int)cs;

    const auto fetch = [&](int o) {
        const int x = (int)(u % p.ntiles) * 64, t = (nk - 1 - o) * kVTokB;
        tma::expect_tx(&full, kNT * kBox);
        tma::load_3d(stage, &maps.h, x, t, (int)bb, &full);
        tma::load_3d(stage + kBox, &maps.a, x, t, (int)bb, &full);
        tma::load_3d(stage + 2 * kBox, &maps.dy, x, t, (int)bb, &full);
        if (HASB) tma::load_3d(stage + 3 * kBox, &maps.b, x, t, (int)bb, &full);
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
        V A, E0;
        const int64_t row = bb * p.d + c0;
        const int left = (int)min64(W, p.d - c0);
        const auto state = [&](int o) {  // the checkpoint at the start of item o
#pragma unroll
            for (int j = 0; j < CP; ++j)
                E0[j] = o < nk ? p.ckpt[((int64_t)u * p.nck + (nk - 1 - o)) * W +
                                        vchan<CP, VEC>(lane, j)]
                               : 0.f;
        };
#pragma unroll
        for (int j = 0; j < CP; ++j) {
            const int ch = vchan<CP, VEC>(lane, j);
            A[j] = p.dx_final && ch < left ? p.dx_final[row + ch] : 0.f;
        }
        state(rank);
        bool alive = true;
        for (int i = 0; i < rounds; ++i) {
            const int par = i & 1, o = i * (int)cs + (int)rank;
            sE[par][lane] = E0;
            if (cs == 1) sA[par][lane] = A;  // known before the item is
            state(o + (int)cs);
            if (TMA && o + (int)cs < nk) {
                if (lane == 0) {
                    if (!mbar_wait(&empty, par, kTmaPolls))
                        status_timeout<false>(p);
                    fetch(o + cs);
                }
                __syncwarp();
            }
            named_bar(1, kVThreads);  // the warps' sums are there
            VPair<CP> c = {vset<CP>(1.f), vset<CP>(0.f)};
#pragma unroll
            for (int w = kVWarps - 1; w >= 0; --w) {
                const V g = sagg[par][w][lane].P;
                c.P = c.P * g;
                c.X = vfma(g, c.X, srev[par][w][lane]);
            }
            // (a block whose wait ran out sends nothing from then on)
            if (cs > 1 && alive && !(p.fault_skip_publish && i == 0 && rank == 0))
                ex.send(i, rank, cs, lane, c);
            if (cs > 1) {
                sA[par][lane] = ex.template fold<false>(i, rank, cs, lane, A, alive, p);
                named_arrive(2, kVThreads);
            } else {
                A = vfma(c.P, A, c.X);
            }
        }
        if (rank == 0 && p.dx0) {
#pragma unroll
            for (int j = 0; j < CP; ++j) {
                const int ch = vchan<CP, VEC>(lane, j);
                if (ch < left) p.dx0[row + ch] = A[j];
            }
        }
    } else {  // ------------------------------------------- compute warps
        const int cl = c0 + vchan<CP, VEC>(lane, 0);
        const int left = (int)p.d - cl;
        const uint32_t stride = (uint32_t)p.d * sizeof(Tout);
        const uint32_t off0 = ((uint32_t)(warp * RUN) * (uint32_t)p.d + cl) * sizeof(Tout);
        const V one = vset<CP>(1.f), minus = vset<CP>(-1.f);
        for (int i = 0; i < rounds; ++i) {
            const int par = i & 1, k = nk - 1 - (i * (int)cs + (int)rank);
            const int64_t tile = (bb * p.L + (int64_t)k * kVTokB) * p.d;  // uniform
            // this warp's tokens (<= 0: none)
            const int n = k >= 0 ? (int)min64(RUN, p.L - k * kVTokB - warp * RUN) : 0;
            // Kept per token: f, i, v = i h, dx, and the factors of g, g and x
            // in da, db and dz: m = f (1 - f), w = h i (1 - i) (coupled: -m h),
            // e = dy SiLU'(z).
            V f[RUN], m[RUN], gi[RUN], v[RUN], w[RUN], dx[RUN], e[RUN];
            V P = one, X = vset<CP>(0.f), R = vset<CP>(0.f);
            if (n > 0) {
                uint32_t rh[RUN], ra[RUN], rb[RUN], rz[RUN], rd[RUN];
                if (TMA) {
                    if (!mbar_wait(&full, par, kTmaPolls))
                        status_timeout<false>(p);
                    const unsigned char* at = stage + warp * RUN * 128 + lane * 4;
                    const auto get = [&](int which, int q) {
                        return *reinterpret_cast<const uint32_t*>(at + which * kBox + q * 128);
                    };
#pragma unroll
                    for (int q = 0; q < RUN; ++q) {
                        rh[q] = get(0, q);
                        ra[q] = get(1, q);
                        rd[q] = get(2, q);
                        if (HASB) rb[q] = get(3, q);
                        if (HASZ) rz[q] = get(kNT - 1, q);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&empty);  // the next tiles may come in
                } else {
#pragma unroll
                    for (int q = 0; q < RUN; ++q) {
                        rh[q] = ra[q] = rb[q] = rz[q] = rd[q] = 0;
                        if (q < n) {
                            const int64_t o = tile + (int64_t)(warp * RUN + q) * p.d;
                            ra[q] = vload<Tin, VEC>(static_cast<const Tin*>(p.a) + o, c0, lane, p.d);
                            rh[q] = vload<Tin, VEC>(static_cast<const Tin*>(p.h) + o, c0, lane, p.d);
                            rd[q] = vload<Tin, VEC>(static_cast<const Tin*>(p.dy) + o, c0, lane,
                                                    p.d);
                            if (HASB)
                                rb[q] = vload<Tin, VEC>(static_cast<const Tin*>(p.b) + o, c0, lane,
                                                        p.d);
                            if (HASZ)
                                rz[q] = vload<Tin, VEC>(static_cast<const Tin*>(p.z) + o, c0, lane,
                                                        p.d);
                        }
                    }
                }
#pragma unroll
                for (int q = 0; q < RUN; ++q) {
                    const V h = VRow<Tin>::unpack(rh[q]), dy = VRow<Tin>::unpack(rd[q]);
                    V r, s;
                    if (HASB) {
                        V r2, s2;
                        gate_rs2<Tin>(ra[q], rb[q], r, s, r2, s2);
                        gi[q] = gate_sel<Tin>(rb[q], r2, s2);
                        w[q] = h * (r2 * s2);
                        m[q] = r * s;
                    } else {
                        gate_rs<Tin>(ra[q], r, s);
                        gi[q] = gate_sel<Tin>(ra[q], s, r);
                        m[q] = r * s;
                        w[q] = m[q] * h * minus;
                    }
                    f[q] = gate_sel<Tin>(ra[q], r, s);
                    v[q] = gi[q] * h;
                    if (HASZ) {
                        const V z = VRow<Tin>::unpack(rz[q]);
                        const V sz = vsigm<CP>(z), zs = z * sz;
                        e[q] = dy * vfma(zs, vfma(sz, minus, one), sz);  // s + z s (1 - s)
                        dx[q] = dy * zs;
                    } else {
                        dx[q] = dy;
                    }
                }
                if (n < RUN) {  // past the sequence: the identity
#pragma unroll
                    for (int q = 0; q < RUN; ++q)
                        if (q >= n) f[q] = one, v[q] = dx[q] = vset<CP>(0.f);
                }
#pragma unroll
                for (int q = 0; q < RUN; ++q) {
                    P = P * f[q];
                    X = vfma(f[q], X, v[q]);
                    const int rq = RUN - 1 - q;
                    R = f[rq] * (dx[rq] + R);
                }
            } else if (TMA && lane == 0) {
                mbar_arrive(&empty);  // (a warp past the sequence's end)
            }
            sagg[par][warp][lane] = {P, X};
            srev[par][warp][lane] = R;
            named_bar(1, kVThreads);
            const auto at = [&](void* t, int q) {
                return reinterpret_cast<Tout*>(
                    reinterpret_cast<char*>(static_cast<Tout*>(t) + tile) + (off0 + q * stride));
            };
            // what needs no exchange goes before the second barrier: the
            // states with dz, and the sums of the warps behind this one
            VPair<CP> c = {one, vset<CP>(0.f)};
            if (n > 0) {
                V x = sE[par][lane];
                for (int o = 0; o < warp; ++o) {
                    const VPair<CP> g = sagg[par][o][lane];
                    x = vfma(g.P, x, g.X);
                }
#pragma unroll
                for (int q = 0; q < RUN; ++q) {
                    m[q] = HASB ? m[q] * x : vfma(m[q], x, w[q]);  // da / g
                    x = vfma(f[q], x, v[q]);
                    if (HASZ && q < n) vstore<Tout, CP, VEC>(at(p.dz, q), left, e[q] * x);
                }
                for (int o = kVWarps - 1; o > warp; --o) {
                    const V g = sagg[par][o][lane].P;
                    c.P = c.P * g;
                    c.X = vfma(g, c.X, srev[par][o][lane]);
                }
            }
            if (cs > 1) named_bar(2, kVThreads);
            if (n <= 0) continue;
            V r = vfma(c.P, sA[par][lane], c.X);  // the adjoint entering from behind
            const auto token = [&](int q) {
                const V g = dx[q] + r;
                r = f[q] * g;
                vstore<Tout, CP, VEC>(at(p.dh, q), left, g * gi[q]);
                vstore<Tout, CP, VEC>(at(p.da, q), left, g * m[q]);
                if (HASB) vstore<Tout, CP, VEC>(at(p.db, q), left, g * w[q]);
            };
            if (n == RUN) {
#pragma unroll
                for (int q = RUN - 1; q >= 0; --q) token(q);
            } else {
#pragma unroll
                for (int q = RUN - 1; q >= 0; --q)
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
static cudaError_t bwd_k(const VscanParams& p, const VscanBwdMaps& maps, cudaStream_t st) {
    const int smem = TMA ? (3 + HASB + HASZ) * kVTokB * 128 : 0;
    static std::atomic<uint64_t> ready{0};
    return vscan_launch(vscan_bwd_kernel<Tin, Tout, HASB, HASZ, TMA, VEC>, p, maps, smem, ready,
                        st);
}

template <typename Tin, typename Tout, bool TMA, bool VEC>
static cudaError_t bwd_t(const VscanParams& p, const VscanBwdMaps& m, cudaStream_t st) {
    if (p.b)
        return p.z ? bwd_k<Tin, Tout, true, true, TMA, VEC>(p, m, st)
                   : bwd_k<Tin, Tout, true, false, TMA, VEC>(p, m, st);
    return p.z ? bwd_k<Tin, Tout, false, true, TMA, VEC>(p, m, st)
               : bwd_k<Tin, Tout, false, false, TMA, VEC>(p, m, st);
}

cudaError_t launch_vscan_bwd(const VscanParams& p, int dtype, int out_dtype, cudaStream_t st) {
    typedef __nv_bfloat16 bf;
    const int64_t Bt = p.units / p.ntiles;
    VscanBwdMaps m{};
    if (vscan_tma(p.d, dtype)) {
        const auto enc = [&](CUtensorMap* map, const void* base) {
            return !base || vscan_map(map, base, Bt, p.L, p.d, dtype, kVTokB);
        };
        if (!(enc(&m.h, p.h) && enc(&m.a, p.a) && enc(&m.b, p.b) && enc(&m.z, p.z) &&
              enc(&m.dy, p.dy)))
            return cudaErrorInvalidValue;
        if (dtype == NAJU_F32) return bwd_t<float, float, true, true>(p, m, st);
        return out_dtype == NAJU_BF16 ? bwd_t<bf, bf, true, true>(p, m, st)
                                      : bwd_t<bf, float, true, true>(p, m, st);
    }
    if (dtype == NAJU_F32) return bwd_t<float, float, false, true>(p, m, st);
    if (p.d % 2 == 0)
        return out_dtype == NAJU_BF16 ? bwd_t<bf, bf, false, true>(p, m, st)
                                      : bwd_t<bf, float, false, true>(p, m, st);
    return out_dtype == NAJU_BF16 ? bwd_t<bf, bf, false, false>(p, m, st)
                                  : bwd_t<bf, float, false, false>(p, m, st);
}

}  // namespace naju
