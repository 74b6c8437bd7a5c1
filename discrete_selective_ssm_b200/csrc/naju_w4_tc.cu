// 4-bit projections on the 5th-generation tensor cores (sm_100a): bf16 x.
//
// A block owns 128 rows of W (tensor-memory lanes) and N rows of x (accumulator
// columns) and walks its share of the inputs in blocks of 128:
//   loader  (1 warp): TMA of the packed weights (128 rows x 64 bytes, swizzled
//           so that a thread reads its row without bank conflicts) and of x
//           (128-byte swizzled K-major operand tiles, straight from memory);
//   unpackers (4 warps, a thread a row): 4-bit words to bf16 (q - 8) / 1024,
//           exact, into tensor memory as the A operand: no trip through
//           shared memory, whose bandwidth would bound it;
//   issuer  (1 warp): tcgen05.mma kind::f16, A from tensor memory, one
//           accumulator per scale group, two in turn;
//   adders  (4 warps, a thread a row): a finished group's N sums times its
//           scale into fp32 registers.
// So every product and every sum is exact or fp32, as in the warp-level kernel.
// The blocks of a cluster share the inputs and add their sums through
// distributed shared memory in fixed order.
// Bound by the hand-over between the warps, which wait for tensor memory and
// for one another (issue slots 38 to 44 % busy, tensor pipe 13 and 24 %):
// 256 x 2048 -> 4096 17.5 us in groups of 64, 64 x 8192 -> 28672 63 us (235 us
// in the warp-level form).  Groups of 32 with 64 rows of x spill 212 bytes:
// 256 x 2048 -> 4096 28 us.
#include <cooperative_groups.h>

#include "naju_common.cuh"
#include "naju_kernels.h"
#include "naju_tc.cuh"
#include "naju_tma.h"
#include "naju_w4.cuh"

namespace naju {

using namespace tc;

namespace {

constexpr int kTcThreads = 320;
constexpr int kTcPolls = 1 << 20;

// Shared memory of a stage, two blocks of 128 inputs: packed weights (128 rows
// of 128 bytes), then x (N rows x 256 inputs, four 64-column tiles).
template <int N> struct W4Tc {
    static constexpr int kWBytes = 128 * 128, kXBytes = N * 512;
    static constexpr int kStage = kWBytes + kXBytes;
    static constexpr int kStages = N == 16 ? 4 : N == 32 ? 3 : 2;  // two blocks on an SM
    static constexpr int kRing = kStages * kStage;
    static constexpr int kRed = N * 128 * 4;  // the sums, over the ring when it is done
    static constexpr int kSmem = (kRing > kRed ? kRing : kRed) + 1024;
    // tensor memory: two accumulators, two A blocks (128 bf16 = 64 columns)
    static constexpr int kA = 2 * N, kCols = 256;
    static_assert(2 * N + 128 <= kCols, "two blocks share an SM's 512 columns");
};

// D[tmem] (+)= A[tmem] * B[smem]^T, one K = 16 step of bf16 operands.
__device__ __forceinline__ void mma_bf16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
        "%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(
            taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
        "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]),
        "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]),
        "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}

// Bounded wait of a whole warp for a phase; once one has run out (*bad), none
// waits any more.
__device__ __forceinline__ void wait_phase(uint64_t* bar, uint32_t phase, int* bad) {
    int polls = 0;
    while (!mbar_try_wait(bar, phase)) {
        if (++polls > kTcPolls) *bad = 1;
        if (*(volatile int*)bad) break;
    }
}

}  // namespace

template <int G, int N>
__global__ void __launch_bounds__(kTcThreads, 2)
w4_tc_kernel(const __grid_constant__ W4Params p, const __grid_constant__ CUtensorMap wmap,
             const __grid_constant__ CUtensorMap xmap) {
    typedef W4Tc<N> C;
    typedef __nv_bfloat16 bf;
    constexpr int S = C::kStages, GPB = 128 / G, kSteps = G / 16;
    namespace cg = cooperative_groups;
    extern __shared__ unsigned char raw[];
    unsigned char* ring = raw + (-smem_u32(raw) & 1023u);
    __shared__ __align__(8) uint64_t full[S], empty[S], afull[2], aempty[2], dfull[2], dempty[2];
    __shared__ uint32_t s_tmem;
    __shared__ int s_bad;  // a wait ran out: the result is NaN
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const unsigned rank = blockIdx.x % p.split;
    const int64_t row0 = (int64_t)(blockIdx.x / p.split) * 128;
    const int col0 = blockIdx.y * N;
    const int b0 = (int)(p.nb * rank / p.split), b1 = (int)(p.nb * (rank + 1) / p.split);

    if (tid == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 5);  // four unpacking warps, the products that read x
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&afull[i], 4);
            mbar_init(&aempty[i], 1);
            mbar_init(&dfull[i], 1);
            mbar_init(&dempty[i], 4);
        }
        s_bad = 0;
        fence_proxy_async();
    }
    if (warp == 0) {
        tmem_alloc(&s_tmem, C::kCols);
        tmem_relinquish();
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tm = s_tmem;
    if (warp < 4) {  // --------------------------------------------- unpackers
        const PairBits bits;
        const uint32_t lanes = (uint32_t)(warp * 32) << 16;
        for (int b = b0; b < b1; ++b) {
            const int i = b - b0, st = i >> 1, s = st % S, ab = i & 1;
            if (!(i & 1)) wait_phase(&full[s], (st / S) & 1, &s_bad);
            const unsigned char* line = ring + s * C::kStage + tid * 128;
            uint4 w[4];
#pragma unroll
            for (int c = 0; c < 4; ++c)  // 128-byte swizzle: chunk ^ row % 8
                w[c] = *reinterpret_cast<const uint4*>(
                    line + ((((i & 1) * 4 + c) ^ (tid & 7)) << 4));
            uint32_t v[64];  // column: two inputs
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        v[16 * j + 4 * c + q] =
                            unpack_pair(reinterpret_cast<const uint32_t*>(&w[c])[j], q, bits);
            __syncwarp();
            if (lane == 0 && ((i & 1) || b + 1 == b1)) mbar_arrive(&empty[s]);
            wait_phase(&aempty[ab], ((i >> 1) & 1) ^ 1, &s_bad);
            fence_after_sync();
            const uint32_t a = tm + lanes + C::kA + ab * 64;
            tmem_st32(a, v);
            tmem_st32(a + 32, v + 32);
            tmem_st_wait();
            fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&afull[ab]);
        }
    } else if (warp < 8) {  // ---------------------------------------- adders
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const int r = tid - 128;
        const int64_t row = row0 + r;
        const bf* sc = p.scales + (row < p.n_out ? row : 0) * p.ng;
        const auto scale = [&](int g) {
            return g < p.ng && row < p.n_out ? __bfloat162float(sc[g]) : 0.f;
        };
        float2 acc[N / 2];
#pragma unroll
        for (int n = 0; n < N / 2; ++n) acc[n] = make_float2(0.f, 0.f);
        float next[GPB];
#pragma unroll
        for (int g = 0; g < GPB; ++g) next[g] = scale(b0 * GPB + g);
        int u = 0;  // groups so far
        for (int b = b0; b < b1; ++b) {
            float cur[GPB];
#pragma unroll
            for (int g = 0; g < GPB; ++g) {
                cur[g] = next[g];
                next[g] = scale((b + 1) * GPB + g);
            }
#pragma unroll
            for (int g = 0; g < GPB; ++g, ++u) {
                wait_phase(&dfull[u & 1], (u >> 1) & 1, &s_bad);
                fence_after_sync();
                const uint32_t d = tm + lanes + (u & 1) * N;
                const float2 s2 = make_float2(cur[g], cur[g]);
#pragma unroll
                for (int n = 0; n < N; n += 16) {
                    float t[16];
                    tmem_ld16(d + n, t);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        acc[n / 2 + e] = __ffma2_rn(s2, make_float2(t[2 * e], t[2 * e + 1]),
                                                    acc[n / 2 + e]);
                }
                fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&dempty[u & 1]);
            }
        }
        // all products are done: the ring becomes the sums [column][row]
        float* red = reinterpret_cast<float*>(ring);
#pragma unroll
        for (int n = 0; n < N / 2; ++n) {
            red[(2 * n) * 128 + r] = acc[n].x;
            red[(2 * n + 1) * 128 + r] = acc[n].y;
        }
    } else if (warp == 8) {  // --------------------------------------- loader
        for (int b = b0; b < b1; b += 2) {
            const int i = (b - b0) >> 1, s = i % S;
            wait_phase(&empty[s], ((i / S) & 1) ^ 1, &s_bad);
            if (lane == 0) {
                unsigned char* st = ring + s * C::kStage;
                tma::expect_tx(&full[s], C::kStage);
                tma::load_3d(st, &wmap, b * 32, (int)row0, 0, &full[s]);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    tma::load_3d(st + C::kWBytes + q * N * 128, &xmap, b * 128 + q * 64, col0, 0,
                                 &full[s]);
            }
        }
    } else {  // ------------------------------------------------------ issuer
        constexpr uint32_t idesc = idesc_bf16(128, N);
        int u = 0;
        for (int b = b0; b < b1; ++b) {
            const int i = b - b0, st = i >> 1, s = st % S, ab = i & 1;
            // (the unpackers have seen the stage full before they say so here)
            wait_phase(&afull[ab], (i >> 1) & 1, &s_bad);
            fence_after_sync();
            const uint32_t xb =
                smem_u32(ring + s * C::kStage + C::kWBytes + (i & 1) * N * 256);
            const uint32_t a = tm + C::kA + ab * 64;
#pragma unroll
            for (int g = 0; g < GPB; ++g, ++u) {
                wait_phase(&dempty[u & 1], ((u >> 1) & 1) ^ 1, &s_bad);
                fence_after_sync();
                if (lane == 0) {
#pragma unroll
                    for (int k = 0; k < kSteps; ++k) {
                        const int ks = g * kSteps + k;
                        mma_bf16_ts(tm + (u & 1) * N, a + 8 * ks, sdesc_bfw_k(xb, N, ks), idesc,
                                    k > 0);
                    }
                    mma_commit(&dfull[u & 1]);
                    if (g == GPB - 1) {
                        mma_commit(&aempty[ab]);
                        if ((i & 1) || b + 1 == b1) mma_commit(&empty[s]);
                    }
                }
                __syncwarp();
            }
        }
    }
    __syncwarp();
    fence_before_sync();
    cg::cluster_group cl = cg::this_cluster();
    if (p.split > 1)
        cl.sync();
    else
        __syncthreads();
    if (warp == 0) {
        fence_after_sync();
        tmem_dealloc(tm, C::kCols);
    }
    const float* red = reinterpret_cast<const float*>(ring);
    bool bad = s_bad;
    for (int s = 0; p.split > 1 && s < p.split; ++s) bad |= *cl.map_shared_rank(&s_bad, s) != 0;
#pragma unroll 2
    for (int e = rank * kTcThreads + tid; e < N * 32; e += kTcThreads * p.split) {
        const int64_t o = row0 + e % 32 * 4, m = col0 + e / 32;
        if (o >= p.n_out || m >= p.m) continue;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int s = 0; s < p.split; ++s) {  // in fixed order
            const float* from = p.split > 1 ? cl.map_shared_rank(red, s) : red;
            v = v + reinterpret_cast<const float4*>(from)[e];
        }
        if (bad) v = make_float4(NAN, NAN, NAN, NAN);
        w4_finish<bf>(p, m, o, v);
    }
    if (p.split > 1) cl.sync();  // no block leaves while another reads from it
}

template <int G, int N>
static cudaError_t tc_run(W4Params p, int sms, cudaStream_t st) {
    typedef W4Tc<N> C;
    static std::atomic<uint64_t> ready{0};
    CUtensorMap wmap, xmap;
    if (!tma_encode_bf16_3d_sw128(&wmap, p.wq, 1, p.n_out, p.nb * 32, 128) ||
        !tma_encode_bf16_3d_sw128(&xmap, p.x, 1, p.m, p.n_in, N))
        return cudaErrorInvalidValue;
    const int64_t rt = (p.n_out + 127) / 128, ct = (p.m + N - 1) / N;
    const int64_t slots = 2 * (int64_t)sms;
    p.split = 1;
    // Blocks per row tile: the fewest rounds of blocks, each as long as its
    // share of the inputs plus what a block takes to start and to add up
    // (about eight blocks of inputs).
    double best = 1e30;
    for (int s = 1; s <= 8 && s <= p.nb; ++s) {
        const double c = (double)((rt * ct * s + slots - 1) / slots) *
                         (double)((p.nb + s - 1) / s + 8);
        if (c < best - 1e-9) {
            best = c;
            p.split = s;
        }
    }
    return w4_launch(w4_tc_kernel<G, N>, dim3((unsigned)(rt * p.split), (unsigned)ct), kTcThreads,
                     C::kSmem, p.split, ready, st, p, wmap, xmap);
}

template <int G>
static cudaError_t tc_pick(const W4Params& p, int sms, cudaStream_t st) {
    if (p.m <= 16) return tc_run<G, 16>(p, sms, st);
    if (p.m <= 32) return tc_run<G, 32>(p, sms, st);
    return tc_run<G, 64>(p, sms, st);  // (128 at a time: no faster, 256 x 2048 -> 4096)
}

cudaError_t launch_w4_tc(const W4Params& p, int group, int sms, cudaStream_t st) {
    if (group == 32) return tc_pick<32>(p, sms, st);
    if (group == 64) return tc_pick<64>(p, sms, st);
    return tc_pick<128>(p, sms, st);
}

}  // namespace naju
