// 4-bit projections: quantiser and y = x W^T (+ bias) (+ residual) for a few
// rows of x (sm_100a; bound by reading the weights once).
//
// W[o, k] = s[o, k / G] (q[o, k] - 8).  q - 8 is exact in bf16, so the product
// runs on the tensor cores over the integers themselves: a group's sum
// sum_k (q - 8) x is accumulated in fp32 (every product exact) and multiplied
// by the group's scale once, in fp32.  Nothing is rounded to bf16 but the
// result.  fp32 x is split into three bf16 parts that add up to it exactly,
// three products instead of one.
//
// mma.m16n8k16 with the weights as the 16-row operand and x as the 8-column
// one.  Only a few columns of x exist, so the tensor rate does not matter and
// the warp-level form saves what tcgen05 needs on top: a weight goes from its
// 4 bits in a register to the operand fragment in the same register (shift,
// mask, subtract), with no trip through shared memory.  The K order of a
// fragment is free as long as both operands agree: the packed words are laid
// out so that a lane's 16 bytes are its fragments of eight k-steps, and four
// lanes' j-th words are one run of 32 inputs (so that groups of 32 work).
#include <cooperative_groups.h>

#include <atomic>

#include "naju_common.cuh"
#include "naju_kernels.h"

namespace naju {

// -------------------------------------------------------------- quantiser
// One warp per (row, 128-input block); lane l handles inputs 4 l .. 4 l + 3
// and a group's maximum is taken over G / 4 lanes.
template <typename T>
__global__ void __launch_bounds__(128)
w4_quantize_kernel(int64_t n_out, int64_t n_in, int group, const T* __restrict__ W,
                   uint32_t* __restrict__ wq, __nv_bfloat16* __restrict__ scales) {
    __shared__ unsigned char sq[4][128];
    const int64_t nb = (n_in + 127) / 128, ng = (n_in + group - 1) / group;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t id = (int64_t)blockIdx.x * 4 + warp;
    if (id >= n_out * nb) return;
    const int64_t row = id / nb, b = id % nb;
    float v[4], m = 0.f;
    bool bad = false;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int64_t k = b * 128 + lane * 4 + e;
        v[e] = k < n_in ? to_f(W[row * n_in + k]) : 0.f;
        m = fmaxf(m, fabsf(v[e]));
        bad |= !(fabsf(v[e]) < INFINITY);
    }
    if (bad) m = INFINITY;
    for (int o = 1; o < group / 4; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const __nv_bfloat16 s16 = __float2bfloat16_rn(m < INFINITY ? __fdiv_rn(m, 7.f) : NAN);
    const float s = __bfloat162float(s16);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float q = s > 0.f ? rintf(__fdiv_rn(v[e], s)) : 0.f;
        sq[warp][lane * 4 + e] = (unsigned char)(8 + (int)fminf(fmaxf(q, -8.f), 7.f));
    }
    const int64_t k0 = b * 128 + lane * 4;
    if (k0 % group == 0 && k0 < n_in) scales[row * ng + k0 / group] = s16;
    __syncwarp();
    if (lane < 16) {  // word 4 c + j: inputs 32 j + 8 c .. + 7
        const unsigned char* q = &sq[warp][32 * (lane & 3) + 8 * (lane >> 2)];
        uint32_t w = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) w |= (uint32_t)q[e] << (4 * (e / 2 + 4 * (e & 1)));
        wq[id * 16 + lane] = w;
    }
}

cudaError_t launch_w4_quantize(int64_t n_out, int64_t n_in, int group, int dtype, const void* W,
                               void* wq, void* scales, cudaStream_t st) {
    const int64_t blocks = (n_out * ((n_in + 127) / 128) + 3) / 4;
    if (dtype == NAJU_F32)
        w4_quantize_kernel<float><<<(unsigned)blocks, 128, 0, st>>>(
            n_out, n_in, group, static_cast<const float*>(W), static_cast<uint32_t*>(wq),
            static_cast<__nv_bfloat16*>(scales));
    else
        w4_quantize_kernel<__nv_bfloat16><<<(unsigned)blocks, 128, 0, st>>>(
            n_out, n_in, group, static_cast<const __nv_bfloat16*>(W), static_cast<uint32_t*>(wq),
            static_cast<__nv_bfloat16*>(scales));
    return cudaGetLastError();
}

// ---------------------------------------------------------------- product
__device__ __forceinline__ void mma_bf16(float* d, uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Nibbles i and i + 4 of a word (inputs 2 i, 2 i + 1) as two bf16 of
// (q - 8) / 1024: or-ing q into the bits of 128 gives 128 + q, exactly.  The
// factor keeps a group's sum (at most 128 * 8 values of x) in range for every
// finite x; the sums are multiplied by 1024 once, at the end.
__device__ __forceinline__ uint32_t unpack_pair(uint32_t w, int i) {
    uint32_t t = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;
    const __nv_bfloat162 r =
        __hfma2(*reinterpret_cast<__nv_bfloat162*>(&t), __float2bfloat162_rn(1.f / 1024.f),
                __float2bfloat162_rn(-136.f / 1024.f));
    return *reinterpret_cast<const uint32_t*>(&r);
}

// fp32 as three bf16 that add up to it (each takes the leading 8 bits of what
// is left, cut off, so nothing overflows); an infinity or a NaN in the first.
__device__ __forceinline__ void split3(float x, uint32_t& h, uint32_t& m, uint32_t& l) {
    if (!(fabsf(x) < INFINITY)) {
        h = __bfloat16_as_ushort(__float2bfloat16_rn(x));
        m = l = 0;
        return;
    }
    const uint32_t hb = __float_as_uint(x) & 0xffff0000u;
    const float r = x - __uint_as_float(hb);
    const uint32_t mb = __float_as_uint(r) & 0xffff0000u;
    h = hb >> 16;
    m = mb >> 16;
    l = __float_as_uint(r - __uint_as_float(mb)) >> 16;
}

struct W4Params {
    const void* x;
    const uint4* wq;
    const __nv_bfloat16* scales;
    const float* bias;
    const void* residual;
    void* y;
    int64_t m, n_in, n_out, nb, ng;  // nb: 128-input blocks of a row, ng: groups of a row
    int split;                       // blocks of a cluster, each with a share of the inputs
};

// General form.  WR warps along the rows of W (16 each), WK along the inputs;
// NT tiles of 8 rows of x.  A chunk is BPW blocks of 128 inputs for each of the
// WK warps; the next chunk's x comes into the other half of the stage and its
// weights into registers while this one is computed.
template <typename T, int WR, int WK, int NT, int G>
__global__ void __launch_bounds__(256) w4_linear_kernel(const W4Params p) {
    constexpr int SP = sizeof(T) == 4 ? 3 : 1;   // bf16 parts of an x value
    constexpr int BPW = SP == 1 ? 2 : 1, KC = BPW * WK;  // blocks per warp and chunk, per chunk
    constexpr int GPB = 128 / G;                 // groups per block
    constexpr int ROWS = 16 * WR, COLS = 8 * NT;
    static_assert(WR * WK == 8, "eight warps");
    // x as operand fragments, twice: [part][block][j][tile][n][c] of 16 bytes (8 inputs)
    extern __shared__ __align__(16) unsigned char smem[];
    uint4* xs0 = reinterpret_cast<uint4*>(smem);
    float* red = reinterpret_cast<float*>(smem);  // [WK][COLS][ROWS] after the last chunk
    constexpr int PART = KC * 4 * NT * 32;        // 16-byte units of one part
    namespace cg = cooperative_groups;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int wr = warp % WR, wk = warp / WR;
    const unsigned rank = blockIdx.x % p.split;
    const int64_t row0 = (int64_t)(blockIdx.x / p.split) * ROWS;
    const int64_t col0 = (int64_t)blockIdx.y * COLS;
    const int r = lane >> 2, c = lane & 3;
    const int64_t ra = row0 + wr * 16 + r, rb = ra + 8;
    // this block's share of the chunks
    const int64_t nch = (p.nb + KC - 1) / KC;
    const int64_t ch0 = nch * rank / p.split, ch1 = nch * (rank + 1) / p.split;

    uint4 wa[BPW], wb[BPW];
    __nv_bfloat16 sa[BPW][GPB], sb[BPW][GPB];
    const auto load_w = [&](int64_t ch) {
#pragma unroll
        for (int i = 0; i < BPW; ++i) {
            const int64_t b = ch * KC + i * WK + wk;
            wa[i] = wb[i] = make_uint4(0, 0, 0, 0);
            if (b < p.nb) {
                if (ra < p.n_out) wa[i] = __ldg(p.wq + (ra * p.nb + b) * 4 + c);
                if (rb < p.n_out) wb[i] = __ldg(p.wq + (rb * p.nb + b) * 4 + c);
            }
#pragma unroll
            for (int g = 0; g < GPB; ++g) {
                const int64_t gi = b * GPB + g;
                const bool ok = b < p.nb && gi < p.ng;
                sa[i][g] = ok && ra < p.n_out ? p.scales[ra * p.ng + gi] : __nv_bfloat16(0.f);
                sb[i][g] = ok && rb < p.n_out ? p.scales[rb * p.ng + gi] : __nv_bfloat16(0.f);
            }
        }
    };
    const T* x = static_cast<const T*>(p.x);
    const bool xvec = p.n_in % (16 / sizeof(T)) == 0;  // rows start on 16 bytes
    const auto stage_x = [&](int64_t ch, uint4* xs) {
        for (int e = tid; e < KC * 16 * COLS; e += 256) {
            const int unit = e % (KC * 16), n = e / (KC * 16);  // 8 inputs of one row of x
            const int64_t k = ch * KC * 128 + unit * 8, row = col0 + n;
            const int b = unit / 16, j = unit % 16 / 4, cc = unit % 4;
            const int at = ((b * 4 + j) * NT + n / 8) * 32 + n % 8 * 4 + cc;
            const bool in = row < p.m;
            if constexpr (SP == 1) {
                const __nv_bfloat16* src = x + row * p.n_in + k;
                if (xvec) {
                    const bool ok = in && k < p.n_in;
                    cp_async16(xs + at, ok ? src : x, ok ? 16 : 0);
                } else {
                    uint32_t h[8];
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        h[q] = in && k + q < p.n_in ? __bfloat16_as_ushort(src[q]) : 0u;
                    xs[at] = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16,
                                        h[6] | h[7] << 16);
                }
            } else {
                float f[8];
                const float* src = x + row * p.n_in + k;
                if (in && xvec && k + 8 <= p.n_in) {
                    load8(src, f);
                } else {
#pragma unroll
                    for (int q = 0; q < 8; ++q) f[q] = in && k + q < p.n_in ? src[q] : 0.f;
                }
                uint32_t h[8], m[8], l[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) split3(f[q], h[q], m[q], l[q]);
                const auto pack = [](const uint32_t* u) {
                    return make_uint4(u[0] | u[1] << 16, u[2] | u[3] << 16, u[4] | u[5] << 16,
                                      u[6] | u[7] << 16);
                };
                xs[at] = pack(h);
                xs[PART + at] = pack(m);
                xs[2 * PART + at] = pack(l);
            }
        }
    };

    float acc[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[t][e] = 0.f;

    if (ch0 < ch1) {
        load_w(ch0);
        stage_x(ch0, xs0);
        cp_async_commit();
    }
    for (int64_t ch = ch0; ch < ch1; ++ch) {
        const uint4* xs = xs0 + ((ch - ch0) & 1) * SP * PART;
        cp_async_wait<0>();
        __syncthreads();  // this chunk's x is there, the other half is read
        uint4 ca[BPW], cb[BPW];
        float fa[BPW][GPB], fb[BPW][GPB];
#pragma unroll
        for (int i = 0; i < BPW; ++i) {
            ca[i] = wa[i];
            cb[i] = wb[i];
#pragma unroll
            for (int g = 0; g < GPB; ++g) {
                fa[i][g] = __bfloat162float(sa[i][g]);
                fb[i][g] = __bfloat162float(sb[i][g]);
            }
        }
        if (ch + 1 < ch1) {
            load_w(ch + 1);
            stage_x(ch + 1, xs0 + ((ch + 1 - ch0) & 1) * SP * PART);
            cp_async_commit();
        }
#pragma unroll
        for (int i = 0; i < BPW; ++i) {
            const uint32_t* ua = reinterpret_cast<const uint32_t*>(&ca[i]);
            const uint32_t* ub = reinterpret_cast<const uint32_t*>(&cb[i]);
            const int b = i * WK + wk;
            float part[NT][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (j % (4 / GPB) == 0) {
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int e = 0; e < 4; ++e) part[t][e] = 0.f;
                }
                uint32_t pa[4], pb[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    pa[q] = unpack_pair(ua[j], q);
                    pb[q] = unpack_pair(ub[j], q);
                }
#pragma unroll
                for (int s = 0; s < SP; ++s) {
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const uint4 v = xs[s * PART + ((b * 4 + j) * NT + t) * 32 + lane];
                        mma_bf16(part[t], pa[0], pb[0], pa[1], pb[1], v.x, v.y);
                        mma_bf16(part[t], pa[2], pb[2], pa[3], pb[3], v.z, v.w);
                    }
                }
                if ((j + 1) % (4 / GPB) == 0) {
                    const int g = j / (4 / GPB);
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        acc[t][0] = fmaf(fa[i][g], part[t][0], acc[t][0]);
                        acc[t][1] = fmaf(fa[i][g], part[t][1], acc[t][1]);
                        acc[t][2] = fmaf(fb[i][g], part[t][2], acc[t][2]);
                        acc[t][3] = fmaf(fb[i][g], part[t][3], acc[t][3]);
                    }
                }
            }
        }
    }
    __syncthreads();

    // sums over the WK warps, then over the cluster's blocks, in fixed order
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int col = t * 8 + c * 2 + (e & 1), row = wr * 16 + r + (e >> 1) * 8;
            red[(wk * COLS + col) * ROWS + row] = acc[t][e];
        }
    }
    cg::cluster_group cl = cg::this_cluster();
    if (p.split > 1)
        cl.sync();
    else
        __syncthreads();
    for (int e = rank * 256 + tid; e < ROWS * COLS; e += 256 * p.split) {
        const int row = e % ROWS, col = e / ROWS;
        const int64_t o = row0 + row, m = col0 + col;
        if (o >= p.n_out || m >= p.m) continue;
        float v = 0.f;
        for (int s = 0; s < p.split; ++s) {
            const float* from = p.split > 1 ? cl.map_shared_rank(red, s) : red;
#pragma unroll
            for (int k = 0; k < WK; ++k) v += from[(k * COLS + col) * ROWS + row];
        }
        v *= 1024.f;
        if (p.bias) v += p.bias[o];
        if (p.residual) v += to_f(static_cast<const T*>(p.residual)[m * p.n_out + o]);
        static_cast<T*>(p.y)[m * p.n_out + o] = from_f<T>(v);
    }
    if (p.split > 1) cl.sync();  // no block leaves while another reads from it
}

// Up to eight rows of bf16 x that start on 16 bytes (the decode of a few
// sessions, where the time is that of reading the weights): no stage and no
// barrier before the sum.  Eight warps share 16 rows of W, each takes every
// eighth block of the inputs (of this block's share), the x of its fragments
// straight from global memory (L1 holds it: all rows of W use the same), and
// has the weights of its next UB blocks in flight.
template <int G>
__global__ void __launch_bounds__(256, 2) w4_rows_kernel(const W4Params p) {
    constexpr int GPB = 128 / G, UB = 4;
    __shared__ float red[8][8][16];  // [warp][row of x][row of W]
    namespace cg = cooperative_groups;
    typedef __nv_bfloat16 bf;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const unsigned rank = blockIdx.x % p.split;
    const int64_t row0 = (int64_t)(blockIdx.x / p.split) * 16;
    const int r = lane >> 2, c = lane & 3;
    const bool oka = row0 + r < p.n_out, okb = row0 + r + 8 < p.n_out;
    const int nb = (int)p.nb, step = 8 * p.split;
    const uint4* wa = p.wq + (oka ? (row0 + r) * p.nb * 4 : 0) + c;
    const uint4* wb = p.wq + (okb ? (row0 + r + 8) * p.nb * 4 : 0) + c;
    const bf* sa = p.scales + (oka ? (row0 + r) * p.ng : 0);
    const bf* sb = p.scales + (okb ? (row0 + r + 8) * p.ng : 0);
    const bool okx = r < p.m;
    const bf* x = static_cast<const bf*>(p.x) + (okx ? r * p.n_in : 0) + 8 * c;

    uint4 qa[UB], qb[UB];
    bf fa[UB][GPB], fb[UB][GPB];
    const auto load = [&](int b0) {
#pragma unroll
        for (int i = 0; i < UB; ++i) {
            const int b = b0 + i * step;
            qa[i] = qb[i] = make_uint4(0, 0, 0, 0);
            if (b < nb) {
                if (oka) qa[i] = __ldg(wa + (int64_t)b * 4);
                if (okb) qb[i] = __ldg(wb + (int64_t)b * 4);
            }
#pragma unroll
            for (int g = 0; g < GPB; ++g) {
                const int gi = b * GPB + g;
                const bool ok = b < nb && gi < p.ng;
                fa[i][g] = ok && oka ? sa[gi] : bf(0.f);
                fb[i][g] = ok && okb ? sb[gi] : bf(0.f);
            }
        }
    };
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    int b0 = rank * 8 + warp;
    load(b0);
    for (; b0 < nb; b0 += UB * step) {
        uint4 ca[UB], cb[UB];
        float ga[UB][GPB], gb[UB][GPB];
#pragma unroll
        for (int i = 0; i < UB; ++i) {
            ca[i] = qa[i];
            cb[i] = qb[i];
#pragma unroll
            for (int g = 0; g < GPB; ++g) {
                ga[i][g] = __bfloat162float(fa[i][g]);
                gb[i][g] = __bfloat162float(fb[i][g]);
            }
        }
        load(b0 + UB * step);
#pragma unroll
        for (int i = 0; i < UB; ++i) {
            const int b = b0 + i * step;
            if (b >= nb) break;
            uint4 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int k = b * 128 + 32 * j;
                v[j] = make_uint4(0, 0, 0, 0);
                if (okx && k + 8 * c < p.n_in) v[j] = __ldg(reinterpret_cast<const uint4*>(x + k));
            }
            const uint32_t* ua = reinterpret_cast<const uint32_t*>(&ca[i]);
            const uint32_t* ub = reinterpret_cast<const uint32_t*>(&cb[i]);
            float part[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (j % (4 / GPB) == 0) part[0] = part[1] = part[2] = part[3] = 0.f;
                mma_bf16(part, unpack_pair(ua[j], 0), unpack_pair(ub[j], 0), unpack_pair(ua[j], 1),
                         unpack_pair(ub[j], 1), v[j].x, v[j].y);
                mma_bf16(part, unpack_pair(ua[j], 2), unpack_pair(ub[j], 2), unpack_pair(ua[j], 3),
                         unpack_pair(ub[j], 3), v[j].z, v[j].w);
                if ((j + 1) % (4 / GPB) == 0) {
                    const int g = j / (4 / GPB);
                    acc[0] = fmaf(ga[i][g], part[0], acc[0]);
                    acc[1] = fmaf(ga[i][g], part[1], acc[1]);
                    acc[2] = fmaf(gb[i][g], part[2], acc[2]);
                    acc[3] = fmaf(gb[i][g], part[3], acc[3]);
                }
            }
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) red[warp][c * 2 + (e & 1)][r + (e >> 1) * 8] = acc[e];
    cg::cluster_group cl = cg::this_cluster();
    if (p.split > 1)
        cl.sync();
    else
        __syncthreads();
    for (int e = rank * 256 + tid; e < 128; e += 256 * p.split) {
        const int row = e % 16, col = e / 16;
        const int64_t o = row0 + row;
        if (o >= p.n_out || col >= p.m) continue;
        float v = 0.f;
        for (int s = 0; s < p.split; ++s) {
            const float* from = p.split > 1 ? cl.map_shared_rank(&red[0][0][0], s) : &red[0][0][0];
#pragma unroll
            for (int k = 0; k < 8; ++k) v += from[(k * 8 + col) * 16 + row];
        }
        v *= 1024.f;
        if (p.bias) v += p.bias[o];
        if (p.residual) v += to_f(static_cast<const bf*>(p.residual)[col * p.n_out + o]);
        static_cast<bf*>(p.y)[col * p.n_out + o] = from_f<bf>(v);
    }
    if (p.split > 1) cl.sync();
}

// Launches clusters of p.split blocks.  `ready`: the devices on which this
// kernel's attributes are set.
static cudaError_t w4_launch(void (*kern)(const W4Params), const W4Params& p, dim3 grid, int smem,
                             std::atomic<uint64_t>& ready, cudaStream_t st) {
    cudaError_t e = smem_once(reinterpret_cast<const void*>(kern), smem, ready);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)p.split;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int G>
static cudaError_t w4_rows(W4Params p, int sms, cudaStream_t st) {
    static std::atomic<uint64_t> ready{0};
    const int64_t rt = (p.n_out + 15) / 16;
    // share the inputs out while the blocks do not fill two per SM and every
    // warp keeps a block of them
    p.split = 1;
    while (p.split < 8 && 16 * p.split <= p.nb && rt * p.split * 2 <= 4LL * sms) p.split *= 2;
    return w4_launch(w4_rows_kernel<G>, p, dim3((unsigned)(rt * p.split)), 0, ready, st);
}

template <typename T, int WR, int WK, int NT, int G>
static cudaError_t w4_run(W4Params p, int sms, cudaStream_t st) {
    constexpr int SP = sizeof(T) == 4 ? 3 : 1, KC = (SP == 1 ? 2 : 1) * WK;
    constexpr int xbytes = 2 * SP * KC * 4 * NT * 32 * 16, rbytes = WK * 8 * NT * 16 * WR * 4;
    constexpr int smem = xbytes > rbytes ? xbytes : rbytes;
    const int64_t rt = (p.n_out + 16 * WR - 1) / (16 * WR), ct = (p.m + 8 * NT - 1) / (8 * NT);
    const int64_t nch = (p.nb + KC - 1) / KC;
    p.split = 1;
    while (p.split < 8 && 2 * p.split <= nch && rt * ct * p.split < 3LL * sms) p.split *= 2;
    static std::atomic<uint64_t> ready{0};
    return w4_launch(w4_linear_kernel<T, WR, WK, NT, G>, p,
                     dim3((unsigned)(rt * p.split), (unsigned)ct), smem, ready, st);
}

template <typename T, int G>
static cudaError_t w4_pick(const W4Params& p, int sms, cudaStream_t st) {
    if constexpr (sizeof(T) == 2) {
        if (p.m <= 8 && p.n_in % 8 == 0) return w4_rows<G>(p, sms, st);
    }
    if (p.m <= 8) return w4_run<T, 1, 8, 1, G>(p, sms, st);
    if (p.m <= 16) return w4_run<T, 2, 4, 2, G>(p, sms, st);
    if (p.m <= 32) return w4_run<T, 4, 2, 4, G>(p, sms, st);
    return w4_run<T, 8, 1, 8, G>(p, sms, st);
}

cudaError_t launch_w4_linear(int64_t m, int64_t n_in, int64_t n_out, int group, int dtype,
                             const void* x, const void* wq, const void* scales, const float* bias,
                             const void* residual, void* y, int sms, cudaStream_t st) {
    W4Params p{};
    p.x = x;
    p.wq = static_cast<const uint4*>(wq);
    p.scales = static_cast<const __nv_bfloat16*>(scales);
    p.bias = bias;
    p.residual = residual;
    p.y = y;
    p.m = m;
    p.n_in = n_in;
    p.n_out = n_out;
    p.nb = (n_in + 127) / 128;
    p.ng = (n_in + group - 1) / group;
    const bool f32 = dtype == NAJU_F32;
    if (group == 32)
        return f32 ? w4_pick<float, 32>(p, sms, st) : w4_pick<__nv_bfloat16, 32>(p, sms, st);
    if (group == 64)
        return f32 ? w4_pick<float, 64>(p, sms, st) : w4_pick<__nv_bfloat16, 64>(p, sms, st);
    return f32 ? w4_pick<float, 128>(p, sms, st) : w4_pick<__nv_bfloat16, 128>(p, sms, st);
}

}  // namespace naju
