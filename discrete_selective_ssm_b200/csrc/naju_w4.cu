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

#include "naju_common.cuh"
#include "naju_kernels.h"
#include "naju_w4.cuh"

namespace naju {

// -------------------------------------------------------------- quantiser
// One warp per (row, 128-input block); lane l handles inputs 4 l .. 4 l + 3
// and a group's maximum is taken over G / 4 lanes.  Runs once per weight, as
// weights are laid out: 28672 x 8192 bf16 668 us (its bytes alone: 92), from
// scalar loads and a division for every weight.
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

    const PairBits bits;
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
                    pa[q] = unpack_pair(ua[j], q, bits);
                    pb[q] = unpack_pair(ub[j], q, bits);
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
    // four rows of W at a time (an access to another block takes as long as a
    // dozen of these sums)
#pragma unroll 2
    for (int e = rank * 256 + tid; e < ROWS * COLS / 4; e += 256 * p.split) {
        const int row = e % (ROWS / 4) * 4, col = e / (ROWS / 4);
        const int64_t o = row0 + row, m = col0 + col;
        if (o >= p.n_out || m >= p.m) continue;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int s = 0; s < p.split; ++s) {
            const float* from = p.split > 1 ? cl.map_shared_rank(red, s) : red;
#pragma unroll
            for (int k = 0; k < WK; ++k)
                v = v + *reinterpret_cast<const float4*>(from + (k * COLS + col) * ROWS + row);
        }
        w4_finish<T>(p, m, o, v);
    }
    if (p.split > 1) cl.sync();  // no block leaves while another reads from it
}

// One or two rows of x (the decode of one or two sessions: the time is that of
// reading the weights), on the CUDA cores.  A warp takes kR rows of W and 1024
// inputs of each (a slice) at a time, 16 bytes a lane, so its loads are whole
// lines and a value of x serves kR weights.  A nibble becomes a float without
// a conversion: or-ed into the bits of 2^23 at nibble place i (0 to 3) it reads
// 2^23 + 16^i q, and a packed addition of two such leaves 16^i (q - 8),
// exactly; the 16^-i (and the 1 / 1024 of unpack_pair) is in the x that is
// staged.  A word's eight products are summed unscaled and enter the row's sum
// with its group's scale.
// 28 instructions for eight weights: 1 x 8192 -> 28672 bf16 45 to 46 us (2.7
// TB/s; a plain sum over the same bytes takes 27.6), 1 x 1024 -> 4096 3.0 us.
// No unit is full (issue slots 60 %, logic and shifts 55 %, HBM 32 %); the
// warps wait for weights most often.  Two rows a warp 50 us, eight 52, two
// resident blocks 49: three were chosen on this form (groups of 128, one row
// of x), whose 78 registers they allow without a spill.  Groups of 64 and 32
// and two rows of x spill 32 to 220 bytes there: 47, 54 and (groups of 128 /
// 32) 65, 94 us; two resident blocks were not timed for those.
constexpr int kR = 4;           // rows of W per warp
constexpr int kRowsSlices = 8;  // slices of x in shared memory at a time

// Nibbles i of the two halves of a word (inputs 2 i, 2 i + 1): 16^i (q - 8).
__device__ __forceinline__ float2 nibble_pair(uint32_t lo, uint32_t hi, int i, uint32_t magic) {
    const float c = -(8388608.f + (float)(8 << (4 * i)));
    return __fadd2_rn(make_float2(__uint_as_float(and_or(lo, 0xfu << (4 * i), magic)),
                                  __uint_as_float(and_or(hi, 0xfu << (4 * i), magic))),
                      make_float2(c, c));
}

template <typename T, int G, int MR>
__global__ void __launch_bounds__(256, 3) w4_rows_kernel(const W4Params p) {
    constexpr int GPB = 128 / G;
    extern __shared__ __align__(16) unsigned char smem[];
    float4* xs = reinterpret_cast<float4*>(smem);  // [row of x][slice][j][half][lane]
    __shared__ float red[8][kR][MR];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int wk = p.split, ks = warp % wk;  // wk warps share their rows' inputs
    const int64_t row0 = ((int64_t)blockIdx.x * (8 / wk) + warp / wk) * kR;
    const int64_t col0 = (int64_t)blockIdx.y * MR;
    const int nsl = (int)((p.nb + 7) / 8);
    const int slices = min(nsl, kRowsSlices);
    const T* x = static_cast<const T*>(p.x) + col0 * p.n_in;
    // rows past the end read the last one and are not stored
    const int64_t last = p.n_out - 1;
    const uint4* w = p.wq + min64(row0, last) * p.nb * 4 + lane;
    const __nv_bfloat16* sc = p.scales + min64(row0, last) * p.ng;
    const int rows = (int)min64(kR, p.n_out - row0);
    const uint32_t magic = held(0x4b000000u);
    uint4 q[kR];
    __nv_bfloat16 s[kR][GPB];
    const auto load = [&](int sl) {
        const int b = sl * 8 + (lane >> 2);
        const uint4* wp = w + (int64_t)sl * 32;
        const __nv_bfloat16* sp = sc + (int64_t)b * GPB;
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            q[r] = b < p.nb ? __ldg(wp) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int g = 0; g < GPB; ++g)
                s[r][g] = b * GPB + g < p.ng ? sp[g] : __nv_bfloat16(0.f);
            if (r + 1 < rows) {
                wp += p.nb * 4;
                sp += p.ng;
            }
        }
    };
    float2 acc[kR][MR];
#pragma unroll
    for (int r = 0; r < kR; ++r)
#pragma unroll
        for (int m = 0; m < MR; ++m) acc[r][m] = make_float2(0.f, 0.f);
    if (ks < nsl) load(ks);
    const bool xvec = p.n_in % (16 / sizeof(T)) == 0;
    for (int s0 = 0; s0 < nsl; s0 += slices) {
        const int n = min(slices, nsl - s0);
        if (s0 > 0) __syncthreads();
#pragma unroll
        for (int m = 0; m < MR; ++m) {
            const bool in = col0 + m < p.m;
            for (int unit = tid; unit < n * 128; unit += 256) {  // eight inputs each
                const int64_t k = (int64_t)s0 * 1024 + unit * 8;
                float f[8];
                if (in && xvec && k + 8 <= p.n_in) {
                    load8(x + m * p.n_in + k, f);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        f[i] = in && k + i < p.n_in ? to_f(x[m * p.n_in + k + i]) : 0.f;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] *= 1.f / (1024.f * (float)(1 << (4 * (i / 2))));
                const int b = unit / 16, j = unit % 16 / 4, c = unit % 4;
                float4* at = xs + ((m * slices + b / 8) * 4 + j) * 64 + b % 8 * 4 + c;
                at[0] = make_float4(f[0], f[1], f[2], f[3]);
                at[32] = make_float4(f[4], f[5], f[6], f[7]);
            }
        }
        __syncthreads();
        // (slices is a multiple of wk or all of them: a warp's slices go on
        // from one stage to the next in steps of wk)
        for (int sl = s0 + ks; sl < s0 + n; sl += wk) {
            uint4 cq[kR];
            float2 cs[kR][GPB];
#pragma unroll
            for (int r = 0; r < kR; ++r) {
                cq[r] = q[r];
#pragma unroll
                for (int g = 0; g < GPB; ++g) {
                    const float f = __bfloat162float(s[r][g]);
                    cs[r][g] = make_float2(f, f);
                }
            }
            if (sl + wk < nsl) load(sl + wk);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float4 xa[MR], xb[MR];
#pragma unroll
                for (int m = 0; m < MR; ++m) {
                    const float4* at = xs + ((m * slices + sl - s0) * 4 + j) * 64 + lane;
                    xa[m] = at[0];
                    xb[m] = at[32];
                }
#pragma unroll
                for (int r = 0; r < kR; ++r) {
                    const uint32_t word = reinterpret_cast<const uint32_t*>(&cq[r])[j];
                    const uint32_t hi = word >> 16;
                    const float2 d0 = nibble_pair(word, hi, 0, magic);
                    const float2 d1 = nibble_pair(word, hi, 1, magic);
                    const float2 d2 = nibble_pair(word, hi, 2, magic);
                    const float2 d3 = nibble_pair(word, hi, 3, magic);
#pragma unroll
                    for (int m = 0; m < MR; ++m) {
                        float2 t = __fmul2_rn(d0, make_float2(xa[m].x, xa[m].y));
                        t = __ffma2_rn(d1, make_float2(xa[m].z, xa[m].w), t);
                        t = __ffma2_rn(d2, make_float2(xb[m].x, xb[m].y), t);
                        t = __ffma2_rn(d3, make_float2(xb[m].z, xb[m].w), t);
                        acc[r][m] = __ffma2_rn(cs[r][j / (4 / GPB)], t, acc[r][m]);
                    }
                }
            }
        }
    }
    // the lanes' sums, then the wk warps', in fixed order
#pragma unroll
    for (int r = 0; r < kR; ++r) {
#pragma unroll
        for (int m = 0; m < MR; ++m) {
            float v = acc[r][m].x + acc[r][m].y;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            if (lane == 0) red[warp][r][m] = v;
        }
    }
    __syncthreads();
    if (ks == 0 && lane < kR * MR) {
        const int r = lane % kR, m = lane / kR;
        const int64_t o = row0 + r, col = col0 + m;
        if (o < p.n_out && col < p.m) {
            float v = 0.f;
            for (int k = 0; k < wk; ++k) v += red[warp + k][r][m];
            v *= 1024.f;
            if (p.bias) v += p.bias[o];
            if (p.residual) v += to_f(static_cast<const T*>(p.residual)[col * p.n_out + o]);
            static_cast<T*>(p.y)[col * p.n_out + o] = from_f<T>(v);
        }
    }
}

template <typename T, int G, int MR>
static cudaError_t w4_rows(W4Params p, int sms, cudaStream_t st) {
    static std::atomic<uint64_t> ready{0};
    const int64_t tiles = (p.n_out + kR - 1) / kR, nsl = (p.nb + 7) / 8;
    // warps share their rows' inputs while there are fewer than sixteen warps
    // per SM and each keeps a slice
    p.split = 1;
    while (p.split < 8 && 2 * p.split <= nsl && tiles * p.split < 16LL * sms) p.split *= 2;
    const int smem = MR * (int)min64(nsl, kRowsSlices) * 4096;
    const cudaError_t e = smem_once(reinterpret_cast<const void*>(w4_rows_kernel<T, G, MR>),
                                    MR * kRowsSlices * 4096, ready);
    if (e != cudaSuccess) return e;
    const int64_t per = 8 / p.split;
    w4_rows_kernel<T, G, MR><<<dim3((unsigned)((tiles + per - 1) / per),
                                    (unsigned)((p.m + MR - 1) / MR)), 256, smem, st>>>(p);
    return cudaGetLastError();
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
    return w4_launch(w4_linear_kernel<T, WR, WK, NT, G>,
                     dim3((unsigned)(rt * p.split), (unsigned)ct), 256, smem, p.split, ready, st,
                     p);
}

template <typename T, int G>
static cudaError_t w4_pick(const W4Params& p, int impl, int sms, cudaStream_t st) {
    // One or two rows: CUDA cores (1 x 8192 -> 28672 bf16: 45 us, against 61 for
    // the warp-level tensor-core form; 1 x 1024 -> 4096: 3.0 and 4.2 us).
    if (impl == 0 && p.m == 1) return w4_rows<T, G, 1>(p, sms, st);
    if (impl == 0 && p.m == 2) return w4_rows<T, G, 2>(p, sms, st);
    // tcgen05 from about 2^28 products on (x in whole tiles of 8 rows): its
    // blocks take 6 to 8 us to start, share out and add up, the warp-level
    // form runs at 64 T products a second (64 x 2048 -> 4096: 11 and 22 us,
    // 16 x 4096 -> 4096: 10.7 and 10.9, 16 x 2048 -> 4096: 9.3 and 5.8).
    if constexpr (sizeof(T) == 2) {
        const bool can = p.n_in % 8 == 0 && p.n_in > 128;
        const double products = (double)((p.m + 7) / 8 * 8) * (double)p.n_in * (double)p.n_out;
        if (can && (impl == 2 || (impl == 0 && p.m > 8 && products >= 268435456.0)))
            return launch_w4_tc(p, G, sms, st);
    }
    if (p.m <= 8) return w4_run<T, 1, 8, 1, G>(p, sms, st);
    if (p.m <= 16) return w4_run<T, 2, 4, 2, G>(p, sms, st);
    if (p.m <= 32) return w4_run<T, 4, 2, 4, G>(p, sms, st);
    return w4_run<T, 8, 1, 8, G>(p, sms, st);
}

cudaError_t launch_w4_linear(int64_t m, int64_t n_in, int64_t n_out, int group, int dtype,
                             const void* x, const void* wq, const void* scales, const float* bias,
                             const void* residual, void* y, int impl, int sms,
                             cudaStream_t st) {
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
        return f32 ? w4_pick<float, 32>(p, impl, sms, st) : w4_pick<__nv_bfloat16, 32>(p, impl, sms, st);
    if (group == 64)
        return f32 ? w4_pick<float, 64>(p, impl, sms, st) : w4_pick<__nv_bfloat16, 64>(p, impl, sms, st);
    return f32 ? w4_pick<float, 128>(p, impl, sms, st) : w4_pick<__nv_bfloat16, 128>(p, impl, sms, st);
}

}  // namespace naju
