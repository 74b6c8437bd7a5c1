// Device pieces shared by the vector-state scan's forward and backward
// (sm_100a, CUDA cores; memory-bound).
//
// The recurrence is the block's (Naju reproduction README, "Core equations")
// with one state value per channel instead of a d_state row:
//   x_t = f_t x_{t-1} + i_t h_t,  f = sigmoid(a), i = sigmoid(b) or 1 - f.
// A run of tokens acts on its entering state as x -> P x + X (P the product
// of its f, X its result from a zero state), so runs compose without ever
// dividing by a decay: f = 0 (a = -inf, a document's first token) and f = 1,
// i = 0 (a = +inf, b = -inf, padding) need no special case.
//
// Work item: 8 * RUN consecutive tokens x one tile of 32 * CP channels of one
// batch element (a unit).  Eight compute warps take RUN consecutive tokens
// each, every lane CP channels (4 bytes of a row, so a warp reads and writes
// whole 128-byte lines).  A cluster of CS blocks owns a unit and walks it in
// rounds of CS consecutive items, one per block: each block sends its item's
// (P, X) to the shared memory of all of them (st.async, which signals the
// receiver's mbarrier with the data), then every block folds the ones before
// its own onto the round's entering state, and all of them onto the next
// round's.  So a unit's tokens are read once, nothing goes through global
// memory between blocks, no block waits for another cluster, and the order of
// every sum is fixed.  A ninth warp, the scout, does the exchange and has the
// next item's tiles brought in by TMA as soon as the compute warps have read
// the present one's.  Measured against items taken from a ticket with a
// look-back through global flags (16 x 4096 x 2048 bf16 / 1 x 65536 x 2048):
// forward 305 / 803 us there, 252 / 352 us here (5.3 and 3.8 TB/s); backward
// 1031 / 2231 and 564 / 592 us (4.3 and 4.1 TB/s).  What bounds them is the
// latency of a round (barriers, exchange, tile wait) with the warps that fit:
// issue slots are 51 and 49 % busy, no unit more than half (the forward's
// MUFU 48 %), HBM 38 and 39 % on 4 x 2048 x 2048.
#pragma once
#include "naju_common.cuh"
#include "naju_kernels.h"
#include "naju_tc.cuh"
#include "naju_tma.h"

namespace naju {

using namespace tc;

constexpr int kVWarps = 8;                      // compute warps
constexpr int kVThreads = 32 * (kVWarps + 1);
constexpr int kVRunF = 8, kVRunB = 4;           // tokens per warp and item, forward, backward
constexpr int kVTokF = kVWarps * kVRunF;        // tokens per forward item
constexpr int kVTokB = kVWarps * kVRunB;        // per backward item, and per checkpoint

constexpr long long kTmaPolls = 1LL << 22;      // before a wait for a tile gives up

constexpr int kVMaxCluster = 16;

// ------------------------------------------------- CP channels of one lane
// Two channels go through the packed fp32 instructions (one issue slot for
// both).
template <int CP> struct Vf;
template <> struct Vf<1> {
    float x;
    __device__ __forceinline__ float& operator[](int) { return x; }
    __device__ __forceinline__ float operator[](int) const { return x; }
};
template <> struct Vf<2> {
    float2 x;
    __device__ __forceinline__ float& operator[](int j) { return j ? x.y : x.x; }
    __device__ __forceinline__ float operator[](int j) const { return j ? x.y : x.x; }
};
template <int CP> __device__ __forceinline__ Vf<CP> vset(float v) {
    Vf<CP> r;
#pragma unroll
    for (int j = 0; j < CP; ++j) r[j] = v;
    return r;
}
__device__ __forceinline__ Vf<1> operator*(Vf<1> a, Vf<1> b) { return {a.x * b.x}; }
__device__ __forceinline__ Vf<1> operator+(Vf<1> a, Vf<1> b) { return {a.x + b.x}; }
__device__ __forceinline__ Vf<1> vfma(Vf<1> a, Vf<1> b, Vf<1> c) { return {fmaf(a.x, b.x, c.x)}; }
__device__ __forceinline__ Vf<2> operator*(Vf<2> a, Vf<2> b) { return {__fmul2_rn(a.x, b.x)}; }
__device__ __forceinline__ Vf<2> operator+(Vf<2> a, Vf<2> b) { return {__fadd2_rn(a.x, b.x)}; }
__device__ __forceinline__ Vf<2> vfma(Vf<2> a, Vf<2> b, Vf<2> c) {
    return {__ffma2_rn(a.x, b.x, c.x)};
}

// CP values of one row in 4 bytes.
template <typename T> struct VRow;
template <> struct VRow<float> {
    static constexpr int CP = 1;
    static constexpr uint32_t kAbs = 0x7fffffffu;
    static __device__ __forceinline__ Vf<1> unpack(uint32_t r) { return {__uint_as_float(r)}; }
    static __device__ __forceinline__ bool neg(uint32_t r, int) { return (int)r < 0; }
};
template <> struct VRow<__nv_bfloat16> {
    static constexpr int CP = 2;
    static constexpr uint32_t kAbs = 0x7fff7fffu;
    static __device__ __forceinline__ Vf<2> unpack(uint32_t r) {
        return {make_float2(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u))};
    }
    static __device__ __forceinline__ bool neg(uint32_t r, int j) {
        return j ? (int)r < 0 : (r & 0x8000u) != 0;
    }
};

// --------------------------------------------------------------- the gates
constexpr float kLog2e = 1.4426950408889634f;

// Both sides of sigmoid(a) without overflow: with t = e^{-|a|} <= 1 and r =
// 1 / (1 + t), the larger of sigmoid(a) and 1 - sigmoid(a) is r and the smaller
// s = t r.  s is off by about |a| + 6 roundings of itself (the argument's own
// in a base-2 exponential, its two steps, sum, reciprocal, product) and zero
// past |a| of about 87, where t leaves fp32's normal range; r is exactly one
// where t is nothing against one.  For fp32 logits r is 1 - s instead: half a
// rounding where the sum and the reciprocal make up to two, which shows in a
// state that sums 150 tokens (8 x 512 x 192: 2.2e-7 from 64 bits instead of
// 4.8e-7; 16 x 4096 x 1024 without z 161 -> 167 us, with z the same).  With
// bf16 logits it would cost 4 % for what the results' rounding hides.  A NaN
// logit makes both NaN.
template <typename T>
__device__ __forceinline__ void gate_rs(uint32_t a, Vf<VRow<T>::CP>& r, Vf<VRow<T>::CP>& s) {
    constexpr int CP = VRow<T>::CP;
    Vf<CP> t = VRow<T>::unpack(a & VRow<T>::kAbs) * vset<CP>(-kLog2e);
#pragma unroll
    for (int j = 0; j < CP; ++j) t[j] = exp2a_(t[j]);
    r = t + vset<CP>(1.0f);
#pragma unroll
    for (int j = 0; j < CP; ++j) r[j] = rcpa_(r[j]);
    s = t * r;
    if (CP == 1) r[0] = 1.0f - s[0];
}
// The same for two logits with one reciprocal: 1 / (Da Db) gives both (the
// MUFU unit, at 16 lanes a clock, is the forward's busiest; both denominators
// lie in [1, 2]), for two more products in each s.  The larger
// side is 1 - s here: r Db need not be one where Da is, and a saturated gate
// has to keep its state bit for bit whatever the other gate is.
template <typename T>
__device__ __forceinline__ void gate_rs2(uint32_t a, uint32_t b, Vf<VRow<T>::CP>& ra,
                                         Vf<VRow<T>::CP>& sa, Vf<VRow<T>::CP>& rb,
                                         Vf<VRow<T>::CP>& sb) {
    constexpr int CP = VRow<T>::CP;
    const Vf<CP> one = vset<CP>(1.0f), c = vset<CP>(-kLog2e);
    Vf<CP> ta = VRow<T>::unpack(a & VRow<T>::kAbs) * c, tb = VRow<T>::unpack(b & VRow<T>::kAbs) * c;
#pragma unroll
    for (int j = 0; j < CP; ++j) ta[j] = exp2a_(ta[j]), tb[j] = exp2a_(tb[j]);
    const Vf<CP> da = ta + one, db = tb + one;
    Vf<CP> r = da * db;
#pragma unroll
    for (int j = 0; j < CP; ++j) r[j] = rcpa_(r[j]);
    sa = ta * (r * db);
    sb = tb * (r * da);
#pragma unroll
    for (int j = 0; j < CP; ++j) ra[j] = 1.0f - sa[j], rb[j] = 1.0f - sb[j];
}
// sigmoid(a) of the two sides (with r and s exchanged: 1 - sigmoid(a)).
template <typename T>
__device__ __forceinline__ Vf<VRow<T>::CP> gate_sel(uint32_t a, const Vf<VRow<T>::CP>& r,
                                                    const Vf<VRow<T>::CP>& s) {
    Vf<VRow<T>::CP> g;
#pragma unroll
    for (int j = 0; j < VRow<T>::CP; ++j) g[j] = VRow<T>::neg(a, j) ? s[j] : r[j];
    return g;
}
// sigmoid alone: 1 / (1 + e^{-v}) saturates cleanly (e^{-v} = inf gives 0).
template <int CP> __device__ __forceinline__ Vf<CP> vsigm(Vf<CP> v) {
    v = v * vset<CP>(-kLog2e);
#pragma unroll
    for (int j = 0; j < CP; ++j) v[j] = exp2a_(v[j]);
    v = v + vset<CP>(1.0f);
#pragma unroll
    for (int j = 0; j < CP; ++j) v[j] = rcpa_(v[j]);
    return v;
}

// ------------------------------------------------------------ rows, stores
// Channel of a lane's j-th value inside the tile.  VEC: adjacent channels,
// one 4-byte access (needs rows that start on 4 bytes: an even d for bf16);
// otherwise 32 apart, so that 2-byte accesses still coalesce.
template <int CP, bool VEC>
__device__ __forceinline__ int vchan(int lane, int j) {
    return VEC ? lane * CP + j : lane + 32 * j;
}

template <typename T, bool VEC>
__device__ __forceinline__ uint32_t vload(const T* row, int64_t c0, int lane, int64_t d) {
    constexpr int CP = VRow<T>::CP;
    if constexpr (VEC) {
        const int64_t c = c0 + lane * CP;
        return c < d ? __ldg(reinterpret_cast<const uint32_t*>(row + c)) : 0u;
    } else {
        const unsigned short* p = reinterpret_cast<const unsigned short*>(row);
        const int64_t c = c0 + lane;
        const uint32_t lo = c < d ? __ldg(p + c) : 0u;
        const uint32_t hi = c + 32 < d ? __ldg(p + c + 32) : 0u;
        return lo | hi << 16;
    }
}

// Stores a lane's CP values of one row at `at` (the lane's first channel).
// left: how many channels from there on exist.  Outputs are read by a later
// kernel, not by this one: streaming stores.
template <typename Tout, int CP, bool VEC>
__device__ __forceinline__ void vstore(Tout* at, int64_t left, const Vf<CP>& v) {
    if (left <= 0) return;
    if constexpr (VEC && CP == 2) {
        if constexpr (sizeof(Tout) == 2) {
            const __nv_bfloat162 w = __floats2bfloat162_rn(v[0], v[1]);
            __stcs(reinterpret_cast<unsigned*>(at), *reinterpret_cast<const unsigned*>(&w));
        } else {
            __stcs(reinterpret_cast<float2*>(at), v.x);
        }
    } else {
        at[0] = from_f<Tout>(v[0]);
        if constexpr (CP == 2) {
            if (left > 32) at[32] = from_f<Tout>(v[1]);
        }
    }
}

// ------------------------------------------------------ cluster exchange
// Shared-memory address of the same variable in block `rank` of the cluster.
__device__ __forceinline__ uint32_t map_rank(const void* p, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}
// A lane's (P, X), and its way to another block's shared memory: the store
// counts its bytes on that block's mbarrier.
template <int CP> struct __align__(8 * CP) VPair {
    Vf<CP> P, X;
};
__device__ __forceinline__ void send_pair(uint32_t dst, const VPair<1>& v, uint32_t mbar) {
    asm volatile(
        "st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];" ::"r"(
            dst),
        "r"(__float_as_uint(v.P.x)), "r"(__float_as_uint(v.X.x)), "r"(mbar)
        : "memory");
}
__device__ __forceinline__ void send_pair(uint32_t dst, const VPair<2>& v, uint32_t mbar) {
    asm volatile(
        "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, "
        "[%5];" ::"r"(dst),
        "r"(__float_as_uint(v.P.x.x)), "r"(__float_as_uint(v.P.x.y)),
        "r"(__float_as_uint(v.X.x.x)), "r"(__float_as_uint(v.X.x.y)), "r"(mbar)
        : "memory");
}
// Releases this thread's mbarrier initialisations (and those alone) to the
// cluster: after the last of them, before cluster_sync.
__device__ __forceinline__ void mbar_init_release() {
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}
// All blocks of the cluster have come this far.  Relaxed: nothing but the
// mbarriers' initialisation (released by mbar_init_release) and the right to
// leave depends on it, so a block does not wait for its stores here.
__device__ __forceinline__ void cluster_sync() {
    asm volatile(
        "barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
            : "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// Arrive on a named barrier without waiting for it.
__device__ __forceinline__ void named_arrive(int id, int count) {
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(count) : "memory");
}

// ---------------------------------------------------------- status word
// 32 bits of flags and, above them, the number of the forward call that they
// belong to: whichever comes first, the call's first block or a wait that runs
// out in any other, makes the word this call's, so neither undoes the other
// (blocks of different clusters are not ordered, and a memset before the
// launch would cost 3.5 us of the shortest forward's 2.9).
typedef unsigned long long StatusWord;
__device__ __forceinline__ StatusWord* status_word(const VscanParams& p) {
    return reinterpret_cast<StatusWord*>(p.status);
}
// The first block: flags of other calls go; what was there is looked at only
// when the block is done (status_keep), so nothing waits for it.
__device__ __forceinline__ StatusWord status_begin(const VscanParams& p) {
    return atomicExch(status_word(p), (StatusWord)p.call << 32);
}
__device__ __forceinline__ void status_keep(const VscanParams& p, StatusWord was) {
    if ((uint32_t)(was >> 32) == p.call && (uint32_t)was) atomicOr(p.status, (int)(uint32_t)was);
}
static __device__ __noinline__ void status_timeout_of(int* status, uint32_t call) {
    const StatusWord flag = 1u << NAJU_ERR_TIMEOUT;
    StatusWord* word = reinterpret_cast<StatusWord*>(status);
    StatusWord old = atomicOr(word, 0ULL);
    for (;;) {
        const bool ours = (uint32_t)(old >> 32) == call;
        const StatusWord next = ours ? old | flag : (StatusWord)call << 32 | flag;
        const StatusWord seen = atomicCAS(word, old, next);
        if (seen == old) return;
        old = seen;
    }
}
// A wait has run out.  The backward adds to its forward's flags (and has no
// room for a function call: 567 -> 577 us on 16 x 4096 x 2048 bf16).
template <bool FWD> __device__ __forceinline__ void status_timeout(const VscanParams& p) {
    if (FWD)
        status_timeout_of(p.status, p.call);
    else
        atomicOr(p.status, 1 << NAJU_ERR_TIMEOUT);
}

// The scout's side of a round's exchange: every block's (P, X) arrives here.
template <int CP> struct VExchange {
    VPair<CP> pair[2][kVMaxCluster][32];  // by round parity
    uint64_t mbar[2];

    __device__ __forceinline__ void init() {
        mbar_init(&mbar[0], 1);
        mbar_init(&mbar[1], 1);
    }
    __device__ __forceinline__ void send(int i, uint32_t rank, uint32_t cs, int lane,
                                         const VPair<CP>& v) {
        const int par = i & 1;
        if (lane == 0) tma::expect_tx(&mbar[par], cs * 32 * (uint32_t)sizeof(VPair<CP>));
        __syncwarp();
#pragma unroll 4
        for (uint32_t r = 0; r < cs; ++r)
            send_pair(map_rank(&pair[par][rank][lane], r), v, map_rank(&mbar[par], r));
    }
    // Waits (bounded) for all blocks' pairs and folds them in the order of the
    // items: E, the round's entering value, becomes the next round's; returns
    // this block's own.
    template <bool FWD>
    __device__ __forceinline__ Vf<CP> fold(int i, uint32_t rank, uint32_t cs, int lane, Vf<CP>& E,
                                           bool& alive, const VscanParams& p) {
        const int par = i & 1;
        long long it = 0;
        while (alive && !mbar_try_wait(&mbar[par], (i >> 1) & 1)) {
            if (++it > p.wait_limit) alive = false;
        }
        alive = __all_sync(0xffffffffu, alive);
        if (!alive && lane == 0) status_timeout<FWD>(p);
        Vf<CP> mine = E;
#pragma unroll 4
        for (uint32_t r = 0; r < cs; ++r) {
            const VPair<CP> g = pair[par][r][lane];
            if (r == rank) mine = E;
            E = vfma(g.P, E, g.X);
        }
        return mine;
    }
};

// Launches a kernel over p.units clusters of p.cluster blocks.
template <typename Maps>
inline cudaError_t vscan_launch(void (*kern)(VscanParams, Maps), const VscanParams& p,
                                const Maps& maps, int smem, std::atomic<uint64_t>& ready,
                                cudaStream_t st) {
    const cudaError_t e = smem_once(reinterpret_cast<const void*>(kern), smem, ready);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(p.units * p.cluster));
    cfg.blockDim = dim3(kVThreads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)p.cluster;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p, maps);
}

}  // namespace naju
