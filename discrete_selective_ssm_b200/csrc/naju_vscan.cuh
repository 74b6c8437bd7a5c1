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
// Work item: kVTok consecutive tokens x one tile of 32 * CP channels of one
// batch element; each of the block's 8 warps takes kVRun consecutive tokens,
// each lane CP channels (4 bytes of a row, so a warp reads and writes whole
// 128-byte lines).  Items are taken in time order from a ticket, so an item
// only ever waits for items that a running block already holds.
#pragma once
#include "naju_common.cuh"

namespace naju {

constexpr int kVWarps = 8;
constexpr int kVRun = 8;                    // tokens per warp and item
constexpr int kVTok = kVWarps * kVRun;      // tokens per item (checkpoint spacing)

// Flag values of a work item.
constexpr int kVAgg = 1;   // its (P, X) are published
constexpr int kVIncl = 2;  // the state leaving it is published

// f and 1 - f of a logit, each to full relative accuracy and without
// overflow: t = e^{-|a|} <= 1 and r = 1 / (1 + t) give max(f, 1 - f) = r and
// min = t r.
__device__ __forceinline__ void gate2(float a, float& f, float& fc) {
    const float t = expa_(-fabsf(a));
    const float r = rcpa_(1.0f + t);
    const float s = t * r;
    f = a >= 0.f ? r : s;
    fc = a >= 0.f ? s : r;
    if (a != a) f = fc = a;  // a NaN logit stays one
}
__device__ __forceinline__ float sigm(float v) { return rcpa_(1.0f + expa_(-v)); }

// A gate in one register: min(g, 1 - g) with the sign bit set when g is the
// smaller one.  gate_of gives both back, the larger as 1 - min (exact to
// 2^-25), so each keeps its relative accuracy however the gate saturates.
__device__ __forceinline__ float gate_pack(float a) {
    const float t = expa_(-fabsf(a));
    const float s = a != a ? a : t * rcpa_(1.0f + t);
    return __int_as_float(__float_as_int(s) | (__float_as_int(a) & 0x80000000));
}
__device__ __forceinline__ void gate_of(float packed, float& g, float& gc) {
    const float lo = fabsf(packed), hi = 1.0f - lo;
    const bool small = __float_as_int(packed) < 0;
    g = small ? lo : hi;
    gc = small ? hi : lo;
}

// CP values of one row in 4 bytes.
template <typename T> struct VRow;
template <> struct VRow<float> {
    static constexpr int CP = 1;
    static __device__ __forceinline__ void unpack(uint32_t r, float* o) {
        o[0] = __uint_as_float(r);
    }
};
template <> struct VRow<__nv_bfloat16> {
    static constexpr int CP = 2;
    static __device__ __forceinline__ void unpack(uint32_t r, float* o) {
        o[0] = __uint_as_float(r << 16);
        o[1] = __uint_as_float(r & 0xffff0000u);
    }
};

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

// Stores a lane's CP values of one row (outputs are read by a later kernel,
// not by this one: streaming stores).
template <typename Tout, int CP, bool VEC>
__device__ __forceinline__ void vstore(Tout* row, int64_t c0, int lane, int64_t d,
                                       const float* v) {
    if constexpr (VEC && CP == 2) {
        const int64_t c = c0 + lane * 2;
        if (c >= d) return;
        if constexpr (sizeof(Tout) == 2) {
            const __nv_bfloat162 w = __floats2bfloat162_rn(v[0], v[1]);
            __stcs(reinterpret_cast<unsigned*>(row + c), *reinterpret_cast<const unsigned*>(&w));
        } else {
            __stcs(reinterpret_cast<float2*>(row + c), make_float2(v[0], v[1]));
        }
    } else {
#pragma unroll
        for (int j = 0; j < CP; ++j) {
            const int64_t c = c0 + vchan<CP, VEC>(lane, j);
            if (c < d) row[c] = from_f<Tout>(v[j]);
        }
    }
}

// Waits, with all lanes of one warp, until the nearest item whose leaving
// state is published is reached through items whose (P, X) are: returns its
// distance (1 = the direct neighbour), or 0 when the bounded wait ran out.
// `flags` points at the neighbour's flag, `step` is -1 (forward) or +1
// (backward), `avail` the number of items on that side.
__device__ __forceinline__ int vlook(const int* flags, int step, int64_t avail, int lane,
                                     int* status, long long limit) {
    long long it = 0;
    unsigned ns = 32;
    for (;;) {
        const int fl = lane < avail ? ld_acquire(flags + (int64_t)step * lane) : 0;
        const unsigned done = __ballot_sync(0xffffffffu, fl == kVIncl);
        const unsigned any = __ballot_sync(0xffffffffu, fl != 0);
        if (done) {
            const int first = __ffs(done) - 1;
            const unsigned need = 0xffffffffu >> (31 - first);
            if ((any & need) == need) return first + 1;
        }
        if (++it > limit) {
            if (lane == 0) atomicOr(status, 1 << NAJU_ERR_TIMEOUT);
            return 0;
        }
        __nanosleep(ns);
        if (ns < 256) ns <<= 1;
    }
}

// Publishes what the warp's lanes have just written.
__device__ __forceinline__ void vpublish(int* flag, int value, int lane) {
    __threadfence();
    __syncwarp();
    if (lane == 0) st_release(flag, value);
}

}  // namespace naju
