// Device helpers shared by the suffix and decode operators.
#pragma once
#include "gdn_index.h"
#include "gdn_ops.h"

namespace gdn {

typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(2))) float f32x2;
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;
typedef __attribute__((ext_vector_type(4))) short i16x4;

// Two floats to a bf16 pair (round to nearest even), the first in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}
__device__ __forceinline__ float bf16_lo(uint32_t p) { return __uint_as_float(p << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t p) { return __uint_as_float(p & 0xffff0000u); }

// The element types of the operators: storage, and one 16-byte vector as floats and back.
struct ElemBF16 {
    typedef uint16_t T;
    static constexpr int V = 8;      // elements of a 16-byte vector
    static __device__ __forceinline__ float one(const T *p) { return __uint_as_float((uint32_t)*p << 16); }
    static __device__ __forceinline__ void unpack(u32x4 r, float *f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) { f[2 * i] = bf16_lo(r[i]); f[2 * i + 1] = bf16_hi(r[i]); }
    }
    static __device__ __forceinline__ u32x4 pack(const float *f) {
        u32x4 r;
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
        return r;
    }
};
struct ElemF32 {
    typedef float T;
    static constexpr int V = 4;
    static __device__ __forceinline__ float one(const T *p) { return *p; }
    static __device__ __forceinline__ void unpack(u32x4 r, float *f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(r[i]);
    }
    static __device__ __forceinline__ u32x4 pack(const float *f) {
        return u32x4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
    }
};
__device__ __forceinline__ u32x4 load16(const void *p) { return *reinterpret_cast<const u32x4 *>(p); }
__device__ __forceinline__ void store16(void *p, u32x4 v) { *reinterpret_cast<u32x4 *>(p) = v; }

// Workgroups go to the eight XCDs in turn.  This numbers them so that each run of `unit` consecutive
// ones, which read the same memory, is on one XCD and shares its L2, and runs take the XCDs in turn.
__device__ __forceinline__ uint32_t xcd_block(uint32_t unit) {
    const uint32_t b = blockIdx.x, whole = gridDim.x / (8 * unit) * (8 * unit);
    if (b >= whole) return b;
    const uint32_t x = b % 8, i = b / 8;
    return ((i / unit) * 8 + x) * unit + i % unit;
}

// e^a for a <= 0, below 2^-126 0.  The exponential's argument is kept in two floats.  Arguments under -150 are
// taken as that (0 as well): the second float's product would overflow at the type's lowest.  NaN stays NaN.
__device__ __forceinline__ float exp_down(float a) {
    a = a < -150.0f ? -150.0f : a;
    const float p = a * 1.4426950408889634f;
    const float r = fmaf(a, 1.4426950408889634f, -p) + a * 1.925963033500e-8f;     // log2 e in two floats
    return __builtin_amdgcn_exp2f(p) * fmaf(r, 0.6931471805599453f, 1.0f);
}
// ln(1 + e^x) = max(x, 0) + ln(1 + z), z = e^-|x| in [0, 1]; ln(1 + z) = 2 atanh(s), s = z / (2 + z) <= 1/3, by its
// series up to s^15 (the next term is below 3e-9 of the sum), which also keeps the small values of very
// negative x.
__device__ __forceinline__ float softplus(float x) {
    const float z = exp_down(-fabsf(x));
    const float d = 2.0f + z;
    float q = __builtin_amdgcn_rcpf(d);
    q = fmaf(fmaf(-d, q, 1.0f), q, q);
    const float s = z * q, t = s * s;
    float u = 1.0f / 15.0f;
    u = fmaf(u, t, 1.0f / 13.0f);
    u = fmaf(u, t, 1.0f / 11.0f);
    u = fmaf(u, t, 1.0f / 9.0f);
    u = fmaf(u, t, 1.0f / 7.0f);
    u = fmaf(u, t, 1.0f / 5.0f);
    u = fmaf(u, t, 1.0f / 3.0f);
    return fmaxf(x, 0.0f) + 2.0f * fmaf(s * t, u, s);
}

// The value, in a register of its own: what is computed from it in a loop stays in the loop instead
// of being kept in registers over it.
__device__ __forceinline__ uint32_t here(uint32_t v) {
    asm volatile("" : "+v"(v));
    return v;
}
// Orders the LDS accesses of one wave's lanes: what any lane wrote before is read after.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__device__ __forceinline__ void set_status(int32_t *status) { atomicOr(status, kStatusBitInput); }

// The last n in [0, n_seqs) with before(n), or 0, found by the whole wave: 64 candidates a step,
// so up to 64 sequences cost one load.  before holds for a first part of the sequences; where a
// bad cu breaks that, the result is still in [0, n_seqs) and the caller checks its range.  The
// same in every lane.
template <class F>
__device__ __forceinline__ int last_before(int n_seqs, F before) {
    const int lane = threadIdx.x & 63;
    int lo = 0, n = n_seqs;                       // the answer is in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 63) >> 6;
        const int64_t i = (int64_t)lane * step;
        const bool is = i < n && before(lo + (int)i);
        const int c = __popcll(__ballot(is));     // lanes 0..c-1
        const int at = (c > 0 ? c - 1 : 0) * step;
        n = n - at < step ? n - at : step;
        lo += at;
    }
    return __builtin_amdgcn_readfirstlane(lo);
}
// The sequence that owns tile index t, and the one that owns token t.
__device__ __forceinline__ int tile_sequence(const int32_t *cu, int n_seqs, int64_t t, int mul, int tile) {
    return last_before(n_seqs, [&](int n) { return first_tile(cu[n], n, mul, tile) <= t; });
}
__device__ __forceinline__ int token_sequence(const int32_t *cu, int n_seqs, int64_t t) {
    return last_before(n_seqs, [&](int n) { return cu[n] <= t; });
}
// The whole of cu, by one wave: a sequence that no tile reaches (behind a descending entry) is
// found here.
__device__ __forceinline__ void check_cu(const int32_t *cu, int n_seqs, int64_t total, int32_t *status) {
    const int lane = threadIdx.x & 63;
    bool bad = false;
    for (int n = lane; n < n_seqs; n += 64)
        bad |= !range_ok(cu[n], cu[n + 1], total) || (n == 0 && cu[0] != 0);
    if (__any(bad) && lane == 0) set_status(status);
}

// The state that row `row` of a single-token call uses, or -1 for a row that is left alone: a
// padded row (slot -1), or one whose slot is out of range or already taken by an earlier row
// (both recorded in the status word).  The same in every lane of the wave.
__device__ __forceinline__ int slot_of_row(const int32_t *slots, int row, int n_slots, int32_t *status) {
    if (!slots) return row;
    const int lane = threadIdx.x & 63;
    const int s = __builtin_amdgcn_readfirstlane(slots[row]);
    if (s == -1) return -1;
    bool bad = s < 0 || s >= n_slots;
    for (int i = lane; i < row; i += 64) bad |= slots[i] == s;
    if (__any(bad)) {
        if (lane == 0) set_status(status);
        return -1;
    }
    return s;
}

}  // namespace gdn
