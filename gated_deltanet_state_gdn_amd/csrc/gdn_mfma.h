// Matrix-core fragments of the suffix operators, for bf16 and fp32 elements alike.
//
// A fragment is eight elements a lane along the contraction, 32 deep over the four lane groups of
// a 16-row tile.  bf16: one 16x16x32 product.  fp32: eight 16x16x4 products, the j-th taking slot
// j of every lane.  Which contraction index slot j of lane group g stands for is free as long as
// both operands agree; two maps are used:
//     nat: 8 g + j                     (one contiguous 16-byte read of a bf16 row)
//     acc: 4 g + j % 4 + 16 (j / 4)    (the rows that two 16 x 16 accumulator tiles hold in lane
//                                       group g, so accumulators become operands where they are)
// The accumulator of a 16 x 16 product holds row 4 g + i, column l % 16 in element i.
#pragma once
#include "gdn_ops_device.h"

namespace gdn {

typedef __attribute__((address_space(3))) i16x4 *lds_i16x4;

__device__ __forceinline__ bf16x8 frag_of(u32x2 a, u32x2 b) {
    return __builtin_bit_cast(bf16x8, u32x4{a.x, a.y, b.x, b.y});
}
__device__ __forceinline__ u32x2 read_tr(const uint16_t *p) {
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4)p));
}

struct MfmaBF16 : ElemBF16 {
    typedef bf16x8 Frag;
    static constexpr int PAD = 8;        // elements behind each LDS row
    static __device__ __forceinline__ f32x4 mma(f32x4 c, const Frag &a, const Frag &b) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    // row l % 16 of M (row-major), contraction along the row
    static __device__ __forceinline__ Frag row_nat(const T *M, int stride, int lane) {
        return __builtin_bit_cast(Frag, load16(M + (lane & 15) * stride + 8 * (lane >> 4)));
    }
    static __device__ __forceinline__ Frag row_acc(const T *M, int stride, int lane) {
        const T *p = M + (lane & 15) * stride + 4 * (lane >> 4);
        return frag_of(*reinterpret_cast<const u32x2 *>(p), *reinterpret_cast<const u32x2 *>(p + 16));
    }
    // column l % 16 of M (in LDS), contraction down the rows in the acc map.  The transposing read
    // gives lane n of every 16 lanes column n of the 4 rows x 16 columns whose 8-byte pieces the
    // lanes point at (lane 4 y + x: row y, columns 4 x .. 4 x + 3).
    static __device__ __forceinline__ Frag col_acc(const T *M, int stride, int lane) {
        const T *p = M + (4 * (lane >> 4) + ((lane & 15) >> 2)) * stride + 4 * (lane & 3);
        return frag_of(read_tr(p), read_tr(p + 16 * stride));
    }
    static __device__ __forceinline__ void to_floats(const Frag &f, float *x) { unpack(__builtin_bit_cast(u32x4, f), x); }
    static __device__ __forceinline__ Frag from_floats(const float *x) { return __builtin_bit_cast(Frag, pack(x)); }
    // four consecutive elements
    static __device__ __forceinline__ void store4(T *p, const float *x) {
        *reinterpret_cast<u32x2 *>(p) = u32x2{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])};
    }
    static __device__ __forceinline__ void load4(const T *p, float *x) {
        const u32x2 r = *reinterpret_cast<const u32x2 *>(p);
        x[0] = bf16_lo(r.x); x[1] = bf16_hi(r.x); x[2] = bf16_lo(r.y); x[3] = bf16_hi(r.y);
    }
};

struct MfmaF32 : ElemF32 {
    struct Frag { float x[8]; };
    static constexpr int PAD = 4;
    static __device__ __forceinline__ f32x4 mma(f32x4 c, const Frag &a, const Frag &b) {
#pragma unroll
        for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.x[j], b.x[j], c, 0, 0, 0);
        return c;
    }
    static __device__ __forceinline__ Frag row_nat(const T *M, int stride, int lane) {
        Frag f;
        const T *p = M + (lane & 15) * stride + 8 * (lane >> 4);
        unpack(load16(p), f.x);
        unpack(load16(p + 4), f.x + 4);
        return f;
    }
    static __device__ __forceinline__ Frag row_acc(const T *M, int stride, int lane) {
        Frag f;
        const T *p = M + (lane & 15) * stride + 4 * (lane >> 4);
        unpack(load16(p), f.x);
        unpack(load16(p + 16), f.x + 4);
        return f;
    }
    static __device__ __forceinline__ Frag col_acc(const T *M, int stride, int lane) {
        Frag f;
        const T *p = M + 4 * (lane >> 4) * stride + (lane & 15);
#pragma unroll
        for (int j = 0; j < 8; ++j) f.x[j] = p[((j & 3) + 16 * (j >> 2)) * stride];
        return f;
    }
    static __device__ __forceinline__ void to_floats(const Frag &f, float *x) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = f.x[j];
    }
    static __device__ __forceinline__ Frag from_floats(const float *x) {
        Frag f;
#pragma unroll
        for (int j = 0; j < 8; ++j) f.x[j] = x[j];
        return f;
    }
    static __device__ __forceinline__ void store4(T *p, const float *x) { store16(p, pack(x)); }
    static __device__ __forceinline__ void load4(const T *p, float *x) { unpack(load16(p), x); }
};

}  // namespace gdn
