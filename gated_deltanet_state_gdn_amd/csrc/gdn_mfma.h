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
// The transposing read of LDS: gives lane n of every 16 lanes column n of the 4 rows x 16 columns whose 8-byte
// pieces the lanes point at (lane 4 y + x: row y, columns 4 x .. 4 x + 3).
__device__ __forceinline__ u32x2 read_tr(const uint16_t *p) {
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4)p));
}

struct MfmaBF16 : ElemBF16 {
    typedef bf16x8 Frag;
    static __device__ __forceinline__ f32x4 mma(f32x4 c, const Frag &a, const Frag &b) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    // row l % 16 of M (row-major), contraction along the row
    static __device__ __forceinline__ Frag row_nat(const T *M, int stride, int lane) {
        return __builtin_bit_cast(Frag, load16(M + (lane & 15) * stride + 8 * (lane >> 4)));
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
    static constexpr int PAD = 4;        // elements behind each LDS row
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

// A tile of ROWS x COLS elements in LDS for products whose contraction runs along the rows or down
// them.
//
// bf16: the nat map, rows without padding; 16-byte chunk c of row r sits at chunk c ^ swz(r).  The
// swizzles are ones that measured free of bank conflicts for 16-byte reads of 16 rows at one chunk
// and that leave the 8-byte transposing reads at their full rate (256-byte rows: the three low row
// bits, reversed, on chunk bits 3..1).
// An accumulator tile kt whose rows are the contraction index of a later product along COLS holds
// the entries state_row(kt, g, i) in element i of lane group g, so that it is that product's operand
// where it is; spread(kb, kt) reads this tile's columns in that order.
template <class M, int ROWS, int COLS>
struct Tile2;

template <int ROWS, int COLS>
struct Tile2<MfmaBF16, ROWS, COLS> {
    typedef MfmaBF16::Frag Frag;
    static constexpr int RB = COLS * 2;
    static constexpr int LANE = 8, HALF = 4;        // contraction slots j of lane group g: 8 g + j
    static_assert(RB == 256 || RB == 128, "rows of 128 or 64 elements");
    alignas(16) char d[ROWS * RB];

    static __device__ __forceinline__ int swz(int r) {
        return RB == 256 ? (((r & 1) << 3) | ((r & 2) << 1) | ((r & 4) >> 1)) : ((((r >> 1) & 1) << 2) | ((r >> 2) & 3));
    }
    static constexpr int NEXT4 = RB == 256 ? 32 : 16;               // what r -> r + 4 (r & 4 = 0) does to a chunk's place
    static __device__ __forceinline__ int state_row(int kt, int g, int i) { return 32 * (kt >> 1) + 8 * g + 4 * (kt & 1) + i; }
    __device__ __forceinline__ char *four(int r, int c) {           // columns c .. c + 3, c a multiple of 4
        return d + r * RB + 16 * ((c >> 3) ^ swz(r)) + 8 * ((c >> 2) & 1);
    }
    __device__ __forceinline__ const char *four(int r, int c) const { return const_cast<Tile2 *>(this)->four(r, c); }
    __device__ __forceinline__ void put16(int r, int c, u32x4 v) { store16(d + r * RB + 16 * ((c >> 3) ^ swz(r)), v); }
    __device__ __forceinline__ void put4(int r, int c, const float *x) { MfmaBF16::store4(reinterpret_cast<uint16_t *>(four(r, c)), x); }
    __device__ __forceinline__ void get4(int r, int c, float *x) const { MfmaBF16::load4(reinterpret_cast<const uint16_t *>(four(r, c)), x); }
    // row r0 + l % 16 (r0 a multiple of 16), columns from 32 kb
    __device__ __forceinline__ Frag row(int r0, int kb, int lane) const {
        const int r = lane & 15;
        return __builtin_bit_cast(Frag, load16(d + r0 * RB + ((r * RB + 16 * ((lane >> 4) ^ swz(r))) ^ (64 * kb))));
    }
    // rows from 32 kb; column 16 ct + l % 16
    __device__ __forceinline__ Frag col(int kb, int ct, int lane) const {
        const int x = lane & 3, r = 8 * (lane >> 4) + ((lane & 15) >> 2);
        return pair(kb, (r * RB + 16 * ((x >> 1) ^ swz(r)) + 8 * (x & 1)) ^ (32 * ct));
    }
    // rows from 32 kb; column state_row(kt, l / 4 % 4, l % 4)
    __device__ __forceinline__ Frag spread(int kb, int kt, int lane) const {
        const int x = lane & 3, r = 8 * (lane >> 4) + ((lane & 15) >> 2);
        return pair(kb, ((r * RB + 16 * (x ^ swz(r))) ^ (64 * (kt >> 1))) + 8 * (kt & 1));
    }
    __device__ __forceinline__ Frag pair(int kb, uint32_t at) const {
        return frag_of(read_tr(reinterpret_cast<const uint16_t *>(d + 32 * kb * RB + at)),
                       read_tr(reinterpret_cast<const uint16_t *>(d + (32 * kb + 4) * RB + (at ^ NEXT4))));
    }
};

template <int ROWS, int COLS>
struct Tile2<MfmaF32, ROWS, COLS> {
    typedef MfmaF32::Frag Frag;
    static constexpr int ST = COLS + MfmaF32::PAD;
    static constexpr int LANE = 4, HALF = 16;       // the acc map
    alignas(16) float d[ROWS * ST];
    static __device__ __forceinline__ int state_row(int kt, int g, int i) { return 16 * kt + 4 * g + i; }
    __device__ __forceinline__ void put16(int r, int c, u32x4 v) { store16(d + r * ST + c, v); }
    __device__ __forceinline__ void put4(int r, int c, const float *x) { MfmaF32::store4(d + r * ST + c, x); }
    __device__ __forceinline__ void get4(int r, int c, float *x) const { MfmaF32::load4(d + r * ST + c, x); }
    __device__ __forceinline__ Frag row(int r0, int kb, int lane) const { return MfmaF32::row_acc(d + r0 * ST + 32 * kb, ST, lane); }
    __device__ __forceinline__ Frag col(int kb, int ct, int lane) const { return MfmaF32::col_acc(d + 32 * kb * ST + 16 * ct, ST, lane); }
    __device__ __forceinline__ Frag spread(int kb, int kt, int lane) const { return col(kb, kt, lane); }
};

}  // namespace gdn
