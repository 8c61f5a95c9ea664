// Selective state space scan over packed sequences, in chunks of C = 64 tokens.
//
//     S_t = a_t S_{t-1} + dt_t B_t x_t^T,   y_t = S_t^T C_t + D x_t,   a_t = exp(dt_t A)
//
// per (sequence, head), B and C shared by the heads of a group.  With G the running sum of log a
// inside a chunk and S the state in front of it,
//     M_ij = (C_i . B_j) exp(G_i - G_j) dt_j   (j <= i),
//     Y    = M X + diag(exp G) C S + D X,
//     S   <- exp(G_last) S + B^T diag(exp(G_last - G_j) dt_j) X,
// which is the recurrence exactly in exact arithmetic.  All exponents are sums of the log a of a
// stretch of tokens, formed as differences of a 64-bit running sum kept as two floats: strong
// decays in front of weak ones cost the weak ones nothing.
//
// Work decomposition: a workgroup takes 64 or 128 columns (whole heads of one group, or half of one)
// over one segment of one sequence, chunk by chunk.  The columns of S (d_v of every head) do not mix, so every wave owns a
// 16-column tile of S whole, in its accumulators; M is the only product the waves share, and
// goes through LDS.  Y is formed transposed (Y^T = S^T C^T + X^T M^T): accumulators of S become
// operands where they are, and a lane ends with four consecutive entries of one token's y.
//
// The decay is one number per head and token, so segments join elementwise: with more than one
// segment, a first launch forms every segment's state from zero and its decay, a second chains
// them (S_start(s+1) = decay_s S_start(s) + local_s), and a third forms the outputs.
//
// Precision: S, G and every sum are fp32 or wider.  bf16 inputs enter the matrix products as they
// are; M, and S in C S, are rounded to bf16 once (half a bf16 step of each term, as the output itself is
// of the sum).  The state is an fp32 output: there diag(w) X is split into three bf16 terms, 24 bits, and
// multiplied with B exactly as B is; the launch that only forms outputs takes two terms, 16 bits.  fp32
// inputs use fp32 products throughout.
//
// Measured: one bf16 sequence of 32768 tokens, 32 heads of 128 x 64: 194 to 201 us by the box (305 MB, which the
// copy would take 61 us for); in a trace states 71 to 83, chain 13, outputs 126 to 150.  Half of the waves'
// cycles are waits, at a chunk's three barriers and for one product's operands from another; no unit is
// full (outputs: LDS 42 % of its cycles, a quarter of them conflicts, vector issue 37 %, matrix cores 21 %;
// states: 32, 34 and 29 %).  fp32, 24 ragged sequences, 7001 tokens, 4 heads of 64 x 64: 44 us.
#include "gdn_mfma.h"

namespace gdn {
namespace {

constexpr int CH = kScanChunk;   // tokens of a chunk
constexpr int NT = 256;
constexpr int MODE_FULL = 0, MODE_STATE = 1, MODE_OUT = 2;

// Columns of a workgroup, for a launch over so many in all.  128 (two heads of 64 of a group, or one
// of 128) read B and C and form C B^T half as often; 64 spread over twice as many CUs, which counts
// where there are few workgroups, and for fp32, whose products keep a CU busy alone.
int scan_columns(int32_t h_qk, int32_t h_v, int32_t d_v, int bf16, int64_t columns)
{
    if (!bf16 || columns / 128 < 256) return 64;
    return d_v == 128 || (h_v / h_qk) % 2 == 0 ? 128 : 64;
}

// The window of sequence n: its tokens [beg, end), false if cu or r is bad.
__device__ __forceinline__ bool window(const ScanArgs &a, int n, int64_t &beg, int64_t &end) {
    const int32_t b = a.cu[n], e = a.cu[n + 1];
    if (!range_ok(b, e, a.total)) return false;
    int32_t len = e - b;
    if (a.r) {
        const int32_t r = a.r[n];
        if (r < 0 || r > len) return false;
        len = r;
    }
    beg = e - len;
    end = e;
    return true;
}
// Output row of sequence n's first token: its own token, or with replay lengths the sum of those
// before it (a wave's sum; -1 if it does not fit).
__device__ __forceinline__ int64_t out_row(const ScanArgs &a, int n, int64_t beg, int64_t len) {
    int64_t row = beg;
    if (a.r) {
        int64_t s = 0;
        for (int i = threadIdx.x & 63; i < n; i += 64) {
            int64_t b, e;
            if (window(a, i, b, e)) s += e - b;
        }
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) s += __shfl_xor(s, off);
        row = s;
    }
    return row + len <= a.total_out ? row : -1;
}
__device__ __forceinline__ int chunks_per_segment(int64_t len, int segs) {
    const int64_t c = (len + CH - 1) / CH;
    return (int)((c + segs - 1) / segs);
}

// Inclusive sum over the lanes of a wave, by lane-shift operands (no LDS): within rows of 16 lanes,
// then the rows' last lanes into the rows behind.
template <int CTRL, int ROWS>
__device__ __forceinline__ double shifted(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROWS, 0xf, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, ROWS, 0xf, false);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);    // 0.0 where there is no such lane
}
__device__ __forceinline__ double wave_scan(double v) {
    v += shifted<0x111, 0xf>(v);         // row_shr 1, 2, 4, 8
    v += shifted<0x112, 0xf>(v);
    v += shifted<0x114, 0xf>(v);
    v += shifted<0x118, 0xf>(v);
    v += shifted<0x142, 0xa>(v);         // lane 15 of rows 0, 2 into rows 1, 3
    v += shifted<0x143, 0xc>(v);         // lane 31 into rows 2, 3
    return v;
}
__device__ __forceinline__ double lane_value(double v, int lane) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, lane), hi = __builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

__device__ __forceinline__ float lane_value(float v, int lane) {
    return __uint_as_float(__builtin_amdgcn_readlane((int)__float_as_uint(v), lane));
}

// What a chunk's gates are to the products, per head and token.
struct Gates {
    float hi[CH], lo[CH];                // G log2 e in two floats
    float dt[CH], w[CH];                 // dt_j and exp(G_last - G_j) dt_j
    float e[CH];                         // exp(G_i)
    // Tiles of M left of the diagonal one in tile row t: exp(G_i - G_j) dt_j = row[i] col[t - 1][j],
    // split at token 16 t - 1 (both exponents <= 0, so neither factor overflows)
    float row[CH], col[3][CH];
    float last;                          // exp(G_last)
};
// COLS columns of a workgroup: HB = COLS / DV whole heads, or 64 of a head's 128.
template <class M, int DK, int COLS, int HB>
struct Lds {
    Tile2<M, CH, DK> B, C;
    Tile2<M, CH, COLS> X;
    Tile2<M, CH, CH> Mx[HB];             // M, row i
    alignas(16) Gates gate[2][HB];       // this chunk's and the next one's
};
// 16-column tiles of S that a wave owns.  Two would halve the reads of C and B^T (which every wave
// reads whole) and leave two waves a SIMD instead of four: one sequence of 32768 tokens, 32 heads took
// 82 + 143 us with two and 75 + 133 us with one (states, outputs; the latter's state then in one term).
constexpr int WT = 1;

template <class M, int DK, int DV, int COLS, int MODE>
__global__ void __launch_bounds__(COLS * 4 / WT, M::V == 8 && COLS == 128 ? 4 : 2) scan_kernel(ScanArgs a)
{
    constexpr int HB = COLS >= DV ? COLS / DV : 1, PARTS = COLS >= DV ? 1 : DV / COLS;
    typedef typename M::T T;
    typedef typename M::Frag Frag;
    typedef Lds<M, DK, COLS, HB> L;
    typedef Tile2<M, CH, DK> Bt;
    constexpr int V = M::V;
    constexpr int WAVES = COLS / 16 / WT, NTH = 64 * WAVES;
    constexpr bool Y = MODE != MODE_STATE;
    __shared__ L s;
    const int lane = threadIdx.x & 63, g = lane >> 4, col = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

    if (blockIdx.x == 0 && threadIdx.x < 64) check_cu(a.cu, a.n_seqs, a.total, a.status);
    // the heads of a segment next to each other: those of a group read the same B and C
    const int hblocks = a.h_v / HB * PARTS;
    const uint32_t block = xcd_block(a.h_v / a.h_qk / HB * PARTS);
    const int hb = block % hblocks;
    const int n = block / hblocks / a.segs;
    // turned by the sequence's number: a multiple of 8 blocks for each would give all the first segments,
    // which no sequence is too short for, to the same XCD
    const int seg = (int)((block / hblocks + (uint32_t)n) % (uint32_t)a.segs);
    const int h0 = hb / PARTS * HB, part = hb % PARTS * COLS;   // first head; first column of its part
    int64_t beg, end;
    if (!window(a, n, beg, end)) {
        if (threadIdx.x == 0) set_status(a.status);
        return;
    }
    const int64_t len = end - beg;
    int64_t row0 = 0;
    if (Y) {
        row0 = out_row(a, n, beg, len);
        if (row0 < 0) {
            if (threadIdx.x == 0) set_status(a.status);
            return;
        }
    }
    const int cps = chunks_per_segment(len, a.segs);
    const int64_t sbeg = beg + (int64_t)seg * cps * CH;
    const int64_t send = sbeg + (int64_t)cps * CH < end ? sbeg + (int64_t)cps * CH : end;
    if (a.segs > 1 && sbeg >= end) return;           // an empty segment: nothing reads its state
    const int nch = sbeg < send ? (int)((send - sbeg + CH - 1) / CH) : 0;

    const int c0 = wave * 16 * WT;                   // this wave's columns within the block's
    const int hl = c0 / DV, h = h0 + hl;             // their head
    const int p0 = part + c0 - hl * DV;              // and within the head
    const int64_t state = (((int64_t)n * a.segs + seg) * a.h_v + h) * DK * DV;
    const float *Sin = nullptr;
    if (MODE == MODE_OUT) Sin = a.seg_state + state;
    else if (a.segs == 1 && a.S0) Sin = a.S0 + state;

    f32x4 S[DK / 16][WT];
    if (Sin) {
#pragma unroll
        for (int kt = 0; kt < DK / 16; ++kt)
#pragma unroll
            for (int pt = 0; pt < WT; ++pt)
#pragma unroll
                for (int i = 0; i < 4; ++i) S[kt][pt][i] = Sin[Bt::state_row(kt, g, i) * DV + p0 + 16 * pt + col];
    } else {
#pragma unroll
        for (int kt = 0; kt < DK / 16; ++kt)
#pragma unroll
            for (int pt = 0; pt < WT; ++pt) S[kt][pt] = f32x4{0, 0, 0, 0};
    }

    if (Y) {   // the tiles right of the diagonal that share a 32-deep step with it stay zero
        for (uint32_t i = threadIdx.x; i < sizeof(s.Mx) / 16; i += NTH) reinterpret_cast<u32x4 *>(s.Mx)[i] = u32x4{0, 0, 0, 0};
    }

    const int gq = h0 / (a.h_v / a.h_qk);            // the group's B and C
    const T *Bp = static_cast<const T *>(a.B) + (int64_t)gq * DK;
    const T *Cp = static_cast<const T *>(a.C) + (int64_t)gq * DK;
    const T *Xp = static_cast<const T *>(a.x) + (int64_t)h0 * DV + part;
    constexpr int NBK = CH * DK / V / NTH, NX = CH * COLS / V / NTH;
    static_assert(NBK >= 1 && NX >= 1, "every thread has vectors of a chunk to bring in");
    u32x4 rb[NBK], rc[NBK], rx[NX];
    // A thread's vectors of a chunk are NTH V elements apart: whole rows, one column.  Their places are
    // 32-bit offsets (the host has checked that a chunk spans less than 2 GiB) from scalar addresses.
    constexpr int RBK = NTH * V / DK, RX = NTH * V / COLS;         // rows from one vector to the next
    static_assert(RBK * DK == NTH * V && RX * COLS == NTH * V, "whole rows");
    const uint32_t bk_row = threadIdx.x * V / DK, bk_col = threadIdx.x * V % DK;
    const uint32_t x_row = threadIdx.x * V / COLS, x_col = threadIdx.x * V % COLS;
    const uint32_t b_at = bk_row * (uint32_t)a.bs + bk_col, c_at = bk_row * (uint32_t)a.cs + bk_col;
    const uint32_t x_at = x_row * (uint32_t)a.xs + x_col;
    auto fetch = [&](int64_t t0) {
        const T *b = Bp + t0 * a.bs, *c = Cp + t0 * a.cs, *x = Xp + t0 * a.xs;
        if (send - t0 >= CH) {
#pragma unroll
            for (int i = 0; i < NBK; ++i) {
                rb[i] = load16(b + i * RBK * a.bs + b_at);
                if (Y) rc[i] = load16(c + i * RBK * a.cs + c_at);
            }
#pragma unroll
            for (int i = 0; i < NX; ++i) rx[i] = load16(x + i * RX * a.xs + x_at);
        } else {
            // rows behind the segment's end repeat its last one: their dt is 0, so they add nothing
            const uint32_t lastrow = (uint32_t)(send - t0 - 1);
#pragma unroll
            for (int i = 0; i < NBK; ++i) {
                const uint32_t row = min(bk_row + i * RBK, lastrow);
                rb[i] = load16(b + row * (uint32_t)a.bs + bk_col);
                if (Y) rc[i] = load16(c + row * (uint32_t)a.cs + bk_col);
            }
#pragma unroll
            for (int i = 0; i < NX; ++i) rx[i] = load16(x + min(x_row + i * RX, lastrow) * (uint32_t)a.xs + x_col);
        }
    };
    // The gates of one head, by one of the last waves (the first ones have more of M): a chunk ahead,
    // from a dt that was loaded a chunk before that.
    const int gw = WAVES - 1 - wave;
    const bool gates = gw < HB;
    const int gh = gates ? h0 + gw : h0;
    const float gA = a.A[gh], gbias = a.dt_bias ? a.dt_bias[gh] : 0.0f;
    const T *dtp = static_cast<const T *>(a.dt) + gh;
    auto fetch_dt = [&](int64_t t0) {
        const int64_t t = t0 + lane < send ? t0 + lane : send - 1;
        return M::one(dtp + t * a.dts);
    };
    const double gL = (double)gA * 1.4426950408889634;
    double total = 0.0;                              // log2 of the decay since the segment's start
    auto form_gates = [&](int64_t t0, float raw, Gates &o) {
        const bool in = t0 + lane < send;
        float dt = raw + gbias;
        if (a.softplus) dt = softplus(dt);
        dt = in ? dt : 0.0f;
        // log2 a; below -1000 it is 0 in fp32 whatever follows, and stays finite here
        const double G = wave_scan(in ? fmax((double)dt * gL, -1000.0) : 0.0), all = lane_value(G, 63);
        const float hi = (float)G, lo = (float)(G - (double)hi);
        // 2^(G at lane l - G), and the reverse
        auto from = [&](int l) { return (lane_value(hi, l) - hi) + (lane_value(lo, l) - lo); };
        o.hi[lane] = hi;
        o.lo[lane] = lo;
        o.dt[lane] = dt;
        o.w[lane] = __builtin_amdgcn_exp2f(from(63)) * dt;
        if (lane == 0) o.last = __builtin_amdgcn_exp2f((float)all);
        if (Y) {
            o.e[lane] = __builtin_amdgcn_exp2f(hi);
            float at = 0.0f;                         // G - G at the token in front of this lane's tile
#pragma unroll
            for (int t = 1; t < 4; ++t) {
                const float b = from(16 * t - 1);
                if (lane >= 16 * t) at = b;
                o.col[t - 1][lane] = __builtin_amdgcn_exp2f(b) * dt;   // read for lane < 16 t
            }
            o.row[lane] = __builtin_amdgcn_exp2f(-at);
        }
        total += all;
    };
    float rdt = 0.0f;
    if (nch > 0) {
        fetch(sbeg);
        if (gates) {
            form_gates(sbeg, fetch_dt(sbeg), s.gate[0][gw]);
            if (nch > 1) rdt = fetch_dt(sbeg + CH);
        }
    }

    for (int ch = 0; ch < nch; ++ch) {
        const int64_t t0 = sbeg + (int64_t)ch * CH;
        __syncthreads();                             // the last chunk's readers are done
#pragma unroll
        for (int i = 0; i < NBK; ++i) {
            s.B.put16(bk_row + i * RBK, bk_col, rb[i]);
            if (Y) s.C.put16(bk_row + i * RBK, bk_col, rc[i]);
        }
#pragma unroll
        for (int i = 0; i < NX; ++i) s.X.put16(x_row + i * RX, x_col, rx[i]);
        __syncthreads();
        if (ch + 1 < nch) fetch(t0 + CH);
        const Gates &gt = s.gate[ch & 1][hl];
        const int lane = (int)here(threadIdx.x & 63), g = lane >> 4, col = lane & 15;
        const int left = send - t0 < CH ? (int)(send - t0) : CH;
        // fp32, which its products bound: half chunks behind the segment's end are left out (one token each of
        // 7 sequences, 4 heads of 64 x 64: 9.4 -> 7.0 us); bf16 waits for other things
        auto beyond = [&](int row) { return V == 4 && row >= left; };

        if (Y) {
            // M: the ten 16 x 16 tiles on and below the diagonal, shared out among the waves;
            // C B^T is the same for the block's heads.  Rows j in the accumulator, column i.
            for (int t = wave; t < 10; t += WAVES) {
                const int it = t < 1 ? 0 : t < 3 ? 1 : t < 6 ? 2 : 3;
                const int jt = t - it * (it + 1) / 2;
                if (beyond(16 * it)) break;
                f32x4 cb = {0, 0, 0, 0};
#pragma unroll
                for (int kb = 0; kb < DK / 32; ++kb)
                    cb = M::mma(cb, s.B.row(16 * jt, kb, lane), s.C.row(16 * it, kb, lane));
                const int i = 16 * it + col, j0 = 16 * jt + 4 * g;
#pragma unroll
                for (int q = 0; q < HB; ++q) {
                    const Gates &z = s.gate[ch & 1][q];
                    float m[4];
                    if (jt < it) {
                        const float f = z.row[i];
                        const f32x4 cj = *reinterpret_cast<const f32x4 *>(&z.col[it - 1][j0]);
#pragma unroll
                        for (int k = 0; k < 4; ++k) m[k] = cb[k] * (f * cj[k]);
                    } else {
                        const float hi = z.hi[i], lo = z.lo[i];
                        const f32x4 hj = *reinterpret_cast<const f32x4 *>(&z.hi[j0]), lj = *reinterpret_cast<const f32x4 *>(&z.lo[j0]);
                        const f32x4 dj = *reinterpret_cast<const f32x4 *>(&z.dt[j0]);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float d = (hi - hj[k]) + (lo - lj[k]);
                            m[k] = j0 + k <= i ? cb[k] * (__builtin_amdgcn_exp2f(d) * dj[k]) : 0.0f;
                        }
                    }
                    s.Mx[q].put4(i, j0, m);
                }
            }
        }
        if (gates && ch + 1 < nch) {
            form_gates(t0 + CH, rdt, s.gate[(ch + 1) & 1][gw]);
            if (ch + 2 < nch) rdt = fetch_dt(t0 + 2 * CH);
        }
        f32x4 yt[4][WT];
        if (Y) {
            // exp(G_i) (S^T C^T)
#pragma unroll
            for (int it = 0; it < 4; ++it)
#pragma unroll
                for (int pt = 0; pt < WT; ++pt) yt[it][pt] = f32x4{0, 0, 0, 0};
            constexpr int PASS = V == 4 ? 2 : 4;     // tiles of rows at a time
#pragma unroll
            for (int i0 = 0; i0 < 4; i0 += PASS) {
                if (beyond(16 * i0)) break;
#pragma unroll
                for (int kb = 0; kb < DK / 32; ++kb) {
                    Frag St[WT];
#pragma unroll
                    for (int pt = 0; pt < WT; ++pt) {
                        float f[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) f[i] = S[2 * kb + (i >> 2)][pt][i & 3];
                        St[pt] = M::from_floats(f);
                    }
#pragma unroll
                    for (int it = i0; it < i0 + PASS; ++it) {
                        const Frag cf = s.C.row(16 * it, kb, lane);
#pragma unroll
                        for (int pt = 0; pt < WT; ++pt) yt[it][pt] = M::mma(yt[it][pt], St[pt], cf);
                    }
                }
            }
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                const float e = gt.e[16 * it + col];
#pragma unroll
                for (int pt = 0; pt < WT; ++pt) yt[it][pt] *= e;
            }
        }
        if (Y) __syncthreads();                      // M is whole
        // X^T: rows p for Y^T, and (the same registers) columns p for the state
        Frag xf[2][WT];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int pt = 0; pt < WT; ++pt) xf[kb][pt] = s.X.col(kb, c0 / 16 + pt, lane);
        if (Y) {
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                if (it % 2 == 0 && beyond(16 * it)) break;
#pragma unroll
                for (int kb = 0; kb <= it / 2; ++kb) {
                    const Frag mf = s.Mx[hl].row(16 * it, kb, lane);
#pragma unroll
                    for (int pt = 0; pt < WT; ++pt) yt[it][pt] = M::mma(yt[it][pt], xf[kb][pt], mf);
                }
            }
            const float D = a.D ? a.D[h] : 0.0f;
            T *yp = static_cast<T *>(a.y) + (row0 + (t0 - beg)) * a.ys + (int64_t)h * DV + p0;
            const uint32_t y_at = col * (uint32_t)a.ys + 4 * g;
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                const int i = 16 * it + col;
                T *yi = yp + 16 * it * a.ys + y_at;
#pragma unroll
                for (int pt = 0; pt < WT; ++pt) {
                    float x[4], o[4];
                    s.X.get4(i, c0 + 16 * pt + 4 * g, x);
#pragma unroll
                    for (int k = 0; k < 4; ++k) o[k] = fmaf(D, x[k], yt[it][pt][k]);
                    if (i < left) M::store4(yi + 16 * pt, o);
                }
            }
        }
        // the state; the outputs alone (MODE_OUT) need it to less than the rounding of S in C S: two terms,
        // 16 bits (one would be a third rounding of y, and one that is there only in segments; the second
        // costs the long sequence above 7 us)
        if (MODE == MODE_OUT && ch + 1 == nch) break;
        const float last = gt.last;
#pragma unroll
        for (int kt = 0; kt < DK / 16; ++kt)
#pragma unroll
            for (int pt = 0; pt < WT; ++pt) S[kt][pt] *= last;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            if (beyond(32 * kb)) break;
            constexpr int TERMS = V == 4 ? 1 : MODE == MODE_OUT ? 2 : 3;
            const f32x4 w0 = *reinterpret_cast<const f32x4 *>(&gt.w[32 * kb + Bt::LANE * g]);
            const f32x4 w1 = *reinterpret_cast<const f32x4 *>(&gt.w[32 * kb + Bt::LANE * g + Bt::HALF]);
            Frag wx[WT][TERMS];
#pragma unroll
            for (int pt = 0; pt < WT; ++pt) {
                float x[8];
                M::to_floats(xf[kb][pt], x);
#pragma unroll
                for (int j = 0; j < 4; ++j) { x[j] *= w0[j]; x[4 + j] *= w1[j]; }
#pragma unroll
                for (int term = 0; term < TERMS; ++term) {
                    wx[pt][term] = M::from_floats(x);
                    if (term + 1 < TERMS) {
                        float got[8];
                        M::to_floats(wx[pt][term], got);
#pragma unroll
                        for (int j = 0; j < 8; ++j) x[j] -= got[j];
                    }
                }
            }
#pragma unroll
            for (int kt = 0; kt < DK / 16; ++kt) {
                const Frag bf = s.B.spread(kb, kt, lane);
#pragma unroll
                for (int pt = 0; pt < WT; ++pt)
#pragma unroll
                    for (int term = TERMS - 1; term >= 0; --term) S[kt][pt] = M::mma(S[kt][pt], bf, wx[pt][term]);
            }
        }
    }
    if (MODE == MODE_OUT) return;
    float *So = a.segs > 1 ? a.seg_state + state : a.S_out + state;
#pragma unroll
    for (int kt = 0; kt < DK / 16; ++kt)
#pragma unroll
        for (int pt = 0; pt < WT; ++pt)
#pragma unroll
            for (int i = 0; i < 4; ++i) So[Bt::state_row(kt, g, i) * DV + p0 + 16 * pt + col] = S[kt][pt][i];
    if (a.segs > 1 && gates && part == 0 && lane == 0)
        a.seg_decay[((int64_t)n * a.segs + seg) * a.h_v + gh] = (float)exp2(total);
}

// Chains the segments of a state: every segment's local state is replaced by the state in front
// of it, and the last one goes to S_out.  One thread per four entries.
__global__ void __launch_bounds__(NT) chain_kernel(ScanArgs a, int elems)
{
    const int64_t q = (int64_t)blockIdx.x * NT + threadIdx.x;
    const int per = elems / 4;
    const int64_t chain = q / per;
    if (chain >= (int64_t)a.n_seqs * a.h_v) return;
    const int n = (int)(chain / a.h_v), h = (int)(chain % a.h_v);
    const int64_t at = (q % per) * 4;
    int64_t beg, end;
    if (!window(a, n, beg, end)) return;
    const int cps = chunks_per_segment(end - beg, a.segs);
    const int act = cps > 0 ? (int)(((end - beg + CH - 1) / CH + cps - 1) / cps) : 0;
    f32x4 run = {0, 0, 0, 0};
    if (a.S0) run = *reinterpret_cast<const f32x4 *>(a.S0 + chain * elems + at);
    float *p = a.seg_state + ((int64_t)n * a.segs * a.h_v + h) * elems + at;
    const float *d = a.seg_decay + (int64_t)n * a.segs * a.h_v + h;
    const int64_t next = (int64_t)a.h_v * elems;
    constexpr int U = 8;                              // loads in flight: the chain itself is short
    for (int s0 = 0; s0 < act; s0 += U) {
        f32x4 l[U];
        float f[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int s = s0 + u < act ? s0 + u : act - 1;
            l[u] = *reinterpret_cast<const f32x4 *>(p + s * next);
            f[u] = d[(int64_t)s * a.h_v];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (s0 + u >= act) break;
            *reinterpret_cast<f32x4 *>(p + (s0 + u) * next) = run;
            run = run * f[u] + l[u];
        }
    }
    *reinterpret_cast<f32x4 *>(a.S_out + chain * elems + at) = run;
}

// Output row offsets of replay windows, for a caller that asks for them.
__global__ void __launch_bounds__(64) offsets_kernel(ScanArgs a)
{
    int64_t run = 0;
    for (int n0 = 0; n0 <= a.n_seqs; n0 += 64) {
        const int n = n0 + threadIdx.x;
        int64_t v = 0;
        if (n < a.n_seqs) {
            int64_t b = 0, e = 0;
            if (window(a, n, b, e)) v = e - b;
        }
        int64_t sum = v;
#pragma unroll
        for (int off = 1; off < 64; off *= 2) {
            const int64_t up = __shfl_up(sum, off);
            if ((int)threadIdx.x >= off) sum += up;
        }
        if (n <= a.n_seqs) a.cu_out[n] = (int32_t)(run + sum - v);
        run += __shfl(sum, 63);
    }
}

template <int DV, int COLS>
int64_t scan_blocks(const ScanArgs &a) { return (int64_t)a.n_seqs * a.segs * ((int64_t)a.h_v * DV / COLS); }

template <class M, int DK, int DV, int COLS, int MODE>
hipError_t scan_m(const ScanArgs &a, hipStream_t stream)
{
    auto k = scan_kernel<M, DK, DV, COLS, MODE>;
    hipLaunchKernelGGL(k, dim3((unsigned)scan_blocks<DV, COLS>(a)), dim3(COLS * 4 / WT), 0, stream, a);
    return hipGetLastError();
}

template <class M, int DK, int DV, int COLS>
hipError_t scan_c(const ScanArgs &a, hipStream_t stream)
{
    const int64_t chains = a.segs > 1 ? ((int64_t)a.n_seqs * a.h_v * (DK * DV / 4) + NT - 1) / NT : 1;   // blocks of chain_kernel
    if (!grid_ok(scan_blocks<DV, COLS>(a), COLS * 4 / WT) || !grid_ok(chains, NT)) return hipErrorInvalidConfiguration;
    if (a.cu_out) {
        hipLaunchKernelGGL(offsets_kernel, dim3(1), dim3(64), 0, stream, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (a.segs == 1) return a.y ? scan_m<M, DK, DV, COLS, MODE_FULL>(a, stream) : scan_m<M, DK, DV, COLS, MODE_STATE>(a, stream);
    hipError_t e = scan_m<M, DK, DV, COLS, MODE_STATE>(a, stream);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(chain_kernel, dim3((unsigned)chains), dim3(NT), 0, stream, a, DK * DV);
    e = hipGetLastError();
    if (e != hipSuccess || !a.y) return e;
    return scan_m<M, DK, DV, COLS, MODE_OUT>(a, stream);
}

template <class M, int DK>
hipError_t scan_v(const ScanArgs &a, int d_v, hipStream_t stream)
{
    const int cols = scan_columns(a.h_qk, a.h_v, d_v, M::V == 8, (int64_t)a.n_seqs * a.segs * a.h_v * d_v);
    if constexpr (M::V == 8)
        if (cols == 128) return d_v == 128 ? scan_c<M, DK, 128, 128>(a, stream) : scan_c<M, DK, 64, 128>(a, stream);
    return d_v == 128 ? scan_c<M, DK, 128, 64>(a, stream) : scan_c<M, DK, 64, 64>(a, stream);
}

}  // namespace

hipError_t launch_scan(const ScanArgs &a, int bf16, int d_k, int d_v, hipStream_t stream)
{
    if (bf16) return d_k == 128 ? scan_v<MfmaBF16, 128>(a, d_v, stream) : scan_v<MfmaBF16, 64>(a, d_v, stream);
    return d_k == 128 ? scan_v<MfmaF32, 128>(a, d_v, stream) : scan_v<MfmaF32, 64>(a, d_v, stream);
}

}  // namespace gdn
