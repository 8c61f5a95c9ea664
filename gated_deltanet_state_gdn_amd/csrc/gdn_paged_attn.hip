// Attention of new tokens over a paged cache.
//
// Token i of a sequence with L new tokens and kv_len cached ones (the new ones among them) sits at
// position p = kv_len - L + i and attends to the keys 0..p of its sequence; v-head group: query
// head h reads cache head floor(h h_kv / h_q).
//     o = sum_{j <= p} exp(s_j - lse) v_j,   s_j = scale q . k_j,   lse = ln sum_{j <= p} exp s_j
//
// The G = h_q / h_kv query heads of a cache head are rows of the same product: row m = i G + h % G,
// so a tile of rows shares every key and value that it reads, for one token as for many.  Both
// products are formed transposed, S^T = K Q^T and O^T = V^T P^T: a lane then holds scores of ONE
// row, the softmax runs inside the lane and over two lane exchanges, P^T goes from accumulators to
// operand without moving, and the running rescale of O is one factor a lane.  One pass over the
// keys with the running maximum m and sum l; long caches are cut into splits of keys whose (O, m,
// l) a second kernel joins.  Scores are in log2 units.
//
// Two kernels.  Few rows per sequence (single tokens): bound by the reads of K and V; the four
// waves of a workgroup take different keys, K goes from memory to registers as operands, V through
// LDS for its transposition, and the waves' results are joined at the end.  Many rows: bound by
// the matrix products; the waves take different rows and share the keys' tiles in LDS.
//
// Precision: scores, maximum, sum, O are fp32.  With bf16 elements the products take q, k and v as
// they are, and P (0 <= P <= 1) is rounded to bf16 once, half a bf16 step as the output is; the sum
// l takes the unrounded P.  Keys behind kv_len are never read: whatever a page holds there (or an
// unused page) does not matter.
#include "gdn_mfma.h"

namespace gdn {
namespace {

constexpr int NT = 256;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// A block's rows: rows [m0, m0 + count) of sequence n, row m = (token i, head i_h).
struct Rows {
    int n, G;
    int32_t beg, kv, pos0;      // first token, cached tokens, position of token 0
    int32_t m0, count;
};
__device__ __forceinline__ bool find_rows(const AttnArgs &a, int64_t tile, int rows, Rows &r)
{
    r.G = a.h_q / a.h_kv;
    r.n = tile_sequence(a.cu, a.n_seqs, tile, r.G, rows);
    const int32_t b = a.cu[r.n], e = a.cu[r.n + 1];
    if (!range_ok(b, e, a.total)) return false;          // recorded by check_cu
    r.beg = b;
    r.kv = a.kv_len[r.n];
    if (!kv_ok(r.kv, a.max_kv, a.page_size, a.max_pages)) {
        if (threadIdx.x == 0) set_status(a.status);
        return false;
    }
    r.pos0 = r.kv - (e - b);
    const int64_t k = tile - first_tile(b, r.n, r.G, rows);
    const int64_t all = (int64_t)(e - b) * r.G, m0 = k * rows;
    if (k < 0 || m0 >= all) return false;
    r.m0 = (int32_t)m0;
    r.count = (int32_t)(all - m0 < rows ? all - m0 : rows);
    return true;
}
// Keys that row m sees: its position + 1 (0 or less: none).
__device__ __forceinline__ int32_t row_limit(const Rows &r, int32_t m) { return r.pos0 + m / r.G + 1; }

// Element offset of key j's row in the caches (head 0), or -1 behind `end` or for a bad page.
__device__ __forceinline__ int64_t key_offset(const AttnArgs &a, const int32_t *table, int32_t j, int32_t end)
{
    if (j >= end) return -1;
    bool bad = false;
    const int64_t at = cache_offset(table, j, a.page_size, a.n_pages, a.page_stride, a.token_stride, bad);
    if (bad) set_status(a.status);
    return at;
}

// Q^T operands of 16 NB rows: row l % 16 of tile b, entries in the nat map.
template <class M, int D, int NB>
__device__ __forceinline__ void load_q(const AttnArgs &a, const Rows &r, int hk, int first, int lane,
                                       typename M::Frag (&q)[NB][D / 32])
{
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const int m = first + 16 * b + (lane & 15);
        const int mm = r.m0 + (m < r.count ? m : 0);     // rows past the end repeat the first; they are not stored
        const typename M::T *p = static_cast<const typename M::T *>(a.q) + (int64_t)(r.beg + mm / r.G) * a.qs +
                                 (int64_t)(hk * r.G + mm % r.G) * D;
#pragma unroll
        for (int kb = 0; kb < D / 32; ++kb) q[b][kb] = M::row_nat(p + 32 * kb, 0, lane);
    }
}

// One step of the running softmax over 32 keys (two accumulator tiles of 16) for one tile of 16
// rows: scores to probabilities, O^T and the lane's share of l rescaled.
template <class M, int D>
__device__ __forceinline__ typename M::Frag soft_step(f32x4 (&st)[2], float scale, int32_t key0, int32_t limit, bool masked,
                                                      float &m, float &l, f32x4 (&o)[D / 16])
{
    float s[8];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float v = st[t][i] * scale;
            s[4 * t + i] = masked && key0 + 16 * t + i >= limit ? -INFINITY : v;
        }
    float top = s[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) top = fmaxf(top, s[i]);
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    const float mn = fmaxf(m, top);
    const float base = mn == -INFINITY ? 0.0f : mn;      // a row that has seen nothing yet
    const float f = exp2f(m - base);
    m = mn;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        s[i] = exp2f(s[i] - base);
        sum += s[i];
    }
    l = l * f + sum;
#pragma unroll
    for (int d = 0; d < D / 16; ++d) o[d] *= f;
    return M::from_floats(s);
}

// The finished rows: normalised outputs, or a split's share.
template <class M, int D>
__device__ __forceinline__ void store_share(const AttnArgs &a, const Rows &r, int hk, int split, int m, int d4, f32x4 o, float mx, float l)
{
    const int mm = r.m0 + m;
    const int64_t t = r.beg + mm / r.G;
    const int h = hk * r.G + mm % r.G;
    if (a.splits == 1) {
        const float inv = l > 0.0f ? 1.0f / l : 0.0f;
        float x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = o[i] * inv;
        M::store4(static_cast<typename M::T *>(a.o) + t * a.os + (int64_t)h * D + d4, x);
        if (a.lse && d4 == 0) a.lse[t * a.h_q + h] = l > 0.0f ? mx * kLn2 + logf(l) : -INFINITY;
        return;
    }
    const int64_t at = ((int64_t)split * a.total + t) * a.h_q + h;
    *reinterpret_cast<f32x4 *>(a.part_o + at * D + d4) = o;
    if (d4 == 0) *reinterpret_cast<f32x2 *>(a.part_ml + at * 2) = f32x2{mx, l};
}

// ------------------------------------------------------------- few rows: waves over the keys
template <class M, int D, int NB>
__global__ void __launch_bounds__(NT) decode_kernel(AttnArgs a)
{
    typedef typename M::T T;
    typedef typename M::Frag Frag;
    constexpr int ROWS = 16 * NB, SD = D + M::PAD, KT = 32;
    constexpr int VW = KT * SD * sizeof(T), OW = ROWS * (D + 4) * 4;
    constexpr int WB = VW > OW ? VW : OW;                // a wave's LDS: its V tile, later its O
    extern __shared__ __align__(16) char smem[];
    __shared__ float sm[4][ROWS], sl[4][ROWS];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, col = lane & 15;
    if (blockIdx.x == 0 && threadIdx.x < 64) check_cu(a.cu, a.n_seqs, a.total, a.status);
    const int hk = blockIdx.x % a.h_kv;
    const int split = (blockIdx.x / a.h_kv) % a.splits;
    const int64_t tile = blockIdx.x / a.h_kv / a.splits;
    Rows r;
    if (!find_rows(a, tile, ROWS, r)) return;
    const int32_t most = row_limit(r, r.m0 + r.count - 1);        // keys that the tile's last row sees
    const int32_t k_beg = split * a.split_keys;
    if (split > 0 && k_beg >= most) return;                       // nothing here for any row
    const int32_t k_end = most < k_beg + a.split_keys ? most : k_beg + a.split_keys;
    const int32_t *table = a.table + (int64_t)r.n * a.max_pages;
    const T *kc = static_cast<const T *>(a.kc) + hk * a.head_stride;
    const T *vc = static_cast<const T *>(a.vc) + hk * a.head_stride;
    T *Vs = reinterpret_cast<T *>(smem + wave * WB);

    Frag q[NB][D / 32];
    load_q<M, D, NB>(a, r, hk, 0, lane, q);
    int32_t limit[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) limit[b] = row_limit(r, r.m0 + 16 * b + col);
    const int32_t least = row_limit(r, r.m0);
    const float scale = a.scale * kLog2e;
    float m[NB], l[NB];
    f32x4 o[NB][D / 16];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        m[b] = -INFINITY;
        l[b] = 0.0f;
#pragma unroll
        for (int d = 0; d < D / 16; ++d) o[b][d] = f32x4{0, 0, 0, 0};
    }
    constexpr int NV = KT * D / M::V / 64;
    for (int32_t k0 = k_beg + wave * KT; k0 < k_end; k0 += 4 * KT) {
        // V: rows to LDS, 16 bytes a lane
        u32x4 rv[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = (lane + i * 64) * M::V;
            const int64_t at = key_offset(a, table, k0 + e / D, k_end);
            rv[i] = at >= 0 ? load16(vc + at + e % D) : u32x4{0, 0, 0, 0};
        }
        f32x4 st[NB][2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int64_t at = key_offset(a, table, k0 + 16 * t + col, k_end);
            Frag kf[D / 32];
#pragma unroll
            for (int kb = 0; kb < D / 32; ++kb) {
                if (at >= 0) kf[kb] = M::row_nat(kc + at + 32 * kb, 0, lane);
                else kf[kb] = Frag{};
            }
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                st[b][t] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int kb = 0; kb < D / 32; ++kb) st[b][t] = M::mma(st[b][t], kf[kb], q[b][kb]);
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = (lane + i * 64) * M::V;
            store16(Vs + e / D * SD + e % D, rv[i]);
        }
        wave_sync();
        Frag p[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b)
            p[b] = soft_step<M, D>(st[b], scale, k0 + 4 * g, limit[b], k0 + KT > least, m[b], l[b], o[b]);
#pragma unroll
        for (int d = 0; d < D / 16; ++d) {
            const Frag vf = M::col_acc(Vs + 16 * d, SD, lane);
#pragma unroll
            for (int b = 0; b < NB; ++b) o[b][d] = M::mma(o[b][d], vf, p[b]);
        }
        wave_sync();
    }
    // join the waves: every wave's (m, l, O) to LDS, then one thread per four entries of a row
    float *Os = reinterpret_cast<float *>(smem + wave * WB);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        l[b] += __shfl_xor(l[b], 16);
        l[b] += __shfl_xor(l[b], 32);
        if (g == 0) { sm[wave][16 * b + col] = m[b]; sl[wave][16 * b + col] = l[b]; }
#pragma unroll
        for (int d = 0; d < D / 16; ++d)
            *reinterpret_cast<f32x4 *>(Os + (16 * b + col) * (D + 4) + 16 * d + 4 * g) = o[b][d];
    }
    __syncthreads();
    for (int e = threadIdx.x * 4; e < r.count * D; e += NT * 4) {
        const int row = e / D, d4 = e % D;
        float mx = sm[0][row];
#pragma unroll
        for (int w = 1; w < 4; ++w) mx = fmaxf(mx, sm[w][row]);
        const float base = mx == -INFINITY ? 0.0f : mx;
        f32x4 sum = {0, 0, 0, 0};
        float ll = 0.0f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float f = exp2f(sm[w][row] - base);
            sum += *reinterpret_cast<const f32x4 *>(reinterpret_cast<const float *>(smem + w * WB) + row * (D + 4) + d4) * f;
            ll += sl[w][row] * f;
        }
        store_share<M, D>(a, r, hk, split, row, d4, sum, mx, ll);
    }
}

// ------------------------------------------------------------- many rows: waves over the rows
template <class M, int D, int NB, int KT>
__global__ void __launch_bounds__(NT) prefill_kernel(AttnArgs a)
{
    typedef typename M::T T;
    typedef typename M::Frag Frag;
    constexpr int ROWS = 64 * NB, SD = D + M::PAD;
    extern __shared__ __align__(16) char smem[];
    T *Ks = reinterpret_cast<T *>(smem), *Vs = Ks + KT * SD;
    __shared__ int64_t off[KT];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, col = lane & 15;
    if (blockIdx.x == 0 && threadIdx.x < 64) check_cu(a.cu, a.n_seqs, a.total, a.status);
    const int hk = blockIdx.x % a.h_kv;
    const int split = (blockIdx.x / a.h_kv) % a.splits;
    const int64_t tile = blockIdx.x / a.h_kv / a.splits;
    Rows r;
    if (!find_rows(a, tile, ROWS, r)) return;
    const int32_t most = row_limit(r, r.m0 + r.count - 1);
    const int32_t k_beg = split * a.split_keys;
    if (split > 0 && k_beg >= most) return;
    const int32_t k_end = most < k_beg + a.split_keys ? most : k_beg + a.split_keys;
    const int32_t *table = a.table + (int64_t)r.n * a.max_pages;
    const T *kc = static_cast<const T *>(a.kc) + hk * a.head_stride;
    const T *vc = static_cast<const T *>(a.vc) + hk * a.head_stride;
    const int first = wave * 16 * NB;

    Frag q[NB][D / 32];
    load_q<M, D, NB>(a, r, hk, first, lane, q);
    int32_t limit[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) limit[b] = row_limit(r, r.m0 + first + 16 * b + col);
    const int32_t least = row_limit(r, r.m0 + first);
    const float scale = a.scale * kLog2e;
    float m[NB], l[NB];
    f32x4 o[NB][D / 16];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        m[b] = -INFINITY;
        l[b] = 0.0f;
#pragma unroll
        for (int d = 0; d < D / 16; ++d) o[b][d] = f32x4{0, 0, 0, 0};
    }
    constexpr int NV = KT * D / M::V / NT;
    for (int32_t k0 = k_beg; k0 < k_end; k0 += KT) {
        __syncthreads();                                 // the last tile's readers are done
        if (threadIdx.x < KT) off[threadIdx.x] = key_offset(a, table, k0 + threadIdx.x, k_end);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = (threadIdx.x + i * NT) * M::V;
            const int64_t at = off[e / D];
            store16(Ks + e / D * SD + e % D, at >= 0 ? load16(kc + at + e % D) : u32x4{0, 0, 0, 0});
            store16(Vs + e / D * SD + e % D, at >= 0 ? load16(vc + at + e % D) : u32x4{0, 0, 0, 0});
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < KT; k += 32) {
            f32x4 st[NB][2];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
#pragma unroll
                for (int b = 0; b < NB; ++b) st[b][t] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int kb = 0; kb < D / 32; ++kb) {
                    const Frag kf = M::row_nat(Ks + (k + 16 * t) * SD + 32 * kb, SD, lane);
#pragma unroll
                    for (int b = 0; b < NB; ++b) st[b][t] = M::mma(st[b][t], kf, q[b][kb]);
                }
            }
            Frag p[NB];
#pragma unroll
            for (int b = 0; b < NB; ++b)
                p[b] = soft_step<M, D>(st[b], scale, k0 + k + 4 * g, limit[b], k0 + k + 32 > least, m[b], l[b], o[b]);
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
                const Frag vf = M::col_acc(Vs + k * SD + 16 * d, SD, lane);
#pragma unroll
                for (int b = 0; b < NB; ++b) o[b][d] = M::mma(o[b][d], vf, p[b]);
            }
        }
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        l[b] += __shfl_xor(l[b], 16);
        l[b] += __shfl_xor(l[b], 32);
        const int row = first + 16 * b + col;
        if (row >= r.count) continue;
#pragma unroll
        for (int d = 0; d < D / 16; ++d) store_share<M, D>(a, r, hk, split, row, 16 * d + 4 * g, o[b][d], m[b], l[b]);
    }
}

// ------------------------------------------------------------- the splits of a row, joined
// One wave per row: the splits that hold keys of the row, in order.
template <class M, int D>
__global__ void __launch_bounds__(NT) join_kernel(AttnArgs a)
{
    typedef typename M::T T;
    constexpr int E = D / 64;                            // entries of a lane
    const int lane = threadIdx.x & 63;
    const int64_t row = (int64_t)blockIdx.x * (NT / 64) + (threadIdx.x >> 6);
    if (row >= a.total * a.h_q) return;
    const int64_t t = row / a.h_q;
    const int n = token_sequence(a.cu, a.n_seqs, t);
    const int32_t b = a.cu[n], e = a.cu[n + 1];
    if (!range_ok(b, e, a.total) || t < b || t >= e) return;
    const int32_t kv = a.kv_len[n];
    if (!kv_ok(kv, a.max_kv, a.page_size, a.max_pages)) return;
    const int32_t limit = kv - (e - (int32_t)t) + 1;
    const int act = limit > 0 ? (limit + a.split_keys - 1) / a.split_keys : 1;
    const int64_t step = a.total * a.h_q;
    float mx = -INFINITY;
    for (int s = lane; s < act; s += 64) mx = fmaxf(mx, a.part_ml[(s * step + row) * 2]);
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) mx = fmaxf(mx, __shfl_xor(mx, off));
    const float base = mx == -INFINITY ? 0.0f : mx;
    float l = 0.0f, acc[E];
#pragma unroll
    for (int i = 0; i < E; ++i) acc[i] = 0.0f;
    for (int s = 0; s < act; ++s) {
        const f32x2 ml = *reinterpret_cast<const f32x2 *>(a.part_ml + (s * step + row) * 2);
        const float f = exp2f(ml.x - base);
        l += ml.y * f;
        const float *p = a.part_o + (s * step + row) * D + lane * E;
#pragma unroll
        for (int i = 0; i < E; ++i) acc[i] = fmaf(p[i], f, acc[i]);
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    T *o = static_cast<T *>(a.o) + t * a.os + (row % a.h_q) * D + lane * E;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        if constexpr (M::V == 8) o[i] = (uint16_t)pack_bf16(acc[i] * inv, 0.0f);
        else o[i] = acc[i] * inv;
    }
    if (a.lse && lane == 0) a.lse[row] = l > 0.0f ? mx * kLn2 + logf(l) : -INFINITY;
}

template <class K>
hipError_t start(K k, int64_t blocks, int lds, const AttnArgs &a, hipStream_t stream)
{
    if (blocks > kMaxBlocks) return hipErrorInvalidConfiguration;
    if (blocks <= 0) return hipSuccess;
    if (lds > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(k), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(k, dim3((unsigned)blocks), dim3(NT), lds, stream, a);
    return hipGetLastError();
}

template <class M, int D>
hipError_t attn_d(const AttnArgs &a, const AttnPlan &p, hipStream_t stream)
{
    constexpr int SD = D + M::PAD;
    const int G = a.h_q / a.h_kv;
    hipError_t e;
    if (p.decode) {
        constexpr int VW = 32 * SD * sizeof(typename M::T), OW = 16 * (D + 4) * 4;
        const int64_t blocks = (a.total * G / 16 + a.n_seqs) * a.splits * a.h_kv;
        e = start(decode_kernel<M, D, 1>, blocks, 4 * (VW > OW ? VW : OW), a, stream);
    } else {
        constexpr int NB = 2, KT = M::V == 8 ? 64 : 32;
        const int64_t blocks = (a.total * G / (64 * NB) + a.n_seqs) * a.splits * a.h_kv;
        e = start(prefill_kernel<M, D, NB, KT>, blocks, 2 * KT * SD * (int)sizeof(typename M::T), a, stream);
    }
    if (e != hipSuccess || a.splits == 1) return e;
    return start(join_kernel<M, D>, (a.total * a.h_q + 3) / 4, 0, a, stream);
}

template <class M>
hipError_t attn_m(const AttnArgs &a, const AttnPlan &p, int d, hipStream_t stream)
{
    switch (d) {
    case 64: return attn_d<M, 64>(a, p, stream);
    case 128: return attn_d<M, 128>(a, p, stream);
    case 256: return attn_d<M, 256>(a, p, stream);
    default: return hipErrorNotSupported;
    }
}

}  // namespace

AttnPlan attn_plan(int64_t total, int32_t n_seqs, int32_t h_q, int32_t h_kv, int32_t d, int32_t max_kv, int bf16)
{
    const int64_t G = h_q / h_kv;
    AttnPlan p;
    p.decode = total * G <= 32 * (int64_t)n_seqs;
    const int rows = p.decode ? 16 : 128;
    const int64_t tiles = (total * G / rows + n_seqs) * h_kv;
    int64_t want = (p.decode ? 1024 : 512) / (tiles > 0 ? tiles : 1);
    if (want < 1) want = 1;
    int64_t keys = (max_kv + want - 1) / want;
    const int64_t least = p.decode ? 128 : 1024;
    if (keys < least) keys = least;
    p.split_keys = (int32_t)((keys + 127) / 128 * 128);
    p.splits = max_kv > 0 ? (max_kv + p.split_keys - 1) / p.split_keys : 1;
    (void)d;
    (void)bf16;
    return p;
}

hipError_t launch_attn(const AttnArgs &a, const AttnPlan &p, int bf16, int d, hipStream_t stream)
{
    return bf16 ? attn_m<MfmaBF16>(a, p, d, stream) : attn_m<MfmaF32>(a, p, d, stream);
}

}  // namespace gdn
