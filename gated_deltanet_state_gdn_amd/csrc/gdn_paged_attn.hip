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

// Q^T operands of 16 NB rows: row l % 16 of tile b, entries in the nat map; negated for a negative
// scale, which the kernels then take as a positive one.
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
        for (int kb = 0; kb < D / 32; ++kb) {
            q[b][kb] = M::row_nat(p + 32 * kb, 0, lane);
            if (a.scale < 0.0f) {
                float f[8];
                M::to_floats(q[b][kb], f);
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] = -f[i];
                q[b][kb] = M::from_floats(f);
            }
        }
    }
}

// The running softmax of NB tiles of 16 rows, a step being 32 keys (two accumulator tiles of 16):
// scores to probabilities exp2(s - base).  base is the row's maximum of some step, not always the
// running one: it moves only when a score passes it by more than 8, so that probabilities stay
// below 2^8 (their relative accuracy is the same there) and most steps neither exchange maxima
// between lanes nor rescale O.
template <int NB>
struct Soft {
    // -base, and the lane's share of the sum.  Before a row's first key base is lower than any score
    // (-3e38): masked scores (-inf) still give 0, and the first key moves it.
    float neg[NB], l[NB];
    __device__ __forceinline__ Soft() {
#pragma unroll
        for (int b = 0; b < NB; ++b) { neg[b] = 3e38f; l[b] = 0.0f; }
    }
    // The whole row's base (-inf if it has seen nothing) and sum.
    __device__ __forceinline__ void whole(int b, float &m, float &sum) const {
        sum = l[b] + __shfl_xor(l[b], 16);
        sum += __shfl_xor(sum, 32);
        m = sum > 0.0f ? -neg[b] : -INFINITY;
    }
    // scale > 0; the lane's keys are key0 + i and key0 + 16 + i, i = 0..3
    template <class M, int D>
    __device__ __forceinline__ void step(f32x4 (&st)[NB][2], float scale, int32_t key0, const int32_t (&limit)[NB],
                                         bool masked, f32x4 (&o)[NB][D / 16], typename M::Frag (&p)[NB]) {
        float top[NB], over = -INFINITY;
        if (masked) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) st[b][t][i] = key0 + 16 * t + i >= limit[b] ? -INFINITY : st[b][t][i];
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            top[b] = fmaxf(fmaxf(fmaxf(st[b][0][0], st[b][0][1]), fmaxf(st[b][0][2], st[b][0][3])),
                           fmaxf(fmaxf(st[b][1][0], st[b][1][1]), fmaxf(st[b][1][2], st[b][1][3])));
            over = fmaxf(over, fmaf(top[b], scale, neg[b]));
        }
        if (__any(over > 8.0f)) {
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                float t = fmaxf(top[b], __shfl_xor(top[b], 16));
                t = fmaxf(t, __shfl_xor(t, 32)) * scale;
                const float base = fmaxf(t, -neg[b]);
                const float f = exp2f(-neg[b] - base);   // 0 at the first key
                neg[b] = -base;
                l[b] *= f;
#pragma unroll
                for (int d = 0; d < D / 16; ++d) o[b][d] *= f;
            }
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            float s[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                s[i] = __builtin_amdgcn_exp2f(fmaf(st[b][i >> 2][i & 3], scale, neg[b]));
                l[b] += s[i];
            }
            p[b] = M::from_floats(s);
        }
    }
};

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
    const float scale = fmaxf(fabsf(a.scale) * kLog2e, 1e-30f);   // 0: every score is as good as 0
    Soft<NB> sf;
    f32x4 o[NB][D / 16];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int d = 0; d < D / 16; ++d) o[b][d] = f32x4{0, 0, 0, 0};
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
        sf.template step<M, D>(st, scale, k0 + 4 * g, limit, k0 + KT > least, o, p);
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
        float mx, l;
        sf.whole(b, mx, l);
        if (g == 0) { sm[wave][16 * b + col] = mx; sl[wave][16 * b + col] = l; }
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
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(1))) const void global_void;

// A tile of KT keys or values in LDS, rows of D elements without padding: 16-byte chunk c of row r
// sits at chunk c ^ sw(r), so that the fragment reads spread over the banks.  It is filled by loads
// that go from memory to LDS by themselves (64 lanes x 16 bytes in a row of LDS; the lane picks
// its chunk's source).
template <class M, int D>
struct Tile {
    typedef typename M::T T;
    static constexpr int RB = D * sizeof(T), CPR = RB / 16;
    // keys are read 16 rows at one chunk: the low four row bits
    static __device__ __forceinline__ int sw_k(int r) { return r & (CPR < 16 ? CPR - 1 : 15); }
    // values are read 4 rows at a time (lane group g, rows 4 g ..): bf16 2 chunks wide, fp32 4 wide
    static __device__ __forceinline__ int sw_v(int r) {
        return M::V == 8 ? (2 * r) & (CPR - 1) & 31 : (4 * ((r >> 2) & 3)) & (CPR - 1);
    }
    // The lane's part of the addresses; the rest of a fragment's address is an XOR of bits that the
    // row does not reach and a constant.
    static __device__ __forceinline__ uint32_t key_lane(int lane) {
        const int r = lane & 15, g = lane >> 4;
        return r * RB + 16 * ((M::V == 8 ? g : 2 * g) ^ sw_k(r));
    }
    static __device__ __forceinline__ uint32_t value_lane(int lane) {
        const int g = lane >> 4, c = lane & 15, r = 4 * g + (M::V == 8 ? c >> 2 : 0);
        return r * RB + (M::V == 8 ? 8 * (c & 3) : 4 * c) + 16 * sw_v(r);
    }
    // K, 32 entries from 32 kb of the 16 rows from 16 t: row l % 16, nat map
    static __device__ __forceinline__ typename M::Frag key(const char *K, int t, int kb, uint32_t at) {
        const char *p = K + 16 * t * RB;
        if constexpr (M::V == 8) {
            return __builtin_bit_cast(typename M::Frag, load16(p + (at ^ (64 * kb))));
        } else {
            typename M::Frag f;
            M::unpack(load16(p + (at ^ (128 * kb))), f.x);
            M::unpack(load16(p + (at ^ (128 * kb) ^ 16)), f.x + 4);
            return f;
        }
    }
    // V^T, entries 16 d + l % 16 of the 32 rows from k, acc map
    static __device__ __forceinline__ typename M::Frag value(const char *Vt, int k, int d, uint32_t at) {
        if constexpr (M::V == 8) {
            const char *p = Vt + k * RB + (at ^ (32 * d));
            return frag_of(read_tr(reinterpret_cast<const uint16_t *>(p)),
                           read_tr(reinterpret_cast<const uint16_t *>(p + 16 * RB)));
        } else {                                       // rows 4 g + j: one swizzle for all of them
            typename M::Frag f;
            const char *p = Vt + k * RB + (at ^ (64 * d));
#pragma unroll
            for (int j = 0; j < 8; ++j) f.x[j] = *reinterpret_cast<const float *>(p + ((j & 3) + 16 * (j >> 2)) * RB);
            return f;
        }
    }
};
// The value, in a register of its own: what is computed from it in a loop stays in the loop instead
// of being kept in registers over it.
__device__ __forceinline__ uint32_t here(uint32_t v) {
    asm volatile("" : "+v"(v));
    return v;
}

// KT: keys of a tile.  Two tiles of K and V each: the next one comes in while this one is used, one
// barrier a tile.
template <class M, int D, int NB, int WAVES, int KT>
__global__ void __launch_bounds__(64 * WAVES) prefill_kernel(AttnArgs a)
{
    typedef typename M::T T;
    typedef typename M::Frag Frag;
    typedef Tile<M, D> Tl;
    constexpr bool FENCE = D == 256;
    constexpr int ROWS = 16 * NB * WAVES, RB = Tl::RB, CPR = Tl::CPR;
    constexpr int NI = KT * RB / 1024 / WAVES;           // 1 KB loads of a wave for one tile of K or V
    static_assert(NI >= 1, "a tile has work for every wave");
    __shared__ __align__(1024) char K0[KT * RB], V0[KT * RB], K1[KT * RB], V1[KT * RB];
    __shared__ int64_t off[2][KT];                       // byte offsets of the keys' rows
    const int lane = threadIdx.x & 63, g = lane >> 4, col = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
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
    const char *kc = reinterpret_cast<const char *>(static_cast<const T *>(a.kc) + hk * a.head_stride);
    const char *vc = reinterpret_cast<const char *>(static_cast<const T *>(a.vc) + hk * a.head_stride);
    const int first = wave * 16 * NB;
    const uint32_t key_at = Tl::key_lane(lane), value_at = Tl::value_lane(lane);

    Frag q[NB][D / 32];
    load_q<M, D, NB>(a, r, hk, first, lane, q);
    int32_t limit[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) limit[b] = row_limit(r, r.m0 + first + 16 * b + col);
    const int32_t least = row_limit(r, r.m0 + first);
    const float scale = fmaxf(fabsf(a.scale) * kLog2e, 1e-30f);   // 0: every score is as good as 0
    Soft<NB> sf;
    f32x4 o[NB][D / 16];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int d = 0; d < D / 16; ++d) o[b][d] = f32x4{0, 0, 0, 0};

    const int nt = k_end > k_beg ? (k_end - k_beg + KT - 1) / KT : 0;
    // The row of a key behind the end is the last key's (its score is masked), that of a bad page the
    // first page's (recorded): every address is one of the cache's, and P = 0 meets numbers.
    auto row_of = [&](int t) -> int64_t {
        int32_t j = k_beg + t * KT + (int)threadIdx.x;
        j = j < k_end ? j : k_end - 1;
        bool bad = false;
        const int64_t at = cache_offset(table, j, a.page_size, a.n_pages, a.page_stride, a.token_stride, bad);
        if (bad) set_status(a.status);
        return bad ? 0 : at * (int64_t)sizeof(T);
    };
    auto stage = [&](int t, char *Kb, char *Vb) {
        const int ln = (int)here(lane);
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int at = (wave * NI + i) * 64 + ln, row = at / CPR, pc = at % CPR;
            const int64_t src = off[t & 1][row];
            __builtin_amdgcn_global_load_lds((global_void *)(kc + src + 16 * (pc ^ Tl::sw_k(row))),
                                             (lds_void *)(Kb + (wave * NI + i) * 1024), 16, 0, 0);
            __builtin_amdgcn_global_load_lds((global_void *)(vc + src + 16 * (pc ^ Tl::sw_v(row))),
                                             (lds_void *)(Vb + (wave * NI + i) * 1024), 16, 0, 0);
        }
    };
    auto compute = [&](int t, const char *Kb, const char *Vb) {
        const int32_t k0 = k_beg + t * KT;
#pragma unroll
        for (int k = 0; k < KT; k += 32) {
            const uint32_t ka = here(key_at), va = here(value_at);
            f32x4 st[NB][2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int b = 0; b < NB; ++b) st[b][h] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int kb = 0; kb < D / 32; ++kb) {
                    const Frag kf = Tl::key(Kb, k / 16 + h, kb, ka);
#pragma unroll
                    for (int b = 0; b < NB; ++b) st[b][h] = M::mma(st[b][h], kf, q[b][kb]);
                    if (FENCE && kb % 4 == 3) __builtin_amdgcn_sched_barrier(0);
                }
            }
            Frag p[NB];
            sf.template step<M, D>(st, scale, k0 + k + 4 * g, limit, k0 + k + 32 > least, o, p);
            if (FENCE) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
                const Frag vf = Tl::value(Vb, k, d, va);
#pragma unroll
                for (int b = 0; b < NB; ++b) o[b][d] = M::mma(o[b][d], vf, p[b]);
                if (FENCE && d % 4 == 3) __builtin_amdgcn_sched_barrier(0);
            }
        }
    };
    auto turn = [&](int t, char *Kb, char *Vb, char *Kn, char *Vn) {
        __syncthreads();                                 // this tile is here, the other buffer is free
        const bool ahead = t + 2 < nt && threadIdx.x < KT;
        int64_t row = 0;
        if (ahead) row = row_of(t + 2);
        if (t + 1 < nt) stage(t + 1, Kn, Vn);
        if (FENCE) __builtin_amdgcn_sched_barrier(0);
        compute(t, Kb, Vb);
        if (ahead) off[t & 1][threadIdx.x] = row;
    };
    if (nt > 0) {
        if (a.n_pages == 0) {                            // no page at all: nothing can be read
            if (threadIdx.x == 0) set_status(a.status);
            return;
        }
        if (threadIdx.x < KT) {
            off[0][threadIdx.x] = row_of(0);
            if (nt > 1) off[1][threadIdx.x] = row_of(1);
        }
        __syncthreads();
        stage(0, K0, V0);
        for (int t = 0; t < nt; t += 2) {
            turn(t, K0, V0, K1, V1);
            if (t + 1 < nt) turn(t + 1, K1, V1, K0, V0);
        }
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        float mx, l;
        sf.whole(b, mx, l);
        const int row = first + 16 * b + col;
        if (row >= r.count) continue;
#pragma unroll
        for (int d = 0; d < D / 16; ++d) store_share<M, D>(a, r, hk, split, row, 16 * d + 4 * g, o[b][d], mx, l);
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
hipError_t start(K k, int64_t blocks, int lds, const AttnArgs &a, hipStream_t stream, int threads = NT)
{
    if (blocks > kMaxBlocks) return hipErrorInvalidConfiguration;
    if (blocks <= 0) return hipSuccess;
    if (lds > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(k), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(k, dim3((unsigned)blocks), dim3(threads), lds, stream, a);
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
        // fp32 rows of 256 entries: the operands and sums of 16 rows fill a wave's registers
        constexpr bool WIDE = D * sizeof(typename M::T) > 512;
        constexpr int NB = WIDE ? 1 : 2, KT = WIDE ? 32 : 64;
        const int64_t blocks = (a.total * G / p.rows + a.n_seqs) * a.splits * a.h_kv;
        if constexpr (WIDE) e = start(prefill_kernel<M, D, NB, 8, KT>, blocks, 0, a, stream, 512);
        else if (p.rows == 256) e = start(prefill_kernel<M, D, NB, 8, KT>, blocks, 0, a, stream, 512);
        else e = start(prefill_kernel<M, D, NB, 4, KT>, blocks, 0, a, stream, 256);
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
    p.rows = p.decode ? 16 : bf16 && total * G >= 192 * (int64_t)n_seqs ? 256 : 128;
    const int64_t tiles = (total * G / p.rows + n_seqs) * h_kv;
    int64_t want = (p.decode ? 1024 : 256 * (256 / p.rows)) / (tiles > 0 ? tiles : 1);
    if (want < 1) want = 1;
    int64_t keys = (max_kv + want - 1) / want;
    const int64_t least = p.decode ? 128 : 1024;
    if (keys < least) keys = least;
    p.split_keys = (int32_t)((keys + 127) / 128 * 128);
    p.splits = max_kv > 0 ? (max_kv + p.split_keys - 1) / p.split_keys : 1;
    (void)d;
    return p;
}

hipError_t launch_attn(const AttnArgs &a, const AttnPlan &p, int bf16, int d, hipStream_t stream)
{
    return bf16 ? attn_m<MfmaBF16>(a, p, d, stream) : attn_m<MfmaF32>(a, p, d, stream);
}

}  // namespace gdn
