// Kernels of the attention of new tokens over a paged cache.
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
// Two kernels.  Few rows per sequence (single tokens): bound by the reads of K and V; the
// waves of a workgroup take different keys, K goes from memory to registers as operands, V through
// LDS for its transposition, and the waves' results are joined at the end.  Many rows: bound by
// the matrix products; the waves take different rows and share the keys' tiles in LDS.
//
// Precision: scores, maximum, sum, O are fp32.  With bf16 elements the products take q, k and v as
// they are; P is rounded to bf16 once where the products are the bound (half a bf16 step of each term p v; a
// second term would be half as many products again), and taken in two bf16 terms in the form of few rows, where memory is,
// and where a batch of few rows a sequence has a prefix in the form of many: which form that takes is the plan's
// choice, not the caller's.  The sum l takes the unrounded P.  Relative error of the outputs, 2-norm, in the measured
// cases: 2.3e-3 with one term, 1.7e-3 with two, which is the outputs' own rounding.
// Keys behind kv_len are never read: whatever a page holds there (or an unused page) does not matter.
#pragma once
#include "gdn_mfma.h"

namespace gdn {
namespace {

constexpr int NT = 256;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Which keys a launch is over.  kWhole: a sequence's own rows over all of its keys.  kShared: sequences of a group
// share their first P tokens, and a block is of one of two sides: Prefix takes the rows of a whole group over the keys [0,
// P), read through the block table of its first sequence, Own a sequence's rows over the keys from P on.  Both leave their
// share to the join.
enum Side { kWhole, kShared };

// A block's rows: rows [m0, m0 + count) of sequence n, row m = (token i, head i_h); of a group, from
// the first token of its first sequence n on.
struct Rows {
    int n, G;
    int32_t beg, kv, pos0;      // first token, cached tokens (Prefix: P), position of token 0
    int32_t m0, count;
    // kShared
    bool prefix;                // the side
    int32_t from, behind;       // Own: P; Prefix: 0, the sequence behind the group's last
    int32_t splits, split_keys, part;      // of the side; its first part
    uint32_t block;             // the block's number in it
};
// The side of a block, and its number there: the prefixes' come first.
template <Side S>
__device__ __forceinline__ void find_side(const AttnArgs &a, Rows &r)
{
    r.block = blockIdx.x;
    r.prefix = S == kShared && blockIdx.x < a.prefix_blocks;
    r.splits = S == kShared && r.prefix ? a.prefix_splits : a.splits;
    r.split_keys = S == kShared && r.prefix ? a.prefix_keys : a.split_keys;
    r.part = S == kShared && !r.prefix ? a.prefix_splits : 0;
    if (S == kShared && !r.prefix) r.block -= a.prefix_blocks;
}
__device__ __forceinline__ bool prefix_ok(const AttnArgs &a, int32_t P)
{
    return kv_ok(P, a.max_prefix, a.page_size, a.max_pages);
}
// Group g's sequences, if they are a range of them.
__device__ __forceinline__ bool group_range(const AttnArgs &a, int g, int32_t &first, int32_t &behind)
{
    first = a.groups[g];
    behind = a.groups[g + 1];
    return range_ok(first, behind, a.n_seqs);
}
// The whole of cu_groups, by one wave.
__device__ __forceinline__ void check_groups(const AttnArgs &a)
{
    const int lane = threadIdx.x & 63;
    bool bad = false;
    for (int g = lane; g < a.n_groups; g += 64) {
        int32_t first, behind;
        bad |= !group_range(a, g, first, behind) || (g == 0 && first != 0) || (g == a.n_groups - 1 && behind != a.n_seqs);
    }
    if (__any(bad) && lane == 0) set_status(a.status);
}
// The prefix of sequence n, and whether its group, prefix and cached tokens are in range.
__device__ __forceinline__ bool find_prefix(const AttnArgs &a, int n, int32_t kv, int32_t &P)
{
    const int g = last_before(a.n_groups, [&](int i) { return a.groups[i] <= n; });
    int32_t first, behind;
    if (!group_range(a, g, first, behind) || n < first || n >= behind) return false;
    P = a.prefix_len[g];
    return prefix_ok(a, P) && kv - P <= a.max_own;
}
__device__ __forceinline__ bool find_group(const AttnArgs &a, int64_t tile, int rows, Rows &r)
{
    const int g = last_before(a.n_groups, [&](int i) {
        const int32_t n = a.groups[i];
        return first_tile(a.cu[n < 0 ? 0 : n > a.n_seqs ? a.n_seqs : n], i, r.G, rows) <= tile;
    });
    int32_t first;
    if (!group_range(a, g, first, r.behind)) return false;   // recorded by check_groups
    const int32_t b = a.cu[first], e = a.cu[r.behind];
    if (!range_ok(b, e, a.total)) return false;              // recorded by check_cu
    r.n = first;
    r.beg = b;
    r.kv = a.prefix_len[g];
    const int64_t k = tile - first_tile(b, g, r.G, rows);
    const int64_t all = (int64_t)(e - b) * r.G, m0 = k * rows;
    if (k < 0 || m0 >= all) return false;
    if (!prefix_ok(a, r.kv)) {
        if (threadIdx.x == 0) set_status(a.status);
        return false;
    }
    r.m0 = (int32_t)m0;
    r.count = (int32_t)(all - m0 < rows ? all - m0 : rows);
    r.from = r.pos0 = 0;
    return true;
}
template <Side S>
__device__ __forceinline__ bool find_rows(const AttnArgs &a, int64_t tile, int rows, Rows &r)
{
    r.G = a.h_q / a.h_kv;
    if constexpr (S == kShared)
        if (r.prefix) return find_group(a, tile, rows, r);
    r.from = 0;
    r.n = tile_sequence(a.cu, a.n_seqs, tile, r.G, rows);
    const int32_t b = a.cu[r.n], e = a.cu[r.n + 1];
    if (!range_ok(b, e, a.total)) return false;          // recorded by check_cu
    r.beg = b;
    r.kv = a.kv_len[r.n];
    if (!kv_ok(r.kv, a.max_kv, a.page_size, a.max_pages)) {
        if (threadIdx.x == 0) set_status(a.status);
        return false;
    }
    if constexpr (S == kShared) {
        if (!find_prefix(a, r.n, r.kv, r.from)) {
            if (threadIdx.x == 0) set_status(a.status);
            return false;
        }
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
// Keys of the prefix that row m of a group sees: all, but for a row whose position is inside it.
__device__ __forceinline__ int32_t prefix_limit(const AttnArgs &a, const Rows &r, int32_t m)
{
    const int32_t t = r.beg + m / r.G;
    int lo = r.n, hi = r.behind;                             // the row's sequence: the last with cu[n] <= t
    while (hi - lo > 1) {
        const int mid = lo + (hi - lo) / 2;
        if (a.cu[mid] <= t) lo = mid;
        else hi = mid;
    }
    const int64_t limit = (int64_t)a.kv_len[lo] - a.cu[lo + 1] + t + 1;
    return limit < 0 ? 0 : limit < r.kv ? (int32_t)limit : r.kv;
}
// The keys that NB tiles of 16 rows see, for the row l % 16 of each, and the least of them (rows past the end
// count as the last one).
template <int NB>
__device__ __forceinline__ int32_t shared_limits(const AttnArgs &a, const Rows &r, int first, int lane, int32_t (&lim)[NB])
{
    int32_t least = 0x7fffffff;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const int m = first + 16 * b + (lane & 15), mm = r.m0 + (m < r.count ? m : r.count - 1);
        lim[b] = r.prefix ? prefix_limit(a, r, mm) : row_limit(r, mm);
        least = lim[b] < least ? lim[b] : least;
    }
#pragma unroll
    for (int off = 8; off >= 1; off >>= 1) {
        const int32_t other = __shfl_xor(least, off);
        least = other < least ? other : least;
    }
    return __builtin_amdgcn_readfirstlane(least);
}

// Where key j of a sequence is, in two steps, so that the block table's entry can be on its way while
// other work goes on: the entry, and the byte offset of the key's row in the caches (head 0).  A key
// behind the end stands for the last one (its score is masked), one of a bad page for the first
// page's first (recorded): every address is one of the cache's, and P = 0 meets numbers.
struct Key {
    int32_t j, page;
};
__device__ __forceinline__ Key find_key(const AttnArgs &a, const int32_t *table, int32_t j, int32_t end)
{
    Key k;
    k.j = j < end ? j : end - 1;
    k.page = table[k.j / a.page_size];
    return k;
}
__device__ __forceinline__ int64_t key_row(const AttnArgs &a, const Key &k, int elem_bytes)
{
    bool bad = false;
    const int64_t at = page_offset(k.page, k.j % a.page_size, a.n_pages, a.page_stride, a.token_stride, bad);
    if (bad) set_status(a.status);
    return bad ? 0 : at * elem_bytes;
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
        for (int kb = 0; kb < D / 32; ++kb) q[b][kb] = M::row_nat(p + 32 * kb, 0, lane);
    }
    if (a.scale < 0.0f)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int kb = 0; kb < D / 32; ++kb) {
                float f[8];
                M::to_floats(q[b][kb], f);
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] = -f[i];
                q[b][kb] = M::from_floats(f);
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
    // scale > 0; the lane's keys are key0 + i and key0 + 16 + i, i = 0..3; limit(b): keys that its row sees
    // TERMS: P in that many terms of the element type (two bf16 terms hold 16 bits)
    template <class M, int D, int TERMS, class Limit>
    __device__ __forceinline__ void step(f32x4 (&st)[NB][2], float scale, int32_t key0, Limit limit, bool masked,
                                         f32x4 (&o)[NB][D / 16], typename M::Frag (&p)[NB][TERMS]) {
        float top[NB], over = -INFINITY;
        if (masked) {
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const int32_t end = limit(b) - key0;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) st[b][t][i] = 16 * t + i >= end ? -INFINITY : st[b][t][i];
            }
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
                const float f = __builtin_amdgcn_exp2f(-neg[b] - base);   // 0 at the first key
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
#pragma unroll
            for (int t = 0; t < TERMS; ++t) {
                p[b][t] = M::from_floats(s);
                if (t + 1 < TERMS) {
                    float got[8];
                    M::to_floats(p[b][t], got);
#pragma unroll
                    for (int i = 0; i < 8; ++i) s[i] -= got[i];
                }
            }
            __builtin_amdgcn_sched_barrier(0);           // one row tile's temporaries at a time
        }
    }
};

// The finished rows: normalised outputs, or a split's share.
template <class M, int D, Side S>
__device__ __forceinline__ void store_share(const AttnArgs &a, const Rows &r, int hk, int split, int m, int d4, f32x4 o, float mx, float l)
{
    const int mm = r.m0 + m;
    const int64_t t = r.beg + mm / r.G;
    const int h = hk * r.G + mm % r.G;
    if (S == kWhole && a.splits == 1) {
        const float inv = l > 0.0f ? 1.0f / l : 0.0f;
        float x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = o[i] * inv;
        M::store4(static_cast<typename M::T *>(a.o) + t * a.os + (int64_t)h * D + d4, x);
        if (a.lse && d4 == 0) a.lse[t * a.h_q + h] = l > 0.0f ? mx * kLn2 + logf(l) : -INFINITY;
        return;
    }
    const int64_t at = ((int64_t)(S == kWhole ? split : r.part + split) * a.total + t) * a.h_q + h;
    *reinterpret_cast<f32x4 *>(a.part_o + at * D + d4) = o;
    if (d4 == 0) *reinterpret_cast<f32x2 *>(a.part_ml + at * 2) = f32x2{mx, l};
}

// ------------------------------------------------------------- tiles of keys and values in LDS
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
// The factor of the scores, in a scalar register: log2 units, positive (0 becomes a number so small
// that every score is as good as 0).
__device__ __forceinline__ float score_scale(const AttnArgs &a) {
    const float s = fmaxf(fabsf(a.scale) * kLog2e, 1e-30f);
    return __uint_as_float(__builtin_amdgcn_readfirstlane((int)__float_as_uint(s)));
}

// Waits until at most N of the wave's last loads are on their way (they return in order), and until
// all its LDS reads are done.  The compiler counts with these builtins, and no access moves over them.
__device__ __forceinline__ void fence() { asm volatile("" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_loads() {
    fence();
    __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
    fence();
}
__device__ __forceinline__ void wait_reads() {
    fence();
    __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (0 << 8) | (3 << 14));
    fence();
}

// ------------------------------------------------------------- few rows: waves over the keys
// A wave has 32 keys at a time, and a tile of K and one of V of its own: the next keys' K comes in
// from the moment the scores are formed, their V from the moment O is.  No barrier before the join.
// Bound by the reads of K and V, or by latency.  Measured, 16 bf16 query heads on 2 of 256: 64 requests of
// 1K to 32K cached tokens 412 us with the join (8), 2.29 GB at 5.6 TB/s; one of 8K 13.5 us, of
// which the join is 4.2, 17 MB.
template <class M, int D, int NB, int WAVES, Side S>
__global__ void __launch_bounds__(64 * WAVES, D <= 128 ? 2 : 1) decode_kernel(AttnArgs a)
{
    typedef typename M::T T;
    typedef typename M::Frag Frag;
    typedef Tile<M, D> Tl;
    constexpr int ROWS = 16 * NB, KT = 32, RB = Tl::RB, CPR = Tl::CPR;
    constexpr int NI = KT * RB / 1024;                   // 1 KB loads of one tile
    static_assert(16 * D * 4 <= KT * RB, "the join's O, 16 rows at a time, fits where the keys were");
    __shared__ __align__(1024) char Ks[WAVES][KT * RB], Vs[WAVES][KT * RB];
    __shared__ int64_t off[WAVES][2][KT];
    __shared__ float sm[WAVES][16], sl[WAVES][16];
    const int lane = threadIdx.x & 63, g = lane >> 4, col = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (blockIdx.x == 0 && threadIdx.x < 64) check_cu(a.cu, a.n_seqs, a.total, a.status);
    Rows r;
    find_side<S>(a, r);
    const int hk = r.block % a.h_kv;
    const int64_t tile = r.block / a.h_kv / r.splits;
    // turned by the tile's number: a multiple of 8 blocks for each would give all the first splits, which
    // no context is too short for, to the same XCD
    const int split = (int)((r.block / a.h_kv + tile) % r.splits);
    if (!find_rows<S>(a, tile, ROWS, r)) return;
    const int32_t most = S == kShared && r.prefix ? r.kv : row_limit(r, r.m0 + r.count - 1);   // keys that the tile's last row sees
    const int32_t k_beg = (S == kShared ? r.from : 0) + split * r.split_keys;
    if ((S == kShared || split > 0) && k_beg >= most) return;     // nothing here for any row
    const int32_t k_end = most < k_beg + r.split_keys ? most : k_beg + r.split_keys;
    const int32_t *table = a.table + (int64_t)r.n * a.max_pages;
    const char *kc = reinterpret_cast<const char *>(static_cast<const T *>(a.kc) + hk * a.head_stride);
    const char *vc = reinterpret_cast<const char *>(static_cast<const T *>(a.vc) + hk * a.head_stride);
    if (most > 0 && a.n_pages == 0) {
        if (threadIdx.x == 0) set_status(a.status);
        return;
    }
    char *Kw = Ks[wave], *Vw = Vs[wave];
    const uint32_t key_at = Tl::key_lane(lane), value_at = Tl::value_lane(lane);
    const int nt = k_end > k_beg ? (k_end - k_beg + KT - 1) / KT : 0;

    auto key_of = [&](int t) { return find_key(a, table, k_beg + t * KT + (lane & 31), k_end); };
    // (the fences keep the loads in this order: the counts that are waited for below rely on it)
    auto fetch_k = [&](int slot) {
        fence();
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int at = i * 64 + lane, row = at / CPR, pc = at % CPR;
            __builtin_amdgcn_global_load_lds((global_void *)(kc + off[wave][slot][row] + 16 * (pc ^ Tl::sw_k(row))),
                                             (lds_void *)(Kw + i * 1024), 16, 0, 0);
        }
    };
    auto fetch_v = [&](int slot) {
        fence();
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int at = i * 64 + lane, row = at / CPR, pc = at % CPR;
            __builtin_amdgcn_global_load_lds((global_void *)(vc + off[wave][slot][row] + 16 * (pc ^ Tl::sw_v(row))),
                                             (lds_void *)(Vw + i * 1024), 16, 0, 0);
        }
    };
    Key now = {0, 0}, next = {0, 0};
    if (nt > 0) {
        now = key_of(wave);
        next = key_of(wave + WAVES);
    }
    Frag q[NB][D / 32];
    load_q<M, D, NB>(a, r, hk, 0, lane, q);
    if (wave < nt) {
        if (lane < KT) off[wave][0][lane] = key_row(a, now, sizeof(T));
        wave_sync();
        fetch_k(0);
        fetch_v(0);
        wait_loads<(2 * NI < 63 ? 2 * NI : 63)>();       // what is in registers is here
    }
    int32_t lim[NB], least;
    if constexpr (S == kShared) least = shared_limits<NB>(a, r, 0, lane, lim);
    else least = row_limit(r, r.m0);
    auto limit = [&](int b) { return S == kShared ? lim[b] : row_limit(r, r.m0 + 16 * b + col); };
    const float scale = score_scale(a);
    Soft<NB> sf;
    f32x4 o[NB][D / 16];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int d = 0; d < D / 16; ++d) o[b][d] = f32x4{0, 0, 0, 0};

    for (int t = wave, slot = 1; t < nt; t += WAVES, slot ^= 1) {
        const bool more = t + WAVES < nt;
        if (lane < KT) off[wave][slot][lane] = key_row(a, next, sizeof(T));
        wave_sync();
        wait_loads<NI>();                                // K is here; V, the last NI loads, may not be
        next = key_of(t + 2 * WAVES);
        f32x4 st[NB][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int b = 0; b < NB; ++b) st[b][h] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int kb = 0; kb < D / 32; ++kb) {
                const Frag kf = Tl::key(Kw, h, kb, key_at);
#pragma unroll
                for (int b = 0; b < NB; ++b) st[b][h] = M::mma(st[b][h], kf, q[b][kb]);
            }
        }
        wait_reads();                                    // K is read: its place may be filled
        if (more) fetch_k(slot);
        constexpr int TERMS = M::V == 8 ? 2 : 1;         // the products wait for memory: P costs nothing more
        Frag p[NB][TERMS];
        sf.template step<M, D, TERMS>(st, scale, k_beg + t * KT + 4 * g, limit, k_beg + t * KT + KT > least, o, p);
        if (more) wait_loads<NI + 1>();                  // V is here; `next` and the new K may not be
        else wait_loads<0>();
#pragma unroll
        for (int d = 0; d < D / 16; ++d) {
            const Frag vf = Tl::value(Vw, 0, d, value_at);
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int term = TERMS - 1; term >= 0; --term) o[b][d] = M::mma(o[b][d], vf, p[b][term]);
        }
        wait_reads();
        if (more) fetch_v(slot);
    }
    // join the waves, 16 rows at a time: every wave's (m, l, O) to LDS, then one thread per four
    // entries of a row (16-byte piece c of a row sits at c ^ row: the sixteen rows that a wave writes
    // at once are then in different banks)
    float *Os = reinterpret_cast<float *>(Kw);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        float m, sum;
        sf.whole(b, m, sum);
        if (b > 0) __syncthreads();                      // the last rows are read
        if (g == 0) { sm[wave][col] = m; sl[wave][col] = sum; }
#pragma unroll
        for (int d = 0; d < D / 16; ++d)
            *reinterpret_cast<f32x4 *>(Os + col * D + 4 * ((4 * d + g) ^ col)) = o[b][d];
        __syncthreads();
        const int rows = r.count - 16 * b < 16 ? r.count - 16 * b : 16;
        for (int e = threadIdx.x * 4; e < rows * D; e += 64 * WAVES * 4) {
            const int row = e / D, d4 = e % D;
            float mx = sm[0][row];
#pragma unroll
            for (int w = 1; w < WAVES; ++w) mx = fmaxf(mx, sm[w][row]);
            const float base = mx == -INFINITY ? 0.0f : mx;
            f32x4 all = {0, 0, 0, 0};
            float ll = 0.0f;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) {
                const float f = exp2f(sm[w][row] - base);
                all += *reinterpret_cast<const f32x4 *>(reinterpret_cast<const float *>(Ks[w]) + row * D + 4 * ((d4 / 4) ^ row)) * f;
                ll += sl[w][row] * f;
            }
            store_share<M, D, S>(a, r, hk, split, 16 * b + row, d4, all, mx, ll);
        }
    }
}

// ------------------------------------------------------------- many rows: waves over the rows
// KT: keys of a tile.  Two tiles of K and V each: the next one comes in while this one is used, one
// barrier a tile.
// Bound by the matrix products and the softmax beside them.  Measured, 1024 tokens of 16 bf16 query heads
// on 2 of 256 over 31744 cached ones: 485 to 500 us with the join (16), 1080 to 1115 TFLOP/s (a large
// matrix product: 1355), matrix cores 48 % busy; fp32, 9 ragged sequences, 1501 tokens of 16 heads on 4 of 64,
// up to 4000 cached: 133 us, 76 TFLOP/s (153), the join 7.
// TERMS: of P, as in step.  A prefix of 31744 of 64 requests, 8 heads on each of 2 of 256: 55 us with one, 65 with two.
template <class M, int D, int NB, int WAVES, int KT, Side S, int TERMS = 1>
__global__ void __launch_bounds__(64 * WAVES) prefill_kernel(AttnArgs a)
{
    typedef typename M::T T;
    typedef typename M::Frag Frag;
    typedef Tile<M, D> Tl;
    constexpr int PRE = 6 < D / 16 ? 6 : D / 16;
    constexpr int ROWS = 16 * NB * WAVES, RB = Tl::RB, CPR = Tl::CPR;
    constexpr int NI = KT * RB / 1024 / WAVES;           // 1 KB loads of a wave for one tile of K or V
    static_assert(NI >= 1, "a tile has work for every wave");
    __shared__ __align__(1024) char K0[KT * RB], V0[KT * RB], K1[KT * RB], V1[KT * RB];
    __shared__ int64_t off[2][KT];                       // byte offsets of the keys' rows
    const int lane = threadIdx.x & 63, g = lane >> 4, col = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (blockIdx.x == 0 && threadIdx.x < 64) check_cu(a.cu, a.n_seqs, a.total, a.status);
    Rows r;
    find_side<S>(a, r);
    const int hk = r.block % a.h_kv;
    const int64_t tile = r.block / a.h_kv / r.splits;
    if (!find_rows<S>(a, tile, ROWS, r)) return;
    // turned as above: by the sequence's number in bf16, so that the tiles of a sequence keep a split's keys
    // to one XCD; by the tile's in fp32, where only the even spread counts
    const int split = (int)((r.block / a.h_kv + (M::V == 8 ? r.n : tile)) % r.splits);
    const int32_t most = S == kShared && r.prefix ? r.kv : row_limit(r, r.m0 + r.count - 1);
    const int32_t k_beg = (S == kShared ? r.from : 0) + split * r.split_keys;
    if ((S == kShared || split > 0) && k_beg >= most) return;
    const int32_t k_end = most < k_beg + r.split_keys ? most : k_beg + r.split_keys;
    const int32_t *table = a.table + (int64_t)r.n * a.max_pages;
    const char *kc = reinterpret_cast<const char *>(static_cast<const T *>(a.kc) + hk * a.head_stride);
    const char *vc = reinterpret_cast<const char *>(static_cast<const T *>(a.vc) + hk * a.head_stride);
    const int first = wave * 16 * NB;
    const uint32_t key_at = Tl::key_lane(lane), value_at = Tl::value_lane(lane);

    Frag q[NB][D / 32];
    load_q<M, D, NB>(a, r, hk, first, lane, q);
    int32_t lim[NB], least;
    if constexpr (S == kShared) least = shared_limits<NB>(a, r, first, lane, lim);
    else least = row_limit(r, r.m0 + first);
    auto limit = [&](int b) { return S == kShared ? lim[b] : row_limit(r, r.m0 + first + 16 * b + (int)here(col)); };
    const float scale = score_scale(a);
    Soft<NB> sf;
    f32x4 o[NB][D / 16];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int d = 0; d < D / 16; ++d) o[b][d] = f32x4{0, 0, 0, 0};

    const int nt = k_end > k_beg ? (k_end - k_beg + KT - 1) / KT : 0;
    auto key_at_tile = [&](int t) {
        const int32_t j = k_beg + t * KT + (int)threadIdx.x;
        return j < k_end ? j : k_end - 1;
    };
    auto page_of = [&](int t) { return table[key_at_tile(t) / a.page_size]; };
    auto place = [&](int t, int32_t page) { off[t & 1][threadIdx.x] = key_row(a, Key{key_at_tile(t), page}, sizeof(T)); };
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
#pragma unroll 1
        for (int k = 0; k < KT; k += 32) {
            const uint32_t ka = here(key_at), va = here(value_at);
            // The wave whose products are next goes first: two waves of a SIMD then take turns, one's
            // products beside the other's softmax.
            __builtin_amdgcn_s_setprio(2);
            // Operands are read PRE steps ahead of their products.  The scheduling barriers hold the
            // order: short of registers (D = 256) the compiler would wait for each read where it is
            // used, an LDS latency for every two products.
            f32x4 st[NB][2];
            Frag ring[PRE];
#pragma unroll
            for (int i = 0; i < PRE; ++i) ring[i] = Tl::key(Kb, k / 16 + (i & 1), i >> 1, ka);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {           // entries 32 (i / 2) .. of the keys 16 (i % 2) ..
                const int h = i & 1, kb = i >> 1;
#pragma unroll
                for (int b = 0; b < NB; ++b) st[b][h] = M::mma(kb == 0 ? f32x4{0, 0, 0, 0} : st[b][h], ring[i % PRE], q[b][kb]);
                const int n = i + PRE;
                if (n < D / 16) ring[i % PRE] = Tl::key(Kb, k / 16 + (n & 1), n >> 1, ka);
                __builtin_amdgcn_sched_barrier(0);
            }
            __builtin_amdgcn_s_setprio(0);
            Frag p[NB][TERMS];
            sf.template step<M, D, TERMS>(st, scale, k0 + k + 4 * g, limit, k0 + k + 32 > least, o, p);
#pragma unroll
            for (int i = 0; i < PRE; ++i) ring[i] = Tl::value(Vb, k, i, va);
            __builtin_amdgcn_s_setprio(2);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int term = TERMS - 1; term >= 0; --term) o[b][d] = M::mma(o[b][d], ring[d % PRE], p[b][term]);
                if (d + PRE < D / 16) ring[d % PRE] = Tl::value(Vb, k, d + PRE, va);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };
    auto turn = [&](int t, char *Kb, char *Vb, char *Kn, char *Vn) {
        __syncthreads();                                 // this tile is here, the other buffer is free
        const bool ahead = t + 2 < nt && threadIdx.x < KT;
        int32_t page = 0;
        if (ahead) page = page_of(t + 2);
        fence();
        if (t + 1 < nt) stage(t + 1, Kn, Vn);
        compute(t, Kb, Vb);
        if (ahead) place(t + 2, page);
    };
    if (nt > 0) {
        if (a.n_pages == 0) {                            // no page at all: nothing can be read
            if (threadIdx.x == 0) set_status(a.status);
            return;
        }
        if (threadIdx.x < KT) {
            place(0, page_of(0));
            if (nt > 1) place(1, page_of(1));
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
        for (int d = 0; d < D / 16; ++d) store_share<M, D, S>(a, r, hk, split, row, 16 * d + 4 * g, o[b][d], mx, l);
    }
}

// ------------------------------------------------------------- the splits of a row, joined
// A workgroup takes 256 / (D / 4) / SL rows of one token, four entries a thread, and SL slices of a
// row's splits, which meet in LDS in order.  Few splits: one slice, and every thread for itself.
template <class M, int D, int SL, bool SHARED>
__global__ void __launch_bounds__(NT) join_kernel(AttnArgs a)
{
    typedef typename M::T T;
    constexpr int C = D / 4, RW = NT / C / SL;
    __shared__ __align__(16) f32x4 part[SL][RW][C];
    __shared__ float lpart[SL][RW];
    if constexpr (SHARED)                                // the only launch that is never left out
        if (blockIdx.x == 0 && threadIdx.x < 64) {
            check_cu(a.cu, a.n_seqs, a.total, a.status);
            check_groups(a);
        }
    const int blocks = (a.h_q + RW - 1) / RW;            // of one token
    const int64_t t = blockIdx.x / blocks;
    const int c = threadIdx.x % C, rw = threadIdx.x / C % RW, slice = threadIdx.x / C / RW;
    const int h = (int)(blockIdx.x % blocks) * RW + rw;
    const int n = token_sequence(a.cu, a.n_seqs, t);
    const int32_t b = a.cu[n], e = a.cu[n + 1];
    if (!range_ok(b, e, a.total) || t < b || t >= e) return;
    const int32_t kv = a.kv_len[n];
    // (shared: recorded here, for there may be no block of own keys that would)
    if (!kv_ok(kv, a.max_kv, a.page_size, a.max_pages)) {
        if (SHARED && threadIdx.x == 0) set_status(a.status);
        return;
    }
    const int32_t limit = kv - (e - (int32_t)t) + 1;
    // the parts that the row's keys are in: with a prefix its splits, then the row's own behind them
    int act, pre = 0;
    if constexpr (SHARED) {
        int32_t P;
        if (!find_prefix(a, n, kv, P)) {
            if (threadIdx.x == 0) set_status(a.status);
            return;
        }
        const int32_t seen = limit < 0 ? 0 : limit < P ? limit : P;
        pre = (int)(((int64_t)seen + a.prefix_keys - 1) / a.prefix_keys);
        act = pre + (limit > P ? (int)(((int64_t)limit - P + a.split_keys - 1) / a.split_keys) : 0);
    } else {
        act = limit > 0 ? (limit + a.split_keys - 1) / a.split_keys : 1;
    }
    auto part_of = [&](int s) { return SHARED && s >= pre ? a.prefix_splits + s - pre : s; };
    const int64_t step = a.total * a.h_q, row = t * a.h_q + (h < a.h_q ? h : a.h_q - 1);
    const f32x2 *ml = reinterpret_cast<const f32x2 *>(a.part_ml) + row;
    float mx = -INFINITY;
    if (SL > 1) {                                        // a wave is one row's: its lanes share the splits
        for (int s = threadIdx.x & 63; s < act; s += 64) mx = fmaxf(mx, ml[part_of(s) * step].x);
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) mx = fmaxf(mx, __shfl_xor(mx, off));
    } else {
        for (int s = 0; s < act; ++s) mx = fmaxf(mx, ml[part_of(s) * step].x);
    }
    const float base = mx == -INFINITY ? 0.0f : mx;
    float l = 0.0f;
    f32x4 acc = {0, 0, 0, 0};
    const float *p = a.part_o + row * D + 4 * c;
#pragma unroll 4
    for (int s = slice; s < act; s += SL) {
        const int64_t at = part_of(s) * step;
        const f32x2 v = ml[at];
        const float f = exp2f(v.x - base);
        l += v.y * f;
        acc += *reinterpret_cast<const f32x4 *>(p + at * D) * f;
    }
    if (SL > 1) {
        part[slice][rw][c] = acc;
        if (c == 0) lpart[slice][rw] = l;
        __syncthreads();
        if (slice > 0) return;
#pragma unroll
        for (int s = 1; s < SL; ++s) {
            acc += part[s][rw][c];
            l += lpart[s][rw];
        }
    }
    if (h >= a.h_q) return;
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    float x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = acc[i] * inv;
    M::store4(static_cast<T *>(a.o) + t * a.os + (int64_t)h * D + 4 * c, x);
    if (a.lse && c == 0) a.lse[row] = l > 0.0f ? mx * kLn2 + logf(l) : -INFINITY;
}

template <class K>
hipError_t start(K k, int64_t blocks, const AttnArgs &a, hipStream_t stream, int threads)
{
    if (!grid_ok(blocks, threads)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL(k, dim3((unsigned)blocks), dim3(threads), 0, stream, a);
    return hipGetLastError();
}

}  // namespace
}  // namespace gdn
