// The next token of each row of logits: temperature, top-k, top-p and min-p, with a given uniform number.
//
// In the order of falling logits (ties: rising index) a row's tokens have the weights
//     w_i = exp((x_i - max x) / T),
// every filter keeps a first part of that order (the k largest; the shortest whose mass reaches p of what
// top-k keeps; those with w >= min-p), so all of them together keep one, of mass M, and the token is the
// first at which the running mass passes u M.  T = 0: the first token.
//
// No row is sorted.  Where the running mass passes a target is found by its bin first: bin j of a row are
// the tokens with rint(8 x / T) = j, bins of 1/8 in the exponent, of which the 256 from the largest
// logit's down are kept (what lies below has weights under e^-32).  A chunk of a row forms its own bins in
// LDS, counted from its own largest logit: no maximum of the row is needed first, so the logits come from
// memory once.  A second launch joins a row's chunks, scans the bins, and reads the row's tokens of the few
// bins that the borders fall into once more (from the caches), sorts these, and finds the borders in them.
//
// Precision: 8 x / T and exp are taken in 64 bits (which run at the rate of 32 here).  A token's weight
// enters its bin as an integer of units 2^-35 relative to the bin's centre, so that the sums do not depend
// on the order of the atomics.  It is off by half a unit, and by 2^-40 for the series: by e = 1.13 2^-36 of itself at most,
// for it is at least e^(-1/16) of the centre's.  All masses are, so that the mass in front of a border and the mass u M (or
// p M) that it is compared with differ by 2 e M at most from the formula's, 2^-34.8 M: a token next to the true one is taken
// for it only where u (or p) lies within 2^-34 of the border.  The sums of bins and their factors, 2^-50, are beside that.
//
// Bound by instructions and by the latency of dependent steps, not by memory: 64 rows of 131072 fp32 logits (33.5 MB, 7
// us of a large copy) take 11 us in the first launch and some 40 in the second, whose workgroups are one a row and whose
// slowest row counts: 1.4 us for the chunks' heads, 3.5 for their bins, 3 for the borders' bins, 4 to 14 for the tokens
// about them (the whole row's 131072 are looked through where the wanted bins are everywhere in it), 4 for each border
// among few tokens, 9 among thousands.  Spread over more workgroups in a launch of its own, the looking through gained a
// tenth in some large calls and lost as much and more in small ones.
#include "gdn_ops_device.h"

namespace gdn {
namespace {

constexpr int BINS = kSampleBins, NT1 = 256, NT2 = 1024, FEW = 256;
// of the list: one turn's marks, 16 a thread, and the elements outside of a row's whole pieces, at most 7 at either end
constexpr int ENDS = 2 * 7, CAP = NT2 * 16 + ENDS;
constexpr double kUnit = 34359738368.0;                  // 2^35 units: a weight of 1
constexpr float kHighest = 3.402823466e38f;
constexpr uint64_t kMass = (1ull << 49) - 1;             // a chunk's bin: mass below, count from bit 49

struct ChunkHead {
    double top;                 // the bin of the chunk's largest logit
    float max;                  // -inf: the chunk has no token
    int32_t index;              // T = 0: the first token that is the largest
};

// The settings of a row, and whether they are in range.
struct Row {
    double scale;               // 8 / T
    float T, top_p, min_p, u;
    int32_t top_k;
    bool ok;
};
__device__ __forceinline__ Row settings(const SampleArgs &a, int row)
{
    Row r;
    r.T = a.temperature ? a.temperature[row] : 1.0f;
    r.top_p = a.top_p ? a.top_p[row] : 1.0f;
    r.min_p = a.min_p ? a.min_p[row] : 0.0f;
    r.top_k = a.top_k ? a.top_k[row] : 0;
    r.u = a.u[row];
    r.ok = r.T >= 0.0f && r.T <= kHighest && r.top_p > 0.0f && r.top_p <= 1.0f && r.min_p >= 0.0f && r.min_p <= 1.0f &&
           r.u >= 0.0f && r.u < 1.0f && r.top_k >= 0;
    r.scale = 8.0 / (double)r.T;
    return r;
}

// exp(f / 8) in units, |f| <= 1/2, as the low 52 bits of a number of exponent 2^52: the series to the sixth power,
// off by 7.4e-13 = 2^-40 at most.
struct Series {
    double c6 = 1.0 / 188743680.0;                       // 8^-6 / 6!
    double c5 = 1.0 / 3932160.0, c4 = 1.0 / 98304.0, c3 = 1.0 / 6.0 / 512.0, c2 = 1.0 / 128.0, c1 = 1.0 / 8.0;
    double unit = kUnit, exp52 = 4503599627370496.0;
    // In registers, one operand of each product and sum in scalar ones: as constants, every use costs two moves.
    __device__ __forceinline__ void hold()
    {
        asm("" : "+v"(c6), "+s"(c5), "+s"(c4), "+s"(c3), "+s"(c2), "+s"(c1), "+v"(unit), "+s"(exp52));
    }
    __device__ __forceinline__ uint64_t units_bits(double f) const
    {
        double p = fma(c6, f, c5);
        p = fma(p, f, c4);
        p = fma(p, f, c3);
        p = fma(p, f, c2);
        p = fma(p, f, c1);
        p = fma(p, f, 1.0);
        return (uint64_t)__double_as_longlong(fma(p, unit, exp52));
    }
};
constexpr uint64_t kExp52 = 0x4330000000000000ull;       // the bits of 2^52

// Bins so far from 0 that neighbouring values of x are many apart: all tokens of the first 256 are equal.
__device__ __forceinline__ bool is_far(double t) { return fabs(t) > 1125899906842624.0; }     // 2^50
// rint(d scale): in the low bits of the sum with 1.5 2^52, unless it is far.  The bin of a token is found by this alone,
// so that every kernel and pass puts it in the same one.
constexpr double kRound = 6755399441055744.0;
__device__ __forceinline__ double bin_of_logit(double d, double scale, bool far)
{
    return far ? rint(d * scale) : fma(d, scale, kRound) - kRound;
}

// The wave's sums through each lane, by moves between lanes within an instruction (through LDS each step waits for its
// answer).
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t lane_moved(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xf, false);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double lane_moved(double v)
{
    const uint64_t b = (uint64_t)__double_as_longlong(v);
    return __longlong_as_double((long long)((uint64_t)lane_moved<CTRL, ROWS>((uint32_t)(b >> 32)) << 32 | lane_moved<CTRL, ROWS>((uint32_t)b)));
}
template <class V>
__device__ __forceinline__ void scan16(V &v)
{
    v += lane_moved<0x111, 0xf>(v);                      // from 1, 2, 4, 8 lanes below in the 16
    v += lane_moved<0x112, 0xf>(v);
    v += lane_moved<0x114, 0xf>(v);
    v += lane_moved<0x118, 0xf>(v);
}
template <class V>
__device__ __forceinline__ void scan64(V &v)
{
    scan16(v);
    v += lane_moved<0x142, 0xa>(v);                      // the last of the 16 below, to the second and fourth
    v += lane_moved<0x143, 0xc>(v);                      // the last of the first 32, to the others
}
template <class V>
__device__ __forceinline__ V from_below(V v) { return lane_moved<0x138, 0xf>(v); }      // lane 0: zero

// A row's tokens in 16-byte pieces: piece v holds the elements [v V - lead, v V - lead + V), at the row's ends in
// part (rows start anywhere).  Elements that are not the row's are -inf.
template <class E>
struct RowReader {
    typedef typename E::T T;
    const T *base;
    int32_t vocab, lead, whole0, whole1;                 // pieces [whole0, whole1) are whole
    __device__ __forceinline__ RowReader(const SampleArgs &a, int row)
    {
        base = static_cast<const T *>(a.logits) + (int64_t)row * a.stride;
        vocab = a.vocab;
        lead = (int32_t)(((uintptr_t)base & 15) / sizeof(T));
        whole0 = lead ? 1 : 0;
        whole1 = (vocab + lead) / E::V;
    }
    __device__ __forceinline__ int32_t first(int32_t v) const { return v * E::V - lead; }
    __device__ __forceinline__ bool is_whole(int32_t v) const { return v >= whole0 && v < whole1; }
    // any whole piece for one that is not, so that no load waits for a branch (there is one)
    __device__ __forceinline__ u32x4 load(int32_t v) const
    {
        return load16(base + first(v < whole0 ? whole0 : v < whole1 ? v : whole1 - 1));
    }
    __device__ __forceinline__ float one(int32_t i) const { return i >= 0 && i < vocab ? E::one(base + i) : -INFINITY; }
    __device__ __forceinline__ void unpack(int32_t v, u32x4 raw, float *x) const
    {
        E::unpack(raw, x);
        if (!is_whole(v)) {
#pragma unroll
            for (int i = 0; i < E::V; ++i) x[i] = one(first(v) + i);
        }
    }
};

// ------------------------------------------------------------- the chunks' bins
// 19 instructions and an atomic in LDS a token: 256 rows of 131072 bf16 logits (67 MB) 28 us, 2.4 TB/s.
template <class E, int PIECES>
__global__ void __launch_bounds__(NT1) bins_kernel(SampleArgs a)
{
    constexpr int N = PIECES * E::V;                     // elements of a thread
    __shared__ uint64_t bins[BINS + 1];                  // and one that takes what is behind the last
    __shared__ float wmax[NT1 / 64];
    __shared__ int first;
    const int row = blockIdx.x / a.chunks, c = blockIdx.x % a.chunks;
    const RowReader<E> in(a, row);
    const int32_t v0 = c * PIECES * NT1 + (int)threadIdx.x;
    u32x4 raw[PIECES];
#pragma unroll
    for (int i = 0; i < PIECES; ++i) raw[i] = u32x4{0, 0, 0, 0};
    if (in.whole0 < in.whole1)
#pragma unroll
        for (int i = 0; i < PIECES; ++i) raw[i] = in.load(v0 + i * NT1);
    const Row r = settings(a, row);                      // (behind the loads: they do not wait for these)
    if (!r.ok) return;
    float x[N];
#pragma unroll
    for (int i = 0; i < PIECES; ++i) in.unpack(v0 + i * NT1, raw[i], x + i * E::V);
    // NaN loses against any number here, and every comparison below
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < N; ++i) m = fmaxf(m, x[i]);
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off));
    bins[threadIdx.x] = 0;
    if (threadIdx.x == 0) first = 0x7fffffff;
    if ((threadIdx.x & 63) == 0) wmax[threadIdx.x >> 6] = m;
    __syncthreads();
    m = fminf(fmaxf(fmaxf(wmax[0], wmax[1]), fmaxf(wmax[2], wmax[3])), kHighest);
    ChunkHead *head = static_cast<ChunkHead *>(a.heads) + blockIdx.x;
    if (m == -INFINITY) {
        if (threadIdx.x == 0) head->max = m;
        return;
    }
    if (r.T == 0.0f) {
        int at = 0x7fffffff;
#pragma unroll
        for (int i = N - 1; i >= 0; --i)
            if (x[i] >= m) at = in.first(v0 + i / E::V * NT1) + i % E::V;
        if (at != 0x7fffffff) atomicMin(&first, at);
        __syncthreads();
        if (threadIdx.x == 0) {
            head->max = m;
            head->index = first;
        }
        return;
    }
    typedef unsigned long long u64;
    const bool far = is_far((double)m * r.scale);
    const double top = bin_of_logit((double)m, r.scale, far);
    if (far) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (x[i] >= m) atomicAdd(reinterpret_cast<u64 *>(&bins[0]), (u64)((1ull << 49) + (1ull << 35)));
    } else {
        // what lies below has no bin; with min-p and without top-p, which wants the mass of all, what min-p drops
        double below = 33.0 * (double)r.T;
        if (r.min_p > 0.0f && r.top_p >= 1.0f) below = fmin(below, -1.001 * (double)r.T * log((double)r.min_p));
        // (at least the lowest number: beyond that -inf, which is no token, would have a weight)
        const float low = fmaxf((float)((double)m - below - 1e-6 * fabs((double)m)), -kHighest);
        const uint32_t top_bits = (uint32_t)__double_as_longlong(top + kRound);
        Series series;
        double round = kRound;
        series.hold();
        asm("" : "+s"(round));
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (x[i] >= low) {
                const double d = (double)__builtin_amdgcn_fmed3f(x[i], low, kHighest), k = fma(d, r.scale, round);
                const uint32_t at = top_bits - (uint32_t)__double_as_longlong(k);
                atomicAdd(reinterpret_cast<u64 *>(&bins[at < BINS ? at : BINS]),
                          (u64)(series.units_bits(fma(d, r.scale, round - k)) + ((1ull << 49) - kExp52)));
            }
    }
    __syncthreads();
    a.bins[(int64_t)blockIdx.x * BINS + threadIdx.x] = bins[threadIdx.x];
    if (threadIdx.x == 0) {
        head->top = top;
        head->max = m;
    }
}

// ------------------------------------------------------------- a row's token
// Looking for wanted tokens: 4 instructions for two bf16 elements of an interval, 3 for one of fp32.  CAP: all that one
// turn of a workgroup can mark and the row's ends, which the last turn lists too, so that rows with more are looked through
// that much at a time (no list at all: 64 rows of
// 131072 90 us for 44, 256 with filters 222 for 77).  FEW: what one workgroup sorts by counting.
// Where a first part of the order ends: at its count-th token, at the first token through which the mass is at least or
// more than so much, or behind the last token that is not behind `order`.
struct Border {
    enum Kind { kCount, kMass, kPassed, kOrder } kind;
    uint32_t count;
    double mass;
    uint64_t order;
    // whether tokens of so much mass and count together, the last of them not behind `end`, reach it
    __device__ __forceinline__ bool reached(double m, uint32_t c, uint64_t end) const
    {
        return kind == kCount ? c >= count : kind == kMass ? m >= mass : kind == kPassed ? m > mass : end >= order;
    }
};

// What the first wave wants to see next.  All at once: the tokens of the wanted bins.  Else: those of bin j0, or of so much
// of it that a border is in.
struct Plan {
    Border border;
    uint64_t to;                // no token behind this
    double front;               // mass and count in front of the part (-1: all earlier bins')
    uint32_t before;
    uint32_t from[4], width[4]; // the wanted tokens' logits have bits in [from, from + width),
    int intervals;
    int parts;                  // and they are in so many parts of the row
    int j0;
    bool once, listed, done;
};

struct Shared {
    uint64_t list[CAP];         // tokens about the borders, in no order
    uint64_t few[FEW];          // the tokens that are looked at, in order,
    double run[FEW];            // and the row's mass through each of them
    double factor[BINS];        // exp(-j / 8)
    double mass[BINS];          // the row's mass and count through each bin
    uint32_t count[BINS];
    uint64_t has[BINS];         // the parts of the row that have tokens of a bin
    int32_t part[64];           // the parts that have wanted tokens
    uint8_t want[BINS];
    uint64_t sub[NT2];          // units and counts of the bins, then of a bin's parts
    uint32_t subcount[NT2];
    double wsum[NT2 / 64];
    uint32_t wcount[NT2 / 64];
    Plan plan;
    uint32_t n, listed;
};

// A logit's place in the order: smaller is earlier.  And marks of the elements of some pieces whose bits are in
// [from, from + width).
template <class E> struct Marks;
template <> struct Marks<ElemBF16> {
    static constexpr int PIECES = 4, APART = 2;          // (APART: 16 elements)
    static __device__ __forceinline__ uint32_t key(float x)
    {
        const uint32_t b = __float_as_uint(x + 0.0f) >> 16;      // -0 counts as 0
        return b >> 15 ? b : b ^ 0x7fffu;
    }
    static __device__ __forceinline__ float logit(uint32_t key)
    {
        return fminf(__uint_as_float((key >> 15 ? key : key ^ 0x7fffu) << 16), kHighest);
    }
    // the key of the last logit that is x or more
    static __device__ __forceinline__ uint32_t last_key(float x) { return x > 0.0f ? least(x) ^ 0x7fffu : key(x); }
    static constexpr uint32_t SIGN = 0x8000u;
    static __device__ __forceinline__ uint32_t bits(const uint16_t *p) { return *p; }
    // the bits of the least number from x on, and the largest up to x (x >= 0)
    static __device__ __forceinline__ uint32_t least(float x) { return (__float_as_uint(x) + 0xffffu) >> 16; }
    static __device__ __forceinline__ uint32_t most(float x) { return __float_as_uint(x) >> 16; }
    // two elements at a time: their marks are 16 bits apart
    static __device__ __forceinline__ uint32_t mark(const u32x4 *raw, uint32_t from, uint32_t width)
    {
        typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
        const u16x2 f = {(unsigned short)from, (unsigned short)from}, w = {(unsigned short)width, (unsigned short)width};
        const u16x2 one = {1, 1};
        uint32_t marks = 0;
#pragma unroll
        for (int d = 0; d < 4 * PIECES; ++d) {
            const u16x2 x = __builtin_bit_cast(u16x2, (uint32_t)raw[d / 4][d % 4]);
            marks |= __builtin_bit_cast(uint32_t, __builtin_elementwise_min(__builtin_elementwise_sub_sat(w, (u16x2)(x - f)), one)) << d;
        }
        return marks;
    }
    static __device__ __forceinline__ int piece(int mark) { return (mark & 15) >> 2; }
    static __device__ __forceinline__ int element(int mark) { return 2 * (mark & 3) + (mark >> 4); }
    static constexpr __device__ uint32_t of_piece(int i) { return 0x000f000fu << 4 * i; }
};
template <> struct Marks<ElemF32> {
    static constexpr int PIECES = 4, APART = 4;
    static __device__ __forceinline__ uint32_t key(float x)
    {
        const uint32_t b = __float_as_uint(fminf(x, kHighest) + 0.0f);
        return b >> 31 ? b : b ^ 0x7fffffffu;
    }
    static __device__ __forceinline__ float logit(uint32_t key) { return __uint_as_float(key >> 31 ? key : key ^ 0x7fffffffu); }
    static __device__ __forceinline__ uint32_t last_key(float x) { return key(x); }
    static constexpr uint32_t SIGN = 0x80000000u;
    static __device__ __forceinline__ uint32_t bits(const float *p) { return __float_as_uint(*p); }
    static __device__ __forceinline__ uint32_t least(float x) { return __float_as_uint(x); }
    static __device__ __forceinline__ uint32_t most(float x) { return __float_as_uint(x); }
    static __device__ __forceinline__ uint32_t mark(const u32x4 *raw, uint32_t from, uint32_t width)
    {
        uint32_t marks = 0;
#pragma unroll
        for (int d = 4 * PIECES - 1; d >= 0; --d) marks = marks + marks + (uint32_t)(raw[d / 4][d % 4] - from < width);
        return marks;
    }
    static __device__ __forceinline__ int piece(int mark) { return mark >> 2; }
    static __device__ __forceinline__ int element(int mark) { return mark & 3; }
    static constexpr __device__ uint32_t of_piece(int i) { return 0xfu << 4 * i; }
};
template <class E>
constexpr bool apart_fits = Marks<E>::APART * E::V * NT2 + 2 * (E::V - 1) <= CAP && 2 * (E::V - 1) <= 16;
static_assert(apart_fits<ElemBF16> && apart_fits<ElemF32>, "what is listed apart has places, and each of the ends a thread");

template <class E>
struct Picker {
    Shared &s;
    const Row &r;
    const RowReader<E> &in;
    double top;                 // the bin of the row's largest logit
    bool far;
    int group;                  // units of a piece a thread in a part of the row
    int ibits;                  // of an index: the order of a token is its logit's key, and behind that its index
    int n;                      // tokens that are looked at

    __device__ __forceinline__ uint64_t order_of(uint32_t key, int32_t i) const { return (uint64_t)key << ibits | (uint32_t)i; }
    __device__ __forceinline__ int32_t last_index() const { return (int32_t)((1u << ibits) - 1); }
    __device__ __forceinline__ float logit_of(uint64_t o) const { return Marks<E>::logit((uint32_t)(o >> ibits)); }
    __device__ __forceinline__ int32_t index_of(uint64_t o) const { return (int32_t)o & last_index(); }
    __device__ __forceinline__ double through(int j) const { return j < 0 ? 0.0 : s.mass[j]; }
    __device__ __forceinline__ uint32_t counted(int j) const { return j < 0 ? 0u : s.count[j]; }
    __device__ __forceinline__ double below(float x) const { return top - bin_of_logit((double)x, r.scale, far); }
    __device__ __forceinline__ uint64_t weight_units(float x) const
    {
        const double d = (double)x;
        return far ? 1ull << 35 : Series().units_bits(fma(d, r.scale, -bin_of_logit(d, r.scale, false))) - kExp52;
    }
    static __device__ __forceinline__ int some_bin(double b) { return b >= 0.0 && b < (double)BINS ? (int)b : 0; }
    // All logits of the bins [j0, j1] are in [lo, hi], which is little wider.
    __device__ __forceinline__ void span(int j0, int j1, float &lo, float &hi) const
    {
        const double l = (top - j1 - 0.75) / r.scale, h = (top - j0 + 0.75) / r.scale;
        lo = fmaxf((float)(l - fabs(l) * 1e-6), -kHighest);      // (-inf is no token)
        hi = (float)(h + fabs(h) * 1e-6);
        hi = hi >= kHighest ? INFINITY : hi;             // +inf counts as the highest value
    }
    // Lists the tokens of the row whose logits are in the plan's intervals, in no order; `apart`: those of the next 16 elements
    // a thread, from piece `seq` of the parts that have such tokens on.  Whether there is more to list.
    // A workgroup's waves are bound by the instructions here, and code that is not in the instruction cache yet costs more
    // than the tokens.  So a thread first marks the tokens of four pieces, by their bits and without a branch, and writes
    // down where the marked ones are; these are read again, many at a time, when all are known.
    __device__ __forceinline__ bool list_tokens(bool apart, int &seq) const
    {
        typedef Marks<E> M;
        const int step = apart ? M::APART : M::PIECES, intervals = __builtin_amdgcn_readfirstlane(s.plan.intervals);
        const int pieces = in.whole0 < in.whole1 ? __builtin_amdgcn_readfirstlane(s.plan.parts) * group : 0;
        const int part_of = s.part[threadIdx.x & 63];
        const char *from = reinterpret_cast<const char *>(in.base - in.lead);
        const uint32_t per_group = (1u << 20) / (uint32_t)group + 1;       // n per_group >> 20 = n / group, n < 4096 as it is
        auto unit_of = [&](int n, auto part) {
            if (group == 1) return part(n);
            const int q = (int)((uint32_t)n * per_group >> 20);
            return part(q) * group + n - q * group;
        };
        auto load = [&](int at, u32x4 (&raw)[M::PIECES]) {
            uint32_t real = ~0u;
#pragma unroll
            for (int i = 0; i < M::PIECES; ++i) {
                const bool wanted = i < step && at + i < pieces;
                const int unit = unit_of(wanted ? at + i : 0, [&](int q) { return __builtin_amdgcn_readlane(part_of, q); });
                const int32_t v = unit * NT2 + (int)threadIdx.x, last = in.whole1 - 1;
                raw[i] = load16(from + (uint32_t)(v < in.whole0 ? in.whole0 : v < last ? v : last) * 16u);
                if (!wanted || unit == 0 || (unit + 1) * NT2 > in.whole1)        // (else all of the unit's pieces are whole)
                    real &= wanted && in.is_whole(v) ? ~0u : ~M::of_piece(i);
            }
            return real;
        };
        // the row's ends: elements in front of the first whole piece, and behind the last
        const bool any = in.whole0 < in.whole1;
        const int32_t front = any ? in.first(in.whole0) : in.vocab, back = any ? in.first(in.whole1) : in.vocab;
        const int32_t end = (int)threadIdx.x < front ? (int)threadIdx.x : back + (int)threadIdx.x - front;
        uint32_t marks, code, at_end = 0;
        if (threadIdx.x < 16 && end < in.vocab) at_end = Marks<E>::bits(in.base + end);
        auto put = [&] {
            // places for the wave's marks, a lane's behind those of the lanes in front
            uint32_t n = (uint32_t)__popc(marks), to = n;
            scan64(to);
            const uint32_t all = (uint32_t)__builtin_amdgcn_readlane((int)to, 63);
            if (all == 0) return;
            uint32_t first = 0;
            if ((threadIdx.x & 63) == 0) first = atomicAdd(&s.listed, all);
            first = (uint32_t)__builtin_amdgcn_readfirstlane((int)first);
            if (first + all > CAP) return;               // too many
            to += first - n;
#pragma unroll 1
            while (marks) {
                s.list[to++] = code | (uint32_t)__builtin_ctz(marks);
                marks &= marks - 1;
            }
        };
        int at = seq;
        if (at < pieces) {
            u32x4 raw[M::PIECES];
            uint32_t real = load(at, raw);
#pragma unroll 1
            for (;;) {
                u32x4 next[M::PIECES];
                const bool more = !apart && at + step < pieces;
                // (without a branch: behind one, every load would be waited for)
                const uint32_t next_real = load(at + step, next);
                marks = 0;
#pragma unroll 1
                for (int k = 0; k < intervals; ++k)
                    marks |= M::mark(raw, (uint32_t)__builtin_amdgcn_readfirstlane((int)s.plan.from[k]),
                                     (uint32_t)__builtin_amdgcn_readfirstlane((int)s.plan.width[k]));
                marks &= real;
                code = (uint32_t)at << 15 | threadIdx.x << 5;
                put();
                at += step;
                if (!more) break;
                real = next_real;
#pragma unroll
                for (int i = 0; i < M::PIECES; ++i) raw[i] = next[i];
            }
        }
        const bool more = at < pieces;
        if (!more && threadIdx.x < 64) {
            marks = 0;
            for (int k = 0; k < intervals; ++k) marks |= at_end - s.plan.from[k] < s.plan.width[k] ? 1u : 0u;
            if (threadIdx.x >= 16 || end >= in.vocab) marks = 0;
            code = 1u << 31 | threadIdx.x << 5;
            put();
        }
        seq = at;
        __syncthreads();
        const int all = s.listed <= CAP ? (int)s.listed : 0;
#pragma unroll 4
        for (int i = threadIdx.x; i < all; i += NT2) {
            const uint32_t c = (uint32_t)s.list[i];
            const int k = (int)(c & 31), t = (int)(c >> 5 & 1023);
            const int unit = unit_of((int)(c >> 15 & 0xffff) + M::piece(k), [&](int q) { return s.part[q]; });
            const int32_t e = c >> 31 ? (t < front ? t : back + t - front) : in.first(unit * NT2 + t) + M::element(k);
            s.list[i] = order_of(M::key(E::one(in.base + e)), e);
        }
        return more;
    }
    // The passes over the listed tokens, or over the row's, listed 16 elements a thread at a time (one function: its code is read
    // in once):
    enum Mode { kList, kParts, kFew };
    // makes the list; the tokens of the plan's bin from `from` to `to` into 1024 parts, 2^shift orders each; those that the plan
    // wants, into the few.
    __device__ __forceinline__ void pass(Mode mode, bool listed, uint64_t from, uint64_t to, int shift) const
    {
        const bool once = s.plan.once;
        const int j = s.plan.j0;
        int seq = 0;
        bool more = !listed;
#pragma unroll 1
        for (;;) {
            if (more) {
                if (mode != kList) {
                    __syncthreads();
                    if (threadIdx.x == 0) s.listed = 0;
                    __syncthreads();
                }
                more = list_tokens(mode != kList, seq);
                if (mode == kList) return;
            }
            // (a thread takes the tokens that it wrote)
            const int all = s.listed <= CAP ? (int)s.listed : 0;
#pragma unroll 1
            for (int i = threadIdx.x; i < all; i += NT2) {
                const uint64_t o = s.list[i];
                const float x = logit_of(o);
                if (o < from || o > to) continue;
                const double b = below(x);
                if (!(b >= 0.0 && b < (double)BINS) || !(once ? s.want[(int)b] : (int)b == j)) continue;
                if (mode == kParts) {
                    const int p = (int)((o - from) >> shift);
                    atomicAdd(reinterpret_cast<unsigned long long *>(&s.sub[p]), (unsigned long long)weight_units(x));
                    atomicAdd(&s.subcount[p], 1u);
                } else {
                    const uint32_t at = atomicAdd(&s.n, 1u);
                    if (at < FEW) s.few[at] = o;
                }
            }
            if (!more) return;
        }
    }
    // Sums over the workgroup in front of each thread.
    __device__ __forceinline__ void scan(double v, uint32_t c, double &front, uint32_t &cfront) const
    {
        const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
        double t = v;
        uint32_t n = c;
        scan64(t);
        scan64(n);
        if (lane == 63) {
            s.wsum[wave] = t;
            s.wcount[wave] = n;
        }
        front = from_below(t);
        cfront = n - c;
        __syncthreads();
        double all = s.wsum[lane & 15];                  // through wave lane % 16
        uint32_t call = s.wcount[lane & 15];
        scan16(all);
        scan16(call);
        if (wave > 0) {
            front += __shfl(all, wave - 1);
            cfront += (uint32_t)__builtin_amdgcn_readlane((int)call, wave - 1);
        }
    }
    __device__ __forceinline__ double mass_of(float x) const
    {
        return (double)weight_units(x) * (1.0 / kUnit) * s.factor[some_bin(below(x))];
    }
    // The mass that a token brings: its own, and that of the bins in front of it that none of the few is of.
    __device__ __forceinline__ double brings(int i) const
    {
        const float x = logit_of(s.few[i]);
        const double b = below(x);
        double w = mass_of(x);
        if (i == 0) {
            w += s.plan.front >= 0.0 ? s.plan.front : through(some_bin(b) - 1);
        } else {
            const double last = below(logit_of(s.few[i - 1]));
            if (b > last + 1.0) w += through(some_bin(b) - 1) - through(some_bin(last));
        }
        return w;
    }
    // Puts the few in order.  A token's place is the number of earlier ones, which four threads count; then the first wave has
    // the mass through each.
    __device__ __forceinline__ void sort_few()
    {
        n = s.n < FEW ? (int)s.n : FEW;
        const int t = (int)threadIdx.x >> 2, part = (int)threadIdx.x & 3;
        const uint64_t mine = t < n ? s.few[t] : 0;
        int at = 0;
        if ((int)threadIdx.x < 4 * n) {
#pragma unroll 4
            for (int i = part; i < n; i += 4) at += s.few[i] < mine ? 1 : 0;
            at += __shfl_xor(at, 1);
            at += __shfl_xor(at, 2);
        }
        __syncthreads();
        if (part == 0 && t < n) s.few[at] = mine;
        __syncthreads();
        if (threadIdx.x >= 64) return;
        double run = 0.0;
#pragma unroll 1
        for (int i0 = 0; i0 < n; i0 += 64) {
            const int i = i0 + (int)threadIdx.x;
            double w = i < n ? brings(i) : 0.0;
            scan64(w);
            w += run;
            if (i < n) s.run[i] = w;
            run = __shfl(w, 63);
        }
        wave_sync();
    }
    // The few: the tokens that the plan wants, in order.  Of a bin that holds more than FEW, the part that the border is in.
    __device__ __forceinline__ void look(bool make_list, bool &listed)
    {
        const int j = s.plan.j0;
        const bool once = s.plan.once;
        uint64_t from = 0, to = s.plan.to;
        double front = through(j - 1);
        uint32_t before = counted(j - 1), inside = counted(j) - before;
        if (once) inside = 0;
        const bool whole = inside <= FEW;
        if (!whole) {
            float lo, hi;
            span(j, j, lo, hi);
            from = order_of(Marks<E>::key(hi), 0);
            const uint64_t end = order_of(Marks<E>::key(lo), last_index());
            to = end < to ? end : to;
        }
        const double unit = s.factor[j] * (1.0 / kUnit);
        Mode mode = make_list ? kList : inside > FEW ? kParts : kFew;
#pragma unroll 1
        for (;;) {
            const int bits = 64 - __clzll((long long)(to - from)), shift = bits > 10 ? bits - 10 : 0;
            if (mode == kParts) {                        // a 1024th of the range each time
                __syncthreads();
                s.sub[threadIdx.x] = 0;
                s.subcount[threadIdx.x] = 0;
                if (threadIdx.x == 0) s.n = 0xffffffffu;
                __syncthreads();
            }
            pass(mode, listed, from, to, shift);
            __syncthreads();
            if (mode == kFew) break;
            if (mode == kList) {
                listed = s.listed <= CAP;
            } else {
                // whole numbers of units: these sums are exact below 2^53, up to 2^18 tokens in a bin, then to 2^-53
                const double u = (double)s.sub[threadIdx.x];
                const uint32_t c = s.subcount[threadIdx.x];
                double u0;
                uint32_t c0;
                scan(u, c, u0, c0);
                const uint64_t start = from + ((uint64_t)threadIdx.x << shift), end = start + ((1ull << shift) - 1);
                // the first part that reaches the border, else (by rounding) the last that has tokens
                const bool reaches = s.plan.border.reached(front + (u0 + u) * unit, before + c0 + c, end);
                const uint32_t wave0 = threadIdx.x & ~63u;
                const uint64_t here = __ballot(c > 0), there = __ballot(c > 0 && reaches);
                if (threadIdx.x == wave0 && there) atomicMin(&s.n, wave0 + (uint32_t)__builtin_ctzll(there));
                __syncthreads();
                if (s.n == 0xffffffffu) {
                    __syncthreads();
                    if (threadIdx.x == 0) s.n = 0;
                    __syncthreads();
                    if (threadIdx.x == wave0 && here) atomicMax(&s.n, wave0 + 63 - (uint32_t)__builtin_clzll(here));
                    __syncthreads();
                }
                const uint32_t at = s.n;
                if (threadIdx.x == at) {
                    s.wsum[0] = u0;
                    s.wcount[0] = c0;
                }
                __syncthreads();
                front += s.wsum[0] * unit;
                before += s.wcount[0];
                inside = s.subcount[at];
                const uint64_t first = from + ((uint64_t)at << shift), last = first + ((1ull << shift) - 1);
                from = first;
                to = last < to ? last : to;
                if (threadIdx.x == 0) s.n = 0;
                __syncthreads();
            }
            mode = inside > FEW ? kParts : kFew;
        }
        if (threadIdx.x == 0 && !whole) {
            s.plan.front = front;
            s.plan.before = before;
        }
        if (threadIdx.x == 0 && whole) s.plan.before = before;
        sort_few();
    }
    // (by one wave) The first of the few with is(i), which holds from some i on; n if none.
    template <class F>
    __device__ __forceinline__ int first_that(F is) const
    {
        for (int i0 = 0; i0 < n; i0 += 64) {
            const int i = i0 + ((int)threadIdx.x & 63);
            const uint64_t at = __ballot(i < n && is(i < n ? i : 0));
            if (at) return i0 + __ffsll((unsigned long long)at) - 1;
        }
        return n;
    }
    // The mass in front of the few.  There may be none: tokens of a bin that min-p drops are not wanted.
    __device__ __forceinline__ double in_front() const { return s.plan.front >= 0.0 ? s.plan.front : through(s.plan.j0 - 1); }
    __device__ __forceinline__ double mass_at(int i) const { return n == 0 ? in_front() : s.run[i < n ? i : n - 1]; }
};

// The first wave's part: borders, the tokens to look at, and the token.
template <class E>
struct Chooser {
    const Picker<E> &p;
    float m;                    // the row's largest logit
    uint64_t last;              // min-p: the last order that stays
    int jk, jm, step;
    double mk, kept;
    uint32_t ahead;
    bool once, need_k, need_p, need_m, by_p;

    // The bin that a border is in, one that has tokens (the first has: the largest logit).
    __device__ __forceinline__ int bin_of(const Border &b) const
    {
        const int lane = threadIdx.x & 63;
        int mine = BINS;
#pragma unroll
        for (int i = 3; i >= 0; --i) mine = b.reached(p.s.mass[4 * lane + i], p.s.count[4 * lane + i], 0) ? 4 * lane + i : mine;
        const uint64_t at = __ballot(mine < BINS);
        int j = at ? __builtin_amdgcn_readlane(mine, __ffsll((unsigned long long)at) - 1) : BINS - 1;
        while (j > 0 && p.s.count[j] == p.s.count[j - 1]) --j;
        return j;
    }
    __device__ __forceinline__ void start()
    {
        Shared &s = p.s;
        const Row &r = p.r;
        const int lane = threadIdx.x & 63;
        double v = 0.0, mass[4];                         // through the bins 4 lane ..
        uint32_t c = 0, count[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v += (double)s.sub[4 * lane + i] * (1.0 / kUnit) * s.factor[4 * lane + i];
            c += s.subcount[4 * lane + i];
            mass[i] = v;
            count[i] = c;
        }
        scan64(v);
        scan64(c);
        v = from_below(v);
        c = from_below(c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            mass[i] += v;
            count[i] += c;
            s.mass[4 * lane + i] = mass[i];
            s.count[4 * lane + i] = count[i];
        }
        wave_sync();
        // Between which masses each filter's part ends, and the bins that this may be in.  The running mass of
        // the bins carries rounding errors of 2^-50; `slack` covers them.
        const double total = s.mass[BINS - 1], slack = 1e-13;
        last = ~0ull;
        const bool by_k = r.top_k > 0 && (uint32_t)r.top_k < s.count[BINS - 1];
        by_p = r.top_p < 1.0f;
        jk = 0;
        double klo = total, khi = total, plo = total, phi = total, mlo = total, mhi = total;
        if (by_k) {
            jk = bin_of(Border{Border::kCount, (uint32_t)r.top_k, 0.0, 0});
            klo = p.through(jk - 1);
            khi = p.through(jk);
        }
        int jp0 = 0, jp1 = 0;
        if (by_p) {
            jp0 = jp1 = bin_of(Border{Border::kMass, 0, (double)r.top_p * klo * (1.0 - slack), 0});
            const double most = (double)r.top_p * khi * (1.0 + slack);
            if (!(s.mass[jp1] >= most)) jp1 = bin_of(Border{Border::kMass, 0, most, 0});
            plo = p.through(jp0 - 1);
            phi = p.through(jp1);
        }
        jm = 0;
        bool by_m = false;
        if (r.min_p > 0.0f) {                            // w >= min-p: the least logit that stays
            const double least = (double)m + (double)r.T * log((double)r.min_p);
            float x = (float)least + 0.0f;
            if ((double)x < least) x = x < 0.0f ? __uint_as_float(__float_as_uint(x) - 1) : __uint_as_float(__float_as_uint(x) + 1);
            last = p.order_of(Marks<E>::last_key(x), p.last_index());
            const double b = p.top - bin_of_logit(least, r.scale, p.far);
            by_m = b < (double)BINS;
            if (by_m) {
                jm = b > 0.0 ? __builtin_amdgcn_readfirstlane((int)b) : 0;
                mlo = p.through(jm - 1);
                mhi = p.counted(jm) > p.counted(jm - 1) ? p.through(jm) : mlo;      // (sums through empty bins may differ by roundings)
            }
        }
        const double hi = fmin(fmin(khi, phi), mhi), lo = fmin(fmin(klo, plo), mlo);
        need_p = by_p && plo < hi;
        need_m = by_m && mlo < hi;
        need_k = by_k && (klo < hi || need_p);
        const int js0 = bin_of(Border{Border::kPassed, 0, (double)r.u * lo * (1.0 - slack), 0});
        const double most = (double)r.u * hi * (1.0 + slack);
        int js1 = js0;
        if (!(s.mass[js0] > most)) js1 = bin_of(Border{Border::kPassed, 0, most, 0});
        mk = total;
        kept = hi;                                       // (a filter that needs no looking keeps at least hi)
        // One reading of the row for all borders if their bins have not too many tokens, else one for each.
        uint32_t looked = 0, prev = __shfl_up(count[3], 1);
        uint64_t has = 0;
        ahead = 0;
        if (lane == 0) prev = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = 4 * lane + i;
            const bool want = (j >= js0 && j <= js1) || (need_k && j == jk) || (need_p && j >= jp0 && j <= jp1) || (need_m && j == jm);
            s.want[j] = want;
            looked += want ? count[i] - prev : 0;
            ahead += want && j < jk ? count[i] - prev : 0;   // the list's tokens in front of the bin jk
            prev = count[i];
            has |= want ? s.has[j] : 0;
        }
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) {
            looked += __shfl_xor(looked, off);
            ahead += __shfl_xor(ahead, off);
            has |= __shfl_xor(has, off);
        }
        looked = (uint32_t)__builtin_amdgcn_readfirstlane((int)looked);
        if (has >> lane & 1) s.part[__popcll(has & ((1ull << lane) - 1))] = lane;
        once = looked <= FEW;
        step = 0;
        // the bins' logits in two ranges: the token's, and the filters'
        int j0 = BINS, j1 = -1;
        if (need_k) { j0 = jk < j0 ? jk : j0; j1 = jk > j1 ? jk : j1; }
        if (need_p) { j0 = jp0 < j0 ? jp0 : j0; j1 = jp1 > j1 ? jp1 : j1; }
        if (need_m) { j0 = jm < j0 ? jm : j0; j1 = jm > j1 ? jm : j1; }
        const int top0 = j0 < js0 ? j0 : js0, last1 = j1 > js1 ? j1 : js1;
        // one range where the two meet
        const bool meet = j1 < 0 || (j0 <= js1 + 1 && j1 >= js0 - 1);
        int intervals = range(0, meet ? top0 : js0, meet ? last1 : js1);
        if (!meet) intervals = range(intervals, j0, j1);
        if (lane == 0) {
            s.plan.once = once;
            s.plan.parts = __popcll(has);
            s.plan.intervals = intervals;
            s.plan.listed = looked <= CAP * 3 / 4;       // (the ranges hold more)
            s.plan.done = false;
            s.listed = 0;
        }
        if (once) ask(0, Border{Border::kCount, 0, 0.0, 0});
        else next();
    }
    // The bins' logits as intervals of their bits, from number n on: those that are not negative, and the others.
    __device__ __forceinline__ int range(int n, int j0, int j1)
    {
        float lo, hi;
        p.span(j0, j1, lo, hi);
        auto add = [&](uint32_t sign, float a, float b) {        // magnitudes from a to b
            const uint32_t from = Marks<E>::least(a), to = Marks<E>::most(b);
            if (!(a <= b) || from > to) return;
            if ((threadIdx.x & 63) == 0) {
                p.s.plan.from[n] = sign | from;
                p.s.plan.width[n] = to - from + 1;
            }
            ++n;
        };
        if (hi >= 0.0f) add(0, fmaxf(lo, 0.0f), hi);
        if (lo <= 0.0f) add(Marks<E>::SIGN, fmaxf(-hi, 0.0f), -lo);
        return n;
    }
    __device__ __forceinline__ void ask(int j, Border b)
    {
        Shared &s = p.s;
        if ((threadIdx.x & 63) == 0) {
            // without top-p, the bins lack some of what min-p drops: it stays out
            s.plan.border = b;
            s.plan.to = by_p ? ~0ull : last;
            s.plan.front = -1.0;
            s.plan.j0 = j;
            s.n = 0;
        }
    }
    __device__ __forceinline__ bool needed() const { return step == 0 ? need_k : step == 1 ? need_p : step == 2 ? need_m : true; }
    // Asks for the tokens of the next step's bin.
    __device__ __forceinline__ void next()
    {
        while (!needed()) ++step;
        Border b;
        b.kind = step == 0 ? Border::kCount : step == 1 ? Border::kMass : step == 2 ? Border::kOrder : Border::kPassed;
        b.count = (uint32_t)p.r.top_k;
        b.mass = step == 1 ? (double)p.r.top_p * mk : (double)p.r.u * kept;
        b.order = last;
        const int j = step == 0 ? jk : step == 2 ? jm : bin_of(b);
        ask(j, b);
    }
    // Takes a step, or all of them, on the list; the token's place in it, or -1 if there are more steps.
    __device__ __forceinline__ int take()
    {
        Shared &s = p.s;
        for (;; ++step) {
            if (!needed()) continue;
            if (step == 0) {
                // the count-th token: in the list the tokens of the wanted bins in front of its own, and of its own, are before it;
                // where it is none of the few, for min-p drops it, those of its bin that stay
                mk = p.mass_at((int)((uint32_t)p.r.top_k - 1 + (once ? ahead - p.counted(jk - 1) : 0u - s.plan.before)));
                mk = fmax(mk, once ? p.through(jk - 1) : p.in_front());
                kept = fmin(kept, mk);
            } else if (step == 1) {
                const double want = (double)p.r.top_p * mk;
                kept = fmin(kept, p.mass_at(p.first_that([&](int i) { return s.run[i] >= want; })));
            } else if (step == 2) {
                const int end = p.first_that([&](int i) { return s.few[i] > last; });
                kept = fmin(kept, fmax(end > 0 ? p.mass_at(end - 1) : 0.0, once ? p.through(jm - 1) : p.in_front()));
            } else {
                const double want = (double)p.r.u * kept;
                const int at = p.first_that([&](int i) { return s.run[i] > want; });
                return at < p.n ? at : p.n > 0 ? p.n - 1 : 0;
            }
            if (!once) {
                ++step;
                next();
                return -1;
            }
        }
    }
};

template <class E>
__global__ void __launch_bounds__(NT2) pick_kernel(SampleArgs a)
{
    __shared__ Shared s;
    __shared__ float wmax[NT2 / 64];
    __shared__ int first;
    const int row = blockIdx.x, lane = threadIdx.x & 63;
    const ChunkHead *heads = static_cast<const ChunkHead *>(a.heads) + (int64_t)row * a.chunks;
    const ChunkHead mine = heads[(int)threadIdx.x < a.chunks ? threadIdx.x : 0];      // (does not wait for the settings)
    const Row r = settings(a, row);
    if (!r.ok) {
        if (threadIdx.x == 0) {
            set_status(a.status);
            a.token[row] = -1;
            if (a.logprob) a.logprob[row] = -INFINITY;
        }
        return;
    }
    ChunkHead *near = reinterpret_cast<ChunkHead *>(s.list);
    float m = -INFINITY;
    if ((int)threadIdx.x < a.chunks) {                   // the first ones stay at hand
        m = fmaxf(m, mine.max);
        near[threadIdx.x] = mine;
    }
#pragma unroll 1
    for (int c = NT2 + threadIdx.x; c < a.chunks; c += NT2) m = fmaxf(m, heads[c].max);
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off));
    if (lane == 0) wmax[threadIdx.x >> 6] = m;
    if (threadIdx.x == 0) first = 0x7fffffff;
    if (threadIdx.x < BINS) {
        s.sub[threadIdx.x] = 0;
        s.subcount[threadIdx.x] = 0;
        s.has[threadIdx.x] = 0;
        s.factor[threadIdx.x] = exp(-0.125 * (int)threadIdx.x);
    }
    __syncthreads();
    m = wmax[lane & (NT2 / 64 - 1)];
#pragma unroll
    for (int off = 8; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off));
    m = __uint_as_float(__builtin_amdgcn_readfirstlane((int)__float_as_uint(m)));
    if (m == -INFINITY || r.T == 0.0f) {                 // nothing to choose from, or nothing to choose
        if (m != -INFINITY) {
            for (int c = threadIdx.x; c < a.chunks; c += NT2)
                if (heads[c].max == m) atomicMin(&first, heads[c].index);
            __syncthreads();
        }
        if (threadIdx.x == 0) {
            a.token[row] = m == -INFINITY ? -1 : first;
            if (a.logprob) a.logprob[row] = m == -INFINITY ? -INFINITY : 0.0f;
        }
        return;
    }
    const bool far = is_far((double)m * r.scale);
    const double top = bin_of_logit((double)m, r.scale, far);
    const RowReader<E> in(a, row);
    const int units = (in.vocab + in.lead + E::V * NT2 - 1) / (E::V * NT2), group = (units + 63) / 64;
    // the chunks' bins, counted from the row's largest logit
    {
        constexpr int PARTS = NT2 / BINS;
        const int bin = threadIdx.x % BINS;
        const uint64_t *bins = a.bins + (int64_t)row * a.chunks * BINS;
        uint64_t mass = 0, has = 0;
        uint32_t count = 0;
        const int pieces = a.chunk / E::V;               // of a chunk: 256 to 2048
        auto part = [&](int unit) { return 1ull << (group == 1 ? unit : unit / group); };
#pragma unroll 1
        for (int c0 = __builtin_amdgcn_readfirstlane((int)threadIdx.x / BINS); c0 < a.chunks; c0 += 8 * PARTS) {
            uint64_t b[8];
            bool some[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int c = c0 + i * PARTS < a.chunks ? c0 + i * PARTS : c0;
                const ChunkHead h = c < NT2 ? near[c] : heads[c];
                const double off = top - h.top;
                some[i] = c0 + i * PARTS < a.chunks && h.max != -INFINITY && off <= (double)bin;
                b[i] = bins[(int64_t)c * BINS + (some[i] ? bin - (int)off : 0)];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int c = c0 + i * PARTS < a.chunks ? c0 + i * PARTS : c0;
                const uint64_t parts = part(c * pieces / NT2) | part(((c + 1) * pieces - 1) / NT2);
                b[i] = some[i] ? b[i] : 0;
                mass += b[i] & kMass;
                count += (uint32_t)(b[i] >> 49);
                has |= b[i] >> 49 ? parts : 0;
            }
        }
        if (has) atomicOr(reinterpret_cast<unsigned long long *>(&s.has[bin]), (unsigned long long)has);
        atomicAdd(reinterpret_cast<unsigned long long *>(&s.sub[bin]), (unsigned long long)mass);
        atomicAdd(&s.subcount[bin], count);
    }
    Picker<E> p = {s, r, in, top, far, group, 32 - __clz(a.vocab), 0};
    Chooser<E> choose = {p, m};
    const bool chooses = threadIdx.x < 64;
    __syncthreads();
    if (chooses) choose.start();
    __syncthreads();
    bool listed = false;
    for (bool make = s.plan.listed;; make = false) {
        p.look(make, listed);
        if (chooses) {
            const int at = choose.take();
            if (at >= 0 && lane == 0) {
                const uint64_t o = s.few[at];
                a.token[row] = p.index_of(o);
                // by the weight that its mass has: zero where it is the only one
                if (a.logprob) a.logprob[row] = (float)(0.0 - log(choose.kept / p.mass_of(p.logit_of(o))));
                s.plan.done = true;
            }
        }
        __syncthreads();
        if (s.plan.done) return;
    }
}

template <class E>
hipError_t sample_e(const SampleArgs &a, hipStream_t stream)
{
    constexpr int V = E::V;
    const int64_t blocks = (int64_t)a.rows * a.chunks;
    if (!grid_ok(blocks, NT1) || !grid_ok(a.rows, NT2)) return hipErrorInvalidConfiguration;
    if (a.chunk == 2048) hipLaunchKernelGGL((bins_kernel<E, 2048 / NT1 / V>), dim3((unsigned)blocks), dim3(NT1), 0, stream, a);
    else hipLaunchKernelGGL((bins_kernel<E, 8192 / NT1 / V>), dim3((unsigned)blocks), dim3(NT1), 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(pick_kernel<E>, dim3((unsigned)a.rows), dim3(NT2), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_sample(const SampleArgs &a, int bf16, hipStream_t stream)
{
    return bf16 ? sample_e<ElemBF16>(a, stream) : sample_e<ElemF32>(a, stream);
}

}  // namespace gdn
