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
// on the order of the atomics; a bin's mass is off by half a unit a token, 2^-36 of it at most, and by
// less the more tokens it has.  A token of the true border's neighbourhood is taken for it only where u (or
// p) lies that close.
#include "gdn_ops_device.h"

namespace gdn {
namespace {

constexpr int BINS = kSampleBins, NT1 = 256, NT2 = 1024, CAP = 4096;
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

// A logit: NaN is taken as -inf, +inf as the highest value, -0 as 0.
__device__ __forceinline__ float logit(float x) { return x != x ? -INFINITY : fminf(x, kHighest) + 0.0f; }

// exp(f / 8) in units, |f| <= 1/2: the series to the sixth power, off by 7.4e-13 = 2^-40 at most.  `far`: bins so far
// from 0 that a bin is a single value of x; all of them weigh the same.
__device__ __forceinline__ uint64_t units(double f, bool far)
{
    double p = 1.0 / 188743680.0;                        // 8^-6 / 6!
    p = fma(p, f, 1.0 / 3932160.0);
    p = fma(p, f, 1.0 / 98304.0);
    p = fma(p, f, 1.0 / 3072.0);
    p = fma(p, f, 1.0 / 128.0);
    p = fma(p, f, 1.0 / 8.0);
    p = fma(p, f, 1.0);
    // 2^52 + p 2^35, whose last bits are the rounded units
    const uint64_t bits = (uint64_t)__double_as_longlong(fma(p, kUnit, 4503599627370496.0)) & ((1ull << 52) - 1);
    return far ? 1ull << 35 : bits;
}

// A row's tokens in 16-byte pieces: piece v holds the elements [v V - lead, v V - lead + V), whole or at the row's ends in
// part (rows start anywhere).  Elements that are not the row's are -inf.
template <class E>
struct RowReader {
    typedef typename E::T T;
    const T *base;
    int32_t vocab, lead;
    __device__ __forceinline__ RowReader(const SampleArgs &a, int row)
    {
        base = static_cast<const T *>(a.logits) + (int64_t)row * a.stride;
        vocab = a.vocab;
        lead = (int32_t)(((uintptr_t)base & 15) / sizeof(T));
    }
    __device__ __forceinline__ int32_t first(int32_t v) const { return v * E::V - lead; }
    __device__ __forceinline__ int32_t pieces() const { return (vocab + lead + E::V - 1) / E::V; }
    __device__ __forceinline__ void read(int32_t v, float *x) const
    {
        const int32_t i0 = first(v);
        if (i0 >= 0 && i0 + E::V <= vocab) {
            E::unpack(load16(base + i0), x);
#pragma unroll
            for (int i = 0; i < E::V; ++i) x[i] = logit(x[i]);
        } else {
#pragma unroll
            for (int i = 0; i < E::V; ++i) x[i] = i0 + i >= 0 && i0 + i < vocab ? logit(E::one(base + i0 + i)) : -INFINITY;
        }
    }
};

// ------------------------------------------------------------- the chunks' bins
template <class E, int PIECES>
__global__ void __launch_bounds__(NT1) bins_kernel(SampleArgs a)
{
    constexpr int N = PIECES * E::V;                     // elements of a thread
    __shared__ uint64_t bins[BINS];
    __shared__ float wmax[NT1 / 64];
    __shared__ int first;
    const int row = blockIdx.x / a.chunks, c = blockIdx.x % a.chunks;
    const Row r = settings(a, row);
    if (!r.ok) return;
    const RowReader<E> in(a, row);
    float x[N];
#pragma unroll
    for (int i = 0; i < PIECES; ++i) in.read((c * PIECES + i) * NT1 + (int)threadIdx.x, x + i * E::V);
    float m = x[0];
#pragma unroll
    for (int i = 1; i < N; ++i) m = fmaxf(m, x[i]);
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off));
    bins[threadIdx.x] = 0;
    if (threadIdx.x == 0) first = 0x7fffffff;
    if ((threadIdx.x & 63) == 0) wmax[threadIdx.x >> 6] = m;
    __syncthreads();
    m = fmaxf(fmaxf(wmax[0], wmax[1]), fmaxf(wmax[2], wmax[3]));
    ChunkHead *head = static_cast<ChunkHead *>(a.heads) + blockIdx.x;
    if (m == -INFINITY) {
        if (threadIdx.x == 0) head->max = m;
        return;
    }
    if (r.T == 0.0f) {
        int at = 0x7fffffff;
#pragma unroll
        for (int i = N - 1; i >= 0; --i)
            if (x[i] == m) at = in.first((c * PIECES + i / E::V) * NT1 + (int)threadIdx.x) + i % E::V;
        if (at != 0x7fffffff) atomicMin(&first, at);
        __syncthreads();
        if (threadIdx.x == 0) {
            head->max = m;
            head->index = first;
        }
        return;
    }
    const double t0 = (double)m * r.scale, top = rint(t0);
    const bool far = fabs(t0) > 1125899906842624.0;      // 2^50
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const double d = (double)x[i], b = rint(d * r.scale), below = top - b;
        if (below < (double)BINS) atomicAdd(reinterpret_cast<unsigned long long *>(&bins[(int)below]), (unsigned long long)(units(fma(d, r.scale, -b), far) + (1ull << 49)));
    }
    __syncthreads();
    a.bins[(int64_t)blockIdx.x * BINS + threadIdx.x] = bins[threadIdx.x];
    if (threadIdx.x == 0) {
        head->top = top;
        head->max = m;
    }
}

// ------------------------------------------------------------- a row's token
// Tokens in their order: smaller is earlier.
__device__ __forceinline__ uint64_t order_of(float x, int32_t i)
{
    const uint32_t b = __float_as_uint(x);
    return (uint64_t)(b >> 31 ? b : ~b & 0x7fffffffu) << 32 | (uint32_t)i;
}
__device__ __forceinline__ float logit_of(uint64_t o)
{
    const uint32_t k = (uint32_t)(o >> 32);
    return __uint_as_float(k >> 31 ? k : ~k & 0x7fffffffu);
}
__device__ __forceinline__ int32_t index_of(uint64_t o) { return (int32_t)(uint32_t)o; }

// The first i in [lo, hi) with is(i), which holds from some i on; hi if none.
template <class F>
__device__ __forceinline__ int first_that(int lo, int hi, F is)
{
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (is(mid)) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

struct Shared {
    uint64_t list[CAP];         // tokens of the bins that are looked at, in order
    double run[CAP];            // the row's mass through each of them
    double mass[BINS];          // the row's mass through each bin
    uint32_t count[BINS];
    uint64_t sub[NT2];          // units and counts of the bins, then of a bin's parts
    uint32_t subcount[NT2];
    double wsum[NT2 / 64];
    uint32_t n;
};

// Where a first part of the order ends: at its count-th token, at the first token through which the mass is at least or
// more than so much, or behind the last token that is not behind `order`.
struct Border {
    enum Kind { kCount, kMass, kPassed, kOrder } kind;
    double mass;
    uint32_t count;
    uint64_t order;
    // whether tokens of so much mass and count together, the last of them not behind `end`, reach it
    __device__ __forceinline__ bool reached(double m, uint32_t c, uint64_t end) const
    {
        return kind == kCount ? c >= count : kind == kMass ? m >= mass : kind == kPassed ? m > mass : end >= order;
    }
};

template <class E>
struct Picker {
    Shared &s;
    const SampleArgs &a;
    const Row &r;
    RowReader<E> in;
    double top;                 // the bin of the row's largest logit
    bool far;
    double base;                // mass and count in front of the list
    uint32_t before;
    int n;                      // tokens in the list

    __device__ __forceinline__ double through(int j) const { return j < 0 ? 0.0 : s.mass[j]; }
    __device__ __forceinline__ uint32_t counted(int j) const { return j < 0 ? 0u : s.count[j]; }
    __device__ __forceinline__ double below(float x) const { return top - rint((double)x * r.scale); }
    __device__ __forceinline__ uint64_t weight_units(float x) const
    {
        const double d = (double)x;
        return units(fma(d, r.scale, -rint(d * r.scale)), far);
    }
    __device__ __forceinline__ double weight(float x) const
    {
        return (double)weight_units(x) * (1.0 / kUnit) * exp(-0.125 * below(x));
    }

    // All logits of the bins [j0, j1] are in [xlo, xhi], which is little wider.
    __device__ __forceinline__ void span(int j0, int j1, float &xlo, float &xhi) const
    {
        const double lo = (top - j1 - 0.75) / r.scale, hi = (top - j0 + 0.75) / r.scale;
        xlo = (float)(lo - fabs(lo) * 1e-6);
        xhi = fminf((float)(hi + fabs(hi) * 1e-6), kHighest);
    }
    // f(token, logit) for every token of the bins [j0, j1]
    template <class F>
    __device__ __forceinline__ void each(int j0, int j1, F f) const
    {
        float xlo, xhi;                                  // a coarse test in 32 bits in front of the exact one
        span(j0, j1, xlo, xhi);
        const int pieces = in.pieces();
        for (int v = threadIdx.x; v < pieces; v += NT2) {
            float x[E::V];
            in.read(v, x);
#pragma unroll
            for (int i = 0; i < E::V; ++i)
                if (x[i] >= xlo && x[i] <= xhi) {
                    const double b = below(x[i]);
                    if (b >= (double)j0 && b <= (double)j1) f(in.first(v) + i, x[i]);
                }
        }
    }
    // Sums over the workgroup in front of each thread, and of all.
    __device__ __forceinline__ double scan(double v, double &all)
    {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        double t = v;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const double o = __shfl_up(t, off);
            if (lane >= off) t += o;
        }
        __syncthreads();
        if (lane == 63) s.wsum[wave] = t;
        const double in_front = __shfl_up(t, 1);
        __syncthreads();
        double front = 0.0;
        all = 0.0;
#pragma unroll
        for (int w = 0; w < NT2 / 64; ++w) {
            if (w == wave) front = all;
            all += s.wsum[w];
        }
        return front + (lane ? in_front : 0.0);
    }
    // The list: the tokens of the bins [j0, j1] from `from` to `to`, at most CAP, sorted, with the running mass from `mass0`.
    __device__ __forceinline__ void gather(int j0, int j1, uint64_t from, uint64_t to, double mass0, uint32_t count0)
    {
        __syncthreads();
        if (threadIdx.x == 0) s.n = 0;
        __syncthreads();
        each(j0, j1, [&](int32_t i, float x) {
            const uint64_t o = order_of(x, i);
            if (o < from || o > to) return;
            const uint32_t at = atomicAdd(&s.n, 1u);
            if (at < CAP) s.list[at] = o;
        });
        __syncthreads();
        n = s.n < CAP ? (int)s.n : CAP;
        int all = 64;
        while (all < n) all <<= 1;
        for (int i = n + threadIdx.x; i < all; i += NT2) s.list[i] = ~0ull;
        for (int k = 2; k <= all; k <<= 1)
            for (int j = k >> 1; j > 0; j >>= 1) {
                __syncthreads();
                for (int p = threadIdx.x; p < all / 2; p += NT2) {
                    const int i = (p & ~(j - 1)) * 2 + (p & (j - 1)), o = i | j;
                    const uint64_t x = s.list[i], y = s.list[o];
                    if ((x > y) == ((i & k) == 0)) {
                        s.list[i] = y;
                        s.list[o] = x;
                    }
                }
            }
        __syncthreads();
        constexpr int PER = CAP / NT2;
        double w[PER], sum = 0.0, ignored;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int at = threadIdx.x * PER + i;
            w[i] = at < n ? weight(logit_of(s.list[at])) : 0.0;
            sum += w[i];
        }
        double run = mass0 + scan(sum, ignored);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int at = threadIdx.x * PER + i;
            run += w[i];
            if (at < n) s.run[at] = run;
        }
        base = mass0;
        before = count0;
        __syncthreads();
    }
    // The list of a single bin; where it holds more than CAP tokens, of the part of it that the border is in.
    __device__ __forceinline__ void open(int j, const Border &b)
    {
        uint64_t from = 0, to = ~0ull;
        double mass0 = through(j - 1);
        uint32_t count0 = counted(j - 1), inside = counted(j) - count0;
        const double unit = exp(-0.125 * j) * (1.0 / kUnit);
        if (inside > CAP) {
            float xlo, xhi;
            span(j, j, xlo, xhi);
            from = order_of(xhi + 0.0f, 0);
            to = order_of(xlo + 0.0f, -1);
        }
        while (inside > CAP) {                           // a 1024th of the range each time
            const int bits = 64 - __clzll((long long)(to - from)), shift = bits > 10 ? bits - 10 : 0;
            __syncthreads();
            s.sub[threadIdx.x] = 0;
            s.subcount[threadIdx.x] = 0;
            if (threadIdx.x == 0) s.n = 0xffffffffu;
            __syncthreads();
            each(j, j, [&](int32_t i, float x) {
                const uint64_t o = order_of(x, i);
                if (o < from || o > to) return;
                const int p = (int)((o - from) >> shift);
                atomicAdd(reinterpret_cast<unsigned long long *>(&s.sub[p]), (unsigned long long)weight_units(x));
                atomicAdd(&s.subcount[p], 1u);
            });
            __syncthreads();
            // whole numbers below 2^53 and 2^24: these sums are exact
            const double u = (double)s.sub[threadIdx.x], c = (double)s.subcount[threadIdx.x];
            double ignored;
            const double u0 = scan(u, ignored), c0 = scan(c, ignored);
            const uint64_t start = from + ((uint64_t)threadIdx.x << shift), end = start + ((1ull << shift) - 1);
            // the first part that reaches the border, else (by rounding) the last that has tokens
            const bool reaches = b.reached(mass0 + (u0 + u) * unit, count0 + (uint32_t)(c0 + c), end);
            if (c > 0.0 && reaches) atomicMin(&s.n, (uint32_t)threadIdx.x);
            __syncthreads();
            if (s.n == 0xffffffffu) {
                __syncthreads();
                if (threadIdx.x == 0) s.n = 0;
                __syncthreads();
                if (c > 0.0) atomicMax(&s.n, (uint32_t)threadIdx.x);
                __syncthreads();
            }
            const uint32_t at = s.n;
            if (threadIdx.x == at) {
                s.wsum[0] = u0;
                s.wsum[1] = c0;
            }
            __syncthreads();
            mass0 += s.wsum[0] * unit;
            count0 += (uint32_t)s.wsum[1];
            inside = s.subcount[at];
            const uint64_t first = from + ((uint64_t)at << shift), last = first + ((1ull << shift) - 1);
            from = first;
            to = last < to ? last : to;
        }
        gather(j, j, from, to, mass0, count0);
    }
    // Places in the list.
    __device__ __forceinline__ double mass_at(int i) const { return i < 0 ? base : s.run[i < n ? i : n - 1]; }
    // The bin that a border is in, one that has tokens (the first has: the largest logit).
    __device__ __forceinline__ int bin_of(const Border &b) const
    {
        int j = first_that(0, BINS - 1, [&](int i) { return b.reached(s.mass[i], s.count[i], 0); });
        while (j > 0 && s.count[j] == s.count[j - 1]) --j;
        return j;
    }
};

template <class E>
__global__ void __launch_bounds__(NT2) pick_kernel(SampleArgs a)
{
    __shared__ Shared s;
    __shared__ float wmax[NT2 / 64];
    __shared__ int first;
    const int row = blockIdx.x;
    const Row r = settings(a, row);
    if (!r.ok) {
        if (threadIdx.x == 0) {
            set_status(a.status);
            a.token[row] = -1;
            if (a.logprob) a.logprob[row] = -INFINITY;
        }
        return;
    }
    const ChunkHead *heads = static_cast<const ChunkHead *>(a.heads) + (int64_t)row * a.chunks;
    float m = -INFINITY;
    for (int c = threadIdx.x; c < a.chunks; c += NT2) m = fmaxf(m, heads[c].max);
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off));
    if ((threadIdx.x & 63) == 0) wmax[threadIdx.x >> 6] = m;
    if (threadIdx.x == 0) first = 0x7fffffff;
    s.sub[threadIdx.x] = 0;
    if (threadIdx.x < BINS) s.subcount[threadIdx.x] = 0;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NT2 / 64; ++w) m = fmaxf(m, wmax[w]);
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
    const double t0 = (double)m * r.scale, top = rint(t0);
    // the chunks' bins, counted from the row's largest logit
    {
        constexpr int PARTS = NT2 / BINS;
        const int bin = threadIdx.x % BINS;
        uint64_t mass = 0;
        uint32_t count = 0;
        for (int c = threadIdx.x / BINS; c < a.chunks; c += PARTS) {
            const ChunkHead h = heads[c];
            const double off = top - h.top;
            if (h.max == -INFINITY || !(off <= (double)bin)) continue;
            const uint64_t b = a.bins[((int64_t)row * a.chunks + c) * BINS + bin - (int)off];
            mass += b & kMass;
            count += (uint32_t)(b >> 49);
        }
        atomicAdd(reinterpret_cast<unsigned long long *>(&s.sub[bin]), (unsigned long long)mass);
        atomicAdd(&s.subcount[bin], count);
    }
    __syncthreads();
    Picker<E> p = {s, a, r, RowReader<E>(a, row), top, fabs(t0) > 1125899906842624.0, 0.0, 0, 0};
    {
        const bool mine = threadIdx.x < BINS;
        const double v = mine ? (double)s.sub[threadIdx.x] * (1.0 / kUnit) * exp(-0.125 * (int)threadIdx.x) : 0.0;
        const double c = mine ? (double)s.subcount[threadIdx.x] : 0.0;
        double all;
        const double v0 = p.scan(v, all), c0 = p.scan(c, all);
        if (mine) {
            s.mass[threadIdx.x] = v0 + v;
            s.count[threadIdx.x] = (uint32_t)(c0 + c);
        }
    }
    __syncthreads();
    // Between which masses each filter's part ends, and the bins that this may be in.  The running mass of
    // the bins carries rounding errors of 2^-50; `slack` covers them.
    const double total = s.mass[BINS - 1], slack = 1e-13;
    Border k = {Border::kCount, 0.0, (uint32_t)r.top_k, 0}, pm = {Border::kMass, 0.0, 0, 0}, u = {Border::kPassed, 0.0, 0, 0};
    Border f = {Border::kOrder, 0.0, 0, 0};
    const bool by_k = r.top_k > 0 && (uint32_t)r.top_k < s.count[BINS - 1], by_p = r.top_p < 1.0f;
    const int jk = by_k ? p.bin_of(k) : 0;
    const double klo = by_k ? p.through(jk - 1) : total, khi = by_k ? s.mass[jk] : total;
    pm.mass = (double)r.top_p * klo * (1.0 - slack);
    const int jp0 = by_p ? p.bin_of(pm) : 0;
    pm.mass = (double)r.top_p * khi * (1.0 + slack);
    const int jp1 = by_p ? p.bin_of(pm) : 0;
    const double plo = by_p ? p.through(jp0 - 1) : total, phi = by_p ? s.mass[jp1] : total;
    double jm_ = (double)BINS;
    if (r.min_p > 0.0f) {                                // w >= min-p: the least logit that stays
        const double least = (double)m + (double)r.T * log((double)r.min_p);
        float x = (float)least + 0.0f;
        if ((double)x < least) x = x < 0.0f ? __uint_as_float(__float_as_uint(x) - 1) : __uint_as_float(__float_as_uint(x) + 1);
        f.order = order_of(x + 0.0f, -1);
        jm_ = top - rint(least * r.scale);
    }
    const bool by_m = jm_ < (double)BINS;
    const int jm = by_m && jm_ > 0.0 ? (int)jm_ : 0;
    const double mlo = by_m ? p.through(jm - 1) : total, mhi = by_m ? s.mass[jm] : total;
    const double hi = fmin(fmin(khi, phi), mhi), lo = fmin(fmin(klo, plo), mlo);
    const bool need_p = by_p && plo < hi, need_m = by_m && mlo < hi, need_k = by_k && (klo < hi || need_p);
    u.mass = (double)r.u * lo * (1.0 - slack);
    int j0 = p.bin_of(u);
    u.mass = (double)r.u * hi * (1.0 + slack);
    int j1 = p.bin_of(u);
    if (need_k) { j0 = jk < j0 ? jk : j0; j1 = jk > j1 ? jk : j1; }
    if (need_p) { j0 = jp0 < j0 ? jp0 : j0; j1 = jp1 > j1 ? jp1 : j1; }
    if (need_m) { j0 = jm < j0 ? jm : j0; j1 = jm > j1 ? jm : j1; }
    // One reading for all of them if that is not too many tokens, else one for each.
    const bool once = s.count[j1] - p.counted(j0 - 1) <= CAP;
    double mk = total, mass = hi;                        // (a filter that needs no looking keeps at least hi)
    int at = 0;
#pragma unroll 1
    for (int step = once ? -1 : 0; step < 4; ++step) {
        if ((step == 0 && !need_k) || (step == 1 && !need_p) || (step == 2 && !need_m)) continue;
        if (step == 1) pm.mass = (double)r.top_p * mk;
        if (step == 3) u.mass = (double)r.u * mass;
        if (step < 0) {
            p.gather(j0, j1, 0, ~0ull, p.through(j0 - 1), p.counted(j0 - 1));
            continue;
        }
        if (!once) p.open(step == 0 ? jk : step == 1 ? p.bin_of(pm) : step == 2 ? jm : p.bin_of(u), step == 0 ? k : step == 1 ? pm : step == 2 ? f : u);
        if (step == 0) {
            mk = p.mass_at((int)(k.count - 1 - p.before));
            mass = fmin(mass, mk);
        } else if (step == 1) {
            mass = fmin(mass, p.mass_at(first_that(0, p.n, [&](int i) { return s.run[i] >= pm.mass; })));
        } else if (step == 2) {
            mass = fmin(mass, p.mass_at(first_that(0, p.n, [&](int i) { return s.list[i] > f.order; }) - 1));
        } else {
            at = first_that(0, p.n, [&](int i) { return s.run[i] > u.mass; });
            at = at < p.n ? at : p.n - 1;
        }
    }
    if (threadIdx.x == 0) {
        const uint64_t o = s.list[at];
        a.token[row] = index_of(o);
        // masses are relative to the centre of the first bin
        if (a.logprob) a.logprob[row] = (float)((p.far ? 0.0 : 0.125 * fma((double)logit_of(o), r.scale, -top)) - log(mass));
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
