// A step's bookkeeping on a paged cache: what follows from the requests' new lengths.
//
// Request n had kv_len[n] cached tokens, or starts behind prefix p = prefix_of[n] with base = prefix_len[p];
// it gets new_len[n] tokens more.  With ps tokens to a page,
//     need_n = ceil((base_n + new_n) / ps) - ceil(base_n / ps),   first_n = free_at + sum_{m < n} need_m,
//     block_table[n, ceil(base_n / ps) + j] = free_pages[first_n + j],   j < need_n,
//     cu[n + 1] = cu[n] + new_n,   token i of n: position base_n + i, slot = page ps + position % ps.
// Scans over the requests, then one entry of the tables or one token a thread.  Nothing but the latency of
// a few dependent loads and of the launches bounds it.  All of a step is checked before any of it is
// written: a step that does not fit takes nothing.
//
// Little work: one workgroup does it all, in LDS (alone_kernel).  Else one workgroup scans and a second launch of
// many fills the tables and slots.
#include "gdn_ops_device.h"

namespace gdn {
namespace {

constexpr int NT = 1024, NA = 256;
constexpr int kAlone = 1024;    // requests, and entries of tables and tokens together, that one workgroup takes alone

// What the first launch leaves for the second.  Per request: its base, the first of its free pages, and its
// table entries in front of it; in the plan's first two words the tokens and entries of all (0: nothing).
struct Request {
    int32_t base, first;
    int64_t entries;
};

__device__ __forceinline__ int32_t pages_of(int64_t tokens, int32_t ps) { return (int32_t)(((uint32_t)tokens + (uint32_t)ps - 1) / (uint32_t)ps); }

struct Wants {
    int32_t base, tokens, need, entries;
    int prefix;                 // -1: none
    bool ok;
};
__device__ __forceinline__ Wants wants(const ExtendArgs &a, int n)
{
    Wants w;
    const int32_t add = a.new_len[n], kv = a.kv_len[n];
    int32_t base = kv;
    w.prefix = a.prefix_of ? a.prefix_of[n] : -1;
    w.ok = add >= 0 && w.prefix >= -1 && w.prefix < a.n_prefixes;
    if (w.ok && w.prefix >= 0) {
        base = a.prefix_len[w.prefix];
        w.ok = base >= 0 && base % a.page_size == 0 && base / a.page_size <= a.max_prefix_pages;
    }
    w.ok = w.ok && base >= 0 && (int64_t)base + add <= 0x7fffffffLL && ((int64_t)base + add + a.page_size - 1) / a.page_size <= a.max_pages;
    if (!w.ok) base = 0;
    w.base = base;
    w.tokens = w.ok ? add : 0;
    w.need = w.ok ? pages_of((int64_t)base + add, a.page_size) - pages_of(base, a.page_size) : 0;
    w.entries = w.need + (w.prefix >= 0 ? base / a.page_size : 0);
    return w;
}

// Sums over the workgroup's threads in front of this one, of three values at once; `all` are the totals.
template <class T>
struct Three {
    T x[3];
};
template <int THREADS, class T>
__device__ __forceinline__ Three<T> scan(Three<T> v, Three<T> &all, Three<T> *part)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    Three<T> s = v;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1)
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const T o = __shfl_up(s.x[i], off);
            if (lane >= off) s.x[i] += o;
        }
    __syncthreads();                                     // the last use of part is over
    if (lane == 63) part[wave] = s;
    __syncthreads();
    all = Three<T>{{0, 0, 0}};
#pragma unroll 2
    for (int w = 0; w < THREADS / 64; ++w) {
        const Three<T> p = part[w];
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            if (w < wave) s.x[i] += p.x[i];
            all.x[i] += p.x[i];
        }
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) s.x[i] -= v.x[i];
    return s;
}

__device__ __forceinline__ Request *requests(const ExtendArgs &a) { return reinterpret_cast<Request *>(a.plan + 2); }

// One entry of a table: entry j of those that request n (base, first free page) gets.
__device__ __forceinline__ void put_entry(const ExtendArgs &a, int n, int32_t base, int32_t first, int32_t j)
{
    const int p = a.prefix_of ? a.prefix_of[n] : -1;
    const int32_t ps = a.page_size, whole = p >= 0 ? base / ps : 0;
    const int32_t page = j < whole ? a.prefix_table[(int64_t)p * a.max_prefix_pages + j] : a.free_pages[first + j - whole];
    a.table[(int64_t)n * a.max_pages + (p >= 0 ? 0 : pages_of(base, ps)) + j] = page;
}
// One token's place: token i of request n.  Its page is an entry from before, or one of the free pages.
__device__ __forceinline__ void put_token(const ExtendArgs &a, int64_t t, int n, int32_t base, int32_t first, int32_t i)
{
    const int32_t ps = a.page_size, pos = base + i, have = pages_of(base, ps), j = pos / ps;
    if (a.positions) a.positions[t] = pos;
    if (!a.slots) return;
    const int32_t page = j < have ? a.table[(int64_t)n * a.max_pages + j] : a.free_pages[first + j - have];
    a.slots[t] = (int64_t)page * ps + pos % ps;
}
__device__ __forceinline__ void put_nothing(const ExtendArgs &a, int64_t t)
{
    if (a.slots) a.slots[t] = -1;
    if (a.positions) a.positions[t] = -1;
}

// Up to kAlone requests, and tokens and table entries together: every sum fits 32 bits, and the scans' results LDS.
// Bound by the latency of its dependent loads and barriers.  64 requests with a token each: 4.2 us; the call 5.6, 8.8 by the
// two launches below; 1000 of them 9.3 and 11.8, and 64 prompts of 900 tokens together 6.6 and 9.5.
__global__ void __launch_bounds__(NA) alone_kernel(ExtendArgs a)
{
    constexpr int PER = kAlone / NA;
    __shared__ Three<int32_t> part[NA / 64];
    __shared__ int32_t cu[kAlone + 1], entries[kAlone + 1], base[kAlone], first[kAlone];
    __shared__ int bad;
    const int32_t at = *a.free_at;
    if (threadIdx.x == 0) bad = 0;
    const int per = (a.n_seqs + NA - 1) / NA, n0 = threadIdx.x * per;
    Wants w[PER];
    Three<int32_t> mine = {{0, 0, 0}}, all;
    bool ok = true;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        w[i] = Wants{};
        if (i < per && n0 + i < a.n_seqs) {
            w[i] = wants(a, n0 + i);
            ok &= w[i].ok & (w[i].tokens <= a.total) & (w[i].need <= kAlone) & (w[i].entries <= 2 * kAlone);
            if (!ok) w[i] = Wants{};
            mine.x[0] += w[i].tokens;
            mine.x[1] += w[i].need;
            mine.x[2] += w[i].entries;
        }
    }
    __syncthreads();
    if (!ok) bad = 1;
    Three<int32_t> s = scan<NA>(mine, all, part);        // (its barriers show `bad` to all)
    const bool fits = !bad && at >= 0 && at <= a.n_free && all.x[0] <= a.total && all.x[1] <= a.n_free - at;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int n = n0 + i;
        if (i >= per || n >= a.n_seqs) continue;
        cu[n] = fits ? s.x[0] : 0;
        entries[n] = s.x[2];
        base[n] = w[i].base;
        first[n] = at + s.x[1];
        a.cu[n] = fits ? s.x[0] : 0;
        if (fits) a.kv_out[n] = w[i].base + w[i].tokens;
        else if (a.kv_out != a.kv_len) a.kv_out[n] = a.kv_len[n];
        s.x[0] += w[i].tokens;
        s.x[1] += w[i].need;
        s.x[2] += w[i].entries;
    }
    if (threadIdx.x == 0) {
        if (!fits) set_status(a.status);
        a.cu[a.n_seqs] = fits ? all.x[0] : 0;
        *a.free_out = fits ? at + all.x[1] : at;
    }
    __syncthreads();
    auto owner = [&](const int32_t *starts, int32_t i) { // the last request that starts at or before i
        int lo = 0, hi = a.n_seqs;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (starts[mid] <= i) lo = mid;
            else hi = mid;
        }
        return lo;
    };
    if (fits)
        for (int e = threadIdx.x; e < all.x[2]; e += NA) {
            const int n = owner(entries, e);
            put_entry(a, n, base[n], first[n], e - entries[n]);
        }
    if (!a.slots && !a.positions) return;
    for (int t = threadIdx.x; t < a.total; t += NA) {
        if (fits && t < all.x[0]) {
            const int n = owner(cu, t);
            put_token(a, t, n, base[n], first[n], t - cu[n]);
        } else {
            put_nothing(a, t);
        }
    }
}

// More than that: the scans, 5.9 us for 700 requests (dependent loads and the barriers of one scan), and behind them the
// tables and slots, 5.5 us for 65536 tokens behind prefixes (0.8 MB written: a launch and the two searches).
__global__ void __launch_bounds__(NT) plan_kernel(ExtendArgs a)
{
    __shared__ Three<int64_t> part[NT / 64];
    __shared__ int bad;
    const int32_t at = *a.free_at;
    if (threadIdx.x == 0) bad = 0;
    __syncthreads();
    // so many neighbouring requests a thread, looked at twice if they are more than one (2000 requests: 13.8 us for 19.6 in
    // rounds of one a thread, with a scan each)
    const int64_t per = ((int64_t)a.n_seqs + NT - 1) / NT, n0 = (int64_t)threadIdx.x * per;
    const int64_t n1 = n0 + per < a.n_seqs ? n0 + per : a.n_seqs;
    Wants w = {};
    Three<int64_t> mine = {{0, 0, 0}}, all;
    bool ok = true;
    for (int64_t n = n0; n < n1; ++n) {
        w = wants(a, (int)n);
        ok &= w.ok;
        mine.x[0] += w.tokens;
        mine.x[1] += w.need;
        mine.x[2] += w.entries;
    }
    if (!ok) bad = 1;
    Three<int64_t> s = scan<NT>(mine, all, part);        // (its barriers show `bad` to all)
    const bool fits = !bad && at >= 0 && at <= a.n_free && all.x[0] <= a.total && all.x[1] <= a.n_free - at;
    Request *req = requests(a);
    for (int64_t n = n0; n < n1; ++n) {
        if (per > 1) w = wants(a, (int)n);
        if (fits) {
            req[n] = Request{w.base, (int32_t)(at + s.x[1]), s.x[2]};
            a.cu[n] = (int32_t)s.x[0];
            a.kv_out[n] = w.base + w.tokens;
        } else {
            a.cu[n] = 0;
            a.kv_out[n] = a.kv_len[n];
        }
        s.x[0] += w.tokens;
        s.x[1] += w.need;
        s.x[2] += w.entries;
    }
    if (threadIdx.x == 0) {
        if (!fits) set_status(a.status);
        a.cu[a.n_seqs] = fits ? (int32_t)all.x[0] : 0;
        *a.free_out = fits ? (int32_t)(at + all.x[1]) : at;
        a.plan[0] = fits ? all.x[0] : 0;
        a.plan[1] = fits ? all.x[2] : 0;
    }
}

// A wave takes 64 neighbouring entries or tokens: the request of the first by a search of 64 candidates a step, those of the
// others among the next 64 requests, whose starts the lanes hold, and by a search where that is not enough.
template <class F>
__device__ __forceinline__ int owner_of_lane(const ExtendArgs &a, int64_t first, int64_t mine, F start)
{
    const int lane = threadIdx.x & 63;
    const int n0 = last_before(a.n_seqs, [&](int n) { return start(n) <= first; });
    const int64_t next = n0 + 1 + lane < a.n_seqs ? start(n0 + 1 + lane) : 0x7fffffffffffffffLL;
    int lo = 0;                                          // requests behind n0 that start at or before mine
#pragma unroll
    for (int step = 32; step >= 1; step >>= 1) lo += __shfl(next, lo + step - 1) <= mine ? step : 0;
    lo += __shfl(next, lo) <= mine ? 1 : 0;
    if (lo < 64) return n0 + lo;
    int from = n0 + 64, to = a.n_seqs;
    while (to - from > 1) {
        const int mid = from + (to - from) / 2;
        if (start(mid) <= mine) from = mid;
        else to = mid;
    }
    return from;
}

__global__ void __launch_bounds__(256) fill_kernel(ExtendArgs a)
{
    const int64_t tokens = a.plan[0], entries = a.plan[1], step = (int64_t)gridDim.x * 256, lane = threadIdx.x & 63;
    const Request *req = requests(a);
    for (int64_t e0 = (int64_t)blockIdx.x * 256 + threadIdx.x - lane; e0 < entries; e0 += step) {
        const int64_t e = e0 + lane;
        const int n = owner_of_lane(a, e0, e, [&](int i) { return req[i].entries; });
        if (e >= entries) continue;
        const Request r = req[n];
        put_entry(a, n, r.base, r.first, (int32_t)(e - r.entries));
    }
    if (!a.slots && !a.positions) return;
    for (int64_t t0 = (int64_t)blockIdx.x * 256 + threadIdx.x - lane; t0 < a.total; t0 += step) {
        const int64_t t = t0 + lane;
        if (t0 >= tokens) {
            if (t < a.total) put_nothing(a, t);
            continue;
        }
        const int n = owner_of_lane(a, t0, t, [&](int i) { return (int64_t)a.cu[i]; });
        if (t < tokens) {
            const Request r = req[n];
            put_token(a, t, n, r.base, r.first, (int32_t)(t - a.cu[n]));
        } else if (t < a.total) {
            put_nothing(a, t);
        }
    }
}

}  // namespace

hipError_t launch_extend(const ExtendArgs &a, hipStream_t stream)
{
    const int64_t prefixes = a.n_prefixes > 0 ? (int64_t)a.n_seqs * (a.max_prefix_pages < a.max_pages ? a.max_prefix_pages : a.max_pages) : 0;
    const int64_t items = a.total + prefixes;
    if (a.n_seqs <= kAlone && items <= kAlone) {
        hipLaunchKernelGGL(alone_kernel, dim3(1), dim3(NA), 0, stream, a);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(plan_kernel, dim3(1), dim3(NT), 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t blocks = (items + a.n_seqs + 255) / 256;
    hipLaunchKernelGGL(fill_kernel, dim3((unsigned)(blocks < 2048 ? blocks : 2048)), dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace gdn
