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
// One workgroup scans; where the rest is little it does that too, else a second launch of many does.
#include "gdn_ops_device.h"

namespace gdn {
namespace {

constexpr int NT = 1024;

// What the first launch leaves for the second.  Per request: its base, the first of its free pages, and its
// table entries in front of it; in the plan's first two words the tokens and entries of all (0: nothing).
struct Request {
    int32_t base, first;
    int64_t entries;
};

__device__ __forceinline__ int32_t pages_of(int64_t tokens, int32_t ps) { return (int32_t)((tokens + ps - 1) / ps); }

struct Wants {
    int64_t base, tokens, need, entries;
    int prefix;                 // -1: none
    bool ok;
};
__device__ __forceinline__ Wants wants(const ExtendArgs &a, int n)
{
    Wants w;
    const int32_t add = a.new_len[n];
    int32_t base = a.kv_len[n];
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
struct Three {
    int64_t x[3];
};
__device__ __forceinline__ Three scan(Three v, Three &all, Three *part)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    Three s = v;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1)
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const int64_t o = __shfl_up(s.x[i], off);
            if (lane >= off) s.x[i] += o;
        }
    __syncthreads();                                     // the last use of part is over
    if (lane == 63) part[wave] = s;
    __syncthreads();
    all = Three{{0, 0, 0}};
#pragma unroll 2
    for (int w = 0; w < NT / 64; ++w) {
        const Three p = part[w];
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

// The request that owns token t or entry e: the last whose start is not behind it.  before(n): its start.
template <class F>
__device__ __forceinline__ int owner(int lo, int hi, F before)
{
    while (hi - lo > 1) {
        const int mid = lo + (hi - lo) / 2;
        if (before(mid)) lo = mid;
        else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ void fill(const ExtendArgs &a, int64_t at, int64_t step, int64_t tokens, int64_t entries)
{
    const Request *req = requests(a);
    const int32_t ps = a.page_size;
    for (int64_t e = at; e < entries; e += step) {
        const int n = owner(0, a.n_seqs, [&](int i) { return req[i].entries <= e; });
        const Request r = req[n];
        const int p = a.prefix_of ? a.prefix_of[n] : -1;
        const int32_t j = (int32_t)(e - r.entries), whole = p >= 0 ? r.base / ps : 0;
        const int32_t page = j < whole ? a.prefix_table[(int64_t)p * a.max_prefix_pages + j] : a.free_pages[r.first + j - whole];
        a.table[(int64_t)n * a.max_pages + (p >= 0 ? 0 : pages_of(r.base, ps)) + j] = page;
    }
    if (!a.slots && !a.positions) return;
    for (int64_t t = at; t < a.total; t += step) {
        int64_t slot = -1;
        int32_t pos = -1;
        if (t < tokens) {
            const int n = owner(0, a.n_seqs, [&](int i) { return a.cu[i] <= t; });
            const Request r = req[n];
            pos = r.base + (int32_t)(t - a.cu[n]);
            const int32_t have = pages_of(r.base, ps), j = pos / ps;
            const int32_t page = j < have ? a.table[(int64_t)n * a.max_pages + j] : a.free_pages[r.first + j - have];
            slot = (int64_t)page * ps + pos % ps;
        }
        if (a.slots) a.slots[t] = slot;
        if (a.positions) a.positions[t] = pos;
    }
}

template <bool ALONE>
__global__ void __launch_bounds__(NT) plan_kernel(ExtendArgs a)
{
    __shared__ Three part[NT / 64];
    __shared__ int bad;
    const int32_t at = *a.free_at;
    if (threadIdx.x == 0) bad = 0;
    __syncthreads();
    Three all = {{0, 0, 0}};
    {
        Three mine = {{0, 0, 0}};
        bool ok = true;
        for (int n = threadIdx.x; n < a.n_seqs; n += NT) {
            const Wants w = wants(a, n);
            ok &= w.ok;
            mine.x[0] += w.tokens;
            mine.x[1] += w.need;
            mine.x[2] += w.entries;
        }
        if (!ok) bad = 1;
        scan(mine, all, part);
    }
    const bool fits = !bad && at >= 0 && at <= a.n_free && all.x[0] <= a.total && all.x[1] <= a.n_free - at;
    Three done = {{0, 0, 0}};
    Request *req = requests(a);
    for (int n0 = 0; n0 < a.n_seqs; n0 += NT) {
        const int n = n0 + threadIdx.x;
        Wants w = {};
        if (n < a.n_seqs && fits) w = wants(a, n);
        Three sum;
        const Three s = scan(Three{{w.tokens, w.need, w.entries}}, sum, part);
        if (n < a.n_seqs) {
            req[n] = Request{(int32_t)w.base, (int32_t)(at + done.x[1] + s.x[1]), done.x[2] + s.x[2]};
            a.cu[n] = (int32_t)(done.x[0] + s.x[0]);
            a.kv_out[n] = fits ? (int32_t)(w.base + w.tokens) : a.kv_len[n];
        }
#pragma unroll
        for (int i = 0; i < 3; ++i) done.x[i] += sum.x[i];
    }
    if (threadIdx.x == 0) {
        if (!fits) set_status(a.status);
        a.cu[a.n_seqs] = (int32_t)done.x[0];
        *a.free_out = fits ? (int32_t)(at + done.x[1]) : at;
        a.plan[0] = done.x[0];
        a.plan[1] = done.x[2];
    }
    if constexpr (ALONE) {
        __syncthreads();                                 // (the barrier makes the workgroup's stores visible in it)
        fill(a, threadIdx.x, NT, done.x[0], done.x[2]);
    }
}

__global__ void __launch_bounds__(256) fill_kernel(ExtendArgs a)
{
    fill(a, (int64_t)blockIdx.x * 256 + threadIdx.x, (int64_t)gridDim.x * 256, a.plan[0], a.plan[1]);
}

}  // namespace

hipError_t launch_extend(const ExtendArgs &a, hipStream_t stream)
{
    const int64_t prefixes = a.n_prefixes > 0 ? (int64_t)a.n_seqs * (a.max_prefix_pages < a.max_pages ? a.max_prefix_pages : a.max_pages) : 0;
    const int64_t items = a.total + prefixes;
    if (items <= 4096) {
        hipLaunchKernelGGL(plan_kernel<true>, dim3(1), dim3(NT), 0, stream, a);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(plan_kernel<false>, dim3(1), dim3(NT), 0, stream, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t blocks = (items + 255) / 256;
    hipLaunchKernelGGL(fill_kernel, dim3((unsigned)(blocks < 2048 ? blocks : 2048)), dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace gdn
