// Norm of q and k per head, position rotation, and the append of k and v to a paged cache, in one
// pass:  q' = rot(q / rms(q) * wq),  k' = rot(k / rms(k) * wk),  rms(x)^2 = mean(x^2) + eps; the
// first `rot` entries of a head turn by the angles of the token's position, in pairs (i, i +
// rot / 2) or (2 i, 2 i + 1); k' and v go to the cache at the token's place.
//
// Bound by memory and, for few tokens, by latency: q, k, v are read once and written once.  D / 8
// lanes hold one head's vector, 8 entries each; the sum of squares runs over those lanes, a pair's
// other half is a lane exchange (rot is a multiple of 16, so it is a whole lane away).  A block
// takes one token, so its sequence and page are found once, and its groups of lanes share the
// token's heads out among them.
// Measured: 1024 tokens of 16 + 2 + 2 bf16 heads of 256: 9.0 us, 21 MB, of which some 5 are the launch and
// the chain sequence - table - place - store; 33 single tokens, fp32: 5.3 us.
#include "gdn_ops_device.h"

namespace gdn {
namespace {

constexpr int NT = 256;

template <int N>
__device__ __forceinline__ void loadf(const float *p, float *f) {
#pragma unroll
    for (int i = 0; i < N; i += 4) ElemF32::unpack(load16(p + i), f + i);
}
// Where the last round of heads ends, for groups of `per` heads taken `per` at a time from any start
__device__ __forceinline__ int first_end(int heads, int per) { return (heads + per - 1) / per * per; }
template <class E>
__device__ __forceinline__ void store8(typename E::T *p, const float *f) {
    store16(p, E::pack(f));
    if (E::V == 4) store16(p + 4, E::pack(f + 4));
}

template <class E, int D, bool INTER>
__global__ void __launch_bounds__(NT) rope_kernel(RopeArgs a)
{
    typedef typename E::T T;
    constexpr int L = D / 8;                       // lanes of one head
    constexpr int MOST = 4;                        // heads that a group of lanes has on their way
    const int64_t t = blockIdx.x;
    if (t == 0 && threadIdx.x < 64) check_cu(a.cu, a.n_seqs, a.total, a.status);
    // the first heads' vectors are asked for before the token's place is looked up
    const int l = threadIdx.x & (L - 1), e0 = 8 * l;
    const int heads = a.h_q + 2 * a.h_kv;
    u32x4 raw[MOST][8 / E::V];
    auto fetch = [&](int h0) {
#pragma unroll
        for (int k = 0; k < MOST; ++k) {
            const int h = h0 + k * (NT / L);
            const int hh = h < heads ? h : heads - 1;
            const T *src = hh < a.h_q ? static_cast<const T *>(a.q) + t * a.qs + (int64_t)hh * D
                         : hh < a.h_q + a.h_kv ? static_cast<const T *>(a.k) + t * a.ks + (int64_t)(hh - a.h_q) * D
                                               : static_cast<const T *>(a.v) + t * a.vs + (int64_t)(hh - a.h_q - a.h_kv) * D;
#pragma unroll
            for (int i = 0; i < 8 / E::V; ++i) raw[k][i] = load16(src + e0 + i * E::V);
        }
    };
    fetch(threadIdx.x / L);
    const int n = token_sequence(a.cu, a.n_seqs, t);
    const int32_t beg = a.cu[n], end = a.cu[n + 1];
    if (!range_ok(beg, end, a.total) || t < beg || t >= end) return;   // bad, or behind the last sequence
    const int32_t kv = a.kv_len[n];
    const int32_t place = kv_ok(kv, a.max_kv, a.page_size, a.max_pages) ? kv - (end - (int32_t)t) : -1;
    const int32_t pos = a.positions ? a.positions[t] : place;
    bool bad = place < 0;
    int64_t cell = -1;
    if (!bad) cell = cache_offset(a.table + (int64_t)n * a.max_pages, place, a.page_size, a.n_pages, a.page_stride, a.token_stride, bad);
    const bool stores = !bad;
    const bool turns = a.rot == 0 || (pos >= 0 && pos < a.max_pos);
    if (threadIdx.x == 0 && !(stores && turns)) set_status(a.status);
    if (!turns) return;

    // the angles of this lane's entries, and the weight of the pair's other half
    const int half = a.rot / 2;
    float c[8], s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) { c[i] = 1.0f; s[i] = 0.0f; }
    if (e0 < a.rot) {
        const float *cs = a.cos_sin + (int64_t)pos * a.rot;
        if (INTER) {                               // entry e is one of pair e / 2
            float cp[4], sp[4];
            loadf<4>(cs + e0 / 2, cp);
            loadf<4>(cs + half + e0 / 2, sp);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                c[i] = cp[i / 2];
                s[i] = i & 1 ? sp[i / 2] : -sp[i / 2];
            }
        } else {                                   // entries e and e + half are pair e
            const int f = e0 < half ? e0 : e0 - half;
            loadf<8>(cs + f, c);
            loadf<8>(cs + half + f, s);
#pragma unroll
            for (int i = 0; i < 8; ++i) s[i] = e0 < half ? -s[i] : s[i];
        }
    }
    const int other = INTER ? l : e0 < half ? l + half / 8 : e0 < a.rot ? l - half / 8 : l;
    const int lane = threadIdx.x & 63;
    const int from = (lane & ~(L - 1)) + other;

    cell += e0;
    float wq[8], wk[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) { wq[i] = 1.0f; wk[i] = 1.0f; }
    if (a.qw) loadf<8>(a.qw + e0, wq);
    if (a.kw) loadf<8>(a.kw + e0, wk);
    // every group of lanes goes round equally often: the exchanges are between all lanes
    for (int h0 = threadIdx.x / L; h0 < first_end(heads, NT / L); h0 += MOST * (NT / L)) {
        if (h0 >= MOST * (NT / L)) fetch(h0);
#pragma unroll
        for (int k = 0; k < MOST; ++k) {
            const int h = h0 + k * (NT / L);
            const bool is_q = h < a.h_q, is_k = !is_q && h < a.h_q + a.h_kv;
            const int hk = is_q ? h : is_k ? h - a.h_q : h - a.h_q - a.h_kv;
            float x[8], y[8], z[8];
            E::unpack(raw[k][0], x);
            if (E::V == 4) E::unpack(raw[k][E::V == 4], x + 4);
            float inv = 1.0f;
            if (a.norm) {
                float ss = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
                for (int off = 1; off < L; off *= 2) ss += __shfl_xor(ss, off);
                inv = 1.0f / sqrtf(ss * (1.0f / D) + a.eps);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = x[i] * inv * (is_q ? wq[i] : wk[i]);
#pragma unroll
            for (int i = 0; i < 8; ++i) z[i] = INTER ? y[i ^ 1] : __shfl(y[i], from);
#pragma unroll
            for (int i = 0; i < 8; ++i) z[i] = e0 < a.rot ? fmaf(y[i], c[i], z[i] * s[i]) : y[i];
            if (h >= heads) continue;
            if (is_q) store8<E>(static_cast<T *>(a.qo) + t * a.qos + (int64_t)hk * D + e0, z);
            else if (stores && is_k) store8<E>(static_cast<T *>(a.kc) + cell + hk * a.head_stride, z);
            else if (stores) store8<E>(static_cast<T *>(a.vc) + cell + hk * a.head_stride, x);
        }
    }
}

template <class E, bool INTER>
hipError_t rope_e(const RopeArgs &a, int d, hipStream_t stream)
{
    if (!grid_ok(a.total, NT)) return hipErrorInvalidConfiguration;
    const dim3 grid((unsigned)a.total);
    switch (d) {
    case 64: hipLaunchKernelGGL((rope_kernel<E, 64, INTER>), grid, dim3(NT), 0, stream, a); break;
    case 128: hipLaunchKernelGGL((rope_kernel<E, 128, INTER>), grid, dim3(NT), 0, stream, a); break;
    case 256: hipLaunchKernelGGL((rope_kernel<E, 256, INTER>), grid, dim3(NT), 0, stream, a); break;
    default: return hipErrorNotSupported;
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rope(const RopeArgs &a, int bf16, int d, bool interleaved, hipStream_t stream)
{
    if (bf16) return interleaved ? rope_e<ElemBF16, true>(a, d, stream) : rope_e<ElemBF16, false>(a, d, stream);
    return interleaved ? rope_e<ElemF32, true>(a, d, stream) : rope_e<ElemF32, false>(a, d, stream);
}

}  // namespace gdn
