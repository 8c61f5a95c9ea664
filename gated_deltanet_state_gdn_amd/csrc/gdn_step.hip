// One token of the two recurrences, for many requests at once: every row has a state of its own
// in a pool of slots, read once and written back once.
//     state space:  S <- a S + k (dt v)^T,                 o = S^T q + D v,   a = exp(dt A)
//     gated delta:  S <- a S + k u^T,  u = b (v - a S^T k),  o = scale S^T q,  a = exp(g)
// (k, q, v are B, C, x of a state space layer; the delta form is the gated delta rule's single
// step with S^T k taken before the decay is applied.)
//
// Bound by memory: 8 d_k d_v bytes of state per row and head against d_k + d_v inputs.  The
// columns of S do not mix, so a wave owns 32 columns of one state whole: lane l has columns
// 4 (l % 8) .. + 3 of the d_k / 8 rows of row group l / 8, as float4s.  The sums over d_k run in
// registers and then over three lane exchanges; there is no LDS and no barrier, and all of a
// wave's loads (16 KB of state at d_k = 128) are in flight before the first use.
// Measured: 64 rows of 32 heads, 128 x 64 (state space): 23 us, 135 MB at 5.9 TB/s; 48 rows of 32 heads,
// 128 x 128 (gated delta): 37 us, 203 MB at 5.5 TB/s (a large copy: 5.0; part of the pool stays in the
// last-level cache between calls).
#include "gdn_ops_device.h"

namespace gdn {
namespace {

// Sum over the eight row groups of a wave (lanes l, l ^ 8, l ^ 16, ...).
__device__ __forceinline__ f32x4 sum_groups(f32x4 s) {
#pragma unroll
    for (int off = 8; off < 64; off *= 2)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] += __shfl_xor(s[i], off);
    return s;
}

template <class E, int DK, bool DELTA>
__global__ void __launch_bounds__(256) step_kernel(StepArgs a, int d_v)
{
    typedef typename E::T T;
    constexpr int R = DK / 8;                       // rows of a lane
    const int lane = threadIdx.x & 63;
    const int slices = d_v / 32;
    const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int64_t head_row = w / slices;
    if (head_row >= (int64_t)a.rows * a.h_v) return;
    const int row = (int)(head_row / a.h_v), h = (int)(head_row % a.h_v);
    const int slot = slot_of_row(a.slots, row, a.n_slots, a.status);
    if (slot < 0) return;
    const int c = (int)(w % slices) * 32 + 4 * (lane & 7);
    const int r0 = (lane >> 3) * R;
    float *Sp = a.S + (((int64_t)slot * a.h_v + h) * DK + r0) * d_v + c;

    f32x4 S[R];
#pragma unroll
    for (int i = 0; i < R; ++i) S[i] = *reinterpret_cast<const f32x4 *>(Sp + (int64_t)i * d_v);
    const int hq = h / (a.h_v / a.h_qk);
    const T *kp = static_cast<const T *>(a.k) + row * a.ks + hq * DK + r0;
    const T *qp = static_cast<const T *>(a.q) + row * a.qs + hq * DK + r0;
    float k[R], q[R], v[4];
#pragma unroll
    for (int i = 0; i < R; i += E::V) {
        E::unpack(load16(kp + i), k + i);
        E::unpack(load16(qp + i), q + i);
    }
    const T *vp = static_cast<const T *>(a.v) + row * a.vs + (int64_t)h * d_v + c;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = E::one(vp + i);

    float decay;
    f32x4 u;
    if (DELTA) {
        decay = expf(a.g[(int64_t)row * a.h_v + h]);
        const float beta = a.beta[(int64_t)row * a.h_v + h];
        f32x4 p = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < R; ++i) p += S[i] * k[i];
        p = sum_groups(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = beta * (v[i] - decay * p[i]);
    } else {
        float dt = E::one(static_cast<const T *>(a.dt) + row * a.dts + h) + (a.dt_bias ? a.dt_bias[h] : 0.0f);
        if (a.softplus) dt = softplus(dt);
        decay = expf(dt * a.A[h]);
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = dt * v[i];
    }
    f32x4 o = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            S[i][j] = fmaf(k[i], u[j], decay * S[i][j]);
            o[j] = fmaf(q[i], S[i][j], o[j]);
        }
        *reinterpret_cast<f32x4 *>(Sp + (int64_t)i * d_v) = S[i];
    }
    o = sum_groups(o);
    if (lane >= 8) return;
    const float D = !DELTA && a.D ? a.D[h] : 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = DELTA ? a.scale * o[j] : fmaf(D, v[j], o[j]);
    const int64_t at = row * a.os + (int64_t)h * d_v + c;
    if (E::V == 4 || a.o_f32) *reinterpret_cast<f32x4 *>(static_cast<float *>(a.o) + at) = o;
    else *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(a.o) + at) = u32x2{pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3])};
}

template <class E, bool DELTA>
hipError_t step_e(const StepArgs &a, int d_k, int d_v, hipStream_t stream)
{
    const int64_t blocks = ((int64_t)a.rows * a.h_v * (d_v / 32) + 3) / 4;
    if (!grid_ok(blocks, 256)) return hipErrorInvalidConfiguration;
    if (d_k == 64) hipLaunchKernelGGL((step_kernel<E, 64, DELTA>), dim3((unsigned)blocks), dim3(256), 0, stream, a, d_v);
    else hipLaunchKernelGGL((step_kernel<E, 128, DELTA>), dim3((unsigned)blocks), dim3(256), 0, stream, a, d_v);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_step(const StepArgs &a, int bf16, int d_k, int d_v, bool delta, hipStream_t stream)
{
    if (bf16) return delta ? step_e<ElemBF16, true>(a, d_k, d_v, stream) : step_e<ElemBF16, false>(a, d_k, d_v, stream);
    return delta ? step_e<ElemF32, true>(a, d_k, d_v, stream) : step_e<ElemF32, false>(a, d_k, d_v, stream);
}

}  // namespace gdn
