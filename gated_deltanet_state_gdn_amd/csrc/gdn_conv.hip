// Short causal convolution over packed sequences, one filter per channel, and its
// single-token form:
//     y[t, c] = act(bias[c] + sum_{j < W} w[c, j] x[t - (W - 1) + j, c]),
// with the W - 1 inputs in front of a sequence taken from its state (zero without one), and the
// last W - 1 inputs of the extended sequence as the new state.
//
// Bound by memory: each input is read once and each output written once, 2 W operations per
// channel.  A thread owns one 16-byte vector of channels and TT consecutive tokens of one
// sequence; its window of W inputs slides through registers, so only the W - 1 rows in front of
// a thread's tokens are read twice (from L2, where the neighbouring tile left them).  All TT + W
// - 1 loads are issued before the first use.
// Workgroups are single waves of 512 channels or fewer: those of neighbouring tokens then mostly run on
// the same XCD.  Measured: 16 suffixes, 8200 tokens of 8192 bf16 channels, 270 MB: 61 us, 4.4 TB/s (a
// large copy: 5.0); in workgroups of 128 threads 62, of 256 66 us; 8 tokens a thread 83 us, 24 as 16.  One
// token of 64 requests, fp32: 5.0 us, 17 MB, the length of a launch.
#include "gdn_ops_device.h"

namespace gdn {
namespace {

constexpr int NT = 64;

// y / (1 + e^-y).  fp32: as y (1 or z) / (1 + z) with z = e^-|y|, whose argument is kept in two floats: at most
// 10 halves of a step off down to y = -87, where z passes 2^-126 and is 0 (the form below, 64 at y = -80: the
// argument's rounding grows with |y|).  bf16: with the hardware's exponential and reciprocal alone, 2^-18 off
// there, a 1000th of the output's half step.
template <class E>
__device__ __forceinline__ float act(float y, int silu) {
    if (!silu) return y;
    if constexpr (E::V == 8) {
        return y * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(y * -1.4426950408889634f));
    } else {
        const float z = exp_down(-fabsf(y));
        return (y < 0.0f ? y * z : y) * __builtin_amdgcn_rcpf(1.0f + z);
    }
}

// W taps of V channels, [channels, W] row-major
template <int W, int V>
__device__ __forceinline__ void load_taps(const float *w, const float *bias, int c, float (&tap)[W][V], float (&b)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int j = 0; j < W; ++j) tap[j][i] = w[(int64_t)(c + i) * W + j];
        b[i] = bias ? bias[c + i] : 0.0f;
    }
}

// cols: 16-byte vectors that a block covers (a power of two, at most NT); the block's NT / cols
// groups of threads take TT tokens each.
template <class E, int W, int TT>
__global__ void __launch_bounds__(NT) conv_kernel(ConvArgs a, int cols, uint32_t wide)
{
    typedef typename E::T T;
    constexpr int V = E::V;
    const int64_t bt = blockIdx.x / wide;                     // tile
    if (blockIdx.x == 0 && threadIdx.x < 64) check_cu(a.cu, a.n_seqs, a.total, a.status);
    const int groups = NT / cols, tile = groups * TT;
    const int n = tile_sequence(a.cu, a.n_seqs, bt, 1, tile);
    const int32_t beg = a.cu[n], end = a.cu[n + 1];
    if (!range_ok(beg, end, a.total)) return;                 // recorded by check_cu
    const int64_t k = bt - first_tile(beg, n, 1, tile);
    const int c = ((int)(blockIdx.x % wide) * cols + (threadIdx.x & (cols - 1))) * V;
    if (k < 0 || c >= a.channels) return;
    const T *x = static_cast<const T *>(a.x) + c;
    const T *s0 = a.state0 ? static_cast<const T *>(a.state0) + (int64_t)n * (W - 1) * a.channels + c : nullptr;
    const int group = threadIdx.x / cols;
    const int64_t t0 = beg + k * tile + (int64_t)group * TT;
    const bool keeps = a.state && k == 0 && group == 0;       // this thread writes the new state
    if (t0 >= end && !keeps) return;

    // input at position t of the extended sequence (t >= beg - (W - 1))
    auto input = [&](int64_t t) -> u32x4 {
        if (t >= beg) return load16(x + t * a.xs);
        return s0 ? load16(s0 + (t - beg + (W - 1)) * a.channels) : u32x4{0, 0, 0, 0};
    };
    u32x4 in[TT + W - 1];
#pragma unroll
    for (int i = 0; i < TT + W - 1; ++i) {
        const int64_t t = t0 - (W - 1) + i;
        in[i] = t < end ? input(t) : u32x4{0, 0, 0, 0};
    }
    // The new state, from the thread that also reads the old one: state may be state0's memory.
    if (keeps) {
        u32x4 last[W - 1];
#pragma unroll
        for (int i = 0; i < W - 1; ++i) last[i] = input((int64_t)end - (W - 1) + i);
        T *so = static_cast<T *>(a.state) + (int64_t)n * (W - 1) * a.channels + c;
#pragma unroll
        for (int i = 0; i < W - 1; ++i) store16(so + (int64_t)i * a.channels, last[i]);
    }
    float tap[W][V], b[V];
    load_taps<W, V>(a.w, a.bias, c, tap, b);
    T *y = static_cast<T *>(a.y) + c;
    float win[W][V];                                          // the window, each input unpacked once
#pragma unroll
    for (int i = 0; i < W - 1; ++i) E::unpack(in[i], win[i]);
#pragma unroll
    for (int i = 0; i < TT; ++i) {
        const int64_t t = t0 + i;
        if (t >= end) break;
        E::unpack(in[i + W - 1], win[(i + W - 1) % W]);
        float acc[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            acc[v] = b[v];
#pragma unroll
            for (int j = 0; j < W; ++j) acc[v] = fmaf(tap[j][v], win[(i + j) % W][v], acc[v]);
            acc[v] = act<E>(acc[v], a.silu);
        }
        store16(y + t * a.ys, E::pack(acc));
    }
}

template <class E, int W>
__global__ void __launch_bounds__(64) conv_step_kernel(ConvArgs a, uint32_t wide)
{
    typedef typename E::T T;
    constexpr int V = E::V;
    const int row = blockIdx.x / wide;
    const int slot = slot_of_row(a.slots, row, a.n_slots, a.status);
    const int c = ((int)(blockIdx.x % wide) * 64 + threadIdx.x) * V;
    if (slot < 0 || c >= a.channels) return;
    T *s = static_cast<T *>(a.state) + (int64_t)slot * (W - 1) * a.channels + c;
    u32x4 in[W];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) in[j] = load16(s + (int64_t)j * a.channels);
    in[W - 1] = load16(static_cast<const T *>(a.x) + row * a.xs + c);
    float tap[W][V], acc[V];
    load_taps<W, V>(a.w, a.bias, c, tap, acc);
#pragma unroll
    for (int j = 0; j < W; ++j) {
        float f[V];
        E::unpack(in[j], f);
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] = fmaf(tap[j][v], f[v], acc[v]);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = act<E>(acc[v], a.silu);
    store16(static_cast<T *>(a.y) + row * a.ys + c, E::pack(acc));
#pragma unroll
    for (int j = 0; j < W - 1; ++j) store16(s + (int64_t)j * a.channels, in[j + 1]);
}

template <class E, int W>
hipError_t conv_w(const ConvArgs &a, bool step, hipStream_t stream)
{
    const int vecs = a.channels / E::V;
    if (step) {
        const int64_t wide = (vecs + 63) / 64;
        if (!grid_ok(wide * a.n_seqs, 64)) return hipErrorInvalidConfiguration;
        hipLaunchKernelGGL((conv_step_kernel<E, W>), dim3((unsigned)(wide * a.n_seqs)), dim3(64), 0, stream, a, (uint32_t)wide);
        return hipGetLastError();
    }
    int cols = 1;
    while (cols < vecs && cols < NT) cols *= 2;
    const int64_t wide = (vecs + cols - 1) / cols;
    const int groups = NT / cols;
    auto tiles = [&](int tt) { return a.total / (groups * tt) + a.n_seqs; };
    const bool small = wide * tiles(16) < 512;
    const int64_t n = tiles(small ? 4 : 16) * wide;
    if (!grid_ok(n, NT)) return hipErrorInvalidConfiguration;
    if (small) hipLaunchKernelGGL((conv_kernel<E, W, 4>), dim3((unsigned)n), dim3(NT), 0, stream, a, cols, (uint32_t)wide);
    else hipLaunchKernelGGL((conv_kernel<E, W, 16>), dim3((unsigned)n), dim3(NT), 0, stream, a, cols, (uint32_t)wide);
    return hipGetLastError();
}

template <class E>
hipError_t conv_t(const ConvArgs &a, int width, bool step, hipStream_t stream)
{
    switch (width) {
    case 2: return conv_w<E, 2>(a, step, stream);
    case 3: return conv_w<E, 3>(a, step, stream);
    case 4: return conv_w<E, 4>(a, step, stream);
    default: return hipErrorNotSupported;
    }
}

}  // namespace

hipError_t launch_conv(const ConvArgs &a, int bf16, int width, hipStream_t stream)
{
    return bf16 ? conv_t<ElemBF16>(a, width, false, stream) : conv_t<ElemF32>(a, width, false, stream);
}
hipError_t launch_conv_step(const ConvArgs &a, int bf16, int width, hipStream_t stream)
{
    return bf16 ? conv_t<ElemBF16>(a, width, true, stream) : conv_t<ElemF32>(a, width, true, stream);
}

}  // namespace gdn
