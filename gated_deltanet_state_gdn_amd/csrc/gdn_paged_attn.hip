// Attention of new tokens over a paged cache: launches of the kernels in gdn_attn.h.
#include "gdn_attn.h"

namespace gdn {
namespace {

template <class M, int D, int WAVES>
hipError_t decode_n(const AttnArgs &a, const AttnPlan &p, int64_t blocks, hipStream_t stream)
{
    if (p.rows == 16) return start(decode_kernel<M, D, 1, WAVES, kWhole>, blocks, a, stream, 64 * WAVES);
    if constexpr (M::V == 8 && D != 128) return start(decode_kernel<M, D, 2, WAVES, kWhole>, blocks, a, stream, 64 * WAVES);
    return hipErrorNotSupported;                         // the plan has no such rows
}

template <class M, int D>
hipError_t attn_d(const AttnArgs &a, const AttnPlan &p, hipStream_t stream)
{
    const int G = a.h_q / a.h_kv;
    constexpr int R = NT / (D / 4);                      // rows of a join's workgroup without slices
    // slices where splits are many, or rows few (48 rows of 8 splits: 9.1 us with the attention, 12.0 without)
    const bool sliced = a.splits > 8 || (a.splits > 2 && a.total * a.h_q <= 4096);
    const int64_t blocks = (a.total * G / p.rows + a.n_seqs) * a.splits * a.h_kv;
    const int64_t joins = a.splits == 1 ? 1 : a.total * (sliced ? a.h_q : (a.h_q + R - 1) / R);
    if (!grid_ok(joins, NT)) return hipErrorInvalidConfiguration;
    hipError_t e;
    if (p.decode) {
        constexpr int WAVES = decode_waves(Tile<M, D>::RB);
        if (p.waves == WAVES) e = decode_n<M, D, WAVES>(a, p, blocks, stream);
        else if constexpr (decode_wide(Tile<M, D>::RB)) e = decode_n<M, D, 2 * WAVES>(a, p, blocks, stream);
        else e = hipErrorNotSupported;                   // the plan has no such waves
    } else {
        if constexpr (M::V == 4) e = start(prefill_kernel<M, D, 1, 4, 32, kWhole>, blocks, a, stream, 256);
        else if (p.rows == 256) e = start(prefill_kernel<M, D, 2, 8, 64, kWhole>, blocks, a, stream, 512);
        else e = start(prefill_kernel<M, D, 2, 4, 64, kWhole>, blocks, a, stream, 256);
    }
    if (e != hipSuccess || a.splits == 1) return e;
    if (sliced) return start(join_kernel<M, D, R, false>, joins, a, stream, NT);
    return start(join_kernel<M, D, 1, false>, joins, a, stream, NT);
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

hipError_t launch_attn(const AttnArgs &a, const AttnPlan &p, int bf16, int d, hipStream_t stream)
{
    return bf16 ? attn_m<MfmaBF16>(a, p, d, stream) : attn_m<MfmaF32>(a, p, d, stream);
}

}  // namespace gdn
