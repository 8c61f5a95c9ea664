// Attention over a paged cache for groups of sequences that share a prefix.
//
// The sequences of group g hold the same keys and values in their first P = prefix_len[g] tokens.  A row
// at position p then attends to the prefix's keys [0, min(P, p + 1)), which are the same for every row
// of the group, and to its sequence's own [P, p]:
//     m = max(m1, m2),  l = l1 e^(m1 - m) + l2 e^(m2 - m),  o = (O1 e^(m1 - m) + O2 e^(m2 - m)) / l,
// (O, m, l) the unnormalised output, maximum and sum over either side.  Prefix: the rows of the whole
// group, tokens times query heads on a cache head, are the rows of one product over the keys that the
// first sequence's block table names, so the prefix is read once for as many rows as a workgroup holds
// instead of once a sequence.  Own: as in attention without groups, from key P on.  Then the join of
// both sides' splits.  Kernels: gdn_attn.h.
#include "gdn_attn.h"

namespace gdn {
namespace {

template <class M, int D, int WAVES, Side S>
hipError_t decode_n(const AttnArgs &a, const AttnPlan &p, int64_t blocks, hipStream_t stream)
{
    if (p.rows == 16) return start(decode_kernel<M, D, 1, WAVES, S>, blocks, a, stream, 64 * WAVES);
    if constexpr (M::V == 8 && D != 128) return start(decode_kernel<M, D, 2, WAVES, S>, blocks, a, stream, 64 * WAVES);
    return hipErrorNotSupported;                         // the plan has no such rows
}

template <class M, int D, Side S>
hipError_t side(AttnArgs a, const AttnPlan &p, int32_t units, int32_t part_first, hipStream_t stream)
{
    a.splits = p.splits;
    a.split_keys = p.split_keys;
    a.part_first = part_first;
    const int64_t blocks = (a.total * (a.h_q / a.h_kv) / p.rows + units) * a.splits * a.h_kv;
    if (p.decode) {
        constexpr int WAVES = decode_waves(Tile<M, D>::RB);
        if (p.waves == WAVES) return decode_n<M, D, WAVES, S>(a, p, blocks, stream);
        if constexpr (decode_wide(Tile<M, D>::RB)) return decode_n<M, D, 2 * WAVES, S>(a, p, blocks, stream);
        return hipErrorNotSupported;                     // the plan has no such waves
    }
    if constexpr (M::V == 4) return start(prefill_kernel<M, D, 1, 4, 32, S>, blocks, a, stream, 256);
    else if (p.rows == 256) return start(prefill_kernel<M, D, 2, 8, 64, S>, blocks, a, stream, 512);
    else return start(prefill_kernel<M, D, 2, 4, 64, S>, blocks, a, stream, 256);
}

template <class M, int D>
hipError_t shared_d(AttnArgs a, const SharedPlan &p, hipStream_t stream)
{
    constexpr int R = NT / (D / 4);                      // rows of a join's workgroup without slices
    const int splits = p.prefix.splits + p.own.splits;
    const bool sliced = splits > 8 || (splits > 2 && a.total * a.h_q <= 4096);
    const int64_t joins = a.total * (sliced ? a.h_q : (a.h_q + R - 1) / R);
    const int64_t G = a.h_q / a.h_kv;
    if (!grid_ok(joins, NT)) return hipErrorInvalidConfiguration;
    if (p.prefix.splits > 0 && !grid_ok((a.total * G / p.prefix.rows + a.n_groups) * p.prefix.splits * a.h_kv, 512)) return hipErrorInvalidConfiguration;
    if (p.own.splits > 0 && !grid_ok((a.total * G / p.own.rows + a.n_seqs) * p.own.splits * a.h_kv, 512)) return hipErrorInvalidConfiguration;
    hipError_t e = hipSuccess;
    if (p.prefix.splits > 0) e = side<M, D, kPrefix>(a, p.prefix, a.n_groups, 0, stream);
    if (e == hipSuccess && p.own.splits > 0) e = side<M, D, kOwn>(a, p.own, a.n_seqs, p.prefix.splits, stream);
    if (e != hipSuccess) return e;
    a.splits = splits;
    a.split_keys = p.own.split_keys;
    a.prefix_keys = p.prefix.split_keys;
    a.part_first = p.prefix.splits;
    if (sliced) return start(join_kernel<M, D, R, true>, joins, a, stream, NT);
    return start(join_kernel<M, D, 1, true>, joins, a, stream, NT);
}

template <class M>
hipError_t shared_m(const AttnArgs &a, const SharedPlan &p, int d, hipStream_t stream)
{
    switch (d) {
    case 64: return shared_d<M, 64>(a, p, stream);
    case 128: return shared_d<M, 128>(a, p, stream);
    case 256: return shared_d<M, 256>(a, p, stream);
    default: return hipErrorNotSupported;
    }
}

}  // namespace

hipError_t launch_shared_attn(const AttnArgs &a, const SharedPlan &p, int bf16, int d, hipStream_t stream)
{
    return bf16 ? shared_m<MfmaBF16>(a, p, d, stream) : shared_m<MfmaF32>(a, p, d, stream);
}

}  // namespace gdn
