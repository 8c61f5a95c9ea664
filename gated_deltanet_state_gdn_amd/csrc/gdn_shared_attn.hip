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
//
// Bound as attention without groups is: few rows by the reads of keys and values, or at the smallest calls by two
// launches, many rows by the matrix products; and by the splits' shares, which are written and read in fp32 (16 heads
// of 256, 64 tokens in 64 splits: 67 MB each way).  Measured, bf16: the next token of two requests behind 1024 tokens
// 13.5 us (9.4 and the join's 4.1 to 5); of 64 behind 31744, 16 heads on 2 of 256, 108 (prefix 65, own 22, join 15);
// of 96 behind 7 prefixes of up to 8192, 32 heads on 8 of 128, 135 (52, 73, 12); 12 prompts, 1501 tokens behind 16384,
// 411 to 429.
#include "gdn_attn.h"

namespace gdn {
namespace {

template <class M, int D, int WAVES>
hipError_t decode_n(const AttnArgs &a, const AttnPlan &p, int64_t blocks, hipStream_t stream)
{
    if (p.rows == 16) return start(decode_kernel<M, D, 1, WAVES, kShared>, blocks, a, stream, 64 * WAVES);
    if constexpr (M::V == 8 && D != 128) return start(decode_kernel<M, D, 2, WAVES, kShared>, blocks, a, stream, 64 * WAVES);
    return hipErrorNotSupported;                         // the plan has no such rows
}

// One launch of so many blocks of prefixes and of own keys, in a plan's form.  fine: probabilities in two bf16 terms, as the
// form of few rows always has them.
template <class M, int D>
hipError_t sides(AttnArgs a, const AttnPlan &p, bool fine, int64_t prefix, int64_t own, hipStream_t stream)
{
    const int64_t blocks = prefix + own;
    a.prefix_blocks = (uint32_t)prefix;
    if (p.decode) {
        constexpr int WAVES = decode_waves(Tile<M, D>::RB);
        if (p.waves == WAVES) return decode_n<M, D, WAVES>(a, p, blocks, stream);
        if constexpr (decode_wide(Tile<M, D>::RB)) return decode_n<M, D, 2 * WAVES>(a, p, blocks, stream);
        return hipErrorNotSupported;                     // the plan has no such waves
    }
    if constexpr (M::V == 4) return start(prefill_kernel<M, D, 1, 4, 32, kShared>, blocks, a, stream, 256);
    else if (p.rows == 256) return start(fine ? prefill_kernel<M, D, 2, 8, 64, kShared, 2> : prefill_kernel<M, D, 2, 8, 64, kShared>, blocks, a, stream, 512);
    else return start(fine ? prefill_kernel<M, D, 2, 4, 64, kShared, 2> : prefill_kernel<M, D, 2, 4, 64, kShared>, blocks, a, stream, 256);
}

template <class M, int D>
hipError_t shared_d(AttnArgs a, const SharedPlan &p, hipStream_t stream)
{
    constexpr int R = NT / (D / 4);                      // rows of a join's workgroup without slices
    a.splits = p.own.splits;
    a.split_keys = p.own.split_keys;
    a.prefix_splits = p.prefix.splits;
    a.prefix_keys = p.prefix.split_keys;
    const int splits = p.prefix.splits + p.own.splits;
    const bool sliced = splits > 8 || (splits > 2 && a.total * a.h_q <= 4096);
    const int64_t G = a.h_q / a.h_kv, joins = a.total * (sliced ? a.h_q : (a.h_q + R - 1) / R);
    const int64_t prefix = (a.total * G / p.prefix.rows + a.n_groups) * p.prefix.splits * a.h_kv;
    const int64_t own = (a.total * G / p.own.rows + a.n_seqs) * p.own.splits * a.h_kv;
    if (!grid_ok(joins, NT) || !grid_ok(prefix + own + 1, 512)) return hipErrorInvalidConfiguration;
    // one launch where both sides take the same form
    const bool same = p.prefix.decode == p.own.decode && p.prefix.rows == p.own.rows && (!p.own.decode || p.prefix.waves == p.own.waves);
    hipError_t e = hipSuccess;
    if (same && prefix + own > 0) e = sides<M, D>(a, p.own, p.fine, prefix, own, stream);
    if (!same && prefix > 0) e = sides<M, D>(a, p.prefix, p.fine, prefix, 0, stream);
    if (!same && own > 0 && e == hipSuccess) e = sides<M, D>(a, p.own, p.fine, 0, own, stream);
    if (e != hipSuccess) return e;
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
