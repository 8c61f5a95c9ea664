// Internal declarations of the suffix and decode operators (convolution, state space scan,
// single-token steps, norm + rotation + cache append, paged attention), shared by the host
// side and the gfx950 kernels.  Not part of the public interface (that is include/gdn.h).
#pragma once
#include "gdn_common.h"
#include "gdn_plan.h"

namespace gdn {

// Whether one launch holds so many blocks: a grid has at least one and fewer than 2^32 threads.  Every
// launch of a call is checked before the first one is enqueued.
constexpr bool grid_ok(int64_t blocks, int threads) { return blocks >= 1 && blocks <= 0xffffffffLL / threads; }

struct ConvArgs {
    const void *x;              // [T, channels], rows x_stride apart
    const float *w, *bias;      // [channels, width], [channels] nullable
    const int32_t *cu;          // [n_seqs + 1] (null for a step)
    const int32_t *slots;       // [n_seqs] (step), nullable
    const void *state0;         // [n_seqs, width - 1, channels], nullable (zero)
    void *state;                // prompts: the state behind each sequence, nullable; step: [n_slots, width - 1, channels]
    void *y;
    int32_t *status;
    int64_t total, xs, ys;
    int32_t n_seqs, n_slots, channels, silu;
};
hipError_t launch_conv(const ConvArgs &a, int bf16, int width, hipStream_t stream);
hipError_t launch_conv_step(const ConvArgs &a, int bf16, int width, hipStream_t stream);

struct StepArgs {
    const void *q, *k, *v;      // q = C, k = B, v = x for the state space step
    const float *g, *beta;      // gated delta rule
    const void *dt;             // state space: [rows, h_v] in the element type
    const float *A, *dt_bias, *D;
    const int32_t *slots;
    float *S;
    void *o;
    int32_t *status;
    int64_t qs, ks, vs, dts, os;   // elements between rows
    int32_t rows, n_slots, h_qk, h_v, softplus, o_f32;
    float scale;
};
hipError_t launch_step(const StepArgs &a, int bf16, int d_k, int d_v, bool delta, hipStream_t stream);

struct ScanArgs {
    const void *x, *B, *C, *dt;
    const float *A, *dt_bias, *D;
    const int32_t *cu, *r;      // r nullable: whole sequences
    const float *S0;            // nullable
    float *S_out;
    void *y;                    // nullable
    int32_t *cu_out;            // nullable
    int32_t *status;
    float *seg_state;           // [n_seqs, segs, h_v, d_k, d_v] with more than one segment
    float *seg_decay;           // [n_seqs, segs, h_v]
    int64_t xs, bs, cs, dts, ys, total, total_out;
    int32_t n_seqs, h_qk, h_v, softplus, segs;
};
hipError_t launch_scan(const ScanArgs &a, int bf16, int d_k, int d_v, hipStream_t stream);

struct RopeArgs {
    const void *q, *k, *v;
    const float *qw, *kw, *cos_sin;
    void *kc, *vc, *qo;
    const int32_t *table, *cu, *kv_len, *positions;
    int32_t *status;
    int64_t qs, ks, vs, qos, page_stride, token_stride, head_stride, total;
    int32_t n_seqs, h_q, h_kv, page_size, n_pages, max_pages, rot, norm, max_pos, max_kv;
    float eps;
};
hipError_t launch_rope(const RopeArgs &a, int bf16, int d, bool interleaved, hipStream_t stream);

struct AttnArgs {
    const void *q, *kc, *vc;
    const int32_t *table, *cu, *kv_len;
    void *o;
    float *lse;                 // [T, h_q], nullable
    float *part_o, *part_ml;    // split partials: [splits, T, h_q, d] and [splits, T, h_q, 2]
    int32_t *status;
    int64_t qs, os, page_stride, token_stride, head_stride, total;
    int32_t n_seqs, h_q, h_kv, page_size, n_pages, max_pages, max_kv;
    int32_t splits, split_keys; // split s covers keys [s split_keys, (s + 1) split_keys)
    float scale;
    // shared prefixes: cu_groups [n_groups + 1], prefix_len [n_groups]
    const int32_t *groups, *prefix_len;
    int32_t n_groups, max_prefix, max_own;
    uint32_t prefix_blocks;     // of this launch
    int32_t prefix_splits, prefix_keys;    // of a prefix; splits and split_keys are the own keys' then
};
hipError_t launch_attn(const AttnArgs &a, const AttnPlan &p, int bf16, int d, hipStream_t stream);
hipError_t launch_shared_attn(const AttnArgs &a, const SharedPlan &p, int bf16, int d, hipStream_t stream);

struct ExtendArgs {
    const int32_t *new_len, *kv_len, *free_pages, *free_at;
    const int32_t *prefix_of, *prefix_table, *prefix_len;      // nullable together
    int32_t *table, *kv_out, *free_out, *cu;
    int64_t *slots;             // [total], nullable
    int32_t *positions;         // [total], nullable
    int32_t *status;
    int64_t *plan;              // workspace: per request, and what the second launch has to do
    int64_t total;
    int32_t n_seqs, page_size, max_pages, n_free, n_prefixes, max_prefix_pages;
};
hipError_t launch_extend(const ExtendArgs &a, hipStream_t stream);

struct SampleArgs {
    const void *logits;
    const float *u, *temperature, *top_p, *min_p;              // all but u nullable
    const int32_t *top_k;       // nullable
    int32_t *token;
    float *logprob;             // nullable
    int32_t *status;
    void *heads;                // workspace: a ChunkHead for each chunk of a row
    uint64_t *bins;             // workspace: kSampleBins for each chunk of a row
    int64_t stride;
    int32_t rows, vocab, chunk, chunks;
};
hipError_t launch_sample(const SampleArgs &a, int bf16, hipStream_t stream);

}  // namespace gdn
