// C ABI of the suffix and decode operators: host-side validation, workspace carving and launches.
// Declarations and the contract of every entry point are in include/gdn.h.
#include <math.h>
#include <stdio.h>
#include <stdlib.h>

#include "../../include/gdn.h"
#include "gdn_ops.h"

namespace {

constexpr size_t kWorkspaceBytes = 256;   // status word, padded to one cache line

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
bool aligned4(const void *p) { return ((uintptr_t)p & 3u) == 0; }
size_t up256(size_t b) { return (b + 255) & ~(size_t)255; }

int32_t refuse(int32_t code, const char *msg)
{
    static const int on = [] {
        const char *e = getenv("GDN_DEBUG");
        return e && e[0] == '1';
    }();
    if (on) fprintf(stderr, "gdn: %s\n", msg);
    return code;
}

bool known_dtype(int32_t t) { return t == GDN_F32 || t == GDN_BF16; }
int64_t elem_bytes(int32_t t) { return t == GDN_BF16 ? 2 : 4; }
// a row stride: rows do not overlap and every row starts on 16 bytes
bool stride_ok(int64_t stride, int64_t row, int32_t dtype)
{
    return stride >= row && stride <= 0x7fffffffLL && stride * elem_bytes(dtype) % 16 == 0;
}
int32_t launched(hipError_t e)
{
    if (e == hipErrorNotSupported) return GDN_ERR_UNSUPPORTED;
    if (e == hipErrorInvalidConfiguration) return refuse(GDN_ERR_SHAPE, "more workgroups than one grid holds");
    return e == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}
int32_t check_ws(const void *ws, size_t bytes, size_t need)
{
    if (!ws) return GDN_ERR_NULL;
    if (!aligned16(ws)) return refuse(GDN_ERR_ALIGN, "the workspace is not 16-byte aligned");
    if (bytes < need) return refuse(GDN_ERR_WORKSPACE, "workspace too small");
    return GDN_OK;
}

// ---------------------------------------------------------------- convolution
int32_t check_conv(const gdn_conv_desc *d, bool step)
{
    if (!d) return GDN_ERR_NULL;
    if (!known_dtype(d->dtype)) return refuse(GDN_ERR_DTYPE, "unknown dtype code");
    if (d->n_seqs < 0 || d->channels <= 0 || d->total_tokens < 0 || d->total_tokens > 0x7fffffffLL ||
        (d->silu != 0 && d->silu != 1))
        return refuse(GDN_ERR_SHAPE, "convolution: bad sizes or activation code");
    if (step && (d->n_slots < 0 || d->total_tokens != d->n_seqs))
        return refuse(GDN_ERR_SHAPE, "convolution step: one token per row, n_slots >= 0");
    if (d->width < 2 || d->width > 4) return refuse(GDN_ERR_UNSUPPORTED, "convolution width must be 2, 3 or 4");
    if (d->channels * elem_bytes(d->dtype) % 16 != 0)
        return refuse(GDN_ERR_ALIGN, "the channels of a token must fill whole 16-byte vectors");
    if (!stride_ok(d->x_stride, d->channels, d->dtype) || !stride_ok(d->y_stride, d->channels, d->dtype))
        return refuse(GDN_ERR_ALIGN, "x_stride and y_stride: at least the channels, a multiple of 16 bytes");
    return GDN_OK;
}

// ---------------------------------------------------------------- state space
int32_t check_ssm(const gdn_ssm_desc *d, bool step)
{
    if (!d) return GDN_ERR_NULL;
    if (!known_dtype(d->dtype)) return refuse(GDN_ERR_DTYPE, "unknown dtype code");
    if (d->n_seqs < 0 || d->h_qk <= 0 || d->h_v <= 0 || d->h_v % d->h_qk != 0 || d->d_k <= 0 || d->d_v <= 0 ||
        d->total_tokens < 0 || d->total_tokens > 0x7fffffffLL || d->total_out_tokens < 0 ||
        d->total_out_tokens > 0x7fffffffLL || (d->softplus != 0 && d->softplus != 1))
        return refuse(GDN_ERR_SHAPE, "state space: bad sizes, h_v not a multiple of h_qk, or softplus code");
    if (step && (d->n_slots < 0 || d->total_tokens != d->n_seqs))
        return refuse(GDN_ERR_SHAPE, "state space step: one token per row, n_slots >= 0");
    if ((d->d_k != 64 && d->d_k != 128) || (d->d_v != 64 && d->d_v != 128))
        return refuse(GDN_ERR_UNSUPPORTED, "unsupported head dims: d_k and d_v must be 64 or 128");
    const int64_t x = (int64_t)d->h_v * d->d_v, k = (int64_t)d->h_qk * d->d_k;
    if (!stride_ok(d->x_stride, x, d->dtype) || !stride_ok(d->b_stride, k, d->dtype) ||
        !stride_ok(d->c_stride, k, d->dtype) || !stride_ok(d->y_stride, x, d->dtype))
        return refuse(GDN_ERR_ALIGN, "x, B, C, y strides: at least a token's row, a multiple of 16 bytes");
    const int64_t widest = d->x_stride > d->y_stride ? d->x_stride : d->y_stride, groups = d->b_stride > d->c_stride ? d->b_stride : d->c_stride;
    if (!step && (widest > groups ? widest : groups) * 64 * elem_bytes(d->dtype) >= 0x7fffffffLL)
        return refuse(GDN_ERR_SHAPE, "state space: a 64-token chunk must span less than 2 GiB");
    if (d->dt_stride < d->h_v || d->dt_stride >= (1LL << 40)) return refuse(GDN_ERR_SHAPE, "dt_stride below h_v");
    return GDN_OK;
}
struct ScanPlan {
    int32_t segs;
    size_t state, decay, bytes;
};
ScanPlan scan_plan(const gdn_ssm_desc *d)
{
    ScanPlan p;
    p.segs = gdn::scan_segments(d->n_seqs, d->h_v, d->d_k, d->d_v, d->dtype == GDN_BF16, d->total_out_tokens);
    const size_t chains = (size_t)d->n_seqs * (size_t)p.segs * (size_t)d->h_v;
    p.state = kWorkspaceBytes;
    p.decay = p.state + chains * (size_t)d->d_k * (size_t)d->d_v * sizeof(float);
    p.bytes = p.segs > 1 ? p.decay + up256(chains * sizeof(float)) : kWorkspaceBytes;
    return p;
}

// ---------------------------------------------------------------- paged attention
int32_t check_paged(const gdn_paged_desc *d)
{
    if (!d) return GDN_ERR_NULL;
    if (!known_dtype(d->dtype)) return refuse(GDN_ERR_DTYPE, "unknown dtype code");
    if (d->n_seqs < 0 || d->h_q <= 0 || d->h_kv <= 0 || d->h_q % d->h_kv != 0 || d->d <= 0 || d->page_size <= 0 ||
        d->n_pages < 0 || d->max_pages < 0 || d->max_kv_len < 0 || d->max_kv_len > (1 << 30) ||
        d->total_tokens < 0 || d->total_tokens > 0x7fffffffLL || d->total_tokens * d->h_q > 0x7fffffffLL)
        return refuse(GDN_ERR_SHAPE, "paged cache: bad sizes, h_q not a multiple of h_kv, or too many rows");
    if (d->d != 64 && d->d != 128 && d->d != 256)
        return refuse(GDN_ERR_UNSUPPORTED, "unsupported head dim: d must be 64, 128 or 256");
    if ((int64_t)d->h_q * d->d > 0x7fffffffLL) return refuse(GDN_ERR_SHAPE, "a token's row is longer than a stride may be");
    const int64_t e = elem_bytes(d->dtype);
    if (d->page_stride < 0 || d->token_stride < d->d || d->head_stride < d->d ||
        d->page_stride >= (1LL << 40) || d->token_stride >= (1LL << 40) || d->head_stride >= (1LL << 40) ||
        d->page_stride * e % 16 || d->token_stride * e % 16 || d->head_stride * e % 16)
        return refuse(GDN_ERR_ALIGN, "cache strides: at least a head's entries, multiples of 16 bytes");
    return GDN_OK;
}
struct PagedPlan {
    gdn::AttnPlan attn;
    size_t o, ml, bytes;
};
PagedPlan paged_plan(const gdn_paged_desc *d)
{
    PagedPlan p;
    p.attn = gdn::attn_plan(d->total_tokens, d->n_seqs, d->h_q, d->h_kv, d->d, d->max_kv_len, d->dtype == GDN_BF16);
    const size_t rows = (size_t)p.attn.splits * (size_t)d->total_tokens * (size_t)d->h_q;
    p.o = kWorkspaceBytes;
    p.ml = p.o + rows * (size_t)d->d * sizeof(float);
    p.bytes = p.attn.splits > 1 ? p.ml + up256(rows * 2 * sizeof(float)) : kWorkspaceBytes;
    return p;
}

}  // namespace

extern "C" {

int32_t gdn_conv(const gdn_conv_desc *d, const void *x, const float *weight, const float *bias, const int32_t *cu,
                 const void *state0, void *state_out, void *y, void *ws, size_t ws_bytes, void *stream)
{
    int32_t st = check_conv(d, false);
    if (st != GDN_OK) return st;
    if (!cu || !weight || (d->total_tokens > 0 && (!x || !y))) return GDN_ERR_NULL;
    if (!aligned16(x) || !aligned16(y) || !aligned16(state0) || !aligned16(state_out) || !aligned4(weight) ||
        !aligned4(bias) || !aligned4(cu))
        return refuse(GDN_ERR_ALIGN, "pointer alignment: 16 bytes required (4 for weight, bias and integer arrays)");
    st = check_ws(ws, ws_bytes, kWorkspaceBytes);
    if (st != GDN_OK || d->n_seqs == 0) return st;
    gdn::ConvArgs a = {};
    a.x = x; a.w = weight; a.bias = bias; a.cu = cu; a.state0 = state0; a.state = state_out; a.y = y;
    a.status = static_cast<int32_t *>(ws);
    a.total = d->total_tokens; a.xs = d->x_stride; a.ys = d->y_stride;
    a.n_seqs = d->n_seqs; a.channels = d->channels; a.silu = d->silu;
    return launched(gdn::launch_conv(a, d->dtype == GDN_BF16, d->width, static_cast<hipStream_t>(stream)));
}

int32_t gdn_conv_step(const gdn_conv_desc *d, const void *x, const float *weight, const float *bias, void *state,
                      const int32_t *slots, void *y, void *ws, size_t ws_bytes, void *stream)
{
    int32_t st = check_conv(d, true);
    if (st != GDN_OK) return st;
    if (!slots && d->n_slots < d->n_seqs) return refuse(GDN_ERR_SHAPE, "fewer slots than rows");
    if (!weight || (d->n_seqs > 0 && (!x || !y || !state))) return GDN_ERR_NULL;
    if (!aligned16(x) || !aligned16(y) || !aligned16(state) || !aligned4(weight) || !aligned4(bias) || !aligned4(slots))
        return refuse(GDN_ERR_ALIGN, "pointer alignment: 16 bytes required (4 for weight, bias and integer arrays)");
    st = check_ws(ws, ws_bytes, kWorkspaceBytes);
    if (st != GDN_OK || d->n_seqs == 0) return st;
    gdn::ConvArgs a = {};
    a.x = x; a.w = weight; a.bias = bias; a.slots = slots; a.state = state; a.y = y;
    a.status = static_cast<int32_t *>(ws);
    a.xs = d->x_stride; a.ys = d->y_stride;
    a.n_seqs = d->n_seqs; a.n_slots = d->n_slots; a.channels = d->channels; a.silu = d->silu;
    return launched(gdn::launch_conv_step(a, d->dtype == GDN_BF16, d->width, static_cast<hipStream_t>(stream)));
}

size_t gdn_ssm_workspace_bytes(const gdn_ssm_desc *d)
{
    return check_ssm(d, false) == GDN_OK ? scan_plan(d).bytes : 0;
}

int32_t gdn_ssm_scan(const gdn_ssm_desc *d, const void *x, const void *B, const void *C, const void *dt, const float *A,
                     const float *dt_bias, const float *D, const int32_t *cu, const int32_t *r, const float *S0,
                     float *S_out, void *y, int32_t *cu_out, void *ws, size_t ws_bytes, void *stream)
{
    int32_t st = check_ssm(d, false);
    if (st != GDN_OK) return st;
    if (r ? d->total_out_tokens > d->total_tokens : d->total_out_tokens != d->total_tokens)
        return refuse(GDN_ERR_SHAPE, "total_out_tokens: total_tokens, or at most that with replay lengths");
    if (!cu || !S_out || !A || (d->total_tokens > 0 && (!x || !B || !C || !dt))) return GDN_ERR_NULL;
    if (!aligned16(x) || !aligned16(B) || !aligned16(C) || !aligned16(y) || !aligned16(S0) || !aligned16(S_out) ||
        ((uintptr_t)dt & (uintptr_t)(elem_bytes(d->dtype) - 1)) || !aligned4(A) || !aligned4(dt_bias) || !aligned4(D) ||
        !aligned4(cu) || !aligned4(r) || !aligned4(cu_out))
        return refuse(GDN_ERR_ALIGN, "pointer alignment: 16 bytes required (an element's for dt, 4 for parameters and integer arrays)");
    const ScanPlan p = scan_plan(d);
    st = check_ws(ws, ws_bytes, p.bytes);
    if (st != GDN_OK || d->n_seqs == 0) return st;
    char *w = static_cast<char *>(ws);
    gdn::ScanArgs a = {};
    a.x = x; a.B = B; a.C = C; a.dt = dt; a.A = A; a.dt_bias = dt_bias; a.D = D;
    a.cu = cu; a.r = r; a.S0 = S0; a.S_out = S_out; a.y = y; a.cu_out = cu_out;
    a.status = reinterpret_cast<int32_t *>(w);
    a.seg_state = reinterpret_cast<float *>(w + p.state);
    a.seg_decay = reinterpret_cast<float *>(w + p.decay);
    a.xs = d->x_stride; a.bs = d->b_stride; a.cs = d->c_stride; a.dts = d->dt_stride; a.ys = d->y_stride;
    a.total = d->total_tokens; a.total_out = d->total_out_tokens;
    a.n_seqs = d->n_seqs; a.h_qk = d->h_qk; a.h_v = d->h_v; a.softplus = d->softplus; a.segs = p.segs;
    return launched(gdn::launch_scan(a, d->dtype == GDN_BF16, d->d_k, d->d_v, static_cast<hipStream_t>(stream)));
}

int32_t gdn_ssm_step(const gdn_ssm_desc *d, const void *x, const void *B, const void *C, const void *dt, const float *A,
                     const float *dt_bias, const float *D, float *S, const int32_t *slots, void *y, void *ws,
                     size_t ws_bytes, void *stream)
{
    int32_t st = check_ssm(d, true);
    if (st != GDN_OK) return st;
    if (!slots && d->n_slots < d->n_seqs) return refuse(GDN_ERR_SHAPE, "fewer slots than rows");
    if (!A || (d->n_seqs > 0 && (!x || !B || !C || !dt || !S || !y))) return GDN_ERR_NULL;
    if (!aligned16(x) || !aligned16(B) || !aligned16(C) || !aligned16(y) || !aligned16(S) ||
        ((uintptr_t)dt & (uintptr_t)(elem_bytes(d->dtype) - 1)) || !aligned4(A) || !aligned4(dt_bias) || !aligned4(D) ||
        !aligned4(slots))
        return refuse(GDN_ERR_ALIGN, "pointer alignment: 16 bytes required (an element's for dt, 4 for parameters and integer arrays)");
    st = check_ws(ws, ws_bytes, kWorkspaceBytes);
    if (st != GDN_OK || d->n_seqs == 0) return st;
    gdn::StepArgs a = {};
    a.q = C; a.k = B; a.v = x; a.dt = dt; a.A = A; a.dt_bias = dt_bias; a.D = D;
    a.slots = slots; a.S = S; a.o = y; a.status = static_cast<int32_t *>(ws);
    a.qs = d->c_stride; a.ks = d->b_stride; a.vs = d->x_stride; a.dts = d->dt_stride; a.os = d->y_stride;
    a.rows = d->n_seqs; a.n_slots = d->n_slots; a.h_qk = d->h_qk; a.h_v = d->h_v; a.softplus = d->softplus;
    a.scale = 1.0f;
    return launched(gdn::launch_step(a, d->dtype == GDN_BF16, d->d_k, d->d_v, false, static_cast<hipStream_t>(stream)));
}

int32_t gdn_step(const gdn_desc *d, const void *q, const void *k, const void *v, const float *g, const float *beta,
                 float *S, int32_t n_slots, const int32_t *slots, void *o, void *ws, size_t ws_bytes, void *stream)
{
    if (!d) return GDN_ERR_NULL;
    if (d->n_seqs < 0 || d->h_qk <= 0 || d->h_v <= 0 || d->h_v % d->h_qk != 0 || d->d_k <= 0 || d->d_v <= 0 ||
        d->total_tokens != d->n_seqs || d->total_out_tokens != d->n_seqs || n_slots < 0)
        return refuse(GDN_ERR_SHAPE, "step: bad sizes, h_v not a multiple of h_qk, or not one token per row");
    if (!known_dtype(d->qkv_dtype) || !known_dtype(d->o_dtype) || (d->o_dtype != d->qkv_dtype && d->o_dtype != GDN_F32))
        return refuse(GDN_ERR_DTYPE, "unknown dtype code, or o_dtype neither qkv_dtype nor fp32");
    if ((d->d_k != 64 && d->d_k != 128) || (d->d_v != 64 && d->d_v != 128))
        return refuse(GDN_ERR_UNSUPPORTED, "unsupported head dims: d_k and d_v must be 64 or 128");
    if (!slots && n_slots < d->n_seqs) return refuse(GDN_ERR_SHAPE, "fewer slots than rows");
    if (d->n_seqs > 0 && (!q || !k || !v || !g || !beta || !S || !o)) return GDN_ERR_NULL;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned4(g) || !aligned4(beta) || !aligned16(S) ||
        !aligned16(o) || !aligned4(slots))
        return refuse(GDN_ERR_ALIGN, "pointer alignment: 16 bytes required (4 for g, beta and slots)");
    const int32_t st = check_ws(ws, ws_bytes, kWorkspaceBytes);
    if (st != GDN_OK || d->n_seqs == 0) return st;
    gdn::StepArgs a = {};
    a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.slots = slots; a.S = S; a.o = o;
    a.status = static_cast<int32_t *>(ws);
    a.qs = a.ks = (int64_t)d->h_qk * d->d_k;
    a.vs = a.os = (int64_t)d->h_v * d->d_v;
    a.rows = d->n_seqs; a.n_slots = n_slots; a.h_qk = d->h_qk; a.h_v = d->h_v;
    a.o_f32 = d->o_dtype == GDN_F32;
    a.scale = d->scale;
    return launched(gdn::launch_step(a, d->qkv_dtype == GDN_BF16, d->d_k, d->d_v, true, static_cast<hipStream_t>(stream)));
}

int32_t gdn_qk_norm_rope(const gdn_paged_desc *d, const void *q, const void *k, const void *v, const float *q_weight,
                         const float *k_weight, const float *cos_sin, const int32_t *block_table, const int32_t *cu,
                         const int32_t *kv_len, const int32_t *positions, void *k_cache, void *v_cache, void *q_out,
                         void *ws, size_t ws_bytes, void *stream)
{
    int32_t st = check_paged(d);
    if (st != GDN_OK) return st;
    if (d->rot_dim < 0 || d->rot_dim > d->d || d->rot_dim % 16 != 0 || d->max_pos < 0 ||
        (d->interleaved != 0 && d->interleaved != 1) || (d->norm != 0 && d->norm != 1) || !(d->eps >= 0.0f))
        return refuse(GDN_ERR_SHAPE, "rotation: rot_dim a multiple of 16 in [0, d], max_pos >= 0, flags 0 or 1, eps >= 0");
    const int64_t qr = (int64_t)d->h_q * d->d, kr = (int64_t)d->h_kv * d->d;
    if (!stride_ok(d->q_stride, qr, d->dtype) || !stride_ok(d->o_stride, qr, d->dtype) ||
        !stride_ok(d->k_stride, kr, d->dtype) || !stride_ok(d->v_stride, kr, d->dtype))
        return refuse(GDN_ERR_ALIGN, "q, k, v, output strides: at least a token's row, a multiple of 16 bytes");
    if (!cu || !kv_len || (d->total_tokens > 0 && (!q || !k || !v || !block_table || !k_cache || !v_cache || !q_out ||
                                                    (d->rot_dim > 0 && !cos_sin))))
        return GDN_ERR_NULL;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(q_out) ||
        !aligned16(q_weight) || !aligned16(k_weight) || !aligned16(cos_sin) || !aligned4(block_table) || !aligned4(cu) ||
        !aligned4(kv_len) || !aligned4(positions))
        return refuse(GDN_ERR_ALIGN, "pointer alignment: 16 bytes required (4 for integer arrays)");
    st = check_ws(ws, ws_bytes, kWorkspaceBytes);
    if (st != GDN_OK || d->n_seqs == 0 || d->total_tokens == 0) return st;
    gdn::RopeArgs a = {};
    a.q = q; a.k = k; a.v = v; a.qw = d->norm ? q_weight : nullptr; a.kw = d->norm ? k_weight : nullptr;
    a.cos_sin = cos_sin; a.kc = k_cache; a.vc = v_cache; a.qo = q_out;
    a.table = block_table; a.cu = cu; a.kv_len = kv_len; a.positions = positions;
    a.status = static_cast<int32_t *>(ws);
    a.qs = d->q_stride; a.ks = d->k_stride; a.vs = d->v_stride; a.qos = d->o_stride;
    a.page_stride = d->page_stride; a.token_stride = d->token_stride; a.head_stride = d->head_stride;
    a.total = d->total_tokens;
    a.n_seqs = d->n_seqs; a.h_q = d->h_q; a.h_kv = d->h_kv;
    a.page_size = d->page_size; a.n_pages = d->n_pages; a.max_pages = d->max_pages;
    a.rot = d->rot_dim; a.norm = d->norm; a.max_pos = d->max_pos; a.max_kv = d->max_kv_len;
    a.eps = d->eps;
    return launched(gdn::launch_rope(a, d->dtype == GDN_BF16, d->d, d->interleaved != 0, static_cast<hipStream_t>(stream)));
}

size_t gdn_paged_workspace_bytes(const gdn_paged_desc *d)
{
    return check_paged(d) == GDN_OK ? paged_plan(d).bytes : 0;
}

int32_t gdn_paged_attn(const gdn_paged_desc *d, const void *q, const void *k_cache, const void *v_cache,
                       const int32_t *block_table, const int32_t *cu, const int32_t *kv_len, void *o, float *lse,
                       void *ws, size_t ws_bytes, void *stream)
{
    int32_t st = check_paged(d);
    if (st != GDN_OK) return st;
    if (!isfinite(d->scale)) return refuse(GDN_ERR_SHAPE, "the score scale is not finite");
    const int64_t row = (int64_t)d->h_q * d->d;
    if (!stride_ok(d->q_stride, row, d->dtype) || !stride_ok(d->o_stride, row, d->dtype))
        return refuse(GDN_ERR_ALIGN, "q and output strides: at least a token's row, a multiple of 16 bytes");
    if (!cu || !kv_len || (d->total_tokens > 0 && (!q || !o)) ||
        (d->total_tokens > 0 && d->max_kv_len > 0 && (!k_cache || !v_cache || !block_table)))
        return GDN_ERR_NULL;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(o) || !aligned4(lse) ||
        !aligned4(block_table) || !aligned4(cu) || !aligned4(kv_len))
        return refuse(GDN_ERR_ALIGN, "pointer alignment: 16 bytes required (4 for lse and integer arrays)");
    const PagedPlan p = paged_plan(d);
    st = check_ws(ws, ws_bytes, p.bytes);
    if (st != GDN_OK || d->n_seqs == 0 || d->total_tokens == 0) return st;
    char *w = static_cast<char *>(ws);
    gdn::AttnArgs a = {};
    a.q = q; a.kc = k_cache; a.vc = v_cache; a.table = block_table; a.cu = cu; a.kv_len = kv_len;
    a.o = o; a.lse = lse; a.status = reinterpret_cast<int32_t *>(w);
    a.part_o = reinterpret_cast<float *>(w + p.o);
    a.part_ml = reinterpret_cast<float *>(w + p.ml);
    a.qs = d->q_stride; a.os = d->o_stride;
    a.page_stride = d->page_stride; a.token_stride = d->token_stride; a.head_stride = d->head_stride;
    a.total = d->total_tokens;
    a.n_seqs = d->n_seqs; a.h_q = d->h_q; a.h_kv = d->h_kv;
    a.page_size = d->page_size; a.n_pages = d->n_pages; a.max_pages = d->max_pages; a.max_kv = d->max_kv_len;
    a.splits = p.attn.splits; a.split_keys = p.attn.split_keys;
    a.scale = d->scale;
    return launched(gdn::launch_attn(a, p.attn, d->dtype == GDN_BF16, d->d, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
