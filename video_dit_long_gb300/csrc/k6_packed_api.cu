// k6_packed_api.cu -- entry points of the packed-sequence calls: argument checks
// on the host, then the launches.  Nothing here allocates or aborts.
#include <stdint.h>

#include "k6_packed_tma.h"

using namespace k6;

namespace {

// Token rows [n][width elements of `elem` bytes], `stride` elements apart.
struct Rows {
    const char *name;
    const void *p;
    long n, stride, width;
    int elem;
    uintptr_t begin() const { return reinterpret_cast<uintptr_t>(p); }
    size_t extent() const { return n > 0 ? (size_t)(((n - 1) * stride + width) * elem) : 0; }
};

// Whether two sets of rows share a byte.  Views of one buffer with the same
// stride (the q, k and v parts of a fused projection) interleave without
// sharing any; other overlapping extents count as shared.
bool share(const Rows &a, const Rows &b) {
    if (!overlap(a.p, a.extent(), b.p, b.extent())) return false;
    const uintptr_t sa = (uintptr_t)a.stride * a.elem, sb = (uintptr_t)b.stride * b.elem;
    if (sa != sb) return true;
    const uintptr_t wa = (uintptr_t)a.width * a.elem, wb = (uintptr_t)b.width * b.elem;
    const uintptr_t delta = a.begin() <= b.begin() ? (b.begin() - a.begin()) % sa : sa - (a.begin() - b.begin()) % sa;
    return !(delta >= wa && delta + wb <= sa);
}

k6attn_status check_rows(const char *fn, const Rows &r) {
    if (r.n == 0) return K6ATTN_OK;
    if (!r.p) return set_error(K6ATTN_ERR_INVALID_ARG, "%s: null %s", fn, r.name);
    if (!aligned16(r.p)) return set_error(K6ATTN_ERR_INVALID_ARG, "%s: %s must be 16-byte aligned", fn, r.name);
    if (r.stride < r.width || (r.stride * r.elem) % 16 || r.stride >= (1L << 31))
        return set_error(K6ATTN_ERR_INVALID_ARG,
                         "%s: the token stride of %s is %ld elements; at least %ld, a multiple of 16 bytes and below "
                         "2^31 wanted",
                         fn, r.name, r.stride, r.width);
    return K6ATTN_OK;
}

k6attn_status check_apart(const char *fn, const Rows *out, int n_out, const Rows *in, int n_in) {
    for (int i = 0; i < n_out; i++) {
        for (int j = 0; j < n_in; j++)
            if (share(out[i], in[j]))
                return set_error(K6ATTN_ERR_INVALID_ARG, "%s: %s overlaps %s", fn, out[i].name, in[j].name);
        for (int j = i + 1; j < n_out; j++)
            if (share(out[i], out[j]))
                return set_error(K6ATTN_ERR_INVALID_ARG, "%s: %s overlaps %s", fn, out[i].name, out[j].name);
    }
    return K6ATTN_OK;
}

// `bytes` bytes at p as one row.
Rows flat(const char *name, const void *p, size_t bytes) {
    return {name, p, p && bytes ? 1 : 0, (long)bytes, (long)bytes, 1};
}

k6attn_status check_norm(const char *fn, k6attn_t h, long tokens, int kv_heads, const int *cu, int n_seq,
                         const int *positions, const float *q_weight, const float *k_weight, float eps) {
    k6attn_status s = check_handle(fn, h);
    if (s != K6ATTN_OK) return s;
    if (tokens < 0 || kv_heads < 1)
        return set_error(K6ATTN_ERR_INVALID_ARG, "%s: tokens must be >= 0 and kv_heads >= 1", fn);
    if (tokens >= (1L << 30) || kv_heads > (1 << 16) || tokens * (h->g.H + kv_heads) >= (1L << 31))
        return set_error(K6ATTN_ERR_UNSUPPORTED, "%s: %ld tokens of %d + %d heads are too many", fn, tokens, h->g.H,
                         kv_heads);
    if (tokens > 0 && !positions) return set_error(K6ATTN_ERR_INVALID_ARG, "%s: null positions", fn);
    if (cu && (n_seq < 1 || n_seq >= (1 << 24)))
        return set_error(K6ATTN_ERR_INVALID_ARG, "%s: n_seq must be in [1, 2^24) with offsets", fn);
    if ((q_weight == nullptr) != (k_weight == nullptr))
        return set_error(K6ATTN_ERR_INVALID_ARG, "%s: give both norm weights, or neither", fn);
    if (!(eps >= 0.f)) return set_error(K6ATTN_ERR_INVALID_ARG, "%s: eps must be >= 0", fn);
    if ((reinterpret_cast<uintptr_t>(positions) | reinterpret_cast<uintptr_t>(q_weight) |
         reinterpret_cast<uintptr_t>(k_weight) | reinterpret_cast<uintptr_t>(cu)) & 3)
        return set_error(K6ATTN_ERR_INVALID_ARG, "%s: offsets, positions and weights must be 4-byte aligned", fn);
    return K6ATTN_OK;
}

// Whether the library takes the batch: host arithmetic alone, whichever device is current.
k6attn_status check_sizes(const char *fn, k6attn_t h, const k6attn_packed *b) {
    if (!h) return set_error(K6ATTN_ERR_INVALID_ARG, "%s: null handle", fn);
    if (!b) return set_error(K6ATTN_ERR_INVALID_ARG, "%s: null batch", fn);
    if (h->g.dtype != K6ATTN_BF16) return set_error(K6ATTN_ERR_UNSUPPORTED, "%s: needs a bf16 handle (d = 128)", fn);
    if (b->n_seq < 1 || b->q_tokens < 0 || b->k_tokens < 0)
        return set_error(K6ATTN_ERR_INVALID_ARG, "%s: n_seq must be >= 1, q_tokens and k_tokens >= 0", fn);
    if (b->kv_heads < 1 || h->g.H % b->kv_heads)
        return set_error(K6ATTN_ERR_INVALID_ARG, "%s: %d query heads are not divisible by %d key heads", fn, h->g.H,
                         b->kv_heads);
    if (h->g.H / b->kv_heads > 128)
        return set_error(K6ATTN_ERR_UNSUPPORTED, "%s: more than 128 query heads per key head", fn);
    if (b->mask_block < 0 || b->mask_block >= (1 << 30))
        return set_error(K6ATTN_ERR_INVALID_ARG, "%s: mask_block must be in [0, 2^30)", fn);
    if (h->sms > 512) return set_error(K6ATTN_ERR_UNSUPPORTED, "%s: more than 512 SMs", fn);
    if (b->q_tokens >= (1L << 30) || b->k_tokens >= (1L << 30) || b->n_seq >= (1 << 24) ||
        b->kv_heads >= (1 << 16) || (b->q_tokens + b->n_seq) * h->g.H >= (1L << 31) ||
        (b->k_tokens + b->n_seq) * b->kv_heads >= (1L << 31))
        return set_error(K6ATTN_ERR_UNSUPPORTED, "%s: batch too large", fn);
    return K6ATTN_OK;
}

k6attn_status check_batch(const char *fn, k6attn_t h, const k6attn_packed *b) {
    const k6attn_status s = check_handle(fn, h);
    return s != K6ATTN_OK ? s : check_sizes(fn, h, b);
}

k6attn_status check_plan(const char *fn, const void *plan) {
    if (!plan || !aligned16(plan))
        return set_error(K6ATTN_ERR_INVALID_ARG, "%s: null plan, or one that is not 16-byte aligned", fn);
    return K6ATTN_OK;
}

}  // namespace

extern "C" {

k6attn_status k6attn_packed_norm_rope(k6attn_t h, long tokens, int kv_heads, const int *cu, int n_seq,
                                      const int *positions, const void *q,
                                      long q_stride, const void *k, long k_stride, const float *q_weight,
                                      const float *k_weight, float eps, void *q_out, long q_out_stride, void *k_out,
                                      long k_out_stride, k6attn_dtype out_dtype, void *stream) {
    const char *fn = "packed_norm_rope";
    clear_error();
    k6attn_status s = check_norm(fn, h, tokens, kv_heads, cu, n_seq, positions, q_weight, k_weight, eps);
    if (s != K6ATTN_OK) return s;
    const Geom &g = h->g;
    if (out_dtype != g.dtype && !(g.dtype == K6ATTN_BF16 && out_dtype == K6ATTN_F16))
        return set_error(K6ATTN_ERR_INVALID_ARG, "%s: output type %d not allowed for this handle", fn, (int)out_dtype);
    const long wq = (long)g.H * g.d, wk = (long)kv_heads * g.d;
    const Rows in[] = {{"q", q, tokens, q_stride, wq, g.elem}, {"k", k, tokens, k_stride, wk, g.elem}};
    const Rows out[] = {{"q_out", q_out, tokens, q_out_stride, wq, g.elem},
                        {"k_out", k_out, tokens, k_out_stride, wk, g.elem}};
    for (int i = 0; i < 2; i++) {
        if ((s = check_rows(fn, in[i])) != K6ATTN_OK || (s = check_rows(fn, out[i])) != K6ATTN_OK) return s;
    }
    for (int i = 0; i < 2; i++) {
        const bool in_place = out[i].p == in[i].p && out[i].stride == in[i].stride && out_dtype == g.dtype;
        const Rows others[] = {in[1 - i], in_place ? flat("", nullptr, 0) : in[i],
                               flat("the positions", positions, (size_t)tokens * 12),
                               flat("a weight", q_weight, q_weight ? g.d * 4 : 0),
                               flat("a weight", k_weight, k_weight ? g.d * 4 : 0),
                               flat("the offsets", cu, cu ? ((size_t)n_seq + 1) * 4 : 0)};
        if ((s = check_apart(fn, out + i, 1, others, 6)) != K6ATTN_OK) return s;
    }
    if ((s = check_apart(fn, out, 2, nullptr, 0)) != K6ATTN_OK) return s;
    PackedNormRope p = {};
    p.tokens = tokens, p.Hkv = kv_heads, p.cu = cu, p.n_seq = n_seq, p.positions = positions, p.turns = h->turns;
    p.x[0] = q, p.x_stride[0] = q_stride, p.x[1] = k, p.x_stride[1] = k_stride;
    p.z[0] = q_out, p.z_stride[0] = q_out_stride, p.z[1] = k_out, p.z_stride[1] = k_out_stride;
    p.w[0] = q_weight, p.w[1] = k_weight, p.eps = eps, p.sms = h->sms, p.err = h->err;
    return cuda_check(launch_packed_norm_rope(g, p, out_dtype, static_cast<cudaStream_t>(stream)),
                      "packed_norm_rope launch");
}

size_t k6attn_packed_norm_rope_backward_workspace_bytes(k6attn_t h, long tokens, int kv_heads) {
    (void)kv_heads;
    if (!h || tokens < 1) return 0;
    return packed_norm_rope_bwd_workspace(h->g, tokens, h->sms);
}

k6attn_status k6attn_packed_norm_rope_backward(k6attn_t h, long tokens, int kv_heads, const int *cu, int n_seq,
                                               const int *positions,
                                               const void *dq_out, long dq_out_stride, const void *dk_out,
                                               long dk_out_stride, const void *q, long q_stride, const void *k,
                                               long k_stride, const float *q_weight, const float *k_weight, float eps,
                                               void *dq, long dq_stride, void *dk, long dk_stride, float *dq_weight,
                                               float *dk_weight, void *workspace, size_t workspace_bytes,
                                               void *stream) {
    const char *fn = "packed_norm_rope_backward";
    clear_error();
    k6attn_status s = check_norm(fn, h, tokens, kv_heads, cu, n_seq, positions, q_weight, k_weight, eps);
    if (s != K6ATTN_OK) return s;
    const Geom &g = h->g;
    const bool norm = q_weight != nullptr;
    if (norm && (!dq_weight || !dk_weight))
        return set_error(K6ATTN_ERR_INVALID_ARG, "%s: null gradient of a norm weight", fn);
    if ((reinterpret_cast<uintptr_t>(dq_weight) | reinterpret_cast<uintptr_t>(dk_weight)) & 3)
        return set_error(K6ATTN_ERR_INVALID_ARG, "%s: gradients of the weights must be 4-byte aligned", fn);
    const long wq = (long)g.H * g.d, wk = (long)kv_heads * g.d;
    const Rows grad[] = {{"dq_out", dq_out, tokens, dq_out_stride, wq, g.elem},
                         {"dk_out", dk_out, tokens, dk_out_stride, wk, g.elem}};
    const Rows in[] = {{"q", q, norm ? tokens : 0, q_stride, wq, g.elem},
                       {"k", k, norm ? tokens : 0, k_stride, wk, g.elem}};
    const Rows out[] = {{"dq", dq, tokens, dq_stride, wq, g.elem}, {"dk", dk, tokens, dk_stride, wk, g.elem}};
    for (int i = 0; i < 2; i++)
        if ((s = check_rows(fn, grad[i])) != K6ATTN_OK || (s = check_rows(fn, in[i])) != K6ATTN_OK ||
            (s = check_rows(fn, out[i])) != K6ATTN_OK)
            return s;
    const size_t need = norm ? packed_norm_rope_bwd_workspace(g, tokens, h->sms) : 0;
    if (need && (!workspace || workspace_bytes < need))
        return set_error(K6ATTN_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", fn, need,
                         workspace ? workspace_bytes : (size_t)0);
    if (need && !aligned16(workspace)) return set_error(K6ATTN_ERR_INVALID_ARG, "%s: workspace misaligned", fn);
    const Rows wide[] = {flat("dq_weight", dq_weight, norm ? g.d * 4 : 0), flat("dk_weight", dk_weight, norm ? g.d * 4 : 0),
                         flat("the workspace", workspace, need)};
    const Rows fixed[] = {in[0],
                          in[1],
                          grad[0],
                          grad[1],
                          out[0],
                          out[1],
                          flat("the positions", positions, (size_t)tokens * 12),
                          flat("a weight", q_weight, norm ? g.d * 4 : 0),
                          flat("a weight", k_weight, norm ? g.d * 4 : 0),
                          flat("the offsets", cu, cu ? ((size_t)n_seq + 1) * 4 : 0)};
    if ((s = check_apart(fn, wide, 3, fixed, 10)) != K6ATTN_OK) return s;
    for (int i = 0; i < 2; i++) {
        const bool in_place = out[i].p == grad[i].p && out[i].stride == grad[i].stride;
        const Rows others[] = {in[0], in[1], grad[1 - i], in_place ? flat("", nullptr, 0) : grad[i], fixed[6], fixed[7],
                               fixed[8], fixed[9]};
        if ((s = check_apart(fn, out + i, 1, others, 8)) != K6ATTN_OK) return s;
    }
    if ((s = check_apart(fn, out, 2, nullptr, 0)) != K6ATTN_OK) return s;
    PackedNormRope p = {};
    p.tokens = tokens, p.Hkv = kv_heads, p.cu = cu, p.n_seq = n_seq, p.positions = positions, p.turns = h->turns;
    p.x[0] = q, p.x_stride[0] = q_stride, p.x[1] = k, p.x_stride[1] = k_stride;
    p.z[0] = const_cast<void *>(dq_out), p.z_stride[0] = dq_out_stride;
    p.z[1] = const_cast<void *>(dk_out), p.z_stride[1] = dk_out_stride;
    p.dx[0] = dq, p.dx_stride[0] = dq_stride, p.dx[1] = dk, p.dx_stride[1] = dk_stride;
    p.w[0] = q_weight, p.w[1] = k_weight, p.eps = eps, p.sms = h->sms, p.err = h->err;
    return cuda_check(launch_packed_norm_rope_bwd(g, p, dq_weight, dk_weight, workspace,
                                                  static_cast<cudaStream_t>(stream)),
                      "packed_norm_rope_backward launch");
}

size_t k6attn_packed_plan_bytes(k6attn_t h, const k6attn_packed *batch) {
    if (check_sizes("packed_plan_bytes", h, batch) != K6ATTN_OK) return 0;
    return packed_plan_bytes(packed_geom(h->g, *batch, h->sms));
}

k6attn_status k6attn_packed_plan(k6attn_t h, const k6attn_packed *batch, const int *cu_q, const int *cu_k, void *plan,
                                 size_t plan_bytes, void *stream) {
    const char *fn = "packed_plan";
    clear_error();
    k6attn_status s = check_batch(fn, h, batch);
    if (s != K6ATTN_OK) return s;
    if (!cu_q) return set_error(K6ATTN_ERR_INVALID_ARG, "%s: null cu_q", fn);
    if (!cu_k && batch->q_tokens != batch->k_tokens)
        return set_error(K6ATTN_ERR_INVALID_ARG, "%s: cu_k may be null only where q and k have the same tokens", fn);
    if ((reinterpret_cast<uintptr_t>(cu_q) | reinterpret_cast<uintptr_t>(cu_k)) & 3)
        return set_error(K6ATTN_ERR_INVALID_ARG, "%s: offsets must be 4-byte aligned", fn);
    const PackedGeom g = packed_geom(h->g, *batch, h->sms);
    if ((s = check_plan(fn, plan)) != K6ATTN_OK) return s;
    const size_t need = packed_plan_bytes(g);
    if (plan_bytes < need)
        return set_error(K6ATTN_ERR_WORKSPACE, "%s: plan of %zu bytes needed, %zu given", fn, need, plan_bytes);
    const size_t cu = ((size_t)batch->n_seq + 1) * 4;
    if (overlap(plan, need, cu_q, cu) || overlap(plan, need, cu_k, cu))
        return set_error(K6ATTN_ERR_INVALID_ARG, "%s: the plan overlaps the offsets", fn);
    return cuda_check(launch_packed_plan(g, cu_q, cu_k ? cu_k : cu_q, plan, h->err, static_cast<cudaStream_t>(stream)),
                      "packed_plan launch");
}

size_t k6attn_packed_workspace_bytes(k6attn_t h, const k6attn_packed *batch) {
    if (check_sizes("packed_workspace_bytes", h, batch) != K6ATTN_OK) return 0;
    return packed_fwd_workspace(packed_geom(h->g, *batch, h->sms));
}

k6attn_status k6attn_packed_forward(k6attn_t h, const k6attn_packed *batch, const void *plan, const void *q,
                                    long q_stride, const void *k, long k_stride, const void *v, long v_stride,
                                    k6attn_dtype qk_dtype, void *out, long out_stride, float *lse, void *workspace,
                                    size_t workspace_bytes, void *stream) {
    const char *fn = "packed_forward";
    clear_error();
    k6attn_status s = check_batch(fn, h, batch);
    if (s != K6ATTN_OK) return s;
    if (qk_dtype != K6ATTN_BF16 && qk_dtype != K6ATTN_F16)
        return set_error(K6ATTN_ERR_INVALID_ARG, "%s: q/k type must be BF16 or F16", fn);
    const PackedGeom g = packed_geom(h->g, *batch, h->sms);
    if ((s = check_plan(fn, plan)) != K6ATTN_OK) return s;
    const long wq = (long)g.H * 128, wk = (long)g.Hkv * 128;
    const size_t need = packed_fwd_workspace(g);
    if (need && (!workspace || workspace_bytes < need))
        return set_error(K6ATTN_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", fn, need,
                         workspace ? workspace_bytes : (size_t)0);
    if (need && !aligned16(workspace)) return set_error(K6ATTN_ERR_INVALID_ARG, "%s: workspace misaligned", fn);
    if (reinterpret_cast<uintptr_t>(lse) & 3) return set_error(K6ATTN_ERR_INVALID_ARG, "%s: lse misaligned", fn);
    const Rows in[] = {{"q", q, g.Tq, q_stride, wq, 2},
                       {"k", k, g.Tk, k_stride, wk, 2},
                       {"v", v, g.Tk, v_stride, wk, 2},
                       flat("the plan", plan, packed_plan_bytes(g))};
    const Rows out_[] = {{"out", out, g.Tq, out_stride, wq, 2},
                         flat("lse", lse, (size_t)g.Tq * g.H * 4),
                         flat("the workspace", workspace, need)};
    for (int i = 0; i < 3; i++)
        if ((s = check_rows(fn, in[i])) != K6ATTN_OK) return s;
    if ((s = check_rows(fn, out_[0])) != K6ATTN_OK || (s = check_apart(fn, out_, 3, in, 4)) != K6ATTN_OK) return s;
    const PackedPtrs t{q, k, v, q_stride, k_stride, v_stride, qk_dtype == K6ATTN_F16, plan, h->wait_limit_ns, h->err};
    const char *why = nullptr;
    const cudaError_t e = launch_packed_fwd(g, t, out, out_stride, lse, workspace, static_cast<cudaStream_t>(stream), &why);
    if (e != cudaSuccess && why) return set_error(K6ATTN_ERR_CUDA, "%s: %s", fn, why);
    return cuda_check(e, "packed_forward launch");
}

size_t k6attn_packed_backward_workspace_bytes(k6attn_t h, const k6attn_packed *batch) {
    if (check_sizes("packed_backward_workspace_bytes", h, batch) != K6ATTN_OK) return 0;
    return packed_bwd_workspace(packed_geom(h->g, *batch, h->sms));
}

k6attn_status k6attn_packed_backward(k6attn_t h, const k6attn_packed *batch, const void *plan, const void *q,
                                     long q_stride, const void *k, long k_stride, const void *v, long v_stride,
                                     k6attn_dtype qk_dtype, const void *out, long out_stride, const void *dout,
                                     long dout_stride, const float *lse, void *dq, long dq_stride, void *dk,
                                     long dk_stride, void *dv, long dv_stride, void *workspace,
                                     size_t workspace_bytes, void *stream) {
    const char *fn = "packed_backward";
    clear_error();
    k6attn_status s = check_batch(fn, h, batch);
    if (s != K6ATTN_OK) return s;
    if (qk_dtype != K6ATTN_BF16 && qk_dtype != K6ATTN_F16)
        return set_error(K6ATTN_ERR_INVALID_ARG, "%s: q/k type must be BF16 or F16", fn);
    const PackedGeom g = packed_geom(h->g, *batch, h->sms);
    if ((s = check_plan(fn, plan)) != K6ATTN_OK) return s;
    const long wq = (long)g.H * 128, wk = (long)g.Hkv * 128;
    const size_t need = packed_bwd_workspace(g);
    if (!workspace || workspace_bytes < need)
        return set_error(K6ATTN_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", fn, need,
                         workspace ? workspace_bytes : (size_t)0);
    if (!aligned16(workspace)) return set_error(K6ATTN_ERR_INVALID_ARG, "%s: workspace misaligned", fn);
    if (g.Tq && (!lse || (reinterpret_cast<uintptr_t>(lse) & 3)))
        return set_error(K6ATTN_ERR_INVALID_ARG, "%s: null or misaligned lse", fn);
    const Rows in[] = {{"q", q, g.Tq, q_stride, wq, 2},
                       {"k", k, g.Tk, k_stride, wk, 2},
                       {"v", v, g.Tk, v_stride, wk, 2},
                       {"out", out, g.Tq, out_stride, wq, 2},
                       {"dout", dout, g.Tq, dout_stride, wq, 2},
                       flat("lse", lse, (size_t)g.Tq * g.H * 4),
                       flat("the plan", plan, packed_plan_bytes(g))};
    const Rows grads[] = {{"dq", dq, g.Tq, dq_stride, wq, 2},
                          {"dk", dk, g.Tk, dk_stride, wk, 2},
                          {"dv", dv, g.Tk, dv_stride, wk, 2},
                          flat("the workspace", workspace, need)};
    for (int i = 0; i < 5; i++)
        if ((s = check_rows(fn, in[i])) != K6ATTN_OK) return s;
    for (int i = 0; i < 3; i++)
        if ((s = check_rows(fn, grads[i])) != K6ATTN_OK) return s;
    if ((s = check_apart(fn, grads, 4, in, 7)) != K6ATTN_OK) return s;
    const PackedPtrs t{q, k, v, q_stride, k_stride, v_stride, qk_dtype == K6ATTN_F16, plan, h->wait_limit_ns, h->err};
    const char *why = nullptr;
    const cudaError_t e = launch_packed_bwd(g, t, out, out_stride, dout, dout_stride, lse, dq, dq_stride, dk, dk_stride,
                                            dv, dv_stride, workspace, static_cast<cudaStream_t>(stream), &why);
    if (e != cudaSuccess && why) return set_error(K6ATTN_ERR_CUDA, "%s: %s", fn, why);
    return cuda_check(e, "packed_backward launch");
}

}  // extern "C"
