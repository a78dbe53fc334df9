// serve_api.cu -- the C ABI's serving operators (include/msa.h): host-side
// validation, workspace layout and dispatch of the rotary positions, the
// paged cache write and the full causal attention.  Nothing here allocates
// device memory, and nothing is enqueued for a call that is refused.
#include <math.h>

#include <algorithm>

#include "full_attn.cuh"

namespace msa {
namespace {

constexpr size_t kAlign = 256;
size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
msa_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? MSA_OK : MSA_ERR_CUDA; }
int elem(int dtype) { return dtype == MSA_BF16 ? 2 : 4; }

// A token stride: 0 selects the dense one; tokens must not overlap and must
// stay 16-byte aligned, and every offset must fit 62 bits.
bool stride_ok(int64_t &stride, int64_t dense, int64_t tokens, int dtype) {
    if (stride == 0) stride = dense;
    if (stride < dense || (stride * elem(dtype)) % 16 != 0) return false;
    return (double)stride * (double)std::max<int64_t>(tokens, 1) < 4e18 / 4;
}

// Memory that a call reads or writes: n rows of `row` bytes, `step` bytes from
// one to the next.
struct Span {
    int64_t at, row, step, n;
    int64_t end() const { return at + (n - 1) * step + row; }
};
Span rows_of(const void *p, int64_t n, int64_t row, int64_t step) {
    if (p == nullptr || row <= 0) n = 0;
    if (step == row && n > 1) return Span{(int64_t)(uintptr_t)p, row * n, row * n, 1};
    return Span{(int64_t)(uintptr_t)p, row, step, n};
}
Span bytes_of(const void *p, double bytes) {             // (more than memory holds: as much as that)
    const int64_t n = (int64_t)std::min(bytes, (double)(1ll << 56));
    return rows_of(p, 1, n, n);
}
// Some row of b overlaps row i of a.
bool row_meets(const Span &a, int64_t i, const Span &b) {
    const int64_t x = a.at + i * a.step, past = x - b.at - b.row;
    const int64_t j = past < 0 ? 0 : past / b.step + 1;   // the first row of b that ends behind x
    return j < b.n && b.at + j * b.step < x + a.row;
}
// Two spans share a byte.  Slices of one fused tensor have equal steps: which
// rows meet depends on the distance of their numbers alone, and those of all
// distances are among the first row of one against the other.
bool overlap(const Span &a, const Span &b) {
    if (a.n <= 0 || b.n <= 0 || a.end() <= b.at || b.end() <= a.at) return false;
    if (a.step == b.step) return row_meets(a, 0, b) || row_meets(b, 0, a);
    if (a.n > b.n) return overlap(b, a);
    for (int64_t i = 0; i < a.n; ++i)
        if (row_meets(a, i, b)) return true;
    return false;
}
// An output overlaps an input or another output.
template <int kOut, int kIn>
bool outputs_overlap(const Span (&out)[kOut], const Span (&in)[kIn]) {
    for (int o = 0; o < kOut; ++o) {
        for (int i = 0; i < kIn; ++i)
            if (overlap(out[o], in[i])) return true;
        for (int i = 0; i < o; ++i)
            if (overlap(out[o], out[i])) return true;
    }
    return false;
}
// An output that overlaps its input is the input, with its stride.
bool in_place_or_apart(const Span &out, const Span &in) {
    return (out.at == in.at && out.row == in.row && out.step == in.step) || !overlap(out, in);
}

// Validate and convert the rotary parameters; Hq or Hkv becomes 0 where the
// tensor is NULL.
msa_status_t make_rope(const msa_rope_params_t *p, const void *Q, const void *Q_out, const void *K,
                       const void *K_out, const double *inv_freq, bool cache, RopeArgs *a) {
    if (p == nullptr) return MSA_ERR_INVALID_ARG;
    if (p->tokens < 0 || p->Hq <= 0 || p->Hkv <= 0 || p->d <= 0 || p->rot_dim <= 0 ||
        p->rot_dim > p->d || p->Hq > 1024 || p->Hkv > 1024)
        return MSA_ERR_INVALID_ARG;
    if (p->layout != MSA_ROPE_HALF && p->layout != MSA_ROPE_INTERLEAVED) return MSA_ERR_INVALID_ARG;
    if (p->dtype != MSA_F32 && p->dtype != MSA_BF16) return MSA_ERR_INVALID_ARG;
    if (p->inverse != 0 && p->inverse != 1) return MSA_ERR_INVALID_ARG;
    if (!isfinite(p->mscale)) return MSA_ERR_INVALID_ARG;
    if (p->d % 16 != 0 || p->d > 256 || p->rot_dim % 16 != 0) return MSA_ERR_UNSUPPORTED;
    if (p->tokens > 0x7fffffff) return MSA_ERR_UNSUPPORTED;
    if ((Q == nullptr) != (Q_out == nullptr) || (K == nullptr) != (K_out == nullptr) ||
        (Q == nullptr && K == nullptr) || inv_freq == nullptr)
        return MSA_ERR_INVALID_ARG;
    if (!aligned16(Q) || !aligned16(K) || !aligned16(Q_out) || !aligned16(K_out) ||
        ((uintptr_t)inv_freq & 7u) != 0)
        return MSA_ERR_INVALID_ARG;
    a->q_stride = p->q_stride; a->k_stride = p->k_stride;
    a->qo_stride = p->q_out_stride; a->ko_stride = cache ? 0 : p->k_out_stride;
    const int64_t dq = (int64_t)p->Hq * p->d, dk = (int64_t)p->Hkv * p->d;
    if (Q != nullptr && (!stride_ok(a->q_stride, dq, p->tokens, p->dtype) ||
                         !stride_ok(a->qo_stride, dq, p->tokens, p->dtype)))
        return MSA_ERR_INVALID_ARG;
    if (K != nullptr && (!stride_ok(a->k_stride, dk, p->tokens, p->dtype) ||
                         !stride_ok(a->ko_stride, dk, p->tokens, p->dtype)))
        return MSA_ERR_INVALID_ARG;
    if ((Q != nullptr && Q == Q_out && a->q_stride != a->qo_stride) ||
        (K != nullptr && K == K_out && a->k_stride != a->ko_stride))
        return MSA_ERR_INVALID_ARG;
    a->Q = Q; a->K = K; a->Q_out = (void *)Q_out; a->K_out = (void *)K_out;
    a->positions = nullptr;
    a->inv_freq = inv_freq;
    a->tokens = p->tokens;
    a->Hq = Q ? p->Hq : 0;
    a->Hkv = K ? p->Hkv : 0;
    a->d = p->d; a->rot = p->rot_dim; a->inverse = p->inverse;
    a->mscale = p->mscale;
    return MSA_OK;
}

// The tokens of a call with such parameters.
struct RopeSpans {
    Span q, k, q_out, k_out;
    RopeSpans(const RopeArgs &a, int dtype) {
        const int64_t e = elem(dtype), dq = (int64_t)a.Hq * a.d * e, dk = (int64_t)a.Hkv * a.d * e;
        q = rows_of(a.Q, a.tokens, dq, a.q_stride * e);
        k = rows_of(a.K, a.tokens, dk, a.k_stride * e);
        q_out = rows_of(a.Q_out, a.tokens, dq, a.qo_stride * e);
        k_out = rows_of(a.K_out, a.tokens, dk, a.ko_stride * e);
    }
};

// Validate an attention call's sizes.
msa_status_t make_full(const msa_attn_params_t *p, bool paged, FullShape *s) {
    if (p == nullptr) return MSA_ERR_INVALID_ARG;
    if (p->tokens < 0 || p->B <= 0 || p->Hq <= 0 || p->Hkv <= 0 || p->d <= 0 ||
        p->Hq % p->Hkv != 0 || (!paged && p->key_tokens < 0))
        return MSA_ERR_INVALID_ARG;
    if (p->dtype != MSA_F32 && p->dtype != MSA_BF16) return MSA_ERR_INVALID_ARG;
    if (!(p->scale == p->scale) || isinf(p->scale)) return MSA_ERR_INVALID_ARG;
    if (paged && (p->page_size <= 0 || p->max_pages <= 0 || p->num_pages <= 0))
        return MSA_ERR_INVALID_ARG;
    if (p->d != 64 && p->d != 128) return MSA_ERR_UNSUPPORTED;
    if (p->Hq / p->Hkv > 64 || p->Hq > 1024 || p->B > (1 << 20)) return MSA_ERR_UNSUPPORTED;
    if (p->tokens > 0x7fffff00ll || (!paged && p->key_tokens > 0x7fffff00ll))
        return MSA_ERR_UNSUPPORTED;
    // key positions are 32-bit, cache rows too (they are TMA coordinates)
    if (paged && ((int64_t)p->max_pages * p->page_size > 0x7fffff00ll ||
                  (int64_t)p->num_pages * p->page_size > 0x7fffff00ll))
        return MSA_ERR_UNSUPPORTED;
    if (paged && p->dtype == MSA_BF16 && p->page_size % 8 != 0) return MSA_ERR_UNSUPPORTED;
    s->tokens = p->tokens;
    s->key_tokens = paged ? (int64_t)p->num_pages * p->page_size : p->key_tokens;
    s->B = p->B; s->Hq = p->Hq; s->Hkv = p->Hkv; s->R = p->Hq / p->Hkv; s->d = p->d;
    s->dtype = p->dtype;
    s->scale = p->scale > 0.f ? p->scale : 1.0f / sqrtf((float)p->d);
    s->q_stride = p->q_stride;
    s->k_stride = paged ? 0 : p->k_stride;
    s->v_stride = paged ? 0 : p->v_stride;
    const int64_t dq = (int64_t)s->Hq * s->d, dk = (int64_t)s->Hkv * s->d;
    if (!stride_ok(s->q_stride, dq, s->tokens, s->dtype) ||
        !stride_ok(s->k_stride, dk, s->key_tokens, s->dtype) ||
        !stride_ok(s->v_stride, dk, s->key_tokens, s->dtype))
        return MSA_ERR_INVALID_ARG;
    // the strides of a tensor map are under 2^40 bytes
    if (s->dtype == MSA_BF16 && std::max({s->q_stride, s->k_stride, s->v_stride}) * 2 >= 1ll << 40)
        return MSA_ERR_UNSUPPORTED;
    s->paged = paged;
    s->page_size = p->page_size; s->max_pages = p->max_pages; s->num_pages = p->num_pages;
    return MSA_OK;
}

FullCut full_cut(const FullShape &s) {
    return s.dtype == MSA_BF16 ? full_tc_cut(s) : full_simt_cut(s);
}

// Workspace: [error word][plan][sequences][partial O][partial lse][sums of long runs' pieces]
struct FullLayout {
    size_t plan, seqs, part_o, part_lse, carry, total;
};
FullLayout full_layout(const FullShape &s, const FullCut &c) {
    FullLayout L;
    size_t o = kErrorBytes;
    L.plan = o;     o += kPlanBytes;
    L.seqs = o;     o += align_up(sizeof(FullSeq) * (size_t)s.B);
    const size_t rows = c.max_parts > 1 ? (size_t)c.max_parts * 2 * s.tokens * s.Hq : 0;
    L.part_o = o;   o += align_up(rows * s.d * sizeof(float));
    L.part_lse = o; o += align_up(rows * sizeof(float));
    L.carry = o;     o += align_up(c.carry_floats * sizeof(float));
    L.total = o;
    return L;
}

// Items of the plan fit 31 bits.
bool full_items_fit(const FullShape &s, const FullCut &c) {
    const double units = (double)s.tokens / c.unit_tokens + s.B;
    return units * s.Hkv * c.max_parts < 2.0e9;
}

msa_status_t run_full(const msa_attn_params_t *params, bool paged, const void *Q, const void *K,
                      const void *V, const FullSeqs &q, void *O, float *lse, void *workspace,
                      size_t workspace_bytes, void *stream) {
    FullShape s;
    const msa_status_t rc = make_full(params, paged, &s);
    if (rc != MSA_OK) return rc;
    if (!q.cu_q || (paged ? (!q.seq_lens || !q.block_table) : !q.cu_k)) return MSA_ERR_INVALID_ARG;
    if (s.tokens > 0 && (!Q || !O || !lse)) return MSA_ERR_INVALID_ARG;
    if (s.key_tokens > 0 && (!K || !V)) return MSA_ERR_INVALID_ARG;
    if (!aligned16(Q) || !aligned16(K) || !aligned16(V) || !aligned16(O) || !aligned16(lse) ||
        ((uintptr_t)q.cu_q & 3u) || ((uintptr_t)q.cu_k & 3u) || ((uintptr_t)q.seq_lens & 3u) ||
        ((uintptr_t)q.block_table & 3u))
        return MSA_ERR_INVALID_ARG;
    const FullCut c = full_cut(s);
    if (!full_items_fit(s, c)) return MSA_ERR_UNSUPPORTED;
    const FullLayout L = full_layout(s, c);
    if (!workspace || ((uintptr_t)workspace % kAlign) != 0 || workspace_bytes < L.total)
        return MSA_ERR_WORKSPACE;
    // a row may be written while another row's inputs are still read
    const int64_t e = elem(s.dtype), dq = (int64_t)s.Hq * s.d * e, dk = (int64_t)s.Hkv * s.d * e;
    const Span out[] = {bytes_of(O, (double)s.tokens * dq), bytes_of(lse, 4.0 * s.tokens * s.Hq),
                        bytes_of(workspace, (double)L.total)};
    const Span in[] = {rows_of(Q, s.tokens, dq, s.q_stride * e),
                       rows_of(K, s.key_tokens, dk, s.k_stride * e),
                       rows_of(V, s.key_tokens, dk, s.v_stride * e),
                       bytes_of(q.cu_q, 4.0 * (s.B + 1)), bytes_of(q.cu_k, 4.0 * (s.B + 1)),
                       bytes_of(q.seq_lens, 4.0 * s.B),
                       bytes_of(q.block_table, 4.0 * s.B * s.max_pages)};
    if (outputs_overlap(out, in)) return MSA_ERR_INVALID_ARG;
    char *ws = (char *)workspace;
    uint32_t *err = (uint32_t *)ws;
    FullPlan *plan = (FullPlan *)(ws + L.plan);
    FullSeq *seqs = (FullSeq *)(ws + L.seqs);
    cudaStream_t st = (cudaStream_t)stream;
    cudaError_t done = launch_full_plan(s, q, c, plan, seqs, err, st);
    if (s.tokens == 0) return cuda_status(done);
    if (s.dtype == MSA_F32) {
        if (done == cudaSuccess) done = launch_full_simt(s, q, c, plan, seqs, Q, K, V, O, lse, st);
        return cuda_status(done);
    }
    float *part_o = (float *)(ws + L.part_o), *part_lse = (float *)(ws + L.part_lse);
    if (done == cudaSuccess)
        done = launch_full_tc(s, q, c, plan, seqs, Q, K, V, O, lse, part_o, part_lse,
                              (float *)(ws + L.carry), err, st);
    if (done == cudaSuccess && c.max_parts > 1)
        done = launch_full_combine(s, q, c, plan, seqs, part_o, part_lse, O, lse, st);
    return cuda_status(done);
}

}  // namespace
}  // namespace msa

using namespace msa;

extern "C" {

msa_status_t msa_rope_frequencies(int32_t rot_dim, double base, int32_t scaling, double factor,
                                  double context, double slow, double fast, double *inv_freq) {
    if (inv_freq == nullptr || rot_dim < 2 || rot_dim % 2 != 0 || !(base > 1.0) || isinf(base))
        return MSA_ERR_INVALID_ARG;
    if (scaling < MSA_ROPE_SCALE_NONE || scaling > MSA_ROPE_SCALE_PARTS) return MSA_ERR_INVALID_ARG;
    if (scaling != MSA_ROPE_SCALE_NONE && (!(factor > 0.0) || isinf(factor)))
        return MSA_ERR_INVALID_ARG;
    if (scaling == MSA_ROPE_SCALE_BASE && rot_dim < 4) return MSA_ERR_INVALID_ARG;
    if (scaling == MSA_ROPE_SCALE_PARTS &&
        (!(context > 0.0) || !(slow >= 0.0) || !(fast > slow) || isinf(fast) || isinf(context)))
        return MSA_ERR_INVALID_ARG;
    if (scaling == MSA_ROPE_SCALE_BASE)
        base *= pow(factor, (double)rot_dim / (double)(rot_dim - 2));
    for (int i = 0; i < rot_dim / 2; ++i) {
        double f = pow(base, -2.0 * i / rot_dim);
        if (scaling == MSA_ROPE_SCALE_LINEAR) f /= factor;
        if (scaling == MSA_ROPE_SCALE_PARTS) {
            const double turns = context * f / 6.283185307179586;
            const double w = std::min(1.0, std::max(0.0, (turns - slow) / (fast - slow)));
            f = w * f + (1.0 - w) * (f / factor);
        }
        inv_freq[i] = f;
    }
    return MSA_OK;
}

msa_status_t msa_rope(const msa_rope_params_t *params, const void *Q, const void *K,
                      const int32_t *positions, const double *inv_freq, void *Q_out, void *K_out,
                      void *stream) {
    RopeArgs a;
    const msa_status_t rc = make_rope(params, Q, Q_out, K, K_out, inv_freq, false, &a);
    if (rc != MSA_OK) return rc;
    if (positions == nullptr || ((uintptr_t)positions & 3u) != 0) return MSA_ERR_INVALID_ARG;
    a.positions = positions;
    const RopeSpans r(a, params->dtype);
    const Span out[] = {r.q_out, r.k_out};
    const Span in[] = {bytes_of(positions, 4.0 * a.tokens), bytes_of(inv_freq, 4.0 * a.rot)};
    if (a.tokens > 0 &&
        (outputs_overlap(out, in) || !in_place_or_apart(r.q_out, r.q) ||
         !in_place_or_apart(r.k_out, r.k) || overlap(r.q_out, r.k) || overlap(r.k_out, r.q)))
        return MSA_ERR_INVALID_ARG;
    return cuda_status(launch_rope(a, params->dtype, params->layout == MSA_ROPE_INTERLEAVED,
                                   (cudaStream_t)stream));
}

msa_status_t msa_rope_append_paged(
    const msa_rope_params_t *params, int32_t B, const int32_t *cu_seqlens,
    const int32_t *seq_lens, const int32_t *block_table, int32_t page_size, int32_t max_pages,
    int32_t num_pages, const void *Q, const void *K, const void *V, int64_t v_stride,
    const void *k_idx, int32_t d_idx, const double *inv_freq, void *Q_out, void *K_cache,
    void *V_cache, void *k_idx_cache, void *workspace, size_t workspace_bytes, void *stream) {
    RopeArgs a;
    const bool none = params != nullptr && params->tokens == 0;   // tokens' pointers may be NULL
    msa_rope_params_t dense;
    if (none) {
        dense = *params;
        dense.q_stride = dense.q_out_stride = dense.k_stride = v_stride = 0;
        params = &dense;
        Q = Q_out = nullptr;
        if (K == nullptr) K = K_cache;
        if (V == nullptr) V = V_cache;
    }
    const msa_status_t rc = make_rope(params, Q, Q_out, K, K_cache, inv_freq, true, &a);
    if (rc != MSA_OK) return rc;
    if (params->inverse != 0 || B <= 0 || page_size <= 0 || max_pages <= 0 || num_pages <= 0)
        return MSA_ERR_INVALID_ARG;
    if (!cu_seqlens || !seq_lens || !block_table || !K || !V || !V_cache) return MSA_ERR_INVALID_ARG;
    if ((k_idx == nullptr) != (k_idx_cache == nullptr) && !(none && k_idx == nullptr))
        return MSA_ERR_INVALID_ARG;
    if (k_idx != nullptr && d_idx <= 0) return MSA_ERR_INVALID_ARG;
    if (!aligned16(V) || !aligned16(V_cache) || !aligned16(k_idx) || !aligned16(k_idx_cache) ||
        ((uintptr_t)cu_seqlens & 3u) || ((uintptr_t)seq_lens & 3u) || ((uintptr_t)block_table & 3u))
        return MSA_ERR_INVALID_ARG;
    if (!stride_ok(v_stride, (int64_t)params->Hkv * params->d, params->tokens, params->dtype))
        return MSA_ERR_INVALID_ARG;
    if (k_idx != nullptr && (d_idx % 16 != 0 || d_idx > 128)) return MSA_ERR_UNSUPPORTED;
    // sequences and key positions are counted in 32 bits, in steps of 256 and 32
    if (B > 0x7fffff00 || (int64_t)max_pages * page_size > 0x7fffff00ll) return MSA_ERR_UNSUPPORTED;
    if (!workspace || ((uintptr_t)workspace % kAlign) != 0 || workspace_bytes < kErrorBytes)
        return MSA_ERR_WORKSPACE;
    const RopeSpans r(a, params->dtype);
    const int64_t e = elem(params->dtype), dk = (int64_t)params->Hkv * params->d * e, n = a.tokens;
    const double rows = (double)num_pages * page_size;
    const Span out[] = {r.q_out, bytes_of(K_cache, rows * dk), bytes_of(V_cache, rows * dk),
                        bytes_of(k_idx_cache, rows * d_idx * e), bytes_of(workspace, kErrorBytes)};
    const Span in[] = {r.k, rows_of(V, n, dk, v_stride * e),
                       bytes_of(k_idx, (double)n * d_idx * e), bytes_of(cu_seqlens, 4.0 * (B + 1.0)),
                       bytes_of(seq_lens, 4.0 * B), bytes_of(block_table, 4.0 * B * max_pages),
                       bytes_of(inv_freq, 4.0 * a.rot)};
    if (outputs_overlap(out, in) || !in_place_or_apart(r.q_out, r.q)) return MSA_ERR_INVALID_ARG;
    for (int i = 1; i < 5; ++i)
        if (overlap(out[i], r.q)) return MSA_ERR_INVALID_ARG;
    AppendArgs c;
    c.cu_seqlens = cu_seqlens; c.seq_lens = seq_lens; c.block_table = block_table;
    c.V = V; c.k_idx = k_idx; c.V_cache = V_cache; c.k_idx_cache = k_idx_cache;
    c.v_stride = v_stride;
    c.B = B; c.page_size = page_size; c.max_pages = max_pages; c.num_pages = num_pages;
    c.d_idx = k_idx ? d_idx : 0;
    c.err = (uint32_t *)workspace;
    return cuda_status(launch_rope_append(a, c, params->dtype,
                                          params->layout == MSA_ROPE_INTERLEAVED,
                                          (cudaStream_t)stream));
}

size_t msa_attn_workspace_size(const msa_attn_params_t *params, int paged) {
    FullShape s;
    if (make_full(params, paged != 0, &s) != MSA_OK) return 0;
    const FullCut c = full_cut(s);
    return full_items_fit(s, c) ? full_layout(s, c).total : 0;
}

msa_status_t msa_attn_packed(const msa_attn_params_t *params, const void *Q, const void *K,
                             const void *V, const int32_t *cu_seqlens_q,
                             const int32_t *cu_seqlens_k, void *O, float *lse, void *workspace,
                             size_t workspace_bytes, void *stream) {
    const FullSeqs q{cu_seqlens_q, cu_seqlens_k, nullptr, nullptr};
    return run_full(params, false, Q, K, V, q, O, lse, workspace, workspace_bytes, stream);
}

msa_status_t msa_attn_paged(const msa_attn_params_t *params, const void *Q, const void *K_cache,
                            const void *V_cache, const int32_t *cu_seqlens,
                            const int32_t *seq_lens, const int32_t *block_table, void *O,
                            float *lse, void *workspace, size_t workspace_bytes, void *stream) {
    const FullSeqs q{cu_seqlens, nullptr, seq_lens, block_table};
    return run_full(params, true, Q, K_cache, V_cache, q, O, lse, workspace, workspace_bytes,
                    stream);
}

}  // extern "C"
