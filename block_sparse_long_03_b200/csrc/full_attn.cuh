// full_attn.cuh -- what the translation units of the full (not block-sparse)
// causal attention share: the call's sizes, the plan that a first kernel
// writes into the workspace, and how a work item is read from it.
#pragma once

#include "msa_internal.cuh"

namespace msa {

// Sizes of one call after host-side validation.
struct FullShape {
    int64_t tokens, key_tokens;          // rows of Q; rows of packed K and V
    int B, Hq, Hkv, R, d, dtype;
    float scale;                         // resolved softmax scale
    int64_t q_stride, k_stride, v_stride;   // elements between tokens
    bool paged;
    int page_size, max_pages, num_pages;
};

// What the caller's device arrays say about the sequences: queries of
// sequence b are rows [cu_q[b], cu_q[b + 1]) of Q; its keys are rows
// [cu_k[b], cu_k[b + 1]) of K and V (packed) or the seq_lens[b] first rows
// of its pages (paged).
struct FullSeqs {
    const int32_t *cu_q, *cu_k, *seq_lens, *block_table;
};

// One sequence of the plan: its queries q0 .. q0 + T of Q at the last T of L
// positions, its first key row (packed), and how its work is cut: `units`
// runs of consecutive queries, each over `parts` runs of `tiles` key tiles.
// A sequence with L = 0 attends nothing (also one whose pages are invalid).
struct FullSeq {
    int32_t q0, T, L, k0, units, parts, tiles, first_item;
};

// Plan header, in the workspace after the error word.  Items are numbered
// through the sequences: item first_item[b] + ((g * parts + part) * units + u)
// is KV head g, key run `part` and query run units - 1 - u of sequence b
// (late queries, which see the most keys, first).
struct FullPlan {
    int32_t items, invalid;              // invalid: the offsets are unusable, no row is written
    int32_t next;                        // items handed out beyond each CTA's first
};
constexpr size_t kPlanBytes = 256;

constexpr int kFullKeys = 128;           // keys of a tile
constexpr int kMaxParts = 64;            // key runs of a unit, at most (twice as many partial
                                         // results where two row tiles share a run)

// How a kernel's tiles cut the work: unit_tokens queries a unit; with
// split > 0 the key runs are sized for about `split` items in all, at most
// max_parts runs a unit.
struct FullCut {
    int unit_tokens, half_tokens, split, max_parts, min_tiles;
    size_t carry_floats;                  // workspace for the sums carried along key runs
};

// Key runs that the partial results of a row of sequence s are kept for: 0
// where its output is written directly.  A unit of at most half_tokens
// queries takes one of the kernel's two row tiles; the second then takes
// half of the key run.
__host__ __device__ __forceinline__ int full_row_parts(const FullSeq &s, const FullCut &c, int t) {
    const int u = t / c.unit_tokens;
    const bool half = c.half_tokens > 0 && s.T - u * c.unit_tokens <= c.half_tokens;
    const int n = s.parts * (half && c.max_parts > 1 ? 2 : 1);
    return n > 1 ? n : 0;
}

// The lse of a partial result whose weights are all 0 and whose O has a NaN (0
// times an infinite value): the merge has to see it where other parts have
// weights.  -infinity: nothing to add, and nothing may be stored.
constexpr float kNanPart = -3.402823466e+38f;

cudaError_t launch_full_plan(const FullShape &s, const FullSeqs &q, const FullCut &c,
                             FullPlan *plan, FullSeq *seqs, uint32_t *err, cudaStream_t st);
// O and lse of the rows kept in parts: part_o [parts, tokens, Hq, d] fp32
// (normalised) and part_lse [parts, tokens, Hq].
cudaError_t launch_full_combine(const FullShape &s, const FullSeqs &q, const FullCut &c,
                                const FullPlan *plan, const FullSeq *seqs, const float *part_o,
                                const float *part_lse, void *O, float *lse, cudaStream_t st);

// CUDA-core kernel (fp32).
FullCut full_simt_cut(const FullShape &s);
cudaError_t launch_full_simt(const FullShape &s, const FullSeqs &q, const FullCut &c,
                             const FullPlan *plan, const FullSeq *seqs, const void *Q,
                             const void *K, const void *V, void *O, float *lse, cudaStream_t st);

// Tensor-core kernel (bf16, full_attn_tc.cu).
FullCut full_tc_cut(const FullShape &s);
cudaError_t launch_full_tc(const FullShape &s, const FullSeqs &q, const FullCut &c,
                           const FullPlan *plan, const FullSeq *seqs, const void *Q,
                           const void *K, const void *V, void *O, float *lse, float *part_o,
                           float *part_lse, float *carry, uint32_t *err, cudaStream_t st);

// The call's kernels follow one another closely (programmatic dependent
// launch): the next one may be set up as soon as every block of this one has
// called launch_next() or ended, and waits in wait_previous() until this one
// has ended and its writes are visible; before that it touches no memory that
// another kernel of the call writes.
__device__ __forceinline__ void launch_next() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_previous() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
template <typename... P, typename... A>
cudaError_t launch_after(void (*k)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                         A... args) {
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, static_cast<P>(args)...);
}

// The sequence that item `i` belongs to, searched from sequence b on (items
// are visited in ascending order), by one warp.
__device__ __forceinline__ int full_find_seq(const FullSeq *seqs, int B, int b, int i, int lane) {
    while (true) {
        const int x = b + 1 + lane;
        const bool later = x >= B || seqs[x].first_item > i;
        const unsigned m = __ballot_sync(0xffffffffu, later);
        if (m) return b + __ffs(m) - 1;
        b += 32;
    }
}

}  // namespace msa
