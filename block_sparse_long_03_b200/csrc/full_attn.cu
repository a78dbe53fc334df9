// full_attn.cu -- full causal attention of packed queries over packed or
// paged keys: the plan kernel, the merge of rows whose keys were split, and
// the CUDA-core kernel that serves fp32.
//
//   p(t) = L - T + t                  position of query t of a sequence
//   O[t, h, :] = sum_{j <= p(t)} softmax(scale Q[t, h] . K[j, g])_j V[j, g, :]
//   lse[t, h]  = log sum_{j <= p(t)} exp(scale Q[t, h] . K[j, g])
//
// with g = h / R.  The lengths are device data, so the cut of the work into
// items is made on the device too: one CTA checks the offsets, lengths and
// page ids, and writes each sequence's share of the item list.
#include <math.h>

#include <algorithm>

#include "full_attn.cuh"

namespace msa {
namespace {

// ---------------------------------------------------------------- plan

constexpr int kPlanThreads = 1024;

constexpr int kRowPages = 256;           // pages a warp looks at in one go
constexpr int kLongRows = 1024;

__device__ __forceinline__ int pages_of(int32_t L, int page_size) {
    return (int)(((uint32_t)L + (uint32_t)page_size - 1u) / (uint32_t)page_size);
}

// Marks the sequences b0 .. b0 + kSeqs - 1 that have a bad page id (k0 = -1; L
// is still being read).  A warp's lanes take 32 pages of each at a time, eight
// loads in flight.  Rows of more than `limit` pages are left out.
template <int kSeqs>
__device__ __forceinline__ void check_rows(const FullShape &s, const int32_t *table, FullSeq *seqs,
                                           int b0, int limit, int lane, uint32_t *err) {
    int n[kSeqs], most = 0;
#pragma unroll
    for (int j = 0; j < kSeqs; ++j) {
        n[j] = b0 + j < s.B ? pages_of(seqs[b0 + j].L, s.page_size) : 0;
        if (n[j] > limit) n[j] = 0;
        most = max(most, n[j]);
    }
    const int32_t *row = table + (int64_t)b0 * s.max_pages + lane;
    unsigned wrong = 0;
    for (int i0 = 0; i0 < most; i0 += 8 / kSeqs * 32) {
        int32_t pg[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int i = i0 + u / kSeqs * 32;
            pg[u] = i + lane < n[u % kSeqs] ? row[(int64_t)(u % kSeqs) * s.max_pages + i] : 0;
        }
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (pg[u] < 0 || pg[u] >= s.num_pages) wrong |= 1u << u % kSeqs;
    }
    wrong = __reduce_or_sync(0xffffffffu, wrong);
    if (lane < kSeqs && (wrong >> lane & 1)) {
        record_error(err, MSA_ERR_BAD_PAGE_TABLE, 3);
        seqs[b0 + lane].k0 = -1;
    }
}

// One CTA: checks what the device arrays say, sizes the key runs and numbers
// the items.  Latency is all it costs, so loads go out in batches: a warp
// takes one to eight short rows of the block table at a time, and the long
// ones are cut over all warps.
__global__ void __launch_bounds__(kPlanThreads)
full_plan_kernel(FullShape s, FullSeqs q, FullCut c, FullPlan *plan, FullSeq *seqs,
                 uint32_t *err) {
    __shared__ int64_t warp_sum[32];
    __shared__ int64_t total_tiles;
    __shared__ int32_t base, n_long;
    __shared__ int2 long_rows[kLongRows];          // sequence, pages
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    launch_next();
    if (tid < (int)(kErrorBytes / 4)) err[tid] = 0u;
    if (tid == 0) n_long = 0;
    // offsets: ascending, inside the arrays
    bool bad = false;
    for (int b = tid; b < s.B; b += kPlanThreads) {
        const int32_t lo = q.cu_q[b], hi = q.cu_q[b + 1];
        bad |= lo < 0 || hi < lo || hi > s.tokens;
        if (!s.paged) {
            const int32_t kl = q.cu_k[b], kh = q.cu_k[b + 1];
            bad |= kl < 0 || kh < kl || kh > s.key_tokens;
        }
    }
    if (__syncthreads_or(bad)) {
        if (tid == 0) {
            record_error(err, MSA_ERR_BAD_OFFSETS, 3);
            plan->items = 0;
            plan->invalid = 1;
            plan->next = 0;
        }
        return;
    }
    // lengths; a paged sequence with a length outside [T, capacity] or a bad
    // page id gets L = 0, and so does one without queries, whose length and
    // pages nothing reads (an idle slot may hold anything)
    for (int b = tid; b < s.B; b += kPlanThreads) {
        const int32_t q0 = q.cu_q[b], T = q.cu_q[b + 1] - q0;
        int32_t L, k0 = 0;
        if (s.paged) {
            L = T > 0 ? q.seq_lens[b] : 0;
            if (L < T || (int64_t)L > (int64_t)s.max_pages * s.page_size) {
                L = 0;
                record_error(err, MSA_ERR_BAD_PAGE_TABLE, 3);
            }
            const int n = pages_of(L, s.page_size);
            if (n > kRowPages) {
                const int i = atomicAdd(&n_long, 1);
                if (i < kLongRows) long_rows[i] = make_int2(b, n);
            }
        } else {
            k0 = q.cu_k[b];
            L = q.cu_k[b + 1] - k0;
        }
        seqs[b].q0 = q0;
        seqs[b].T = T;
        seqs[b].L = L;
        seqs[b].k0 = k0;
    }
    __syncthreads();
    if (s.paged) {
        const bool listed = n_long <= kLongRows;
        const int limit = listed ? kRowPages : 0x7fffffff;
        if (s.B > 128)
            for (int b = warp * 8; b < s.B; b += 256)
                check_rows<8>(s, q.block_table, seqs, b, limit, lane, err);
        else if (s.B > 64) {
            if (warp * 4 < s.B) check_rows<4>(s, q.block_table, seqs, warp * 4, limit, lane, err);
        } else if (s.B > 32) {
            if (warp * 2 < s.B) check_rows<2>(s, q.block_table, seqs, warp * 2, limit, lane, err);
        } else if (warp < s.B)
            check_rows<1>(s, q.block_table, seqs, warp, limit, lane, err);
        int turn = 0;                              // the warp whose turn it is
        for (int e = 0; listed && e < n_long; ++e) {
            const int2 r = long_rows[e];
            const int32_t *row = q.block_table + (int64_t)r.x * s.max_pages;
            const int pieces = (r.y + kRowPages - 1) / kRowPages;
            bool wrong = false;
            for (int p = (warp - turn) & 31; p < pieces; p += 32) {
                int32_t pg[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const int i = p * kRowPages + u * 32 + lane;
                    pg[u] = i < r.y ? row[i] : 0;
                }
#pragma unroll
                for (int u = 0; u < 8; ++u) wrong |= pg[u] < 0 || pg[u] >= s.num_pages;
            }
            if (__any_sync(0xffffffffu, wrong) && lane == 0) {
                record_error(err, MSA_ERR_BAD_PAGE_TABLE, 3);
                seqs[r.x].k0 = -1;
            }
            turn = (turn + pieces) & 31;
        }
        __syncthreads();
        for (int b = tid; b < s.B; b += kPlanThreads)
            if (seqs[b].k0 < 0) {
                seqs[b].L = 0;
                seqs[b].k0 = 0;
            }
    }
    // key tiles of all units, for the length of a key run
    int64_t mine = 0;
    for (int b = tid; b < s.B; b += kPlanThreads) {
        const int units = (seqs[b].T + c.unit_tokens - 1) / c.unit_tokens;
        mine += (int64_t)units * s.Hkv * ((seqs[b].L + kFullKeys - 1) / kFullKeys);
    }
    for (int off = 16; off > 0; off /= 2) mine += __shfl_xor_sync(0xffffffffu, mine, off);
    if (lane == 0) warp_sum[warp] = mine;
    if (tid == 0) base = 0;
    __syncthreads();
    if (tid == 0) {
        int64_t n = 0;
        for (int w = 0; w < 32; ++w) n += warp_sum[w];
        total_tiles = n;
    }
    __syncthreads();
    const int64_t run = c.split > 0 ? max((int64_t)c.min_tiles, (total_tiles + c.split - 1) / c.split)
                                    : (int64_t)1 << 30;
    // items of each sequence, and their running sum
    for (int b0 = 0; b0 < s.B; b0 += kPlanThreads) {
        const int b = b0 + tid;
        int n = 0;
        if (b < s.B) {
            const int tiles = (seqs[b].L + kFullKeys - 1) / kFullKeys;
            const int units = (seqs[b].T + c.unit_tokens - 1) / c.unit_tokens;
            int parts = (int)min((int64_t)max(1, c.max_parts), (tiles + run - 1) / run);
            parts = max(parts, 1);
            const int per = max(1, (tiles + parts - 1) / parts);
            seqs[b].units = units;
            seqs[b].parts = parts;
            seqs[b].tiles = per;
            n = units * parts * s.Hkv;
        }
        int sum = n;                               // inclusive over the warp, then the CTA
        for (int off = 1; off < 32; off *= 2) {
            const int o = __shfl_up_sync(0xffffffffu, sum, off);
            if (lane >= off) sum += o;
        }
        if (lane == 31) warp_sum[warp] = sum;
        __syncthreads();
        int before = base;
        for (int w = 0; w < warp; ++w) before += (int)warp_sum[w];
        if (b < s.B) seqs[b].first_item = before + sum - n;
        __syncthreads();
        if (tid == kPlanThreads - 1) base = before + sum;
        __syncthreads();
    }
    if (tid == 0) {
        plan->items = base;
        plan->invalid = 0;
        plan->next = 0;
    }
}

// ---------------------------------------------------------------- merge

constexpr int kMergeThreads = 256;

// Adds parts i0 .. i0 + N - 1 (in that order) to a row: lane i % 32 of mine
// holds part i's lse.  All N loads are in flight at once.
template <int N, int kPer>
__device__ __forceinline__ void add_parts(int i0, int parts, float mine, float m, const float *src,
                                          int64_t part_step, float &sum, float (&acc)[kPer]) {
    float l[N], x[N][kPer];
#pragma unroll
    for (int u = 0; u < N; ++u) {
        l[u] = __shfl_sync(0xffffffffu, mine, (i0 + u) % 32);
        if (i0 + u >= parts) l[u] = -INFINITY;
        // a part without weights for this row may have stored nothing
        const bool use = l[u] != -INFINITY;
        const float *p = src + (i0 + u) * part_step;
        if constexpr (kPer == 4) {
            const float4 v = use ? *(const float4 *)p : make_float4(0.f, 0.f, 0.f, 0.f);
            x[u][0] = v.x; x[u][1] = v.y; x[u][2] = v.z; x[u][3] = v.w;
        } else {
            const float2 v = use ? *(const float2 *)p : make_float2(0.f, 0.f);
            x[u][0] = v.x; x[u][1] = v.y;
        }
    }
#pragma unroll
    for (int u = 0; u < N; ++u) {
        const float w = l[u] == -INFINITY ? 0.f : expf(l[u] - m);
        sum += w;
#pragma unroll
        for (int k = 0; k < kPer; ++k) acc[k] = fmaf(w, x[u][k], acc[k]);
    }
}

// Rows of a token whose keys were split: weights exp(lse_i - max lse), summed
// in the order of the parts.  One warp a (token, head), lane l channels
// (D / 32) l ...; N parts' loads are in flight at a time (bound: HBM or L2,
// the partial results once; for few rows of many parts the loads' latency).
template <int D, int N>
__global__ void __launch_bounds__(kMergeThreads)
full_combine_kernel(FullShape s, FullSeqs q, FullCut c, const FullPlan *plan, const FullSeq *seqs,
                    const float *__restrict__ part_o, const float *__restrict__ part_lse,
                    __nv_bfloat16 *__restrict__ O, float *__restrict__ lse) {
    const int lane = threadIdx.x % 32;
    const int64_t row = ((int64_t)blockIdx.x * kMergeThreads + threadIdx.x) / 32;
    const int64_t step = s.tokens * s.Hq;
    wait_previous();
    if (row >= step || plan->invalid) return;
    const int64_t n = row / s.Hq;
    const int b = seq_of_token(q.cu_q, s.B, n);
    if (b >= s.B) return;
    const FullSeq sq = seqs[b];
    if (n < sq.q0) return;
    const int parts = full_row_parts(sq, c, (int)(n - sq.q0));
    if (parts == 0) return;
    constexpr int kPer = D / 32;
    // lane l holds the lse of part l, and in turn those of parts l + 32 ...
    // (loops, so that the code of a cold call stays small)
    const float *row_lse = part_lse + row;
    float mine = lane < parts ? row_lse[lane * step] : -INFINITY, m = mine;
#pragma unroll 1
    for (int i = 32 + lane; i < parts; i += 32) m = fmaxf(m, row_lse[i * step]);
    for (int off = 16; off > 0; off /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    float sum = 0.f, acc[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) acc[k] = 0.f;
    const float *src = part_o + row * D + lane * kPer;
#pragma unroll 1
    for (int i0 = 0; i0 < parts; i0 += N) {
        if (i0 > 0 && i0 % 32 == 0)
            mine = i0 + lane < parts ? row_lse[(i0 + lane) * step] : -INFINITY;
        add_parts<N>(i0, parts, mine, m, src, step * D, sum, acc);
    }
    if (m == kNanPart && sum == sum) {                 // no part has weights
        sum = 0.f;
#pragma unroll
        for (int k = 0; k < kPer; ++k) acc[k] = 0.f;
    }
    const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
    __nv_bfloat162 o[kPer / 2];
#pragma unroll
    for (int k = 0; k < kPer / 2; ++k)
        o[k] = __floats2bfloat162_rn(acc[2 * k] * inv, acc[2 * k + 1] * inv);
    if constexpr (kPer == 4) *(uint2 *)(O + row * D + lane * kPer) = *(const uint2 *)o;
    else *(uint32_t *)(O + row * D + lane * kPer) = *(const uint32_t *)o;
    if (lane == 0) lse[row] = sum == 0.f ? -INFINITY : m + logf(sum);
}

// ---------------------------------------------------------------- CUDA cores

constexpr int kSimtThreads = 128;
constexpr int kSimtRows = 64;              // rows = (token, head of the group) pairs
constexpr int kSimtKeys = 32;

// A CTA takes an item's rows: q in shared memory, keys 32 at a time.
// Scores: thread (y, x) owns rows 4 y .. 4 y + 3 and keys x, x + 8, x + 16,
// x + 24; softmax: two threads a row; values: rows 4 y .. and channels
// 4 x + 32 k ...  A score costs d multiply-adds from shared memory and so
// does a weight: 64 of them for each eight 16-byte reads.
template <int D>
__global__ void __launch_bounds__(kSimtThreads)
full_simt_kernel(FullShape s, FullSeqs sq, FullCut c, const FullPlan *plan, const FullSeq *seqs,
                 const float *__restrict__ Q, const float *__restrict__ K,
                 const float *__restrict__ V, float *__restrict__ O, float *__restrict__ lse) {
    constexpr int kLd = D + 4;
    extern __shared__ __align__(16) float sm[];
    float *qs = sm;                                        // [64][D + 4]
    float *ks = qs + kSimtRows * kLd;                      // [32][D + 4]
    float *vs = ks + kSimtKeys * kLd;                      // [32][D]
    float *ps = vs + kSimtKeys * D;                        // [64][36]
    float *alpha = ps + kSimtRows * 36;                    // [64]
    float *inv_l = alpha + kSimtRows;                      // [64]
    const int tid = threadIdx.x, lane = tid % 32;
    const int y = tid / 8, x = tid % 8;
    const int items = plan->items;
    int b = 0;
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
        b = full_find_seq(seqs, s.B, b, item, lane);
        const FullSeq q = seqs[b];
        const int local = item - q.first_item;
        const int g = local / q.units, u = q.units - 1 - local % q.units;
        const int t0 = u * c.unit_tokens, nt = min(c.unit_tokens, q.T - t0);
        const int rows = nt * s.R;
        const int pos0 = q.L - q.T + t0;                   // position of the first token
        const int last = pos0 + nt;                        // no row sees key `last` or later
        for (int i = tid; i < kSimtRows * (D / 4); i += kSimtThreads) {
            const int r = i / (D / 4), ch = (i % (D / 4)) * 4;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < rows) {
                const float *p = Q + (int64_t)(q.q0 + t0 + r / s.R) * s.q_stride +
                             (int64_t)(g * s.R + r % s.R) * D + ch;
                v = *(const float4 *)p;
            }
            *(float4 *)(qs + r * kLd + ch) = v;
        }
        float acc[4][D / 8];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int k = 0; k < D / 8; ++k) acc[i][k] = 0.f;
        float m = -INFINITY, l = 0.f;                      // of row tid / 2
        for (int j0 = 0; j0 < last; j0 += kSimtKeys) {
            __syncthreads();
            for (int i = tid; i < kSimtKeys * (D / 4); i += kSimtThreads) {
                const int r = i / (D / 4), ch = (i % (D / 4)) * 4;
                float4 kv = make_float4(0.f, 0.f, 0.f, 0.f), vv = kv;
                const int j = j0 + r;
                if (j < last) {
                    int64_t kr = (int64_t)q.k0 + j;
                    bool in = true;
                    if (s.paged) {
                        const int pg = sq.block_table[(int64_t)b * s.max_pages + j / s.page_size];
                        kr = (int64_t)pg * s.page_size + j % s.page_size;
                        in = MSA_IN_BOUNDS(kr, (int64_t)s.num_pages * s.page_size);
                    }
                    if (in) {
                        const float *kp = K + kr * s.k_stride + (int64_t)g * D + ch;
                        const float *vp = V + kr * s.v_stride + (int64_t)g * D + ch;
                        kv = *(const float4 *)kp;
                        vv = *(const float4 *)vp;
                    }
                }
                *(float4 *)(ks + r * kLd + ch) = kv;
                *(float4 *)(vs + r * D + ch) = vv;
            }
            __syncthreads();
            float sc[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) sc[i][k] = 0.f;
#pragma unroll 4
            for (int ch = 0; ch < D; ch += 4) {
                float4 qv[4], kv[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) qv[i] = *(const float4 *)(qs + (4 * y + i) * kLd + ch);
#pragma unroll
                for (int k = 0; k < 4; ++k) kv[k] = *(const float4 *)(ks + (x + 8 * k) * kLd + ch);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        sc[i][k] = fmaf(qv[i].x, kv[k].x, fmaf(qv[i].y, kv[k].y,
                                   fmaf(qv[i].z, kv[k].z, fmaf(qv[i].w, kv[k].w, sc[i][k]))));
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 4 * y + i, p = pos0 + r / s.R;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    ps[r * 36 + x + 8 * k] = j0 + x + 8 * k <= p ? sc[i][k] * s.scale : -INFINITY;
            }
            __syncthreads();
            {
                float *pr = ps + (tid / 2) * 36 + (tid % 2) * 16;
                float top = m;
#pragma unroll
                for (int k = 0; k < 16; ++k) top = fmaxf(top, pr[k]);
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                const float at = top == -INFINITY ? 0.f : top;
                float sum = 0.f;
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const float w = expf(pr[k] - at);
                    pr[k] = w;
                    sum += w;
                }
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                const float a = m == -INFINITY ? 0.f : expf(m - at);
                l = l * a + sum;
                m = top;
                if (tid % 2 == 0) alpha[tid / 2] = a;
            }
            __syncthreads();
            // The tile's weighted values are summed by themselves and then added:
            // one value after another onto the sum of 2^18 equal ones is 0.26 %
            // off, this way 0.002 to 0.005 %.
            float t[4][D / 8];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int k = 0; k < D / 8; ++k) t[i][k] = 0.f;
            // a tile that some row sees only in part: that row leaves the
            // later values out (they may be infinite or NaN)
            const bool whole = j0 + kSimtKeys <= pos0 + 1;
            // (unrolled whole the loop spills at D = 128: 2.1 ms for 512 tokens of 32
            // heads over 4096 keys, by eight 1.62)
#pragma unroll 8
            for (int j = 0; j < kSimtKeys; ++j) {
                float4 v[D / 32];
#pragma unroll
                for (int k = 0; k < D / 32; ++k) v[k] = *(const float4 *)(vs + j * D + 4 * x + 32 * k);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (!whole && j0 + j > pos0 + (4 * y + i) / s.R) continue;
                    const float w = ps[(4 * y + i) * 36 + j];
#pragma unroll
                    for (int k = 0; k < D / 32; ++k) {
                        t[i][4 * k] = fmaf(w, v[k].x, t[i][4 * k]);
                        t[i][4 * k + 1] = fmaf(w, v[k].y, t[i][4 * k + 1]);
                        t[i][4 * k + 2] = fmaf(w, v[k].z, t[i][4 * k + 2]);
                        t[i][4 * k + 3] = fmaf(w, v[k].w, t[i][4 * k + 3]);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float a = alpha[4 * y + i];
#pragma unroll
                for (int k = 0; k < D / 8; ++k) acc[i][k] = fmaf(acc[i][k], a, t[i][k]);
            }
        }
        if (tid % 2 == 0) {
            const int r = tid / 2;
            inv_l[r] = l == 0.f ? 0.f : 1.f / l;
            if (r < rows)
                lse[(int64_t)(q.q0 + t0 + r / s.R) * s.Hq + g * s.R + r % s.R] =
                    l == 0.f ? -INFINITY : m + logf(l);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 4 * y + i;
            if (r >= rows) continue;
            float *dst = O + ((int64_t)(q.q0 + t0 + r / s.R) * s.Hq + g * s.R + r % s.R) * D;
            const float inv = inv_l[r];
            // no weights (no key, or every score -infinity): 0, whatever the
            // values were
            if (inv == 0.f) {
#pragma unroll
                for (int k = 0; k < D / 8; ++k) acc[i][k] = 0.f;
            }
#pragma unroll
            for (int k = 0; k < D / 32; ++k)
                *(float4 *)(dst + 4 * x + 32 * k) =
                    make_float4(acc[i][4 * k] * inv, acc[i][4 * k + 1] * inv,
                                acc[i][4 * k + 2] * inv, acc[i][4 * k + 3] * inv);
        }
        __syncthreads();
    }
}

template <int D>
cudaError_t launch_simt(const FullShape &s, const FullSeqs &q, const FullCut &c,
                          const FullPlan *plan, const FullSeq *seqs, const void *Q, const void *K,
                          const void *V, void *O, float *lse, cudaStream_t st) {
    const size_t smem = sizeof(float) * ((size_t)(kSimtRows + kSimtKeys) * (D + 4) + kSimtKeys * D +
                                         kSimtRows * 36 + 2 * kSimtRows);
    auto k = full_simt_kernel<D>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const int64_t most = (s.tokens / c.unit_tokens + s.B) * s.Hkv;
    k<<<(unsigned)std::min<int64_t>(most, 148 * 3 * 16), kSimtThreads, smem, st>>>(
        s, q, c, plan, seqs, (const float *)Q, (const float *)K, (const float *)V, (float *)O, lse);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_full_plan(const FullShape &s, const FullSeqs &q, const FullCut &c,
                             FullPlan *plan, FullSeq *seqs, uint32_t *err, cudaStream_t st) {
    full_plan_kernel<<<1, kPlanThreads, 0, st>>>(s, q, c, plan, seqs, err);
    count_launches(1);
    return cudaGetLastError();
}

cudaError_t launch_full_combine(const FullShape &s, const FullSeqs &q, const FullCut &c,
                                const FullPlan *plan, const FullSeq *seqs, const float *part_o,
                                const float *part_lse, void *O, float *lse, cudaStream_t st) {
    // Up to 16 warps an SM, all resident at sixteen loads a lane in flight
    // (64 rows of 128 parts among 2048: 20 us; four loads: 33); beyond, four, which
    // leave room for 48 warps (a 2048-token step of 65 sequences: 415 us in
    // all; sixteen loads: 460).
    const int64_t warps = s.tokens * s.Hq;
    const bool few = warps <= 148 * 16;
    auto k = s.d == 64 ? (few ? full_combine_kernel<64, 16> : full_combine_kernel<64, 4>)
                       : (few ? full_combine_kernel<128, 16> : full_combine_kernel<128, 4>);
    count_launches(1);
    return launch_after(k, dim3((unsigned)((warps * 32 + kMergeThreads - 1) / kMergeThreads)),
                        dim3(kMergeThreads), 0, st, s, q, c, plan, seqs, part_o, part_lse,
                        (__nv_bfloat16 *)O, lse);
}

FullCut full_simt_cut(const FullShape &s) { return FullCut{kSimtRows / s.R, 0, 0, 1, 1, 0}; }

cudaError_t launch_full_simt(const FullShape &s, const FullSeqs &q, const FullCut &c,
                             const FullPlan *plan, const FullSeq *seqs, const void *Q,
                             const void *K, const void *V, void *O, float *lse, cudaStream_t st) {
    return s.d == 64 ? launch_simt<64>(s, q, c, plan, seqs, Q, K, V, O, lse, st)
                     : launch_simt<128>(s, q, c, plan, seqs, Q, K, V, O, lse, st);
}

}  // namespace msa
