// rope.cu -- rotary positions, and rotary positions with the write of new
// tokens into the paged caches.
//
// A head's first rot channels are taken as rot/2 pairs (x_i, x_{i+rot/2}) or
// (x_{2i}, x_{2i+1}); pair i of a token at position p is turned by the angle
// p * theta_i and scaled:
//   y_a = mscale (x_a cos - x_b sin),   y_b = mscale (x_b cos + x_a sin)
// (the transposed turn negates the sine); the other channels are copied.
//
// Bound: HBM.  Every value is read and written once and costs three
// operations; the only other work is one cosine and sine per (token, pair),
// shared by all heads.  So one CTA takes one token: its rot/2 cosines and
// sines go to shared memory first, then its threads stream all of the
// token's heads, 16 bytes (bf16) a load.
//
// Angles: p * theta is reduced to a part of a turn in fp64 (at p = 2^20 an
// fp32 product would be off by up to 0.06 radians), and the remainder, at
// most half a turn, is rounded to fp32 for sincospif: an error of at most
// 2^-25 turns, 2e-7 radians, at every position.
#include <math.h>

#include "msa_internal.cuh"

namespace msa {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxHalf = 128;                 // pairs of a head (rot <= 256)

// Eight channels as fp32.
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&x)[8]) {
    const uint4 u = *(const uint4 *)p;
    const __nv_bfloat162 *h = (const __nv_bfloat162 *)&u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __bfloat1622float2(h[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ void load8(const float *p, float (&x)[8]) {
    *(float4 *)x = *(const float4 *)p;
    *(float4 *)(x + 4) = *(const float4 *)(p + 4);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&x)[8]) {
    uint4 u;
    __nv_bfloat162 *h = (__nv_bfloat162 *)&u;
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    *(uint4 *)p = u;
}
__device__ __forceinline__ void store8(float *p, const float (&x)[8]) {
    *(float4 *)p = *(const float4 *)x;
    *(float4 *)(p + 4) = *(const float4 *)(x + 4);
}
__device__ __forceinline__ void copy8(__nv_bfloat16 *d, const __nv_bfloat16 *s) {
    *(uint4 *)d = *(const uint4 *)s;
}
__device__ __forceinline__ void copy8(float *d, const float *s) {
    const uint4 a = *(const uint4 *)s, b = *(const uint4 *)(s + 4);
    *(uint4 *)d = a;
    *(uint4 *)(d + 4) = b;
}

// Unit u of a head: its first rot/16 (halves) or rot/8 (side by side) units
// turn 8 or 4 pairs, the following ones copy eight channels each.  A unit's
// values are all read before any is written, so in and out may be the same.
template <typename T, bool kSide>
__device__ __forceinline__ void turn_unit(const T *in, T *out, int u, int rot, const float2 *cs) {
    if (kSide) {
        if (8 * u >= rot) {
            copy8(out + 8 * u, in + 8 * u);
            return;
        }
        float x[8];
        load8(in + 8 * u, x);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 t = cs[4 * u + i];
            const float a = x[2 * i], b = x[2 * i + 1];
            x[2 * i] = a * t.x - b * t.y;
            x[2 * i + 1] = b * t.x + a * t.y;
        }
        store8(out + 8 * u, x);
    } else {
        const int turned = rot / 16;
        if (u >= turned) {
            const int c = rot + 8 * (u - turned);
            copy8(out + c, in + c);
            return;
        }
        float a[8], b[8];
        load8(in + 8 * u, a);
        load8(in + rot / 2 + 8 * u, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 t = cs[8 * u + i];
            const float x = a[i], y = b[i];
            a[i] = x * t.x - y * t.y;
            b[i] = y * t.x + x * t.y;
        }
        store8(out + 8 * u, a);
        store8(out + rot / 2 + 8 * u, b);
    }
}

// mscale times the cosine and (signed) sine of each pair's angle at position p.
__device__ __forceinline__ void fill_turns(float2 *cs, int64_t p, const double *inv_freq, int half,
                                           float mscale, bool inverse) {
    for (int i = threadIdx.x; i < half; i += kThreads) {
        double turns = (double)p * (inv_freq[i] * 0.15915494309189535);   // 1 / (2 pi)
        turns -= rint(turns);
        float s, c;
        sincospif(2.f * (float)turns, &s, &c);
        cs[i] = make_float2(mscale * c, mscale * (inverse ? -s : s));
    }
}

template <typename T, bool kSide>
__global__ void __launch_bounds__(kThreads)
rope_kernel(RopeArgs a) {
    __shared__ float2 cs[kMaxHalf];
    const int64_t n = blockIdx.x;
    fill_turns(cs, a.positions[n], a.inv_freq, a.rot / 2, a.mscale, a.inverse);
    __syncthreads();
    const T *q = (const T *)a.Q + n * a.q_stride, *k = (const T *)a.K + n * a.k_stride;
    T *qo = (T *)a.Q_out + n * a.qo_stride, *ko = (T *)a.K_out + n * a.ko_stride;
    const int per = kSide ? a.d / 8 : a.rot / 16 + (a.d - a.rot) / 8;      // units of a head
    const int nq = a.Hq * per, total = nq + a.Hkv * per;
    for (int i = threadIdx.x; i < total; i += kThreads) {
        const bool is_q = i < nq;
        const int j = is_q ? i : i - nq;
        const int h = j / per, u = j % per;
        if (is_q) turn_unit<T, kSide>(q + (int64_t)h * a.d, qo + (int64_t)h * a.d, u, a.rot, cs);
        else turn_unit<T, kSide>(k + (int64_t)h * a.d, ko + (int64_t)h * a.d, u, a.rot, cs);
    }
}

// Number of threads of the CTA for which `pred` holds, over strided indices
// [0, n): the sequence of token t is the number of sequences that end at or
// before it.
__device__ __forceinline__ int count_ends(const int32_t *cu, int B, int64_t t) {
    int c = 0;
    for (int b0 = 0; b0 < B; b0 += kThreads) {
        const int b = b0 + threadIdx.x;
        c += __syncthreads_count(b < B && cu[b + 1] <= t);
    }
    return c;
}

template <typename T, bool kSide>
__global__ void __launch_bounds__(kThreads)
rope_append_kernel(RopeArgs a, AppendArgs c) {
    __shared__ float2 cs[kMaxHalf];
    const int64_t n = blockIdx.x;
    const int b = count_ends(c.cu_seqlens, c.B, n);
    if (b >= c.B) return;                                   // behind the last sequence
    const int64_t lo = c.cu_seqlens[b], hi = c.cu_seqlens[b + 1], L = c.seq_lens[b];
    if (b == 0 && n < lo) return;                           // before the first one
    // the token's position, cache row and the checks that keep both in range
    const int64_t p = L - hi + n;
    const bool ok = lo >= 0 && lo <= n && n < hi && hi <= a.tokens && hi - lo <= L &&
                    L <= (int64_t)c.max_pages * c.page_size;
    int64_t row = -1;
    if (ok) {
        const int pg = c.block_table[(int64_t)b * c.max_pages + p / c.page_size];
        if (pg >= 0 && pg < c.num_pages) row = (int64_t)pg * c.page_size + p % c.page_size;
    }
    if (row < 0 || !MSA_IN_BOUNDS(row, (int64_t)c.num_pages * c.page_size)) {
        if (threadIdx.x == 0) record_error(c.err, MSA_ERR_BAD_PAGE_TABLE, 3);
        return;
    }
    fill_turns(cs, p, a.inv_freq, a.rot / 2, a.mscale, false);
    __syncthreads();
    const T *q = (const T *)a.Q + n * a.q_stride, *k = (const T *)a.K + n * a.k_stride;
    const T *v = (const T *)c.V + n * c.v_stride, *x = (const T *)c.k_idx + n * c.d_idx;
    const int64_t kv_row = (int64_t)a.Hkv * a.d;
    T *qo = (T *)a.Q_out + n * a.qo_stride, *ko = (T *)a.K_out + row * kv_row;
    T *vo = (T *)c.V_cache + row * kv_row, *xo = (T *)c.k_idx_cache + row * c.d_idx;
    const int per = kSide ? a.d / 8 : a.rot / 16 + (a.d - a.rot) / 8;
    const int nq = a.Hq * per, nk = nq + a.Hkv * per, nv = nk + (int)(kv_row / 8);
    const int total = nv + c.d_idx / 8;
    for (int i = threadIdx.x; i < total; i += kThreads) {
        if (i < nk) {
            const int j = i < nq ? i : i - nq;
            const int h = j / per, u = j % per;
            if (i < nq) turn_unit<T, kSide>(q + (int64_t)h * a.d, qo + (int64_t)h * a.d, u, a.rot, cs);
            else turn_unit<T, kSide>(k + (int64_t)h * a.d, ko + (int64_t)h * a.d, u, a.rot, cs);
        } else if (i < nv) {
            copy8(vo + 8 * (i - nk), v + 8 * (i - nk));
        } else {
            copy8(xo + 8 * (i - nv), x + 8 * (i - nv));
        }
    }
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &a, int dtype, bool side, cudaStream_t st) {
    if (a.tokens == 0) return cudaSuccess;
    const unsigned grid = (unsigned)a.tokens;
    if (dtype == MSA_BF16) {
        if (side) rope_kernel<__nv_bfloat16, true><<<grid, kThreads, 0, st>>>(a);
        else rope_kernel<__nv_bfloat16, false><<<grid, kThreads, 0, st>>>(a);
    } else {
        if (side) rope_kernel<float, true><<<grid, kThreads, 0, st>>>(a);
        else rope_kernel<float, false><<<grid, kThreads, 0, st>>>(a);
    }
    count_launches(1);
    return cudaGetLastError();
}

cudaError_t launch_rope_append(const RopeArgs &a, const AppendArgs &c, int dtype, bool side,
                               cudaStream_t st) {
    if (a.tokens == 0) return cudaSuccess;
    const unsigned grid = (unsigned)a.tokens;
    if (dtype == MSA_BF16) {
        if (side) rope_append_kernel<__nv_bfloat16, true><<<grid, kThreads, 0, st>>>(a, c);
        else rope_append_kernel<__nv_bfloat16, false><<<grid, kThreads, 0, st>>>(a, c);
    } else {
        if (side) rope_append_kernel<float, true><<<grid, kThreads, 0, st>>>(a, c);
        else rope_append_kernel<float, false><<<grid, kThreads, 0, st>>>(a, c);
    }
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace msa
