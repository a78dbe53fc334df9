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
// shared by all heads.  A warp takes a token, or a share of its heads where
// there are few tokens: its lanes cover whole heads a step, 16 (bf16) or 32
// contiguous bytes each and always the same channels, so a lane's cosines and
// sines stay in registers, its addresses advance by one addition, and no
// barrier is needed.  32K tokens of 72 heads of 128 channels, bf16: 190 us,
// 6.3 TB/s, 97 % of a copy.  (One CTA a token with the turns in shared memory
// and places worked out by division: 256 us, bound by instruction issue.)
//
// Angles: p * theta is reduced to a part of a turn in fp64 (at p = 2^20 an
// fp32 product would be off by up to 0.06 radians), and the remainder, at
// most half a turn, is rounded to fp32 for sincospif: an error of at most
// 2^-25 turns, 2e-7 radians, and that of the fp64 steps, up to |p theta| 2^-51
// radians (1.5e-8 for theta = 1 at p = 2^25, 1e-6 at 2^31).  fp32 outputs are 1.3 times as far
// from 64 bits as with cosines in fp64 (6.2e-8 against 4.6e-8).
#include <math.h>

#include "msa_internal.cuh"

namespace msa {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxHalf = 128;                 // pairs of a head (rot <= 256)
// Heads a lane has in flight (two, three, four: 217, 209, 190 us for the 32K
// prompt's Q and K; six spill).
constexpr int kUnits = 4;

// Eight channels as they are in memory.
template <typename T> struct Raw8;
template <> struct Raw8<__nv_bfloat16> {
    uint4 v;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { v = *(const uint4 *)p; }
    __device__ __forceinline__ void store(__nv_bfloat16 *p) const { *(uint4 *)p = v; }
    __device__ __forceinline__ Raw8 from(int lane) const {   // another lane's
        Raw8 r;
        r.v = make_uint4(__shfl_sync(0xffffffffu, v.x, lane), __shfl_sync(0xffffffffu, v.y, lane),
                         __shfl_sync(0xffffffffu, v.z, lane), __shfl_sync(0xffffffffu, v.w, lane));
        return r;
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const __nv_bfloat162 *h = (const __nv_bfloat162 *)&v;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __bfloat1622float2(h[i]);
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
    __device__ __forceinline__ void put(const float (&x)[8]) {
        __nv_bfloat162 *h = (__nv_bfloat162 *)&v;
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    }
};
template <> struct Raw8<float> {
    float4 v[2];
    __device__ __forceinline__ void load(const float *p) {
        v[0] = *(const float4 *)p;
        v[1] = *(const float4 *)(p + 4);
    }
    __device__ __forceinline__ void store(float *p) const {
        *(float4 *)p = v[0];
        *(float4 *)(p + 4) = v[1];
    }
    __device__ __forceinline__ Raw8 from(int lane) const {
        Raw8 r;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            r.v[i] = make_float4(__shfl_sync(0xffffffffu, v[i].x, lane),
                                 __shfl_sync(0xffffffffu, v[i].y, lane),
                                 __shfl_sync(0xffffffffu, v[i].z, lane),
                                 __shfl_sync(0xffffffffu, v[i].w, lane));
        return r;
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        *(float4 *)x = v[0];
        *(float4 *)(x + 4) = v[1];
    }
    __device__ __forceinline__ void put(const float (&x)[8]) {
        v[0] = *(const float4 *)x;
        v[1] = *(const float4 *)(x + 4);
    }
};
template <typename T>
__device__ __forceinline__ void copy8(T *d, const T *s) {
    Raw8<T> r;
    r.load(s);
    r.store(d);
}

// mscale times the cosine and (signed) sine of a pair's angle at position p.
__device__ __forceinline__ float2 turn_of(int64_t p, double inv_freq, float mscale, bool inverse) {
    double turns = (double)p * (inv_freq * 0.15915494309189535);   // 1 / (2 pi)
    turns -= rint(turns);
    float s, c;
    sincospif(2.f * (float)turns, &s, &c);
    return make_float2(mscale * c, mscale * (inverse ? -s : s));
}

// How a warp covers heads of d channels: d / 8 lanes a head, eight channels
// each (c0 ..), `heads` heads a step; lanes past heads * d / 8 are idle.  With
// channels in halves, a turned lane's pairs are with the channels of another
// lane of its head, `mate`: the first half's lanes turn (own, mate's), the
// second half's (mate's, own).  Side by side, a lane has its pairs itself.
struct Lanes {
    int heads, h, c0, mate;
    bool active, turned, second;
};
template <bool kSide>
__device__ __forceinline__ Lanes make_lanes(int d, int rot) {
    Lanes l;
    const int per = d / 8, lane = threadIdx.x % 32, u = lane % per, half = rot / 16;
    l.heads = 32 / per;
    l.h = lane / per;
    l.active = l.h < l.heads;
    l.c0 = 8 * u;
    l.turned = l.active && l.c0 < rot;
    l.second = !kSide && l.turned && u >= half;
    l.mate = kSide || !l.turned ? lane : l.second ? lane - half : lane + half;
    return l;
}

// Heads share * l.heads + ..., of one token, shares * l.heads apart, kUnits at
// a time.  The first ones are loaded by begin(), so that it may run before the
// turns are known.  A step's values are all read before any is written.
template <typename T, bool kSide>
struct Heads {
    Raw8<T> x[kUnits];
    const T *in;
    int h;
    __device__ __forceinline__ void load(const Lanes &l, const RopeArgs &a, int n, int64_t hop) {
#pragma unroll
        for (int k = 0; k < kUnits; ++k)
            if (l.active && h + k * hop < n) x[k].load(in + k * hop * a.d);
    }
    __device__ __forceinline__ void begin(const Lanes &l, const RopeArgs &a, const T *token, int n,
                                          int share, int shares) {
        h = share * l.heads + l.h;
        in = token + (int64_t)h * a.d + l.c0;
        load(l, a, n, shares * l.heads);
    }
    __device__ __forceinline__ void turn(Raw8<T> &v, const Lanes &l, const float2 *cs) {
        float x[8];
        if (kSide) {
            if (!l.turned) return;
            v.get(x);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float p = x[2 * i], q = x[2 * i + 1];
                x[2 * i] = p * cs[i].x - q * cs[i].y;
                x[2 * i + 1] = q * cs[i].x + p * cs[i].y;
            }
        } else {
            const Raw8<T> m = v.from(l.mate);            // (all lanes take part)
            if (!l.turned) return;
            float y[8];
            v.get(x);
            m.get(y);
            // own * cos -+ mate's * sin: the sine carries the lane's sign
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = x[i] * cs[i].x + y[i] * cs[i].y;
        }
        v.put(x);
    }
    __device__ __forceinline__ void run(const Lanes &l, const RopeArgs &a, T *token, int n,
                                        int shares, const float2 *cs) {
        const int hop = shares * l.heads;
        T *out = token + (int64_t)h * a.d + l.c0;
        // the same number of steps for every lane: they exchange values
        for (int base = h - l.h; base < n; base += kUnits * hop) {
#pragma unroll
            for (int k = 0; k < kUnits; ++k) {
                if (base + k * hop < n) turn(x[k], l, cs);
                if (l.active && h + k * hop < n) x[k].store(out + (int64_t)k * hop * a.d);
            }
            h += kUnits * hop;
            in += (int64_t)kUnits * hop * a.d;
            out += (int64_t)kUnits * hop * a.d;
            load(l, a, n, hop);
        }
    }
};

// The lane's turns, in registers: the warp works out each pair's once.
template <bool kSide>
__device__ __forceinline__ void lane_turns(float2 (&mine)[kSide ? 4 : 8], float2 *shared,
                                           const Lanes &l, const RopeArgs &a, int64_t p,
                                           bool inverse) {
    for (int i = threadIdx.x % 32; i < a.rot / 2; i += 32)
        shared[i] = turn_of(p, a.inv_freq[i], a.mscale, inverse);
    __syncwarp();
    if (!l.turned) return;
    const int first = kSide ? l.c0 / 2 : l.second ? l.c0 - a.rot / 2 : l.c0;
#pragma unroll
    for (int i = 0; i < (kSide ? 4 : 8); ++i) {
        mine[i] = shared[first + i];
        if (!kSide && !l.second) mine[i].y = -mine[i].y;
    }
}

// `shares` warps a token.
template <typename T, bool kSide>
__global__ void __launch_bounds__(kThreads)
rope_kernel(RopeArgs a, int shares) {
    __shared__ float2 cs[kThreads / 32][kMaxHalf];
    const int warp = threadIdx.x / 32;
    const int64_t w = (int64_t)blockIdx.x * (kThreads / 32) + warp, n = w / shares;
    const int share = (int)(w % shares);
    if (n >= a.tokens) return;
    const Lanes l = make_lanes<kSide>(a.d, a.rot);
    Heads<T, kSide> q, k;
    q.begin(l, a, (const T *)a.Q + n * a.q_stride, a.Hq, share, shares);
    float2 mine[kSide ? 4 : 8];
    lane_turns<kSide>(mine, cs[warp], l, a, a.positions[n], a.inverse);
    q.run(l, a, (T *)a.Q_out + n * a.qo_stride, a.Hq, shares, mine);
    k.begin(l, a, (const T *)a.K + n * a.k_stride, a.Hkv, share, shares);
    k.run(l, a, (T *)a.K_out + n * a.ko_stride, a.Hkv, shares, mine);
}

// Sequence b's offsets and length are usable: T = hi - lo new tokens, the last
// of L positions.
__device__ __forceinline__ bool usable(const RopeArgs &a, const AppendArgs &c, int64_t lo,
                                       int64_t hi, int64_t L) {
    return lo >= 0 && lo <= hi && hi <= a.tokens && hi - lo <= L &&
           L <= (int64_t)c.max_pages * c.page_size;
}

// The error word of the call, by one CTA of its own (so that no separate clear
// is needed): what the other CTAs skip is found again here.  A thread takes a
// sequence, and warps together those with new tokens on more than four pages
// (the call for 300 single tokens: 5.5 us; with a warp a sequence 33).
__device__ __forceinline__ void append_check(const RopeArgs &a, const AppendArgs &c) {
    __shared__ int4 many[kThreads];                // sequence, first and last page
    __shared__ int n_many;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    auto bad_page = [&](int b, int64_t i) {
        const int pg = c.block_table[(int64_t)b * c.max_pages + i];
        return pg < 0 || pg >= c.num_pages;
    };
    int bad = 0;
    for (int b0 = 0; b0 < c.B; b0 += kThreads) {
        if (tid == 0) n_many = 0;
        __syncthreads();
        const int b = b0 + tid;
        if (b < c.B) {
            const int64_t lo = c.cu_seqlens[b], hi = c.cu_seqlens[b + 1], L = c.seq_lens[b];
            if (lo != hi && !usable(a, c, lo, hi, L)) {
                ++bad;
            } else if (lo != hi) {
                const int first = (int)((L - (hi - lo)) / c.page_size), last = (int)((L - 1) / c.page_size);
                if (last - first >= 4) {
                    many[atomicAdd(&n_many, 1)] = make_int4(b, first, last, 0);
                } else {
                    bool wrong = false;
#pragma unroll
                    for (int i = 0; i < 4; ++i) wrong |= first + i <= last && bad_page(b, first + i);
                    bad += wrong;
                }
            }
        }
        __syncthreads();
        for (int e = warp; e < n_many; e += kThreads / 32) {
            const int4 r = many[e];
            bool wrong = false;
            for (int i = r.y + lane; i <= r.z; i += 32) wrong |= bad_page(r.x, i);
            wrong = __any_sync(0xffffffffu, wrong);
            bad += lane == 0 && wrong;
        }
        __syncthreads();
    }
    __shared__ int total;
    if (tid == 0) total = 0;
    __syncthreads();
    if (bad) atomicAdd(&total, bad);
    __syncthreads();
    if (threadIdx.x < kErrorBytes / 4)
        c.err[threadIdx.x] = threadIdx.x == 0 ? (total ? MSA_ERR_BAD_PAGE_TABLE : MSA_OK)
                             : threadIdx.x == 3 ? total : 0;
}

// A warp's share of `n8` groups of eight channels, copied.
template <typename T>
__device__ __forceinline__ void copy_share(T *out, const T *in, int n8, int share, int shares) {
    const int step = 32 * shares;
    for (int i0 = 32 * share + threadIdx.x % 32; i0 < n8; i0 += 4 * step) {
        Raw8<T> x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i0 + k * step < n8) x[k].load(in + 8 * (i0 + k * step));
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i0 + k * step < n8) x[k].store(out + 8 * (i0 + k * step));
    }
}

// `shares` warps a token; the last CTA checks the call.
template <typename T, bool kSide>
__global__ void __launch_bounds__(kThreads)
rope_append_kernel(RopeArgs a, AppendArgs c, int shares) {
    __shared__ float2 cs[kThreads / 32][kMaxHalf];
    if (blockIdx.x == gridDim.x - 1) {
        append_check(a, c);
        return;
    }
    const int warp = threadIdx.x / 32;
    const int64_t w = (int64_t)blockIdx.x * (kThreads / 32) + warp, n = w / shares;
    const int share = (int)(w % shares);
    if (n >= a.tokens) return;
    const Lanes l = make_lanes<kSide>(a.d, a.rot);
    Heads<T, kSide> q, k;
    q.begin(l, a, (const T *)a.Q + n * a.q_stride, a.Hq, share, shares);
    // the token's sequence, position and cache row
    const int b = seq_of_token(c.cu_seqlens, c.B, n);
    if (b >= c.B) return;                                   // behind the last sequence
    const int64_t lo = c.cu_seqlens[b], hi = c.cu_seqlens[b + 1], L = c.seq_lens[b];
    if (n < lo || n >= hi || !usable(a, c, lo, hi, L)) return;
    const int64_t p = L - hi + n;
    const int pg = c.block_table[(int64_t)b * c.max_pages + p / c.page_size];
    if (pg < 0 || pg >= c.num_pages) return;
    const int64_t row = (int64_t)pg * c.page_size + p % c.page_size;
    if (!MSA_IN_BOUNDS(row, (int64_t)c.num_pages * c.page_size)) return;
    float2 mine[kSide ? 4 : 8];
    lane_turns<kSide>(mine, cs[warp], l, a, p, false);
    q.run(l, a, (T *)a.Q_out + n * a.qo_stride, a.Hq, shares, mine);
    k.begin(l, a, (const T *)a.K + n * a.k_stride, a.Hkv, share, shares);
    k.run(l, a, (T *)a.K_out + row * a.ko_stride, a.Hkv, shares, mine);
    copy_share((T *)c.V_cache + row * a.ko_stride, (const T *)c.V + n * c.v_stride,
               (int)(a.ko_stride / 8), share, shares);
    if (c.d_idx > 0 && share == shares - 1)
        copy_share((T *)c.k_idx_cache + row * c.d_idx, (const T *)c.k_idx + n * c.d_idx, c.d_idx / 8,
                   0, 1);
}

// Warps a token: eight where there are few tokens (a decode step of 64 then
// has 512 warps at work), one from 16 warps an SM on (two or four from there on
// are 0 to 30 % slower: each works the token's turns out again).
int shares_of(int64_t tokens) {
    return tokens < 148 * 2 ? 8 : tokens < 148 * 8 ? 4 : tokens < 148 * 16 ? 2 : 1;
}

template <typename T, bool kSide, bool kAppend>
cudaError_t launch_rope_t(const RopeArgs &a, const AppendArgs *c, cudaStream_t st) {
    const int shares = shares_of(a.tokens);
    const unsigned ctas = (unsigned)((a.tokens * shares * 32 + kThreads - 1) / kThreads);
    if constexpr (kAppend)
        rope_append_kernel<T, kSide><<<ctas + 1, kThreads, 0, st>>>(a, *c, shares);
    else
        rope_kernel<T, kSide><<<ctas, kThreads, 0, st>>>(a, shares);
    count_launches(1);
    return cudaGetLastError();
}

template <bool kAppend>
cudaError_t launch_any(const RopeArgs &a, const AppendArgs *c, int dtype, bool side, cudaStream_t st) {
    if (dtype == MSA_BF16)
        return side ? launch_rope_t<__nv_bfloat16, true, kAppend>(a, c, st)
                    : launch_rope_t<__nv_bfloat16, false, kAppend>(a, c, st);
    return side ? launch_rope_t<float, true, kAppend>(a, c, st)
                : launch_rope_t<float, false, kAppend>(a, c, st);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &a, int dtype, bool side, cudaStream_t st) {
    return a.tokens == 0 ? cudaSuccess : launch_any<false>(a, nullptr, dtype, side, st);
}

cudaError_t launch_rope_append(const RopeArgs &a, const AppendArgs &c, int dtype, bool side,
                               cudaStream_t st) {
    return launch_any<true>(a, &c, dtype, side, st);
}

}  // namespace msa
