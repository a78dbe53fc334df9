// full_attn_tc.cu -- full causal attention on the tensor cores (bf16), over
// packed or paged keys, from one query token to whole prompts.
//
//   O = softmax(scale Q K^T + causal) V,   lse = log sum exp(scale Q K^T)
//
// A row tile is 128 (token, head of the KV group) rows: 128 / R tokens with
// their R query heads, so that K and V are read once for the group.  A CTA
// holds two of them in flight (streams 0 and 1), each with its own softmax
// warpgroup and its own product-issuing thread.  A unit of work is two row
// tiles of consecutive tokens against the same keys; one of at most 128 / R
// tokens (decode, ends of prompts) is a single row tile whose key run the two
// streams share half and half.
//
//   S = Q K^T      tcgen05, operands from shared memory, fp32 in TMEM
//   P = 2^(scale log2(e) (S - m))    in registers, bf16 over S in TMEM
//   O += P V       tcgen05, P from TMEM, O (fp32) in TMEM
//
// K and V come in tiles of 128 keys; S and P go in halves of 64, two buffers
// a stream (TMEM: streams' buffers in columns 0, 64 and 128, 192; O in 256
// and 384), so that the scores of the next half are ready when the softmax of
// this one ends.  With one 128-key buffer a stream (all that fits beside O)
// every softmax waited for the product before it, the scores after it and two
// hand-overs, 1400 of 3800 cycles a tile, while neither the tensor cores nor
// the special-function units were half busy.
//
// The running maximum m that a row's P is taken against moves only when a
// half's maximum would make P larger than 2^8: P keeps the same relative
// rounding in bf16, far from fp32's range, and O is rarely rescaled.  The fp32
// row sum is of the unrounded P.  P is rounded to bf16 because one product's
// operands have one type and V is bf16 (in fp32, or as two bf16 terms, the
// product would cost two to four times as much): its errors, up to 2^-8 a weight
// and independent of one another, leave O 1.2 to 1.4 times as far from the
// 64-bit value as an fp32 computation that rounds once.  The exponentials are
// ex2.approx, good to 2^-22, far under that.
//
// Measured (one B200 at its 1000 W limit, 1.65 to 1.8 GHz): one 32768-token
// prompt of 32 heads, d = 128, 8.0 to 8.4 ms, 1.05 to 1.10 PFLOP/s on the
// causal flops, 64 to 67 % of a measured 8192^3 matrix product; tensor pipe 53 %
// busy, special-function units 53 %.  The products alone (no softmax) take
// 6.2 to 6.8 ms of that, the softmax alone 5.9 to 6.5.  A decode step of 64
// sequences of 2K to 16K keys: 440 us for this kernel by itself, 5.9 TB/s, 90 %
// of a copy (with the plan and the merge 466, the call in a loop 500).
// Tried and slower: S released as soon as the softmax has it in registers, P
// in columns of its own (8.5 ms); four softmax warpgroups, two a stream taking
// halves in turn (8.9 ms); a quarter to a half of the exponentials as
// polynomials on the multiply-add pipe (no gain).
#include <math.h>

#include <algorithm>
#include <atomic>

#include "full_attn.cuh"
#include "tc.cuh"

namespace msa {
namespace {

constexpr int kThreads = 384;            // loads + MMA + value check, two softmax warpgroups
constexpr int kRows = 128;               // rows of a row tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMaxLag = 8.f;           // log2 of how far P may pass 1
constexpr int kHalf = 64;                // keys of one S / P buffer
constexpr int kMaxCtas = 148;            // SMs of a B200

// Halves whose products are summed in TMEM at most: an item of longer key runs
// is handed out in pieces, each one's sums carried to the next in memory.  The
// tensor core adds to its fp32 sums four keys at a time and cuts the result off,
// towards 0: over 2^20 keys at once O came out 0.66 % too small, over 2^22 2.6 %,
// over 2^26 a third; over 2^16, this many, 0.04 %, a tenth of bf16's rounding.
// (Carried inside the loop over the halves instead, the loop's registers made
// every call of short sequences 2 to 4 % slower.)
constexpr int kPieceHalves = 1024;
constexpr int kCarryIn = 1, kCarryOut = 2;   // Item::carry: pieces before this one, behind it

template <int D> constexpr int ring_slots() { return D == 128 ? 5 : 10; }
template <int D> constexpr size_t tc_smem() {
    return 1024 + (2 + (size_t)ring_slots<D>()) * 128 * D * 2 + 1024;
}

struct TcArgs {
    FullShape s;
    FullSeqs q;
    FullCut c;
    const FullPlan *plan;
    const FullSeq *seqs;
    int *next;                           // the next item to take
    const __nv_bfloat16 *Q, *K, *V;      // Q, K: read for infinite values' weights only
    __nv_bfloat16 *O;
    float *lse, *part_o, *part_lse;
    float *carry;                        // [CTA][stream][row][d + 8]: earlier pieces' sums
    uint32_t *err;
    int box;                             // key rows of one TMA box
    bool wide;                           // O is 32-byte aligned
    float scale_log2, lag;               // lag: kMaxLag in units of raw scores
};

// A work item as the loading warp hands it to the others.
struct Item {
    int valid, b, g, q0;                 // q0: row of Q of the unit's first token
    int nt, pos0, k0, pair;              // tokens; position of the first; packed key row 0
    int a0, a1, h0, h1;                  // each stream's first key tile and number of halves
    int part, parts, carry, pad;         // key run, and how many the rows' results come in
};

__device__ __forceinline__ int stream_a(const Item &w, int s) { return s ? w.a1 : w.a0; }
__device__ __forceinline__ int stream_h(const Item &w, int s) { return s ? w.h1 : w.h0; }
__device__ __forceinline__ int stream_n(const Item &w, int s) { return (stream_h(w, s) + 1) / 2; }
// The streams read the same key tiles (a pair of row tiles, or one stream idle).
__device__ __forceinline__ bool shared_keys(const Item &w) { return w.pair || w.h1 == 0; }
// Some row of the unit does not attend all of key tile t.
__device__ __forceinline__ bool edge_tile(const Item &w, int t) {
    return (t + 1) * kFullKeys > w.pos0 + 1;
}

__device__ __forceinline__ Item make_item(const TcArgs &a, const FullSeq &q, int b, int item) {
    Item w;
    const int local = item - q.first_item, per = q.units * q.parts;
    const int r = local % per;
    const int u = q.units - 1 - r % q.units;
    w.valid = 1;
    w.b = b;
    w.g = local / per;
    w.part = r / q.units;
    const int t0 = u * a.c.unit_tokens;
    w.nt = min(a.c.unit_tokens, q.T - t0);
    w.q0 = q.q0 + t0;
    w.pos0 = q.L - q.T + t0;
    w.k0 = q.k0;
    w.pair = w.nt > a.c.half_tokens;
    w.parts = full_row_parts(q, a.c, t0);
    w.carry = 0;
    const int lo = w.part * q.tiles;
    auto run = [&](int tokens) {         // halves of this part that the first tokens see
        const int seen = (max(0, w.pos0 + tokens) + kHalf - 1) / kHalf;
        return max(0, min(seen, 2 * (lo + q.tiles)) - 2 * lo);
    };
    const int h = run(w.nt);
    w.a0 = w.a1 = lo;
    if (w.pair) {
        w.h0 = run(a.c.half_tokens);
        w.h1 = h;
    } else if (a.c.max_parts > 1) {
        const int tiles = ((h + 1) / 2 + 1) / 2;         // the first half of the tiles
        w.h0 = min(h, 2 * tiles);
        w.h1 = h - w.h0;
        w.a1 = lo + tiles;
        w.part *= 2;
    } else {
        w.h0 = h;
        w.h1 = 0;
    }
    return w;
}

struct Bars {
    // a slot's tile has landed; was read by its products; an edge tile's load
    // was issued (the check warps skip the other tiles, so they cannot follow
    // `full` by its phases alone); an edge tile's values are in order
    uint64_t full[10], empty[10], issued[10], fixed[10];
    uint64_t q_full, q_empty, s_full[2][2], p_full[2][2], o_prev[2], o_full[2], item_full[2], item_empty[2];
    Item item[2];
    volatile int odd[2];                 // item count + 1 where an edge tile held inf or NaN
    uint32_t tmem;
    volatile int abort;
};
static_assert(sizeof(Bars) <= 1024, "barrier block");

// One lane's arrival, without a branch and without the release fence of a
// plain arrival (together about 150 cycles of a softmax tile).  What it
// announces is in TMEM, ordered by tcgen05.wait::st and the fences around it.
__device__ __forceinline__ void arrive_if(bool pred, uint64_t *bar) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "@p mbarrier.arrive.relaxed.cta.shared::cta.b64 _, [%0];\n\t}\n"
        ::"r"(tc::smem_u32(bar)), "r"((uint32_t)pred) : "memory");
}

// Ring position: slot and phase parity.
struct Ring {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void step(int slots) {
        if (++slot == slots) {
            slot = 0;
            phase ^= 1;
        }
    }
};

// Calls k(stream, j) and v(stream, j) for the key and value tiles of an item
// in the order they go through the ring (stream 0 stands for both where the
// keys are shared); false as soon as one of them fails.
template <typename FK, typename FV>
__device__ __forceinline__ bool for_tiles(const Item &w, FK k, FV v) {
    const int n0 = stream_n(w, 0), n1 = stream_n(w, 1);
    if (shared_keys(w)) {
        const int n = max(n0, n1);
        if (n > 0 && !k(0, 0)) return false;
        for (int j = 0; j < n; ++j) {
            if (!v(0, j)) return false;
            if (j + 1 < n && !k(0, j + 1)) return false;
        }
        return true;
    }
    if (!k(0, 0) || !k(1, 0)) return false;              // both streams have a tile
    for (int j = 0; j < n0; ++j)                          // n0 >= n1
        for (int s = 0; s < 2; ++s) {
            const int n = s ? n1 : n0;
            if (j < n && !v(s, j)) return false;
            if (j + 1 < n && !k(s, j + 1)) return false;
        }
    return true;
}

// ---------------------------------------------------------------- loads

template <int D, bool kPaged>
__device__ void load_role(const TcArgs &a, Bars *bar, uint8_t *sQ, uint8_t *sKV,
                          const CUtensorMap *tm_q, const CUtensorMap *tm_q1,
                          const CUtensorMap *tm_k, const CUtensorMap *tm_v) {
    constexpr int kAtoms = D / 64, kSlots = ring_slots<D>();
    constexpr uint32_t kTile = 128 * D * 2;
    const int lane = threadIdx.x % 32;
    const int items = a.plan->items;
    const uint32_t q_tile_bytes = (uint32_t)(a.c.half_tokens * a.s.R) * 128 * kAtoms;
    Ring ring;
    int b = 0, q_uses = 0, left0 = 0, left1 = 0;         // the streams' halves from this piece on
    bool ok = true;
    Item w{};
    for (int k = 0;; ++k) {
        const int slot = k & 1;
        if (w.carry & kCarryOut) {
            w.a0 += kPieceHalves / 2;
            w.a1 += kPieceHalves / 2;
            left0 -= w.h0;
            left1 -= w.h1;
            w.carry = kCarryIn;
        } else {
            int item = blockIdx.x;
            if (k > 0) {
                if (lane == 0) item = gridDim.x + atomicAdd(a.next, 1);
                item = __shfl_sync(0xffffffffu, item, 0);
            }
            w = Item{};
            if (item < items) {
                b = full_find_seq(a.seqs, a.s.B, b, item, lane);
                w = make_item(a, a.seqs[b], b, item);
            }
            left0 = w.h0;
            left1 = w.h1;
        }
        w.h0 = min(left0, kPieceHalves);
        w.h1 = min(left1, kPieceHalves);
        if (max(left0, left1) > kPieceHalves) w.carry |= kCarryOut;
        const int limit = w.pos0 + w.nt;                 // no row attends key `limit` or later
        // paged: this lane's box, the cache row of each stream's tile, and of
        // its next one (whose page id is on its way meanwhile)
        int row[2] = {0, 0}, next_pg[2] = {0, 0}, next_at[2] = {0, 0};
        auto look_up = [&](int s, int j) {
            const int first = (stream_a(w, s) + j) * kFullKeys + lane * a.box;
            if (lane * a.box >= kFullKeys || first >= limit) return;
            const int i = first / a.s.page_size, at = first - i * a.s.page_size;
            const int pg = __ldg(a.q.block_table + (int64_t)w.b * a.s.max_pages + i);
            if (s) { next_pg[1] = pg; next_at[1] = at; } else { next_pg[0] = pg; next_at[0] = at; }
        };
        if (kPaged && w.h0 + w.h1 > 0) {
            look_up(0, 0);
            if (!shared_keys(w)) look_up(1, 0);
        }
        if (!tc::mbar_wait(&bar->item_empty[slot], ((k >> 1) & 1) ^ 1, a.err, &bar->abort)) break;
        if (lane == 0) {
            bar->item[slot] = w;
            tc::mbar_arrive(&bar->item_full[slot]);
        }
        if (!w.valid) break;
        if (w.h0 + w.h1 > 0) {
            if (!tc::mbar_wait(&bar->q_empty, (q_uses & 1) ^ 1, a.err, &bar->abort)) break;
            ++q_uses;
            const int tiles = w.pair ? 2 : 1;
            const bool one = w.nt == 1;
            if (lane == 0)
                tc::mbar_expect_tx(&bar->q_full, one ? (uint32_t)a.s.R * 128 * kAtoms
                                                     : q_tile_bytes * tiles);
            __syncwarp();
            if (one) {
                // one token: its heads alone.  The other rows then stay 0 in a
                // decode step, and the products on them cost little power,
                // which bounds the clock (1000 W at 1.7 GHz with the rows of
                // other sequences there).
                if (lane < kAtoms)
                    tc::tma_load_3d(sQ + lane * 16384, tm_q1, &bar->q_full, lane * 64,
                                    w.g * a.s.R, w.q0);
            } else if (lane < tiles * kAtoms) {
                const int t = lane / kAtoms, at = lane % kAtoms;
                tc::tma_load_3d(sQ + t * kTile + at * 16384, tm_q, &bar->q_full, at * 64,
                                w.g * a.s.R, w.q0 + t * a.c.half_tokens);
            }
        }
        auto load = [&](const CUtensorMap *tm, int s, int j, bool is_key) {
            if (!tc::mbar_wait(&bar->empty[ring.slot], ring.phase ^ 1, a.err, &bar->abort))
                return false;
            uint8_t *dst = sKV + ring.slot * kTile;
            uint64_t *full = &bar->full[ring.slot];
            const int key = (stream_a(w, s) + j) * kFullKeys;
            if (!kPaged) {
                if (lane == 0) tc::mbar_expect_tx(full, kTile);
                __syncwarp();
                if (lane < kAtoms)
                    tc::tma_load_3d(dst + lane * 16384, tm, full, lane * 64, w.g, w.k0 + key);
            } else {
                const int first = key + lane * a.box;    // this lane's box
                const bool mine = lane * a.box < kFullKeys && first < limit;
                if (is_key) {
                    if (s) row[1] = next_pg[1] * a.s.page_size + next_at[1];
                    else row[0] = next_pg[0] * a.s.page_size + next_at[0];
                }
                const int boxes = __popc(__ballot_sync(0xffffffffu, mine));
                if (lane == 0) tc::mbar_expect_tx(full, (uint32_t)boxes * a.box * 128 * kAtoms);
                __syncwarp();
                if (mine) {
                    const int rw = s ? row[1] : row[0];
#pragma unroll
                    for (int at = 0; at < kAtoms; ++at)
                        tc::tma_load_3d(dst + at * 16384 + lane * a.box * 128, tm, full, at * 64,
                                        w.g, rw);
                }
                if (is_key) look_up(s, j + 1);
            }
            if (!is_key && lane == 0 && edge_tile(w, stream_a(w, s) + j))
                tc::mbar_arrive(&bar->issued[ring.slot]);
            ring.step(kSlots);
            return true;
        };
        ok = for_tiles(w, [&](int s, int j) { return load(tm_k, s, j, true); },
                       [&](int s, int j) { return load(tm_v, s, j, false); });
        if (!ok) break;
    }
    if (bar->abort) {
        // copies in flight land before the CTA may end (each slot's latest
        // load), with a limit
        for (int i = 0; i < kSlots; ++i) {
            const bool this_lap = i < ring.slot;
            if (!this_lap && ring.phase == 0) continue;  // never loaded
            const uint32_t parity = this_lap ? ring.phase : ring.phase ^ 1;
            for (int n = 0; n < 1000 && !tc::mbar_try_wait(&bar->full[i], parity); ++n) {}
        }
        for (int n = 0; q_uses > 0 && n < 1000 &&
                        !tc::mbar_try_wait(&bar->q_full, (q_uses - 1) & 1); ++n) {}
    }
}

// ---------------------------------------------------------------- MMA

// A shared-memory matrix descriptor (128-byte swizzle, 8-row groups 1024 bytes
// apart) from its low word: the address / 16, with the leading byte offset
// / 16 in the upper half.  Kept in this form because one thread issues all
// products, and an address step is then one addition: 16 products in 1032
// cycles where building each descriptor from its address took 1097 (ideal
// 1024).
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) {
    return (saddr >> 4) | ((lbo >> 4) << 16);
}
__device__ __forceinline__ uint64_t desc(uint32_t lo) {
    constexpr uint32_t hi = (1024u >> 4) | (1u << 14) | (2u << 29);   // group stride, version, swizzle
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
    return d;
}

// One thread issues the products of one stream: S(0), S(1), then for each half
// i, once its P is there, O += P(i) V(i) and S(i + 2), which takes the buffer
// P(i) was in.  The two streams' threads sit in different warps and do not
// wait for each other: with one thread for both, its waits and commits (900
// cycles a tile) were the kernel's bound.  S of 64 keys runs at 49 cycles a
// product (its operands come from shared memory at 128 bytes a clock) where
// 32 would be ideal, which the other stream's products partly fill.
template <int D>
__device__ void mma_role(const TcArgs &a, Bars *bar, uint32_t tmem, uint32_t sQ, uint32_t sKV,
                         int me) {
    constexpr int kSlots = ring_slots<D>();
    constexpr uint32_t kTile = 128 * D * 2;
    constexpr uint32_t idesc_s = tc::idesc_bf16(kRows, kHalf, 0, 0);
    constexpr uint32_t idesc_o = tc::idesc_bf16(kRows, D, 0, 1);
    const uint32_t tS = tmem + me * 128, tO = tmem + 256 + me * 128;
    Ring ring;
    uint32_t fix_phase = 0;                              // per slot
    uint32_t p_phase = 0;                                // per buffer
    int q_uses = 0;
    for (int k = 0;; ++k) {
        const int slot = k & 1;
        if (!tc::mbar_wait(&bar->item_full[slot], (k >> 1) & 1, a.err, &bar->abort)) return;
        const Item w = bar->item[slot];
        tc::mbar_arrive(&bar->item_empty[slot]);
        if (!w.valid) return;
        if (w.h0 + w.h1 == 0) continue;
        if (!tc::mbar_wait(&bar->q_full, q_uses & 1, a.err, &bar->abort)) return;
        ++q_uses;
        const bool shared = shared_keys(w);
        const int h = stream_h(w, me), n = (h + 1) / 2;
        if (h == 0) tc::mbar_arrive(&bar->q_empty);
        const uint32_t qa = desc_lo(sQ + (w.pair && me ? kTile : 0), 16);
        // Both threads wait for every tile and release every tile, so that
        // neither can be a lap of the ring ahead of the other (a phase's
        // parity tells one lap only).
        auto scores = [&](int i, uint32_t k_tile) {      // half i, of the key tile at k_tile
            const uint32_t ka = desc_lo(k_tile, 16) + (i & 1) * 512;
#pragma unroll
            for (int c = 0; c < D / 16; ++c)
                tc::mma_ss(tS + (i & 1) * kHalf, desc(qa + (c / 4) * 1024 + (c % 4) * 2),
                           desc(ka + (c / 4) * 1024 + (c % 4) * 2), idesc_s, c > 0);
            tc::mma_commit(&bar->s_full[me][i & 1]);
            if (i + 1 == h) tc::mma_commit(&bar->q_empty);
        };
        auto product = [&](int i, uint32_t va) {         // half i, of the value tile at va
            const int b = i & 1;
            if (!tc::mbar_wait(&bar->p_full[me][b], (p_phase >> b) & 1, a.err, &bar->abort))
                return false;
            p_phase ^= 1u << b;
            tc::tc_fence_after();
#pragma unroll
            for (int c = 0; c < kHalf / 16; ++c)
                tc::mma_ts(tO, tS + b * kHalf + c * 8, desc(va + (b * 4 + c) * 128), idesc_o,
                           (i > 0 || c > 0) ? 1u : 0u);
            if (i + 2 == h) tc::mma_commit(&bar->o_prev[me]);
            if (i + 1 == h) tc::mma_commit(&bar->o_full[me]);
            return true;
        };
        auto key = [&](int s, int j) {
            const int at = ring.slot;
            const uint32_t phase = ring.phase;
            ring.step(kSlots);
            const bool mine = shared ? j < n : s == me;
            if (mine && j > 0) return true;              // its scores went with the values before
            if (!tc::mbar_wait(&bar->full[at], phase, a.err, &bar->abort)) return false;
            if (!mine) {
                tc::mbar_arrive(&bar->empty[at]);
                return true;
            }
            tc::tc_fence_after();
            scores(0, sKV + at * kTile);
            if (h > 1) scores(1, sKV + at * kTile);
            tc::mma_commit(&bar->empty[at]);
            return true;
        };
        auto value = [&](int s, int j) {
            const int at = ring.slot;
            const uint32_t phase = ring.phase;
            ring.step(kSlots);
            const bool edge = edge_tile(w, stream_a(w, s) + j);
            const uint32_t fixed = (fix_phase >> at) & 1;
            if (edge) fix_phase ^= 1u << at;
            if (!tc::mbar_wait(&bar->full[at], phase, a.err, &bar->abort)) return false;
            if (!(shared ? j < n : s == me)) {
                tc::mbar_arrive(&bar->empty[at]);
                return true;
            }
            if (edge && !tc::mbar_wait(&bar->fixed[at], fixed, a.err, &bar->abort)) return false;
            const uint32_t va = desc_lo(sKV + at * kTile, 16384);
            const int next = ring.slot;                  // the next key tile follows in the ring
            if (!product(2 * j, va)) return false;
            if (2 * j + 2 < h) {
                if (!tc::mbar_wait(&bar->full[next], ring.phase, a.err, &bar->abort)) return false;
                scores(2 * j + 2, sKV + next * kTile);
            }
            if (2 * j + 1 < h && !product(2 * j + 1, va)) return false;
            tc::mma_commit(&bar->empty[at]);
            if (2 * j + 3 < h) scores(2 * j + 3, sKV + next * kTile);
            if (2 * j + 2 < h) tc::mma_commit(&bar->empty[next]);
            return true;
        };
        if (!for_tiles(w, key, value)) return;
    }
}

// ---------------------------------------------------------------- value check

// One warp.  In a tile that some row attends only in part, P is 0 at the
// keys the row does not attend, and 0 times infinity or NaN would reach it:
// rows of V that no row attends (other sequences, what a page held before)
// are set to 0, and in rows that only later tokens attend, infinities and
// NaN are (the epilogue adds them, times their weights, for the rows that do
// attend them).
template <int D>
__device__ void check_role(const TcArgs &a, Bars *bar, uint8_t *sKV) {
    constexpr int kSlots = ring_slots<D>(), kChunks = D / 8;
    const int lane = threadIdx.x % 32;
    Ring ring;
    uint32_t edge_phase = 0;                             // per slot
    for (int k = 0;; ++k) {
        const int slot = k & 1;
        if (!tc::mbar_wait(&bar->item_full[slot], (k >> 1) & 1, a.err, &bar->abort)) return;
        const Item w = bar->item[slot];
        if (w.valid) {
            const int limit = w.pos0 + w.nt;
            auto key = [&](int, int) {
                ring.step(kSlots);
                return true;
            };
            auto value = [&](int s, int j) {
                const int t = stream_a(w, s) + j;
                if (edge_tile(w, t)) {
                    if (!tc::mbar_wait(&bar->issued[ring.slot], (edge_phase >> ring.slot) & 1,
                                       a.err, &bar->abort))
                        return false;
                    edge_phase ^= 1u << ring.slot;
                    if (!tc::mbar_wait(&bar->full[ring.slot], ring.phase, a.err, &bar->abort))
                        return false;
                    uint8_t *base = sKV + ring.slot * (128 * D * 2);
                    const int from = max(0, w.pos0 + 1 - t * kFullKeys);
                    bool odd = false;
                    for (int i = lane; i < (kFullKeys - from) * kChunks; i += 32) {
                        const int r = from + i / kChunks, ch = i % kChunks;
                        uint4 *p = (uint4 *)(base + (ch / 8) * 16384 + r * 128 +
                                             (((ch % 8) ^ (r & 7)) << 4));
                        if (t * kFullKeys + r >= limit) {
                            *p = make_uint4(0u, 0u, 0u, 0u);
                            continue;
                        }
                        uint4 v = *p;
                        uint32_t *x = (uint32_t *)&v;
                        bool hit = false;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if ((x[e] & 0x7f80u) == 0x7f80u) { x[e] &= 0xffff0000u; hit = true; }
                            if ((x[e] & 0x7f800000u) == 0x7f800000u) { x[e] &= 0xffffu; hit = true; }
                        }
                        if (hit) {
                            *p = v;
                            odd = true;
                        }
                    }
                    if (odd) bar->odd[slot] = k + 1;
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __threadfence_block();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&bar->fixed[ring.slot]);
                }
                ring.step(kSlots);
                return true;
            };
            if (!for_tiles(w, key, value)) return;
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bar->item_empty[slot]);
        if (!w.valid) return;
    }
}

// ---------------------------------------------------------------- softmax

// Two fp32 values in one 64-bit register: the packed operations do two
// additions or multiply-adds an issue slot.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t r, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
// 32 bytes in one store of a whole sector where the tensor's base allows it
// (`wide`: a multiple of 32), else in two.
__device__ __forceinline__ void store32(void *dst, const uint32_t *v, bool wide) {
    if (!wide) {
        ((uint4 *)dst)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        ((uint4 *)dst)[1] = make_uint4(v[4], v[5], v[6], v[7]);
        return;
    }
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 ::"l"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]),
                   "r"(v[6]), "r"(v[7]) : "memory");
}
// max(a, b, c), NaN if one of them is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// The maximum of a row's 64 scores.
__device__ __forceinline__ float row_max(const uint32_t (&v)[kHalf]) {
    float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int c = 0; c < kHalf; c += 8)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            m[i] = max3_nan(m[i], __uint_as_float(v[c + 2 * i]), __uint_as_float(v[c + 2 * i + 1]));
    return max3_nan(max3_nan(m[0], m[1], m[2]), m[3], m[3]);
}

// P = 2^(scale_log2 S - mb) of a half, as bf16 over S; returns the fp32 row
// sum.  (A quarter of the exponentials as polynomials on the multiply-add pipe
// gains nothing here: the special-function unit is busy 53 % of the time.)
__device__ __forceinline__ float weights(const uint32_t (&v)[kHalf], uint32_t tP, uint64_t scale2,
                                         uint64_t mb2) {
    uint64_t l0 = 0, l1 = 0;                             // (0, 0)
#pragma unroll
    for (int h = 0; h < kHalf; h += 32) {
        uint32_t pk[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) {
            const uint64_t x2 = fma2(pack2(__uint_as_float(v[h + 2 * c]),
                                           __uint_as_float(v[h + 2 * c + 1])), scale2, mb2);
            float e0, e1;
            unpack2(x2, e0, e1);
            e0 = tc::ex2_approx(e0);
            e1 = tc::ex2_approx(e1);
            if (c & 1) l1 = add2(l1, pack2(e0, e1)); else l0 = add2(l0, pack2(e0, e1));
            __nv_bfloat162 b = __floats2bfloat162_rn(e0, e1);
            pk[c] = *(uint32_t *)&b;
        }
        tc::tmem_st16(tP + h / 2, pk);
    }
    float x, y;
    unpack2(add2(l0, l1), x, y);
    return x + y;
}

// The sums of the pieces so far of a row of this CTA's stream s: O (not yet
// divided), the maximum it is taken against, the weights.
template <int D>
__device__ __forceinline__ float *carried_row(const TcArgs &a, int s, int row) {
    return a.carry + ((blockIdx.x * 2 + s) * (int64_t)kRows + row) * (D + 8);
}

// What is left of a stored row (`out`: carried on, a partial result or O) where `odd` (its item has
// infinities or NaN that the products left out) or its weights are all 0.
// The infinities and NaN among the values of keys lo .. hi enter with the weights
// of their keys, worked out again against the running maximum m: a weight of 0 (a
// score of -infinity, or far below m) gives NaN, as in a product.  Returns whether
// the row has a NaN.  Apart from the epilogue's loop, and on what it stored, so
// that the loop stays small.
template <int D, bool kPaged, typename T>
__device__ __forceinline__ bool finish_row(const TcArgs &a, const Item &w, bool odd, int64_t q_row,
                                           int head, int lo, int hi, float m, T *out) {
    const __nv_bfloat16 *q = a.Q + q_row * a.s.q_stride + (int64_t)(w.g * a.s.R + head) * D;
    for (int j = lo; odd && j <= hi; ++j) {
        int64_t row = (int64_t)w.k0 + j;
        if (kPaged)
            row = (int64_t)a.q.block_table[(int64_t)w.b * a.s.max_pages + j / a.s.page_size] *
                      a.s.page_size + j % a.s.page_size;
        const __nv_bfloat16 *v = a.V + row * a.s.v_stride + (int64_t)w.g * D;
        float p = -1.f;                                  // not worked out yet
#pragma unroll 1
        for (int c = 0; c < D; ++c) {
            const float f = __bfloat162float(v[c]);
            if (isfinite(f)) continue;
            if (p == -1.f) {
                const __nv_bfloat16 *k = a.K + row * a.s.k_stride + (int64_t)w.g * D;
                float dot = 0.f;
#pragma unroll 4
                for (int e = 0; e < D; ++e)
                    dot = fmaf(__bfloat162float(q[e]), __bfloat162float(k[e]), dot);
                p = tc::ex2_approx(fmaf(dot, a.scale_log2, m == -INFINITY ? 0.f : -m * a.scale_log2));
            }
            out[c] = from_f32<T>(fmaf(p, f, to_f32<T>(out[c])));
        }
    }
    bool nan = false;
#pragma unroll 4
    for (int c = 0; c < D; ++c) nan |= to_f32<T>(out[c]) != to_f32<T>(out[c]);
    return nan;
}
template <int D, bool kPaged>
__device__ __noinline__ bool finish_row(const TcArgs &a, const Item &w, bool odd, int stream, int tok,
                                        int head, int64_t part, float m) {
    const int t = (w.pair ? stream * a.c.half_tokens : 0) + tok, t0 = stream_a(w, stream);
    const int lo = max(t0 * kFullKeys, w.pos0 + 1);
    const int hi = min(w.pos0 + t, (t0 + stream_n(w, stream)) * kFullKeys - 1);
    const int64_t q_row = w.q0 + t;
    if (w.parts > 0 || (w.carry & kCarryOut))
        return finish_row<D, kPaged>(a, w, odd, q_row, head, lo, hi, m,
                                     w.carry & kCarryOut
                                         ? carried_row<D>(a, stream, tok * a.s.R + head)
                                         : a.part_o + part * D);
    return finish_row<D, kPaged>(a, w, odd, q_row, head, lo, hi, m,
                                 a.O + (q_row * a.s.Hq + w.g * a.s.R + head) * D);
}

template <int D, bool kPaged>
__device__ void softmax_role(const TcArgs &a, Bars *bar, uint32_t tmem, int s) {
    const int quad = (threadIdx.x / 32) % 4, lane = threadIdx.x % 32;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const uint32_t tS = tmem + s * 128 + lane_off, tO = tmem + 256 + s * 128 + lane_off;
    const int row = quad * 32 + lane;
    const int tok = row / a.s.R, head = row % a.s.R;
    uint32_t s_phase = 0, o_phase = 0, prev_phase = 0;   // s_phase: per buffer
    const uint64_t scale2 = pack2(a.scale_log2, a.scale_log2);
    for (int k = 0;; ++k) {
        const int slot = k & 1;
        if (!tc::mbar_wait(&bar->item_full[slot], (k >> 1) & 1, a.err, &bar->abort)) return;
        const Item &w = bar->item[slot];                 // read where needed: registers are short
        if (!w.valid) return;
        const int first_tok = w.pair ? s * a.c.half_tokens : 0;
        const int toks = min(a.c.half_tokens, w.nt - first_tok);
        const bool valid = tok < toks;
        const bool busy = quad * 32 < toks * a.s.R;      // the warp holds a row
        const int first_pos = w.pos0 + first_tok;        // of the stream's first token
        const int t0 = stream_a(w, s), h = stream_h(w, s), n = (h + 1) / 2;
        float m = -INFINITY, l = 0.f;
        for (int i = 0; i < h; ++i) {
            const int b = i & 1;
            const uint32_t tB = tS + b * kHalf;
            if (!tc::mbar_wait(&bar->s_full[s][b], (s_phase >> b) & 1, a.err, &bar->abort)) return;
            s_phase ^= 1u << b;
            if (busy) {
                tc::tc_fence_after();
                uint32_t v[kHalf];
                tc::tmem_ld32(tB, *(uint32_t(*)[32])v);
                tc::tmem_ld32(tB + 32, *(uint32_t(*)[32])(v + 32));
                tc::tmem_ld_wait();
                const int key0 = t0 * kFullKeys + i * kHalf;
                const bool edge = key0 + kHalf > first_pos + 1;
                if (edge) {
                    const int lim = first_pos + tok - key0;   // columns above lim are not attended
#pragma unroll
                    for (int c = 0; c < kHalf; ++c)
                        if (c > lim) v[c] = __float_as_uint(-INFINITY);
                }
                const float top = row_max(v);
                const bool move = valid && !(top <= m + a.lag);   // (a NaN moves m too)
                if (i == 0) {
                    m = top;
                } else if (__any_sync(0xffffffffu, move)) {
                    // O is rescaled between the products of halves i - 1 and
                    // i.  The first is complete once S(i + 1), issued after
                    // it, is; at the last half o_prev tells.
                    if (i + 1 < h ? !tc::mbar_wait(&bar->s_full[s][b ^ 1], (s_phase >> (b ^ 1)) & 1,
                                                   a.err, &bar->abort)
                                  : !tc::mbar_wait(&bar->o_prev[s], prev_phase, a.err, &bar->abort))
                        return;
                    tc::tc_fence_after();
                    const float f = move ? tc::ex2_approx((m - top) * a.scale_log2) : 1.f;
                    if (move) m = top;
                    l *= f;
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        uint32_t o[32];
                        tc::tmem_ld32(tO + c, o);
                        tc::tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tc::tmem_st32(tO + c, o);
                    }
                }
                const float mb = m == -INFINITY ? 0.f : -m * a.scale_log2;
                l += weights(v, tB, scale2, pack2(mb, mb));
                tc::tmem_st_wait();
                tc::tc_fence_before();
            }
            __syncwarp();
            arrive_if(lane == 0, &bar->p_full[s][b]);
        }
        // epilogue: O / l and the log-sum-exp, final or as one of the row's parts
        if (h > 0) {
            if (!tc::mbar_wait(&bar->o_full[s], o_phase, a.err, &bar->abort)) return;
            o_phase ^= 1;
            tc::tc_fence_after();
        }
        if (h > 1) prev_phase ^= 1;
        if (busy && (w.pair || s == 0 || a.c.max_parts > 1)) {
            float inv = 1.f, before = 0.f;               // factors of this O and of earlier pieces'
            if (w.carry & kCarryIn) {
                const float *y = carried_row<D>(a, s, row) + D;
                const float top = y[0] != y[0] || y[0] > m ? y[0] : m;   // (NaN where one is)
                if (top != -INFINITY) inv = tc::ex2_approx((m - top) * a.scale_log2);
                before = top != -INFINITY ? tc::ex2_approx((y[0] - top) * a.scale_log2) : 1.f;
                l = l * inv + y[1] * before;
                m = top;
            }
            if (!(w.carry & kCarryOut)) {
                const float r = l == 0.f ? 0.f : 1.f / l;
                inv *= r;
                before *= r;
            }
            const int64_t at = (int64_t)(w.q0 + first_tok + tok) * a.s.Hq + w.g * a.s.R + head;
            const int64_t part = ((int64_t)w.part + (w.pair ? 0 : s)) * a.s.tokens * a.s.Hq + at;
            const bool odd = bar->odd[slot] == k + 1;
            const bool direct = w.parts == 0 && !(w.carry & kCarryOut);
            const bool empty = direct && l == 0.f;       // O = 0
            if (n > 0 || w.parts == 0 || w.carry) {
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32];
                    __syncwarp();
                    if (n > 0) {
                        tc::tmem_ld32(tO + c, o);
                        tc::tmem_ld_wait();
                    }
                    float x[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        x[i] = empty || n == 0 ? 0.f : __uint_as_float(o[i]) * inv;
                    if ((w.carry & kCarryIn) && !empty) {
                        const float *y = carried_row<D>(a, s, row) + c;
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[i] = fmaf(y[i], before, x[i]);
                    }
                    if (valid && !direct) {
                        float *dst = w.carry & kCarryOut ? carried_row<D>(a, s, row) + c
                                                         : a.part_o + part * D + c;
#pragma unroll
                        for (int i = 0; i < 32; i += 8) store32(dst + i, (const uint32_t *)(x + i), true);
                    } else if (valid) {
                        __nv_bfloat16 *dst = a.O + at * D + c;
#pragma unroll
                        for (int i = 0; i < 32; i += 16) {
                            uint32_t u[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                __nv_bfloat162 h = __floats2bfloat162_rn(x[i + 2 * e], x[i + 2 * e + 1]);
                                u[e] = *(uint32_t *)&h;
                            }
                            store32(dst + i, u, a.wide);
                        }
                    }
                }
            }
            bool nan = false;
            if (valid && !empty && (odd || l == 0.f) && (n > 0 || w.carry))
                nan = finish_row<D, kPaged>(a, w, odd, s, tok, head, part, m);
            if (valid) {
                const float out_lse = l != 0.f ? m * a.s.scale + logf(l)
                                               : nan ? kNanPart : -INFINITY;
                if (w.carry & kCarryOut) {
                    float *y = carried_row<D>(a, s, row) + D;
                    y[0] = m;
                    y[1] = l;
                } else if (w.parts > 0) {
                    a.part_lse[part] = out_lse;
                } else {
                    a.lse[at] = out_lse;
                }
            }
            tc::tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bar->item_empty[slot]);
    }
}

template <int D, bool kPaged>
__global__ void __launch_bounds__(kThreads, 1)
full_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_q1,
               const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
               const __grid_constant__ TcArgs a) {
    constexpr int kSlots = ring_slots<D>();
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint8_t *sQ = smem;                                  // [2][D / 64][128][64]
    uint8_t *sKV = sQ + 2 * 128 * D * 2;                 // [kSlots][D / 64][128][64]
    Bars *bar = (Bars *)(sKV + kSlots * 128 * D * 2);
    const int warp = threadIdx.x / 32;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kSlots; ++i) {
            tc::mbar_init(&bar->full[i], 1);
            tc::mbar_init(&bar->empty[i], 2);            // one per stream
            tc::mbar_init(&bar->issued[i], 1);
            tc::mbar_init(&bar->fixed[i], 1);
        }
        tc::mbar_init(&bar->q_full, 1);
        tc::mbar_init(&bar->q_empty, 2);
        for (int i = 0; i < 2; ++i) {
            for (int b = 0; b < 2; ++b) {
                tc::mbar_init(&bar->s_full[i][b], 1);
                tc::mbar_init(&bar->p_full[i][b], 4);    // one per softmax warp
            }
            tc::mbar_init(&bar->o_prev[i], 1);
            tc::mbar_init(&bar->o_full[i], 1);
            tc::mbar_init(&bar->item_full[i], 1);
            tc::mbar_init(&bar->item_empty[i], 2 + 1 + 8);   // MMA, check and softmax warps
            bar->odd[i] = 0;
        }
        bar->abort = 0;
        tc::fence_mbar_init();
    }
    if (warp == 1) tc::tmem_alloc(&bar->tmem, 512);
    // rows of Q that are never loaded are 0
    for (int i = threadIdx.x; i < 2 * 128 * D * 2 / 16; i += kThreads)
        ((uint4 *)sQ)[i] = make_uint4(0u, 0u, 0u, 0u);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    launch_next();
    wait_previous();                                     // the plan
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = bar->tmem;
    if (warp < 4) {
        if (warp == 0) load_role<D, kPaged>(a, bar, sQ, sKV, &tm_q, &tm_q1, &tm_k, &tm_v);
        else if (warp == 3) check_role<D>(a, bar, sKV);
        else if (threadIdx.x % 32 == 0)
            mma_role<D>(a, bar, tmem, tc::smem_u32(sQ), tc::smem_u32(sKV), warp - 1);
    } else {
        softmax_role<D, kPaged>(a, bar, tmem, warp / 4 - 1);
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc::tc_fence_after();
        tc::tmem_free(tmem, 512);
    }
}

// SMs of the current device, and kernel k's shared-memory limit raised there:
// looked up and set once per device (together about 2 us a call).
template <int D, bool kPaged>
cudaError_t device_ready(int *sms) {
    static std::atomic<int> known[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    *sms = dev < 64 ? known[dev].load(std::memory_order_acquire) : 0;
    if (*sms > 0) return cudaSuccess;
    e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(full_tc_kernel<D, kPaged>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, (int)tc_smem<D>());
    if (e == cudaSuccess && dev < 64) known[dev].store(*sms, std::memory_order_release);
    return e;
}

template <int D, bool kPaged>
cudaError_t launch_tc_t(const FullShape &s, const TcArgs &a, const void *Q, const void *K,
                        const void *V, cudaStream_t st) {
    CUtensorMap tq, tq1, tk, tv;
    const uint64_t qdims[3] = {(uint64_t)D, (uint64_t)s.Hq, (uint64_t)s.tokens};
    const uint64_t qstr[2] = {(uint64_t)D * 2, (uint64_t)s.q_stride * 2};
    const uint32_t qbox[3] = {64, (uint32_t)s.R, (uint32_t)a.c.half_tokens};
    const uint32_t qbox1[3] = {64, (uint32_t)s.R, 1};
    if (!make_tmap_bf16(&tq, Q, 3, qdims, qstr, qbox)) return cudaErrorInvalidValue;
    if (!make_tmap_bf16(&tq1, Q, 3, qdims, qstr, qbox1)) return cudaErrorInvalidValue;
    // no keys at all: nothing is loaded, but a map needs an extent
    const uint64_t rows = (uint64_t)std::max<int64_t>(s.key_tokens, 1);
    const uint64_t dims[3] = {(uint64_t)D, (uint64_t)s.Hkv, rows};
    const uint64_t kstr[2] = {(uint64_t)D * 2, (uint64_t)s.k_stride * 2};
    const uint64_t vstr[2] = {(uint64_t)D * 2, (uint64_t)s.v_stride * 2};
    const uint32_t box[3] = {64, 1, (uint32_t)a.box};
    if (!make_tmap_bf16(&tk, s.key_tokens ? K : Q, 3, dims, kstr, box)) return cudaErrorInvalidValue;
    if (!make_tmap_bf16(&tv, s.key_tokens ? V : Q, 3, dims, vstr, box)) return cudaErrorInvalidValue;
    int sms = 0;
    const cudaError_t e = device_ready<D, kPaged>(&sms);
    if (e != cudaSuccess) return e;
    const int64_t most = (s.tokens / a.c.unit_tokens + std::min<int64_t>(s.B, s.tokens)) * s.Hkv *
                         a.c.max_parts;
    count_launches(1);
    return launch_after(full_tc_kernel<D, kPaged>, dim3((unsigned)std::min<int64_t>(most, std::min(sms, kMaxCtas))),
                        dim3(kThreads), tc_smem<D>(), st, tq, tq1, tk, tv, a);
}

}  // namespace

// Two row tiles of 128 / R tokens a unit.  Keys are split into runs while a
// call has too few units to keep every SM busy several times over: about
// kItemsPerSm items an SM (3, 4, 6, 8, on two workloads: a decode step of 64
// sequences 485, 471, 466, 474 us, a mixed step 1112, 1115, 1144, 1160 us; with
// page ids looked up ahead, at four, 463 and 1075).  A run has at least two
// tiles over a paged cache, where a single token may have 1000 keys and every
// SM idle (27 us; at least four: 31 us), and four over packed prompts, whose
// shortest then need no merge (28.7 against 32.8 us).  The partial results
// take at most (items + units) * 256 rows * 2, about 300 MB.  The number of runs
// follows from the tokens of the whole call, not from a sequence's own: beside a
// large chunk a single token has one run and one stream, whatever its length
// (4096 tokens of 64 heads over 8 take 307 us, with a token over 128K keys beside
// them 1.90 ms; that token alone 177 us).
FullCut full_tc_cut(const FullShape &s) {
    constexpr int kItemsPerSm = 4, kSms = kMaxCtas;
    FullCut c;
    c.half_tokens = kRows / s.R;
    c.unit_tokens = 2 * c.half_tokens;
    c.split = kSms * kItemsPerSm;
    c.min_tiles = s.paged ? 2 : 4;
    const int64_t units = std::max<int64_t>(1, (s.tokens + c.unit_tokens - 1) / c.unit_tokens) * s.Hkv;
    const int64_t keys = s.paged ? (int64_t)s.max_pages * s.page_size : s.key_tokens;
    c.carry_floats = keys > kPieceHalves * kHalf ? (size_t)kMaxCtas * 2 * kRows * (s.d + 8) : 0;
    c.max_parts = (int)std::min<int64_t>(kMaxParts, std::max<int64_t>(1, (4 * kSms + units - 1) / units));
    return c;
}

cudaError_t launch_full_tc(const FullShape &s, const FullSeqs &q, const FullCut &c,
                           const FullPlan *plan, const FullSeq *seqs, const void *Q,
                           const void *K, const void *V, void *O, float *lse, float *part_o,
                           float *part_lse, float *carry, uint32_t *err, cudaStream_t st) {
    TcArgs a;
    a.s = s; a.q = q; a.c = c;
    a.plan = plan; a.seqs = seqs;
    a.next = (int *)&plan->next;
    a.Q = (const __nv_bfloat16 *)Q;
    a.K = (const __nv_bfloat16 *)K;
    a.V = (const __nv_bfloat16 *)V;
    a.O = (__nv_bfloat16 *)O;
    a.lse = lse; a.part_o = part_o; a.part_lse = part_lse; a.err = err;
    a.wide = ((uintptr_t)O & 31u) == 0;
    a.scale_log2 = s.scale * kLog2e;
    a.lag = kMaxLag / a.scale_log2;
    a.carry = carry;
    a.box = kFullKeys;                   // the largest power of two that divides pages and tiles
    if (s.paged)
        while (s.page_size % a.box != 0) a.box /= 2;
    if (s.d == 64)
        return s.paged ? launch_tc_t<64, true>(s, a, Q, K, V, st)
                       : launch_tc_t<64, false>(s, a, Q, K, V, st);
    return s.paged ? launch_tc_t<128, true>(s, a, Q, K, V, st)
                   : launch_tc_t<128, false>(s, a, Q, K, V, st);
}

}  // namespace msa
