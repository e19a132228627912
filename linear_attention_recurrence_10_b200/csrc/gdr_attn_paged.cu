// gdr_attn_paged.cu -- attention of the new tokens of packed sequences over
// their pages: row i of sequence s, at position t = cache_len[s] + i, attends
// tokens 0 .. t.
//
//   a_j = scale q . k_j,  y = (sum_{j <= t} e^{a_j} v_j) / (sum e^{a_j}) * sigmoid(gate)
//
// Two kernels on the caller's stream, each a programmatic dependent of the one
// before:
//   attend: one CTA per SM.  A work item is a query tile (128 rows: the group's
//     query heads of 128 / n_rep tokens, so that a key/value tile is read once
//     for all of them) over the tiles of 128 keys that its last row attends.
//     The items of the whole batch, each n_kv tiles long plus a fixed cost,
//     are laid end to end and every CTA takes an equal stretch, so a prompt's
//     triangle of tiles, a ragged batch and one long sequence all load the SMs
//     evenly.  Every CTA derives its stretch from the lengths on the device.
//     An item that a stretch cuts leaves partial results in the workspace.
//   combine: joins the partial results of the items that were cut.
//
// In a CTA, one warp streams K and V through a ring of shared-memory slots with
// TMA tensor copies, page by page, into 128-byte-swizzled tiles; one thread
// issues S = Q K^T (M = 128 rows, N = 128 keys, K = 256) and O += P V (N = 256)
// on tcgen05 with S (two buffers) and O in tensor memory; the softmax warps
// (thread = row, two threads a row, four for codes) keep the running maximum and
// sum, write P over S in tensor memory and rescale O when the maximum has moved
// far.  S of the next tile is computed while the softmax works on this one.
//
// Long chunks over a bf16 cache go by pairs of CTAs: alone, a CTA's 128 rows use each
// 128 KB tile of keys and values for 16.8 MFLOP, and the L2 cache cannot feed 148 of
// them (2970 clocks a tile, a third of them waiting for loads).  The two CTAs of a cluster
// take 256 rows and load half of every tile each (cta_group::2 multiplies both halves
// for both): the waits for loads are short, and a tile takes 2700 clocks, of which the
// products are 2048 and the rest the round from S through the softmax back to P V.
//
// A code cache is multiplied as it is, in e4m3, at twice bf16's rate and with
// nothing to convert: the other operand is split in two 8-bit parts, x ~ hi + lo,
// which hold 8 significant bits as bf16 does.  Q (bf16) times a power of two
// per row, in e4m3 and e4m3, is exact for values within 2^-9 of the row's largest; smaller
// ones are off by up to 2^-17 of the largest.  The
// key scales multiply the scores.  The value scales sv_j enter the
// weights, w_j = 2^(a_j + log2 sv_j - m), which P holds in e4m3 and e5m2, with the maximum taken
// over a_j + log2 sv_j; the softmax's sum is that of w_j / sv_j.  Two more warps split
// Q and prepare the scales.
//
// What bounds it, 16 query heads over 2 key/value heads (clocks by stamps in the kernel, which
// add some per cent):
//   decode, 64 sequences of 4096 tokens: bf16, 107 us, the 0.54 GB of the cache at 5.0 TB/s;
//     codes, 90 us (0.27 GB, 3.0 TB/s): no unit is full (tensor pipe 44%, issue slots 28%).  Of
//     4200 clocks a tile the softmax's warps take 3550 from scores to weights, for which the
//     issuing thread waits 1250; one warp a scheduler has rows, 8 of its 32, so that is one
//     warp's latency.  The products are 2050, of 128 rows.  Spreading those 8 rows' softmax over
//     all warps was no faster.
//   2048 tokens after 6144, bf16: 225 to 228 us, 1.06 PFLOP/s with clocks near 1.5 GHz under the
//     power limit (200 us, 1.2 PFLOP/s, alone on a cool card).  The softmax's warps wait 450
//     clocks of a tile; their round is 2250.  Before the first tile a CTA spends 17000 clocks,
//     most of them on its place in the batch (make_plan: a binary search in 64-bit divisions).
//   4 prompts of 4096, bf16: 560 to 567 us, 0.97 PFLOP/s: 14.5 items a pair, whose ends, output gates
//     most of them, take 10700 clocks each, a fifth of the time, while nothing is multiplied.
//   chunks by codes: the softmax of a tile, 3800 clocks of 4150, four threads a row and three
//     times bf16's instructions a key (scales, two parts).
// P in shared memory with S two tiles ahead (pairs) measured 238 us for 232: P's one buffer
// then makes the softmax wait for P V.
//
// Every wait is bounded (2 s, less in the self-test); on expiry a role records GDR_ERR_TIMEOUT, the
// others run into their own limits, copies and commits in flight are waited
// for (bounded), tensor memory is freed and the CTA returns.
#include "gdr_tmap.cuh"
#include <math.h>

#include <atomic>
#include <type_traits>

#include "gdr.h"
#include "gdr_common.cuh"
#include "gdr_paged.cuh"
#include "gdr_tc.cuh"

namespace gdr {
namespace paged {

using namespace gdr::tc;

constexpr int ROWS = 128;  // query rows per item
constexpr int KEYS = 128;  // keys per tile
// Cost of starting and finishing an item, in tiles: for the items of a sequence with few new
// rows, and for others, whose output, gates and sums are most of it.  Four prompts of 4096
// tokens: 609 us with 2, 563 with 4, 571 with 6; 64 sequences' decode step 106 us with 2, 110 with 4.
constexpr int FEW_ROWS = 32, COST_FEW = 2, COST_MANY = 4;
constexpr int AUX_WARPS = 2;      // split Q, prepare scales: code caches only
constexpr int NRAW = 4;       // tiles of key and value scales in flight
constexpr uint32_t TM_O = 0, TM_S = 256, TM_COLS = 512;
constexpr uint64_t kWaitNs = 2000000000ull;
// Unwinding after an expired wait: arrivals still owed come within microseconds
// if their operations were issued, never if not.
constexpr uint64_t kDrainNs = 1000000ull;
constexpr int kTimeout = GDR_ERR_TIMEOUT;

// Shared memory.  Q tile: 4 boxes of [128 rows][128 bytes]; bf16: box c holds
// dims 64c ..; split e4m3: boxes 2h, 2h + 1 hold the hi and lo parts of dims 128h ...
constexpr uint32_t BOX = 16384;
template <bool E4M3>
struct Layout {
    // Threads that share a row, each with KEYS / PARTS keys of a tile.  Codes take four:
    // their weights cost three times bf16's instructions, and more warps hide more of the
    // latency than their smaller register share costs (a tile: 4400 clocks with two, 3900).
    // bf16 at four: 3300 clocks instead of 2970, the MMA thread having less of its scheduler.
    static constexpr int PARTS = E4M3 ? 4 : 2;
    static constexpr int SOFTMAX = 4 * PARTS;  // softmax warps: 0 ..
    static constexpr int W_LOAD = SOFTMAX, W_MMA = SOFTMAX + 1, W_AUX = SOFTMAX + 2;
    // A tile is two K slots and two V slots.  bf16: K slots are halves of the dims
    // (2 boxes of [128 keys][64 dims]), V slots halves of the keys (4 boxes of
    // [64 keys][64 dims]).  e4m3: both are halves of the dims ([128 keys][128 dims]).
    static constexpr uint32_t SLOT = E4M3 ? BOX : 2 * BOX;
    static constexpr int NSLOT = E4M3 ? 9 : 5;
    static constexpr uint32_t S_Q = 0;
    static constexpr uint32_t S_RING = 4 * BOX;
    static constexpr uint32_t S_RED = S_RING + NSLOT * SLOT;         // [4 quads][2][PARTS][32] floats
    static constexpr uint32_t S_SCALE = S_RED + 1024 * PARTS;  // [2][3][128] floats
    static constexpr uint32_t S_RAW = S_SCALE + (E4M3 ? 6 * 512 : 0);   // [NRAW][2][128] floats
    static constexpr uint32_t S_ROWK = S_RAW + (E4M3 ? NRAW * 1024 : 0);  // [2][128] floats
    static constexpr uint32_t S_BAR = S_ROWK + (E4M3 ? 1024 : 0);
    static constexpr uint32_t S_BYTES = S_BAR + 544;
    static constexpr int THREADS = 32 * (W_AUX + (E4M3 ? AUX_WARPS : 0));
};
static_assert(Layout<false>::S_BYTES <= 232448 && Layout<true>::S_BYTES <= 232448, "shared memory");

struct Desc {  // what a CTA leaves for the combine kernel
    int32_t tail;         // its last item is cut after it: slot 2c + 1 holds the item's first part
    int32_t head;         // slot 2c holds a part of an item begun before: 1, or 2 for its last part
    int32_t row0, n_tok;  // of the item in slot 2c + 1
    int32_t g;
    int32_t status;
    int32_t pad[2];
};

struct AttnParams {
    CUtensorMap tm_q, tm_k, tm_v;
    gdr_attn_paged_args a;
    int shift;        // log2(page_size)
    int n_rep;
    int cta_tok, tile_tok;  // tokens of a CTA's 128 rows, of an item (twice that for a pair)
    int pair;               // CTAs of an item: 1 or 2
    uint32_t rep_inv;  // r / n_rep = r * rep_inv >> 16, for r < 128
    int k_rows, v_rows;  // rows of a K and V box
    int n_rows;       // rows of the cache: a row past the end reads as zeros
    float scale_log2;
    int withhold;       // diagnostic: no Q tile is loaded, so that every wait for one runs out
    uint64_t wait_ns;   // limit of a wait
    int *status;      // workspace
    Desc *desc;       // [CTAs]
    float *part_ml;   // [2 CTAs][128][2]: maximum (log2) and sum
    float *part_o;    // [2 CTAs][64][128][4]: dims 4c .. of row r at [c][r], so that lanes = rows store together
};

// sum_{i < n} floor((a i + b) / m), in the steps of Euclid's algorithm.
__device__ int64_t floor_sum(int64_t n, int64_t m, int64_t a, int64_t b) {
    int64_t sum = 0;
    while (n > 0) {
        if (a >= m) {
            sum += n * (n - 1) / 2 * (a / m);
            a %= m;
        }
        if (b >= m) {
            sum += n * (b / m);
            b %= m;
        }
        const int64_t y = a * n + b;
        if (y < m) break;
        n = y / m;
        b = y % m;
        const int64_t t = m;
        m = a;
        a = t;
    }
    return sum;
}

// A sequence's lengths as the kernels use them.
struct Seq {
    int cu0, q, len;  // first packed row, new tokens, tokens before; len -1: lengths not usable
    int start;        // cost of starting and finishing an item
    // From cu_seqlens[s], cu_seqlens[s + 1] and cache_len[s].
    __device__ __forceinline__ void set(const AttnParams &p, int begin, int end, int before) {
        cu0 = max(begin, 0);
        q = max(min(end, (int)p.a.n_tok) - cu0, 0);
        start = (int64_t)q * p.n_rep <= FEW_ROWS ? COST_FEW : COST_MANY;
        len = before;
        const int64_t total = (int64_t)len + q;
        if (len < 0 || total > ((int64_t)p.a.pages.table_width << p.shift) || total >= kTooLong) len = -1;
    }
    __device__ __forceinline__ void load(const AttnParams &p, int s) {
        const int32_t *cu = p.a.pages.cu_seqlens + s;
        set(p, __ldg(cu), __ldg(cu + 1), __ldg(p.a.cache_len + s));
    }
    __device__ __forceinline__ int tiles(const AttnParams &p) const {
        return (q + p.tile_tok - 1) / p.tile_tok;
    }
    // Key tiles of query tile i.
    __device__ __forceinline__ int keys(const AttnParams &p, int i) const {
        if (len < 0) return 0;
        const int64_t end = (int64_t)len + min((int64_t)q, (int64_t)(i + 1) * p.tile_tok);
        return (int)((end + KEYS - 1) / KEYS);
    }
    // Cost of the first m query tiles of one kv head.
    __device__ __forceinline__ int64_t cost(const AttnParams &p, int m) const {
        int64_t u = (int64_t)m * start;
        if (len < 0 || m == 0) return u;
        const int whole = min(m, q / p.tile_tok);
        u += floor_sum(whole, KEYS, p.tile_tok, (int64_t)len + p.tile_tok + KEYS - 1);
        if (m > whole) u += ((int64_t)len + q + KEYS - 1) / KEYS;
        return u;
    }
};

// A CTA's stretch: `len` units of cost from its beginning; its first item is (s, g, i), whose
// cost starts at u <= 0.
struct Plan {
    int len, u, s, g, i;
};

struct Item {
    int s, g;
    int row0, n_tok;  // packed rows of this CTA
    int pos0;         // position of the first row's token
    int end;          // keys attended by the item's last row (of both CTAs of a pair)
    int n_kv;         // tiles of the whole item; 0: lengths not usable
    int a, b;         // this CTA's tiles
};

// The items of a CTA's stretch, in order.  Every role walks them by itself; the
// lengths of the next sequence are fetched while one is walked.
struct Walk {
    Plan w;
    Seq q;
    int n_tiles;
    int skip;                // tokens of the item before this CTA's
    int next_end, next_len;  // of sequence w.s + 1
    __device__ __forceinline__ Walk(const AttnParams &p, const Plan *plan, int rank)
        : w(*plan), n_tiles(0), skip(rank * p.cta_tok) {
        if (w.u < w.len) {
            q.load(p, w.s);
            n_tiles = q.tiles(p);
            fetch(p);
        }
    }
    __device__ __forceinline__ void fetch(const AttnParams &p) {
        const int s = min(w.s + 1, p.a.pages.n_seq - 1);
        next_end = __ldg(p.a.pages.cu_seqlens + s + 1);
        next_len = __ldg(p.a.cache_len + s);
    }
    __device__ __forceinline__ bool next(const AttnParams &p, Item &it) {
        const gdr_kv_pages &c = p.a.pages;
        while (w.u < w.len) {
            while (w.i >= n_tiles) {
                w.i = 0;
                if (n_tiles == 0 || ++w.g == c.H_kv) {
                    w.g = 0;
                    if (++w.s >= c.n_seq) return false;
                    q.set(p, q.cu0 + q.q, next_end, next_len);
                    n_tiles = q.tiles(p);
                    fetch(p);
                }
            }
            const int first = w.i * p.tile_tok;
            it.s = w.s;
            it.g = w.g;
            it.row0 = q.cu0 + first + skip;
            it.n_tok = min(p.cta_tok, max(q.q - first - skip, 0));
            it.pos0 = q.len + first + skip;
            it.end = q.len + min(first + p.tile_tok, q.q);
            it.n_kv = q.keys(p, w.i);
            const bool begins = w.u >= 0;
            it.a = min(max(-w.u - q.start, 0), it.n_kv);
            it.b = min(max(w.len - w.u - q.start, 0), it.n_kv);
            w.u += q.start + it.n_kv;
            ++w.i;
            if (it.a < it.b || (it.n_kv == 0 && begins)) return true;
        }
        return false;
    }
};

// One block-wide call: this CTA's stretch of the batch's cost.
__device__ void make_plan(const AttnParams &p, int n_thr, int64_t *warp_sum, Plan *plan) {
    const gdr_kv_pages &c = p.a.pages;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n_warps = n_thr >> 5;
    const int per = (c.n_seq + n_thr - 1) / n_thr;
    const int s0 = (int)min((int64_t)tid * per, (int64_t)c.n_seq);
    const int s1 = (int)min((int64_t)s0 + per, (int64_t)c.n_seq);
    int64_t mine = 0;
    for (int s = s0; s < s1; ++s) {
        Seq q;
        q.load(p, s);
        mine += c.H_kv * q.cost(p, q.tiles(p));
    }
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(kFullMask, upto, o);
        if (lane >= o) upto += x;
    }
    if (lane == 31) warp_sum[warp] = upto;
    if (tid == 0) *plan = Plan{0, 0, 0, 0, 0};
    __syncthreads();
    int64_t before = 0, total = 0;
    for (int i = 0; i < n_warps; ++i) {
        if (i < warp) before += warp_sum[i];
        total += warp_sum[i];
    }
    upto += before;
    // (blockIdx * total could overflow.)
    const int64_t n = gridDim.x / p.pair, me = blockIdx.x / p.pair, each = total / n, more = total - each * n;
    const int64_t lo = me * each + min(me, more);
    const int64_t hi = lo + each + (me < more ? 1 : 0);
    int64_t u = upto - mine;
    if (lo < hi && u <= lo && lo < upto) {
        for (int s = s0; s < s1; ++s) {
            Seq q;
            q.load(p, s);
            const int n_tiles = q.tiles(p);
            const int64_t head = q.cost(p, n_tiles), all = head * c.H_kv;
            if (lo < u + all) {
                const int g = (int)((lo - u) / head);
                u += g * head;
                int a = 0, b = n_tiles;  // the last tile that begins at or before lo
                while (b - a > 1) {
                    const int m = a + (b - a) / 2;
                    if (u + q.cost(p, m) <= lo) a = m;
                    else b = m;
                }
                *plan = Plan{(int)min(hi - lo, (int64_t)0x3fffffff), (int)(u + q.cost(p, a) - lo), s, g, a};
                break;
            }
            u += all;
        }
    }
    __syncthreads();
}

// Waits for a barrier's phase, at most `limit` ns.  The first look is inline, the rest a
// call: a CTA's five roles share the instruction cache, and code that is repeated at every wait
// costs more there than the call.
__device__ __noinline__ bool wait_on(uint64_t *bar, uint32_t parity, uint64_t limit) {
    return mbar_wait(bar, parity, limit);
}
__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, uint64_t limit) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}\n"
        : "=r"(done)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return done || wait_on(bar, parity, limit);
}

// The same by looking again and again: for a barrier at which another CTA arrives (a waiting
// thread that the hardware has suspended is woken late by that: by up to 2000 clocks here).
__device__ __noinline__ bool spin_on(uint64_t *bar, uint32_t parity, uint64_t limit) {
    const uint64_t start = global_ns();
    for (uint32_t i = 1;; ++i) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.b32 %0, 1, 0, p;\n\t}\n"
            : "=r"(done)
            : "r"(smem_u32(bar)), "r"(parity)
            : "memory");
        if (done) return true;
        if ((i & 255) == 0 && global_ns() - start > limit) return false;
    }
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mov.b64 c, {%6, %7};\n\tfma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
// Two f16 values as e4m3 codes in two parts, the second what the first leaves.
__device__ __forceinline__ void split2(uint32_t h2, uint16_t &hi, uint16_t &lo) {
    uint32_t back, rest;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(hi) : "r"(h2));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(hi));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(rest) : "r"(h2), "r"(back));
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(lo) : "r"(rest));
}
// a, b times inv and the sigmoids of two bf16 gates, 1 / (1 + 2^u) with u = -g log2(e): one
// reciprocal for both, of the product, which must not overflow, so u is held below 60
// (fminf also keeps a NaN out of its neighbour's value).  Right for gates of a magnitude
// below FAR_GATE (a bf16's bits: 41.75, 2^60.2); rows with others are written again by gate_any.
constexpr uint32_t FAR_GATE = 0x4227;
__device__ __forceinline__ void gate2(float &a, float &b, uint32_t gates, float inv) {
    const float2 u = mul2(make_float2(__uint_as_float(gates << 16), __uint_as_float(gates & 0xffff0000u)),
                          make_float2(-1.4426950408889634f, -1.4426950408889634f));
    const float2 d = add2(make_float2(exp2_fast(fminf(u.x, 60.f)), exp2_fast(fminf(u.y, 60.f))),
                          make_float2(1.f, 1.f));
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d.x * d.y));
    // (r times inv could underflow.)
    const float2 y = mul2(mul2(make_float2(a, b), make_float2(inv, inv)),
                          mul2(make_float2(d.y, d.x), make_float2(r, r)));
    a = y.x;
    b = y.y;
}
// a times the sigmoid of any gate: 0 times a for -inf, NaN for a NaN.
__device__ __forceinline__ float gate_any(float a, float g) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + exp2_fast(g * -1.4426950408889634f)));
    return a * r;
}
// Four weights in two 8-bit parts, e4m3 and what that leaves in e5m2, with integer
// instructions: the conversions run at 16 lanes a clock for the SM, like the exponentials
// beside them.  The weights come times 2^-8, below 2: there f16 has e4m3's exponents (2^-14
// its smallest normal value, where the codes' is 2^-6), so a code is an f16 value rounded to
// 3 bits of mantissa, without its sign's neighbour bit, which is 0.  The rest is at most a
// 16th of the weight (or 2^-10); times 2^8 its f16 value rounded to 2 bits of mantissa is its
// e5m2 code.  Together they are within 2^-8 of the weight, as bf16 is, and within 2^-14
// below 2^-6, where a second part in e4m3, whose smallest step is 2^-9, is within 2^-10.
__device__ __forceinline__ void split4(float a, float b, float c, float d, uint32_t &hi, uint32_t &lo) {
    const uint32_t y[2] = {f16x2(a, b), f16x2(c, d)};
    uint32_t h[2], l[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t t = y[i] + 0x00400040u;  // weights are positive: round by a carry
        uint32_t rest;
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(rest) : "r"(y[i]), "r"(t & 0xff80ff80u));
        asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(rest) : "r"(rest), "r"(0x5c005c00u));  // 2^8; exact
        h[i] = t << 1;
        l[i] = rest + 0x00800080u;  // rounded away from zero, whatever the sign
    }
    hi = __byte_perm(h[0], h[1], 0x7531);
    lo = __byte_perm(l[0], l[1], 0x7531);
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}
__device__ __forceinline__ void st_shared16(uint32_t a, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z),
                 "r"(v.w)
                 : "memory");
}

// Two 16-byte chunks in each of two neighbouring lanes, transposed: the even lane ends
// with the two first chunks, the odd lane with the two second ones (its own inverse).
__device__ __forceinline__ void transpose2(uint4 (&c)[2], int lane) {
    const bool odd = lane & 1;
    uint4 send = odd ? c[0] : c[1];
    send.x = __shfl_xor_sync(kFullMask, send.x, 1);
    send.y = __shfl_xor_sync(kFullMask, send.y, 1);
    send.z = __shfl_xor_sync(kFullMask, send.z, 1);
    send.w = __shfl_xor_sync(kFullMask, send.w, 1);
    if (odd) c[0] = send;
    else c[1] = send;
}

// Uses of the ring by an item of n tiles, in the order the MMA thread takes them: K0, K1,
// V0, K2, V1, ..., V(n-1), each SPT slots.
template <int SPT>
__device__ __forceinline__ int use_k(int i) { return i == 0 ? 0 : SPT * (2 * i - 1); }
template <int SPT>
__device__ __forceinline__ int use_v(int i, int n) { return SPT * (i < n - 1 ? 2 * i + 2 : 2 * n - 1); }

template <bool E4M3, bool PAIR, bool OUT_BF16>
__global__ void __launch_bounds__(Layout<E4M3>::THREADS, 1)
    attn_paged_kernel(const __grid_constant__ AttnParams p) {
    using L = Layout<E4M3>;
    static_assert(!(E4M3 && PAIR), "code caches are not paired");
    constexpr int NSLOT = L::NSLOT, PARTS = L::PARTS, SPT = PAIR ? 1 : 2;
    extern __shared__ __align__(1024) unsigned char sm[];
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + L::S_BAR);  // [NSLOT] slot landed
    uint64_t *empty = full + NSLOT;    // [NSLOT] slot consumed
    uint64_t *q_full = empty + NSLOT;  // Q tile landed
    uint64_t *q_split = q_full + 1;    // Q tile split in hi and lo (aux warps)
    uint64_t *q_free = q_full + 2;     // the item's S products are done
    uint64_t *bar_s = q_full + 3;      // [2] S of a tile in TMEM
    uint64_t *bar_p = q_full + 5;      // [2] P of a tile in TMEM, O rescaled (8 warps)
    uint64_t *bar_o = q_full + 7;      // [2] O += P V of a tile done
    uint64_t *o_free = q_full + 9;     // the item's O has been read (8 warps)
    uint64_t *sc_full = q_full + 10;   // [2] scales of a tile prepared (aux warps)
    uint64_t *raw_full = q_full + 12;  // [NRAW] scales of a tile landed
    uint64_t *peer_full = q_full + 12;  // [NSLOT] pairs: slot landed in the odd CTA (no codes there)
    uint64_t *peer_q = peer_full + NSLOT;  // pairs: Q tile landed in the odd CTA
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + L::S_BAR + 288);
    Plan *plan = reinterpret_cast<Plan *>(sm + L::S_BAR + 304);
    int64_t *warp_sum = reinterpret_cast<int64_t *>(sm + L::S_BAR + 352);  // one a warp
    const gdr_kv_pages &c = p.a.pages;
    // (Through a shuffle, so that the compiler knows the warp's number to be uniform.)
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(kFullMask, tid >> 5, 0);
    const uint32_t sbase = smem_u32(sm);
    const uint32_t ring = sbase + L::S_RING, sq = sbase + L::S_Q;
    const int rank = PAIR ? (int)cluster_rank() : 0;

    if (warp == 0) {
        if constexpr (PAIR) tmem_alloc_pair(tmem_slot, TM_COLS);
        else tmem_alloc(tmem_slot, TM_COLS);
    }
    if (tid == 0) {
        for (int i = 0; i < NSLOT; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1);
        }
        mbar_init(q_full, 1);
        mbar_init(q_split, AUX_WARPS);
        mbar_init(q_free, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar_s + i, 1);
            mbar_init(bar_p + i, (PAIR ? 2 : 1) * L::SOFTMAX);
            mbar_init(bar_o + i, 1);
            mbar_init(sc_full + i, AUX_WARPS);
        }
        for (int i = 0; i < (PAIR ? NSLOT + 1 : NRAW); ++i) mbar_init(raw_full + i, 1);  // (peer_full, peer_q)
        mbar_init(o_free, (PAIR ? 2 : 1) * L::SOFTMAX);
        mbar_fence_init();
    }
    wait_for_predecessor();
    release_dependents();
    Desc *desc = p.desc + blockIdx.x;
    if (tid == 0) *desc = Desc{};
    make_plan(p, L::THREADS, warp_sum, plan);
    fence_before_sync();
    __syncthreads();
    if constexpr (PAIR) cluster_sync();  // the barriers of both CTAs are set up
    fence_after_sync();
    const uint32_t tm = *tmem_slot;
    auto report = [&](int status) { atomicMax(&desc->status, status); };
    auto full_wait = [&](int use) {
        return wait_bar(full + use % NSLOT, (uint32_t)(use / NSLOT) & 1u, p.wait_ns);
    };
    // The swizzled tiles must start on 1024-byte boundaries.
    const bool usable = (sbase & 1023u) == 0;
    if (!usable && tid == 0) report(GDR_ERR_CUDA);

    // Arrivals that the thread which issues the MMAs waits for, in its CTA.
    auto arrive_mma = [&](uint64_t *bar) {
        if (PAIR && rank) mbar_arrive_at(bar, 0);
        else mbar_arrive(bar);
    };
    Walk walk(p, plan, rank);
    Item it;
    if (!usable) {
        // nothing runs
    } else if (warp == L::W_LOAD) {
        // ---------------------------------------------------------- loads
        // Lane 0 keeps the barriers; every lane issues its boxes of a slot.
        bool ok = true, bad = false;
        int n_use = 0, n_item = 0, n_raw = 0;
        if (lane == 0) {
            tma_prefetch_map(&p.tm_q);
            tma_prefetch_map(&p.tm_k);
            tma_prefetch_map(&p.tm_v);
            fence_proxy_async_global();
        }
        __syncwarp();
        const int kr = p.k_rows, vr = p.v_rows;
        while (ok && walk.next(p, it)) {
            if (it.n_kv == 0) {
                bad = true;
                continue;
            }
            // Cache row of each 16 keys of a tile, in lanes 0 .. 7; past the cache's end
            // (zeros) for a page that does not exist.
            auto page_row = [&](int j) {
                const int key = j * KEYS + 16 * lane;
                int row = p.n_rows;
                if (lane < 8 && j < it.b && key < it.end) {
                    const int r = cache_row(c, p.shift, it.s, it.g, key);
                    if (r >= 0) row = r;
                    else bad = true;
                }
                return row;
            };
            // One slot: n_box rows of boxes with n_col boxes each.
            auto acquire = [&](int use) {
                if (use >= NSLOT && lane == 0)
                    ok = wait_bar(empty + use % NSLOT, (uint32_t)(use / NSLOT - 1) & 1u, p.wait_ns);
                ok = __shfl_sync(kFullMask, ok, 0);
                return ok;
            };
            auto load_k = [&](int j, int use0, int row) {
                const int n = min(KEYS, it.end - j * KEYS);
                // Pairs: this CTA's 64 keys, in boxes of 64 dims as V's below.
                const int keys = PAIR ? max(0, min(64, n - 64 * rank)) : n;
                const int parts = (keys + kr - 1) / kr;
                constexpr int NCOL = E4M3 ? 1 : PAIR ? 4 : 2;
                constexpr uint32_t COL = PAIR ? BOX / 2 : BOX;
                for (int h = 0; h < SPT; ++h) {
                    const int use = use0 + h;
                    if (!acquire(use)) return;
                    uint64_t *bar = full + use % NSLOT;
                    if (lane == 0) {
                        if (!PAIR || parts > 0) bulk_expect(bar, (uint32_t)(parts * NCOL * kr * 128));
                        else mbar_arrive(bar);
                    }
                    __syncwarp();
                    const int part = lane / NCOL, col = lane % NCOL;
                    const int r = __shfl_sync(kFullMask, row, (part * (kr >> 4) + (PAIR ? 4 * rank : 0)) & 7);
                    if (part < parts)
                        tma_load_2d(ring + (use % NSLOT) * L::SLOT + col * COL + part * kr * 128,
                                    &p.tm_k, h * 128 + col * 64, r, bar);
                    n_use = use + 1;
                }
                if constexpr (E4M3) {
                    // The tile's scales: lanes 0 .. 7 the keys', 8 .. 15 the values', a part
                    // of kr rows each; none for a page that does not exist.  The stage is
                    // free: its tile's weights were multiplied before K's slot came free.
                    const int part = lane & 7;
                    const int r = __shfl_sync(kFullMask, row, (part * (kr >> 4)) & 7);
                    const bool has = lane < 16 && part < parts && r < p.n_rows;
                    const uint32_t bytes = (uint32_t)kr * 4;
                    const int n_copy = __popc(__ballot_sync(kFullMask, has));
                    uint64_t *bar = raw_full + n_raw % NRAW;
                    if (lane == 0) bulk_expect(bar, bytes * n_copy);
                    __syncwarp();
                    if (has)
                        bulk_copy(sm + L::S_RAW + (n_raw % NRAW) * 1024 + (lane >> 3) * 512 + part * bytes,
                                  (lane < 8 ? c.k_scale : c.v_scale) + r, bytes, bar);
                    ++n_raw;
                }
            };
            auto load_v = [&](int j, int use0, int row) {
                const int n = min(KEYS, it.end - j * KEYS);
                for (int h = 0; h < SPT; ++h) {
                    const int use = use0 + h;
                    if (!acquire(use)) return;
                    uint64_t *bar = full + use % NSLOT;
                    const uint32_t dst = ring + (use % NSLOT) * L::SLOT;
                    // bf16: half of the keys, all dims; pairs and codes: all keys, half of the dims
                    constexpr bool BY_DIMS = E4M3 || PAIR;
                    constexpr int NCOL = E4M3 ? 1 : PAIR ? 2 : 4;
                    constexpr uint32_t COL = PAIR ? BOX : BOX / 2;
                    const int keys = BY_DIMS ? n : max(0, min(64, n - 64 * h));
                    const int parts = (keys + vr - 1) / vr;
                    if (lane == 0) {
                        if (parts > 0) bulk_expect(bar, (uint32_t)(parts * NCOL * vr * 128));
                        else mbar_arrive(bar);
                    }
                    __syncwarp();
                    const int part = lane / NCOL, col = lane % NCOL;
                    const int r = __shfl_sync(kFullMask, row, (part * (vr >> 4) + (BY_DIMS ? 0 : 4 * h)) & 7);
                    if (part < parts)
                        tma_load_2d(dst + col * COL + part * vr * 128, &p.tm_v,
                                    (BY_DIMS ? (PAIR ? rank : h) * 128 : 0) + col * 64, r, bar);
                    n_use = use + 1;
                }
            };
            const int n = it.b - it.a, base = n_use;
            int row = page_row(it.a), row1 = page_row(it.a + 1);
            if (n_item > 0) {
                if (lane == 0) ok = wait_bar(q_free, (uint32_t)(n_item - 1) & 1u, p.wait_ns);
                ok = __shfl_sync(kFullMask, ok, 0);
                if (!ok) break;
            }
            ++n_item;
            if (lane == 0) {
                bulk_expect(q_full, (uint32_t)(4 * 128 * p.n_rep * p.cta_tok));
                for (int b = 0; b < 4 && !p.withhold; ++b)
                    tma_load_3d(sq + b * BOX, &p.tm_q, b * 64, it.g * p.n_rep, it.row0, q_full);
            }
            __syncwarp();
            load_k(it.a, base + use_k<SPT>(0), row);
            for (int i = 0; i < n && ok; ++i) {
                const int row2 = page_row(it.a + i + 2);
                if (i + 1 < n) load_k(it.a + i + 1, base + use_k<SPT>(i + 1), row1);
                if (ok) load_v(it.a + i, base + use_v<SPT>(i, n), row);
                row = row1;
                row1 = row2;
            }
        }
        bad = __any_sync(kFullMask, bad);
        if (lane == 0) {
            if (bad) report(kBadPage);
            if (!ok) report(kTimeout);
            // No copy may land after the CTA ends (where all went well, all have).
            if (n_item > 0) wait_bar(q_full, (uint32_t)(n_item - 1) & 1u, p.wait_ns);
            for (int u = max(0, n_use - NSLOT); u < n_use; ++u)
                wait_bar(full + u % NSLOT, (uint32_t)(u / NSLOT) & 1u, kWaitNs);
            for (int u = max(0, n_raw - NRAW); u < n_raw; ++u)
                wait_bar(raw_full + u % NRAW, (uint32_t)(u / NRAW) & 1u, kWaitNs);
            // Nor may an arrival that a commit owes: the last use of every slot, the
            // last item's Q.
            const uint64_t lim = ok ? p.wait_ns : kDrainNs;
            for (int u = max(0, n_use - NSLOT); u < n_use; ++u)
                wait_bar(empty + u % NSLOT, (uint32_t)(u / NSLOT) & 1u, lim);
            if (n_item > 0) wait_bar(q_free, (uint32_t)(n_item - 1) & 1u, lim);
        }
        __syncwarp();
    } else if (warp == L::W_MMA) {
        // ------------------------------------------------------ MMA issue
        // One elected thread.  Descriptors are a base per operand plus a constant step:
        // what is left to compute per instruction is one addition.
        if (PAIR && rank) {
            // The odd CTA tells the issuing thread what has landed here.
            if (elect_one()) {
                bool ok = true;
                int u = 0, n_item = 0;
                while (ok && walk.next(p, it)) {
                    if (it.n_kv == 0) continue;
                    ok = wait_bar(q_full, (uint32_t)n_item & 1u, p.wait_ns);
                    if (ok) mbar_arrive_at(peer_q, 0);
                    for (const int end = u + 2 * (it.b - it.a); u < end && ok; ++u) {
                        ok = full_wait(u);
                        if (ok) mbar_arrive_at(peer_full + u % NSLOT, 0);
                    }
                    ++n_item;
                }
                if (!ok) report(kTimeout);
            }
        } else if (elect_one()) {
            constexpr Kind KIND = E4M3 ? Kind::E4M3 : Kind::BF16;
            constexpr int M = PAIR ? 256 : 128;
            constexpr uint32_t ID_S = instr_desc<KIND>(M, KEYS, false, false);
            constexpr uint32_t ID_O = instr_desc<KIND>(M, E4M3 ? 128 : 256, false, true);
            constexpr uint32_t ID_O_LO = ID_O | E5M2_A;  // codes: the weights' second parts
            constexpr int STEP = E4M3 ? 32 : 16;  // keys per instruction of P V
            const uint64_t dq = smem_desc_sw128(sq, 16, 1024);
            const uint64_t dk = smem_desc_sw128(ring, 16, 1024);
            const uint64_t dv = smem_desc_sw128(ring, E4M3 || PAIR ? BOX : BOX / 2, 1024);
            auto done = [&](uint64_t *bar) {
                if constexpr (PAIR) commit_pair(smem_u32(bar));
                else commit(smem_u32(bar));
            };
            auto landed = [&](int u) {  // in both CTAs of a pair
                return full_wait(u) && (!PAIR || spin_on(peer_full + u % NSLOT, (uint32_t)(u / NSLOT) & 1u, p.wait_ns));
            };
            auto wait_both = [&](uint64_t *bar, uint32_t parity) {  // for arrivals from both CTAs of a pair
                return PAIR ? spin_on(bar, parity, p.wait_ns) : wait_bar(bar, parity, p.wait_ns);
            };
            bool ok = true;
            int jt = 0, base = 0, n_item = 0;
            // S of tile `tile`, from the ring's uses u, u + 1.
            auto score = [&](int tile, int u) {
                const uint32_t d = tm + TM_S + 128 * (tile & 1);
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    const int use = u + (SPT == 2 ? h : 0);
                    if ((SPT == 2 || h == 0) && !landed(use)) return false;
                    fence_after_sync();
                    const uint64_t a = dq + (uint64_t)h * (2 * BOX >> 4);
                    const uint64_t b = dk + (uint64_t)(use % NSLOT) * (L::SLOT >> 4) + (PAIR ? h * (BOX >> 4) : 0);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        // bf16: box k / 4 of the half (a pair's boxes have 64 keys); e4m3: the hi,
                        // then the lo part
                        constexpr uint32_t KBOX = PAIR ? BOX / 2 : BOX;
                        const uint64_t ak = a + ((k >> 2) * (BOX >> 4) + (k & 3) * 2);
                        const uint64_t bk = b + ((E4M3 ? 0 : (k >> 2) * (KBOX >> 4)) + (k & 3) * 2);
                        if constexpr (PAIR) mma_pair(d, ak, bk, ID_S, k ? 1u : (uint32_t)h);
                        else mma<KIND>(d, ak, bk, ID_S, k ? 1u : (uint32_t)h);
                    }
                }
                done(bar_s + (tile & 1));
                for (int h = 0; h < SPT; ++h) done(empty + (u + h) % NSLOT);
                return true;
            };
            // O (+)= P V of half h of a tile: `steps` instructions, twice (hi, lo) for codes.
            auto weigh = [&](uint32_t pt, int u, int h, int steps, uint32_t more) {
                const uint64_t b = dv + (uint64_t)(u % NSLOT) * (L::SLOT >> 4);
                if constexpr (PAIR) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (k < steps)
                            mma_pair_ta(tm + TM_O, pt + 64 * (k >> 2) + 8 * (k & 3), b + k * (2048 >> 4), ID_O,
                                        k ? 1u : more);
                } else if constexpr (!E4M3) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (k < steps)
                            mma_ta(tm + TM_O, pt + 64 * h + 8 * k, b + k * (2048 >> 4), ID_O,
                                   k ? 1u : more);
                } else {
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        const int part = x >> 2, k = x & 3;
                        if (k < steps)
                            mma_ta_e4m3(tm + TM_O + 128 * h, pt + 32 * k + 8 * part,
                                        b + k * (4096 >> 4), part ? ID_O_LO : ID_O, x ? 1u : more);
                    }
                }
            };
            while (ok && walk.next(p, it)) {
                if (it.n_kv == 0) continue;
                const int n = it.b - it.a;
                ok = wait_bar(E4M3 ? q_split : q_full, (uint32_t)n_item & 1u, p.wait_ns) &&
                     (!PAIR || spin_on(peer_q, (uint32_t)n_item & 1u, p.wait_ns)) && score(jt, base + use_k<SPT>(0));
                if (n == 1 && ok) done(q_free);
                for (int i = 0; i < n && ok; ++i) {
                    if (i + 1 < n) {
                        ok = score(jt + i + 1, base + use_k<SPT>(i + 1));
                        if (i + 2 == n && ok) done(q_free);
                    }
                    if (ok && i == 0 && n_item > 0) ok = wait_both(o_free, (uint32_t)(n_item - 1) & 1u);
                    const int j = jt + i, u0 = base + use_v<SPT>(i, n);
                    ok = ok && wait_both(bar_p + (j & 1), (uint32_t)(j >> 1) & 1u);
                    const int keys = min(KEYS, it.end - (it.a + i) * KEYS);
                    const uint32_t pt = tm + TM_S + 128 * (j & 1);
#pragma unroll 1
                    for (int h = 0; h < SPT; ++h) {
                        ok = ok && landed(u0 + h);
                        if (!ok) break;
                        fence_after_sync();
                        // bf16: a slot holds 64 of the keys
                        weigh(pt, u0 + h, h, ((E4M3 || PAIR ? keys : keys - 64 * h) + STEP - 1) / STEP,
                              i || (!E4M3 && h) ? 1u : 0u);
                    }
                    if (!ok) break;
                    done(bar_o + (j & 1));
                    for (int h = 0; h < SPT; ++h) done(empty + (u0 + h) % NSLOT);
                }
                jt += n;
                base += 2 * SPT * n;
                ++n_item;
            }
            if (!ok) report(kTimeout);
        }
        __syncwarp();
    } else if (E4M3 && warp >= L::W_AUX) {
        // -------------------------------------- Q in two parts, and the scales
        const int t = tid - 32 * L::W_AUX;
        constexpr int NT = 32 * AUX_WARPS;
        float *scales = reinterpret_cast<float *>(sm + L::S_SCALE);
        const float *raw = reinterpret_cast<const float *>(sm + L::S_RAW);
        float *rowk = reinterpret_cast<float *>(sm + L::S_ROWK);
        bool ok = true;
        int jt = 0, n_item = 0;
        while (ok && walk.next(p, it)) {
            if (it.n_kv == 0) continue;
            ok = __all_sync(kFullMask, wait_bar(q_full, (uint32_t)n_item & 1u, p.wait_ns));
            if (!ok) break;
            // Row r: 256 bf16 values, 16-byte chunk j of box b at chunk j ^ (r % 8).  Eight lanes
            // a row, each with 16 values of either half: all of a row is read before any of
            // it is written over.
            const int oct = lane & 7, n_rows = it.n_tok * p.n_rep;
#pragma unroll 1
            for (int r0 = (t >> 5) * 4; r0 < n_rows; r0 += NT / 8) {
                const int r = r0 + (lane >> 3);
                auto chunk = [&](int b, int j) { return sq + r * 128 + b * BOX + ((j ^ (r & 7)) << 4); };
                uint4 x[4];  // values 16 oct .. of half 0 in x[0], x[1], of half 1 in x[2], x[3]
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int j = 2 * oct + (c & 1);
                    x[c] = ld_shared16(chunk(2 * (c >> 1) + (j >> 3), j & 7));
                }
                uint32_t top = 0;  // largest magnitude, as bf16 bits
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    top = __vmaxu2(top, __vmaxu2(__vmaxu2(x[c].x & 0x7fff7fffu, x[c].y & 0x7fff7fffu),
                                                 __vmaxu2(x[c].z & 0x7fff7fffu, x[c].w & 0x7fff7fffu)));
#pragma unroll
                for (int o = 1; o < 8; o <<= 1) top = __vmaxu2(top, __shfl_xor_sync(kFullMask, top, o));
                // A power of two that takes the largest value into [128, 256).
                const int e = min(max((int)max(top >> 16, top & 0xffffu) >> 7, 8), 254);
                const float up = __uint_as_float((uint32_t)(261 - e) << 23);
                if (oct == 0) rowk[(n_item & 1) * ROWS + r] = __uint_as_float((uint32_t)(e - 7) << 23);
                __syncwarp();
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const uint4 v = x[2 * h + (w >> 1)];
                        const uint32_t v0 = w & 1 ? v.z : v.x, v1 = w & 1 ? v.w : v.y;
                        uint16_t h0, h1, l0, l1;
                        split2(f16x2(__uint_as_float(v0 << 16) * up, __uint_as_float(v0 & 0xffff0000u) * up),
                               h0, l0);
                        split2(f16x2(__uint_as_float(v1 << 16) * up, __uint_as_float(v1 & 0xffff0000u) * up),
                               h1, l1);
                        hi[w] = h0 | (uint32_t)h1 << 16;
                        lo[w] = l0 | (uint32_t)l1 << 16;
                    }
                    st_shared16(chunk(2 * h, oct), make_uint4(hi[0], hi[1], hi[2], hi[3]));
                    st_shared16(chunk(2 * h + 1, oct), make_uint4(lo[0], lo[1], lo[2], lo[3]));
                }
            }
            fence_smem_to_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_split);
            for (int j = it.a; j < it.b; ++j, ++jt) {
                ok = wait_bar(raw_full + jt % NRAW, (uint32_t)(jt / NRAW) & 1u, p.wait_ns);
                // The stage was read by the softmax two tiles back.
                if (jt >= 2) ok = ok && wait_bar(bar_p + (jt & 1), (uint32_t)((jt - 2) >> 1) & 1u, p.wait_ns);
                ok = __all_sync(kFullMask, ok);
                if (!ok) break;
                float *st = scales + (jt & 1) * 3 * KEYS;
                const float *from = raw + (jt % NRAW) * 2 * KEYS;
#pragma unroll
                for (int x = t; x < KEYS; x += NT) {
                    const bool in = j * KEYS + x < it.end;
                    // The smallest scale that an append writes stands for zero too: it keeps
                    // the key in the softmax's sum.  Keys past the end: any finite value.
                    const float ks = in ? from[x] : 0.f;
                    const float vs = in ? fmaxf(from[KEYS + x], kScaleMin) : 1.f;
                    st[x] = ks * p.scale_log2;
                    st[KEYS + x] = log2f(vs);
                    st[2 * KEYS + x] = 1.f / vs;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(sc_full + (jt & 1));
            }
            ++n_item;
        }
        if (!ok && lane == 0) report(kTimeout);
    } else if (warp < L::SOFTMAX) {
        // -------------------------------------------------------- softmax
        // The warps w, w + 4, .. share rows 32 (w % 4) ..; each takes KPT of a tile's keys
        // and COLS of O's columns.  They agree on a row's maximum through red[], and
        // to stop, at the same barrier.
        //
        // The reference maximum moves up when a tile's maximum passes it by
        // more than kLazy (log2): then O and the sum are rescaled, which needs
        // the tile before's product finished.  bf16 holds a weight of any size
        // alike; the codes' parts hold at most 448, so there the weights sit 2^6 up
        // and may grow by 2^2.
        //
        // Codes: below 2^-6 a weight is off by up to 2^-14, 2^-20 of the reference.  Where one
        // key's weight is far above the many that follow, that would add up, so there the
        // reference also moves down, to a tile's maximum 2^kSink below it (and no more than
        // 2^kFall below the highest: such weights are nothing beside what is summed, and the
        // sums would overflow).  A tile's reference is then at most 2^5 times its largest
        // weight, and all these errors add up to at most 2^7 2^-20 2^5 = 2^-8 of the sum of
        // the weights, times the largest code, whatever the number of keys.  Scores of
        // random rows of size 1 hardly ever move it: 64 x 4096 80 us, as without; of size 3, 89
        // for 85.  (To the maximum of the last 8 tiles, every 8, 1 below: 85 and 89.)  A tile of
        // which a row attends nothing, its last, moves it too, for nothing; to test for that costs 1%.
        constexpr float kLazy = E4M3 ? 2.f : 8.f;
        constexpr float kUp = E4M3 ? 6.f : 0.f;
        constexpr float kShift = E4M3 ? 8.f : 0.f;  // split4 takes weights times 2^-8
        constexpr float kSink = 5.f, kFall = 40.f;
        constexpr int KPT = KEYS / PARTS, COLS = D / PARTS, NG = 32 * PARTS;
        const int part = warp >> 2, quad = warp & 3, r = 32 * quad + lane;
        const uint32_t lane_off = (uint32_t)(32 * quad) << 16;
        // The quad's own part of the exchange area: the warps of a quad are in step with each
        // other, not with those of other quads.  At an item's end it holds the sums.
        float *red = reinterpret_cast<float *>(sm + L::S_RED) + quad * (2 * PARTS * 32) + lane;
        const int tok = (int)(r * p.rep_inv >> 16), h = r - tok * p.n_rep;
        const float *scales = reinterpret_cast<const float *>(sm + L::S_SCALE);
        const float *rowk = reinterpret_cast<const float *>(sm + L::S_ROWK);
        bool dead = false, fault = false;
        int jt = 0, base = 0, n_item = 0;
        auto wait_o = [&](int tile, uint64_t lim) {
            return wait_bar(bar_o + (tile & 1), (uint32_t)(tile >> 1) & 1u, lim);
        };
        while (!dead && walk.next(p, it)) {
            const bool mine = tok < it.n_tok;  // this row exists
            const bool some = __any_sync(kFullMask, mine);
            const int64_t grow = it.row0 + tok;
            const int gh = it.g * p.n_rep + h;
            if (it.n_kv == 0) {
                // Lengths that cannot be used: zeros.
                if (mine) {
                    for (int d = COLS * part; d < COLS * part + COLS; d += 4) {
                        using T = std::conditional_t<OUT_BF16, __nv_bfloat16, float>;
                        Elem<T>::store4(static_cast<T *>(p.a.out) + grow * p.a.out_stride + gh * D + d,
                                        make_float4(0.f, 0.f, 0.f, 0.f));
                    }
                    if (part == 0 && p.a.lse) p.a.lse[grow * p.a.lse_stride + gh] = -INFINITY;
                }
                continue;
            }
            const int n = it.b - it.a;
            const bool begins = it.a == 0, ends = it.b == it.n_kv, whole = begins && ends;
            if (whole && mine && p.a.gate) {
                // The row's gates come into L2 while its keys are worked on.
                const __nv_bfloat16 *g = static_cast<const __nv_bfloat16 *>(p.a.gate) + grow * p.a.gate_stride +
                                         gh * D + COLS * part;
#pragma unroll
                for (int x = 0; x < COLS; x += 64)
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(g + x));
            }
            float m_ref = -INFINITY, l = 0.f;
            float lowest = -INFINITY;  // codes: how far the reference may go down
            float row_factor = 1.f;
            for (int i = 0; i < n; ++i) {
                const int j = jt + i, k0 = (it.a + i) * KEYS;
                bool ok = wait_bar(bar_s + (j & 1), (uint32_t)(j >> 1) & 1u, p.wait_ns);
                if (E4M3) ok = ok && wait_bar(sc_full + (j & 1), (uint32_t)(j >> 1) & 1u, p.wait_ns);
                ok = __all_sync(kFullMask, ok);
                // bf16: in two chunks of the thread's keys, read twice, which is half the code
                // of holding all of them (the roles share the instruction cache).  Codes: in one
                // that is held, since their scaling costs more than the code.
                constexpr int NCH = KPT / 32;
                const uint32_t st = tm + lane_off + TM_S + 128 * (j & 1) + KPT * part;
                const float *sck = scales + (j & 1) * 3 * KEYS + KPT * part;
                // Keys this row attends, of this thread's (a row that does not exist: all
                // of them, whatever they are).
                const int lim = mine ? it.pos0 + tok + 1 - k0 - KPT * part : KPT;
                const bool masked = __any_sync(kFullMask, lim < KPT);
                auto load = [&](int c, float (&s)[32]) {
                    tmem_ld32(st + 32 * c, s);
                    if constexpr (E4M3) {
                        const float4 *sk = reinterpret_cast<const float4 *>(sck);
                        const float4 *lv = sk + KEYS / 4;
                        const float2 rf = make_float2(row_factor, row_factor);
#pragma unroll
                        for (int x = 0; x < 8; ++x) {
                            const float4 a = sk[x], b = lv[x];
                            const float2 u = fma2(mul2(make_float2(s[4 * x], s[4 * x + 1]), rf),
                                                  make_float2(a.x, a.y), make_float2(b.x, b.y));
                            const float2 v = fma2(mul2(make_float2(s[4 * x + 2], s[4 * x + 3]), rf),
                                                  make_float2(a.z, a.w), make_float2(b.z, b.w));
                            s[4 * x] = u.x;
                            s[4 * x + 1] = u.y;
                            s[4 * x + 2] = v.x;
                            s[4 * x + 3] = v.y;
                        }
                    }
                    if (masked) {
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            if (x + 32 * c >= lim) s[x] = -INFINITY;
                    }
                };
                float top = -INFINITY;
                float s[32];
                if (some && ok) {
                    fence_after_sync();
                    if (E4M3 && i == 0) row_factor = rowk[(n_item & 1) * ROWS + r];
#pragma unroll 1
                    for (int c = 0; c < NCH; ++c) {
                        load(c, s);
                        float t4[4] = {top, s[1], s[2], s[3]};
                        t4[0] = fmaxf(t4[0], s[0]);
#pragma unroll
                        for (int x = 4; x < 32; x += 4) {
                            t4[0] = fmaxf(t4[0], s[x]);
                            t4[1] = fmaxf(t4[1], s[x + 1]);
                            t4[2] = fmaxf(t4[2], s[x + 2]);
                            t4[3] = fmaxf(t4[3], s[x + 3]);
                        }
                        top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
                    }
                    if (!E4M3) top *= p.scale_log2;
                    red[((j & 1) * PARTS + part) * 32] = top;
                }
                dead = group_sync_or(1 + quad, NG, !ok || fault);
                if (dead) break;
                // The MMA takes V's keys in steps of 16 (32 codes): what pages hold between
                // the sequence's end and the step's becomes zero.  (Just before P's arrival instead:
                // 64 ragged sequences of up to 8190 tokens over codes 90.2 us for 88.6, over bf16 and
                // shorter ones alike.)
                const int keys = it.end - k0;
                constexpr int STEP = E4M3 ? 32 : 16;
                const bool clears = keys < KEYS && (keys & (STEP - 1));
                if (clears) {
                    const int up = (keys + STEP - 1) & ~(STEP - 1);
                    // 16 bytes each: bf16, 4 boxes of 8 a key; pairs, 2 boxes; codes, 2 slots.
                    constexpr int CH = E4M3 || PAIR ? 16 : 32;
                    constexpr uint32_t COL = PAIR ? BOX : BOX / 2;
                    const int u0 = base + use_v<SPT>(i, n);
                    const int u = E4M3 || PAIR ? u0 : u0 + (keys >> 6);
                    bool okv = full_wait(u);
                    if (E4M3) okv = okv && full_wait(u0 + 1);
                    fault = fault || !__all_sync(kFullMask, okv);
                    if (!fault) {
                        for (int x = tid; x < (up - keys) * CH; x += 32 * L::SOFTMAX) {
                            const int key = keys + x / CH, ch = x % CH;
                            const int uu = E4M3 ? u0 + (ch >> 3) : u;
                            const uint32_t at = ring + (uu % NSLOT) * L::SLOT + (E4M3 ? 0 : (ch >> 3) * COL) +
                                                (E4M3 || PAIR ? key : key & 63) * 128 + (ch & 7) * 16;
                            st_shared16(at, make_uint4(0, 0, 0, 0));
                        }
                    }
                    fence_smem_to_async();
                }
                if (some) {
                    top = -INFINITY;
#pragma unroll
                    for (int x = 0; x < PARTS; ++x)
                        top = fmaxf(top, red[((j & 1) * PARTS + x) * 32]);
                    const bool first = m_ref == -INFINITY;
                    bool moves = mine && !first && top > m_ref + kLazy;
                    float to = top;
                    if constexpr (E4M3) {
                        lowest = fmaxf(lowest, m_ref - kFall);
                        const float down = fmaxf(top, lowest);
                        if (mine && down < m_ref - kSink) {
                            moves = true;
                            to = down;
                        }
                    }
                    const float alpha = moves ? exp2_fast(m_ref - to) : 1.f;
                    if (first || moves) m_ref = to;
                    l *= alpha;
                    const bool rescale = __any_sync(kFullMask, moves) && i > 0;
                    // -inf (nothing attended yet) as 0: every exponent below is -inf then.
                    const float sub = (m_ref == -INFINITY ? 0.f : m_ref) - kUp + kShift;
                    const float2 sub2 = make_float2(-sub, -sub);
                    float2 l2 = make_float2(0.f, 0.f), l3 = l2;
                    // P goes over the S that this warp has read: bf16, 2 keys a column; codes,
                    // 4 a column, the hi parts of all its keys and then the lo parts.
#pragma unroll 1
                    for (int c = 0; c < NCH; ++c) {
                        if (NCH > 1) load(c, s);
                        uint32_t pk[16];
                        if constexpr (!E4M3) {
                            const float2 cl = make_float2(p.scale_log2, p.scale_log2);
#pragma unroll
                            for (int x = 0; x < 16; x += 2) {
                                const float2 u = fma2(make_float2(s[2 * x], s[2 * x + 1]), cl, sub2);
                                const float2 v = fma2(make_float2(s[2 * x + 2], s[2 * x + 3]), cl, sub2);
                                const float2 a = make_float2(exp2_fast(u.x), exp2_fast(u.y));
                                const float2 b = make_float2(exp2_fast(v.x), exp2_fast(v.y));
                                l2 = add2(l2, a);
                                l3 = add2(l3, b);
                                pk[x] = bf16x2(a.x, a.y);
                                pk[x + 1] = bf16x2(b.x, b.y);
                            }
                        } else {
                            const float4 *rs = reinterpret_cast<const float4 *>(sck + 2 * KEYS);
#pragma unroll
                            for (int x = 0; x < 8; ++x) {
                                const float4 f = rs[x];
                                const float2 u = add2(make_float2(s[4 * x], s[4 * x + 1]), sub2);
                                const float2 v = add2(make_float2(s[4 * x + 2], s[4 * x + 3]), sub2);
                                const float2 a = make_float2(exp2_fast(u.x), exp2_fast(u.y));
                                const float2 b = make_float2(exp2_fast(v.x), exp2_fast(v.y));
                                l2 = fma2(a, make_float2(f.x, f.y), l2);
                                l3 = fma2(b, make_float2(f.z, f.w), l3);
                                split4(a.x, a.y, b.x, b.y, pk[x], pk[8 + x]);
                            }
                        }
                        __syncwarp();
                        tmem_st16(st + 16 * c, pk);
                    }
                    l += (l2.x + l2.y) + (l3.x + l3.y);
                    if (rescale) {
                        fault = !__all_sync(kFullMask, wait_o(j - 1, p.wait_ns)) || fault;
                        if (!fault) {
                            fence_after_sync();
#pragma unroll 1
                            for (int x = 0; x < COLS; x += 32) {
                                float o[32];
                                tmem_ld32(tm + lane_off + TM_O + COLS * part + x, o);
#pragma unroll
                                for (int y = 0; y < 32; ++y) o[y] *= alpha;
                                tmem_st32(tm + lane_off + TM_O + COLS * part + x, o);
                            }
                        }
                    }
                }
                fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    // The whole warp's zeros, which the barrier above has brought to this lane,
                    // before its arrival at the other CTA.
                    if (PAIR && clears) fence_cluster();
                    arrive_mma(bar_p + (j & 1));
                }
            }
            if (dead) break;
            jt += n;
            base += 2 * SPT * n;
            ++n_item;
            // The item's end: the row's sum over its threads, then O.
            l *= E4M3 ? 256.f : 1.f;  // 2^kShift
            group_sync_or(1 + quad, NG, false);  // every maximum has been read
            red[part * 32] = l;
            // For accesses of 32 bytes a row, 16 a lane: the two rows of this lane's pair.
            using T = std::conditional_t<OUT_BF16, __nv_bfloat16, float>;
            constexpr int PER = 16 / sizeof(T);  // values in 16 bytes
            const int odd = lane & 1;
            bool has[2];
            const uint4 *gate_at[2];
            T *out_at[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int r2 = r - odd + k, t2 = (int)(r2 * p.rep_inv >> 16);
                const int col = (it.g * p.n_rep + r2 - t2 * p.n_rep) * D + COLS * part;
                has[k] = t2 < it.n_tok;
                gate_at[k] = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.a.gate) +
                                                             (it.row0 + t2) * p.a.gate_stride + col + 8 * odd);
                out_at[k] = static_cast<T *>(p.a.out) + (it.row0 + t2) * p.a.out_stride + col + PER * odd;
            }
            // Gates of 16 columns of the pair's rows, fetched a block ahead.
            const bool gated = whole && p.a.gate;
            uint4 gates[2] = {};
            auto fetch_gate = [&](int x) {
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    if (gated && has[k] && x < COLS) gates[k] = __ldg(gate_at[k] + x / 8);
            };
            fetch_gate(0);
            const bool ok = wait_o(jt - 1, p.wait_ns);
            dead = group_sync_or(1 + quad, NG, !ok || fault);
            if (dead) break;
            l = 0.f;  // in one order in all its threads
#pragma unroll
            for (int x = 0; x < PARTS; ++x) l += red[x * 32];
            group_sync_or(1 + quad, NG, false);  // the next tile writes there
            fence_after_sync();
            const int slot = 2 * blockIdx.x + (begins ? 1 : 0);
            const float inv = l > 0.f ? 1.f / l : 0.f;
            uint32_t gate_top = 0;  // magnitudes of the row's gates, by halves of a word
            if (some) {
#pragma unroll 1
                for (int x = 0; x < COLS; x += 16) {
                    float o[16];
                    __syncwarp();
                    tmem_ld16(tm + lane_off + TM_O + COLS * part + x, o);
                    if (!whole) {
                        float4 *po = reinterpret_cast<float4 *>(p.part_o) +
                                     ((size_t)slot * (D / 4) + (COLS * part + x) / 4) * ROWS + r;
                        if (mine)
#pragma unroll
                            for (int y = 0; y < 4; ++y)
                                po[y * ROWS] = make_float4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
                        continue;
                    }
                    if (p.a.gate) {
                        uint4 g[2] = {gates[0], gates[1]};
                        fetch_gate(x + 16);
                        transpose2(g, lane);
#pragma unroll
                        for (int y = 0; y < 16; y += 2) {
                            const uint4 c8 = g[y >> 3];
                            const uint32_t w4[4] = {c8.x, c8.y, c8.z, c8.w};
                            gate2(o[y], o[y + 1], w4[(y & 7) >> 1], inv);
                            gate_top = __vmaxu2(gate_top, w4[(y & 7) >> 1] & 0x7fff7fffu);
                        }
                    } else {
#pragma unroll
                        for (int y = 0; y < 16; ++y) o[y] *= inv;
                    }
                    // 32 bytes of its row in each lane become 16 bytes of both rows of the pair.
#pragma unroll
                    for (int y = 0; y < 16; y += 2 * PER) {
                        uint4 q2[2];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const float *v = o + y + PER * k;
                            if constexpr (OUT_BF16)
                                q2[k] = make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]),
                                                   bf16x2(v[6], v[7]));
                            else
                                q2[k] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]),
                                                   __float_as_uint(v[2]), __float_as_uint(v[3]));
                        }
                        transpose2(q2, lane);
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            if (has[k]) *reinterpret_cast<uint4 *>(out_at[k] + x + y) = q2[k];
                    }
                }
                const bool far = mine && max(gate_top >> 16, gate_top & 0xffffu) >= FAR_GATE;
                if (__any_sync(kFullMask, far)) {
                    // (The stores above, by two lanes a row, come before the warp's barrier here.)
                    const int64_t col = gh * D + COLS * part;
                    const __nv_bfloat16 *g = static_cast<const __nv_bfloat16 *>(p.a.gate) + grow * p.a.gate_stride + col;
                    T *to = static_cast<T *>(p.a.out) + grow * p.a.out_stride + col;
#pragma unroll 1
                    for (int x = 0; x < COLS; x += 16) {
                        float o[16];
                        __syncwarp();
                        tmem_ld16(tm + lane_off + TM_O + COLS * part + x, o);
                        if (far)
#pragma unroll
                            for (int y = 0; y < 16; y += 4) {
                                const float4 f = Elem<__nv_bfloat16>::load4(g + x + y);
                                Elem<T>::store4(to + x + y, make_float4(gate_any(o[y] * inv, f.x), gate_any(o[y + 1] * inv, f.y),
                                                                        gate_any(o[y + 2] * inv, f.z),
                                                                        gate_any(o[y + 3] * inv, f.w)));
                            }
                    }
                }
                if (mine && part == 0) {
                    if (!whole) {
                        float *ml = p.part_ml + ((size_t)slot * ROWS + r) * 2;
                        ml[0] = m_ref - kUp;
                        ml[1] = l;
                    } else if (p.a.lse) {
                        p.a.lse[grow * p.a.lse_stride + gh] =
                            l > 0.f ? (m_ref - kUp + __log2f(l)) * 0.6931471805599453f : -INFINITY;
                    }
                }
            }
            fence_before_sync();
            __syncwarp();
            if (lane == 0) arrive_mma(o_free);
            if (!whole && tid == 0) {
                if (!begins) {
                    desc->head = ends ? 2 : 1;
                } else {
                    desc->tail = 1;
                    desc->row0 = it.row0;
                    desc->n_tok = it.n_tok;
                    desc->g = it.g;
                }
            }
        }
        if ((dead || fault) && lane == 0) report(kTimeout);
        // The product before the last is waited for by nobody: its commit must land too.
        if (jt >= 2) wait_o(jt - 2, dead ? kDrainNs : p.wait_ns);
        if (dead && jt >= 1) wait_o(jt - 1, kDrainNs);
    }

    fence_before_sync();
    __syncthreads();
    // Neither CTA of a pair ends before the other's last arrival at it.
    if constexpr (PAIR) cluster_sync();
    if (warp == 0) {
        fence_after_sync();
        if constexpr (PAIR) tmem_free_pair(tm, TM_COLS);
        else tmem_free(tm, TM_COLS);
    }
}

// --------------------------------------------------------------- combine

// COMBINE_SPLIT blocks join the parts of the item that CTA blockIdx.x / COMBINE_SPLIT began
// and did not end: y = (sum_i 2^{m_i - m} O_i) / (sum_i 2^{m_i - m} l_i) * sigmoid(gate).
// A warp takes 8 rows (lane % 8) by 16 dims (4 a lane) at a time, the parts four at once: it
// is a chain of loads, so what counts is how few of them wait for another.
constexpr int COMBINE_SPLIT = 8;
constexpr int COMBINE_WARPS = 8;
template <bool OUT_BF16>
__global__ void __launch_bounds__(32 * COMBINE_WARPS) attn_paged_combine(const AttnParams p, int n_cta) {
    wait_for_predecessor();
    release_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int cta = blockIdx.x / COMBINE_SPLIT, share = blockIdx.x % COMBINE_SPLIT;
    if (blockIdx.x == 0 && warp == 0) {
        int st = 0;
        for (int i = lane; i < n_cta; i += 32) st = max(st, p.desc[i].status);
        st = __reduce_max_sync(kFullMask, st);
        if (lane == 0) *p.status = st;
    }
    // The parts: slot 2 cta + 1, then slots 2 i of the CTAs after it up to the one that ends
    // the item.  None between is without a part: CTAs with nothing to do come last.
    const Desc d = p.desc[cta];
    // (The CTAs of one rank of the pairs, where they work in pairs.)
    int n_part = 1;
    for (int k0 = 1; cta + k0 * p.pair < n_cta; k0 += 32) {
        const int i = cta + (k0 + lane) * p.pair;
        const uint32_t ends = __ballot_sync(kFullMask, i < n_cta && p.desc[i].head == 2);
        if (ends) {
            n_part = k0 + __ffs(ends);
            break;
        }
    }
    if (!d.tail) return;
    const int rows = d.n_tok * p.n_rep;
    const int n_task = ((rows + 7) >> 3) * (D / 16);
    for (int task = share * COMBINE_WARPS + warp; task < n_task; task += COMBINE_SPLIT * COMBINE_WARPS) {
        const int r = (task / (D / 16)) * 8 + (lane & 7), c4 = (task % (D / 16)) * 4 + (lane >> 3);
        if (r >= rows) continue;
        const int tok = r / p.n_rep, gh = d.g * p.n_rep + r - tok * p.n_rep;
        const int64_t grow = d.row0 + tok;
        float4 gate = make_float4(0.f, 0.f, 0.f, 0.f);
        if (p.a.gate)
            gate = Elem<__nv_bfloat16>::load4(static_cast<const __nv_bfloat16 *>(p.a.gate) +
                                              grow * p.a.gate_stride + gh * D + 4 * c4);
        float m = -INFINITY, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k0 = 0; k0 < n_part; k0 += 4) {
            float2 ml[4];
            float4 a[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int i = cta + min(k0 + k, n_part - 1) * p.pair;
                const size_t slot = 2 * i + (i == cta);
                ml[k] = __ldg(reinterpret_cast<const float2 *>(p.part_ml) + slot * ROWS + r);
                a[k] = __ldg(reinterpret_cast<const float4 *>(p.part_o) + (slot * (D / 4) + c4) * ROWS + r);
                if (k0 + k >= n_part) ml[k].x = -INFINITY;
            }
            const float top = fmaxf(fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)), m);
            if (top == -INFINITY) continue;
            const float keep = exp2_fast(m - top);
            m = top;
            l *= keep;
            o = make_float4(o.x * keep, o.y * keep, o.z * keep, o.w * keep);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                // A part in which the row attends nothing has m = -inf and adds nothing.
                const float f = exp2_fast(ml[k].x - top);
                l = fmaf(f, ml[k].y, l);
                o.x = fmaf(f, a[k].x, o.x);
                o.y = fmaf(f, a[k].y, o.y);
                o.z = fmaf(f, a[k].z, o.z);
                o.w = fmaf(f, a[k].w, o.w);
            }
        }
        const float inv = l > 0.f ? 1.f / l : 0.f;
        o = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
        if (p.a.gate) {
            o.x = __fdividef(o.x, 1.f + __expf(-gate.x));
            o.y = __fdividef(o.y, 1.f + __expf(-gate.y));
            o.z = __fdividef(o.z, 1.f + __expf(-gate.z));
            o.w = __fdividef(o.w, 1.f + __expf(-gate.w));
        }
        using T = std::conditional_t<OUT_BF16, __nv_bfloat16, float>;
        Elem<T>::store4(static_cast<T *>(p.a.out) + grow * p.a.out_stride + gh * D + 4 * c4, o);
        if (c4 == 0 && p.a.lse)
            p.a.lse[grow * p.a.lse_stride + gh] =
                l > 0.f ? (m + __log2f(l)) * 0.6931471805599453f : -INFINITY;
    }
}

namespace {

constexpr size_t WS_DESC = 256;
size_t ws_ml(int n_cta) { return WS_DESC + (((size_t)n_cta * sizeof(Desc) + 255) & ~(size_t)255); }
size_t ws_o(int n_cta) { return ws_ml(n_cta) + (size_t)2 * n_cta * ROWS * 2 * 4; }

template <bool E4M3, bool PAIR, bool OUT_BF16>
cudaError_t launch_attn(const AttnParams &p, int dev, int n_cta, cudaStream_t s) {
    using L = Layout<E4M3>;
    const auto kern = attn_paged_kernel<E4M3, PAIR, OUT_BF16>;
    cudaError_t e = cudaSuccess;
    // The kernel's shared-memory limit, raised once per device (setting it twice is harmless).
    static std::atomic<uint64_t> raised{0};
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (!(raised.load(std::memory_order_relaxed) & bit) || !bit) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::S_BYTES);
        if (e != cudaSuccess) {
            (void)cudaGetLastError();
            return e;
        }
        raised.fetch_or(bit, std::memory_order_relaxed);
    }
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)n_cta);
    cfg.blockDim = dim3(L::THREADS);
    cfg.dynamicSmemBytes = L::S_BYTES;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = PAIR ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, kern, p);
    if (e == cudaSuccess) {
        cfg.numAttrs = 1;
        cfg.gridDim = dim3((unsigned)(n_cta * COMBINE_SPLIT));
        cfg.blockDim = dim3(32 * COMBINE_WARPS);
        cfg.dynamicSmemBytes = 0;
        e = cudaLaunchKernelEx(&cfg, attn_paged_combine<OUT_BF16>, p, n_cta);
    }
    if (e != cudaSuccess) (void)cudaGetLastError();
    return e;
}

}  // namespace
}  // namespace paged

size_t attn_paged_workspace_bytes(int n_sm) {
    return paged::ws_o(n_sm) + (size_t)2 * n_sm * paged::ROWS * paged::D * 4;
}

// wait_ns 0: the ordinary limit; otherwise the diagnostic with that limit.
cudaError_t launch_attn_paged(const gdr_attn_paged_args *a, void *workspace, uint64_t wait_ns, cudaStream_t s) {
    using namespace paged;
    const gdr_kv_pages &c = a->pages;
    int dev = 0, n_sm = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return cudaGetLastError();
    AttnParams p = {};
    p.a = *a;
    p.shift = log2_of(c.page_size);
    p.n_rep = a->H_q / c.H_kv;
    p.cta_tok = ROWS / p.n_rep;
    // In pairs where a sequence's new tokens fill a pair's 256 rows on average, which is as much
    // as the host knows: a chunk of 2048 tokens takes 228 us so and 253 alone, while of a decode
    // step's 8 rows a pair would give one CTA none.
    const bool pair = c.kv_dtype == GDR_BF16 && a->n_tok * p.n_rep >= (int64_t)2 * ROWS * c.n_seq;
    p.pair = pair ? 2 : 1;
    p.tile_tok = p.cta_tok * p.pair;
    const int n_cta = n_sm / p.pair * p.pair;
    p.rep_inv = (65536u + p.n_rep - 1) / p.n_rep;
    const bool codes = c.kv_dtype == GDR_E4M3;
    const int k_keys = pair ? KEYS / 2 : KEYS;           // keys of a K slot
    const int v_keys = codes || pair ? KEYS : KEYS / 2;  // of a V slot
    p.k_rows = c.page_size < k_keys ? c.page_size : k_keys;
    p.v_rows = c.page_size < v_keys ? c.page_size : v_keys;
    p.n_rows = c.n_pages * c.H_kv * c.page_size;
    p.scale_log2 = (float)((double)a->scale * 1.4426950408889634);
    p.withhold = wait_ns != 0;
    p.wait_ns = wait_ns ? wait_ns : kWaitNs;
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    p.status = reinterpret_cast<int *>(ws);
    p.desc = reinterpret_cast<Desc *>(ws + WS_DESC);
    p.part_ml = reinterpret_cast<float *>(ws + ws_ml(n_sm));
    p.part_o = reinterpret_cast<float *>(ws + ws_o(n_sm));
    const bool maps =
        encode_bf16_3d(&p.tm_q, a->q, D, a->H_q, a->n_tok, (uint64_t)a->q_stride * 2, 64, p.n_rep, p.cta_tok) &&
        (codes ? encode_u8_2d(&p.tm_k, c.k, D, p.n_rows, 128, p.k_rows) &&
                     encode_u8_2d(&p.tm_v, c.v, D, p.n_rows, 128, p.v_rows)
               : encode_bf16_2d(&p.tm_k, c.k, D, p.n_rows, D * 2, 64, p.k_rows) &&
                     encode_bf16_2d(&p.tm_v, c.v, D, p.n_rows, D * 2, 64, p.v_rows));
    if (!maps) return cudaErrorInvalidValue;
    const bool bf16 = a->out_dtype == GDR_BF16;
    if (codes)
        return bf16 ? launch_attn<true, false, true>(p, dev, n_cta, s) : launch_attn<true, false, false>(p, dev, n_cta, s);
    if (pair)
        return bf16 ? launch_attn<false, true, true>(p, dev, n_cta, s) : launch_attn<false, true, false>(p, dev, n_cta, s);
    return bf16 ? launch_attn<false, false, true>(p, dev, n_cta, s) : launch_attn<false, false, false>(p, dev, n_cta, s);
}

}  // namespace gdr
