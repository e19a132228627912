// gdr_kv.cu -- the paged key/value cache of the gated full-attention layer:
// writing new tokens (rotary embedding, optional 8-bit codes) and reading
// cached ones back.
//
//   append: k' = RoPE(k, t), q' = RoPE(q, t) at position t = cache_len[s] + i
//           (pairs (j, j + rot_dim/2), angle t theta^(-2j/rot_dim)); k' and v
//           go to token t's row, as bf16, or as scale = max(max|x|/448, 2^-40)
//           and codes e4m3(x / scale)
//   gather: rows scale * codes (or the bf16 rows) into packed rows
//
// Both move every byte once, 16 bytes a lane (8 of codes), a row of 256 values a warp.
//
// gather is bound by memory once enough is in flight: a block looks its tokens' pages up
// once, and a warp reads four rows before it writes the first.  64 sequences of 4096
// tokens from codes (0.81 GB): 148 us, 5.5 TB/s; with one row a warp and a look-up a row, 224 us.
//
// append: the angles are taken in double, once per token for all its
// heads.  A row's rotated dims are a quarter of it in the layers this is for, so queries go by
// pairs of 16-byte chunks instead of rows: whole warps rotate, and the rest is copied.  Four
// prompts of 4096 tokens, 16 query and 2 key/value heads, to codes (0.32 GB): 69 us,
// 4.6 TB/s; by rows, 98 us.  To bf16 (0.34 GB, no divisions) it is 71 us.  Neither memory (70% of a
// copy's rate) nor the issue slots (55%) are full: blocks are short, and each searches its
// sequences and takes its pages and angles before most of its loads.
#include <cuda_fp8.h>
#include <math.h>

#include "gdr.h"
#include "gdr_common.cuh"
#include "gdr_paged.cuh"

namespace gdr {
namespace paged {

// Tokens per block: a prompt's blocks take several so that a block's set-up
// (sequence search, pages, angles) is shared; a few tokens spread over the SMs.  Append: 75 us
// with 8, 76 with 16, 80 with 32; gather: 155 us with 16, 148 with 32.
constexpr int APPEND_TOKENS = 8;
constexpr int GATHER_TOKENS = 32;
constexpr int WARPS = 8;
constexpr float kE4m3Max = 448.f;

struct AppendParams {
    gdr_kv_append_args a;
    int shift;      // log2(page_size)
    int tokens;     // per block
    int rows;       // rows a token that warps take whole: (H_q +) 2 H_kv
    int whole_q;    // the q heads are among them (a rot_dim that is not a multiple of 16)
    double log2_theta;
};

// 8 bf16 values of a lane as fp32.
__device__ __forceinline__ void unpack8(const uint4 &u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Where the block's packed rows t0 .. t0 + n - 1 belong (n <= 32): their token's position and
// its row of kv head 0 in the cache, -1 without a valid page, or kNone when no sequence
// owns them.  `before` (may be null) holds each sequence's position of its first row.  Two
// searches find the sequences of the first and the last row; between them each thread
// looks by itself, in most blocks at nothing.
constexpr int kNone = -2;
struct Where {
    int first, last;  // sequences
    int row[32];
    int64_t pos[32];
};
__device__ __forceinline__ void locate(const gdr_kv_pages &c, const int32_t *before, int shift, int64_t t0,
                                       int n, Where &w) {
    const int tid = threadIdx.x, lane = tid & 31;
    if (tid < 64) {
        const int s = find_sequence(c.cu_seqlens, c.n_seq, (int)(tid < 32 ? t0 : t0 + n - 1));
        if (lane == 0) (tid < 32 ? w.first : w.last) = s;
    }
    __syncthreads();
    if (tid < n) {
        const int t = (int)t0 + tid;
        int lo = w.first, hi = w.last;  // the first s in [lo, hi] whose end is past t
        while (lo < hi) {
            const int mid = lo + (hi - lo) / 2;
            if (__ldg(c.cu_seqlens + mid + 1) <= t) lo = mid + 1;
            else hi = mid;
        }
        int row = kNone;
        int64_t pos = 0;
        if (lo < c.n_seq) {
            const int i = t - __ldg(c.cu_seqlens + lo);
            const int from = before ? __ldg(before + lo) : 0;
            if (i >= 0) {
                pos = from < 0 ? -1 : (int64_t)from + i;
                row = cache_row(c, shift, lo, 0, pos);
            }
        }
        w.row[tid] = row;
        w.pos[tid] = pos;
    }
    __syncthreads();
}

// Five blocks an SM (51 registers): 75 us as compiled freely (58 to 64), 69 so, 74 with six.
template <bool E4M3>
__global__ void __launch_bounds__(32 * WARPS, 5) kv_append_kernel(const AppendParams p) {
    __shared__ float2 turn[APPEND_TOKENS][D / 2];
    __shared__ Where where;
    wait_for_predecessor();
    release_dependents();
    const gdr_kv_append_args &a = p.a;
    const gdr_kv_pages &c = a.pages;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t0 = (int64_t)blockIdx.x * p.tokens;
    const int n = (int)min((int64_t)p.tokens, a.n_tok - t0);
    // Rows of the block that a warp takes whole: token by token, its q heads (unless they go
    // by pairs of chunks, below), its k heads, its v heads.
    const int n_rows = n * p.rows, step = gridDim.y * WARPS, q_rows = p.whole_q ? a.H_q : 0;
    auto fetch = [&](int r) {
        const int tt = r / p.rows, h = r - tt * p.rows;
        const int64_t t = t0 + tt;
        const __nv_bfloat16 *src =
            h < q_rows             ? static_cast<const __nv_bfloat16 *>(a.q) + t * a.q_stride + h * D
            : h < q_rows + c.H_kv ? static_cast<const __nv_bfloat16 *>(a.k) + t * a.k_stride + (h - q_rows) * D
                                  : static_cast<const __nv_bfloat16 *>(a.v) + t * a.v_stride +
                                        (h - q_rows - c.H_kv) * D;
        // Not through the read-only path: q_out may be q.
        return *reinterpret_cast<const uint4 *>(src + 8 * lane);
    };
    int r = blockIdx.y * WARPS + warp;
    uint4 next = make_uint4(0, 0, 0, 0);
    if (r < n_rows) next = fetch(r);
    locate(c, a.cache_len, p.shift, t0, n, where);
    const int half = a.rot_dim >> 1;
    for (int i = threadIdx.x; i < n * half; i += 32 * WARPS) {
        const int tt = i / half, j = i - tt * half;
        const double ang = (double)where.pos[tt] * exp2(-(2.0 * j / a.rot_dim) * p.log2_theta);
        double sn, cs;
        sincos(ang, &sn, &cs);
        turn[tt][j] = make_float2((float)cs, (float)sn);
    }
    __syncthreads();
    if (!p.whole_q && a.H_q > 0) {
        // Queries: a thread takes two chunks of 8 values of a row, a chunk to be turned and
        // its partner, or two of those that stay (which in place it leaves), so that the
        // arithmetic of the first kind is done by whole warps.
        const int pairs = half >> 3, others = D / 16 - pairs;
        const int n_head = n * a.H_q, at = blockIdx.y * (32 * WARPS) + threadIdx.x, by = gridDim.y * (32 * WARPS);
        auto q_row = [&](int u, int per, int64_t &from, int64_t &to, int &tt) {
            const int hh = u / per;
            tt = hh / a.H_q;
            const int h = hh - tt * a.H_q;
            from = (t0 + tt) * a.q_stride + h * D;
            to = (t0 + tt) * a.q_out_stride + h * D;
            return u - hh * per;
        };
        const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q);
        __nv_bfloat16 *q_out = static_cast<__nv_bfloat16 *>(a.q_out);
        for (int u = at; u < n_head * pairs; u += by) {
            int64_t from, to;
            int tt;
            const int j = 8 * q_row(u, pairs, from, to, tt);
            if (where.row[tt] == kNone) continue;
            float x[8], y[8], lo[8], hi[8];
            unpack8(*reinterpret_cast<const uint4 *>(q + from + j), x);
            unpack8(*reinterpret_cast<const uint4 *>(q + from + half + j), y);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 cs = turn[tt][j + i];
                lo[i] = x[i] * cs.x - y[i] * cs.y;
                hi[i] = y[i] * cs.x + x[i] * cs.y;
            }
            *reinterpret_cast<uint4 *>(q_out + to + j) = pack8(lo);
            *reinterpret_cast<uint4 *>(q_out + to + half + j) = pack8(hi);
        }
        if (q_out != q)
            for (int u = at; u < n_head * others; u += by) {
                int64_t from, to;
                int tt;
                const int j = a.rot_dim + 16 * q_row(u, others, from, to, tt);
                if (where.row[tt] == kNone) continue;
                const uint4 v0 = *reinterpret_cast<const uint4 *>(q + from + j);
                const uint4 v1 = *reinterpret_cast<const uint4 *>(q + from + j + 8);
                *reinterpret_cast<uint4 *>(q_out + to + j) = v0;
                *reinterpret_cast<uint4 *>(q_out + to + j + 8) = v1;
            }
    }
    for (; r < n_rows; r += step) {
        const uint4 raw = next;
        if (r + step < n_rows) next = fetch(r + step);  // a row ahead
        const int tt = r / p.rows, h = r - tt * p.rows;
        const int row0 = where.row[tt];
        if (row0 == kNone) continue;
        const int64_t t = t0 + tt;
        const bool is_q = h < q_rows, is_v = h >= q_rows + c.H_kv;
        const int g = is_q ? h : is_v ? h - q_rows - c.H_kv : h - q_rows;
        float x[8];
        unpack8(raw, x);
        if (!is_v && half > 0) {
            if ((half & 7) == 0) {
                // Partners sit in another lane, at the same place.
                const int step = half >> 3;
                const bool low = lane < step, in = lane < 2 * step;
                const int from = in ? (low ? lane + step : lane - step) : lane;
                uint4 o;
                o.x = __shfl_sync(kFullMask, raw.x, from);
                o.y = __shfl_sync(kFullMask, raw.y, from);
                o.z = __shfl_sync(kFullMask, raw.z, from);
                o.w = __shfl_sync(kFullMask, raw.w, from);
                if (in) {
                    float y[8];
                    unpack8(o, y);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 cs = turn[tt][8 * (low ? lane : lane - step) + i];
                        x[i] = low ? x[i] * cs.x - y[i] * cs.y : x[i] * cs.x + y[i] * cs.y;
                    }
                }
            } else {
                const __nv_bfloat16 *src = (is_q ? static_cast<const __nv_bfloat16 *>(a.q) + t * a.q_stride
                                                 : static_cast<const __nv_bfloat16 *>(a.k) + t * a.k_stride) +
                                           g * D;
                float y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int d = 8 * lane + i;
                    y[i] = d < a.rot_dim ? __bfloat162float(src[d < half ? d + half : d - half]) : 0.f;
                }
                __syncwarp();  // every lane has read the row before one writes it in place
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int d = 8 * lane + i;
                    if (d < a.rot_dim) {
                        const float2 cs = turn[tt][d < half ? d : d - half];
                        x[i] = d < half ? x[i] * cs.x - y[i] * cs.y : x[i] * cs.x + y[i] * cs.y;
                    }
                }
            }
        }
        if (is_q) {
            __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.q_out) + t * a.q_out_stride + g * D;
            *reinterpret_cast<uint4 *>(dst + 8 * lane) = pack8(x);
            continue;
        }
        if (row0 < 0) {
            if (lane == 0 && a.status) *a.status = kBadPage;
            continue;
        }
        const int row = row0 + g * c.page_size;
        void *pages = is_v ? c.v : c.k;
        if constexpr (!E4M3) {
            __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(pages) + (size_t)row * D;
            *reinterpret_cast<uint4 *>(dst + 8 * lane) = is_v ? raw : pack8(x);
        } else {
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[i]));
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, o));
            const float scale = fmaxf(__fdiv_rn(top, kE4m3Max), kScaleMin);
            // x / scale itself, not x times a rounded reciprocal: values half way between
            // two codes are common (x is bf16), and the quotient decides them.
            uint32_t w[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float2 lo = make_float2(__fdiv_rn(x[4 * i], scale), __fdiv_rn(x[4 * i + 1], scale));
                const float2 hi = make_float2(__fdiv_rn(x[4 * i + 2], scale), __fdiv_rn(x[4 * i + 3], scale));
                w[i] = (uint32_t)__nv_cvt_float2_to_fp8x2(lo, __NV_SATFINITE, __NV_E4M3) |
                       ((uint32_t)__nv_cvt_float2_to_fp8x2(hi, __NV_SATFINITE, __NV_E4M3) << 16);
            }
            unsigned char *dst = static_cast<unsigned char *>(pages) + (size_t)row * D;
            *reinterpret_cast<uint2 *>(dst + 8 * lane) = make_uint2(w[0], w[1]);
            if (lane == 0) (is_v ? c.v_scale : c.k_scale)[row] = scale;
        }
    }
}

struct GatherParams {
    gdr_kv_gather_args a;
    int shift;
    int tokens;
    int sides;  // rows per token and kv head: K and V, or one of them
};

template <bool E4M3, typename TOUT>
__global__ void __launch_bounds__(32 * WARPS) kv_gather_kernel(const GatherParams p) {
    __shared__ Where where;
    wait_for_predecessor();
    release_dependents();
    const gdr_kv_gather_args &a = p.a;
    const gdr_kv_pages &c = a.pages;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t0 = (int64_t)blockIdx.x * p.tokens;
    const int n = (int)min((int64_t)p.tokens, a.n_tok - t0);
    locate(c, a.first, p.shift, t0, n, where);
    // Rows of the block, AHEAD of them in flight a warp.
    constexpr int AHEAD = 4;
    const int per_tok = c.H_kv * p.sides, n_rows = n * per_tok, step = gridDim.y * WARPS;
    // Row r is token tt's row h: kept by additions, a division a row costs a tenth of the time.
    int r = blockIdx.y * WARPS + warp, tt = r / per_tok, h = r - tt * per_tok;
    const int step_t = step / per_tok, step_h = step - step_t * per_tok;
    while (r < n_rows) {
        uint4 raw[AHEAD];  // codes: 8 bytes and the scale
        int64_t at[AHEAD];
        TOUT *to[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            to[k] = nullptr;
            if (r >= n_rows) continue;
            const int t_now = tt, h_now = h, g = h >= c.H_kv ? h - c.H_kv : h;
            r += step;
            tt += step_t;
            h += step_h;
            if (h >= per_tok) {
                h -= per_tok;
                ++tt;
            }
            const int row0 = where.row[t_now];
            if (row0 < 0) {
                if (row0 != kNone && lane == 0 && a.status) *a.status = kBadPage;
                continue;
            }
            const bool is_v = !a.k_out || h_now >= c.H_kv;
            const size_t row = (size_t)row0 + (size_t)g * c.page_size;
            const void *pages = is_v ? c.v : c.k;
            if constexpr (E4M3) {
                const uint2 w = __ldg(reinterpret_cast<const uint2 *>(
                    static_cast<const unsigned char *>(pages) + row * D + 8 * lane));
                raw[k] = make_uint4(w.x, w.y, __float_as_uint(__ldg((is_v ? c.v_scale : c.k_scale) + row)), 0);
            } else {
                raw[k] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(pages) + row * D +
                                                               8 * lane));
            }
            to[k] = static_cast<TOUT *>(is_v ? a.v_out : a.k_out);
            at[k] = (t0 + t_now) * (is_v ? a.v_out_stride : a.k_out_stride) + g * D + 8 * lane;
        }
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            if (!to[k]) continue;
            TOUT *dst = to[k] + at[k];
            float x[8];
            if constexpr (E4M3) {
                const float scale = __uint_as_float(raw[k].z);
                const uint32_t ww[2] = {raw[k].x, raw[k].y};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const __half2_raw h2 = __nv_cvt_fp8x2_to_halfraw2(
                        (__nv_fp8x2_storage_t)(ww[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
                    const float2 f = __half22float2(__half2(h2));
                    x[2 * i] = f.x * scale;
                    x[2 * i + 1] = f.y * scale;
                }
            } else if constexpr (sizeof(TOUT) == 4) {
                unpack8(raw[k], x);
            }
            if constexpr (sizeof(TOUT) == 2) {
                *reinterpret_cast<uint4 *>(dst) = E4M3 ? pack8(x) : raw[k];
            } else {
                reinterpret_cast<float4 *>(dst)[0] = make_float4(x[0], x[1], x[2], x[3]);
                reinterpret_cast<float4 *>(dst)[1] = make_float4(x[4], x[5], x[6], x[7]);
            }
        }
    }
}

// Launch as a programmatic dependent: the kernel waits for its predecessor
// before it reads anything, so only the launch overlaps.
template <typename P>
static cudaError_t launch(void (*kern)(P), const P &p, dim3 grid, cudaStream_t s) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(32 * WARPS);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p);
    if (e != cudaSuccess) (void)cudaGetLastError();
    return e;
}

// Up to this many tokens a block takes one token and its rows are spread over
// several blocks, a warp each; above, a block takes as many as it can.
constexpr int64_t kFewTokens = 592;  // 4 blocks for each of 148 SMs

static dim3 grid_for(int64_t n_tok, int rows, int most, int *tokens) {
    *tokens = n_tok <= kFewTokens ? 1 : most;
    const unsigned y = *tokens == 1 ? (unsigned)((rows + WARPS - 1) / WARPS) : 1u;
    return dim3((unsigned)((n_tok + *tokens - 1) / *tokens), y < 65535u ? y : 65535u);
}

}  // namespace paged

cudaError_t launch_kv_append(const gdr_kv_append_args *a, cudaStream_t s) {
    paged::AppendParams p = {};
    p.a = *a;
    p.shift = paged::log2_of(a->pages.page_size);
    p.whole_q = ((a->rot_dim >> 1) & 7) != 0;
    p.rows = (p.whole_q ? a->H_q : 0) + 2 * a->pages.H_kv;
    p.log2_theta = log2((double)a->rope_theta);
    const dim3 grid = paged::grid_for(a->n_tok, a->H_q + 2 * a->pages.H_kv, paged::APPEND_TOKENS, &p.tokens);
    return a->pages.kv_dtype == GDR_E4M3 ? paged::launch(paged::kv_append_kernel<true>, p, grid, s)
                                         : paged::launch(paged::kv_append_kernel<false>, p, grid, s);
}

cudaError_t launch_kv_gather(const gdr_kv_gather_args *a, cudaStream_t s) {
    paged::GatherParams p = {};
    p.a = *a;
    p.shift = paged::log2_of(a->pages.page_size);
    p.sides = (a->k_out ? 1 : 0) + (a->v_out ? 1 : 0);
    const dim3 grid = paged::grid_for(a->n_tok, p.sides * a->pages.H_kv, paged::GATHER_TOKENS, &p.tokens);
    const bool codes = a->pages.kv_dtype == GDR_E4M3;
    if (a->out_dtype == GDR_BF16)
        return codes ? paged::launch(paged::kv_gather_kernel<true, __nv_bfloat16>, p, grid, s)
                     : paged::launch(paged::kv_gather_kernel<false, __nv_bfloat16>, p, grid, s);
    return codes ? paged::launch(paged::kv_gather_kernel<true, float>, p, grid, s)
                 : paged::launch(paged::kv_gather_kernel<false, float>, p, grid, s);
}

}  // namespace gdr
