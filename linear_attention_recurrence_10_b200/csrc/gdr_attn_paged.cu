// gdr_attn_paged.cu -- attention of the new tokens of packed sequences over
// their pages: row i of sequence s, at position t = cache_len[s] + i, attends
// tokens 0 .. t.
//
//   a_j = scale q . k_j,  y = (sum_{j <= t} e^{a_j} v_j) / (sum e^{a_j}) * sigmoid(gate)
//
// One warp per (token, query head), 8 of the 256 dims a lane; the keys one
// after another with the running maximum and sum of the softmax.
#include <cuda_fp8.h>
#include <math.h>

#include "gdr.h"
#include "gdr_common.cuh"
#include "gdr_paged.cuh"

namespace gdr {
namespace paged {

struct AttnParams {
    gdr_attn_paged_args a;
    int shift;
    int *status;
};

template <bool E4M3>
__device__ __forceinline__ void cached8(const void *pages, const float *scales, int row, int lane,
                                        float (&x)[8]) {
    if constexpr (E4M3) {
        const uint2 w = __ldg(reinterpret_cast<const uint2 *>(
            static_cast<const unsigned char *>(pages) + (size_t)row * D + 8 * lane));
        const float scale = __ldg(scales + row);
        const uint32_t ww[2] = {w.x, w.y};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2_raw h2 = __nv_cvt_fp8x2_to_halfraw2(
                (__nv_fp8x2_storage_t)(ww[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
            const float2 f = __half22float2(__half2(h2));
            x[2 * i] = f.x * scale;
            x[2 * i + 1] = f.y * scale;
        }
    } else {
        const uint4 u = __ldg(reinterpret_cast<const uint4 *>(
            static_cast<const __nv_bfloat16 *>(pages) + (size_t)row * D + 8 * lane));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}

template <bool E4M3, typename TOUT>
__global__ void __launch_bounds__(256) attn_paged_kernel(const AttnParams p) {
    wait_for_predecessor();
    const gdr_attn_paged_args &a = p.a;
    const gdr_kv_pages &c = a.pages;
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (w >= a.n_tok * a.H_q) return;
    const int64_t t = w / a.H_q;
    const int h = (int)(w - t * a.H_q), g = h / (a.H_q / c.H_kv);
    const int s = find_sequence(c.cu_seqlens, c.n_seq, (int)t);
    if (s >= c.n_seq) return;
    const int i = (int)t - __ldg(c.cu_seqlens + s);
    if (i < 0) return;
    const int64_t last = (int64_t)__ldg(a.cache_len + s) + i;
    float q[8], o[8] = {}, m = -INFINITY, l = 0.f;
    cached8<false>(static_cast<const __nv_bfloat16 *>(a.q) + t * a.q_stride + h * D, nullptr, 0,
                   lane, q);
    for (int64_t j = 0; j <= last; ++j) {
        const int row = cache_row(c, p.shift, s, g, j);
        if (row < 0) {
            if (lane == 0) *p.status = kBadPage;
            break;
        }
        float k[8], v[8];
        cached8<E4M3>(c.k, c.k_scale, row, lane, k);
        cached8<E4M3>(c.v, c.v_scale, row, lane, v);
        float x = 0.f;
#pragma unroll
        for (int d = 0; d < 8; ++d) x = fmaf(q[d], k[d], x);
        x = group_sum<32>(x) * a.scale;
        const float top = fmaxf(m, x), f = expf(m - top), e = expf(x - top);
        m = top;
        l = fmaf(l, f, e);
#pragma unroll
        for (int d = 0; d < 8; ++d) o[d] = fmaf(o[d], f, e * v[d]);
    }
    if (last < 0 && lane == 0) *p.status = kBadPage;
    const float r = l > 0.f ? 1.f / l : 0.f;
    const int64_t at = t * a.out_stride + h * D + 8 * lane;
#pragma unroll
    for (int d = 0; d < 8; ++d) {
        float y = o[d] * r;
        if (a.gate)
            y /= 1.f + expf(-__bfloat162float(static_cast<const __nv_bfloat16 *>(
                           a.gate)[t * a.gate_stride + h * D + 8 * lane + d]));
        Elem<TOUT>::store1(static_cast<TOUT *>(a.out) + at + d, y);
    }
    if (lane == 0 && a.lse) a.lse[t * a.lse_stride + h] = m + logf(l);
}

}  // namespace paged

size_t attn_paged_workspace_bytes(int n_sm) { return 256; }

cudaError_t launch_attn_paged(const gdr_attn_paged_args *a, void *workspace, cudaStream_t s) {
    paged::AttnParams p = {};
    p.a = *a;
    p.shift = paged::log2_of(a->pages.page_size);
    p.status = static_cast<int *>(workspace);
    cudaError_t e = cudaMemsetAsync(workspace, 0, 4, s);
    if (e != cudaSuccess) return e;
    const unsigned grid = (unsigned)((a->n_tok * a->H_q + 7) / 8);
    const bool codes = a->pages.kv_dtype == GDR_E4M3, b = a->out_dtype == GDR_BF16;
    if (codes && b) paged::attn_paged_kernel<true, __nv_bfloat16><<<grid, 256, 0, s>>>(p);
    if (codes && !b) paged::attn_paged_kernel<true, float><<<grid, 256, 0, s>>>(p);
    if (!codes && b) paged::attn_paged_kernel<false, __nv_bfloat16><<<grid, 256, 0, s>>>(p);
    if (!codes && !b) paged::attn_paged_kernel<false, float><<<grid, 256, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace gdr
