// scaled_product.cu -- the matrix product of 8-bit floating point numbers with
// a scale for each block of 128:
//   out[t][n] = sum_b (sx[t][b] sw[n / 128][b]) sum_{k in b} x[t][k] w[n][k].
#include <algorithm>

#include "e4m3.cuh"
#include "internal.h"
#include "rows.h"

namespace moe {

namespace {

constexpr int kStatusBytes = 256;

struct ProductParams {
    const uint8_t *x, *w;
    size_t x_stride, w_stride, sx_stride, sw_stride, out_stride;
    const float *sx, *sw;
    int T, N, K;
    void *out;
};

__device__ __forceinline__ float e4m3_value(uint8_t c) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

// 64 x 64 outputs a CTA, 4 x 4 a thread.
template <typename O>
__global__ void __launch_bounds__(256) product_kernel(const ProductParams p) {
    __shared__ float xs[32][65], ws[32][65];
    const int t0 = blockIdx.y * 64, n0 = blockIdx.x * 64, tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float sum[4][4] = {};
    for (int b = 0; b * kScaleBlock < p.K; b++) {
        float part[4][4] = {};
        for (int k0 = b * kScaleBlock; k0 < min(p.K, (b + 1) * kScaleBlock); k0 += 32) {
            for (int i = threadIdx.x; i < 2048; i += 256) {
                const int r = i >> 5, k = i & 31;
                const bool in = k0 + k < p.K;
                xs[k][r] = in && t0 + r < p.T ? e4m3_value(p.x[(size_t)(t0 + r) * p.x_stride + k0 + k]) : 0.0f;
                ws[k][r] = in && n0 + r < p.N ? e4m3_value(p.w[(size_t)(n0 + r) * p.w_stride + k0 + k]) : 0.0f;
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < 32; k++)
#pragma unroll
                for (int i = 0; i < 4; i++)
#pragma unroll
                    for (int j = 0; j < 4; j++) part[i][j] = fmaf(xs[k][ty * 4 + i], ws[k][tx * 4 + j], part[i][j]);
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const int t = t0 + ty * 4 + i, n = n0 + tx * 4 + j;
                if (t < p.T && n < p.N) {
                    const float s = p.sx[(size_t)t * p.sx_stride + b] * p.sw[(size_t)(n / kScaleBlock) * p.sw_stride + b];
                    sum[i][j] = fmaf(s, part[i][j], sum[i][j]);
                }
            }
    }
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const int t = t0 + ty * 4 + i, n = n0 + tx * 4 + j;
            if (t < p.T && n < p.N) static_cast<O *>(p.out)[(size_t)t * p.out_stride + n] = (O)sum[i][j];
        }
}

int check_matrix(const moe_scaled_matrix_desc *wd, const char *who) {
    if (wd == nullptr) return fail(MOE_EINVAL, "%s: descriptor is NULL", who);
    if (wd->N < 1 || wd->K < 1) return fail(MOE_EINVAL, "%s: N=%d K=%d", who, wd->N, wd->K);
    return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_scaled_product_workspace_bytes(const moe_scaled_matrix_desc *wd, int T) {
    if (check_matrix(wd, "scaled_product_workspace_bytes") || T < 0) return 0;
    return kStatusBytes;
}

extern "C" int moe_scaled_product(const moe_scaled_matrix_desc *wd, const void *x, size_t x_stride, const float *x_scales,
                                  size_t x_scale_stride, int T, void *out, int out_dtype, size_t out_stride, void *ws, size_t ws_bytes,
                                  cudaStream_t stream) {
    const char *who = "scaled_product";
    if (int rc = check_matrix(wd, who)) return rc;
    if (T < 0) return fail(MOE_EINVAL, "%s: T=%d", who, T);
    if (out_dtype != MOE_DTYPE_F32 && out_dtype != MOE_DTYPE_BF16) return fail(MOE_EINVAL, "%s: out_dtype=%d", who, out_dtype);
    if (T == 0) return MOE_OK;
    const size_t n = (size_t)T, N = (size_t)wd->N, K = (size_t)wd->K, blocks = (K + kScaleBlock - 1) / kScaleBlock;
    const size_t tall = (N + kScaleBlock - 1) / kScaleBlock, e = bytes_of(out_dtype);
    const Rows in[] = {{"x", x, n, K, x_stride}, {"w", wd->w, N, K, wd->w_stride}, {"x_scales", x_scales, n, blocks * 4, x_scale_stride * 4},
                       {"scales", wd->scales, tall, blocks * 4, wd->scale_stride * 4}};
    const Rows o{"out", out, n, N * e, out_stride * e}, status{"ws", ws, 1, kStatusBytes, 0};
    for (int i = 0; i < 4; i++)
        if (int rc = check_rows(who, in[i], i < 2 ? 16 : 4)) return rc;
    if (int rc = check_rows(who, o)) return rc;
    if (!ws || off(ws, 256) || ws_bytes < kStatusBytes)
        return fail(MOE_ENOSPACE, "%s: workspace of %zu bytes (need %d, 256-byte aligned)", who, ws_bytes, kStatusBytes);
    for (const Rows &i : in)
        if (o.overlaps(i) || status.overlaps(i)) return fail(MOE_EINVAL, "%s: out or ws overlaps %s", who, i.name);
    if (o.overlaps(status)) return fail(MOE_EINVAL, "%s: out overlaps ws", who);
    const ProductParams p{static_cast<const uint8_t *>(x), static_cast<const uint8_t *>(wd->w), x_stride, wd->w_stride, x_scale_stride,
                          wd->scale_stride, out_stride, x_scales, wd->scales, T, wd->N, wd->K, out};
    const dim3 grid((wd->N + 63) / 64, (T + 63) / 64);
    if (out_dtype == MOE_DTYPE_F32) product_kernel<float><<<grid, 256, 0, stream>>>(p);
    else product_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(p);
    return check_launch("product_kernel");
}
