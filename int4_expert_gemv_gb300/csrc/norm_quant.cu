// norm_quant.cu -- the root-mean-square norm with the residual's addition, and
// the quantisation to 8-bit floating point with a scale for each block of 128.
//
// Norm.  h = x + res;  y = h / sqrt(mean(h^2) + eps) * w, everything in fp32
// from numbers read once: a row stays in the registers of the threads that
// have loaded it (8 to 32 numbers each), so that the sum of squares,
// the block's largest size and the result need no second read.  In 8 bits a
// block of 128 numbers belongs to 16 neighbouring lanes, which find its
// largest size by shuffles.  8191 rows of 4096 with a 16-bit residual, sum
// written: to bf16 43.5 us, 91 % of the copy rate; to e4m3 42.4, 82 % (40.2 with
// scales that are powers of two), with 76 % of the issue slots taken (the conversion).  4096 rows of 8192, all fp32 but a bf16 result:
// 73 us, 95 %.  16384 rows of 512: 14.8 us, 59 %: a warp has a row, and its chain of
// load, sum, scale and store too little beside it.  Up to some hundred rows a call
// takes the 2 to 2.5 us of one launch and one such chain.
//
// Quantisation.  16381 rows of 4096 from bf16 39.0 us, 77 % of the copy rate (68 %
// of the issue slots), with scales that are powers of two 35.0, 86 %; from fp32
// 53.3, 93 %.  Weights by 128 x 128, 8192 x 4096: from bf16 24.7 us, 60 %, from
// fp32 28.2, 88 %; 2500 x 2000 fp32 7.4 us (9.4 with 64 numbers a thread).
#include <algorithm>

#include "e4m3.cuh"
#include "fastdiv.cuh"
#include "internal.h"
#include "rows.h"

namespace moe {

namespace {

constexpr int kMaxCols = 1 << 30;         // of a quantised row
constexpr int kNoChunk = kMaxCols / 8;    // behind every row
constexpr int kMaxNormWidth = 32768;      // 1024 threads of 32 numbers

struct NormParams {
    const void *x, *res, *w;
    size_t x_stride, res_stride, sum_stride, y_stride, scale_stride;    // elements
    int T, d, w_bf16;
    float eps;
    void *sum, *y;
    float *scales;
    bool pow2;
};

// The largest of the lanes that hold a block.
template <int LANES>
__device__ __forceinline__ uint32_t most_of(uint32_t m) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}

// X, R: types of x and res (R = void: no residual); Y: type of y (uint8_t:
// e4m3 codes).  A row belongs to a warp (ROWS warps, each with a row of its
// own) or, for ROWS = 1, to the CTA; each thread has NV chunks of 8 numbers.
// Persistent: the next row is on its way while this one is computed.
template <typename X, typename R, typename Y, int NV, int ROWS, int THREADS>
__global__ void __launch_bounds__(THREADS) norm_kernel(const NormParams p) {
    constexpr bool RES = !std::is_void<R>::value, AHEAD = NV < 4;      // (32 numbers and the next 32 do not fit 1024 threads' registers)
    using RT = std::conditional_t<RES, R, float>;
    __shared__ float part[2][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int first = ROWS > 1 ? lane : threadIdx.x, step = ROWS > 1 ? 32 : blockDim.x;
    Raw8<X> a[NV];
    Raw8<RT> b[NV];
    auto load = [&](int64_t t) {
#pragma unroll
        for (int i = 0; i < NV; i++) {
            a[i] = row_load8<X>(static_cast<const X *>(p.x) + (size_t)t * p.x_stride, first + i * step, p.d);
            if (RES) b[i] = row_load8<RT>(static_cast<const RT *>(p.res) + (size_t)t * p.res_stride, first + i * step, p.d);
        }
    };
    const int64_t rows = (int64_t)gridDim.x * ROWS;
    int64_t t = (int64_t)blockIdx.x * ROWS + (ROWS > 1 ? warp : 0);
    if (AHEAD && t < p.T) load(t);
    for (int odd = 0; t < p.T; t += rows, odd ^= 1) {
        float h[NV][8];
        float ss = 0.0f;
        if (!AHEAD) load(t);
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const Floats8 u = a[i].floats(), v = RES ? b[i].floats() : u;
#pragma unroll
            for (int j = 0; j < 8; j++) h[i][j] = RES ? u.x[j] + v.x[j] : u.x[j];
        }
        if (AHEAD && t + rows < p.T) load(t + rows);
#pragma unroll
        for (int i = 0; i < NV; i++) {
            if (RES && p.sum && 8 * (first + i * step) < p.d)
                row_store8(static_cast<RT *>(p.sum) + (size_t)t * p.sum_stride, first + i * step, p.d, h[i]);
#pragma unroll
            for (int j = 0; j < 8; j++) ss = fmaf(h[i][j], h[i][j], ss);
        }
        ss = warp_sum(ss, 32);
        if (ROWS == 1 && warps > 1) {
            if (lane == 0) part[odd][warp] = ss;          // (two sets: a row's are read before the next but one's are written)
            __syncthreads();
            ss = warp_sum(lane < warps ? part[odd][lane] : 0.0f, 32);
        }
        const float by = __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(ss, (float)p.d) + p.eps));
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int c = first + i * step;
            const bool in = 8 * c < p.d;
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; j++) y[j] = h[i][j] * by;
            if (p.w && in) {
                const Floats8 w = p.w_bf16 ? row_load8<__nv_bfloat16>(static_cast<const __nv_bfloat16 *>(p.w), c, p.d).floats()
                                           : row_load8<float>(static_cast<const float *>(p.w), c, p.d).floats();
#pragma unroll
                for (int j = 0; j < 8; j++) y[j] *= w.x[j];
            }
            if constexpr (sizeof(Y) == 1) {
                const float scale = block_scale(most_of<16>(in ? most8(y) : 0u), p.pow2);
                if (in) {
                    row_store8(static_cast<uint8_t *>(p.y) + (size_t)t * p.y_stride, c, p.d, block_codes(y, scale, p.pow2));
                    if (c % 16 == 0) p.scales[(size_t)t * p.scale_stride + c / 16] = scale;
                }
            } else if (in) {
                row_store8(static_cast<Y *>(p.y) + (size_t)t * p.y_stride, c, p.d, y);
            }
        }
    }
}

// The CTAs that the SMs hold, or fewer where there are fewer rows.  (The
// occupancy takes the host a microsecond: not asked for where it does not count.)
template <typename F>
int norm_grid(F kernel, int threads, int64_t rows) {
    int ctas = 1;
    if (rows <= num_sms()) return (int)rows;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&ctas, kernel, threads, 0) != cudaSuccess) cudaGetLastError();
    ctas = std::max(ctas, 1);
    return (int)std::min<int64_t>(rows, (int64_t)ctas * num_sms());
}

template <typename X, typename R, typename Y>
int launch_norm(const NormParams &p, cudaStream_t st) {
    const int chunks = (p.d + 7) / 8;
    auto threads = [&](int nv) { return ((chunks + nv - 1) / nv + 31) / 32 * 32; };
    auto go = [&](auto kernel, int n, int64_t rows) { kernel<<<norm_grid(kernel, n, rows), n, 0, st>>>(p); };
    if (chunks <= 32) go(norm_kernel<X, R, Y, 1, 4, 128>, 128, (p.T + (int64_t)3) / 4);
    else if (chunks <= 64) go(norm_kernel<X, R, Y, 2, 4, 128>, 128, (p.T + (int64_t)3) / 4);
    else if (threads(1) <= 256 && p.T <= 8 * num_sms()) go(norm_kernel<X, R, Y, 1, 1, 256>, threads(1), p.T);
    else if (threads(2) <= 512) go(norm_kernel<X, R, Y, 2, 1, 512>, threads(2), p.T);
    else if (threads(2) <= 1024) go(norm_kernel<X, R, Y, 2, 1, 1024>, threads(2), p.T);
    else go(norm_kernel<X, R, Y, 4, 1, 1024>, threads(4), p.T);
    return check_launch("norm_kernel");
}

template <typename X, typename R>
int launch_norm_y(const NormParams &p, int y_dtype, cudaStream_t st) {
    if (y_dtype == MOE_DTYPE_E4M3) return launch_norm<X, R, uint8_t>(p, st);
    if (y_dtype == MOE_DTYPE_BF16) return launch_norm<X, R, __nv_bfloat16>(p, st);
    return launch_norm<X, R, float>(p, st);
}

template <typename X>
int launch_norm_res(const NormParams &p, int res_dtype, int y_dtype, cudaStream_t st) {
    if (!p.res) return launch_norm_y<X, void>(p, y_dtype, st);
    if (res_dtype == MOE_DTYPE_BF16) return launch_norm_y<X, __nv_bfloat16>(p, y_dtype, st);
    return launch_norm_y<X, float>(p, y_dtype, st);
}

// ---------------------------------------------------------------- quantise
struct QuantParams {
    const void *x;
    size_t x_stride, code_stride, scale_stride;      // elements
    int rows, cols;
    uint8_t *codes;
    float *scales;
    bool pow2;
    FastDiv quads;                                   // four blocks of a row: a warp's
};

// A warp's unit is four blocks of a row, 16 numbers a lane (a block's scale costs
// its lanes two divisions each, so that 8 numbers a lane took 50 us at 16381 x 4096);
// U units are on their way at a time.
template <typename X>
__global__ void __launch_bounds__(256) quant_rows_kernel(const QuantParams p) {
    constexpr int U = sizeof(X) == 2 ? 2 : 1;
    const int lane = threadIdx.x & 31, n = p.rows * p.quads.d, step = gridDim.x * 8;           // (the host keeps n + U step within 2^31)
    for (int u0 = blockIdx.x * 8 + (threadIdx.x >> 5); u0 < n; u0 += U * step) {
        Raw8<X> raw[U][2];
        int r[U], c[U];
#pragma unroll
        for (int j = 0; j < U; j++) {
            const int u = min(u0 + j * step, n - 1);
            r[j] = p.quads.div(u);
            c[j] = u0 + j * step < n ? (u - r[j] * p.quads.d) * 64 + 2 * lane : kNoChunk;
#pragma unroll
            for (int i = 0; i < 2; i++) raw[j][i] = row_load8<X>(static_cast<const X *>(p.x) + (size_t)r[j] * p.x_stride, c[j] + i, p.cols);
        }
#pragma unroll
        for (int j = 0; j < U; j++) {
            const Floats8 f = raw[j][0].floats(), g = raw[j][1].floats();
            const float scale = block_scale(most_of<8>(max(most8(f.x), most8(g.x))), p.pow2);
            if (8 * c[j] < p.cols) {
                uint8_t *row = p.codes + (size_t)r[j] * p.code_stride;
                const uint2 a = block_codes(f.x, scale, p.pow2), b = block_codes(g.x, scale, p.pow2);
                if (8 * c[j] + 16 <= p.cols) {
                    *reinterpret_cast<uint4 *>(row + 8 * (size_t)c[j]) = make_uint4(a.x, a.y, b.x, b.y);
                } else {
                    row_store8(row, c[j], p.cols, a);
                    if (8 * c[j] + 8 < p.cols) row_store8(row, c[j] + 1, p.cols, b);
                }
                if (c[j] % 16 == 0) p.scales[(size_t)r[j] * p.scale_stride + c[j] / 16] = scale;
            }
        }
    }
}

// A CTA takes 128 x 128 numbers, 32 a thread, which stay in its registers.
template <typename X>
__global__ void __launch_bounds__(512) quant_tiles_kernel(const QuantParams p) {
    __shared__ uint32_t part[16];
    const int r0 = blockIdx.y * 128 + (threadIdx.x >> 4), c = blockIdx.x * 16 + (threadIdx.x & 15);
    const bool in = 8 * c < p.cols;
    Raw8<X> raw[4];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; i++)              // (a row behind the last is as one without columns)
        raw[i] = row_load8<X>(static_cast<const X *>(p.x) + (size_t)min(r0 + 32 * i, p.rows - 1) * p.x_stride, c, r0 + 32 * i < p.rows ? p.cols : 0);
#pragma unroll
    for (int i = 0; i < 4; i++) m = max(m, most8(raw[i].floats().x));
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 16; i++) m = max(m, part[i]);
    const float scale = block_scale(m, p.pow2);
    if (threadIdx.x == 0) p.scales[(size_t)blockIdx.y * p.scale_stride + blockIdx.x] = scale;
#pragma unroll
    for (int i = 0; i < 4; i++)
        if (in && r0 + 32 * i < p.rows)
            row_store8(p.codes + (size_t)(r0 + 32 * i) * p.code_stride, c, p.cols, block_codes(raw[i].floats().x, scale, p.pow2));
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_add_rms_norm(const moe_norm_desc *nd, const void *x, int x_dtype, size_t x_stride, const void *res, int res_dtype,
                                size_t res_stride, int T, void *sum, size_t sum_stride, void *y, int y_dtype, size_t y_stride,
                                float *scales, size_t scale_stride, cudaStream_t stream) {
    const char *who = "add_rms_norm";
    if (nd == nullptr) return fail(MOE_EINVAL, "%s: descriptor is NULL", who);
    if (nd->d < 1 || !(nd->eps >= 0.0f) || !(nd->eps < INFINITY) || (nd->pow2 != 0 && nd->pow2 != 1))
        return fail(MOE_EINVAL, "%s: d=%d eps=%g pow2=%d", who, nd->d, (double)nd->eps, nd->pow2);
    if (nd->d > kMaxNormWidth) return fail(MOE_EUNSUPPORTED, "%s: d=%d (at most %d)", who, nd->d, kMaxNormWidth);
    if (nd->weight && nd->w_dtype != MOE_DTYPE_F32 && nd->w_dtype != MOE_DTYPE_BF16)
        return fail(MOE_EINVAL, "%s: w_dtype=%d", who, nd->w_dtype);
    if (x_dtype != MOE_DTYPE_F32 && x_dtype != MOE_DTYPE_BF16) return fail(MOE_EINVAL, "%s: x_dtype=%d", who, x_dtype);
    if (res && res_dtype != MOE_DTYPE_F32 && res_dtype != MOE_DTYPE_BF16) return fail(MOE_EINVAL, "%s: res_dtype=%d", who, res_dtype);
    if (y_dtype != MOE_DTYPE_F32 && y_dtype != MOE_DTYPE_BF16 && y_dtype != MOE_DTYPE_E4M3)
        return fail(MOE_EINVAL, "%s: y_dtype=%d", who, y_dtype);
    if (sum && !res) return fail(MOE_EINVAL, "%s: sum without a residual", who);
    if (T < 0) return fail(MOE_EINVAL, "%s: T=%d", who, T);
    if (T == 0) return MOE_OK;
    const size_t xe = bytes_of(x_dtype), re = bytes_of(res_dtype), ye = bytes_of(y_dtype), n = (size_t)T, d = (size_t)nd->d;
    const bool e4m3 = y_dtype == MOE_DTYPE_E4M3;
    const Rows in[] = {{"x", x, n, d * xe, x_stride * xe}, {"res", res, n, d * re, res_stride * re},
                       {"weight", nd->weight, 1, d * bytes_of(nd->w_dtype), 0}};
    const Rows out[] = {{"sum", sum, n, d * re, sum_stride * re}, {"y", y, n, d * ye, y_stride * ye},
                        {"scales", e4m3 ? scales : nullptr, n, (d + kScaleBlock - 1) / kScaleBlock * 4, scale_stride * 4}};
    if (int rc = check_rows(who, in[0])) return rc;
    if (res)
        if (int rc = check_rows(who, in[1])) return rc;
    if (nd->weight)
        if (int rc = check_rows(who, in[2])) return rc;
    if (sum)
        if (int rc = check_rows(who, out[0])) return rc;
    if (int rc = check_rows(who, out[1])) return rc;
    if (e4m3)
        if (int rc = check_rows(who, out[2], 4)) return rc;
    // A thread reads its numbers of x and res before it writes any.
    const int in_type[] = {x_dtype, res_dtype, -1}, out_type[] = {res_dtype, y_dtype, -2};
    for (int o = 0; o < 3; o++) {
        for (int i = 0; i < 3; i++)
            if (out[o].overlaps(in[i]) && !(out[o].same(in[i]) && out_type[o] == in_type[i]))
                return fail(MOE_EINVAL, "%s: %s overlaps %s", who, out[o].name, in[i].name);
        for (int i = 0; i < o; i++)
            if (out[o].overlaps(out[i])) return fail(MOE_EINVAL, "%s: %s overlaps %s", who, out[o].name, out[i].name);
    }
    const NormParams p{x, res, nd->weight, x_stride, res_stride, sum_stride, y_stride, scale_stride, T, nd->d,
                       nd->w_dtype == MOE_DTYPE_BF16, nd->eps, sum, y, scales, nd->pow2 != 0};
    return x_dtype == MOE_DTYPE_BF16 ? launch_norm_res<__nv_bfloat16>(p, res_dtype, y_dtype, stream)
                                     : launch_norm_res<float>(p, res_dtype, y_dtype, stream);
}

extern "C" int moe_quantise_e4m3(const void *x, int x_dtype, size_t x_stride, int rows, int cols, int block_rows, int pow2,
                                 void *codes, size_t code_stride, float *scales, size_t scale_stride, cudaStream_t stream) {
    const char *who = "quantise_e4m3";
    if (rows < 0 || cols < 0 || (block_rows != 1 && block_rows != kScaleBlock) || (pow2 != 0 && pow2 != 1))
        return fail(MOE_EINVAL, "%s: rows=%d cols=%d block_rows=%d (1 or %d) pow2=%d", who, rows, cols, block_rows, kScaleBlock, pow2);
    if (x_dtype != MOE_DTYPE_F32 && x_dtype != MOE_DTYPE_BF16) return fail(MOE_EINVAL, "%s: x_dtype=%d", who, x_dtype);
    if (rows == 0 || cols == 0) return MOE_OK;
    const int blocks = (cols - 1) / kScaleBlock + 1, quads = (blocks - 1) / 4 + 1, tall = (rows - 1) / kScaleBlock + 1;
    if (cols > kMaxCols || (int64_t)rows * quads >= (int64_t)2000000000 || (block_rows != 1 && tall > 65535))
        return fail(MOE_EUNSUPPORTED, "%s: rows=%d cols=%d", who, rows, cols);
    const size_t xe = bytes_of(x_dtype), n = (size_t)rows;
    const Rows in{"x", x, n, cols * xe, x_stride * xe}, out{"codes", codes, n, (size_t)cols, code_stride},
        sc{"scales", scales, block_rows == 1 ? n : (size_t)tall, (size_t)blocks * 4, scale_stride * 4};
    if (int rc = check_rows(who, in)) return rc;
    if (int rc = check_rows(who, out)) return rc;
    if (int rc = check_rows(who, sc, 4)) return rc;
    if (out.overlaps(in) || sc.overlaps(in) || sc.overlaps(out))
        return fail(MOE_EINVAL, "%s: x, codes and scales overlap", who);
    const QuantParams p{x, x_stride, code_stride, scale_stride, rows, cols, static_cast<uint8_t *>(codes), scales, pow2 != 0, FastDiv(quads)};
    if (block_rows == 1) {
        const unsigned grid = (unsigned)std::min<int64_t>(((int64_t)rows * quads + 7) / 8, (int64_t)num_sms() * 8);
        if (x_dtype == MOE_DTYPE_BF16) quant_rows_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(p);
        else quant_rows_kernel<float><<<grid, 256, 0, stream>>>(p);
    } else {
        const dim3 grid((unsigned)blocks, (unsigned)tall);
        if (x_dtype == MOE_DTYPE_BF16) quant_tiles_kernel<__nv_bfloat16><<<grid, 512, 0, stream>>>(p);
        else quant_tiles_kernel<float><<<grid, 512, 0, stream>>>(p);
    }
    return check_launch("quantise_e4m3");
}
