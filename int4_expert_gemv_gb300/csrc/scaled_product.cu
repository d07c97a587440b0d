// scaled_product.cu -- the matrix product of 8-bit floating point numbers with
// a scale for each block of 128:
//   out[t][n] = sum_b (sx[t][b] sw[n / 128][b]) sum_{k in b} x[t][k] w[n][k].
//
// The kernels feed tcgen05.mma (kind::f8f6f4, e4m3 x e4m3 -> fp32) from
// 128-byte swizzled tiles that TMA brings, one block of K (four instructions of
// K = 32) into a TMEM accumulator of its own; while the next block's runs, a
// set of warps reads it back and adds it to sums in registers, times the
// block's two scales.  Nothing but the inner sum of 128 is left to the tensor
// cores, and any fp32 scale is met exactly.
#include <algorithm>

#include "e4m3.cuh"
#include "gemm_umma.cuh"
#include "internal.h"
#include "rows.h"

namespace moe {

namespace {

constexpr int kStatusBytes = 256;

using pipe::mbar_arrive;
using pipe::mbar_expect_tx;
using pipe::mbar_init;
using pipe::saddr;
using umma::sw128_desc;
using umma::tc_fence_after;
using umma::tc_fence_before;
using umma::uwait;

struct ProductParams {
    const float *sx, *sw;
    size_t sx_stride, sw_stride, out_stride;     // elements
    int T, N, KB;
    void *out;
    int32_t *err;
    uint64_t timeout_ns;
    int stall;
    int split, stages;                           // few_kernel: CTAs of a cluster, stages of the ring
};

// Instruction descriptor of kind::f8f6f4: fp32 accumulator (bits 4-5 = 1), A
// and B e4m3 (bits 7-9, 10-12 = 0), both K-major, N >> 3 in bits 17-22, M >> 4
// in bits 24-28.
__host__ __device__ constexpr uint32_t idesc_e4m3(int m, int n) {
    return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

template <int CTAS>
__device__ __forceinline__ void mma_e4m3(uint32_t tmem_d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    if constexpr (CTAS == 1)
        asm volatile("{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
                     "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n"
                     ::"r"(tmem_d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
    else
        asm volatile("{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
                     "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n"
                     ::"r"(tmem_d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}

// NC accumulator columns of this warp's 32 lanes.
template <int NC>
__device__ __forceinline__ void tmem_ld(uint32_t at, uint32_t (&r)[NC]) {
    if constexpr (NC == 16) umma::tmem_ld_x16(at, r);
    else umma::tmem_ld_x32(at, r);
}

// Every thread of the cluster, once each.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}

__device__ __forceinline__ uint32_t mapped(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

__device__ __forceinline__ void put(float *at, float v) { *at = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *at, float v) { *at = __float2bfloat16_rn(v); }

// ---------------------------------------------------------------- few tokens
// The weights are the 128 rows of the MMA and the tokens its NT columns, so
// that a tile of weights is read once, for a token as for NT.  A cluster of
// `split` CTAs shares a tile's blocks of K and joins the sums through
// distributed shared memory, in the order of its CTAs.
constexpr int kFewThreads = 192;         // warps 0-3 sums, 4 TMA, 5 MMA
constexpr int kFewMaxStages = 12;
constexpr int kFewScales = 64;           // blocks whose scales stand in shared memory at a time
template <int NT>
struct Few {
    static constexpr int kSlots = NT <= 64 ? 4 : 2;                 // accumulators
    static constexpr int kCols = kSlots * NT;                       // TMEM columns: 64 to 256
    static constexpr int kStage = 128 * 128 + NT * 128;
};

// Blocks of a CTA, at most.
__host__ __device__ inline int few_share(int KB, int split) { return (KB + split - 1) / split; }
__host__ __device__ inline int few_scales(int KB, int split) { return min(few_share(KB, split), kFewScales); }

template <int NT>
size_t few_smem(int KB, int split, int stages) {
    return 1024 + (size_t)stages * Few<NT>::kStage + (size_t)few_scales(KB, split) * NT * 4 + (2 * kFewMaxStages + 2 * Few<NT>::kSlots + 1) * 8 + 16;
}

template <int NT, typename O>
__global__ void __launch_bounds__(kFewThreads) few_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                                                          const ProductParams p) {
    using F = Few<NT>;
    extern __shared__ __align__(1024) uint8_t smdyn[];
    uint8_t *stages = smdyn + ((1024u - (saddr(smdyn) & 1023u)) & 1023u);
    float *scales = reinterpret_cast<float *>(stages + (size_t)p.stages * F::kStage);           // [blocks][NT]
    uint64_t *full = reinterpret_cast<uint64_t *>(scales + few_scales(p.KB, p.split) * NT);
    uint64_t *empty = full + kFewMaxStages, *acc_full = empty + kFewMaxStages, *acc_empty = acc_full + F::kSlots;
    uint64_t *stall_bar = acc_empty + F::kSlots;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(stall_bar + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, S = p.split;
    const int tile = blockIdx.x / S, rank = blockIdx.x - tile * S, t0 = blockIdx.y * NT;
    const int kb0 = (int)((int64_t)p.KB * rank / S), nkb = (int)((int64_t)p.KB * (rank + 1) / S) - kb0;
    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; s++) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
        }
        for (int k = 0; k < F::kSlots; k++) {
            mbar_init(acc_full + k, 1);
            mbar_init(acc_empty + k, 4);
        }
        mbar_init(stall_bar, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 5) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(tmem_holder)), "n"(F::kCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;

    if (warp == 4) {
        // the first fills all at once, a lane for each copy
        const int n0 = min(nkb, p.stages);
        if (lane < 2 * n0) {
            const int q = lane >> 1;
            uint8_t *stage = stages + (size_t)q * F::kStage;
            if (lane & 1) {
                pipe::tma_2d(stage + 128 * 128, &xmap, (kb0 + q) * 128, t0, full + q);
            } else {
                mbar_expect_tx(full + q, F::kStage);
                pipe::tma_2d(stage, &wmap, (kb0 + q) * 128, tile * 128, full + q);
            }
        }
        __syncwarp();
        int q = n0;
        for (; q < nkb; q++) {
            const int s = q % p.stages;
            uint8_t *stage = stages + (size_t)s * F::kStage;
            if (!uwait(empty + s, ((q / p.stages) - 1) & 1, p.timeout_ns, abort_flag, p.err)) break;
            if (lane == 0) mbar_expect_tx(full + s, F::kStage);
            __syncwarp();
            if (lane == 0) pipe::tma_2d(stage, &wmap, (kb0 + q) * 128, tile * 128, full + s);
            else if (lane == 1) pipe::tma_2d(stage + 128 * 128, &xmap, (kb0 + q) * 128, t0, full + s);
            __syncwarp();
        }
        // the last fill of each stage lands before the CTA exits
        for (int s = 0; s < p.stages && s < q; s++) {
            const int last = q - 1 - ((q - 1 - s) % p.stages);
            if (!pipe::warp_wait(full + s, (last / p.stages) & 1, p.timeout_ns) && lane == 0) atomicExch(p.err, MOE_ETIMEOUT);
        }
    } else if (warp == 5) {
        for (int q = 0; q < nkb; q++) {
            const int s = q % p.stages, k = q % F::kSlots;
            const bool have = uwait(full + s, (q / p.stages) & 1, p.timeout_ns, abort_flag, p.err);
            const bool free = q < F::kSlots || uwait(acc_empty + k, ((q / F::kSlots) - 1) & 1, p.timeout_ns, abort_flag, p.err);
            tc_fence_after();
            if (lane == 0) {
                if (have && free && !*abort_flag) {
                    const uint64_t a = sw128_desc(saddr(stages + (size_t)s * F::kStage)), b = sw128_desc(saddr(stages + (size_t)s * F::kStage + 128 * 128));
#pragma unroll
                    for (int kk = 0; kk < 4; kk++)                   // 32 bytes of K each
                        mma_e4m3<1>(tmem + k * NT, a + 2 * kk, b + 2 * kk, idesc_e4m3(128, NT), kk > 0);
                }
                umma::umma_commit(empty + s);
                umma::umma_commit(acc_full + k);
            }
            __syncwarp();
        }
    } else {
        const int tid = threadIdx.x;
        if (p.stall && blockIdx.x == 0 && blockIdx.y == 0 && warp == 0) {        // test hook: bytes that no copy sends
            if (lane == 0) mbar_expect_tx(stall_bar, 16);
            __syncwarp();
            uwait(stall_bar, 0, p.timeout_ns, abort_flag, p.err);
        }
        float acc[NT];
#pragma unroll
        for (int j = 0; j < NT; j++) acc[j] = 0.0f;
        const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
        for (int q = 0; q < nkb; q++) {
            const int k = q % F::kSlots;
            if (q % kFewScales == 0) {
                // the products of the next blocks' scales (the first while the tiles are on their way)
                if (q) asm volatile("bar.sync 1, 128;" ::: "memory");
                for (int i = tid; i < min(nkb - q, kFewScales) * NT; i += 128) {
                    const int b = kb0 + q + i / NT, t = t0 + i % NT;
                    scales[i] = t < p.T ? __ldg(p.sx + (size_t)t * p.sx_stride + b) * __ldg(p.sw + (size_t)tile * p.sw_stride + b) : 0.0f;
                }
                asm volatile("bar.sync 1, 128;" ::: "memory");
            }
            const bool ok = uwait(acc_full + k, (q / F::kSlots) & 1, p.timeout_ns, abort_flag, p.err);
            tc_fence_after();
            // tcgen05.ld is warp-collective: the warp goes by lane 0's view
            if (__shfl_sync(0xffffffffu, (int)(ok && !*abort_flag), 0)) {
                constexpr int NC = NT < 32 ? 16 : 32;
                const float4 *sc = reinterpret_cast<const float4 *>(scales + q % kFewScales * NT);
#pragma unroll
                for (int c = 0; c < NT; c += NC) {
                    uint32_t d[NC];
                    tmem_ld<NC>(lanes + k * NT + c, d);
#pragma unroll
                    for (int j = 0; j < NC; j += 4) {
                        const float4 f = sc[(c + j) / 4];
                        acc[c + j] = fmaf(f.x, __uint_as_float(d[j]), acc[c + j]);
                        acc[c + j + 1] = fmaf(f.y, __uint_as_float(d[j + 1]), acc[c + j + 1]);
                        acc[c + j + 2] = fmaf(f.z, __uint_as_float(d[j + 2]), acc[c + j + 2]);
                        acc[c + j + 3] = fmaf(f.w, __uint_as_float(d[j + 3]), acc[c + j + 3]);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(acc_empty + k);
        }
        const int n = tile * 128 + tid, nt = min(NT, p.T - t0);
        if (S == 1) {
            O *out = static_cast<O *>(p.out) + (size_t)t0 * p.out_stride + n;
            if (n < p.N) {
#pragma unroll
                for (int j = 0; j < NT; j++)
                    if (j < nt) put(out + (size_t)j * p.out_stride, acc[j]);
            }
        } else if (!*abort_flag) {
            // over the ring, all of whose copies and products are done: [token][row]
            float *part = reinterpret_cast<float *>(stages);
#pragma unroll
            for (int j = 0; j < NT; j++)
                if (j < nt) part[j * 128 + tid] = acc[j];
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 5) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(F::kCols) : "memory");
    }
    if (S > 1) {
        cluster_sync();
        const int n = tile * 128 + (int)threadIdx.x, nt = min(NT, p.T - t0);
        if (threadIdx.x < 128 && n < p.N) {
            const uint32_t mine = saddr(stages) + threadIdx.x * 4;
            for (int j = rank; j < nt; j += S) {
                float sum = 0.0f;
                for (int r = 0; r < S; r++) {
                    float v;
                    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(mapped(mine + j * 512, r)) : "memory");
                    sum += v;
                }
                put(static_cast<O *>(p.out) + (size_t)(t0 + j) * p.out_stride + n, sum);
            }
        }
        cluster_sync();                  // no CTA's memory goes while another reads it
    }
}

int encode_tile(CUtensorMap *m, const void *base, size_t rows, size_t cols, size_t stride, int box_rows) {
    const cuuint64_t dims[2] = {cols, rows}, strides[1] = {rows > 1 ? stride : align_up(cols, 16)};
    const cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
    return pipe::encode_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int NT, typename O>
int launch_few(const CUtensorMap &wmap, const CUtensorMap &xmap, ProductParams p, cudaStream_t st) {
    const int tiles = (p.N - 1) / 128 + 1, cols = (p.T - 1) / NT + 1;
    p.split = 1;
    while (p.split < 8 && 2 * p.split <= p.KB && (int64_t)tiles * cols * p.split * 2 <= 2 * num_sms()) p.split *= 2;
    p.stages = std::min(std::max(2, few_share(p.KB, p.split)), std::min(kFewMaxStages, (100 << 10) / Few<NT>::kStage));
    p.stages = std::max(p.stages, (NT * 512 + Few<NT>::kStage - 1) / Few<NT>::kStage);       // room for the sums
    const size_t smem = few_smem<NT>(p.KB, p.split, p.stages);
    static OnDevices ready;
    cudaError_t e = ready.once([] { return cudaFuncSetAttribute(few_kernel<NT, O>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 << 10); });
    if (e != cudaSuccess) return fail(MOE_ECUDA, "scaled_product: %s", cudaGetErrorString(e));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * p.split), (unsigned)cols);
    cfg.blockDim = dim3(kFewThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)p.split;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, few_kernel<NT, O>, wmap, xmap, p);
    if (e != cudaSuccess) return fail(MOE_ECUDA, "scaled_product: %s", cudaGetErrorString(e));
    return check_launch("few_kernel");
}

template <typename O>
int launch_product(const void *x, size_t x_stride, const moe_scaled_matrix_desc *wd, const ProductParams &p, cudaStream_t st) {
    CUtensorMap wmap, xmap;
    const int nt = p.T <= 16 ? 16 : p.T <= 32 ? 32 : p.T <= 64 ? 64 : 128;
    if (encode_tile(&wmap, wd->w, wd->N, wd->K, wd->w_stride, 128) || encode_tile(&xmap, x, p.T, wd->K, x_stride, nt))
        return fail(MOE_ECUDA, "scaled_product: no tensor map");
    switch (nt) {
    case 16: return launch_few<16, O>(wmap, xmap, p, st);
    case 32: return launch_few<32, O>(wmap, xmap, p, st);
    case 64: return launch_few<64, O>(wmap, xmap, p, st);
    default: return launch_few<128, O>(wmap, xmap, p, st);
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
    const pipe::WaitCfg wait = pipe::wait_cfg();
    ProductParams p = {};
    p.sx = x_scales, p.sw = wd->scales, p.sx_stride = x_scale_stride, p.sw_stride = wd->scale_stride, p.out_stride = out_stride;
    p.T = T, p.N = wd->N, p.KB = (int)blocks, p.out = out, p.err = static_cast<int32_t *>(ws);
    p.timeout_ns = wait.timeout_ns ? wait.timeout_ns : pipe::kDefaultWaitNs, p.stall = wait.stall;
    return out_dtype == MOE_DTYPE_F32 ? launch_product<float>(x, x_stride, wd, p, stream)
                                      : launch_product<__nv_bfloat16>(x, x_stride, wd, p, stream);
}
