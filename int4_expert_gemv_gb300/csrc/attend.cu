// attend.cu -- attention of one new token per request over a paged key-value
// cache.
//
// One CTA per (request, query head): every warp takes each eighth token, its
// lanes the head's dimensions, with a running maximum and sum per warp that
// the CTA joins at the end.
#include <cuda_fp8.h>

#include "internal.h"

namespace moe {

namespace {

struct AttendParams {
    const uint8_t *k, *v;
    size_t page_stride;
    const float *k_scale, *v_scale;
    int n_pages, Hkv, D, e4m3, G, Hq;
    FastDiv page;
    const void *q;
    int q_dtype;
    size_t q_stride, out_stride;
    const int32_t *seq, *table;
    int max_blocks, window;
    float scale;
    void *out;
    float *lse;
};

__device__ __forceinline__ float cache_num(const uint8_t *p, int i, int e4m3) {
    if (e4m3) {
        __nv_fp8_e4m3 x;
        x.__x = p[i];
        return (float)x;
    }
    return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p)[i]);
}

constexpr int kMaxPer = 8;       // 256 / 32

__global__ void __launch_bounds__(256) attend_kernel(const AttendParams p) {
    __shared__ float sm_m[8], sm_l[8], sm_o[8][256];
    const int b = blockIdx.x / p.Hq, hq = blockIdx.x % p.Hq, h = hq / p.G;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = (p.D + 31) / 32, elt = p.e4m3 ? 1 : 2;
    int len = max(0, p.seq[b]);
    bool bad = (int64_t)len > (int64_t)p.max_blocks * p.page.d;
    if (bad) len = 0;
    const int lo = p.window > 0 ? max(0, len - p.window) : 0;
    const float ks = p.scale * (p.k_scale ? p.k_scale[h] : 1.0f), vs = p.v_scale ? p.v_scale[h] : 1.0f;
    float q[kMaxPer], o[kMaxPer] = {};
    for (int i = 0; i < per; i++) {
        const int c = lane + 32 * i;
        q[i] = c < p.D ? load_act(p.q, p.q_dtype, (size_t)b * p.q_stride + (size_t)hq * p.D + c) : 0.0f;
    }
    float m = -INFINITY, l = 0.0f;
    for (int t = lo + warp; t < len; t += 8) {
        const int blk = p.page.div(t), off = t - blk * p.page.d;
        const int id = p.table[(size_t)b * p.max_blocks + blk];
        if ((unsigned)id >= (unsigned)p.n_pages) {
            bad = true;
            break;
        }
        const size_t at = (size_t)id * p.page_stride + ((size_t)h * p.page.d + off) * p.D * elt;
        float x = 0.0f;
        for (int i = 0; i < per; i++) {
            const int c = lane + 32 * i;
            if (c < p.D) x = fmaf(q[i], cache_num(p.k + at, c, p.e4m3), x);
        }
        x = warp_sum(x, 32) * ks;
        const float mn = fmaxf(m, x), f = m == -INFINITY ? 0.0f : expf(m - mn), e = expf(x - mn);
        l = l * f + e;
        m = mn;
        for (int i = 0; i < per; i++) {
            const int c = lane + 32 * i;
            if (c < p.D) o[i] = fmaf(e, cache_num(p.v + at, c, p.e4m3), o[i] * f);
        }
    }
    if (lane == 0) {
        sm_m[warp] = m;
        sm_l[warp] = l;
    }
    for (int i = 0; i < per; i++) sm_o[warp][lane + 32 * i] = o[i];
    bad = __syncthreads_or(bad);
    m = -INFINITY;
    for (int w = 0; w < 8; w++) m = fmaxf(m, sm_m[w]);
    l = 0.0f;
    float f[8];
    for (int w = 0; w < 8; w++) {
        f[w] = sm_m[w] == -INFINITY ? 0.0f : expf(sm_m[w] - m);
        l += f[w] * sm_l[w];
    }
    const int c = threadIdx.x;
    if (c < p.D) {
        float a = 0.0f;
        for (int w = 0; w < 8; w++)
            if (f[w] > 0.0f) a = fmaf(f[w], sm_o[w][c], a);
        a = bad ? NAN : l > 0.0f ? a / l * vs : 0.0f;
        const size_t i = (size_t)b * p.out_stride + (size_t)hq * p.D + c;
        if (p.q_dtype == MOE_DTYPE_F32) static_cast<float *>(p.out)[i] = a;
        else static_cast<__nv_bfloat16 *>(p.out)[i] = __float2bfloat16(a);
    }
    if (c == 0 && p.lse)
        p.lse[(size_t)b * p.Hq + hq] = bad ? NAN : l > 0.0f ? m + logf(l) : -INFINITY;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" size_t moe_paged_attention_workspace_bytes(const moe_kv_desc *kv, int B, int Hq) {
    if (kv == nullptr || B < 0 || Hq < 1 || kv->Hkv < 1 || Hq % kv->Hkv) return 0;
    return 256;
}

extern "C" int moe_paged_attention(const moe_kv_desc *kv, const void *q, int q_dtype,
                                   size_t q_stride, int B, int Hq, const int32_t *seq_len,
                                   const int32_t *block_table, int max_blocks, float scale,
                                   int window, void *out, size_t out_stride, float *lse, void *ws,
                                   size_t ws_bytes, cudaStream_t stream) {
    if (int rc = check_kv(kv, "paged_attention")) return rc;
    if (B < 0 || B > 65536 || Hq < 1 || Hq > 65536 || Hq % kv->Hkv || max_blocks < 1 || window < 0)
        return fail(MOE_EINVAL, "paged_attention: B=%d Hq=%d Hkv=%d max_blocks=%d window=%d (need "
                                "B, Hq <= 65536, Hq a multiple of Hkv)", B, Hq, kv->Hkv, max_blocks,
                    window);
    if (q_dtype != MOE_DTYPE_F32 && q_dtype != MOE_DTYPE_BF16)
        return fail(MOE_EINVAL, "paged_attention: q_dtype=%d", q_dtype);
    if (!(scale > 0.0f) || !(scale < INFINITY))
        return fail(MOE_EINVAL, "paged_attention: scale=%g (need a positive number)", (double)scale);
    if (B == 0) return MOE_OK;
    const size_t row = (size_t)Hq * kv->D, elt = q_dtype == MOE_DTYPE_F32 ? 4 : 2;
    if (!q || !out || !seq_len || !block_table || reinterpret_cast<uintptr_t>(q) % 16 ||
        reinterpret_cast<uintptr_t>(out) % 16 || reinterpret_cast<uintptr_t>(seq_len) % 4 ||
        reinterpret_cast<uintptr_t>(block_table) % 4 || reinterpret_cast<uintptr_t>(lse) % 4)
        return fail(MOE_EINVAL, "paged_attention: NULL or misaligned pointer");
    if ((B > 1 && (q_stride < row || out_stride < row)) || q_stride * elt % 16 || out_stride * elt % 16)
        return fail(MOE_EINVAL, "paged_attention: strides %zu / %zu (need >= %zu numbers, 16-byte "
                                "multiples)", q_stride, out_stride, row);
    const size_t need = moe_paged_attention_workspace_bytes(kv, B, Hq);
    if (ws == nullptr || ws_bytes < need || reinterpret_cast<uintptr_t>(ws) % 256)
        return fail(MOE_ENOSPACE, "paged_attention: workspace %zu bytes, need %zu (256-aligned)",
                    ws_bytes, need);
    AttendParams p{};
    p.k = static_cast<const uint8_t *>(kv->k);
    p.v = static_cast<const uint8_t *>(kv->v);
    p.page_stride = kv->page_stride;
    p.k_scale = kv->k_scale;
    p.v_scale = kv->v_scale;
    p.n_pages = kv->n_pages;
    p.Hkv = kv->Hkv;
    p.D = kv->D;
    p.e4m3 = kv->dtype == MOE_DTYPE_E4M3;
    p.G = Hq / kv->Hkv;
    p.Hq = Hq;
    p.page = FastDiv(kv->page);
    p.q = q;
    p.q_dtype = q_dtype;
    p.q_stride = q_stride;
    p.out_stride = out_stride;
    p.seq = seq_len;
    p.table = block_table;
    p.max_blocks = max_blocks;
    p.window = window;
    p.scale = scale;
    p.out = out;
    p.lse = lse;
    attend_kernel<<<(unsigned)(B * Hq), 256, 0, stream>>>(p);
    return check_launch("attend_kernel");
}
