// attend.cu -- the paged attention's entry: validation, workspace, choice of
// the kernel by types and head size.
#include "attend.cuh"

namespace moe {

namespace {

struct AttendWs {
    AttendPlan plan;
    int ctas;
    size_t ml, o, total;
};

// {row descriptors, (m, l) and O of two partial rows per CTA}
AttendWs attend_ws(const moe_kv_desc *kv, int Hq) {
    AttendWs w;
    w.plan = attend_plan(kv->D, kv->dtype == MOE_DTYPE_E4M3, Hq / kv->Hkv);
    w.ctas = num_sms() * w.plan.ctas_per_sm;
    const size_t rows = 2 * (size_t)w.ctas * w.plan.rows;
    w.ml = align_up((size_t)w.ctas * sizeof(int4), 256);
    w.o = align_up(w.ml + rows * sizeof(float2), 256);
    w.total = align_up(w.o + rows * w.plan.dp * sizeof(float), 256);
    return w;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" size_t moe_paged_attention_workspace_bytes(const moe_kv_desc *kv, int B, int Hq) {
    if (kv == nullptr || B < 0 || Hq < 1 || kv->Hkv < 1 || Hq % kv->Hkv || kv->D < 16 || kv->D > 256) return 0;
    return attend_ws(kv, Hq).total;
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
    if (kv->page_stride > UINT32_MAX)
        return fail(MOE_EUNSUPPORTED, "paged_attention: page_stride %zu (need below 2^32)", kv->page_stride);
    if ((int64_t)B * Hq > INT32_MAX)
        return fail(MOE_EUNSUPPORTED, "paged_attention: B=%d Hq=%d (need fewer than 2^31 rows)", B, Hq);
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
    const AttendWs wl = attend_ws(kv, Hq);
    const bool f8 = kv->dtype == MOE_DTYPE_E4M3;
    uint8_t *w = static_cast<uint8_t *>(ws);
    AttendParams p{};
    p.k = static_cast<const uint8_t *>(kv->k);
    p.v = static_cast<const uint8_t *>(kv->v);
    p.page_stride = (uint32_t)kv->page_stride;
    p.k_scale = kv->k_scale;
    p.v_scale = kv->v_scale;
    p.n_pages = kv->n_pages;
    p.Hkv = kv->Hkv;
    p.D = kv->D;
    p.B = B;
    p.page = FastDiv(kv->page);
    p.G = Hq / kv->Hkv;
    p.tiles = (p.G + wl.plan.rows - 1) / wl.plan.rows;
    p.q = q;
    p.q_stride = q_stride;
    p.out_stride = out_stride;
    p.Hq = Hq;
    p.seq = seq_len;
    p.table = block_table;
    p.max_blocks = max_blocks;
    p.window = window;
    p.scale = scale;
    p.out = out;
    p.lse = lse;
    p.meta = reinterpret_cast<int4 *>(w);
    p.part_ml = reinterpret_cast<float2 *>(w + wl.ml);
    p.part_o = reinterpret_cast<float *>(w + wl.o);
    const bool f32 = q_dtype == MOE_DTYPE_F32;
    if (f8) return f32 ? launch_attend_e4m3_qf32(p, wl.plan.dp, stream) : launch_attend_e4m3_qbf16(p, wl.plan.dp, stream);
    return f32 ? launch_attend_bf16_qf32(p, wl.plan.dp, stream) : launch_attend_bf16_qbf16(p, wl.plan.dp, stream);
}
