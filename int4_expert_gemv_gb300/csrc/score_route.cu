// score_route.cu -- routing by scores: softmax or sigmoid of the router's
// logits, a balance bias that moves only the choice, groups of experts of
// which a few stay, the K best of those and their renormalised weights.
//
// One warp per token.  The group count is rounded up to a power of two that
// divides the warp, so a group is 32 / that many neighbouring lanes, each
// with NV consecutive experts of it: a group's best two come from log2 steps
// of shuffles for all groups at once, and equal choices resolve to the lowest
// lane, then the lowest register -- the lowest index.  Choices are compared as
// 32-bit keys that order like the numbers, so a round of the top-K is one
// warp-wide integer maximum and a ballot.
#include "internal.h"

namespace moe {

namespace {

struct RouteParams {
    const void *z;
    size_t stride;
    int T, E, K, n_group, gs, lanes, keep, best, renorm;   // gs: experts of a group, lanes: of a group
    float factor;
    const float *bias;
    int32_t *idx;
    float *w;
};

constexpr uint32_t kOut = 0u;                 // no expert, or one of a dropped group

// Orders as the numbers do (NaN excluded); -0 is made +0 first.
__device__ __forceinline__ uint32_t order_key(float c) {
    const uint32_t u = __float_as_uint(c + 0.0f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

template <typename X>
__device__ __forceinline__ float logit(const void *row, int e);
template <>
__device__ __forceinline__ float logit<float>(const void *row, int e) {
    return __ldg(static_cast<const float *>(row) + e);
}
template <>
__device__ __forceinline__ float logit<__nv_bfloat16>(const void *row, int e) {
    return __bfloat162float(static_cast<const __nv_bfloat16 *>(row)[e]);
}

__device__ __forceinline__ float sigmoid_f(float z) { return __fdiv_rn(1.0f, 1.0f + expf(-z)); }

// exp(z - m) with +inf logits sharing the mass
__device__ __forceinline__ float soft_f(float z, float m) { return z == m ? 1.0f : expf(z - m); }

template <typename X, int NV, bool SIGMOID>
__global__ void __launch_bounds__(256) scored_route_kernel(const RouteParams p) {
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (t >= p.T) return;                     // whole warps
    const X *row = static_cast<const X *>(p.z) + (size_t)t * p.stride;
    const int group = lane / p.lanes, first = (lane - group * p.lanes) * NV;
    const int base = group * p.gs + first;
    const int n = group < p.n_group ? min(NV, max(0, p.gs - first)) : 0;   // this lane's experts

    float s[NV];
#pragma unroll
    for (int i = 0; i < NV; i++) s[i] = i < n ? logit<X>(row, base + i) : -INFINITY;
    float m = -INFINITY, inv = 0.0f;
    if (!SIGMOID) {
#pragma unroll
        for (int i = 0; i < NV; i++) m = fmaxf(m, s[i]);          // NaN is passed over
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const bool on = s[i] > -INFINITY;                    // neither -inf nor NaN
            const float e = on ? soft_f(s[i], m) : 0.0f;
            sum += e;
            s[i] = on ? e : -INFINITY;
        }
        sum = warp_sum(sum, 32);
        inv = sum;
    }
    uint32_t key[NV];
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const bool on = s[i] > -INFINITY;
        float c = -INFINITY;
        if (on) {
            c = SIGMOID ? sigmoid_f(s[i]) : __fdiv_rn(s[i], inv);
            if (p.bias) c += __ldg(p.bias + base + i);
            if (c != c) c = -INFINITY;
        }
        key[i] = i < n ? order_key(c) : kOut;
    }

    if (p.keep < p.n_group) {
        uint32_t b1 = kOut, b2 = kOut;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            b2 = max(b2, min(b1, key[i]));
            b1 = max(b1, key[i]);
        }
        for (int o = p.lanes >> 1; o > 0; o >>= 1) {
            const uint32_t o1 = __shfl_xor_sync(0xffffffffu, b1, o);
            const uint32_t o2 = __shfl_xor_sync(0xffffffffu, b2, o);
            b2 = max(max(b2, o2), min(b1, o1));
            b1 = max(b1, o1);
        }
        float g = p.best == 1 ? key_value(b1) : key_value(b1) + key_value(b2);
        if (g != g) g = -INFINITY;
        const uint32_t mine = order_key(g);
        int rank = 0;
        for (int j = 0; j < p.n_group; j++) {
            const uint32_t other = __shfl_sync(0xffffffffu, mine, j * p.lanes);
            rank += other > mine || (other == mine && j < group);
        }
        if (rank >= p.keep) {
#pragma unroll
            for (int i = 0; i < NV; i++) key[i] = kOut;
        }
    }

    int chosen = 0;                           // lane k: the k-th choice
    for (int k = 0; k < p.K; k++) {
        uint32_t b = key[0];
        int bi = 0;
#pragma unroll
        for (int i = 1; i < NV; i++)
            if (key[i] > b) {
                b = key[i];
                bi = i;
            }
        const uint32_t top = __reduce_max_sync(0xffffffffu, b);
        const int src = __ffs(__ballot_sync(0xffffffffu, b == top)) - 1;
        const int e = __shfl_sync(0xffffffffu, base + bi, src);
        if (lane == k) chosen = e;
        if (lane == src) {
#pragma unroll
            for (int i = 0; i < NV; i++)
                if (i == bi) key[i] = kOut;
        }
    }
    float w = 0.0f;
    if (lane < p.K) {
        const float z = logit<X>(row, chosen);
        if (z > -INFINITY) w = SIGMOID ? sigmoid_f(z) : __fdiv_rn(soft_f(z, m), inv);
    }
    if (p.renorm) {
        const float sum = warp_sum(w, 32);
        w = sum > 0.0f ? __fdiv_rn(w, sum) : 0.0f;
    }
    if (lane < p.K) {
        p.idx[(size_t)t * p.K + lane] = chosen;
        p.w[(size_t)t * p.K + lane] = w * p.factor;
    }
}

template <typename X, bool SIGMOID>
void launch_nv(const RouteParams &p, int nv, cudaStream_t st) {
    const int threads = 256;
    const unsigned grid = (unsigned)((p.T + threads / 32 - 1) / (threads / 32));
    if (nv <= 1) scored_route_kernel<X, 1, SIGMOID><<<grid, threads, 0, st>>>(p);
    else if (nv <= 2) scored_route_kernel<X, 2, SIGMOID><<<grid, threads, 0, st>>>(p);
    else if (nv <= 4) scored_route_kernel<X, 4, SIGMOID><<<grid, threads, 0, st>>>(p);
    else if (nv <= 8) scored_route_kernel<X, 8, SIGMOID><<<grid, threads, 0, st>>>(p);
    else if (nv <= 16) scored_route_kernel<X, 16, SIGMOID><<<grid, threads, 0, st>>>(p);
    else if (nv <= 32) scored_route_kernel<X, 32, SIGMOID><<<grid, threads, 0, st>>>(p);
    else scored_route_kernel<X, 64, SIGMOID><<<grid, threads, 0, st>>>(p);
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" int moe_scored_route(const moe_route_desc *rd, const void *logits, int logits_dtype,
                                size_t stride, int T, int32_t *idx, float *w,
                                cudaStream_t stream) {
    if (rd == nullptr) return fail(MOE_EINVAL, "scored_route: descriptor is NULL");
    if (T < 0 || rd->E < 1 || rd->E > 1024 || rd->K < 1 || rd->K > 16)
        return fail(MOE_EINVAL, "scored_route: T=%d E=%d K=%d (need 1<=K<=16, 1<=E<=1024)", T, rd->E,
                    rd->K);
    if (rd->score != MOE_SCORE_SOFTMAX && rd->score != MOE_SCORE_SIGMOID)
        return fail(MOE_EINVAL, "scored_route: score=%d", rd->score);
    if (rd->n_group < 1 || rd->n_group > 32 || rd->E % rd->n_group || rd->keep_group < 1 ||
        rd->keep_group > rd->n_group)
        return fail(MOE_EINVAL, "scored_route: %d of %d groups of E=%d (need 1..32 groups that divide "
                                "E)", rd->keep_group, rd->n_group, rd->E);
    const int gs = rd->E / rd->n_group;
    if (rd->K > rd->keep_group * gs)
        return fail(MOE_EINVAL, "scored_route: K=%d of %d experts in the kept groups", rd->K,
                    rd->keep_group * gs);
    if (rd->group_best < 1 || rd->group_best > 2 || (rd->n_group > 1 && rd->group_best > gs))
        return fail(MOE_EINVAL, "scored_route: group_best=%d with groups of %d", rd->group_best, gs);
    if (logits_dtype != MOE_DTYPE_F32 && logits_dtype != MOE_DTYPE_BF16)
        return fail(MOE_EINVAL, "scored_route: logits_dtype=%d", logits_dtype);
    if (T == 0) return MOE_OK;
    const size_t elt = logits_dtype == MOE_DTYPE_F32 ? 4 : 2;
    if (!logits || !idx || !w) return fail(MOE_EINVAL, "scored_route: NULL pointer");
    if (reinterpret_cast<uintptr_t>(logits) % elt || reinterpret_cast<uintptr_t>(idx) % 4 ||
        reinterpret_cast<uintptr_t>(w) % 4 || reinterpret_cast<uintptr_t>(rd->bias) % 4)
        return fail(MOE_EINVAL, "scored_route: misaligned pointer");
    if (T > 1 && stride < (size_t)rd->E)
        return fail(MOE_EINVAL, "scored_route: stride %zu below E=%d", stride, rd->E);
    RouteParams p{};
    p.z = logits;
    p.stride = stride;
    p.T = T;
    p.E = rd->E;
    p.K = rd->K;
    p.n_group = rd->n_group;
    p.gs = gs;
    int np = 1;
    while (np < rd->n_group) np *= 2;
    p.lanes = 32 / np;
    p.keep = rd->keep_group;
    p.best = rd->group_best;
    p.renorm = rd->renorm != 0;
    p.factor = rd->factor;
    p.bias = rd->bias;
    p.idx = idx;
    p.w = w;
    const int nv = (gs + p.lanes - 1) / p.lanes;      // at most 61: E <= 1024
    const bool sig = rd->score == MOE_SCORE_SIGMOID;
    if (logits_dtype == MOE_DTYPE_F32) {
        if (sig) launch_nv<float, true>(p, nv, stream);
        else launch_nv<float, false>(p, nv, stream);
    } else {
        if (sig) launch_nv<__nv_bfloat16, true>(p, nv, stream);
        else launch_nv<__nv_bfloat16, false>(p, nv, stream);
    }
    return check_launch("scored_route_kernel");
}
