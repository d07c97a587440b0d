// score_route.cu -- routing by scores: softmax or sigmoid of the router's
// logits, a balance bias that moves only the choice, groups of experts of
// which a few stay, the K best of those and their renormalised weights.
//
// Layout.  LT lanes (8 or 32) share a token.  A group's experts stand in
// blocks of 8 (the last one short), block s of the token with lane s mod LT:
// one lane reads 32 or 16 bytes of a row, its neighbours the next ones.  A
// lane keeps each of its blocks' largest choice in a register and all
// choices in shared memory.  A round of the top-K is then a maximum over a
// lane's blocks and over LT lanes, and the chosen block's eight before eight
// lanes: which one it was, and the largest that is left.  With 8 lanes a warp
// does so for four tokens at once, which is what the rounds cost most of;
// with 32 a token has the shorter chain.  Choices are floats: what is off is
// -FLT_MAX (all other choices are kept above it, at kLowest at least), what is
// taken or dropped -inf.
//
// Bound.  The logits are read once (4 E bytes a token, 10.5 us for 65521
// tokens of 256 at the copy rate) and each costs an exponential and a
// reciprocal for its sigmoid: 16 of those a clock and SM make 7 us there.
// Measured 31.0 us with bias and 4 of 8 groups, K = 8: issue slots (68 % taken)
// and the latencies of shared memory and shuffles share it; a round costs 1.2
// us (1.5 past the eighth), the groups 3.8, and the rest 17: loads, scores, the
// way of all choices through shared memory, weights.  Without a bias the
// choices are the logits: 25.0 us without groups (softmax 24.4), 30.5 with
// groups by their best two.  Beside the 32 us of an earlier state, a warp per
// token with a warp-wide integer maximum per round took 68; two or four lanes a
// token 41 (shared memory then halves the warps of an SM); the lane of a block
// going through its eight alone 35; a block's second choice kept in a register
// 36, and 64 instead of 45 with K = 16 (some token of the four always has to
// look for a third); the row asked for ahead into L2 33.
#include <cfloat>
#include <type_traits>

#include "fastdiv.cuh"
#include "internal.h"

namespace moe {

namespace {

struct RouteParams {
    const void *z;
    size_t stride;
    int T, E, K, n_group, gs, nsub, keep, best, renorm;   // gs: experts of a group, nsub: blocks of a token
    FastDiv spg;                                          // blocks of a group
    int vec;                                              // whole blocks, 16-byte aligned
    int tok;                                              // floats of a token in shared memory
    float factor;
    const float *bias;
    int32_t *idx;
    float *w;
};

constexpr int kRouteThreads = 128;

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

template <typename X>
__device__ __forceinline__ void logits8(const void *row, int e, float *f);
template <>
__device__ __forceinline__ void logits8<float>(const void *row, int e, float *f) {
    const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(row) + e);
    const float4 a = __ldg(q), b = __ldg(q + 1);
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}
template <>
__device__ __forceinline__ void logits8<__nv_bfloat16>(const void *row, int e, float *f) {
    const uint4 a = __ldg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(row) + e));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; j++) {
        f[2 * j] = __uint_as_float(w[j] << 16);
        f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
}

// Without a bias the choice goes by the logits themselves: both scores grow
// with them, and what fp32 cannot hold or tell apart (e^-100 beside 1, the
// sigmoids of 20 and 21) still has its order.  With a bias it goes by quick
// scores (2^-21 of exact, of 1; below 2^-126 they are 0), equal for equal
// logits; the weights of the chosen by exact exponentials and quotients.
__device__ __forceinline__ float quick_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float quick_sigmoid(float z) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(1.0f + quick_exp2(z * -1.44269504088896341f)));
    return y;
}
// The lowest choice of an expert that is on; what is off is just below it.
constexpr float kLowest = -0x1.fffffcp127f;

__device__ __forceinline__ float size8(const float *f) {
    return (fabsf(f[0]) + fabsf(f[1])) + (fabsf(f[2]) + fabsf(f[3])) +
           ((fabsf(f[4]) + fabsf(f[5])) + (fabsf(f[6]) + fabsf(f[7])));
}

// A group's score by its two best logits, in an order that is the sums' also
// where they are below fp32's numbers: the sum, or below e^-20 (where sigmoids
// are exponentials to 2^-28) its logarithm, which is negative as no sum is.
template <bool SIGMOID>
__device__ __forceinline__ float pair_score(float b1, float b2, float m) {
    if (b2 == -FLT_MAX) return b2;                  // only one is on, or none
    if (!SIGMOID && m == INFINITY) return b1 + b2;  // (these are scores, of 0 and 1)
    const float x1 = SIGMOID ? b1 : b1 - m, x2 = SIGMOID ? b2 : b2 - m;
    if (x1 < -20.0f) {
        const float sum = x1 + log1pf(expf(b2 - b1));
        if (sum < -20.0f) return fmaxf(sum, kLowest);
    }
    return SIGMOID ? quick_sigmoid(x1) + quick_sigmoid(x2)
                   : quick_exp2(x1 * 1.44269504088896341f) + quick_exp2(x2 * 1.44269504088896341f);
}

template <int LT>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
    for (int o = LT / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
template <int LT>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = LT / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Shared memory of a token: its choices (the first, then the second float4 of
// every block, so that neighbouring lanes meet no bank twice), with groups the
// blocks' best two, the places of the chosen.
inline int route_token_floats(int nsub, bool groups) { return nsub * 8 + (groups ? (nsub + 1) / 2 * 4 : 0) + 16; }

template <typename X, int LT, int SUB, bool SIGMOID, bool VEC>
__global__ void __launch_bounds__(kRouteThreads, SUB <= 4 ? 10 : 1) scored_route_kernel(const RouteParams p) {
    extern __shared__ __align__(16) float smem[];
    constexpr int TOK = kRouteThreads / LT;
    const int NB = p.nsub;
    const int lane = threadIdx.x & 31, sub = threadIdx.x / LT, l = threadIdx.x % LT;
    const uint32_t tt = blockIdx.x * TOK + sub;
    const bool live = tt < (uint32_t)p.T;
    const int t = live ? (int)tt : p.T - 1;        // the last warp's idle lanes repeat a token
    float *c_s = smem + sub * p.tok;
    float4 *c4 = reinterpret_cast<float4 *>(c_s);
    float2 *best_s = reinterpret_cast<float2 *>(c_s + NB * 8);
    int *pick_s = reinterpret_cast<int *>(c_s + p.tok - 16);
    const X *row = static_cast<const X *>(p.z) + (size_t)t * p.stride;
    const bool groups = p.keep < p.n_group;

    // first expert of block s
    auto expert0 = [&](int s) {
        const int grp = p.spg.div(s);
        return grp * p.gs + (s - grp * p.spg.d) * 8;
    };
    // how many of block s's places have an expert (s < nsub)
    auto count = [&](int s) { return VEC ? 8 : p.gs - (s - p.spg.div(s) * p.spg.d) * 8; };
    // block s's eight numbers of a row of E; -inf where there is no expert
    auto read8 = [&](auto *x, int s, float *f) {
        using Y = typename std::remove_const<typename std::remove_pointer<decltype(x)>::type>::type;
        if (VEC) {
            logits8<Y>(x, expert0(s), f);
        } else {
            const int e0 = expert0(s), n = count(s);
#pragma unroll
            for (int i = 0; i < 8; i++) f[i] = i < n ? logit<Y>(x, e0 + i) : -INFINITY;
        }
    };
    auto put8 = [&](int s, const float *f) {
        c4[s] = make_float4(f[0], f[1], f[2], f[3]);
        c4[NB + s] = make_float4(f[4], f[5], f[6], f[7]);
    };
    auto get8 = [&](int s, float *f) {
        const float4 a = c4[s], b = c4[NB + s];
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    };

    const bool raw = p.bias == nullptr;             // the choices are the logits
    float m = -INFINITY, total = 1.0f;
    if (!SIGMOID) {                                 // the maximum
#pragma unroll
        for (int j = 0; j < SUB; j++) {
            const int s = l + LT * j;
            if (s < p.nsub) {
                float f[8];
                read8(row, s, f);
#pragma unroll
                for (int i = 0; i < 8; i++) m = fmaxf(m, f[i]);        // passes NaN over
                put8(s, f);
            }
        }
        m = lanes_max<LT>(m);
    }
    if (!SIGMOID && !(raw && p.renorm)) {           // the exponentials, and their sum
        const bool share = __any_sync(0xffffffffu, m == INFINITY);     // +inf logits share the mass
        const float ref = m == INFINITY || m == -INFINITY ? 0.0f : m;
        total = 0.0f;
#pragma unroll
        for (int j = 0; j < SUB; j++) {
            const int s = l + LT * j;
            if (s < p.nsub) {
                float f[8];
                get8(s, f);
                if (share && m == INFINITY) {
#pragma unroll
                    for (int i = 0; i < 8; i++)
                        if (f[i] > -INFINITY) f[i] = f[i] == INFINITY ? 0.0f : -FLT_MAX;
                }
                // (the maximum's own term is 1 wherever the logits stand, as in the weights below)
                float e[8];
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    e[i] = quick_exp2((f[i] - ref) * 1.44269504088896341f);
                    total += fmaxf(e[i], 0.0f);                        // (passes NaN over)
                }
                if (!raw) {
#pragma unroll
                    for (int i = 0; i < 8; i++) e[i] = f[i] > -INFINITY ? e[i] : -FLT_MAX;   // off: -inf and NaN
                    put8(s, e);
                }
            }
        }
        total = lanes_sum<LT>(total);
    }
    const float inv = SIGMOID ? 1.0f : __fdiv_rn(1.0f, fmaxf(total, FLT_MIN));
    float top[SUB];                                 // the blocks' largest choices
    // (Two loops, by whether there is a bias: a branch within one keeps the next
    // blocks' loads from being asked for ahead of it: 33.4 us against 31.0.)
    auto choices = [&](auto no_bias) {
        constexpr bool RAW = decltype(no_bias)::value;
#pragma unroll
        for (int j = 0; j < SUB; j++) {
            const int s = l + LT * j;
            top[j] = -INFINITY;
            if (s < p.nsub) {
                float f[8];
                // A block whose logits, and whose choices with their bias, are below
                // 2^127 in size all together holds nothing that is off and no choice
                // below kLowest: one test for eight.
                bool plain = true, put = SIGMOID || !RAW || !VEC;
                if (SIGMOID) read8(row, s, f);
                else get8(s, f);
                if constexpr (RAW) {
                    const bool share = !SIGMOID && m == INFINITY;
                    if (!(size8(f) < 0x1p127f) || share) {
#pragma unroll
                        for (int i = 0; i < 8; i++) {
                            const float c = share ? (f[i] == INFINITY ? 1.0f : 0.0f) : fmaxf(f[i], kLowest);
                            f[i] = f[i] > -INFINITY ? c : -FLT_MAX;
                        }
                        put = true;
                    }
                } else if constexpr (SIGMOID) {
                    plain = size8(f) < 0x1p127f;
                    float c[8];
#pragma unroll
                    for (int i = 0; i < 8; i++) c[i] = quick_sigmoid(f[i]);
                    if (!plain) {
#pragma unroll
                        for (int i = 0; i < 8; i++)
                            if (!(f[i] > -INFINITY)) c[i] = -FLT_MAX;
                    }
#pragma unroll
                    for (int i = 0; i < 8; i++) f[i] = c[i];
                }
                if (!RAW) {
                    float c[8];
                    read8(p.bias, s, c);
#pragma unroll
                    for (int i = 0; i < 8; i++) c[i] = fmaf(f[i], inv, c[i]);
                    if (!plain || !(size8(c) < 0x1p127f) || !SIGMOID) {    // (softmax marks what is off by -FLT_MAX)
#pragma unroll
                        for (int i = 0; i < 8; i++) c[i] = f[i] == -FLT_MAX ? f[i] : fmaxf(c[i], kLowest);
                    }
#pragma unroll
                    for (int i = 0; i < 8; i++) f[i] = c[i];
                }
                if (!VEC) {
                    const int n = count(s);
#pragma unroll
                    for (int i = 0; i < 8; i++) f[i] = i < n ? f[i] : -INFINITY;
                }
                if (put) put8(s, f);
                top[j] = fmaxf(fmaxf(fmaxf(f[0], f[1]), fmaxf(f[2], f[3])), fmaxf(fmaxf(f[4], f[5]), fmaxf(f[6], f[7])));
                if (groups) {                           // the best two, by pairs
                    float hi[4], lo[4];
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        hi[i] = fmaxf(f[2 * i], f[2 * i + 1]);
                        lo[i] = fminf(f[2 * i], f[2 * i + 1]);
                    }
#pragma unroll
                    for (int i = 0; i < 3; i++) {       // 0+1, 2+3, then both
                        const int x = i == 2 ? 0 : 2 * i, y = i == 2 ? 2 : 2 * i + 1;
                        lo[x] = fmaxf(fmaxf(lo[x], lo[y]), fminf(hi[x], hi[y]));
                        hi[x] = fmaxf(hi[x], hi[y]);
                    }
                    best_s[s] = make_float2(hi[0], lo[0]);
                }
            }
        }
    };
    if (raw) choices(std::true_type{});
    else choices(std::false_type{});
    if (groups) {
        // scores of groups l, l + LT, ...; then how many groups stand before each
        __syncwarp();
        constexpr int GL = 32 / LT;
        float score[GL];
        int before[GL];
#pragma unroll
        for (int i = 0; i < GL; i++) {
            const int grp = l + LT * i;
            float b1 = -INFINITY, b2 = -INFINITY;
            if (grp < p.n_group)
                for (int q = 0; q < p.spg.d; q++) {
                    const float2 o = best_s[grp * p.spg.d + q];
                    b2 = fmaxf(fmaxf(b2, o.y), fminf(b1, o.x));
                    b1 = fmaxf(b1, o.x);
                }
            score[i] = p.best == 1 ? b1
                       : raw       ? pair_score<SIGMOID>(b1, b2, m)
                       : b2 == -FLT_MAX ? b2
                                        : fmaxf(b1 + b2, kLowest);
            before[i] = 0;
        }
        uint32_t kept = 0;
        if (p.n_group <= LT) {                      // a group a lane
#pragma unroll
            for (int k = 0; k < LT; k++) {
                const float o = __shfl_sync(0xffffffffu, score[0], (lane & ~(LT - 1)) + k);
                if (k < p.n_group) before[0] += o > score[0] || (o == score[0] && k < l);
            }
        } else {
#pragma unroll
            for (int i = 0; i < GL; i++)
                for (int k = 0; k < LT; k++) {
                    const int other = k + LT * i;
                    const float o = __shfl_sync(0xffffffffu, score[i], (lane & ~(LT - 1)) + k);
                    if (other < p.n_group) {
#pragma unroll
                        for (int a = 0; a < GL; a++)
                            before[a] += o > score[a] || (o == score[a] && other < l + LT * a);
                    }
                }
        }
#pragma unroll
        for (int a = 0; a < GL; a++)
            if (l + LT * a < p.n_group && before[a] < p.keep) kept |= 1u << (l + LT * a);
#pragma unroll
        for (int o = LT / 2; o > 0; o >>= 1) kept |= __shfl_xor_sync(0xffffffffu, kept, o);
#pragma unroll
        for (int j = 0; j < SUB; j++) {
            const int grp = p.spg.div(l + LT * j);
            if (grp < p.n_group && !(kept >> grp & 1u)) top[j] = -INFINITY;
        }
    }

    __syncwarp();                                   // the choices, for all lanes
    const uint32_t seg = LT == 32 ? 0xffffffffu : ((1u << (LT & 31)) - 1u) << (lane & ~(LT - 1));
    for (int k = 0; k < p.K; k++) {
        float v = top[0];                           // this lane's best block, the first of equals
        int mine = 0;
#pragma unroll
        for (int j = 1; j < SUB; j++)
            if (top[j] > v) {
                v = top[j];
                mine = j;
            }
        const int s = l + LT * mine;
        const float best = lanes_max<LT>(v);
        uint32_t who = __ballot_sync(0xffffffffu, v == best) & seg;
        if (SUB > 1 && __any_sync(0xffffffffu, who & (who - 1))) {      // equal choices: the lowest block
            int low = v == best ? s : INT32_MAX;
#pragma unroll
            for (int o = LT / 2; o > 0; o >>= 1) low = min(low, __shfl_xor_sync(0xffffffffu, low, o));
            who = __ballot_sync(0xffffffffu, v == best && s == low) & seg;
        }
        // its eight lie before eight lanes: which one it was, and what is left
        const int src = __ffs(who) - 1, block = __shfl_sync(0xffffffffu, s, src), i = l & 7;
        float *mine_c = c_s + (i >> 2) * NB * 4 + block * 4 + (i & 3);
        const float c = *mine_c;
        const uint32_t eq = __ballot_sync(0xffffffffu, c == best) >> (lane & ~(LT - 1)) & 0xffu;
        const int at = __ffs(eq) - 1;
        float next = i == at ? -INFINITY : c;
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) next = fmaxf(next, __shfl_xor_sync(0xffffffffu, next, o));
        if (l == at) {
            *mine_c = -INFINITY;
            pick_s[k] = block * 8 + at;
        }
        if (lane == src) {
#pragma unroll
            for (int j = 0; j < SUB; j++)
                if (j == mine) top[j] = next;
        }
        __syncwarp();
    }

    // Renormalised weights keep their ratios where the scores themselves are
    // below fp32's numbers: softmax's are taken from the largest chosen logit
    // (the sum over the row cancels), sigmoids below e^-64 as exponentials.
    constexpr int KL = (16 + LT - 1) / LT;
    float z[KL], w[KL], sum = 0.0f, ref = -INFINITY;
    int e[KL];
#pragma unroll
    for (int i = 0; i < KL; i++) {
        const int k = l + LT * i;
        z[i] = -INFINITY;
        e[i] = 0;
        if (k < p.K) {
            e[i] = expert0(pick_s[k] >> 3) + (pick_s[k] & 7);
            z[i] = logit<X>(row, e[i]);
        }
        ref = fmaxf(ref, z[i]);
    }
    if (p.renorm) ref = lanes_max<LT>(ref);
    if (!SIGMOID && (!p.renorm || m == INFINITY)) ref = m;
    const bool soft = !SIGMOID || (p.renorm && ref < -64.0f);
#pragma unroll
    for (int i = 0; i < KL; i++) {
        w[i] = 0.0f;
        if (z[i] > -INFINITY) {                     // (otherwise the row's sum may be 0 as well)
            const float x = expf(!soft ? -z[i] : z[i] == ref ? 0.0f : z[i] - ref);   // (+inf logits share the mass)
            w[i] = __fdiv_rn(soft ? x : 1.0f, !soft ? 1.0f + x : p.renorm ? 1.0f : total);
        }
        sum += w[i];
    }
    sum = lanes_sum<LT>(sum);
#pragma unroll
    for (int i = 0; i < KL; i++) {
        const int k = l + LT * i;
        if (!live || k >= p.K) continue;
        const float v = p.renorm ? (sum > 0.0f ? __fdiv_rn(w[i], sum) : 0.0f) : w[i];
        p.idx[(size_t)t * p.K + k] = e[i];
        p.w[(size_t)t * p.K + k] = v * p.factor;
    }
}

template <typename X, bool SIGMOID, int LT, int SUB>
int launch_sub(const RouteParams &p, cudaStream_t st) {
    constexpr int TOK = kRouteThreads / LT;
    const size_t smem = (size_t)TOK * p.tok * sizeof(float);        // at most 16 tokens of 155 blocks: 107 KB
    auto kernel = p.vec ? scored_route_kernel<X, LT, SUB, SIGMOID, true> : scored_route_kernel<X, LT, SUB, SIGMOID, false>;
    if (smem > 48 * 1024) {
        static OnDevices ready[2];
        const cudaError_t e = ready[p.vec].once(
            [&] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 112 * 1024); });
        if (e != cudaSuccess) return fail(MOE_ECUDA, "scored_route_kernel: %s", cudaGetErrorString(e));
    }
    kernel<<<((uint32_t)p.T + TOK - 1) / TOK, kRouteThreads, smem, st>>>(p);
    return check_launch("scored_route_kernel");
}

template <typename X, bool SIGMOID, int LT>
int launch_lt(const RouteParams &p, cudaStream_t st) {
    const int n = (p.nsub + LT - 1) / LT;             // blocks of a lane: 5 or 20 at most (E <= 1024, 32 groups)
    if (n <= 1) return launch_sub<X, SIGMOID, LT, 1>(p, st);
    if (n <= 2) return launch_sub<X, SIGMOID, LT, 2>(p, st);
    if (n <= 4) return launch_sub<X, SIGMOID, LT, 4>(p, st);
    if constexpr (LT == 32) {
        return launch_sub<X, SIGMOID, LT, 5>(p, st);
    } else {
        if (n <= 8) return launch_sub<X, SIGMOID, LT, 8>(p, st);
        if (n <= 16) return launch_sub<X, SIGMOID, LT, 16>(p, st);
        return launch_sub<X, SIGMOID, LT, 20>(p, st);
    }
}

template <typename X, bool SIGMOID>
int launch_route(const RouteParams &p, cudaStream_t st) {
    // 32 lanes a token while that does not fill the SMs.  Measured, 32 against
    // 8 lanes (tokens x experts): 1 x 256 3.8 / 5.5 us, 1216 x 128 4.6 / 4.8,
    // 2525 x 160 6.1 / 6.8, 4096 x 512 4.4 / 6.3, but 4433 x 60 4.3 / 3.1, 9028 x
    // 64 6.1 / 3.2, 8000 x 512 7.1 / 6.7, 65521 x 256 66 / 31.
    const int most = num_sms() * (p.nsub > 16 ? 32 : 8);
    return p.T <= most ? launch_lt<X, SIGMOID, 32>(p, st) : launch_lt<X, SIGMOID, 8>(p, st);
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
    const bool groups = rd->keep_group < rd->n_group;     // all kept: as good as one group
    p.n_group = groups ? rd->n_group : 1;
    p.gs = groups ? gs : rd->E;
    p.keep = groups ? rd->keep_group : 1;
    p.spg = FastDiv((p.gs + 7) / 8);
    p.nsub = p.n_group * p.spg.d;
    p.tok = route_token_floats(p.nsub, groups);
    p.best = rd->group_best;
    p.renorm = rd->renorm != 0;
    p.vec = p.gs % 8 == 0 && stride * elt % 16 == 0 && reinterpret_cast<uintptr_t>(logits) % 16 == 0 &&
            reinterpret_cast<uintptr_t>(rd->bias) % 16 == 0;
    p.factor = rd->factor;
    p.bias = rd->bias;
    p.idx = idx;
    p.w = w;
    const bool sig = rd->score == MOE_SCORE_SIGMOID;
    if (logits_dtype == MOE_DTYPE_F32)
        return sig ? launch_route<float, true>(p, stream) : launch_route<float, false>(p, stream);
    return sig ? launch_route<__nv_bfloat16, true>(p, stream) : launch_route<__nv_bfloat16, false>(p, stream);
}
