// rotary.cu -- rotary embedding: pairs (a, b) of a head's numbers turned by
// place * frequency,  a' = m (a cos - b sin),  b' = m (b cos + a sin).
//
// The angle.  A frequency is kept as the 64 bits behind the point of its turns
// a place, F = 2^64 freq / (2 pi): place * F modulo 2^64 is the angle in turns
// without what is whole, exact but for F's own rounding (a place of 2^20 times
// 2^-53 of a turn), at any distance and for negative places too.  Its top two
// bits, rounded, are the quarter; what is left is within 1/8 of a turn, where
// fp32 holds it to 2^-24 of itself.  No reduction of a large argument is left.
//
// Bytes bound it where there are many tokens: 16381 tokens of 40 heads of 128
// take 53 us from bf16 to bf16, 93 % of the copy rate, 8000 in fp32 50 us, 96 %.
// A token's cosines and sines are made once for all its heads.  Heads whose
// parts are no multiples of 16 bytes go number by number (4000 tokens of 16 heads of
// 80 of which 20 turn: 18 us, 17 %), and with few heads of 256 the table is a
// large part of a CTA's work (4000 tokens of 18: 25 us, 43 %).
#include <algorithm>
#include <cmath>

#include "e4m3.cuh"
#include "fastdiv.cuh"
#include "internal.h"
#include "rows.h"

namespace moe {

namespace {

constexpr int kMaxHead = 1024;

struct TableParams {
    int rot, scaling, trained;
    double base, factor, low, high;
};

__global__ void rotary_table_kernel(const TableParams p, uint64_t *turns) {
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= p.rot / 2) return;
    const double two_pi = 6.283185307179586476925;
    double base = p.base;
    if (p.scaling == MOE_ROTARY_BASE && p.rot > 2) base *= pow(p.factor, (double)p.rot / (p.rot - 2));
    double f = pow(base, -2.0 * i / p.rot);
    if (p.scaling == MOE_ROTARY_LINEAR) {
        f /= p.factor;
    } else if (p.scaling == MOE_ROTARY_YARN) {
        // from the pair that turns `high` times within the trained length to
        // the one that turns `low` times, the frequency goes over to its factor-th part
        const double by = p.rot / (2.0 * log(p.base));
        const double from = fmax(floor(by * log(p.trained / (p.high * two_pi))), 0.0);
        const double to = fmin(ceil(by * log(p.trained / (p.low * two_pi))), p.rot - 1.0);
        const double ramp = fmin(1.0, fmax(0.0, (i - from) / fmax(to - from, 0.001)));
        f = f * (1.0 - ramp) + f / p.factor * ramp;
    } else if (p.scaling == MOE_ROTARY_BANDS) {
        const double keep = fmin(1.0, fmax(0.0, (p.trained * f / two_pi - p.low) / (p.high - p.low)));
        f = f * keep + f / p.factor * (1.0 - keep);
    }
    const double t = f / two_pi;
    turns[i] = (uint64_t)((t - floor(t)) * 0x1p64);
}

// Cosine and sine of place * F, times m.
__device__ __forceinline__ float2 turned(int32_t place, uint64_t F, float m) {
    const uint64_t turn = (uint64_t)(int64_t)place * F;
    const uint32_t quarter = (uint32_t)((turn + ((uint64_t)1 << 61)) >> 62);
    const int64_t rest = (int64_t)(turn - ((uint64_t)quarter << 62));        // -2^61 .. 2^61 - 1
    float s, c;
    sincospif(__ll2float_rn(rest) * 0x1p-63f, &s, &c);
    float cc = quarter & 1 ? s : c, ss = quarter & 1 ? c : s;
    if (quarter == 1 || quarter == 2) cc = -cc;
    if (quarter >= 2) ss = -ss;
    return make_float2(m * cc, m * ss);
}

// One product rounded, the other within the sum, in every variant.
__device__ __forceinline__ void turn(float &a, float &b, float2 w) {
    const float u = a, v = b;
    a = fmaf(u, w.x, -__fmul_rn(v, w.y));
    b = fmaf(v, w.x, __fmul_rn(u, w.y));
}

struct Operand {
    const void *x;
    void *out;
    size_t x_stride, out_stride;         // elements between tokens
};

struct RotaryParams {
    Operand q, k;
    const uint64_t *turns;
    const int32_t *places;
    int T, Hq, D, rot, first, tokens;    // tokens of a CTA
    int turning;                         // chunks of a head that turn; the others are copied
    float m;
    FastDiv per_token, per_head;         // chunks of a token's heads, of a head
    FastDiv pairs;
};

template <typename X, int V>
struct Chunk {                           // V numbers: 16 bytes, or one number
    float f[V];
};
template <typename X, int V>
__device__ __forceinline__ Chunk<X, V> chunk_load(const X *at) {
    Chunk<X, V> c;
    if constexpr (V == 1) {
        c.f[0] = (float)*at;
    } else if constexpr (sizeof(X) == 4) {
        const float4 v = *reinterpret_cast<const float4 *>(at);
        c.f[0] = v.x, c.f[1] = v.y, c.f[2] = v.z, c.f[3] = v.w;
    } else {
        const uint4 raw = *reinterpret_cast<const uint4 *>(at);
        const Floats8 f = floats8<X>(&raw);
#pragma unroll
        for (int j = 0; j < V; j++) c.f[j] = f.x[j];
    }
    return c;
}
template <typename X, int V>
__device__ __forceinline__ void chunk_store(X *at, const Chunk<X, V> &c) {
    if constexpr (V == 1) {
        *at = (X)c.f[0];
    } else if constexpr (sizeof(X) == 4) {
        *reinterpret_cast<float4 *>(at) = make_float4(c.f[0], c.f[1], c.f[2], c.f[3]);
    } else {
        *reinterpret_cast<uint4 *>(at) = bf16x8(c.f);
    }
}

// A CTA takes `tokens` tokens: their cosines and sines into shared memory, a
// pair a thread, then all heads' chunks.  HALF: an item is V pairs (i, i +
// rot / 2), two chunks of V numbers; else V numbers of V / 2 neighbouring
// pairs (two numbers where V = 1).
template <typename X, int V, bool HALF>
__global__ void __launch_bounds__(256) rotary_kernel(const RotaryParams p) {
    extern __shared__ float2 table[];                 // [tokens][rot / 2]
    constexpr int W = !HALF && V == 1 ? 2 : V;        // numbers of a turning item's first chunk
    const int t0 = blockIdx.x * p.tokens, nt = min(p.tokens, p.T - t0), pairs = p.rot / 2;
    for (int i = threadIdx.x; i < nt * pairs; i += blockDim.x) {
        const int t = p.pairs.div(i);
        table[i] = turned(__ldg(p.places + t0 + t), __ldg(p.turns + i - t * pairs), p.m);
    }
    __syncthreads();
    const int n = nt * p.per_token.d;
    for (int it = threadIdx.x; it < n; it += blockDim.x) {
        const int t = p.per_token.div(it), in = it - t * p.per_token.d;
        const int head = p.per_head.div(in);
        int c = in - head * p.per_head.d;
        const bool is_q = head < p.Hq;
        const Operand &o = is_q ? p.q : p.k;
        const size_t at = (size_t)(is_q ? head : head - p.Hq) * p.D;
        const X *x = static_cast<const X *>(o.x) + (size_t)(t0 + t) * o.x_stride + at;
        X *out = static_cast<X *>(o.out) + (size_t)(t0 + t) * o.out_stride + at;
        if (c >= p.turning) {                         // the numbers in front of the part and behind it
            c = (c - p.turning) * V;
            if (c >= p.first) c += p.rot;
            if constexpr (V == 1) out[c] = x[c];
            else *reinterpret_cast<uint4 *>(out + c) = *reinterpret_cast<const uint4 *>(x + c);
            continue;
        }
        const float2 *cs = table + t * pairs;
        if constexpr (HALF) {
            const int i = c * V;
            Chunk<X, V> a = chunk_load<X, V>(x + p.first + i), b = chunk_load<X, V>(x + p.first + pairs + i);
#pragma unroll
            for (int j = 0; j < V; j++) {
                const float2 w = cs[i + j];
                turn(a.f[j], b.f[j], w);
            }
            chunk_store<X, V>(out + p.first + i, a);
            chunk_store<X, V>(out + p.first + pairs + i, b);
        } else {
            const int i = c * W;
            Chunk<X, W> a;
            if constexpr (V == 1) {
                a.f[0] = (float)x[p.first + i];
                a.f[1] = (float)x[p.first + i + 1];
            } else {
                a = chunk_load<X, W>(x + p.first + i);
            }
#pragma unroll
            for (int j = 0; j < W; j += 2) {
                const float2 w = cs[(i + j) / 2];
                turn(a.f[j], a.f[j + 1], w);
            }
            if constexpr (V == 1) {
                out[p.first + i] = (X)a.f[0];
                out[p.first + i + 1] = (X)a.f[1];
            } else {
                chunk_store<X, W>(out + p.first + i, a);
            }
        }
    }
}

template <typename X, int V>
int launch_rotary(const RotaryParams &p, bool half, cudaStream_t st) {
    const unsigned grid = (unsigned)((p.T + (int64_t)p.tokens - 1) / p.tokens);
    const size_t smem = (size_t)p.tokens * (p.rot / 2) * sizeof(float2);
    if (half) rotary_kernel<X, V, true><<<grid, 256, smem, st>>>(p);
    else rotary_kernel<X, V, false><<<grid, 256, smem, st>>>(p);
    return check_launch("rotary_kernel");
}

int check_rotary(const moe_rotary_desc *rd, const char *who) {
    if (rd == nullptr) return fail(MOE_EINVAL, "%s: descriptor is NULL", who);
    if (rd->D < 2 || rd->D > kMaxHead || rd->rot < 2 || rd->rot % 2 || rd->first < 0 || rd->rot > rd->D || rd->first > rd->D - rd->rot)
        return fail(MOE_EINVAL, "%s: D=%d rot=%d first=%d (D up to %d, rot even, the part inside the head)", who, rd->D, rd->rot, rd->first,
                    kMaxHead);
    if (rd->layout != MOE_ROTARY_HALF && rd->layout != MOE_ROTARY_INTERLEAVED) return fail(MOE_EINVAL, "%s: layout=%d", who, rd->layout);
    if (!(std::fabs(rd->amplitude) < INFINITY)) return fail(MOE_EINVAL, "%s: amplitude=%g", who, (double)rd->amplitude);
    return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_rotary_table(const moe_rotary_desc *rd, uint64_t *turns, cudaStream_t stream) {
    const char *who = "rotary_table";
    if (int rc = check_rotary(rd, who)) return rc;
    if (rd->scaling < MOE_ROTARY_PLAIN || rd->scaling > MOE_ROTARY_BANDS) return fail(MOE_EINVAL, "%s: scaling=%d", who, rd->scaling);
    if (!(rd->base > 1.0) || !(rd->base < INFINITY)) return fail(MOE_EINVAL, "%s: base=%g (above 1)", who, rd->base);
    if (rd->scaling != MOE_ROTARY_PLAIN && (!(rd->factor >= 1.0) || !(rd->factor <= 1e6)))
        return fail(MOE_EINVAL, "%s: factor=%g (1 to 10^6)", who, rd->factor);
    if ((rd->scaling == MOE_ROTARY_YARN || rd->scaling == MOE_ROTARY_BANDS) &&
        (rd->trained < 1 || !(rd->low > 0.0) || !(rd->high > rd->low) || !(rd->high < INFINITY)))
        return fail(MOE_EINVAL, "%s: trained=%d low=%g high=%g (0 < low < high)", who, rd->trained, rd->low, rd->high);
    if (!turns || off(turns, 8)) return fail(MOE_EINVAL, "%s: NULL or misaligned turns", who);
    const TableParams p{rd->rot, rd->scaling, rd->trained, rd->base, rd->factor, rd->low, rd->high};
    rotary_table_kernel<<<(rd->rot / 2 + 63) / 64, 64, 0, stream>>>(p, turns);
    return check_launch("rotary_table_kernel");
}

extern "C" int moe_rotary(const moe_rotary_desc *rd, const uint64_t *turns, const int32_t *places, int T, int dtype, const void *q,
                          size_t q_stride, int Hq, void *q_out, size_t q_out_stride, const void *k, size_t k_stride, int Hk, void *k_out,
                          size_t k_out_stride, cudaStream_t stream) {
    const char *who = "rotary";
    if (int rc = check_rotary(rd, who)) return rc;
    if (T < 0 || Hq < 0 || Hk < 0 || Hq > 65536 || Hk > 65536) return fail(MOE_EINVAL, "%s: T=%d Hq=%d Hk=%d", who, T, Hq, Hk);
    if (dtype != MOE_DTYPE_F32 && dtype != MOE_DTYPE_BF16) return fail(MOE_EINVAL, "%s: dtype=%d", who, dtype);
    if (T == 0 || Hq + Hk == 0) return MOE_OK;
    if (!turns || off(turns, 8) || !places || off(places, 4)) return fail(MOE_EINVAL, "%s: NULL or misaligned turns/places", who);
    const size_t e = dtype == MOE_DTYPE_F32 ? 4 : 2, n = (size_t)T, D = (size_t)rd->D;
    const Rows in[] = {{"q", Hq ? q : nullptr, n, Hq * D * e, q_stride * e}, {"k", Hk ? k : nullptr, n, Hk * D * e, k_stride * e},
                       {"turns", turns, 1, (size_t)rd->rot * 4, 0}, {"places", places, 1, n * 4, 0}};
    const Rows out[] = {{"q_out", Hq ? q_out : nullptr, n, Hq * D * e, q_out_stride * e},
                        {"k_out", Hk ? k_out : nullptr, n, Hk * D * e, k_out_stride * e}};
    for (int i = 0; i < 2; i++)
        for (const Rows *r : {&in[i], &out[i]}) {
            if (r->width == 0) continue;
            if (!r->at || off(r->at, e)) return fail(MOE_EINVAL, "%s: NULL or misaligned %s", who, r->name);
            if (n > 1 && (r->stride < r->width || r->stride > (SIZE_MAX >> 1) / n))
                return fail(MOE_EINVAL, "%s: tokens of %s %zu bytes apart (need >= %zu)", who, r->name, r->stride, r->width);
        }
    for (int o = 0; o < 2; o++) {
        for (int i = 0; i < 4; i++)
            if (out[o].overlaps(in[i]) && !(i == o && out[o].same(in[i])))
                return fail(MOE_EINVAL, "%s: %s overlaps %s", who, out[o].name, in[i].name);
        if (o && out[1].overlaps(out[0])) return fail(MOE_EINVAL, "%s: k_out overlaps q_out", who);
    }
    // 16-byte chunks where every chunk of the part and of its two sides is whole
    // and on its boundary; else single numbers (pairs).
    const bool half = rd->layout == MOE_ROTARY_HALF;
    const int vec = (int)(16 / e);
    bool wide = rd->D % vec == 0 && rd->first % vec == 0 && (half ? rd->rot / 2 : rd->rot) % vec == 0;
    for (int i = 0; i < 2; i++)
        for (const Rows *r : {&in[i], &out[i]})
            if (r->width) wide = wide && !off(r->at, 16) && (n <= 1 || r->stride % 16 == 0);
    const int V = wide ? vec : 1;
    const bool in_place = (!Hq || out[0].same(in[0])) && (!Hk || out[1].same(in[1]));
    const int turning = half ? rd->rot / 2 / V : V == 1 ? rd->rot / 2 : rd->rot / V;
    const int per_head = turning + (in_place ? 0 : (rd->D - rd->rot) / V);
    const int64_t per_token = (int64_t)(Hq + Hk) * per_head;
    // Tokens of a CTA: some 1024 items, four a thread (16381 tokens of 40 heads of 128 take 53 us,
    // with 512 items 59, with 2048 57), its table within 16 KB, and a CTA for each SM first.
    int tokens = (int)std::max<int64_t>(1, std::min<int64_t>(1024 / per_token, 2048 / (rd->rot / 2)));
    tokens = (int)std::max<int64_t>(1, std::min<int64_t>(tokens, (T + (int64_t)num_sms() - 1) / num_sms()));
    const RotaryParams p{{q, q_out, q_stride, q_out_stride}, {k, k_out, k_stride, k_out_stride}, turns, places, T, Hq, rd->D, rd->rot, rd->first,
                         tokens, turning, rd->amplitude, FastDiv((int)per_token), FastDiv(per_head), FastDiv(rd->rot / 2)};
    if (dtype == MOE_DTYPE_F32) return wide ? launch_rotary<float, 4>(p, half, stream) : launch_rotary<float, 1>(p, half, stream);
    return wide ? launch_rotary<__nv_bfloat16, 8>(p, half, stream) : launch_rotary<__nv_bfloat16, 1>(p, half, stream);
}
