// attend.cuh -- attention of one new token per request over a paged key-value
// cache: the kernel, templated over the head size, the cache's and the
// query's type and the number of heads that share a key head.
//
// Mathematics.  A CTA walks part of one request's tokens for all (up to 16)
// query heads of one key head, so every key and value is read once.  With
// x_i = q . k_i, c = scale log2(e) (times the key scale) and a running
// reference m near the largest c x_i, it keeps l = sum 2^(c x_i - m) and O =
// sum 2^(c x_i - m) v_i; when m grows, l and O are multiplied by 2^(m_old -
// m_new).  Parts of a row (warps of a CTA, then CTAs) join the same way: m =
// max m_j, l = sum 2^(m_j - m) l_j, O likewise; out = O / l, lse = ln 2 (m +
// log2 l).
//
// What bounds it: the cache's bytes.  Measured on one GB300, of the copy rate
// (6768 GB/s): two requests of 130977 tokens, 8 heads to a key head of 128,
// bf16 161 us (99 %); 64 ragged ones of up to 8192, 4 heads, 143 us (97 %; 151
// with an fp32 q); 96 of up to 16384 over an e4m3 cache 231 us (95 %; 234 with
// an fp32 q).  Small calls are bound by
// their launches and one chain of loads (length, table, keys), fp32 q by a
// tile's own latencies (29 windows of 1000, heads of 80: 25 us, 52 %).  A
// key or value number is used by G heads, 2 G flops for 2 bytes (bf16): far
// below the machine's balance, so the design aims at bytes in flight and few
// instructions per byte, and the products go to the tensor cores only to stay
// out of the way.  mma.sync with its 16-row tile and register operands fits
// that: a tcgen05 tile has 64 rows or more of which G would be used, and its
// accumulator would have to come out of tensor memory for every 64 tokens'
// softmax.
//
// Work split.  The unit is 64 tokens (16 for each of four warps) of one
// (request, key head): a row.  All units, in order of requests, heads and
// places, are cut into one even run per CTA of a grid that is resident at
// once, whatever the lengths: no row is too long and no batch too ragged.  A
// CTA thus holds at most two partial rows, one cut at each end; it stores
// their (O, m, l) and the join kernel adds them in order of the CTAs, so
// results do not depend on timing.  Each CTA finds its run by summing the
// lengths itself.  Short rows are not cut and need no join; where they are
// many, each warp takes rows of its own (SOLO).  One and two warps a CTA
// throughout were slower (e4m3 351 and 256 us against 244): fewer warps split
// q, and there are more parts to join.
//
// Pipeline.  Each warp streams its own 16-token tiles through a ring of NS
// stages in shared memory with 16-byte asynchronous copies and waits only for
// itself; there is no barrier until the row's end.  Rows are stored XOR-
// swizzled so that the fragment loads below touch every bank once.
//
// Fragments.  In S = Q K^T the order of the k index is free as long as both
// operands agree, so a lane's part of a key row is 16 consecutive bytes: k
// steps of 16 numbers take 4 consecutive numbers of each of the row's four
// lanes.  In O = P V the n index is free likewise: lane g's column of tile i
// is dimension 8 g + i, and a lane reads 8 consecutive numbers of its four
// token rows and pairs tokens with byte permutes.  P goes from accumulators to
// operand registers without a shuffle.
//
// Accuracy.  bf16 and e4m3 keys and values are exact operands (e4m3 as fp16).
// What is not exact is split into 16-bit parts that are summed in the fp32
// accumulator: an fp32 q into three bf16 (24 bits) or two fp16 (22 bits, after
// a power of two per row); the weights P into three bf16 with an fp32 result
// over a bf16 cache, two bf16 (16 bits) with a bf16 result, two fp16 (22 bits,
// of 2^8 times the weight so that small ones keep them) over an e4m3 cache.
// With up to 8 heads the second part rides in the tile's otherwise empty rows
// 8-15 and costs nothing; with more it is a tile of its own (64 requests, 12
// heads of 64 over e4m3: 66.9 us, 60.2 with the first part alone; heads of
// 128: no difference).
#pragma once

#include <cfloat>

#include <cuda_fp16.h>

#include "fastdiv.cuh"
#include "internal.h"

namespace moe {

constexpr int kAttWarps = 4;
constexpr int kAttTile = 16;                          // tokens of a warp's tile

constexpr int kMaxLength = INT32_MAX - 65535;         // places past the last tile stay in 32 bits

struct AttendParams {
    const uint8_t *k, *v;
    uint32_t page_stride;            // bytes
    const float *k_scale, *v_scale;
    int n_pages, Hkv, D, B;
    FastDiv page;
    int G, tiles;                    // query heads of a key head; head tiles of them
    const void *q;
    size_t q_stride, out_stride;
    int Hq;
    const int32_t *seq, *table;
    int max_blocks, window, ctas, by_row, whole;
    float scale;
    void *out;
    float *lse;
    int4 *meta;                      // rows in several parts: {parts, row, first CTA, its slot}, by row or by first CTA
    float2 *part_ml;                 // [2 ctas][rows]
    float *part_o;                   // [2 ctas][rows][DP]
};

// ---------------------------------------------------------------- pieces
__device__ __forceinline__ uint32_t smem_addr(const void *p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}

// 16 bytes from global to shared memory, or zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 lds16(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}

__device__ __forceinline__ float exp2_f(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <bool F16>
__device__ __forceinline__ void mma(float *c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                    uint32_t b0, uint32_t b1) {
    if (F16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two numbers as one 16-bit pair, and what the pair leaves of them.
template <bool F16>
__device__ __forceinline__ uint32_t pair_of(float &a, float &b) {
    uint32_t w;
    if (F16) {
        const __half2 h = __floats2half2_rn(a, b);
        const float2 f = __half22float2(h);
        a -= f.x;
        b -= f.y;
        w = *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        w = *reinterpret_cast<const uint32_t *>(&h);
        a -= __uint_as_float(w << 16);
        b -= __uint_as_float(w & 0xffff0000u);
    }
    return w;
}

// Two e4m3 (the low 16 bits) as an fp16 pair, exactly.
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t w) {
    uint32_t r;
    asm("{ .reg .b16 h; cvt.u16.u32 h, %1; cvt.rn.f16x2.e4m3x2 %0, h; }" : "=r"(r) : "r"(w));
    return r;
}

// SOLO: every warp takes rows of its own, whole ones, and no barrier joins it
// to the others.
template <int DP, bool F8, bool QF32, bool FULL, bool SOLO>
struct AttendShape {
    static constexpr int NW = SOLO ? 1 : kAttWarps;           // warps that share a row
    static constexpr int ELT = F8 ? 1 : 2;
    static constexpr int CH = DP * ELT / 16;                  // 16-byte chunks of a row
    static constexpr int NQ = QF32 ? (F8 ? 2 : 3) : 1;        // parts of q
    static constexpr int NP = QF32 && !F8 ? 3 : 2;            // parts of the weights
    static constexpr int ROWS = FULL ? 16 : 8;                // query heads of a tile
    static constexpr int NA = FULL ? NQ : (NQ + 1) / 2;       // operand tiles of q
    static constexpr int NB = FULL ? NP : (NP + 1) / 2;       // of the weights
    static constexpr int STEPS = DP / 16;
    // The weights are 2^LIFT at the reference and pass it by 2^(SLACK - LIFT)
    // at most before it follows: within fp16's 2^16 for an e4m3 cache (2^-22
    // of the reference keeps 11 bits), anywhere in bf16.
    static constexpr float LIFT = F8 ? 8.0f : 0.0f, SLACK = F8 ? 15.0f : 16.0f;
    static constexpr int TILE_B = kAttTile * DP * ELT;        // bytes of a tile's keys
    static constexpr int STAGE = TILE_B + (CH == 12 ? kAttTile * 13 * 16 : TILE_B);
    static constexpr bool HALF_UNIT = DP % 64 != 0;           // the last 32 dimensions are half a unit of values
    // Stages and CTAs per SM, of the shared memory (192 KB of stages) and the
    // registers.  More CTAs hide a tile's own latencies better, more stages
    // the memory's: with an fp32 q in up to 8 rows (more products a tile)
    // three CTAs of two stages beat two of three (29 windows of 1000: 39
    // against 44 us; 64 ragged bf16 requests: 153 against 152).
    static constexpr bool BUSY = QF32 && !FULL;
    static constexpr int NS = SOLO ? 2
                              : F8 ? (DP == 64 ? 8 : DP == 128 ? 4 : 3)
                                   : (DP == 96 || DP == 128 ? (BUSY ? 2 : 3) : DP == 256 ? 3 : 4);
    static constexpr int CTAS = F8 ? (DP == 256 ? 2 : 3) : (DP == 64 ? 3 : DP <= 128 ? (BUSY ? 3 : 2) : 1);
    static constexpr int UNIT = kAttTile * NW;
    static constexpr int RING = NS * STAGE;                   // of one warp
    static constexpr bool HALF = !FULL && NQ == 1;            // operand rows 8-15 of q are zero and not stored
    static constexpr int Q_B = NA * STEPS * (HALF ? 256 : 512);
    static constexpr int LDO = DP + 4;                        // floats of a row of O in the join of the warps
    static constexpr int SMEM = kAttWarps * RING + kAttWarps / NW * Q_B;
    static_assert(SOLO || ROWS * LDO * 4 <= RING, "a warp's O fits its ring");
};

// Chunk c of row r of a tile: keys are read by 8 rows x 4 neighbouring
// chunks, values by rows 2t x 8-byte or 16-byte chunks g.
template <int CH>
__device__ __forceinline__ uint32_t key_at(int r, int c) {
    return CH % 8 == 0 ? (uint32_t)(r * CH + (c ^ ((r & 1) << 2))) * 16 : (uint32_t)(r * CH + c) * 16;
}
template <int CH>
__device__ __forceinline__ uint32_t value_at(int r, int c) {
    if (CH % 8 == 0) return (uint32_t)(r * CH + (c ^ (r & 6))) * 16;
    if (CH == 12) return (uint32_t)(r * 13 + c) * 16;         // an odd stride does the same
    const int pos = (r >> 1) | (r & 1) << 3;                  // rows of 64 bytes: even rows first
    return (uint32_t)(pos * CH + (c ^ (pos & 2))) * 16;
}

template <int UNIT>
__device__ __forceinline__ int units_of(int len, int window, int room) {
    len = min(len, room);
    if (len <= 0) return 0;
    const int lo = window > 0 && len > window ? (len - window) & ~(kAttTile - 1) : 0;
    return (len - lo + UNIT - 1) / UNIT;
}

// A row's weight in the even runs: its units, and what it costs to begin one
// (q, the first table entries and keys, the join of the warps: about as much
// as two units).  The first kBegin places of a row are no units.  Without
// them a CTA could be given a dozen rows of one token: 29 windows of 1000
// took 34 us instead of 25 for one request of length 1 among them.
constexpr int kBegin = 2;
__device__ __forceinline__ int weight_of(int units) { return units > 0 ? units + kBegin : 0; }

// Quotient of a 64-bit number that nearly always fits 32 bits.
__device__ __forceinline__ int64_t quotient(int64_t a, int b) {
    return a >> 31 ? a / b : (int64_t)((int)a / b);
}

template <bool QF32>
__device__ __forceinline__ void store4(void *out, size_t i, float4 f) {
    if (QF32) {
        *reinterpret_cast<float4 *>(static_cast<float *>(out) + i) = f;
    } else {
        const __nv_bfloat162 a = __floats2bfloat162_rn(f.x, f.y), b = __floats2bfloat162_rn(f.z, f.w);
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(out) + i) =
            make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    }
}

// ---------------------------------------------------------------- kernel
template <int DP, bool F8, bool QF32, bool FULL, bool ALIGNED, bool SOLO>
__global__ void __launch_bounds__(32 * kAttWarps, (AttendShape<DP, F8, QF32, FULL, SOLO>::CTAS))
    attend_kernel(const AttendParams p) {
    using S = AttendShape<DP, F8, QF32, FULL, SOLO>;
    constexpr int NW = S::NW, CH = S::CH, NS = S::NS, ROWS = S::ROWS, R = FULL ? 2 : 1, UNIT = S::UNIT;
    constexpr int THREADS = 32 * kAttWarps, TEAMS = kAttWarps / NW;       // a team: the warps of a row
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t sm_sum[kAttWarps];
    __shared__ int sm_top[kAttWarps];
    __shared__ int64_t sm_off[TEAMS], sm_W, sm_end;
    __shared__ int sm_b[TEAMS], sm_bad;
    __shared__ float sm_c[TEAMS][16];
    __shared__ float2 sm_ml[kAttWarps][16];
    const int tid = threadIdx.x, lane = tid & 31, wrp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int team = wrp / NW, warp = wrp % NW, cta = blockIdx.x * TEAMS + team, HT = p.Hkv * p.tiles;
    auto sync = [] {
        if (SOLO) __syncwarp();
        else __syncthreads();
    };
    const int room = (int)min((int64_t)p.max_blocks * p.page.d, (int64_t)kMaxLength);
    asm volatile("griddepcontrol.launch_dependents;");   // the join may take the SMs as they empty
    uint8_t *ring = smem + wrp * S::RING;
    const uint32_t ring_a = smem_addr(ring);
    uint8_t *q_s = smem + kAttWarps * S::RING + team * S::Q_B;

    // where this CTA's run begins
    const int run = (p.B + THREADS - 1) / THREADS;
    const int b0 = min(p.B, tid * run), b1 = min(p.B, b0 + run);
    int64_t sum = 0;
    int top_w = 0;
    for (int b = b0; b < b1; b++) {
        const int w = weight_of(units_of<UNIT>(p.seq[b], p.window, room));
        sum += w;
        top_w = max(top_w, w);
    }
    top_w = __reduce_max_sync(0xffffffffu, top_w);
    int64_t before = sum;
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += u;
    }
    if (lane == 31) {
        sm_sum[wrp] = before;
        sm_top[wrp] = top_w;
    }
    before -= sum;
    for (int i = tid; i < TEAMS * S::Q_B / 16; i += THREADS)
        reinterpret_cast<uint4 *>(smem + kAttWarps * S::RING)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    int64_t W = 0;
#pragma unroll
    for (int w = 0; w < kAttWarps; w++) {
        if (w == wrp) before += W;
        W += sm_sum[w];
        top_w = max(top_w, sm_top[w]);
    }
    W *= HT;
    // a unit for each team while that makes at most 64 parts of a row, then four
    const int n_cta = (int)min((int64_t)p.ctas * TEAMS, max(W / 4, min(W, (int64_t)p.B * HT * 64)));
    if (tid == 0 && !p.by_row && !p.whole) p.meta[cta] = make_int4(0, 0, 0, 0);
    // Rows are not cut either where the lengths turn out to give each CTA one
    // row or less and the longest is little more than an even run: a CTA's two
    // parts and the join cost six units' time (32 requests of 1000 tokens, 8
    // key heads: 29 us cut).
    bool whole_rows = p.whole;
    if (!SOLO && !p.whole && n_cta > 0) {
        const int64_t each = quotient(W, n_cta);
        whole_rows = each <= top_w && top_w <= each + 6;
    }
#pragma unroll
    for (int k = 0; k < TEAMS; k++) {          // a thread in whose requests a team's run begins says so
        const int c = blockIdx.x * TEAMS + k;
        if (c >= n_cta) continue;
        const int64_t u = quotient(c * W, n_cta);
        if (u >= before * HT && u < (before + sum) * HT) {
            int64_t at = before;
            int b = b0;
            for (;; b++) {
                const int n = weight_of(units_of<UNIT>(p.seq[b], p.window, room));
                if (u < (at + n) * HT) break;
                at += n;
            }
            sm_b[k] = b;
            sm_off[k] = u - at * HT;
        }
    }
    if (tid == 0) sm_W = W;                    // (for a cut row's last CTA; not kept in registers meanwhile)
    __syncthreads();

    const bool busy = cta < n_cta;
    const int64_t u0 = busy ? quotient(cta * W, n_cta) : 0, u1 = busy ? quotient((cta + 1) * W, n_cta) : 0;
    int b = busy ? sm_b[team] : 0;
    int64_t off = busy ? sm_off[team] : 0;
    bool first_seg = true;
    for (int64_t u = u0; u < u1;) {
        const int full_len = p.seq[b];
        const int nb = units_of<UNIT>(full_len, p.window, room);
        const int nw = weight_of(nb);
        if (off >= (int64_t)nw * HT) {
            off = 0;
            b++;
            continue;
        }
        const int ht = (int)quotient(off, nw), from = (int)(off - (int64_t)ht * nw);
        if (whole_rows && from > 0) {             // the row belongs to the CTA that its first place fell to
            off += nw - from;
            u += nw - from;
            continue;
        }
        const int n_place = whole_rows ? nw : (int)min((int64_t)(nw - from), u1 - u);
        const int blk = max(0, from - kBegin), n_unit = max(0, from + n_place - kBegin) - blk;
        const int64_t row_end = u - from + nw;
        u += n_place;
        off += n_place;
        if (n_unit == 0) continue;             // the row's units are the next CTA's
        const int h = ht / p.tiles, head0 = h * p.G + (ht - h * p.tiles) * ROWS;
        const int n_rows = min(ROWS, (h + 1) * p.G - head0);
        const int len = min(full_len, room);
        const int lo = p.window > 0 ? max(0, len - p.window) : 0;
        const int tile0 = (lo & ~(kAttTile - 1)) + blk * UNIT;      // this segment's first token
        const int stop = min(len, tile0 + n_unit * UNIT);
        const int n_tile = (stop - tile0 + kAttTile - 1) / kAttTile;
        const int mine = n_tile > warp ? (n_tile - warp + NW - 1) / NW : 0;
        if (!SOLO && tid == 0) {
            sm_bad = full_len > room;
            sm_end = row_end;
        }

        // ---- q: the numbers are loaded before the first tiles are asked for, and split after
        constexpr int QR = ROWS / NW, IT = (DP / 4 + 31) / 32;
        uint4 qx[QR][IT];
#pragma unroll
        for (int k = 0; k < QR; k++)
#pragma unroll
            for (int i = 0; i < IT; i++) {
                const int r = warp + NW * k, d = 4 * (lane + 32 * i);
                qx[k][i] = make_uint4(0, 0, 0, 0);
                if (d < p.D && r < n_rows) {
                    const size_t at = (size_t)b * p.q_stride + (size_t)(head0 + r) * p.D + d;
                    if (QF32) {
                        qx[k][i] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const float *>(p.q) + at));
                    } else {
                        const uint2 f = __ldg(reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(p.q) + at));
                        qx[k][i] = make_uint4(f.x << 16, f.x & 0xffff0000u, f.y << 16, f.y & 0xffff0000u);
                    }
                }
            }
        const float c0 = p.scale * 1.44269504088896341f * (F8 && p.k_scale ? __ldg(p.k_scale + h) : 1.0f);

        // ---- the warp's tiles
        const int row_b = p.D * S::ELT;                            // bytes of a stored row
        const uint8_t *k_h = p.k + (size_t)h * p.page.d * row_b, *v_h = p.v + (size_t)h * p.page.d * row_b;
        const int32_t *tab = p.table + (size_t)b * p.max_blocks;
        int ids = 0, ids8 = 0;          // ALIGNED: the pages of 32 tiles; else of rows lane / 4 and 8 more of the next tile
        bool bad = false;
        auto page_of = [&](int tok) { return tok < stop ? __ldg(tab + p.page.div(tok)) : -1; };
        auto fetch_ids = [&](int i) {   // before tile i is issued
            if (ALIGNED) {
                if ((i & 31) == 0) ids = page_of(tile0 + (warp + NW * (i + lane)) * kAttTile);
            } else {
                const int tok = tile0 + (warp + NW * i) * kAttTile + g;
                ids = page_of(tok);
                ids8 = page_of(tok + 8);
            }
        };
        uint32_t fill = ring_a, read = ring_a;                     // the stages to write and to read next
        auto next = [&](uint32_t &at) { at = at == ring_a + (NS - 1) * S::STAGE ? ring_a : at + S::STAGE; };
        auto issue = [&](int i) {
            if (i < mine) {
                const int tok0 = tile0 + (warp + NW * i) * kAttTile;
                const uint32_t dst = fill;
                next(fill);
                if (ALIGNED) {          // one page: whole rows, row after row
                    const int id = __shfl_sync(0xffffffffu, ids, i & 31);
                    const bool ok0 = (unsigned)id < (unsigned)p.n_pages;
                    const int in = tok0 - p.page.div(tok0) * p.page.d;
                    bad |= !ok0;
                    fetch_ids(i + 1);
                    const uint64_t at0 = (uint64_t)(uint32_t)(ok0 ? id : 0) * p.page_stride + (uint32_t)(in * row_b);
                    const uint8_t *k0 = k_h + at0, *v0 = v_h + at0;
                    if (ok0 && tok0 >= lo && tok0 + kAttTile <= stop && row_b == CH * 16) {
#pragma unroll
                        for (int n = 0; n < CH * kAttTile / 32; n++) {
                            const int e = n * 32 + lane, r = e / CH, ch = e - r * CH;
                            copy16(dst + key_at<CH>(r, ch), k0 + e * 16);
                            copy16(dst + S::TILE_B + value_at<CH>(r, ch), v0 + e * 16);
                        }
                    } else {
#pragma unroll
                        for (int n = 0; n < CH * kAttTile / 32; n++) {
                            const int e = n * 32 + lane, r = e / CH, ch = e - r * CH, tok = tok0 + r;
                            const bool ok = ok0 && tok >= lo && tok < stop && ch * 16 < row_b;
                            const int at = ok ? r * row_b + ch * 16 : 0;
                            copy16(dst + key_at<CH>(r, ch), ok ? k0 + at : p.k, ok);
                            copy16(dst + S::TILE_B + value_at<CH>(r, ch), ok ? v0 + at : p.v, ok);
                        }
                    }
                } else {                // a page per row: four lanes a row, two rows a lane
#pragma unroll
                    for (int hf = 0; hf < 2; hf++) {
                        const int r = g + 8 * hf, tok = tok0 + r, id = hf ? ids8 : ids;
                        const bool in_page = (unsigned)id < (unsigned)p.n_pages, seen = tok >= lo && tok < stop;
                        const bool ok0 = in_page && seen;
                        bad |= seen && !in_page;
                        const int in = tok - p.page.div(tok) * p.page.d;
                        const uint64_t at0 = (uint64_t)(uint32_t)(ok0 ? id : 0) * p.page_stride + (uint32_t)(in * row_b);
                        const uint8_t *k0 = k_h + at0, *v0 = v_h + at0;
#pragma unroll
                        for (int n = 0; n < CH / 4; n++) {
                            const int ch = 4 * n + t;
                            const bool ok = ok0 && ch * 16 < row_b;
                            const int at = ch * 16 < row_b ? ch * 16 : 0;
                            copy16(dst + key_at<CH>(r, ch), k0 + at, ok);
                            copy16(dst + S::TILE_B + value_at<CH>(r, ch), v0 + at, ok);
                        }
                    }
                    fetch_ids(i + 1);
                }
            }
            copy_commit();
        };
        fetch_ids(0);
#pragma unroll
        for (int i = 0; i < NS - 1; i++) issue(i);
        // ---- q, split into parts in the order of the operand's registers
#pragma unroll
        for (int k = 0; k < QR; k++) {
            const int r = warp + NW * k;
            float top = 0.0f;
            if (F8) {
#pragma unroll
                for (int i = 0; i < IT; i++)
                    top = fmaxf(fmaxf(fmaxf(top, fabsf(__uint_as_float(qx[k][i].x))), fabsf(__uint_as_float(qx[k][i].y))),
                                fmaxf(fabsf(__uint_as_float(qx[k][i].z)), fabsf(__uint_as_float(qx[k][i].w))));
            }
            float f = c0 < 0.0f ? -1.0f : 1.0f, c = fabsf(c0);
            if (F8) {                     // fp16 parts: the row's largest number to 2^13 .. 2^14
                for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                const int e = max(27, (int)(__float_as_uint(top) >> 23));       // biased exponent
                if (top > 0.0f && e < 255) {
                    f *= __uint_as_float((uint32_t)(127 + 13 + 127 - e) << 23);
                    c *= __uint_as_float((uint32_t)max(1, e - 13) << 23);
                }
            }
            if (c < FLT_MIN) c = FLT_MIN;     // a scale of 0: alike weights, and no 0 times a masked -inf
            if (lane == 0) sm_c[team][r] = c;
#pragma unroll
            for (int i = 0; i < IT; i++) {
                const int d = 4 * (lane + 32 * i);
                if (d >= DP) break;
                const int per = F8 ? 16 : 8;                       // numbers of a lane in a unit of the row
                const int step = d / (4 * per) * (per / 4) + d % per / 4, tt = d / per % 4;
                float x[4] = {__uint_as_float(qx[k][i].x) * f, __uint_as_float(qx[k][i].y) * f,
                              __uint_as_float(qx[k][i].z) * f, __uint_as_float(qx[k][i].w) * f};
#pragma unroll
                for (int part = 0; part < S::NQ; part++) {
                    const int na = FULL ? part : part / 2, up = FULL ? r >> 3 : part & 1;
                    constexpr int W = S::HALF ? 2 : 4;            // words of a lane
                    uint32_t *w = reinterpret_cast<uint32_t *>(q_s) + ((na * S::STEPS + step) * 32 + (r & 7) * 4 + tt) * W;
                    w[up] = pair_of<F8>(x[0], x[1]);
                    w[W / 2 + up] = pair_of<F8>(x[2], x[3]);
                }
            }
        }
        sync();
        float c[R], m[R], l[R];
#pragma unroll
        for (int r = 0; r < R; r++) {
            c[r] = sm_c[team][g + 8 * r];
            m[r] = -INFINITY;
            l[r] = 0.0f;
        }
        float o[DP / 8][4];
#pragma unroll
        for (int i = 0; i < DP / 8; i++) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;

        for (int i = 0; i < mine; i++) {
            __syncwarp();
            issue(i + NS - 1);
            copy_wait<NS - 1>();
            __syncwarp();
            const uint32_t ks = read, vs = ks + S::TILE_B;
            next(read);
            const int tok0 = tile0 + (warp + NW * i) * kAttTile;

            float sp[2][2][4] = {};                 // two chains of products for each 8 tokens
#pragma unroll
            for (int un = 0; un < CH / 4; un++) {
                const uint4 k0 = lds16(ks + key_at<CH>(g, 4 * un + t));
                const uint4 k1 = lds16(ks + key_at<CH>(g + 8, 4 * un + t));
                const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
                for (int j = 0; j < (F8 ? 4 : 2); j++) {
                    const int step = un * (F8 ? 4 : 2) + j;
                    uint32_t x0, x1, y0, y1;
                    if (F8) {
                        x0 = e4m3_pair(w0[j]), x1 = e4m3_pair(w0[j] >> 16);
                        y0 = e4m3_pair(w1[j]), y1 = e4m3_pair(w1[j] >> 16);
                    } else {
                        x0 = w0[2 * j], x1 = w0[2 * j + 1];
                        y0 = w1[2 * j], y1 = w1[2 * j + 1];
                    }
#pragma unroll
                    for (int na = 0; na < S::NA; na++) {
                        float(*s)[4] = sp[(step + na) & 1];
                        if (S::HALF) {
                            const uint2 a = reinterpret_cast<const uint2 *>(q_s)[(na * S::STEPS + step) * 32 + lane];
                            mma<F8>(s[0], a.x, 0u, a.y, 0u, x0, x1);
                            mma<F8>(s[1], a.x, 0u, a.y, 0u, y0, y1);
                        } else {
                            const uint4 a = reinterpret_cast<const uint4 *>(q_s)[(na * S::STEPS + step) * 32 + lane];
                            mma<F8>(s[0], a.x, a.y, a.z, a.w, x0, x1);
                            mma<F8>(s[1], a.x, a.y, a.z, a.w, y0, y1);
                        }
                    }
                }
            }
            float s[2][4];
#pragma unroll
            for (int n = 0; n < 2; n++)
#pragma unroll
                for (int j = 0; j < 4; j++) s[n][j] = sp[0][n][j] + sp[1][n][j];
            // x[r][4]: tokens 2t, 2t+1, 2t+8, 2t+9 of head g (and g + 8)
            float x[R][4];
#pragma unroll
            for (int n = 0; n < 2; n++)
#pragma unroll
                for (int j = 0; j < 2; j++) {
                    if (FULL) {
                        x[0][2 * n + j] = s[n][j];
                        x[R - 1][2 * n + j] = s[n][2 + j];
                    } else {
                        x[0][2 * n + j] = S::NQ > 1 ? s[n][j] + s[n][2 + j] : s[n][j];
                    }
                }
            if (tok0 < lo || tok0 + kAttTile > stop) {
#pragma unroll
                for (int n = 0; n < 4; n++) {
                    const int tok = tok0 + (n >> 1) * 8 + 2 * t + (n & 1);
                    if (tok < lo || tok >= stop) {
#pragma unroll
                        for (int r = 0; r < R; r++) x[r][n] = -INFINITY;
                    }
                }
            }
            // The reference need not be the maximum: it follows only when a
            // score passes it by 2^SLACK, so most tiles take no maximum over
            // the row's lanes and scale nothing.
            bool over = false;
#pragma unroll
            for (int r = 0; r < R; r++) {
                const float top = fmaxf(fmaxf(x[r][0], x[r][1]), fmaxf(x[r][2], x[r][3]));
                over |= fmaf(top, c[r], -m[r]) > S::SLACK;         // (the first tile: m is -inf)
            }
            if (__any_sync(0xffffffffu, over)) {
                float f[R];
#pragma unroll
                for (int r = 0; r < R; r++) {
                    float top = fmaxf(fmaxf(x[r][0], x[r][1]), fmaxf(x[r][2], x[r][3]));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    const float mn = fmaxf(m[r], top * c[r] - S::LIFT);
                    f[r] = mn > m[r] ? exp2_f(m[r] - mn) : 1.0f;
                    m[r] = mn;
                    l[r] *= f[r];
                }
#pragma unroll
                for (int i2 = 0; i2 < DP / 8; i2++) {
                    o[i2][0] *= f[0];
                    o[i2][1] *= f[0];
                    o[i2][2] *= f[R - 1];
                    o[i2][3] *= f[R - 1];
                }
            }
#pragma unroll
            for (int r = 0; r < R; r++) {
                const float ref = m[r] == -INFINITY ? 0.0f : m[r];
#pragma unroll
                for (int n = 0; n < 4; n++) x[r][n] = exp2_f(fmaf(x[r][n], c[r], -ref));
                l[r] += (x[r][0] + x[r][1]) + (x[r][2] + x[r][3]);
            }
            // the weights as operand tiles
            uint32_t a[S::NB][4];
#pragma unroll
            for (int nb2 = 0; nb2 < S::NB; nb2++) a[nb2][1] = a[nb2][3] = 0u;
#pragma unroll
            for (int r = 0; r < R; r++)
#pragma unroll
                for (int part = 0; part < S::NP; part++) {
                    const int to = FULL ? part : part / 2, up = FULL ? r : part & 1;
                    a[to][up] = pair_of<F8>(x[r][0], x[r][1]);
                    a[to][2 + up] = pair_of<F8>(x[r][2], x[r][3]);
                }
#pragma unroll
            for (int un = 0; un < DP / 64; un++) {
                uint32_t v[2][8];                   // operand registers of the 8 tiles of 8 dimensions
                if (F8) {
                    const int ch = 4 * un + (g >> 1), in = (g & 1) * 8;
                    uint2 w[4];
#pragma unroll
                    for (int j = 0; j < 4; j++)
                        w[j] = lds8(vs + value_at<CH>(2 * t + (j & 1) + (j >> 1) * 8, ch) + in);
#pragma unroll
                    for (int hf = 0; hf < 2; hf++)
#pragma unroll
                        for (int q4 = 0; q4 < 2; q4++) {
                            const uint32_t e = q4 ? w[2 * hf].y : w[2 * hf].x;
                            const uint32_t d = q4 ? w[2 * hf + 1].y : w[2 * hf + 1].x;
                            const uint32_t lo2 = __byte_perm(e, d, 0x5140), hi2 = __byte_perm(e, d, 0x7362);
                            v[hf][4 * q4] = e4m3_pair(lo2);
                            v[hf][4 * q4 + 1] = e4m3_pair(lo2 >> 16);
                            v[hf][4 * q4 + 2] = e4m3_pair(hi2);
                            v[hf][4 * q4 + 3] = e4m3_pair(hi2 >> 16);
                        }
                } else {
#pragma unroll
                    for (int hf = 0; hf < 2; hf++) {
                        const uint4 e = lds16(vs + value_at<CH>(2 * t + 8 * hf, 8 * un + g));
                        const uint4 d = lds16(vs + value_at<CH>(2 * t + 1 + 8 * hf, 8 * un + g));
                        const uint32_t ew[4] = {e.x, e.y, e.z, e.w}, dw[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
                        for (int j = 0; j < 4; j++) {
                            v[hf][2 * j] = __byte_perm(ew[j], dw[j], 0x5410);
                            v[hf][2 * j + 1] = __byte_perm(ew[j], dw[j], 0x7632);
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < 8; j++)
#pragma unroll
                    for (int nb2 = 0; nb2 < S::NB; nb2++)
                        mma<F8>(o[un * 8 + j], a[nb2][0], a[nb2][1], a[nb2][2], a[nb2][3], v[0][j], v[1][j]);
            }
            if (S::HALF_UNIT) {                     // 4 numbers a lane: tile i's column g is dimension 4 g + i of these 32
                uint32_t v[2][4];
#pragma unroll
                for (int hf = 0; hf < 2; hf++) {
                    const int ch = DP / 64 * 8 + (g >> 1), in = (g & 1) * 8;
                    const uint2 e = lds8(vs + value_at<CH>(2 * t + 8 * hf, ch) + in);
                    const uint2 d = lds8(vs + value_at<CH>(2 * t + 1 + 8 * hf, ch) + in);
                    v[hf][0] = __byte_perm(e.x, d.x, 0x5410);
                    v[hf][1] = __byte_perm(e.x, d.x, 0x7632);
                    v[hf][2] = __byte_perm(e.y, d.y, 0x5410);
                    v[hf][3] = __byte_perm(e.y, d.y, 0x7632);
                }
#pragma unroll
                for (int j = 0; j < 4; j++)
#pragma unroll
                    for (int nb2 = 0; nb2 < S::NB; nb2++)
                        mma<F8>(o[DP / 64 * 8 + j], a[nb2][0], a[nb2][1], a[nb2][2], a[nb2][3], v[0][j], v[1][j]);
            }
        }
        copy_wait<0>();
        __syncwarp();

        const float v_scale = F8 && p.v_scale ? p.v_scale[h] : 1.0f;
        if (SOLO) {                     // ---- the warp's row, out of its registers
            bad = __any_sync(0xffffffffu, bad) || full_len > room;
#pragma unroll
            for (int r = 0; r < R; r++) {
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
                if (bad) l[r] = NAN;
                const int row = g + 8 * r;
                if (row >= n_rows) continue;
                const float inv = v_scale / l[r];
                const size_t at = (size_t)b * p.out_stride + (size_t)(head0 + row) * p.D;
#pragma unroll
                for (int un = 0; un < DP / 64; un++)
#pragma unroll
                    for (int hf = 0; hf < 2; hf++) {
                        const int d = un * 64 + 16 * t + 8 * hf;
                        if (d >= p.D) continue;
                        float w[8];
#pragma unroll
                        for (int j = 0; j < 8; j++) {
                            const float *e = o[un * 8 + j];
                            w[j] = (FULL ? e[2 * r + hf] : e[hf] + e[2 + hf]) * inv;
                        }
                        store4<QF32>(p.out, at + d, make_float4(w[0], w[1], w[2], w[3]));
                        store4<QF32>(p.out, at + d + 4, make_float4(w[4], w[5], w[6], w[7]));
                    }
                if (S::HALF_UNIT) {
#pragma unroll
                    for (int hf = 0; hf < 2; hf++) {
                        const int d = DP / 64 * 64 + 8 * t + 4 * hf;
                        if (d >= p.D) continue;
                        float w[4];
#pragma unroll
                        for (int j = 0; j < 4; j++) {
                            const float *e = o[DP / 64 * 8 + j];
                            w[j] = (FULL ? e[2 * r + hf] : e[hf] + e[2 + hf]) * inv;
                        }
                        store4<QF32>(p.out, at + d, make_float4(w[0], w[1], w[2], w[3]));
                    }
                }
                if (t == 0 && p.lse) p.lse[(size_t)b * p.Hq + head0 + row] = 0.69314718055994531f * (m[r] + log2f(l[r]));
            }
            __syncwarp();
            continue;
        }
        // ---- the warps' parts of the row
        if (bad) sm_bad = 1;
        float *o_s = reinterpret_cast<float *>(ring);
#pragma unroll
        for (int r = 0; r < R; r++) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
            if (t == 0) sm_ml[warp][g + 8 * r] = make_float2(m[r], l[r]);
#pragma unroll
            for (int un = 0; un < DP / 64; un++)
#pragma unroll
                for (int hf = 0; hf < 2; hf++)
#pragma unroll
                    for (int q4 = 0; q4 < 2; q4++) {
                        float4 w;
                        float *wf = &w.x;
#pragma unroll
                        for (int j = 0; j < 4; j++) {
                            const float *e = o[un * 8 + 4 * q4 + j];
                            wf[j] = FULL ? e[2 * r + hf] : e[hf] + e[2 + hf];
                        }
                        *reinterpret_cast<float4 *>(o_s + (g + 8 * r) * S::LDO + un * 64 + 16 * t + 8 * hf + 4 * q4) = w;
                    }
            if (S::HALF_UNIT) {
#pragma unroll
                for (int hf = 0; hf < 2; hf++) {
                    float4 w;
                    float *wf = &w.x;
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const float *e = o[DP / 64 * 8 + j];
                        wf[j] = FULL ? e[2 * r + hf] : e[hf] + e[2 + hf];
                    }
                    *reinterpret_cast<float4 *>(o_s + (g + 8 * r) * S::LDO + DP / 64 * 64 + 8 * t + 4 * hf) = w;
                }
            }
        }
        __syncthreads();
        const bool whole = n_unit == nb;
        const int slot = 2 * cta + (first_seg ? 0 : 1);
        for (int i = tid; i < n_rows * (DP / 4); i += THREADS) {
            const int r = i / (DP / 4), d = (i - r * (DP / 4)) * 4;
            float M = -INFINITY, L = 0.0f;
#pragma unroll
            for (int w = 0; w < NW; w++) M = fmaxf(M, sm_ml[w][r].x);
            const float ref = M == -INFINITY ? 0.0f : M;
            float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int w = 0; w < NW; w++) {
                const float2 ml = sm_ml[w][r];
                const float fw = exp2_f(ml.x - ref);
                const float4 e = *reinterpret_cast<const float4 *>(
                    reinterpret_cast<const float *>(smem + w * S::RING) + r * S::LDO + d);
                L = fmaf(fw, ml.y, L);
                acc.x = fmaf(fw, e.x, acc.x);
                acc.y = fmaf(fw, e.y, acc.y);
                acc.z = fmaf(fw, e.z, acc.z);
                acc.w = fmaf(fw, e.w, acc.w);
            }
            if (sm_bad) L = NAN;
            if (whole) {
                const float inv = v_scale / L;
                if (d < p.D)
                    store4<QF32>(p.out, (size_t)b * p.out_stride + (size_t)(head0 + r) * p.D + d,
                                 make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
                if (d == 0 && p.lse) p.lse[(size_t)b * p.Hq + head0 + r] = 0.69314718055994531f * (M + log2f(L));
            } else {
                *reinterpret_cast<float4 *>(p.part_o + ((size_t)slot * ROWS + r) * DP + d) = acc;
                if (d == 0) p.part_ml[(size_t)slot * ROWS + r] = make_float2(M, L);
            }
        }
        if (tid == 0 && blk == 0 && n_unit < nb) {
            const int c1 = (int)((sm_end * n_cta - 1) / sm_W);     // the CTA of the row's last unit
            p.meta[p.by_row ? b * HT + ht : cta] = make_int4(c1 - cta + 1, b * HT + ht, cta, slot);
        } else if (tid == 0 && blk == 0 && p.by_row && !p.whole) {
            p.meta[b * HT + ht] = make_int4(0, 0, 0, 0);
        }
        __syncthreads();
        first_seg = false;
    }

    // rows with nothing to see
    for (int e = blockIdx.x; e < p.B; e += gridDim.x) {
        if (units_of<UNIT>(p.seq[e], p.window, room) > 0) continue;
        for (int i = tid; i < p.Hq * p.D / 4; i += THREADS)
            store4<QF32>(p.out, (size_t)e * p.out_stride + 4 * (size_t)i, make_float4(0.0f, 0.0f, 0.0f, 0.0f));
        if (p.lse)
            for (int i = tid; i < p.Hq; i += THREADS) p.lse[(size_t)e * p.Hq + i] = -INFINITY;
        if (p.by_row && !p.whole)
            for (int i = tid; i < HT; i += THREADS) p.meta[e * HT + i] = make_int4(0, 0, 0, 0);
    }
}

// Joins a row's parts: JW warps for each (row in several parts, head), HB
// heads a CTA.  Warp w of a head takes every JW-th part, its lanes four
// dimensions each (and four more past 128).  Many rows have few parts each,
// and a warp for each head is enough; few rows have many.
template <bool QF32, int JW, int HB>
__global__ void __launch_bounds__(32 * JW * HB) attend_join_kernel(const AttendParams p, int dp, int rows) {
    __shared__ float4 acc_s[JW > 1 ? JW * HB : 1][64];
    __shared__ float2 ml_s[JW * HB];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4 meta = p.meta[blockIdx.x];
    const int n = meta.x, HT = p.Hkv * p.tiles, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = blockIdx.y * HB + warp / JW, w = warp % JW;
    if (n == 0) return;
    const int b = meta.y / HT, ht = meta.y - b * HT, h = ht / p.tiles, head = h * p.G + (ht - h * p.tiles) * rows + r;
    const bool live = r < rows && head < (h + 1) * p.G;
    const int q = dp / 4;                             // float4s of a row: 16 .. 64
    auto slot = [&](int j) { return (j == 0 ? (size_t)meta.w : 2 * ((size_t)meta.z + j)) * rows + r; };
    float M = -INFINITY, L = 0.0f;
    float4 acc[2] = {make_float4(0, 0, 0, 0), make_float4(0, 0, 0, 0)};
    for (int j0 = w; live && j0 < n; j0 += 32 * JW) { // 32 parts of this warp: their (m, l), one a lane
        const int jl = j0 + JW * lane;
        const float2 ml = jl < n ? p.part_ml[slot(jl)] : make_float2(-INFINITY, 0.0f);
        float top = ml.x;
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float Mn = fmaxf(M, top), ref = Mn == -INFINITY ? 0.0f : Mn;
        const float old = exp2_f(M - ref), f = exp2_f(ml.x - ref);
        M = Mn;
        L = fmaf(L, old, warp_sum(f * ml.y, 32));
#pragma unroll
        for (int i = 0; i < 2; i++) acc[i].x *= old, acc[i].y *= old, acc[i].z *= old, acc[i].w *= old;
        const int m = min(32, (n - j0 + JW - 1) / JW);
#pragma unroll 8
        for (int i = 0; i < m; i++) {
            const float fi = __shfl_sync(0xffffffffu, f, i);
            const float *o = p.part_o + slot(j0 + JW * i) * dp;
#pragma unroll
            for (int c = 0; c < 2; c++) {
                if (lane + 32 * c < q) {
                    const float4 e = __ldcg(reinterpret_cast<const float4 *>(o) + lane + 32 * c);
                    acc[c].x = fmaf(fi, e.x, acc[c].x);
                    acc[c].y = fmaf(fi, e.y, acc[c].y);
                    acc[c].z = fmaf(fi, e.z, acc[c].z);
                    acc[c].w = fmaf(fi, e.w, acc[c].w);
                }
            }
        }
    }
    if (JW > 1) {                                     // the warps' sums, by the head's first warp
        acc_s[warp][lane] = acc[0];
        acc_s[warp][lane + 32] = acc[1];
        if (lane == 0) ml_s[warp] = make_float2(M, L);
        __syncthreads();
        if (w != 0) return;
        for (int k = 1; k < JW; k++) M = fmaxf(M, ml_s[warp + k].x);
        const float ref = M == -INFINITY ? 0.0f : M;
        acc[0] = acc[1] = make_float4(0, 0, 0, 0);
        L = 0.0f;
        for (int k = 0; k < JW; k++) {
            const float f = exp2_f(ml_s[warp + k].x - ref);
            L = fmaf(f, ml_s[warp + k].y, L);
#pragma unroll
            for (int c = 0; c < 2; c++) {
                const float4 e = acc_s[warp + k][lane + 32 * c];
                acc[c].x = fmaf(f, e.x, acc[c].x);
                acc[c].y = fmaf(f, e.y, acc[c].y);
                acc[c].z = fmaf(f, e.z, acc[c].z);
                acc[c].w = fmaf(f, e.w, acc[c].w);
            }
        }
    }
    if (!live) return;
    const float inv = (p.v_scale ? p.v_scale[h] : 1.0f) / L;
#pragma unroll
    for (int c = 0; c < 2; c++) {
        const int d = 4 * (lane + 32 * c);
        if (d < p.D)
            store4<QF32>(p.out, (size_t)b * p.out_stride + (size_t)head * p.D + d,
                         make_float4(acc[c].x * inv, acc[c].y * inv, acc[c].z * inv, acc[c].w * inv));
    }
    if (lane == 0 && p.lse) p.lse[(size_t)b * p.Hq + head] = 0.69314718055994531f * (M + log2f(L));
}

// ---------------------------------------------------------------- launch
template <int DP, bool F8, bool QF32, bool FULL, bool ALIGNED, bool SOLO>
int launch_attend_rows(const AttendParams &p, cudaStream_t st) {
    using S = AttendShape<DP, F8, QF32, FULL, SOLO>;
    auto kernel = attend_kernel<DP, F8, QF32, FULL, ALIGNED, SOLO>;
    static OnDevices ready;
    cudaError_t e = ready.once([&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
    });
    if (e == cudaSuccess) {
        kernel<<<p.ctas, 32 * kAttWarps, S::SMEM, st>>>(p);
        e = cudaGetLastError();
    }
    if (e != cudaSuccess) return fail(MOE_ECUDA, "attend_kernel: %s", cudaGetErrorString(e));
    return MOE_OK;
}

template <int DP, bool F8, bool QF32, bool FULL, bool ALIGNED>
int launch_attend_kernel(AttendParams p, cudaStream_t st) {
    using S = AttendShape<DP, F8, QF32, FULL, false>;
    p.ctas = num_sms() * S::CTAS;
    const int64_t rows = (int64_t)p.B * p.Hkv * p.tiles;
    p.by_row = rows <= p.ctas;
    // Rows that are short by the table's width and the window are not cut: a
    // CTA takes those that begin in its run.  That saves the join and its
    // launch (about five units' time), and costs what the run is uneven by: up
    // to four units always, up to eight where the CTAs have rows enough (32
    // requests of up to 500 tokens, 8 key heads: 10.5 us against 12.5).  Where
    // there are many rows, each warp takes rows of its own: a row costs about
    // as much as four tiles of it before its first product, which is then paid
    // for four rows at once (199 requests of up to 3 tokens, heads of 192: 14
    // us against 27).
    const int64_t room = (int64_t)p.max_blocks * p.page.d;
    const int64_t seen = (int64_t)p.window + kAttTile, longest = p.window > 0 && seen < room ? seen : room;
    const int64_t units = (longest + S::UNIT - 1) / S::UNIT, rounds = (rows + p.ctas - 1) / p.ctas;
    p.whole = units <= 4 || (units <= 8 && rounds * (units + kBegin) <= rows * (units + kBegin) / p.ctas + 5);
    if (p.whole) {
        const int64_t tile = (longest + kAttTile - 1) / kAttTile;
        const int64_t shared = rounds * (4 + units);
        const int64_t solo = (rows + 4 * p.ctas - 1) / (4 * p.ctas) * (4 + tile);
        return solo < shared ? launch_attend_rows<DP, F8, QF32, FULL, ALIGNED, true>(p, st)
                             : launch_attend_rows<DP, F8, QF32, FULL, ALIGNED, false>(p, st);
    }
    if (int rc = launch_attend_rows<DP, F8, QF32, FULL, ALIGNED, false>(p, st)) return rc;
    const int64_t parts = p.ctas / rows;              // of a row, when the lengths are alike
    const int heads = min(S::ROWS, p.G), hb = parts > 32 ? 1 : parts > 4 ? 2 : 8;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(p.by_row ? rows : p.ctas), (unsigned)((heads + hb - 1) / hb));
    cfg.blockDim = dim3(parts > 32 ? 512 : 256);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const cudaError_t e =
        parts > 32  ? cudaLaunchKernelEx(&cfg, attend_join_kernel<QF32, 16, 1>, p, DP, (int)S::ROWS)
        : parts > 4 ? cudaLaunchKernelEx(&cfg, attend_join_kernel<QF32, 4, 2>, p, DP, (int)S::ROWS)
                    : cudaLaunchKernelEx(&cfg, attend_join_kernel<QF32, 1, 8>, p, DP, (int)S::ROWS);
    if (e != cudaSuccess) return fail(MOE_ECUDA, "attend_join_kernel: %s", cudaGetErrorString(e));
    return MOE_OK;
}

// Padded head size, tile rows and most CTAs per SM of a shape; the workspace goes by them.
struct AttendPlan {
    int dp, rows, ctas_per_sm;
};
inline AttendPlan attend_plan(int D, bool f8, int G) {
    AttendPlan a;
    a.dp = D <= 64 ? 64 : D <= 96 && !f8 ? 96 : D <= 128 ? 128 : D <= 192 && !f8 ? 192 : 256;
    a.rows = G > 8 ? 16 : 8;
    a.ctas_per_sm = f8 ? (a.dp == 256 ? 2 : 3) : (a.dp <= 128 ? 3 : 1);
    return a;
}

template <bool F8, bool QF32, int DP>
int launch_attend_dp(const AttendParams &p, cudaStream_t st) {
    const bool full = p.G > 8, aligned = p.page.d % kAttTile == 0;
    if (full) return aligned ? launch_attend_kernel<DP, F8, QF32, true, true>(p, st)
                             : launch_attend_kernel<DP, F8, QF32, true, false>(p, st);
    return aligned ? launch_attend_kernel<DP, F8, QF32, false, true>(p, st)
                   : launch_attend_kernel<DP, F8, QF32, false, false>(p, st);
}

int launch_attend_bf16_qf32(const AttendParams &p, int dp, cudaStream_t st);
int launch_attend_bf16_qbf16(const AttendParams &p, int dp, cudaStream_t st);
int launch_attend_e4m3_qf32(const AttendParams &p, int dp, cudaStream_t st);
int launch_attend_e4m3_qbf16(const AttendParams &p, int dp, cudaStream_t st);

}  // namespace moe
