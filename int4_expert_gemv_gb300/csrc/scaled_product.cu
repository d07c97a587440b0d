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

struct ProductParams {
    const float *sx, *sw;
    size_t sx_stride, sw_stride, out_stride;     // elements
    int T, N, KB;
    void *out;
    int32_t *err;
    uint32_t polls;                              // of a wait, at most
    int stall;
    int nt, split, stages;                       // tokens of a tile, CTAs of a cluster, stages of the ring
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

// Waits for the phase of `bar` with `parity`.  Both kinds count polls, and
// where those run out they write MOE_ETIMEOUT.
//
// The threads that issue copies and MMAs sleep between polls: a spinning one
// takes issue slots from the sums' warps (8190 x 5120 x 4096: 136 us with the
// sleep, 143 without; 157 with the hardware's own suspended wait, which wakes late).
struct Bound {
    uint32_t polls;
    int32_t *err;
};
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, const Bound &b) {
#pragma unroll 1
    for (uint32_t i = b.polls; i; i--) {
        if (pipe::mbar_try_wait(bar, parity)) return true;
        __nanosleep(32);
    }
    atomicExch(b.err, MOE_ETIMEOUT);
    return false;
}

// Those that multiply and add go on with what there is when their polls, counted over the
// whole kernel, have run out (the results are invalid then): with a way out of the
// loop over the blocks the MMAs' issue is no longer uniform code to the compiler, and
// 8190 x 5120 x 4096 takes 181 us instead of 136.
template <bool SLEEP>
__device__ __forceinline__ void wait_on(uint64_t *bar, uint32_t parity, int &left) {
#pragma unroll 1
    while (!pipe::mbar_try_wait(bar, parity)) {
        if (--left <= 0) break;
        if (SLEEP) __nanosleep(32);
    }
}

// Polls of a whole kernel of n blocks: a wait's, and what waits take that are in time.
__device__ __forceinline__ int all_polls(uint32_t polls, int n) {
    return (int)min((uint64_t)polls * 2 + (uint64_t)n * 4, (uint64_t)INT32_MAX);
}

// A place in a ring of n, and the parity of the phase that its next turn is
// waited for with.
struct Ring {
    int at = 0;
    uint32_t turn = 0;
    __device__ __forceinline__ void next(int n) {
        if (++at == n) at = 0, turn ^= 1;
    }
};

// One lane of a warp that runs together.  The tensor cores' and TMA's
// instructions take uniform registers, and the compiler keeps what such a lane
// computes there: four MMAs, their two commits and a wait take 190 clocks to
// issue, and 335 behind a test of the lane's number.
__device__ __forceinline__ bool elected() {
    uint32_t one;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(one));
    return one != 0;
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
// The weights are the 128 rows of the MMA and the tokens its `nt` columns, so
// that a tile of weights is read once, for a token as for 64.  A cluster of
// `split` CTAs shares a tile's blocks of K and joins the sums through
// distributed shared memory, in the order of its CTAs.
constexpr int kFewMaxStages = 12;
constexpr int kFewScales = 64;           // blocks whose scales stand in shared memory at a time
template <int MAXN>
struct Few {
    static constexpr int kSumWarps = MAXN >= 64 ? 8 : 4;            // four a half of the columns, or of all
    static constexpr int kCols = MAXN / (kSumWarps / 4);            // columns of a thread, at most
    static constexpr int kSlots = 4;                                // accumulators
    static constexpr int kTmem = kSlots * MAXN;                     // TMEM columns: 64 to 256
    static constexpr int kThreads = 32 * (kSumWarps + 2);           // and a warp for TMA, one for the MMAs
};

// Blocks of a CTA, at most.
__host__ __device__ inline int few_share(int KB, int split) { return (KB + split - 1) / split; }
__host__ __device__ inline int few_scales(int KB, int split) { return min(few_share(KB, split), kFewScales); }
__host__ __device__ inline int few_stage(int nt) { return 128 * 128 + nt * 128; }

template <int MAXN>
size_t few_smem(int KB, int split, int stages, int nt) {
    return 1024 + (size_t)stages * few_stage(nt) + (size_t)few_scales(KB, split) * MAXN * 4 + (2 * kFewMaxStages + 2 * Few<MAXN>::kSlots + 2) * 8 + 16;
}

template <int MAXN, typename O>
__global__ void __launch_bounds__(Few<MAXN>::kThreads) few_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                                                                  const ProductParams p) {
    using F = Few<MAXN>;
    extern __shared__ __align__(1024) uint8_t smdyn[];
    uint8_t *stages = smdyn + ((1024u - (saddr(smdyn) & 1023u)) & 1023u);
    const int NT = p.nt, stage_bytes = few_stage(NT), S = p.split;
    float *scales = reinterpret_cast<float *>(stages + (size_t)p.stages * stage_bytes);         // [blocks][MAXN]
    uint64_t *full = reinterpret_cast<uint64_t *>(scales + few_scales(p.KB, S) * MAXN);
    uint64_t *empty = full + kFewMaxStages, *acc_full = empty + kFewMaxStages, *acc_empty = acc_full + F::kSlots;
    uint64_t *stall_bar = acc_empty + F::kSlots, *drain_bar = stall_bar + 1;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(drain_bar + 1);
    const Bound bound{p.polls, p.err};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tile = blockIdx.x / S, rank = blockIdx.x - tile * S, t0 = 0;
    const int kb0 = (int)((int64_t)p.KB * rank / S), nkb = (int)((int64_t)p.KB * (rank + 1) / S) - kb0;
    const int fills = min(nkb, p.stages);
    if (warp == F::kSumWarps) {
        // The first fills at once, a lane for each copy, before the CTA has come
        // together: the barriers that they tell are this warp's own work.
        if (lane < p.stages) {
            mbar_init(full + lane, 1);
            mbar_init(empty + lane, 1);
        }
        if (lane < F::kSlots) {
            mbar_init(acc_full + lane, 1);
            mbar_init(acc_empty + lane, F::kSumWarps);
        }
        if (lane == 0) {
            mbar_init(stall_bar, 1);
            mbar_init(drain_bar, 1);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane < 2 * fills) {
            const int q = lane >> 1;
            uint8_t *stage = stages + (size_t)q * stage_bytes;
            if (lane & 1) {
                pipe::tma_2d(stage + 128 * 128, &xmap, (kb0 + q) * 128, t0, full + q);
            } else {
                mbar_expect_tx(full + q, stage_bytes);
                pipe::tma_2d(stage, &wmap, (kb0 + q) * 128, tile * 128, full + q);
            }
        }
    }
    if (warp == F::kSumWarps + 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(tmem_holder)), "n"(F::kTmem) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;

    if (warp == F::kSumWarps) {
        int q = fills;
        if (elected()) {
            Ring r;
            for (; q < nkb; q++, r.next(p.stages)) {
                uint8_t *stage = stages + (size_t)r.at * stage_bytes;
                if (!wait(empty + r.at, r.turn, bound)) break;
                mbar_expect_tx(full + r.at, stage_bytes);
                pipe::tma_2d(stage, &wmap, (kb0 + q) * 128, tile * 128, full + r.at);
                pipe::tma_2d(stage + 128 * 128, &xmap, (kb0 + q) * 128, t0, full + r.at);
            }
        }
        q = __reduce_max_sync(0xffffffffu, (unsigned)q);
        // the last fill of each stage lands before the CTA exits
        for (int s = 0; s < p.stages && s < q; s++) {
            const int last = q - 1 - ((q - 1 - s) % p.stages);
            wait(full + s, (last / p.stages) & 1, bound);
        }
    } else if (warp == F::kSumWarps + 1) {
        const uint32_t idesc = idesc_e4m3(128, NT);
        if (elected()) {
            int left = all_polls(p.polls, nkb);
            Ring r;
            for (int q = 0; q < nkb; q++, r.next(p.stages)) {
                const int k = q % F::kSlots;
                wait_on<true>(full + r.at, r.turn, left);
                if (q >= F::kSlots) wait_on<true>(acc_empty + k, ((q / F::kSlots) - 1) & 1, left);
                tc_fence_after();
                const uint32_t at = saddr(stages + (size_t)r.at * stage_bytes);
                const uint64_t a = sw128_desc(at), b = sw128_desc(at + 128 * 128);
#pragma unroll
                for (int kk = 0; kk < 4; kk++)                       // 32 bytes of K each
                    mma_e4m3<1>(tmem + k * MAXN, a + 2 * kk, b + 2 * kk, idesc, kk > 0);
                umma::umma_commit(acc_full + k);
                if (q + p.stages < nkb) umma::umma_commit(empty + r.at);         // (nothing waits for the last ones)
            }
            umma::umma_commit(drain_bar);
            if (left <= 0) atomicExch(p.err, MOE_ETIMEOUT);
        }
        __syncwarp();
        wait(drain_bar, 0, bound);           // what has been issued ends before the memory goes
    } else {
        const int tid = threadIdx.x, row = tid & 127;
        if (p.stall && blockIdx.x == 0 && warp == 0) {        // test hook: bytes that no copy sends
            if (lane == 0) mbar_expect_tx(stall_bar, 16);
            __syncwarp();
            wait(stall_bar, 0, bound);
        }
        // this warp's columns: from c0, nc of them (a multiple of 16)
        const int half = F::kSumWarps == 8 ? (NT / 16 + 1) / 2 * 16 : NT;
        const int c0 = F::kSumWarps == 8 && warp >= 4 ? half : 0, nc = min(half, NT - c0);
        constexpr int NC = F::kCols < 32 ? 16 : 32;
        float acc[F::kCols];
#pragma unroll
        for (int j = 0; j < F::kCols; j++) acc[j] = 0.0f;
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16) + c0;
        int left = all_polls(p.polls, nkb);
        for (int q = 0; q < nkb; q++) {
            const int k = q % F::kSlots;
            if (q % kFewScales == 0) {
                // the products of the next blocks' scales (the first while the tiles are on their way)
                if (q) asm volatile("bar.sync 1, %0;" ::"n"(F::kSumWarps * 32) : "memory");
                const int all = min(nkb - q, kFewScales) * MAXN;
                for (int i0 = tid; i0 < all; i0 += 8 * F::kSumWarps * 32) {
                    float x[8], w[8];
#pragma unroll
                    for (int u = 0; u < 8; u++) {
                        const int i = i0 + u * F::kSumWarps * 32, b = kb0 + q + i / MAXN, j = i % MAXN;
                        const bool in = i < all && j < NT && t0 + j < p.T;
                        x[u] = in ? __ldg(p.sx + (size_t)(t0 + j) * p.sx_stride + b) : 0.0f;
                        w[u] = in ? __ldg(p.sw + (size_t)tile * p.sw_stride + b) : 0.0f;
                    }
#pragma unroll
                    for (int u = 0; u < 8; u++)
                        if (i0 + u * F::kSumWarps * 32 < all) scales[i0 + u * F::kSumWarps * 32] = x[u] * w[u];
                }
                asm volatile("bar.sync 1, %0;" ::"n"(F::kSumWarps * 32) : "memory");
            }
            wait_on<false>(acc_full + k, (q / F::kSlots) & 1, left);
            __syncwarp();
            tc_fence_after();
            const float4 *sc = reinterpret_cast<const float4 *>(scales + q % kFewScales * MAXN + c0);
#pragma unroll
            for (int c = 0; c < F::kCols; c += NC) {
                if (c >= nc) break;
                uint32_t d[NC];
                tmem_ld<NC>(lanes + k * MAXN + c, d);
#pragma unroll
                for (int j = 0; j < NC; j += 4) {
                    const float4 f = sc[(c + j) / 4];
                    acc[c + j] = fmaf(f.x, __uint_as_float(d[j]), acc[c + j]);
                    acc[c + j + 1] = fmaf(f.y, __uint_as_float(d[j + 1]), acc[c + j + 1]);
                    acc[c + j + 2] = fmaf(f.z, __uint_as_float(d[j + 2]), acc[c + j + 2]);
                    acc[c + j + 3] = fmaf(f.w, __uint_as_float(d[j + 3]), acc[c + j + 3]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(acc_empty + k);
        }
        if (left <= 0) atomicExch(p.err, MOE_ETIMEOUT);
        const int n = tile * 128 + row, have = min(nc, p.T - t0 - c0);
        if (S == 1) {
            O *out = static_cast<O *>(p.out) + (size_t)(t0 + c0) * p.out_stride + n;
            if (n < p.N) {
#pragma unroll
                for (int j = 0; j < F::kCols; j++)
                    if (j < have) put(out + (size_t)j * p.out_stride, acc[j]);
            }
        } else if (__all_sync(0xffffffffu, left > 0)) {
            // over the ring, all of whose copies and products are done: [token][row]
            float *part = reinterpret_cast<float *>(stages) + c0 * 128 + row;
#pragma unroll
            for (int j = 0; j < F::kCols; j++)
                if (j < have) part[j * 128] = acc[j];
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == F::kSumWarps + 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(F::kTmem) : "memory");
    }
    if (S > 1) {
        cluster_sync();
        // four rows of a token a thread, in turn among the cluster's threads (a row a
        // thread, one load after the other, took half of a call of 256 tokens)
        const uint32_t base = saddr(stages);
        const int items = min(NT, p.T - t0) * 32;
        for (int i = rank * F::kThreads + threadIdx.x; i < items; i += S * F::kThreads) {
            const int j = i >> 5, n = tile * 128 + (i & 31) * 4;
            float4 v[8];
#pragma unroll
            for (int r = 0; r < 8; r++)
                if (r < S)
                    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v[r].x), "=f"(v[r].y), "=f"(v[r].z), "=f"(v[r].w) : "r"(mapped(base + i * 16, r)) : "memory");
            float sum[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
            for (int r = 1; r < 8; r++)
                if (r < S) sum[0] += v[r].x, sum[1] += v[r].y, sum[2] += v[r].z, sum[3] += v[r].w;
            O *out = static_cast<O *>(p.out) + (size_t)(t0 + j) * p.out_stride + n;
#pragma unroll
            for (int u = 0; u < 4; u++)
                if (n + u < p.N) put(out + u, sum[u]);
        }
        cluster_sync();                  // no CTA's memory goes while another reads it
    }
}

// ---------------------------------------------------------------- many tokens
// A pair of CTAs computes 256 tokens x 256 outputs (or 192, or 128): the tokens
// are the rows of cta_group::2 MMAs (128 in each CTA's TMEM), so that a token's
// scale belongs to a thread and a weight's to a whole warp, and each CTA brings
// the tiles of its 128 tokens and of half of the outputs (a CTA of its own would
// have to bring both halves: 48 KB a block of K instead of 32).  Two
// accumulators of 256 columns fill TMEM, each in two halves that are multiplied,
// read and freed by themselves (an accumulator's turn, from one block's products
// to the next one's, is the shorter); eight warps keep 128 sums a thread.
// Persistent over the tiles, eight rows of tiles at a time, so that the tiles in
// work share what L2 holds.
//
// 8190 x 5120 x 4096 takes 128 us: 2690 TFLOP/s, 1.4 times the measured rate in
// bf16.  Its floor is 90 us at twice that rate.  The sums bound it: a block of K takes 710 to 850 clocks where its MMAs take 513;
// without the sums it takes 105 us, without the scales' loads 123, and a block's
// 128 x 256 numbers of TMEM read and added by eight warps alone take 360 to 400
// clocks.  Sixteen warps with 64 sums a thread took 172 us, packed pairs of sums 164.
template <int TILE>                       // outputs of a tile: 256, 192 or 128
struct Many {
    static constexpr int kParts = TILE > 128 ? 2 : 1;        // MMAs of a step
    static constexpr int kPart = TILE / kParts;              // outputs of one
    static constexpr int kDepth = 4 / kParts;                // accumulators, of kParts times 128 columns
    static constexpr int kStage = (128 + TILE / 2) * 128;
    static constexpr int kStages = TILE == 128 ? 6 : 5;
    // Bytes of a row of the boxes that a warp's TILE / 2 outputs go in.
    template <typename O>
    static constexpr int box_row() { return TILE / 2 * (int)sizeof(O) % 128 ? 64 : 128; }
    static constexpr size_t kSmem = 1024 + kStages * kStage + 8 * 8192 + (2 * kStages + 2 * 4 + 2) * 8 + 16;
};
constexpr int kManyBoxes = 8192;         // staging of a warp's results
constexpr int kManyThreads = 384;        // warps 0-7 sums, 8 TMA, 9 MMA (of the pair's first CTA); 10 and 11 fill the warpgroup
// Registers: 168 a thread at launch; 256 threads with up to 128 sums take 208, the
// other 128 keep 72: 256 * 208 + 128 * 72 <= 384 * 168.
constexpr int kManySumRegs = 208, kManyOtherRegs = 72;
static_assert(256 * kManySumRegs + 128 * kManyOtherRegs <= 384 * 168 && kManyThreads == 384, "within the launch's registers");
constexpr int kManyRows = 8;             // rows of tiles that go together

struct ManyParams {
    const float *sx, *sw;
    size_t sx_stride, sw_stride, out_stride;
    int T, N, KB, tiles_m, tiles_n;
    void *out;
    int32_t *err;
    uint32_t polls;                              // of a wait, at most
    int stall;
};

__device__ __forceinline__ void many_tile(const ManyParams &p, int i, int &m, int &n) {
    const int group = i / (kManyRows * p.tiles_n), rows = min(kManyRows, p.tiles_m - group * kManyRows), in = i - group * kManyRows * p.tiles_n;
    n = in / rows;
    m = group * kManyRows + in - n * rows;
}

// A copy of the pair: into this CTA's memory, told to the first CTA's barrier.
__device__ __forceinline__ void tma_pair(void *dst, const CUtensorMap *m, int x, int y, uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], [%4];"
                 ::"r"(saddr(dst)), "l"(m), "r"(x), "r"(y), "r"(bar) : "memory");
}

__device__ __forceinline__ void commit_pair(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                 ::"r"(saddr(bar)), "h"((uint16_t)3) : "memory");
}

__device__ __forceinline__ void tma_store(const CUtensorMap *m, const void *src, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(m), "r"(x), "r"(y), "r"(saddr(src)) : "memory");
}

template <int TILE, typename O>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kManyThreads, 1)
many_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap omap, const ManyParams p) {
    using M = Many<TILE>;
    constexpr int H = TILE / 2, P = M::kParts, D = M::kDepth;        // H: outputs of a warp
    extern __shared__ __align__(1024) uint8_t smdyn[];
    uint8_t *stages = smdyn + ((1024u - (saddr(smdyn) & 1023u)) & 1023u);
    uint8_t *boxes = stages + M::kStages * M::kStage;
    uint64_t *full = reinterpret_cast<uint64_t *>(boxes + 8 * kManyBoxes);
    uint64_t *empty = full + M::kStages, *acc_full = empty + M::kStages, *acc_empty = acc_full + 4, *stall_bar = acc_empty + 4, *drain_bar = stall_bar + 1;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(drain_bar + 1);
    const Bound bound{p.polls, p.err};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rank = blockIdx.x & 1;
    const int tiles = p.tiles_m * p.tiles_n, pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const int mine = tiles > pair ? (tiles - 1 - pair) / pairs + 1 : 0, nq = mine * p.KB;
    if (threadIdx.x == 0) {
        for (int s = 0; s < M::kStages; s++) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
        }
        for (int k = 0; k < 4; k++) {
            mbar_init(acc_full + k, 1);
            mbar_init(acc_empty + k, 16 / P);
        }
        mbar_init(stall_bar, 1);
        mbar_init(drain_bar, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(saddr(tmem_holder)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kManyOtherRegs));
    if (warp == 8) {
        int q = 0, kb = 0, li = 0, m = 0, n = 0;
        if (nq) many_tile(p, pair, m, n);
        if (elected()) {
            const uint32_t first_full = mapped(saddr(full), 0);
            Ring r;
            for (; q < nq; q++, r.next(M::kStages)) {
                uint8_t *stage = stages + r.at * M::kStage;
                if (q >= M::kStages && !wait(empty + r.at, r.turn ^ 1, bound)) break;
                const uint32_t bar = first_full + r.at * 8;
                if (rank == 0) mbar_expect_tx(full + r.at, 2 * M::kStage);
                tma_pair(stage, &xmap, kb * 128, m * 256 + rank * 128, bar);
#pragma unroll
                for (int h = 0; h < P; h++)
                    tma_pair(stage + (128 + h * M::kPart / 2) * 128, &wmap, kb * 128, n * TILE + h * M::kPart + rank * (M::kPart / 2), bar);
                if (++kb == p.KB) {
                    kb = 0;
                    if (++li < mine) many_tile(p, pair + li * pairs, m, n);
                }
            }
        }
        q = __reduce_max_sync(0xffffffffu, (unsigned)q);
        // A wait has run out: the two CTAs may have asked for different fills, and only
        // the first one's barriers tell of them.  What is on its way lands meanwhile.
        if (q < nq)
            for (int i = 0; i < 64; i++) __nanosleep(1000);
        // the last fill of each stage, the other CTA's part too, lands before the pair exits
        for (int s = 0; rank == 0 && s < M::kStages && s < q; s++) {
            const int last = q - 1 - ((q - 1 - s) % M::kStages);
            wait(full + s, (last / M::kStages) & 1, bound);
        }
    } else if (warp == 9 && rank == 0) {
        if (elected()) {
            int left = all_polls(p.polls, nq);
            Ring r;
            for (int q = 0; q < nq; q++, r.next(M::kStages)) {
                const int k = P * (q % D);
                wait_on<true>(full + r.at, r.turn, left);
                const uint32_t at = saddr(stages + r.at * M::kStage);
                const uint64_t a = sw128_desc(at), b = sw128_desc(at + 128 * 128);
#pragma unroll
                for (int h = 0; h < P; h++) {
                    if (q >= D) wait_on<true>(acc_empty + k + h, (q / D - 1) & 1, left);
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < 4; kk++)
                        mma_e4m3<2>(tmem + (k + h) * 128, a + 2 * kk, b + (h * (M::kPart / 2) * 128 >> 4) + 2 * kk, idesc_e4m3(256, M::kPart), kk > 0);
                    commit_pair(acc_full + k + h);
                }
                commit_pair(empty + r.at);
            }
            commit_pair(drain_bar);
            if (left <= 0) atomicExch(p.err, MOE_ETIMEOUT);
        }
        __syncwarp();
    }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kManySumRegs));
        if (p.stall && blockIdx.x == 0 && warp == 0) {                     // test hook: bytes that no copy sends
            if (lane == 0) mbar_expect_tx(stall_bar, 16);
            __syncwarp();
            wait(stall_bar, 0, bound);
        }
        const int h = warp >> 2;                                           // half of the columns
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        uint8_t *box = boxes + warp * kManyBoxes;
        const uint32_t free_bar = mapped(saddr(acc_empty), 0);
        int q = 0;
        int left = all_polls(p.polls, nq);
        for (int li = 0; li < mine; li++) {
            int m, n;
            many_tile(p, pair + li * pairs, m, n);
            const int t = m * 256 + rank * 128 + (warp & 3) * 32 + lane, n0 = n * TILE + h * H;
            // rows behind the end have scales of 0, columns those of the last block
            const float *sx = p.sx + (size_t)min(t, p.T - 1) * p.sx_stride;
            const float *sw = p.sw + (size_t)min(n0 >> 7, (p.N - 1) >> 7) * p.sw_stride;
            // (96 outputs may lie in two blocks of 128: from `edge` on in the next one)
            const float *sw2 = p.sw + (size_t)min((n0 + H - 1) >> 7, (p.N - 1) >> 7) * p.sw_stride;
            const int edge = 128 - (n0 & 127);
            float acc[H];
#pragma unroll
            for (int j = 0; j < H; j++) acc[j] = 0.0f;
            // the scales are loaded a block ahead and multiplied when their block comes
            float xs = __ldg(sx), ws = __ldg(sw), ws2 = H == 96 ? __ldg(sw2) : 0.0f;
            for (int kb = 0; kb < p.KB; kb++, q++) {
                const int k = P * (q % D) + (P == 2 ? h : 0);
                const float scale = xs * ws, scale2 = xs * ws2;
                if (kb + 1 < p.KB) {
                    xs = __ldg(sx + kb + 1), ws = __ldg(sw + kb + 1);
                    if (H == 96) ws2 = __ldg(sw2 + kb + 1);
                }
                wait_on<false>(acc_full + k, (q / D) & 1, left);
                __syncwarp();
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < H; c += 16) {
                    uint32_t d[16];
                    umma::tmem_ld_x16(lanes + k * 128 + (P == 2 ? 0 : h * H) + c, d);
#pragma unroll
                    for (int j = 0; j < 16; j++) acc[c + j] = fmaf(H == 96 && c >= edge ? scale2 : scale, __uint_as_float(d[j]), acc[c + j]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(free_bar + k * 8) : "memory");
            }
            // this warp's results, in boxes of 32 rows whose 16-byte pieces stand as TMA's
            // swizzle has them (no bank conflicts)
            constexpr int ROW = M::template box_row<O>(), PER = ROW / (int)sizeof(O);      // a box's row: bytes, columns
            constexpr int ROUND = H / PER % 2 ? 1 : 2;                                     // boxes at a time
            const int whole = p.N & ~(16 / (int)sizeof(O) - 1);
            const int t_warp = t - lane;
#pragma unroll
            for (int c = 0; c < H; c += PER * ROUND) {
                if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                __syncwarp();
#pragma unroll
                for (int b = 0; b < ROUND; b++)
#pragma unroll
                    for (int i = 0; i < ROW / 16; i++) {
                        uint4 w;
                        float f[8];
#pragma unroll
                        for (int j = 0; j < 16 / (int)sizeof(O); j++) {
                            const int col = c + b * PER + i * (16 / (int)sizeof(O)) + j;
                            f[j] = acc[col];
                        }
                        if constexpr (sizeof(O) == 2) w = bf16x8(f);
                        else w = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
                        *reinterpret_cast<uint4 *>(box + b * 32 * ROW + lane * ROW + ((i ^ (ROW == 128 ? lane & 7 : lane >> 1 & 3)) << 4)) = w;
                    }
                umma::fence_async_shared();
                __syncwarp();
                if (lane == 0 && t_warp < p.T) {
#pragma unroll
                    for (int b = 0; b < ROUND; b++)
                        if (n0 + c + b * PER < whole) tma_store(&omap, box + b * 32 * ROW, n0 + c + b * PER, t_warp);
                    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                }
            }
            // TMA writes whole 16-byte pieces: what is left of the rows goes by itself
            if (whole < p.N && n0 < p.N && n0 + H > whole && t < p.T) {
                O *out = static_cast<O *>(p.out) + (size_t)t * p.out_stride + n0;
#pragma unroll
                for (int c = 0; c < H; c++)
                    if (n0 + c >= whole && n0 + c < p.N) put(out + c, acc[c]);
            }
        }
        if (left <= 0) atomicExch(p.err, MOE_ETIMEOUT);
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    // The last commit's arrival, which the first CTA's MMAs send to both: none is
    // on its way to a CTA that has gone.
    if (warp == 9) wait(drain_bar, 0, bound);
    cluster_sync();                      // the other CTA's arrivals and products are done too
    if (warp == 9) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

// ---------------------------------------------------------------- host
// The hardware holds a poll that fails for 3.8 us.
uint32_t polls_of(uint64_t ns) { return (uint32_t)std::min<uint64_t>(ns / 3800 + 1, INT32_MAX); }

int encode_tile(CUtensorMap *m, const void *base, size_t rows, size_t cols, size_t stride, int box_rows) {
    const cuuint64_t dims[2] = {cols, rows}, strides[1] = {rows > 1 ? stride : align_up(cols, 16)};
    const cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
    return pipe::encode_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// An error of the runtime, which the next launch's check is not to find again.
int failed(cudaError_t e) {
    cudaGetLastError();
    return fail(MOE_ECUDA, "scaled_product: %s", cudaGetErrorString(e));
}

int no_map() { return fail(MOE_ECUDA, "scaled_product: no tensor map"); }

template <int TILE, typename O>
int launch_many(const void *x, size_t x_stride, const moe_scaled_matrix_desc *wd, const ProductParams &q, cudaStream_t st) {
    CUtensorMap xmap, wmap, omap;
    const cuuint64_t dims[2] = {std::max<cuuint64_t>(16 / sizeof(O), q.N / (16 / sizeof(O)) * (16 / sizeof(O))), (cuuint64_t)q.T}, strides[1] = {(q.T > 1 ? q.out_stride : align_up(q.N, 8)) * sizeof(O)};
    constexpr int row = Many<TILE>::template box_row<O>();
    const cuuint32_t box[2] = {(cuuint32_t)(row / sizeof(O)), 32};
    if (encode_tile(&xmap, x, q.T, wd->K, x_stride, 128) || encode_tile(&wmap, wd->w, wd->N, wd->K, wd->w_stride, Many<TILE>::kPart / 2) ||
        pipe::encode_map(&omap, sizeof(O) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, q.out, dims, strides, box,
                         row == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B))
        return no_map();
    static OnDevices ready;
    const cudaError_t e = ready.once([] { return cudaFuncSetAttribute(many_kernel<TILE, O>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Many<TILE>::kSmem); });
    if (e != cudaSuccess) return failed(e);
    const ManyParams p{q.sx, q.sw, q.sx_stride, q.sw_stride, q.out_stride, q.T, q.N, q.KB, (q.T - 1) / 256 + 1, (q.N - 1) / TILE + 1, q.out, q.err, q.polls, q.stall};
    const int pairs = (int)std::min<int64_t>(num_sms() / 2, (int64_t)p.tiles_m * p.tiles_n);
    many_kernel<TILE, O><<<2 * pairs, kManyThreads, Many<TILE>::kSmem, st>>>(xmap, wmap, omap, p);
    return check_launch("many_kernel");
}

template <int MAXN, typename O>
int launch_few(const void *x, size_t x_stride, const moe_scaled_matrix_desc *wd, ProductParams p, cudaStream_t st) {
    CUtensorMap wmap, xmap;
    if (encode_tile(&wmap, wd->w, wd->N, wd->K, wd->w_stride, 128) || encode_tile(&xmap, x, p.T, wd->K, x_stride, p.nt)) return no_map();
    const int tiles = (p.N - 1) / 128 + 1;
    // Up to two CTAs an SM, and with more than 32 tokens four blocks a CTA: the
    // join goes over all its tokens (64 of 2560 x 2048: 7.2 us with four CTAs a tile, 8.5 with eight;
    // one of 5120 x 4096: 8.2 with four, 9.1 with two).
    p.split = 1;
    while (p.split < 8 && 2 * p.split * (p.nt > 32 ? 4 : 1) <= p.KB && (int64_t)tiles * p.split * 2 <= 2 * num_sms()) p.split *= 2;
    const int stage = few_stage(p.nt), least = p.split > 1 ? std::max(2, (p.nt * 512 + stage - 1) / stage) : 2;      // room for the sums
    p.stages = std::max(least, std::min({few_share(p.KB, p.split), kFewMaxStages, (100 << 10) / stage}));
    static OnDevices ready;
    cudaError_t e = ready.once([] { return cudaFuncSetAttribute(few_kernel<MAXN, O>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 << 10); });
    if (e != cudaSuccess) return failed(e);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * p.split));
    cfg.blockDim = dim3(Few<MAXN>::kThreads);
    cfg.dynamicSmemBytes = few_smem<MAXN>(p.KB, p.split, p.stages, p.nt);
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)p.split;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, few_kernel<MAXN, O>, wmap, xmap, p);
    if (e != cudaSuccess) return failed(e);
    return check_launch("few_kernel");
}

template <typename O>
int launch_product(const void *x, size_t x_stride, const moe_scaled_matrix_desc *wd, ProductParams p, cudaStream_t st) {
    // A kernel by the tokens: with 64 the first takes 11.2 us at 5120 x 4096, pairs
    // 13.2; with 96 its 128 columns took 19.5, pairs 13.4.
    if (p.T <= 64) {
        p.nt = (p.T + 15) / 16 * 16;
        if (p.nt <= 16) return launch_few<16, O>(x, x_stride, wd, p, st);
        if (p.nt <= 32) return launch_few<32, O>(x, x_stride, wd, p, st);
        return launch_few<64, O>(x, x_stride, wd, p, st);
    }
    // Pairs' tiles by the rounds that the grid takes over them: a round of 128
    // outputs takes 16.3 us over 64 blocks of K, one of 192 20.8, one of 256 24.5, beside
    // some 5 us of a call.  256 tokens of 5120 x 4096 take 13.7 us in tiles of 128
    // and 17.8 in tiles of 256, 505 of 5000 x 4000 21.8, 16.0 (192) and 17.8,
    // 2048 of 4096 x 4096 39.3 and 32.0.
    const int64_t pairs = std::max(1, num_sms() / 2), rows = (p.T - 1) / 256 + 1;
    auto rounds = [&](int64_t tile) { return (rows * ((p.N - 1) / tile + 1) + pairs - 1) / pairs; };
    if (rounds(128) * ((int64_t)p.KB + 1) >= INT32_MAX || rounds(128) * pairs >= INT32_MAX) return fail(MOE_EUNSUPPORTED, "scaled_product: T=%d N=%d K=%d", p.T, p.N, wd->K);
    const int64_t c128 = 10 * rounds(128), c192 = 13 * rounds(192), c256 = 15 * rounds(256);
    if (c128 <= c192 && c128 <= c256) return launch_many<128, O>(x, x_stride, wd, p, st);
    return c192 <= c256 ? launch_many<192, O>(x, x_stride, wd, p, st) : launch_many<256, O>(x, x_stride, wd, p, st);
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
    p.polls = polls_of(wait.timeout_ns ? wait.timeout_ns : pipe::kDefaultWaitNs), p.stall = wait.stall;
    return out_dtype == MOE_DTYPE_F32 ? launch_product<float>(x, x_stride, wd, p, stream)
                                      : launch_product<__nv_bfloat16>(x, x_stride, wd, p, stream);
}
