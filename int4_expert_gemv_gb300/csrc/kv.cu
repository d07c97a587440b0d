// kv.cu -- the paged key-value cache around the decode attention: the page
// plan of a scheduler step (block tables, slots, free pages) and the append of
// new keys and values.
//
// Plan.  With b_r = ceil(len_r / page) blocks held, a_r = ceil((len_r + new_r)
// / page) needed and exclusive sums over the requests of new_r, a_r - b_r and
// the returned b_r, every output is a function of its own place: token i
// belongs to the request r with first_r <= i < first_{r+1}, stands at place
// len_r + i - first_r, and its block is either in the table already or the
// (needed_r + block - b_r)-th free page.  So no CTA waits for another: each
// makes the three sums for itself (R <= 16384 lengths, a few kB out of L2)
// and then takes its share of the tokens, the new blocks and the returned
// pages.  In a graph, 4096 requests with 710,000 new tokens take 10.2 us: 5.9
// until the sums stand (4096 of them in each CTA, and a launch), 4.3 for the
// items, a search of 12 steps for each four tokens and 1.7 rounds of the grid;
// 256 requests with a token each 3.4, of them 2.2 until the sums.  13.3 us
// under a profiler, 52 % of the issue slots taken, next to nothing from DRAM.
#include <algorithm>

#include "e4m3.cuh"
#include "fastdiv.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr int kMaxPlanRequests = 16384;     // their three sums fit shared memory
using PlanParts = uint32_t[4][32];          // the warps' sums and flags

struct PlanParams {
    const int32_t *seq, *add;
    int R;
    int32_t *table;
    int max_blocks;
    FastDiv page;
    int32_t *ring;
    int n_pages;
    const int32_t *pool;
    int32_t *seq_out, *first, *slots, *places;
    int cap;
    int32_t *pool_out, *status;
};

// Last r with sum[r] <= i, for i below sum[R]: the request that owns item i.
__device__ __forceinline__ int owner(const int32_t *sum, int R, int i) {
    int lo = 0, n = R;
    while (n > 1) {
        const int half = n >> 1;
        if (sum[lo + half] <= i) {
            lo += half;
            n -= half;
        } else {
            n = half;
        }
    }
    return lo;
}

__device__ __forceinline__ int wrap(int64_t i, int n) { return (int)(i < n ? i : i - n); }

// Sums that stick at 2^32 - 1, far above any that fits.
__device__ __forceinline__ uint32_t add_sat(uint32_t a, uint32_t b) {
    const uint32_t s = a + b;
    return s < b ? 0xffffffffu : s;
}

__device__ __forceinline__ uint32_t scan_sat(uint32_t v, int lane) {       // inclusive, over a warp
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v = add_sat(v, u);
    }
    return v;
}

// A thread's items: single tokens, or four neighbours where there are many.
template <int THREADS>
__global__ void __launch_bounds__(THREADS) kv_plan_kernel(const PlanParams p) {
    constexpr int WARPS = THREADS / 32;
    extern __shared__ int32_t sums[];               // [3][R + 1]
    __shared__ PlanParts part;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, R = p.R;
    const int32_t *s_new = sums, *s_need = sums + R + 1, *s_gone = sums + 2 * (R + 1);
    const int page = p.page.d;
    const int head = p.pool[0], n_free = p.pool[1];
    const int64_t room = (int64_t)p.max_blocks * page;

    // this thread's run of requests
    const int run = (R + THREADS - 1) / THREADS;
    const int r0 = min(R, tid * run), r1 = min(R, r0 + run);
    bool invalid = head < 0 || head >= p.n_pages || n_free < 0 || n_free > p.n_pages;
    bool nospace = false;
    uint32_t sum[3] = {0, 0, 0};
#pragma unroll 4
    for (int r = r0; r < r1; r++) {
        const int len = __ldg(p.seq + r), add = __ldg(p.add + r);
        if (len < 0 || len > room || add < -1) {
            invalid = true;
            continue;
        }
        const int have = p.page.ceil(len);
        int item[3] = {0, 0, 0};                    // kept where their sums will stand
        if (add < 0) {
            item[2] = have;
        } else if ((int64_t)len + add > room || (int64_t)len + add > INT32_MAX) {
            nospace = true;
        } else {
            item[0] = add;
            item[1] = p.page.ceil(len + add) - have;
        }
#pragma unroll
        for (int j = 0; j < 3; j++) {
            sum[j] = add_sat(sum[j], item[j]);
            sums[j * (R + 1) + r] = item[j];
        }
        if (blockIdx.x == 0) p.seq_out[r] = add < 0 ? 0 : len + item[0];
    }
    uint32_t upto[3], total[3];
#pragma unroll
    for (int j = 0; j < 3; j++) {
        upto[j] = scan_sat(sum[j], lane);
        if (lane == 31) part[j][warp] = upto[j];
    }
    invalid = __any_sync(0xffffffffu, invalid);
    nospace = __any_sync(0xffffffffu, nospace);
    if (lane == 0) part[3][warp] = (invalid ? 1u : 0u) | (nospace ? 2u : 0u);
    __syncthreads();
    const uint32_t flags = __reduce_or_sync(0xffffffffu, lane < WARPS ? part[3][lane] : 0u);
#pragma unroll
    for (int j = 0; j < 3; j++) {
        const uint32_t v = scan_sat(lane < WARPS ? part[j][lane] : 0u, lane);
        total[j] = __shfl_sync(0xffffffffu, v, 31);
        const uint32_t before = __shfl_sync(0xffffffffu, v, (warp + 31) & 31);
        upto[j] = upto[j] - sum[j] + (warp > 0 ? before : 0u);      // exact unless a total sticks, which is refused
    }
    // more pages held than there are: the tables and the ring contradict each other
    invalid = (flags & 1u) || (uint64_t)n_free + total[2] > (uint64_t)p.n_pages;
    nospace = (flags & 2u) || total[0] > (uint32_t)p.cap || total[1] > (uint32_t)n_free;
    const int step = gridDim.x * THREADS, me = blockIdx.x * THREADS + tid;
    if (invalid || nospace) {                       // the same answer in every CTA
        if (blockIdx.x == 0)                        // (where this CTA has written its sums)
            for (int r = r0; r < r1; r++) p.seq_out[r] = p.seq[r];
        for (int r = me; r <= R; r += step) p.first[r] = 0;
        for (int64_t i = me; i < p.cap; i += step) {            // (cap may be within a step of 2^31)
            p.slots[i] = -1;
            p.places[i] = 0;
        }
        if (me == 0) {
            p.pool_out[0] = head;
            p.pool_out[1] = n_free;
            p.status[0] = invalid ? MOE_EINVAL : MOE_ENOSPACE;
        }
        return;
    }
    for (int r = r0; r < r1; r++) {
        if (blockIdx.x == 0) p.first[r] = (int)upto[0];
#pragma unroll
        for (int j = 0; j < 3; j++) {
            const int item = sums[j * (R + 1) + r];
            sums[j * (R + 1) + r] = (int)upto[j];
            upto[j] += item;
        }
    }
    const int n_new = (int)total[0], n_need = (int)total[1], n_gone = (int)total[2];
    if (me == 0) {
        p.first[R] = n_new;
        p.pool_out[0] = wrap((int64_t)head + n_need, p.n_pages);
        p.pool_out[1] = n_free - n_need + n_gone;
        p.status[0] = MOE_OK;
    }
    __syncthreads();

    // The items of all three kinds in one run, so that their chains of loads
    // overlap: slots and places, new blocks, returned pages.
    const int four = p.cap > step ? 4 : 1;
    const int64_t n_item = ((int64_t)p.cap + four - 1) / four, all = n_item + n_need + n_gone;
    const bool vec = four == 4 && ((reinterpret_cast<uintptr_t>(p.slots) | reinterpret_cast<uintptr_t>(p.places)) & 15) == 0;
    for (int64_t it = me; it < all; it += step) {
        if (it >= n_item + n_need) {                // behind the ring's free part, where no page is being taken
            const int j = (int)(it - n_item - n_need), r = owner(s_gone, R, j);
            p.ring[wrap((int64_t)head + n_free + j, p.n_pages)] = p.table[(size_t)r * p.max_blocks + j - s_gone[r]];
            continue;
        }
        if (it >= n_item) {
            const int j = (int)(it - n_item), r = owner(s_need, R, j);
            const int b = p.page.ceil(__ldg(p.seq + r)) + j - s_need[r];
            p.table[(size_t)r * p.max_blocks + b] = p.ring[wrap((int64_t)head + j, p.n_pages)];
            continue;
        }
        // one search for the first token, and a new length, block or page
        // only where it changes
        const int64_t i0 = it * four;
        int slot[4] = {-1, -1, -1, -1}, place[4] = {0, 0, 0, 0};
        if (i0 < n_new) {
            int r = owner(s_new, R, (int)i0), next = r + 1 < R ? s_new[r + 1] : n_new;
            int len = __ldg(p.seq + r), have = p.page.ceil(len), blk = -1, id = -1;
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const int i = (int)i0 + j;
                if (j >= four || i >= n_new) break;
                if (i >= next) {
                    do {
                        r++;
                        next = r + 1 < R ? s_new[r + 1] : n_new;
                    } while (i >= next);
                    len = __ldg(p.seq + r);
                    have = p.page.ceil(len);
                    blk = -1;
                }
                place[j] = len + i - s_new[r];
                const int b = p.page.div(place[j]);
                if (b != blk) {
                    blk = b;
                    id = b < have ? p.table[(size_t)r * p.max_blocks + b]
                                  : p.ring[wrap((int64_t)head + s_need[r] + b - have, p.n_pages)];
                }
                if ((unsigned)id < (unsigned)p.n_pages) slot[j] = id * page + place[j] - b * page;
            }
        }
        if (vec && i0 + 4 <= p.cap) {
            *reinterpret_cast<int4 *>(p.slots + i0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
            *reinterpret_cast<int4 *>(p.places + i0) = make_int4(place[0], place[1], place[2], place[3]);
        } else {
            for (int j = 0; j < four && i0 + j < p.cap; j++) {
                p.slots[i0 + j] = slot[j];
                p.places[i0 + j] = place[j];
            }
        }
    }
}

template <int THREADS>
int launch_plan(const PlanParams &p, cudaStream_t st) {
    const size_t smem = 3 * (size_t)(p.R + 1) * sizeof(int32_t);
    if (smem + sizeof(PlanParts) > 48 * 1024) {     // (the limit is on both together)
        static OnDevices ready;
        const cudaError_t e = ready.once([] {
            return cudaFuncSetAttribute(kv_plan_kernel<THREADS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        3 * (kMaxPlanRequests + 1) * (int)sizeof(int32_t));
        });
        if (e != cudaSuccess) return fail(MOE_ECUDA, "kv_plan: %s", cudaGetErrorString(e));
    }
    const int64_t want = ((int64_t)p.cap + 2047) / 2048 + (p.R + 15) / 16;
    const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(want, num_sms()));
    kv_plan_kernel<THREADS><<<grid, THREADS, smem, st>>>(p);
    return check_launch("kv_plan_kernel");
}

// ---------------------------------------------------------------- append
struct AppendParams {
    const void *k, *v;
    size_t k_stride, v_stride;      // elements
    const int32_t *slots;
    int N, n_slots, D;
    FastDiv page, row, head;        // chunks of 8 numbers: of a token, of a head
    uint8_t *ck, *cv;
    size_t page_stride;
    const float *k_scale, *v_scale;
};

// (65521 tokens of 8 heads of 128 from fp32: 116 us dividing all, 107 with the
// division left to where two products differ; from bf16 84 and 77.)
__device__ __forceinline__ void store8_e4m3(uint8_t *dst, const float *f, float scale, float2 inv) {
    *reinterpret_cast<uint2 *>(dst) = e4m3_quotients(f, scale, inv);
}

// One thread takes 8 keys and 8 values of a token: 16-byte loads, neighbours in
// a row.  Bytes bound it: 65521 tokens of 8 heads of 128 take 84 us from bf16 to
// bf16 (94 % of the copy rate), 126 from fp32 to bf16 (95 %), 109 from fp32 to
// e4m3 (91 %), 76 from bf16 to e4m3 (78 %: half the bytes to a conversion).
// Places are 32-bit within a span of tokens: a 64-bit quotient per thread cost
// as much as the rest together.
template <typename X, bool E4M3>
__global__ void __launch_bounds__(256, E4M3 && sizeof(X) == 2 ? 5 : 6) kv_append_kernel(const AppendParams p) {
    // Chunks whose loads are asked for together: one, but two where the loads
    // are short and what follows them long.
    constexpr int U = E4M3 && sizeof(X) == 2 ? 2 : 1;
    const int span = INT32_MAX / p.row.d;
    const uint32_t step = gridDim.x * 256;
    for (int n0 = 0; n0 < p.N; n0 += min(span, p.N - n0)) {
        const uint32_t end = (uint32_t)min(span, p.N - n0) * (uint32_t)p.row.d;
        for (uint32_t c = blockIdx.x * 256 + threadIdx.x; c < end; c += U * step) {
            uint4 a[U][sizeof(X) / 2], b[U][sizeof(X) / 2];
            int slot[U], in[U];
#pragma unroll
            for (int u = 0; u < U; u++) {
                slot[u] = -1;
                if (c + u * step < end) {
                    const int m = p.row.div((int)(c + u * step)), n = n0 + m;
                    in[u] = (int)(c + u * step) - m * p.row.d;
                    slot[u] = __ldg(p.slots + n);
                    const X *k = static_cast<const X *>(p.k) + (size_t)n * p.k_stride + 8 * in[u];
                    const X *v = static_cast<const X *>(p.v) + (size_t)n * p.v_stride + 8 * in[u];
#pragma unroll
                    for (int j = 0; j < (int)sizeof(X) / 2; j++) {
                        // (an fp32 chunk's second half is found in L1)
                        const uint4 *ka = reinterpret_cast<const uint4 *>(k) + j, *va = reinterpret_cast<const uint4 *>(v) + j;
                        a[u][j] = sizeof(X) == 4 ? __ldg(ka) : ld_stream16(ka);
                        b[u][j] = sizeof(X) == 4 ? __ldg(va) : ld_stream16(va);
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < U; u++) {
                if ((unsigned)slot[u] >= (unsigned)p.n_slots) continue;
                const int h = p.head.div(in[u]), i = in[u] - h * p.head.d;
                const int pg = p.page.div(slot[u]), off = slot[u] - pg * p.page.d;
                const size_t at = (size_t)pg * p.page_stride +
                                  (((size_t)h * p.page.d + off) * p.D + 8 * i) * (E4M3 ? 1 : 2);
                if (E4M3) {
                    const float ks = p.k_scale ? __ldg(p.k_scale + h) : 1.0f, vs = p.v_scale ? __ldg(p.v_scale + h) : 1.0f;
                    store8_e4m3(p.ck + at, floats8<X>(a[u]).x, ks, inverses(ks));
                    store8_e4m3(p.cv + at, floats8<X>(b[u]).x, vs, inverses(vs));
                } else if (sizeof(X) == 2) {
                    *reinterpret_cast<uint4 *>(p.ck + at) = a[u][0];
                    *reinterpret_cast<uint4 *>(p.cv + at) = b[u][0];
                } else {
                    store8_bf16(p.ck + at, floats8<X>(a[u]).x);
                    store8_bf16(p.cv + at, floats8<X>(b[u]).x);
                }
            }
        }
    }
}

}  // namespace

int check_kv(const moe_kv_desc *kv, const char *who) {
    if (kv == nullptr) return fail(MOE_EINVAL, "%s: cache descriptor is NULL", who);
    if (kv->n_pages < 1 || kv->page < 1 || kv->page > 65536 || kv->Hkv < 1 || kv->Hkv > 65536 ||
        kv->D < 16 || kv->D > 256 || kv->D % 16)
        return fail(MOE_EINVAL, "%s: n_pages=%d page=%d Hkv=%d D=%d (page 1..65536, Hkv 1..65536, "
                                "D a multiple of 16 up to 256)", who, kv->n_pages, kv->page,
                    kv->Hkv, kv->D);
    if ((int64_t)kv->n_pages * kv->page >= (int64_t)1 << 31)
        return fail(MOE_EUNSUPPORTED, "%s: %d pages of %d tokens (need fewer than 2^31 slots)", who,
                    kv->n_pages, kv->page);
    if (kv->dtype != MOE_DTYPE_BF16 && kv->dtype != MOE_DTYPE_E4M3)
        return fail(MOE_EINVAL, "%s: cache dtype=%d (need MOE_DTYPE_BF16 or MOE_DTYPE_E4M3)", who,
                    kv->dtype);
    if (!kv->k || !kv->v || reinterpret_cast<uintptr_t>(kv->k) % 16 ||
        reinterpret_cast<uintptr_t>(kv->v) % 16)
        return fail(MOE_EINVAL, "%s: NULL or misaligned k/v", who);
    const size_t need = (size_t)kv->Hkv * kv->page * kv->D * (kv->dtype == MOE_DTYPE_E4M3 ? 1 : 2);
    if (kv->page_stride < need || kv->page_stride % 16)
        return fail(MOE_EINVAL, "%s: page_stride %zu (need >= %zu, multiple of 16)", who,
                    kv->page_stride, need);
    if (kv->dtype != MOE_DTYPE_E4M3 && (kv->k_scale || kv->v_scale))
        return fail(MOE_EINVAL, "%s: scales with a bf16 cache", who);
    if (reinterpret_cast<uintptr_t>(kv->k_scale) % 4 || reinterpret_cast<uintptr_t>(kv->v_scale) % 4)
        return fail(MOE_EINVAL, "%s: misaligned scales", who);
    return MOE_OK;
}

}  // namespace moe

using namespace moe;

static bool off4(const void *p) { return reinterpret_cast<uintptr_t>(p) % 4 != 0; }

namespace {
struct Ints {                        // an array of the plan's
    const char *name;
    const int32_t *at;
    size_t n;
    bool overlaps(const Ints &o) const {
        const uintptr_t a = reinterpret_cast<uintptr_t>(at), b = reinterpret_cast<uintptr_t>(o.at);
        return n > 0 && o.n > 0 && a < b + 4 * o.n && b < a + 4 * n;
    }
};
}  // namespace

extern "C" int moe_kv_plan(const int32_t *seq_len, const int32_t *new_len, int R,
                           int32_t *block_table, int max_blocks, int page, int32_t *ring,
                           int n_pages, const int32_t *pool, int32_t *seq_out, int32_t *first,
                           int32_t *slots, int32_t *places, int cap, int32_t *pool_out,
                           int32_t *status, cudaStream_t stream) {
    if (R < 0 || cap < 0 || max_blocks < 1 || page < 1 || page > 65536 || n_pages < 1)
        return fail(MOE_EINVAL, "kv_plan: R=%d cap=%d max_blocks=%d page=%d n_pages=%d", R, cap,
                    max_blocks, page, n_pages);
    if (R > kMaxPlanRequests || (int64_t)n_pages * page >= (int64_t)1 << 31)
        return fail(MOE_EUNSUPPORTED, "kv_plan: R=%d (at most %d), %d pages of %d tokens (fewer than "
                                      "2^31 slots)", R, kMaxPlanRequests, n_pages, page);
    if (!ring || !pool || !first || !pool_out || !status || (cap > 0 && (!slots || !places)) ||
        (R > 0 && (!seq_len || !new_len || !block_table || !seq_out)))
        return fail(MOE_EINVAL, "kv_plan: NULL pointer");
    if (off4(seq_len) || off4(new_len) || off4(block_table) || off4(ring) || off4(pool) ||
        off4(seq_out) || off4(first) || off4(slots) || off4(places) || off4(pool_out) || off4(status))
        return fail(MOE_EINVAL, "kv_plan: misaligned pointer");
    // Every CTA reads the lengths, the pool's state, the table and the ring
    // while others write the outputs.
    const Ints in[] = {{"seq_len", seq_len, (size_t)R}, {"new_len", new_len, (size_t)R}, {"pool", pool, 2},
                       {"block_table", block_table, (size_t)R * max_blocks}, {"ring", ring, (size_t)n_pages}};
    const Ints out[] = {{"seq_out", seq_out, (size_t)R}, {"first", first, (size_t)R + 1}, {"slots", slots, (size_t)cap},
                        {"places", places, (size_t)cap}, {"pool_out", pool_out, 2}, {"status", status, 1}};
    for (const Ints &o : out)
        for (const Ints &i : in)
            if (o.overlaps(i)) return fail(MOE_EINVAL, "kv_plan: %s overlaps %s", o.name, i.name);
    for (int j = 3; j < 5; j++)
        for (int i = 0; i < j; i++)
            if (in[j].overlaps(in[i])) return fail(MOE_EINVAL, "kv_plan: %s overlaps %s", in[j].name, in[i].name);
    const PlanParams p{seq_len, new_len, R, block_table, max_blocks, FastDiv(page), ring, n_pages,
                       pool, seq_out, first, slots, places, cap, pool_out, status};
    return R > 1024 ? launch_plan<1024>(p, stream) : launch_plan<512>(p, stream);
}

extern "C" int moe_kv_append(const moe_kv_desc *kv, const void *k, size_t k_stride, const void *v,
                             size_t v_stride, int x_dtype, const int32_t *slots, int N,
                             cudaStream_t stream) {
    if (int rc = check_kv(kv, "kv_append")) return rc;
    if (N < 0) return fail(MOE_EINVAL, "kv_append: N=%d", N);
    if (x_dtype != MOE_DTYPE_F32 && x_dtype != MOE_DTYPE_BF16)
        return fail(MOE_EINVAL, "kv_append: x_dtype=%d", x_dtype);
    if (N == 0) return MOE_OK;
    const size_t row = (size_t)kv->Hkv * kv->D, elt = x_dtype == MOE_DTYPE_F32 ? 4 : 2;
    if (!k || !v || !slots || reinterpret_cast<uintptr_t>(k) % 16 ||
        reinterpret_cast<uintptr_t>(v) % 16 || off4(slots))
        return fail(MOE_EINVAL, "kv_append: NULL or misaligned k/v/slots");
    if ((N > 1 && (k_stride < row || v_stride < row)) || k_stride * elt % 16 || v_stride * elt % 16)
        return fail(MOE_EINVAL, "kv_append: strides %zu / %zu (need >= %zu numbers, 16-byte "
                                "multiples)", k_stride, v_stride, row);
    const AppendParams p{k, v, k_stride, v_stride, slots, N, kv->n_pages * kv->page, kv->D,
                         FastDiv(kv->page), FastDiv((int)(row / 8)), FastDiv(kv->D / 8),
                         static_cast<uint8_t *>(kv->k), static_cast<uint8_t *>(kv->v),
                         kv->page_stride, kv->k_scale, kv->v_scale};
    const int64_t total = (int64_t)N * (int64_t)(row / 8);
    const unsigned grid = (unsigned)std::min<int64_t>((total + 255) / 256, (int64_t)num_sms() * 8);
    const bool f8 = kv->dtype == MOE_DTYPE_E4M3;
    if (x_dtype == MOE_DTYPE_F32) {
        if (f8) kv_append_kernel<float, true><<<grid, 256, 0, stream>>>(p);
        else kv_append_kernel<float, false><<<grid, 256, 0, stream>>>(p);
    } else {
        if (f8) kv_append_kernel<__nv_bfloat16, true><<<grid, 256, 0, stream>>>(p);
        else kv_append_kernel<__nv_bfloat16, false><<<grid, 256, 0, stream>>>(p);
    }
    return check_launch("kv_append_kernel");
}
