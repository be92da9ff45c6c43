// kvc_sparse.cu -- one-token attention over the pages of a paged cache that a
// cheap score selects ("Persistent KV Cache and Decode Performance Roadmap",
// "Phase 2": fixed-size pages read through a page table).
//
// Every full page keeps, per kv head, 8-bit bounds of its keys: with
// s = max|k| / 127 over the page, hi_d = ceil(max_r k_rd / s) and
// lo_d = floor(min_r k_rd / s).  For a query q no key of the page can exceed
//     q . k <= s * sum_d max(q_d hi_d, q_d lo_d)
//            = s * (sum_d max(q_d, 0) hi_d + sum_d min(q_d, 0) lo_d).
// (With a negative `scale` the weights grow with -q . k: it is -q that is scored.)
// Summed over the heads of a group this needs only the group's sums of the
// positive and of the negative parts of the query, rounded to 8 bits: one
// integer dot product of 2 D codes a page, exact, so that which pages are
// taken does not depend on the order of any sum.
//
//   page_bounds_kernel   the bounds of the pages that a step filled
//   page_select_kernel   scores, and the choice of n pages for each row and kv head
//   sparse_decode_kernel attention over them
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "kvc_common.cuh"
#include "kvc_flat.cuh"
#include "kvc_tc.cuh"

namespace {

// --------------------------------------------------------------------------
// bounds
// --------------------------------------------------------------------------

struct BoundsArgs {
    int8_t *bounds;   // [n_pool, kv_heads, 2, D]
    float *scale;     // [n_pool, kv_heads]
    const void *k_pool;
    const int32_t *table;
    int max_pages, page_size;
    int64_t n_pool;
    kvc_lengths len;
    int kv_heads, D;
    int32_t *status;
};

// x / s rounded up (or down) to a code
__device__ __forceinline__ int bound_code(float x, float s, bool up)
{
    const float y = __fdiv_rn(x, s);
    return max(-127, min(127, up ? __float2int_ru(y) : __float2int_rd(y)));
}

// Packed maximum and minimum in which a NaN wins
template <typename T> __device__ __forceinline__ uint32_t pair_max(uint32_t x, uint32_t y)
{
    uint32_t z;
    if constexpr (std::is_same<T, __half>::value)
        asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(z) : "r"(x), "r"(y));
    else
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(z) : "r"(x), "r"(y));
    return z;
}
template <typename T> __device__ __forceinline__ uint32_t pair_min(uint32_t x, uint32_t y)
{
    uint32_t z;
    if constexpr (std::is_same<T, __half>::value)
        asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(z) : "r"(x), "r"(y));
    else
        asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(z) : "r"(x), "r"(y));
    return z;
}

// A warp takes the page of one head: D / 8 lanes a row, eight columns a lane,
// maximum and minimum of two columns at once, kAhead loads of 16 bytes under way.
// It reads 2 D bytes a row once and no block waits for another warp.
// 64 x 256 pages of 64 rows of 128 (268 MB): 46 us, 6.0 TB/s of reads; 117 us with a
// block a page.
constexpr int kBoundWarps = 8;
template <typename T, int D>
__global__ void __launch_bounds__(32 * kBoundWarps)
page_bounds_kernel(const BoundsArgs a)
{
    constexpr int LPR = D / 8, ROWS = 32 / LPR, kAhead = 16;
    const int lane = threadIdx.x & 31, b = blockIdx.y;
    const int item = blockIdx.x * kBoundWarps + (threadIdx.x >> 5);
    const int h = item % a.kv_heads;
    const int P = a.len.past_abs[b], total = a.len.total_abs[b];
    if (a.len.cache_total[b] < 0)
        return;
    const bool lead = lane == 0 && item < a.kv_heads;
    if (total > (int64_t)a.max_pages * a.page_size || P < 0 || P > total) {
        if (lead && h == 0)
            kvc::raise_status(a.status, KVC_DEV_CAPACITY);
        return;
    }
    // pages [P / page, T / page) became full with this step
    const int j = P / a.page_size + item / a.kv_heads;
    if (j >= total / a.page_size)
        return;
    const int64_t id = a.table[(int64_t)b * a.max_pages + j];
    if (id < 0 || id >= a.n_pool) {
        if (lane == 0)
            kvc::raise_status(a.status, KVC_DEV_INDEX_OOB);
        return;
    }
    const int64_t slice = id * a.kv_heads + h;
    const int col = lane % LPR * 8, r0 = lane / LPR;
    const T *k = static_cast<const T *>(a.k_pool) + (slice * a.page_size + r0) * D + col;
    constexpr uint32_t low = std::is_same<T, __half>::value ? 0xfc00fc00u : 0xff80ff80u;  // -infinity
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        hi[e] = low;
        lo[e] = low & 0x7fff7fffu;
    }
    auto take = [&](const uint4 &v) {
        const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            hi[e] = pair_max<T>(hi[e], x[e]);
            lo[e] = pair_min<T>(lo[e], x[e]);
        }
    };
    int r = 0;
    for (; r + kAhead * ROWS <= a.page_size; r += kAhead * ROWS) {
        uint4 v[kAhead];
#pragma unroll
        for (int e = 0; e < kAhead; ++e)
            v[e] = __ldg(reinterpret_cast<const uint4 *>(k + (int64_t)(r + e * ROWS) * D));
#pragma unroll
        for (int e = 0; e < kAhead; ++e)
            take(v[e]);
    }
    for (; r + r0 < a.page_size; r += ROWS)
        take(__ldg(reinterpret_cast<const uint4 *>(k + (int64_t)r * D)));
#pragma unroll
    for (int d = LPR; d < 32; d <<= 1)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            hi[e] = pair_max<T>(hi[e], __shfl_xor_sync(0xffffffffu, hi[e], d));
            lo[e] = pair_min<T>(lo[e], __shfl_xor_sync(0xffffffffu, lo[e], d));
        }
    const T *mx = reinterpret_cast<const T *>(hi), *mn = reinterpret_cast<const T *>(lo);
    // |x| by its bits, so that a NaN or an infinity is the largest
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        top = max(top, max(__float_as_uint(kvc::Elem<T>::to_f32(mx[e])) & 0x7fffffffu,
                           __float_as_uint(kvc::Elem<T>::to_f32(mn[e])) & 0x7fffffffu));
#pragma unroll
    for (int d = 1; d < LPR; d <<= 1)
        top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
    // a page with a NaN or an infinity: scale infinity, the page is taken first
    const bool finite = top < 0x7f800000u;
    const float s = finite ? __fdiv_rn(__uint_as_float(top), 127.f) : INFINITY;
    if (r0 == 0) {
        uint2 out[2] = {};
        if (finite && s > 0.f) {
            int8_t *c = reinterpret_cast<int8_t *>(out);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                c[e] = (int8_t)bound_code(kvc::Elem<T>::to_f32(mx[e]), s, true);
                c[8 + e] = (int8_t)bound_code(kvc::Elem<T>::to_f32(mn[e]), s, false);
            }
        }
        *reinterpret_cast<uint2 *>(a.bounds + slice * 2 * D + col) = out[0];
        *reinterpret_cast<uint2 *>(a.bounds + slice * 2 * D + D + col) = out[1];
        if (lane == 0)
            a.scale[slice] = s;
    }
}

// --------------------------------------------------------------------------
// selection
// --------------------------------------------------------------------------

constexpr int kSelThreads = 256;
constexpr int kMaxPages = 49152;   // pages a sequence may have: their scores stay in shared memory
constexpr int kMaxCluster = 8;
constexpr int kPagesPerCta = 128;  // pages from which a row is worth another CTA

struct SelectArgs {
    const void *q;
    const int8_t *bounds;
    const float *scale;
    const int32_t *table;
    int max_pages, page_size;
    int64_t n_pool;
    kvc_lengths len;
    int batch, kv_heads, group, n_select, sink, recent;
    int negate;            // score -q
    const float *cos_t, *sin_t;
    int64_t rope_max_pos;
    int32_t *selected;     // [B, kv_heads, n_select] logical pages
    int32_t *sub_table;    // the same as pages of the pool seen one head at a time
    int32_t *done;         // [B * kv_heads] units of work finished, for the attention
    int32_t *status;
};

// scores as unsigned keys that order as the scores do; a NaN score orders
// above all (its page holds what the attention has to see)
__device__ __forceinline__ uint32_t order_key(float f)
{
    if (f != f)
        return 0xffffffffu;
    const uint32_t u = __float_as_uint(f + 0.f);  // -0 as 0
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// the block's sum of v, and in `before` that of the threads before this one
__device__ __forceinline__ int block_scan(int v, int *warp_sum, int &before)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d)
            inc += u;
    }
    __syncthreads();
    if (lane == 31)
        warp_sum[warp] = inc;
    __syncthreads();
    int total = 0, base = 0;
#pragma unroll
    for (int w = 0; w < kSelThreads / 32; ++w) {
        base += w < warp ? warp_sum[w] : 0;
        total += warp_sum[w];
    }
    before = base + inc - v;
    return total;
}

// thread-block clusters: rank, size, barrier, and a 32-bit store
__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// into the shared memory of another CTA of the cluster, at the place of p in this one's
__device__ __forceinline__ void cluster_store(const uint32_t *p, uint32_t rank, uint32_t v)
{
    uint32_t at;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(kvc::smem_u32(p)), "r"(rank));
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}

// A sum and what its roundings dropped (Knuth's exact two-term sum): 48 bits, on a
// part whose 64-bit arithmetic takes a warp's addition in 16 clocks
struct Sum2 {
    float hi = 0.f, lo = 0.f;
    __device__ __forceinline__ void add(float x)
    {
        const float s = __fadd_rn(hi, x), z = __fsub_rn(s, hi);
        lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, z)), __fsub_rn(x, z)));
        hi = s;
    }
};

// One cluster per (batch row, kv head), of one CTA for every kPagesPerCta pages that
// the table holds, eight at most: each CTA scores a run of the pages and sends the
// scores to the first one, which chooses alone.  kAhead pages' bounds are under way
// for each group of lanes, the first of them while the query's codes are made.
// The choice is that of the rest-th largest key, found 8 bits at a time below the
// highest bit in which the keys differ (keys are close together: on their leading
// bits a histogram is one bin, and its atomics one queue).
// 64 rows of up to 2048 pages: 11 to 16 us, each step a chain of its own (ids 2, bounds
// and query 2, scores 2 to 5, n-th largest 2, compaction 2 to 3).  They took 71 us with
// one CTA a row and a page at a time, 24 us with the histograms of eight CTAs joined at
// every step.
template <typename T, int D>
__global__ void __launch_bounds__(kSelThreads, 4)
page_select_kernel(const SelectArgs a, int run_max)
{
    extern __shared__ uint32_t keys[];            // [max_pages] scores as order_key, then the run's page ids
    __shared__ float part[2][D];                  // sums of the positive and negative parts
    __shared__ __align__(16) int8_t code[2 * D];  // their codes
    __shared__ int warp_sum[kSelThreads / 32];
    __shared__ uint32_t hist[256];
    __shared__ uint32_t pick[3];
    __shared__ int order[kSelThreads];
    __shared__ float top_sh[kSelThreads / 32];
    __shared__ uint32_t edge_sh[2][kSelThreads / 32];
    int32_t *ids = reinterpret_cast<int32_t *>(keys + a.max_pages);
    kvc::grid_dep_launch();
    const uint32_t rank = cluster_rank(), ctas = cluster_size();
    const int h = blockIdx.x / ctas, b = blockIdx.y, row = b * a.kv_heads + h;
    const int tid = threadIdx.x;
    const int total = a.len.total_abs[b];
    int L = a.len.cache_total[b];
    const bool lead = tid == 0 && rank == 0;
    if (L >= 0 && (total < 1 || total > (int64_t)a.max_pages * a.page_size)) {
        if (lead && h == 0)
            kvc::raise_status(a.status, KVC_DEV_CAPACITY);
        L = -1;
    }
    if (L >= 0 && a.cos_t && (int64_t)total > a.rope_max_pos) {
        if (lead && h == 0)
            kvc::raise_status(a.status, KVC_DEV_ROPE_RANGE);
        L = -1;
    }
    int32_t *sel = a.selected + (int64_t)row * a.n_select, *sub = a.sub_table + (int64_t)row * a.n_select;
    if (L < 0)  // (every CTA of the cluster)
        return;
    if (lead)
        a.done[row] = 0;
    const int pages = (total + a.page_size - 1) / a.page_size;
    const int take = min(pages, a.n_select);
    // pages [0, sink) and [tail, pages) are always taken
    const int tail = max(0, pages - a.recent), sink = min(a.sink, tail);
    const int rest = take - sink - (pages - tail);  // to choose out of [sink, tail)
    const int middle = tail - sink;
    const bool choose = rest > 0 && rest < middle;
    if (!choose && rank > 0)
        return;
    const int32_t *table = a.table + (int64_t)b * a.max_pages;
    if (choose) {
        // (the first CTA has to run before another writes into it: the wait is below)
        asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
        // this CTA's run of the middle pages
        const int run = (middle + (int)ctas - 1) / (int)ctas;
        const int first = min(middle, (int)rank * run), mine = min(run, middle - first);
        // the group's query, and by the other half of the threads the ids of the run's pages
        if (tid < D / 2) {
            const int p = tid;
            const int64_t pos = (int64_t)total - 1;
            const T *q = static_cast<const T *>(a.q) + (int64_t)row * a.group * D;
            float cs = 1.f, sn = 0.f;
            if (a.cos_t) {
                cs = __ldg(a.cos_t + pos * (D / 2) + p);
                sn = __ldg(a.sin_t + pos * (D / 2) + p);
            }
            // in twice the digits, so that a sum does not hang on the order of the heads
            Sum2 up[2], down[2];
#pragma unroll 4
            for (int r = 0; r < a.group; ++r) {
                float x[2] = {kvc::Elem<T>::to_f32(q[r * D + p]), kvc::Elem<T>::to_f32(q[r * D + D / 2 + p])};
                if (a.cos_t)
                    kvc::rope_pair(x[0], x[1], cs, sn);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    up[e].add(x[e] > 0.f ? x[e] : 0.f);
                    down[e].add(x[e] < 0.f ? x[e] : 0.f);
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                // (the positive parts of -q are the negative ones of q, with the other sign)
                const float u = __fadd_rn(up[e].hi, up[e].lo), w = __fadd_rn(down[e].hi, down[e].lo);
                part[0][p + e * (D / 2)] = a.negate ? -w : u;
                part[1][p + e * (D / 2)] = a.negate ? -u : w;
            }
        } else if (tid >= kSelThreads / 2) {
            for (int j = tid - kSelThreads / 2; j < mine; j += kSelThreads / 2)
                ids[j] = __ldg(table + sink + first + j);
        }
        __syncthreads();

        // ---- bounds: 16 codes a lane, D / 8 lanes a page ----
        constexpr int LPP = D / 8, PPB = kSelThreads / LPP, kAhead = 8;
        const int sub_lane = tid % LPP;
        uint4 v[kAhead];
        float s[kAhead];
        uint32_t bad = 0;
        auto fetch = [&](int j0) {
            bad = 0;
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int32_t id = ids[min(j0 + u * PPB, mine - 1)];
                const bool out = id < 0 || id >= a.n_pool;
                bad |= (uint32_t)out << u;
                const int64_t slice = (int64_t)(out ? 0 : id) * a.kv_heads + h;
                v[u] = __ldg(reinterpret_cast<const uint4 *>(a.bounds + slice * 2 * D) + sub_lane);
                s[u] = __ldg(a.scale + slice);
            }
        };
        if (mine > 0)
            fetch(tid / LPP);

        // ---- the query's codes ----
        float top = 0.f;
        for (int i = tid; i < 2 * D; i += kSelThreads)
            top = fmaxf(top, fabsf(part[i / D][i % D]));
#pragma unroll
        for (int d = 16; d; d >>= 1)
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        if ((tid & 31) == 0)
            top_sh[tid >> 5] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kSelThreads / 32; ++w)
            top = fmaxf(top, top_sh[w]);
        const float sq = __fdiv_rn(top, 127.f);
        for (int i = tid; i < 2 * D; i += kSelThreads) {
            const float x = part[i / D][i % D];
            code[i] = (int8_t)(sq > 0.f ? max(-127, min(127, __float2int_rn(__fdiv_rn(x, sq)))) : 0);
        }
        __syncthreads();

        // ---- scores, to the first CTA ----
        asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
        const uint4 qc = reinterpret_cast<const uint4 *>(code)[sub_lane];
        for (int j0 = tid / LPP; j0 - tid / LPP < mine; j0 += kAhead * PPB) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                int sum = __dp4a((int)v[u].x, (int)qc.x, 0);
                sum = __dp4a((int)v[u].y, (int)qc.y, sum);
                sum = __dp4a((int)v[u].z, (int)qc.z, sum);
                sum = __dp4a((int)v[u].w, (int)qc.w, sum);
#pragma unroll
                for (int d = 1; d < LPP; d <<= 1)
                    sum += __shfl_xor_sync(0xffffffffu, sum, d);
                const int j = j0 + u * PPB;
                if (j < mine && sub_lane == 0) {
                    const bool out = bad >> u & 1u;
                    if (out)
                        kvc::raise_status(a.status, KVC_DEV_INDEX_OOB);
                    // a page that does not exist orders first too: the attention reports it
                    cluster_store(keys + first + j, 0,
                                  out || isinf(s[u]) ? 0xffffffffu : order_key(__fmul_rn(s[u], (float)sum)));
                }
            }
            if (j0 - tid / LPP + kAhead * PPB < mine)
                fetch(j0 + kAhead * PPB);
        }
        cluster_sync();
        if (rank > 0)
            return;  // (nobody reads or writes this CTA's shared memory)
    }

    // ---- the rest-th largest key ----
    uint32_t least = 0;   // a page with a key above it is taken,
    int ties = 0;         // and the first `ties` pages with that key
    if (choose) {
        uint32_t lo = 0xffffffffu, hi = 0;
        for (int j = tid; j < middle; j += kSelThreads) {
            lo = min(lo, keys[j]);
            hi = max(hi, keys[j]);
        }
        lo = __reduce_min_sync(0xffffffffu, lo);
        hi = __reduce_max_sync(0xffffffffu, hi);
        if ((tid & 31) == 0) {
            edge_sh[0][tid >> 5] = lo;
            edge_sh[1][tid >> 5] = hi;
        }
        hist[tid] = 0;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kSelThreads / 32; ++w) {
            lo = min(lo, edge_sh[0][w]);
            hi = max(hi, edge_sh[1][w]);
        }
        int left = hi == lo ? 0 : 32 - __clz(hi - lo);  // bits of key - lo still to find
        uint32_t prefix = 0;                            // the bits found, above them
        int want = rest;
        while (left > 0) {
            const int shift = max(0, left - 8);
            const uint32_t digit = (1u << (left - shift)) - 1;
            for (int j = tid; j < middle; j += kSelThreads) {
                const uint32_t x = keys[j] - lo;
                if (left == 32 || x >> left == prefix)
                    atomicAdd(&hist[x >> shift & digit], 1u);
            }
            __syncthreads();
            // bins from the top: thread i looks at bin 255 - i
            const int n = (int)hist[255 - tid];
            int before;
            block_scan(n, warp_sum, before);
            hist[255 - tid] = 0;
            if (before < want && before + n >= want) {
                pick[0] = 255 - tid;
                pick[1] = want - before;
                pick[2] = n;
            }
            __syncthreads();
            prefix = prefix << (left - shift) | pick[0];
            want = (int)pick[1];
            left = shift;
            if ((int)pick[2] == want)
                break;  // every key with these bits is taken
        }
        // (left bits not looked at: the keys from prefix 0...0 on, all of them, which some key is below)
        least = lo + (prefix << left) - (left > 0 ? 1 : 0);
        ties = left > 0 ? 0 : want;
    }

    // ---- the chosen pages in ascending order: a run of pages a thread ----
    {
        const int each = ((pages + kSelThreads - 1) / kSelThreads) | 1;  // (odd: the runs start in different banks)
        const int j0 = min(pages, tid * each), j1 = min(pages, j0 + each);
        auto rank_of = [&](int j) {  // 2: taken, 1: taken if among the first of its key, 0: not
            if (j < sink || j >= tail)
                return 2;
            if (!choose)
                return rest > 0 ? 2 : 0;
            return keys[j - sink] > least ? 2 : keys[j - sink] == least ? 1 : 0;
        };
        int sure = 0, tied = 0;
        for (int j = j0; j < j1; ++j) {
            const int k = rank_of(j);
            sure += k >> 1;
            tied += k & 1;
        }
        int tied_before = 0, before;
        if (choose)
            block_scan(tied, warp_sum, tied_before);
        block_scan(sure + max(0, min(tied, ties - tied_before)), warp_sum, before);
        auto put = [&](int i, int j) {
            const int32_t id = __ldg(table + j);
            sel[i] = j;
            // an id outside the pool stays outside the one-head pool
            sub[i] = id < 0 || id >= a.n_pool ? -1 : (int32_t)((int64_t)id * a.kv_heads + h);
        };
        // (the first of them by a thread each: their ids come in at once)
        for (int j = j0; j < j1; ++j) {
            const int k = rank_of(j);
            if (k == 2 || (k == 1 && tied_before++ < ties)) {
                if (before < kSelThreads)
                    order[before] = j;
                else
                    put(before, j);
                ++before;
            }
        }
        __syncthreads();
        if (tid < take)
            put(tid, order[tid]);
    }
    for (int i = take + tid; i < a.n_select; i += kSelThreads) {
        sel[i] = -1;
        sub[i] = -1;
    }
}

// --------------------------------------------------------------------------
// attention over the chosen pages
// --------------------------------------------------------------------------

constexpr int kUnit = 64;           // keys of a unit of work: pages are whole units
// units (kvc_flat.cuh) that a row costs beside its keys: sparse-long of perf/operators.py takes
// 48.3 us with 2, 47.5 with 4, 46.5 with 6, 45.7 with 8
constexpr int kRowCost = 8;
constexpr int kWarps = 4;           // that compute, 16 keys of a unit each
constexpr int kDecodeThreads = 32 * (kWarps + 2);
constexpr float kNone = -1e30f;     // a reference maximum before any score (finite: differences stay numbers)
constexpr float kSlack = 8.f;       // log2 units a score may exceed its reference by

struct SparseArgs {
    void *out;
    const void *q;
    const int32_t *sub_table;       // [B * kv_heads, n_select] pages of the pool seen one head at a time
    int32_t *done;                  // [B * kv_heads]
    kvc_lengths len;
    int batch, kv_heads, group, n_select, max_pages, page_size;
    float scale_log2;
    const float *cos_t, *sin_t;
    int64_t rope_max_pos;
    int grid, row_cost;             // row_cost: units that a row costs beside its keys
    float *ws_o, *ws_m, *ws_l;      // [2 * grid][group] (x D)
    int32_t *status;
};

// the keys of a row of batch row b, all of whose chosen pages but the last (that of
// the newest token) are full; 0: the batch row is rejected
__device__ __forceinline__ int chosen_rows(const SparseArgs &a, int b, int &total)
{
    total = a.len.total_abs[b];
    if (a.len.cache_total[b] < 0 || total < 1 || total > (int64_t)a.max_pages * a.page_size ||
        (a.cos_t && (int64_t)total > a.rope_max_pos))
        return 0;
    const int pages = (total - 1) / a.page_size + 1;
    return (min(pages, a.n_select) - 1) * a.page_size + total - (pages - 1) * a.page_size;
}

__host__ __device__ constexpr int ctas_per_sm(int D) { return D == 64 ? 3 : D == 128 ? 2 : 1; }

template <int D, int HB> struct SparseSmem {
    static constexpr int SLAB = kUnit * D * 2;                 // a unit's K or V
    // (deeper, the queues before the memory hold up the joins more than the keys: 45.7 us with 2, 47.6 with 3)
    static constexpr int STAGES = D == 64 ? 4 : 2;
    static constexpr int HEADS = 8 * HB;
    static constexpr int V_OFF = STAGES * SLAB, Q_OFF = 2 * STAGES * SLAB;
    static constexpr int Q_BYTES = D / 16 * HB * 32 * 16;      // a lane's fragments of a k-step: two parts of two words
    static constexpr int O_PITCH = D + 4;                      // floats
    static constexpr int O_BYTES = HEADS * O_PITCH * 4;        // at a segment's end, in the queries' place
    static constexpr int ML_OFF = Q_OFF + (Q_BYTES > O_BYTES ? Q_BYTES : O_BYTES);  // m and l of each warp
    static constexpr int BAR_OFF = ML_OFF + 2 * kWarps * HEADS * 4;
    static constexpr int FLAG_OFF = BAR_OFF + 4 * STAGES * 8;  // the abort flag, and whether this CTA joins
    static constexpr int TOTAL = FLAG_OFF + 16;
    static_assert(ctas_per_sm(D) * (TOTAL + 1024 + 1024) <= 228 * 1024, "resident CTAs");
};

template <typename T>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (std::is_same<T, __half>::value)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void load_tiles(uint32_t (&r)[4], uint32_t at)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ void load_tiles_trans(uint32_t (&r)[4], uint32_t at)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ uint32_t transposed(uint32_t x)
{
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ void compute_bar() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory"); }
// x as a 16-bit number, and what that left
template <typename T> __device__ __forceinline__ void parts_of(float x, T &hi, T &lo)
{
    hi = kvc::Elem<T>::from_f32(x);
    lo = kvc::Elem<T>::from_f32(x - kvc::Elem<T>::to_f32(hi));
}

// Attention of one query over the chosen pages of a flat share of the (batch row,
// kv head) rows (kvc_flat.cuh).  Memory bounds it: two warps bring K and V, 64 rows
// a TMA box (pages are multiples of 64 rows), through a ring that fills the SM's
// shared memory, and four warps take 16 keys each into mma.sync m16n8k16,
//   scores  S^T[key][head] = K[key][:] . Q[head][:]
//   output  O^T[d][head] += V^T[d][key] w[key][head]
// (a group has 16 heads at most: the tensor cores have nine tenths of their time to
// spare).  So the query, rotated in float32, and the weights are sums of two 16-bit
// numbers each, at the price of a second product: of the roundings to 16 bits only
// the result's is left.  (An infinity in V meets both parts of its weight, of which
// the second may be zero or negative: what comes out is NaN or infinite as that falls,
// and is made NaN.)  A row that several CTAs worked on is joined by the one of
// them that finishes last, in the order of the shares whichever that is.
// 64 rows of 64 pages of 64 keys of 128 (134 MB): 33 us alone, of which 20 are the
// bytes; the first bytes come 3 us after the choice of pages is done, and the joins
// take the rest.
template <typename T, int D, int HB>
__global__ void __launch_bounds__(kDecodeThreads, ctas_per_sm(D))
sparse_decode_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                     const SparseArgs a)
{
    using SM = SparseSmem<D, HB>;
    using kvc_tc::wait_or_abort;
    constexpr int HEADS = SM::HEADS, STAGES = SM::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + SM::BAR_OFF), *empty = full + 2 * STAGES;  // K's, then V's
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + SM::FLAG_OFF);
    int *joins = reinterpret_cast<int *>(smem + SM::FLAG_OFF + 4);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = blockIdx.x;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2 * STAGES; ++i) {
            kvc::mbar_init(&full[i], 1);
            kvc::mbar_init(&empty[i], kWarps);
        }
        *abort_flag = 0;
        kvc::fence_mbar_init();
    }
    auto units_of = [&](int b) {
        int total;
        const int n = chosen_rows(a, b, total);
        return n > 0 ? (n + kUnit - 1) / kUnit + a.row_cost : 0;
    };
    int x, x_end, b, base;
    kvc_flat::share_of_cta(a.batch, a.kv_heads, units_of, a.grid, c, x, x_end, b, base);
    __syncthreads();

    // the share's segments, one at a time: units [u0, u1) of row (b, h)
    struct {
        int n, total, line, h, u0, u1;
    } sg;
    auto segment = [&]() -> bool {
        if (x >= x_end)
            return false;
        sg.n = chosen_rows(a, b, sg.total);
        sg.line = (sg.n + kUnit - 1) / kUnit + a.row_cost;
        sg.h = (x - base) / sg.line;
        const int p0 = (x - base) - sg.h * sg.line, p1 = min(sg.line, p0 + (x_end - x));
        // (the units that stand for the row's cost hold no keys)
        sg.u0 = max(0, p0 - a.row_cost);
        sg.u1 = p1 - a.row_cost;
        x += p1 - p0;
        return sg.u1 > sg.u0;
    };
    auto next_row = [&]() {
        if (x == base + sg.line * a.kv_heads && x < x_end) {
            int total;
            base = x;
            do {
                ++b;
            } while (chosen_rows(a, b, total) == 0);
        }
    };

    if (warp >= kWarps) {
        // ======================= TMA producers of K and of V =======================
        const bool is_v = warp == kWarps + 1;
        const CUtensorMap *tmap = is_v ? &tmap_v : &tmap_k;
        uint64_t *my_full = full + (is_v ? STAGES : 0), *my_empty = empty + (is_v ? STAGES : 0);
        uint8_t *ring = smem + (is_v ? SM::V_OFF : 0);
        if (lane == 0)
            kvc::tma_prefetch_desc(tmap);
        kvc::grid_dep_wait();
        int i = 0;  // units so far
        bool ok = true;
        while (ok && segment()) {
            const int32_t *table = a.sub_table + ((int64_t)b * a.kv_heads + sg.h) * a.n_select;
            const int per_page = a.page_size / kUnit;
            int32_t id = 0;
            for (int u = sg.u0; u < sg.u1; ++u, ++i) {
                if (((u - sg.u0) & 31) == 0)
                    id = u + lane < sg.u1 ? __ldg(table + (u + lane) / per_page) : 0;
                const int32_t page = __shfl_sync(0xffffffffu, id, (u - sg.u0) & 31);
                const int slot = i % STAGES;
                if (i >= STAGES)
                    ok = wait_or_abort(&my_empty[slot], (i / STAGES - 1) & 1, abort_flag, a.status);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok)
                    break;
                if (lane == 0) {
                    // a page outside the pool: reported, and the pool's first in its place
                    if (page < 0 && !is_v)
                        kvc::raise_status(a.status, KVC_DEV_INDEX_OOB);
                    const int32_t y = page < 0 ? 0 : page * a.page_size + u % per_page * kUnit;
                    kvc::mbar_arrive_expect_tx(&my_full[slot], SM::SLAB);
                    kvc::tma_load_3d(ring + slot * SM::SLAB, tmap, 0, y, 0, &my_full[slot]);
                }
                __syncwarp();
            }
            next_row();
        }
        if (*abort_flag && lane == 0)
            // wind-down: let the loads in flight land before the CTA exits
            for (int k = max(0, i - STAGES); k < i; ++k)
                kvc::mbar_wait(&my_full[k % STAGES], (k / STAGES) & 1);
        return;
    }

    // ======================= attention =======================
    const int g = lane >> 2, t = lane & 3;
    const uint32_t ring = kvc::smem_u32(smem);
    uint4 *q_frag = reinterpret_cast<uint4 *>(smem + SM::Q_OFF);
    float *o_sh = reinterpret_cast<float *>(smem + SM::Q_OFF);
    float *m_sh = reinterpret_cast<float *>(smem + SM::ML_OFF), *l_sh = m_sh + kWarps * HEADS;
    // this lane's row of the four 8 x 8 tiles of a fragment, in K (rows are keys) and in V (transposed)
    const int k_row = 16 * warp + (lane & 15), v_row = 16 * warp + (lane & 7) + (lane >> 4) * 8;
    const int k_col = lane >> 4, v_col = lane >> 3 & 1;
    auto chunk = [](int row, int col) {  // of a slab: 16 bytes `col` of `row`, 128-byte swizzled
        return (uint32_t)((col >> 3) * (kUnit * 128) + row * 128 + ((col & 7) ^ (row & 7)) * 16);
    };
    int b_none, base_none;
    const kvc_flat::Shares shares(kvc_flat::locate(a.batch, a.kv_heads, units_of, -1, b_none, base_none), a.grid);
    int i = 0;
    bool ok = true, waited = false;
    for (int seg = 0; segment(); ++seg) {
        const int64_t slice = (int64_t)b * a.kv_heads + sg.h;
        const int n = sg.n;
        // ---- the group's queries: rotated, as two parts, in the order of the fragments ----
        {
            const int64_t pos = (int64_t)sg.total - 1;
            const T *q = static_cast<const T *>(a.q) + slice * a.group * D;
            T *to = reinterpret_cast<T *>(q_frag);
            auto place = [&](int r, int d) {  // (in elements) of the upper part of head r's column d
                return (((d >> 4) * HB + (r >> 3)) * 32 + (r & 7) * 4 + (d >> 1 & 3)) * 8 + (d >> 3 & 1) * 2 + (d & 1);
            };
            for (int idx = threadIdx.x; idx < HEADS * (D / 2); idx += 32 * kWarps) {
                const int r = idx / (D / 2), p = idx % (D / 2);
                float lo = 0.f, hi = 0.f;
                if (r < a.group) {
                    lo = kvc::Elem<T>::to_f32(q[r * D + p]);
                    hi = kvc::Elem<T>::to_f32(q[r * D + D / 2 + p]);
                    if (a.cos_t)
                        kvc::rope_pair(lo, hi, __ldg(a.cos_t + pos * (D / 2) + p), __ldg(a.sin_t + pos * (D / 2) + p));
                }
                const int e = place(r, p), f = place(r, p + D / 2);
                parts_of(lo, to[e], to[e + 4]);
                parts_of(hi, to[f], to[f + 4]);
            }
        }
        if (!waited) {
            kvc::grid_dep_wait();
            waited = true;
        }
        compute_bar();

        float o[HB][D / 16][4], m[HB][2], l[HB][2];
#pragma unroll
        for (int hb = 0; hb < HB; ++hb) {
#pragma unroll
            for (int dt = 0; dt < D / 16; ++dt)
                o[hb][dt][0] = o[hb][dt][1] = o[hb][dt][2] = o[hb][dt][3] = 0.f;
            m[hb][0] = m[hb][1] = kNone;
            l[hb][0] = l[hb][1] = 0.f;
        }
        for (int u = sg.u0; u < sg.u1; ++u, ++i) {
            const int slot = i % STAGES, key = u * kUnit + 16 * warp;  // the warp's first
            ok = ok && wait_or_abort(&full[slot], (i / STAGES) & 1, abort_flag, a.status);
            ok = __all_sync(0xffffffffu, ok);
            const bool any = ok && key < n;
            // ---- scores: a chain of products for each part of the query ----
            float s[HB][4], s2[HB][4];
#pragma unroll
            for (int hb = 0; hb < HB; ++hb)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    s[hb][e] = s2[hb][e] = 0.f;
            if (any) {
                const uint32_t at = ring + slot * SM::SLAB;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    uint32_t f[4];
                    load_tiles(f, at + chunk(k_row, 2 * ks + k_col));
#pragma unroll
                    for (int hb = 0; hb < HB; ++hb) {
                        const uint4 qf = q_frag[(ks * HB + hb) * 32 + lane];
                        mma16<T>(s[hb], f, qf.x, qf.y);
                        mma16<T>(s2[hb], f, qf.z, qf.w);
                    }
                }
            }
            __syncwarp();
            if (lane == 0)
                kvc::mbar_arrive(&empty[slot]);

            uint32_t wt[HB][2][2];  // weights: part, keys from 0 or 8 on
            if (any) {
                // ---- softmax ----
                const bool tail = key + 16 > n;
                float z[HB][4], top = kNone;
#pragma unroll
                for (int hb = 0; hb < HB; ++hb)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float v = (s[hb][e] + s2[hb][e]) * a.scale_log2;
                        if (tail && key + g + 8 * (e >> 1) >= n)
                            v = -INFINITY;
                        z[hb][e] = v;
                        top = fmaxf(top, v - m[hb][e & 1]);
                    }
                if (__any_sync(0xffffffffu, top > kSlack)) {
                    // a reference is left behind: raise it to the tile's maximum
#pragma unroll
                    for (int hb = 0; hb < HB; ++hb) {
                        float shrink[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float mx = fmaxf(z[hb][e], z[hb][2 + e]);
#pragma unroll
                            for (int d = 4; d < 32; d <<= 1)
                                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                            mx = fmaxf(mx, m[hb][e]);  // (fmaxf drops a NaN: the reference stays a number)
                            shrink[e] = kvc_tc::fast_exp2(m[hb][e] - mx);
                            l[hb][e] *= shrink[e];
                            m[hb][e] = mx;
                        }
#pragma unroll
                        for (int dt = 0; dt < D / 16; ++dt) {
                            o[hb][dt][0] *= shrink[0];
                            o[hb][dt][1] *= shrink[1];
                            o[hb][dt][2] *= shrink[0];
                            o[hb][dt][3] *= shrink[1];
                        }
                    }
                }
#pragma unroll
                for (int hb = 0; hb < HB; ++hb)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float w0 = kvc_tc::fast_exp2(z[hb][2 * e] - m[hb][0]);
                        const float w1 = kvc_tc::fast_exp2(z[hb][2 * e + 1] - m[hb][1]);
                        l[hb][0] += w0;
                        l[hb][1] += w1;
                        const uint32_t hi = kvc_tc::pack2<T>(w0, w1);
                        const T *back = reinterpret_cast<const T *>(&hi);
                        wt[hb][0][e] = transposed(hi);
                        wt[hb][1][e] = transposed(
                            kvc_tc::pack2<T>(w0 - kvc::Elem<T>::to_f32(back[0]), w1 - kvc::Elem<T>::to_f32(back[1])));
                    }
            }

            // ---- output ----
            ok = ok && wait_or_abort(&full[STAGES + slot], (i / STAGES) & 1, abort_flag, a.status);
            ok = __all_sync(0xffffffffu, ok);
            if (any && ok) {
                const uint32_t at = ring + SM::V_OFF + slot * SM::SLAB;
                // what a row past the last holds does not reach the sums
                const bool tail = key + 16 > n;
                const int k0 = key + 2 * t;
                const uint32_t keep0 = (k0 < n ? 0xffffu : 0u) | (k0 + 1 < n ? 0xffff0000u : 0u);
                const uint32_t keep1 = (k0 + 8 < n ? 0xffffu : 0u) | (k0 + 9 < n ? 0xffff0000u : 0u);
#pragma unroll
                for (int dt = 0; dt < D / 16; ++dt) {
                    uint32_t f[4];
                    load_tiles_trans(f, at + chunk(v_row, 2 * dt + v_col));
                    if (tail) {
                        f[0] &= keep0;
                        f[1] &= keep0;
                        f[2] &= keep1;
                        f[3] &= keep1;
                    }
#pragma unroll
                    for (int hb = 0; hb < HB; ++hb) {
                        mma16<T>(o[hb][dt], f, wt[hb][0][0], wt[hb][0][1]);
                        mma16<T>(o[hb][dt], f, wt[hb][1][0], wt[hb][1][1]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0)
                kvc::mbar_arrive(&empty[STAGES + slot]);
        }

        // ---- join the warps: m, l, then O relative to the common m, one warp after another ----
#pragma unroll
        for (int hb = 0; hb < HB; ++hb)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1)
                    l[hb][e] += __shfl_xor_sync(0xffffffffu, l[hb][e], d);
                if (g == 0) {
                    m_sh[warp * HEADS + hb * 8 + 2 * t + e] = m[hb][e];
                    l_sh[warp * HEADS + hb * 8 + 2 * t + e] = l[hb][e];
                }
            }
        compute_bar();
        float f[HB][2];
#pragma unroll
        for (int hb = 0; hb < HB; ++hb)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float top = -INFINITY;
#pragma unroll
                for (int w = 0; w < kWarps; ++w)
                    top = fmaxf(top, m_sh[w * HEADS + hb * 8 + 2 * t + e]);
                f[hb][e] = exp2f(m[hb][e] - top);
            }
        auto o_at = [&](int hb, int dt, int e) {
            return (hb * 8 + 2 * t + (e & 1)) * SM::O_PITCH + dt * 16 + g + 8 * (e >> 1);
        };
        for (int w = 0; w < kWarps; ++w) {
            if (warp == w) {
#pragma unroll
                for (int hb = 0; hb < HB; ++hb) {
                    // (every load before the first store: they may not pass one another)
                    if (w > 0) {
#pragma unroll
                        for (int dt = 0; dt < D / 16; ++dt)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                o[hb][dt][e] = fmaf(o[hb][dt][e], f[hb][e & 1], o_sh[o_at(hb, dt, e)]);
                    } else {
#pragma unroll
                        for (int dt = 0; dt < D / 16; ++dt)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                o[hb][dt][e] *= f[hb][e & 1];
                    }
#pragma unroll
                    for (int dt = 0; dt < D / 16; ++dt)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o_sh[o_at(hb, dt, e)] = o[hb][dt][e];
                }
            }
            compute_bar();
        }
        const bool whole = sg.u0 == 0 && sg.u1 == sg.line - a.row_cost;
        const int64_t part = 2 * (int64_t)c + (seg == 0 ? 0 : 1);
        if (ok) {
            for (int idx = threadIdx.x; idx < a.group * D; idx += 32 * kWarps) {
                const int r = idx / D, d = idx % D;
                float top = -INFINITY, sum = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w)
                    top = fmaxf(top, m_sh[w * HEADS + r]);
#pragma unroll
                for (int w = 0; w < kWarps; ++w)
                    sum += l_sh[w * HEADS + r] * exp2f(m_sh[w * HEADS + r] - top);
                const float v = o_sh[r * SM::O_PITCH + d];
                if (whole) {
                    static_cast<T *>(a.out)[slice * a.group * D + idx] =
                        kvc::Elem<T>::from_f32(kvc_tc::finite_or_nan(v / sum));
                } else {
                    a.ws_o[(part * a.group + r) * D + d] = v;
                    if (d == 0) {
                        a.ws_m[part * a.group + r] = top;
                        a.ws_l[part * a.group + r] = sum;
                    }
                }
            }
        }
        if (!whole) {
            // (after a wait that gave up the count stays short, and nobody joins)
            __threadfence();
            compute_bar();
            if (threadIdx.x == 0) {
                const int mine = ok ? sg.u1 - sg.u0 : 0;
                *joins = ok && atomicAdd(a.done + slice, mine) + mine == sg.line - a.row_cost;
                __threadfence();
            }
            compute_bar();
            if (*joins) {
                const int x0 = base + sg.h * sg.line;
                const int c0 = shares.of(x0 + a.row_cost), parts = shares.of(x0 + sg.line - 1) - c0 + 1;
                // the row's segment is the first of its CTA, but in CTA c0 if that began before the row
                const int slot0 = shares.begin(c0) < x0 ? 1 : 0;
                for (int r = warp; r < a.group; r += kWarps) {
                    // eight parts under way at a time
                    constexpr int AHEAD = 8;
                    float top = -INFINITY, sum = 0.f, acc[D / 32];
#pragma unroll
                    for (int e = 0; e < D / 32; ++e)
                        acc[e] = 0.f;
                    for (int k0 = 0; k0 < parts; k0 += AHEAD) {
                        float pm[AHEAD], pl[AHEAD], po[AHEAD][D / 32], was = top;
#pragma unroll
                        for (int k = 0; k < AHEAD; ++k) {
                            const int kk = min(k0 + k, parts - 1);
                            const int64_t at = (2 * (int64_t)(c0 + kk) + (kk == 0 ? slot0 : 0)) * a.group + r;
                            pm[k] = k0 + k < parts ? __ldcg(a.ws_m + at) : -INFINITY;
                            pl[k] = __ldcg(a.ws_l + at);
#pragma unroll
                            for (int e = 0; e < D / 32; ++e)
                                po[k][e] = __ldcg(a.ws_o + at * D + lane + 32 * e);
                        }
#pragma unroll
                        for (int k = 0; k < AHEAD; ++k)
                            top = fmaxf(top, pm[k]);
                        const float shrink = exp2f(was - top);
                        sum *= shrink;
#pragma unroll
                        for (int e = 0; e < D / 32; ++e)
                            acc[e] *= shrink;
#pragma unroll
                        for (int k = 0; k < AHEAD; ++k) {
                            const float w = exp2f(pm[k] - top);
                            // (a part that is not there has no weight, whatever was read in its place)
                            if (k0 + k < parts) {
                                sum = fmaf(w, pl[k], sum);
#pragma unroll
                                for (int e = 0; e < D / 32; ++e)
                                    acc[e] = fmaf(w, po[k][e], acc[e]);
                            }
                        }
                    }
#pragma unroll
                    for (int e = 0; e < D / 32; ++e)
                        static_cast<T *>(a.out)[(slice * a.group + r) * D + lane + 32 * e] =
                            kvc::Elem<T>::from_f32(kvc_tc::finite_or_nan(acc[e] / sum));
                }
            }
        }
        compute_bar();  // shared memory may be written again
        next_row();
    }
}

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// One wave of resident CTAs over all rows, or, where the rows are so few that this
// leaves each too many parts: a unit takes a CTA 0.4 us, and joining eight parts of
// four heads 0.9, so that a row of t units is done soonest by about sqrt(3.6 t) CTAs
// (one row of 500 units of 8 heads: 96 us with 304).  Rows then begin with a CTA each
// and cost nothing beside their keys.
struct Grid {
    int ctas, row_cost;
};
Grid decode_grid(int batch, int kv_heads, int group, int page_size, int n_select, int D)
{
    const int64_t rows = (int64_t)batch * kv_heads, t = (int64_t)n_select * page_size / kUnit;
    const int64_t wave = (int64_t)kvc_host::sm_count() * ctas_per_sm(D);
    const int64_t few = std::min(t, (int64_t)std::ceil(std::sqrt(3.6 * (double)t / ((group + 3) / 4))));
    if (rows * few <= wave)
        return {(int)std::max<int64_t>(1, rows * few), 0};
    return {(int)std::min(rows * (t + kRowCost), wave), kRowCost};
}

// the parts of the workspace: the chosen pages, the counts, the partial results
struct SparseLayout {
    size_t done, o, m, l, total;
};
SparseLayout sparse_layout(int batch, int q_heads, int kv_heads, int page_size, int n_select, int D)
{
    SparseLayout l;
    const size_t rows = (size_t)batch * kv_heads;
    const size_t parts = 2 * (size_t)decode_grid(batch, kv_heads, q_heads / kv_heads, page_size, n_select, D).ctas *
                         (q_heads / kv_heads);
    l.done = align256(rows * n_select * 4);
    l.o = l.done + align256(rows * 4);
    l.m = l.o + parts * D * 4;
    l.l = l.m + parts * 4;
    l.total = l.l + parts * 4;
    return l;
}

template <typename T, int D, int HB>
kvc_status launch_decode(const SparseArgs &a, const void *k_pool, const void *v_pool, int64_t n_pool,
                         cudaStream_t stream)
{
    using SM = SparseSmem<D, HB>;
    const CUtensorMapDataType type = std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                                    : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const uint64_t rows = (uint64_t)n_pool * a.kv_heads * a.page_size;
    CUtensorMap tk, tv;
    if (!kvc_host::encode_3d_sw128(&tk, k_pool, rows, D, kUnit, D / 64, type) ||
        !kvc_host::encode_3d_sw128(&tv, v_pool, rows, D, kUnit, D / 64, type))
        return KVC_ERR_CUDA;
    auto kern = sparse_decode_kernel<T, D, HB>;
    const int smem = SM::TOTAL + 1024;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return KVC_ERR_CUDA;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(a.grid);
    cfg.blockDim = dim3(kDecodeThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, tk, tv, a) != cudaSuccess)
        return KVC_ERR_CUDA;
    return kvc_host::launch_status();
}

template <typename T>
kvc_status launch_decode_dim(const SparseArgs &a, const void *k, const void *v, int64_t n_pool, int D,
                             cudaStream_t stream)
{
    const bool two = a.group > 8;
    switch (D) {
    case 64:
        return two ? launch_decode<T, 64, 2>(a, k, v, n_pool, stream) : launch_decode<T, 64, 1>(a, k, v, n_pool, stream);
    case 128:
        return two ? launch_decode<T, 128, 2>(a, k, v, n_pool, stream) : launch_decode<T, 128, 1>(a, k, v, n_pool, stream);
    default:
        return two ? launch_decode<T, 256, 2>(a, k, v, n_pool, stream) : launch_decode<T, 256, 1>(a, k, v, n_pool, stream);
    }
}

bool sizes_ok(int batch, int q_heads, int kv_heads, int page_size, int n_select, int D)
{
    return batch >= 0 && q_heads >= 1 && kv_heads >= 1 && q_heads % kv_heads == 0 && n_select >= 1 &&
           page_size >= 64 && page_size % 64 == 0 && D >= 1;
}

template <typename T, int D> kvc_status launch_select_dim(const SelectArgs &a, cudaStream_t stream)
{
    int ctas = 1;
    while (ctas < kMaxCluster && ctas * kPagesPerCta < a.max_pages)
        ctas *= 2;
    const int run = (a.max_pages + ctas - 1) / ctas, smem = (a.max_pages + run) * 4;
    if (smem > 32 * 1024 && cudaFuncSetAttribute(page_select_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 smem) != cudaSuccess)
        return KVC_ERR_CUDA;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(a.kv_heads * ctas, a.batch);
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ctas;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, page_select_kernel<T, D>, a, run) != cudaSuccess)
        return KVC_ERR_CUDA;
    return kvc_host::launch_status();
}

template <typename T> kvc_status launch_select(const SelectArgs &a, int D, cudaStream_t stream)
{
    switch (D) {
    case 64:
        return launch_select_dim<T, 64>(a, stream);
    case 128:
        return launch_select_dim<T, 128>(a, stream);
    default:
        return launch_select_dim<T, 256>(a, stream);
    }
}

template <typename T> kvc_status launch_bounds(const BoundsArgs &a, int batch, int S, cudaStream_t stream)
{
    // at most ceil(S / page) pages of a batch row become full, a warp for each of their heads
    const int64_t most = ((int64_t)S + a.page_size - 1) / a.page_size * a.kv_heads;
    if (most > (int64_t)INT32_MAX - kBoundWarps)
        return KVC_ERR_SHAPE;
    const dim3 grid((unsigned)((most + kBoundWarps - 1) / kBoundWarps), batch);
    switch (a.D) {
    case 64:
        page_bounds_kernel<T, 64><<<grid, 32 * kBoundWarps, 0, stream>>>(a);
        break;
    case 128:
        page_bounds_kernel<T, 128><<<grid, 32 * kBoundWarps, 0, stream>>>(a);
        break;
    default:
        page_bounds_kernel<T, 256><<<grid, 32 * kBoundWarps, 0, stream>>>(a);
    }
    return kvc_host::launch_status();
}

} // namespace

KVC_API kvc_status kvc_page_bounds(void *bounds, float *bound_scale, const void *k_pool, const int32_t *block_table,
                                   int max_pages, int64_t n_pool_pages, int page_size, kvc_lengths len, int batch,
                                   int kv_heads, int new_tokens, int head_dim, int dtype, int32_t *dev_status,
                                   void *stream_)
{
    if (kvc_host::elem_bytes_of(dtype) == 0)
        return KVC_ERR_DTYPE;
    if (dtype == KVC_F32 || (head_dim != 64 && head_dim != 128 && head_dim != 256))
        return KVC_ERR_UNSUPPORTED;
    if (batch < 0 || batch > 65535 || kv_heads < 1 || new_tokens < 1 || max_pages < 1 ||
        n_pool_pages < 1 || page_size < 1)
        return KVC_ERR_SHAPE;
    if ((int64_t)max_pages * page_size > (int64_t)INT32_MAX)
        return KVC_ERR_CAPACITY;
    if (batch == 0)
        return KVC_OK;
    if (!bounds || !bound_scale || !k_pool || !block_table || !kvc_host::lengths_ok(len))
        return KVC_ERR_NULL;
    for (const void *p : {(const void *)bounds, (const void *)bound_scale, k_pool})
        if (!kvc_host::aligned16(p))
            return KVC_ERR_ALIGN;
    const size_t slices = (size_t)n_pool_pages * kv_heads;
    if (kvc_host::overlaps(bounds, slices * 2 * head_dim, bound_scale, slices * 4) ||
        kvc_host::overlaps(bounds, slices * 2 * head_dim, k_pool, slices * page_size * head_dim * 2) ||
        kvc_host::overlaps(bound_scale, slices * 4, k_pool, slices * page_size * head_dim * 2))
        return KVC_ERR_SHAPE;
    BoundsArgs a{static_cast<int8_t *>(bounds), bound_scale, k_pool, block_table, max_pages, page_size, n_pool_pages,
                 len, kv_heads, head_dim, dev_status};
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    return dtype == KVC_BF16 ? launch_bounds<__nv_bfloat16>(a, batch, new_tokens, stream)
                             : launch_bounds<__half>(a, batch, new_tokens, stream);
}

KVC_API size_t kvc_gqa_decode_sparse_workspace_size(int batch, int q_heads, int kv_heads, int page_size,
                                                    int n_select, int head_dim, int dtype)
{
    if (!sizes_ok(batch, q_heads, kv_heads, page_size, n_select, head_dim) || batch < 1 ||
        (int64_t)n_select * page_size > (int64_t)INT32_MAX || (int64_t)batch * kv_heads > 65535)
        return 0;
    if (kvc_host::elem_bytes_of(dtype) == 0 || (head_dim != 64 && head_dim != 128 && head_dim != 256))
        return 0;
    return sparse_layout(batch, q_heads, kv_heads, page_size, n_select, head_dim).total;
}

KVC_API kvc_status kvc_gqa_decode_sparse(void *out, const void *q, const void *k_pool, const void *v_pool,
                                         const void *bounds, const float *bound_scale, const int32_t *block_table,
                                         int max_pages, int64_t n_pool_pages, int page_size, kvc_lengths len, int batch,
                                         int q_heads, int kv_heads, int head_dim, int dtype, int n_select,
                                         int sink_pages, int recent_pages, int32_t *selected, float scale,
                                         const float *rope_cos, const float *rope_sin, int64_t rope_max_pos,
                                         void *workspace, size_t workspace_bytes, int32_t *dev_status, void *stream_)
{
    if (kvc_host::elem_bytes_of(dtype) == 0)
        return KVC_ERR_DTYPE;
    if (dtype == KVC_F32)
        return KVC_ERR_UNSUPPORTED;
    if (!sizes_ok(batch, q_heads, kv_heads, page_size, n_select, head_dim) || max_pages < 1 || n_pool_pages < 1 ||
        sink_pages < 0 || recent_pages < 1 || (int64_t)sink_pages + recent_pages > n_select)
        return KVC_ERR_SHAPE;
    if ((head_dim != 64 && head_dim != 128 && head_dim != 256) || q_heads / kv_heads > 16)
        return KVC_ERR_UNSUPPORTED;
    if ((int64_t)batch * kv_heads > 65535)
        return KVC_ERR_SHAPE;
    if (max_pages > kMaxPages || (int64_t)max_pages * page_size > (int64_t)INT32_MAX ||
        (int64_t)n_select * page_size > (int64_t)INT32_MAX ||
        n_pool_pages * kv_heads * (int64_t)page_size > (int64_t)INT32_MAX ||
        (int64_t)batch * kv_heads * ((int64_t)n_select * page_size / kUnit + kRowCost) > (int64_t)INT32_MAX)
        return KVC_ERR_CAPACITY;
    if ((rope_cos == nullptr) != (rope_sin == nullptr))
        return KVC_ERR_NULL;
    if (rope_cos && rope_max_pos < 1)
        return KVC_ERR_SHAPE;
    if (batch == 0)
        return KVC_OK;
    if (!out || !q || !k_pool || !v_pool || !bounds || !bound_scale || !block_table || !selected ||
        !kvc_host::lengths_ok(len))
        return KVC_ERR_NULL;
    for (const void *p : {(const void *)out, q, k_pool, v_pool, bounds, (const void *)bound_scale})
        if (!kvc_host::aligned16(p))
            return KVC_ERR_ALIGN;
    const SparseLayout l = sparse_layout(batch, q_heads, kv_heads, page_size, n_select, head_dim);
    if (!workspace || workspace_bytes < l.total)
        return KVC_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u)
        return KVC_ERR_ALIGN;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    SelectArgs a{};
    a.q = q;
    a.bounds = static_cast<const int8_t *>(bounds);
    a.scale = bound_scale;
    a.table = block_table;
    a.max_pages = max_pages;
    a.page_size = page_size;
    a.n_pool = n_pool_pages;
    a.len = len;
    a.batch = batch;
    a.kv_heads = kv_heads;
    a.group = q_heads / kv_heads;
    a.n_select = n_select;
    a.sink = sink_pages;
    a.recent = recent_pages;
    a.negate = scale < 0.f;
    a.cos_t = rope_cos;
    a.sin_t = rope_sin;
    a.rope_max_pos = rope_max_pos;
    a.selected = selected;
    a.sub_table = reinterpret_cast<int32_t *>(ws);
    a.done = reinterpret_cast<int32_t *>(ws + l.done);
    a.status = dev_status;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    const kvc_status st =
        dtype == KVC_BF16 ? launch_select<__nv_bfloat16>(a, head_dim, stream) : launch_select<__half>(a, head_dim, stream);
    if (st != KVC_OK)
        return st;
    SparseArgs d{};
    d.out = out;
    d.q = q;
    d.sub_table = a.sub_table;
    d.done = a.done;
    d.len = len;
    d.batch = batch;
    d.kv_heads = kv_heads;
    d.group = a.group;
    d.n_select = n_select;
    d.max_pages = max_pages;
    d.page_size = page_size;
    d.scale_log2 = (scale == 0.f ? 1.f / sqrtf((float)head_dim) : scale) * 1.44269504088896340736f;
    d.cos_t = rope_cos;
    d.sin_t = rope_sin;
    d.rope_max_pos = rope_max_pos;
    const Grid grid = decode_grid(batch, kv_heads, a.group, page_size, n_select, head_dim);
    d.grid = grid.ctas;
    d.row_cost = grid.row_cost;
    d.ws_o = reinterpret_cast<float *>(ws + l.o);
    d.ws_m = reinterpret_cast<float *>(ws + l.m);
    d.ws_l = reinterpret_cast<float *>(ws + l.l);
    d.status = dev_status;
    return dtype == KVC_BF16 ? launch_decode_dim<__nv_bfloat16>(d, k_pool, v_pool, n_pool_pages, head_dim, stream)
                             : launch_decode_dim<__half>(d, k_pool, v_pool, n_pool_pages, head_dim, stream);
}
