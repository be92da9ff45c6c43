// kvc_ragged.cu -- a serving step whose requests bring different numbers of
// new tokens, packed one behind the other ("Persistent KV Cache and Decode
// Performance Roadmap", "Phase 2": fixed-size pages read through a page table).
//
//   page_release_kernel  pages of ended requests go back onto the free stack
//   ragged_plan_kernel   lengths -> pages taken, offsets, positions, slots
//   rope_tables_kernel   cos and sin of every position, stretched for long contexts
//   ragged_append_kernel norm of each head's query and key, their rotation, K and
//                        V rows to their slots, in one pass
#include <algorithm>
#include <climits>
#include <cmath>
#include <type_traits>

#include "kvc_common.cuh"
#include "kvc_tc.cuh"

namespace {

constexpr int kPlanThreads = 256;
constexpr int kPlanTokens = 4 * kPlanThreads;  // tokens of a block
constexpr int kMaxRequests = 16384;            // two words of shared memory each
constexpr int kMaxTokens = INT_MAX - 1023;     // (a last block's tokens are numbered past the end)

// Inclusive prefix sum over the block's threads; `sums` holds a word a warp.
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t *sums, int64_t &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d)
            x += y;
    }
    if (lane == 31)
        sums[warp] = x;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        if (w == warp)
            x += total;
        total += sums[w];
    }
    __syncthreads();
    return x;
}

__device__ __forceinline__ int64_t pages_of(int64_t tokens, int page_size)
{
    return (tokens + page_size - 1) / page_size;
}

struct Stack {
    const int32_t *count;  // free pages before the call
    int64_t n_pool;
    // 0 for a count that no stack of the pool has
    __device__ __forceinline__ int64_t depth(int32_t *status) const
    {
        const int64_t n = *count;
        if (n >= 0 && n <= n_pool)
            return n;
        if (threadIdx.x == 0)
            kvc::raise_status(status, KVC_DEV_INDEX_OOB);
        return 0;
    }
};

struct ReleaseArgs {
    const int32_t *released, *table;
    int max_pages, page_size;
    int32_t *free_pages;
    Stack stack;
    int32_t *left;
    int batch;
    int32_t *status;
};

// Every block finds the place of every row's first page on the stack (a prefix
// sum over the rows) and copies the pages of its own rows, a warp a row.
__global__ void __launch_bounds__(kPlanThreads)
page_release_kernel(const ReleaseArgs a)
{
    extern __shared__ int32_t place[];  // [batch], -1: nothing goes back
    __shared__ int64_t sums[kPlanThreads / 32];
    kvc::grid_dep_wait();
    const int64_t depth = a.stack.depth(a.status);
    int64_t before = 0;
    int given = 0;  // pages that rows of this thread give back, for the number left
    for (int b0 = 0; b0 < a.batch; b0 += kPlanThreads) {
        const int b = b0 + threadIdx.x;
        int64_t n = 0;
        if (b < a.batch) {
            const int t = a.released[b];
            n = t > 0 ? pages_of(t, a.page_size) : 0;
            if (t < 0 || n > a.max_pages) {
                if (blockIdx.x == 0)
                    kvc::raise_status(a.status, KVC_DEV_SEQLEN_RANGE);
                n = 0;
            }
        }
        int64_t total;
        const int64_t end = before + block_scan(n, sums, total);
        if (b < a.batch) {
            const bool fits = depth + end <= a.stack.n_pool;
            if (n > 0 && !fits && blockIdx.x == 0)
                kvc::raise_status(a.status, KVC_DEV_CAPACITY);
            place[b] = n > 0 && fits ? (int32_t)(depth + end - n) : -1;
            given += n > 0 && fits ? (int)n : 0;
        }
        before += total;
    }
    int64_t total;
    block_scan(given, sums, total);
    if (blockIdx.x == 0 && threadIdx.x == 0)
        *a.left = (int32_t)(depth + total);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int b = blockIdx.x * (kPlanThreads / 32) + warp; b < a.batch; b += gridDim.x * (kPlanThreads / 32)) {
        const int at = place[b];
        if (at < 0)
            continue;
        const int n = (int)pages_of(a.released[b], a.page_size);
        for (int j = lane; j < n; j += 32) {
            const int32_t id = a.table[(int64_t)b * a.max_pages + j];
            if (id < 0 || id >= a.stack.n_pool)
                kvc::raise_status(a.status, KVC_DEV_INDEX_OOB);
            a.free_pages[at + j] = id;
        }
    }
}

struct PlanArgs {
    const int32_t *cached, *fresh;
    int32_t *table;
    int max_pages, page_size;
    const int32_t *free_pages;
    Stack stack;
    int32_t *left;
    int batch, tokens;
    int32_t *offsets;
    kvc_lengths len;
    int32_t *positions, *slots;
    int32_t *status;
};

// Every block finds where every request's tokens begin and which pages it
// takes (two prefix sums over the requests, in shared memory), block 0 writes
// that down, and each block fills in the places of its 1024 tokens: a token
// that begins a page that its request did not hold writes the page's id into the table.
// (One launch: a second one for the tokens would cost as much as the sums.)
// A chain of loads and barriers bounds both kernels: 6.3 us the two for 32 requests, 10.2
// for 256 with 16 prompts (17000 tokens).
__global__ void __launch_bounds__(kPlanThreads)
ragged_plan_kernel(const PlanArgs a)
{
    extern __shared__ int32_t plan[];
    __shared__ int64_t sums[kPlanThreads / 32];
    int32_t *begin = plan;                // [batch + 1] first token
    int32_t *taken = plan + a.batch + 1;  // [batch] pages that requests before it take, -1: rejected
    kvc::grid_dep_wait();
    const int64_t depth = a.stack.depth(a.status), capacity = (int64_t)a.max_pages * a.page_size;
    const bool writer = blockIdx.x == 0;
    int64_t tokens_before = 0, pages_before = 0, left = depth;
    if (threadIdx.x == 0)
        begin[0] = 0;
    for (int b0 = 0; b0 < a.batch; b0 += kPlanThreads) {
        const int b = b0 + threadIdx.x;
        int64_t P = 0, n = 0;
        uint32_t bad = 0;
        if (b < a.batch) {
            P = a.cached[b];
            n = a.fresh[b];
            if (P < 0 || n < 0 || P + n > INT32_MAX) {
                bad = KVC_DEV_SEQLEN_RANGE;
                P = n = 0;
            }
        }
        int64_t total;
        const int64_t end = tokens_before + block_scan(n, sums, total);
        tokens_before += total;
        int64_t want = 0;
        if (b < a.batch && !bad) {
            if (P + n > capacity || (n > 0 && end > a.tokens)) {
                bad = KVC_DEV_CAPACITY;
            } else if (n > 0 && P % a.page_size) {
                // new tokens go on in a page that the request holds
                const int32_t id = a.table[(int64_t)b * a.max_pages + P / a.page_size];
                if (id < 0 || id >= a.stack.n_pool)
                    bad = KVC_DEV_INDEX_OOB;
            }
            if (!bad)
                want = pages_of(P + n, a.page_size) - pages_of(P, a.page_size);
        }
        const int64_t upto = pages_before + block_scan(want, sums, total);
        pages_before += total;
        if (want > 0 && upto > depth)
            bad = KVC_DEV_CAPACITY;
        else if (want > 0)
            left = depth - upto;
        if (b < a.batch) {
            begin[b + 1] = (int32_t)(end < a.tokens ? end : a.tokens);
            taken[b] = bad ? -1 : (int32_t)(upto - want);
            if (writer) {
                if (bad)
                    kvc::raise_status(a.status, bad);
                a.offsets[b + 1] = begin[b + 1];
                a.len.past_abs[b] = a.len.cache_past[b] = bad ? -1 : (int32_t)P;
                a.len.total_abs[b] = a.len.cache_total[b] = bad ? -1 : (int32_t)(P + n);
                a.len.evict[b] = bad ? -1 : 0;
            }
        }
    }
    if (writer) {
        if (threadIdx.x == 0)
            a.offsets[0] = 0;
        // the least that any thread's requests leave (those that take pages are the first of those that want some)
        __shared__ int least;
        if (threadIdx.x == 0)
            least = (int)depth;
        __syncthreads();
        atomicMin(&least, (int)left);
        __syncthreads();
        if (threadIdx.x == 0)
            *a.left = least;
    }
    __syncthreads();

    const int t0 = blockIdx.x * kPlanTokens + threadIdx.x * 4;
    if (t0 >= a.tokens)
        return;
    // the last request that begins at t0 or before (empty ones begin where the next does)
    int lo = 0, hi = a.batch;
    while (hi - lo > 0) {
        const int mid = (lo + hi + 1) >> 1;
        if (begin[mid] <= t0)
            lo = mid;
        else
            hi = mid - 1;
    }
    int b = lo, P = 0;
    if (b < a.batch)
        P = a.cached[b];
    int32_t pos[4], slot[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int t = t0 + e;
        pos[e] = slot[e] = -1;
        if (b < a.batch && t >= begin[b + 1]) {
            do
                ++b;
            while (b < a.batch && t >= begin[b + 1]);
            if (b < a.batch)
                P = a.cached[b];
        }
        if (b >= a.batch || t >= a.tokens || taken[b] < 0)
            continue;
        const int p = P + (t - begin[b]);
        const int j = p / a.page_size, at = p - j * a.page_size;
        const int held = (int)pages_of(P, a.page_size);
        int32_t *entry = a.table + (int64_t)b * a.max_pages + j;
        const int32_t id = j < held ? *entry : a.free_pages[depth - 1 - (taken[b] + (j - held))];
        const bool there = id >= 0 && id < a.stack.n_pool;
        if (!there)
            kvc::raise_status(a.status, KVC_DEV_INDEX_OOB);
        if (j >= held && at == 0)
            *entry = there ? id : -1;
        pos[e] = p;
        slot[e] = there ? id * a.page_size + at : -1;
    }
    if (t0 + 4 <= a.tokens) {
        *reinterpret_cast<int4 *>(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        *reinterpret_cast<int4 *>(a.slots + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
    } else {
        for (int e = 0; t0 + e < a.tokens; ++e) {
            a.positions[t0 + e] = pos[e];
            a.slots[t0 + e] = slot[e];
        }
    }
}

kvc_status check_pages(int batch, int max_pages, int page_size, int64_t n_pool_pages)
{
    if (batch < 0 || max_pages < 1 || page_size < 1 || n_pool_pages < 1)
        return KVC_ERR_SHAPE;
    if (batch > kMaxRequests)
        return KVC_ERR_UNSUPPORTED;
    // slots and lengths are 32-bit
    if ((int64_t)max_pages * page_size > INT32_MAX || n_pool_pages > INT32_MAX || n_pool_pages * page_size > INT32_MAX)
        return KVC_ERR_CAPACITY;
    return KVC_OK;
}

// Asked for at any size: a kernel has 48 KB without, what it holds beside the dynamic part included.  And what the
// most requests take, whatever the call's: another thread's smaller call must not lower it before this one's launch.
template <int BYTES, typename Kernel> bool allow_smem(Kernel kern)
{
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, BYTES) == cudaSuccess;
}
constexpr int words_of_release(int batch) { return batch; }
constexpr int words_of_plan(int batch) { return 2 * batch + 1; }

// --------------------------------------------------------------------------
// rotation tables
// --------------------------------------------------------------------------

constexpr int kMaxPairs = 128;

// What a position adds to each pair's angle, in units of 2^-64 of a turn: the
// angle of position p is p times that modulo 2^64.  The rate is within one unit of
// the speed's, so that the last position, 2^31, is off by 2^-33 of a turn (in
// float32 an angle of 10^5 is known to 2^-7 only, and float64 arithmetic is slow on
// this machine).
struct TurnRates {
    uint64_t per[kMaxPairs];
};
constexpr int64_t kMaxPositions = (int64_t)1 << 31;

// x in [0, 1] in units of 2^-64, modulo 2^64
uint64_t units_of(double x)
{
    const double high = std::ldexp(x, 32), whole = std::floor(high);
    return ((uint64_t)whole << 32) + (uint64_t)std::nearbyint(std::ldexp(high - whole, 32));
}

// Turns a position of `speed` radians a position, the whole ones left out.  1 / 2 pi and
// the product are sums of two float64: with one, an error of 2^-53 of the turns would
// grow with the position (a speed of 8: 17 * 2^-24 radians at 2^31).
uint64_t turns_of(double speed)
{
    constexpr double kInverse = 0x1.45f306dc9c883p-3, kRest = -0x1.6b01ec5417056p-57;  // of 1 / 2 pi
    const double turns = speed * kInverse, error = std::fma(speed, kInverse, -turns) + speed * kRest;
    const uint64_t more = units_of(std::fabs(error) - std::floor(std::fabs(error)));
    return units_of(turns - std::floor(turns)) + (error < 0.0 ? 0 - more : more);
}

// cos and sin of x / 2^32 turns, times `magnitude`, two at a time: the nearest quarter
// turn in whole numbers, the rest u, at most an eighth of a turn, by the Taylor series of sin
// and cos of 2 pi u (terms (2 pi)^k / k!; the first left out are below 2^-29).  With
// sincospif, which reduces its argument again, the 131072 x 64 table took 34 us; one at a
// time, each position's angle a product, in three waves of blocks 14.7; now 11.1 to 12.2, 81
// to 89 % of the copy rate.
__device__ __forceinline__ void turns2(const uint32_t (&x)[2], float magnitude, float *c, float *s)
{
    using kvc_tc::fma2;
    using kvc_tc::mul2;
    uint32_t q[2];
    float v[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        q[e] = (x[e] + (1u << 29)) >> 30;
        v[e] = (float)(int32_t)(x[e] - (q[e] << 30));
    }
    auto both = [](float k) { return make_float2(k, k); };
    const float2 u = mul2(make_float2(v[0], v[1]), both(0x1p-32f)), z = mul2(u, u);
    float2 sn = both(42.0586939f), cs = both(-26.4262568f);
    sn = fma2(sn, z, both(-76.7058598f));
    sn = fma2(sn, z, both(81.6052493f));
    sn = fma2(sn, z, both(-41.3417022f));
    sn = mul2(fma2(sn, z, both(6.28318531f)), u);
    cs = fma2(cs, z, both(60.2446414f));
    cs = fma2(cs, z, both(-85.4568172f));
    cs = fma2(cs, z, both(64.939394f));
    cs = fma2(cs, z, both(-19.7392088f));
    cs = fma2(cs, z, both(1.f));
    sn = mul2(sn, both(magnitude));
    cs = mul2(cs, both(magnitude));
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        // an odd number of quarter turns exchanges the two; one or two of them make the cosine negative, two or
        // three the sine
        const float a = e ? sn.y : sn.x, b = e ? cs.y : cs.x;
        const uint32_t flip_c = (q[e] + 1u) << 30 & 0x80000000u, flip_s = q[e] << 30 & 0x80000000u;
        c[e] = __uint_as_float(__float_as_uint(q[e] & 1u ? a : b) ^ flip_c);
        s[e] = __uint_as_float(__float_as_uint(q[e] & 1u ? b : a) ^ flip_s);
    }
}

// VEC columns a thread, of every `step`-th position: its angles go on by the same steps,
// exactly.
constexpr int kTableBlock = 4 * 256;  // pieces of a block, at least
template <int VEC>
__global__ void __launch_bounds__(256, 6)
rope_tables_kernel(float *__restrict__ cos_t, float *__restrict__ sin_t, int64_t first, int64_t positions, int half,
                   const __grid_constant__ TurnRates rates, float magnitude)
{
    const uint32_t pieces = half / VEC, w = blockIdx.x * blockDim.x + threadIdx.x;
    const uint32_t step = gridDim.x * blockDim.x / pieces, p0 = w / pieces;
    const int i0 = (int)(w - p0 * pieces) * VEC;
    if (p0 >= step)
        return;
    constexpr int N = VEC == 1 ? 2 : VEC;  // (a single column is computed twice)
    uint64_t angle[N], by[N];
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const uint64_t rate = rates.per[i0 + (VEC == 1 ? 0 : e)];
        angle[e] = (uint64_t)(first + p0) * rate + 0x80000000u;  // (rounded to 2^-32 of a turn)
        by[e] = step * rate;
    }
#pragma unroll 1
    for (int64_t p = p0; p < positions; p += step) {
        float c[N], s[N];
#pragma unroll
        for (int e = 0; e < N; e += 2) {
            const uint32_t x[2] = {(uint32_t)(angle[e] >> 32), (uint32_t)(angle[e + 1] >> 32)};
            turns2(x, magnitude, c + e, s + e);
            angle[e] += by[e];
            angle[e + 1] += by[e + 1];
        }
        const int64_t at = p * half + i0;
        if constexpr (VEC == 4) {
            *reinterpret_cast<float4 *>(cos_t + at) = make_float4(c[0], c[1], c[2], c[3]);
            *reinterpret_cast<float4 *>(sin_t + at) = make_float4(s[0], s[1], s[2], s[3]);
        } else {
            cos_t[at] = c[0];
            sin_t[at] = s[0];
        }
    }
}

// --------------------------------------------------------------------------
// norm, rotation and append
// --------------------------------------------------------------------------

struct AppendArgs {
    void *q_out, *k_pool, *v_pool;
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;  // elements from token to token
    const void *q_weight, *k_weight;       // NULL: no norm
    float eps;
    const int32_t *positions, *slots;
    int tokens, q_heads, kv_heads, D, page_size;
    int64_t rows;  // of the pool: pages * page_size
    int turned;    // columns rotated
    int interleaved;
    const float *cos_t, *sin_t;
    int64_t rope_max_pos;
    int part;      // of a token's rows, that a block has (gridDim.y parts)
    int32_t *status;
};

// two 16-bit values -> float32, and back
template <typename T> __device__ __forceinline__ float2 unpack2(uint32_t w)
{
    if constexpr (std::is_same<T, __half>::value)
        return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    else
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// A row (one head of one token) is LPR lanes of eight columns each.  A block holds
// 256 / LPR / share tokens and the same part of each one's rows (its queries, keys and
// values one behind the other), which `share` groups of LPR lanes have between them.  A
// column of a query or key becomes
//     (x cos w + x' sin w') / rms
// with its partner x' (of the lane that holds the pair's other half, or the same
// word), the sine negative for a pair's first; cos w and sin w' are made once for the
// token's rows that a group has (with three rows a group, making them took more
// instructions than the rows).  Products and the sum are rounded separately: without a norm w and 1 / rms
// are 1 and the bits those of the other calls' rotation.  A lane asks for kAhead rows
// before it works on the first (one at a time held the pass to 2.6 TB/s).
// 16384 tokens of 48 rows of 128, normed and rotated: 79 us, 5.2 TB/s or 76 % of the copy
// rate, with 55 % of the issue slots taken; 1543 of 80 rows of 64: 9.4 us; 32 tokens: 3.7.
constexpr int kAhead = 4;
enum Turn { kNoTurn, kHalves, kNeighbours };

template <typename T, int LPR, bool NORM, int TURN>
__device__ __forceinline__ void append_rows(const AppendArgs &a, int first, int end, int step, bool mine, uint32_t peers,
                                            const T *from, T *to, int64_t to_step, bool turns, int other,
                                            const float2 (&cs)[4], const float2 (&sn)[4])
{
    using kvc_tc::add2;
    using kvc_tc::mul2;
    const float by_d = 1.f / (float)a.D;
    const int64_t from_step = (int64_t)a.D * step;
    from += first * (int64_t)a.D;
    to += first * to_step;
    to_step *= step;
    for (int r0 = first; r0 < end; r0 += kAhead * step) {
        uint4 raw[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            raw[u] = make_uint4(0, 0, 0, 0);
            if (mine && r0 + u * step < end)
                raw[u] = *reinterpret_cast<const uint4 *>(from);
            from += from_step;
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u, to += to_step) {
            if (r0 + u * step >= end)
                break;
            if constexpr (NORM || TURN != kNoTurn) {
                uint32_t w[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
                float2 x[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[e] = unpack2<T>(w[e]);
                float by = 1.f;
                if constexpr (NORM) {
                    float2 s2 = mul2(x[0], x[0]);
#pragma unroll
                    for (int e = 1; e < 4; ++e)
                        s2 = kvc_tc::fma2(x[e], x[e], s2);
                    float sum = s2.x + s2.y;
#pragma unroll
                    for (int d = LPR / 2; d; d >>= 1)
                        sum += __shfl_xor_sync(peers, sum, d, LPR);
                    by = rsqrtf(fmaf(sum, by_d, a.eps));
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float2 z = mul2(x[e], cs[e]);
                    if constexpr (TURN != kNoTurn) {
                        const uint32_t o = TURN == kHalves ? __shfl_sync(peers, w[e], other, LPR) : __byte_perm(w[e], 0, 0x1032);
                        // (a column that is not turned has no partner)
                        z = add2(z, mul2(unpack2<T>(turns ? o : 0u), sn[e]));
                    }
                    if constexpr (NORM)
                        z = mul2(z, make_float2(by, by));
                    const uint32_t y = kvc_tc::pack2<T>(z.x, z.y);
                    w[e] = NORM || turns ? y : w[e];
                }
                raw[u] = make_uint4(w[0], w[1], w[2], w[3]);
            }
            if (mine)
                *reinterpret_cast<uint4 *>(to) = raw[u];
        }
    }
}

template <typename T, int LPR>
__global__ void __launch_bounds__(256, 4)
ragged_append_kernel(const AppendArgs a, int share)
{
    const int group = threadIdx.x / LPR, lane = threadIdx.x % LPR;
    const int t = blockIdx.x * (256 / LPR / share) + group / share;
    const int c0 = lane * 8;
    // (a warp's groups may be at different tokens)
    const uint32_t peers = LPR == 32 ? 0xffffffffu : ((1u << (LPR & 31)) - 1u) << (threadIdx.x & 31 & ~(LPR - 1));
    const int r0 = blockIdx.y * a.part, r1 = min(r0 + a.part, a.q_heads + 2 * a.kv_heads);  // of the token's rows
    const int lead = group % share;
    kvc::grid_dep_wait();
    const int slot = t < a.tokens ? a.slots[t] : -1;
    const int pos = t < a.tokens ? a.positions[t] : -1;
    if (slot < 0)
        return;
    const uint32_t bad = (slot >= a.rows ? KVC_DEV_INDEX_OOB : 0u) |
                         (a.cos_t && (pos < 0 || pos >= a.rope_max_pos) ? KVC_DEV_ROPE_RANGE : 0u);
    if (bad) {
        if (lane == 0)
            kvc::raise_status(a.status, bad);
        return;
    }
    const bool mine = c0 < a.D;
    const int half = a.turned / 2;
    const bool turns = a.cos_t && c0 < a.turned;  // (a multiple of 16: whole lanes turn or stay)
    const bool low = c0 < half;
    // the lane that holds the other half of this one's pairs
    const int other = a.interleaved || !turns ? lane : low ? lane + half / 8 : lane - half / 8;
    auto factors = [&](const void *weight, float2 (&cs)[4], float2 (&sn)[4]) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            cs[e] = make_float2(1.f, 1.f);
            sn[e] = make_float2(0.f, 0.f);
        }
        if (turns && a.interleaved) {
            const int64_t at = (int64_t)pos * half + c0 / 2;
            const float4 x = *reinterpret_cast<const float4 *>(a.cos_t + at);
            const float4 y = *reinterpret_cast<const float4 *>(a.sin_t + at);
            cs[0] = make_float2(x.x, x.x), cs[1] = make_float2(x.y, x.y), cs[2] = make_float2(x.z, x.z), cs[3] = make_float2(x.w, x.w);
            sn[0] = make_float2(-y.x, y.x), sn[1] = make_float2(-y.y, y.y), sn[2] = make_float2(-y.z, y.z), sn[3] = make_float2(-y.w, y.w);
        } else if (turns) {
            const int64_t at = (int64_t)pos * half + (low ? c0 : c0 - half);
            const float sign = low ? -1.f : 1.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float4 x = *reinterpret_cast<const float4 *>(a.cos_t + at + 4 * e);
                const float4 y = *reinterpret_cast<const float4 *>(a.sin_t + at + 4 * e);
                cs[2 * e] = make_float2(x.x, x.y), cs[2 * e + 1] = make_float2(x.z, x.w);
                sn[2 * e] = make_float2(sign * y.x, sign * y.y), sn[2 * e + 1] = make_float2(sign * y.z, sign * y.w);
            }
        }
        if (weight) {
            uint4 w4 = make_uint4(0, 0, 0, 0);
            if (mine)
                w4 = *reinterpret_cast<const uint4 *>(static_cast<const T *>(weight) + c0);
            const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t o = a.interleaved ? __byte_perm(w[e], 0, 0x1032) : __shfl_sync(peers, w[e], other, LPR);
                cs[e] = kvc_tc::mul2(cs[e], unpack2<T>(w[e]));
                // (a column that is not turned keeps its zero: that times an infinite weight is none)
                if (turns)
                    sn[e] = kvc_tc::mul2(sn[e], unpack2<T>(o));
            }
        }
    };
    const int page = slot / a.page_size, in_page = slot - page * a.page_size;
    const int64_t kv_to = ((int64_t)page * a.kv_heads * a.page_size + in_page) * a.D + c0, kv_step = (int64_t)a.page_size * a.D;
    const int k0 = a.q_heads, v0 = k0 + a.kv_heads;
#pragma unroll 1
    for (int kind = 0; kind < 3; ++kind) {
        // the block's rows of the token's queries, keys or values
        const int from = kind == 0 ? 0 : kind == 1 ? k0 : v0, to = kind == 0 ? k0 : kind == 1 ? v0 : v0 + a.kv_heads;
        const int begin = max(r0, from) - from + lead, end = min(r1, to) - from;
        if (r0 >= to || r1 <= from)
            continue;
        const T *src = kind == 0   ? static_cast<const T *>(a.q) + t * a.q_stride
                       : kind == 1 ? static_cast<const T *>(a.k) + t * a.k_stride
                                   : static_cast<const T *>(a.v) + t * a.v_stride;
        T *dst = kind == 0   ? static_cast<T *>(a.q_out) + (int64_t)t * a.q_heads * a.D + c0
                 : kind == 1 ? static_cast<T *>(a.k_pool) + kv_to
                             : static_cast<T *>(a.v_pool) + kv_to;
        const int64_t dst_step = kind == 0 ? a.D : kv_step;
        const void *weight = kind == 0 ? a.q_weight : kind == 1 ? a.k_weight : nullptr;
        float2 cs[4], sn[4];
        auto run = [&](auto norm, auto turn) {
            append_rows<T, LPR, decltype(norm)::value, decltype(turn)::value>(a, begin, end, share, mine, peers, src + c0, dst,
                                                                              dst_step, turns, other, cs, sn);
        };
        using std::integral_constant;
        if (kind == 2 || (!weight && !a.cos_t)) {
            run(std::false_type{}, integral_constant<int, kNoTurn>{});
            continue;
        }
        factors(weight, cs, sn);
        if (!a.cos_t)
            run(std::true_type{}, integral_constant<int, kNoTurn>{});
        else if (a.interleaved && weight)
            run(std::true_type{}, integral_constant<int, kNeighbours>{});
        else if (a.interleaved)
            run(std::false_type{}, integral_constant<int, kNeighbours>{});
        else if (weight)
            run(std::true_type{}, integral_constant<int, kHalves>{});
        else
            run(std::false_type{}, integral_constant<int, kHalves>{});
    }
}

template <typename T> cudaError_t launch_append(const AppendArgs &a, cudaStream_t stream)
{
    const int rows = a.q_heads + 2 * a.kv_heads;
    int lpr = 2;
    while (lpr * 8 < a.D)
        lpr *= 2;
    const int groups = 256 / lpr, sms = kvc_host::sm_count();
    // Rows of a group: as few as make three blocks an SM, or all of a token's (rows are taken four at a time, and a
    // group makes cos, sin and weights once; a dozen at most and four blocks, rounded down, took 83 for 79 us with 16384
    // tokens of 48 rows, 13.2 for 9.3 with 1543 of 80, 7.9 for 5.7 with 512 of 48, 3.7 with 32 either way).  Where
    // blocks of whole tokens leave the last wave of four an SM mostly empty, 24 at most (12000 tokens of 48: 67 -> 60 us).
    // The groups of a token in parts of its rows, at least three where there are that many groups, so that most
    // have to do with one kind alone.
    const int64_t wanted = (int64_t)groups * 3 * sms, blocks = (a.tokens + (int64_t)groups - 1) / groups, wave = 4 * sms;
    const bool uneven = blocks > wave && 10 * blocks < 7 * ((blocks + wave - 1) / wave * wave);
    const int most = uneven ? std::min(rows, 24) : rows;
    const int each = (int)std::max<int64_t>(1, std::min<int64_t>(most, ((int64_t)a.tokens * rows + wanted - 1) / wanted));
    int share = 1;
    while (share < groups && 2 * share * 3 * each <= rows)
        share *= 2;
    const int per_block = groups / share;
    AppendArgs b = a;
    const int parts = (rows + share * each - 1) / (share * each);
    b.part = (rows + parts - 1) / parts;
    const dim3 grid((a.tokens + per_block - 1) / per_block, (rows + b.part - 1) / b.part);
    switch (lpr) {
    case 2:
        return kvc_host::launch_chained(ragged_append_kernel<T, 2>, grid, 256, 0, stream, b, share);
    case 4:
        return kvc_host::launch_chained(ragged_append_kernel<T, 4>, grid, 256, 0, stream, b, share);
    case 8:
        return kvc_host::launch_chained(ragged_append_kernel<T, 8>, grid, 256, 0, stream, b, share);
    case 16:
        return kvc_host::launch_chained(ragged_append_kernel<T, 16>, grid, 256, 0, stream, b, share);
    default:
        return kvc_host::launch_chained(ragged_append_kernel<T, 32>, grid, 256, 0, stream, b, share);
    }
}

} // namespace

KVC_API kvc_status kvc_page_release(const int32_t *released, const int32_t *block_table, int max_pages, int page_size,
                                    int32_t *free_pages, int64_t n_pool_pages, const int32_t *free_count,
                                    int32_t *free_left, int batch, int32_t *dev_status, void *stream_)
{
    const kvc_status st = check_pages(batch, max_pages, page_size, n_pool_pages);
    if (st != KVC_OK)
        return st;
    if (!free_pages || !free_count || !free_left || (batch > 0 && (!released || !block_table)))
        return KVC_ERR_NULL;
    const size_t rows = (size_t)batch * sizeof(int32_t), one = sizeof(int32_t);
    if (kvc_host::collide({{free_pages, n_pool_pages * one}, {free_left, one}},
                          {{released, rows}, {block_table, rows * max_pages}, {free_count, one}}))
        return KVC_ERR_SHAPE;
    const ReleaseArgs a{released, block_table, max_pages, page_size, free_pages, {free_count, n_pool_pages}, free_left,
                        batch, dev_status};
    const size_t smem = words_of_release(batch) * sizeof(int32_t);
    if (!allow_smem<words_of_release(kMaxRequests) * (int)sizeof(int32_t)>(page_release_kernel))
        return kvc_host::cuda_failed();
    const int warps = kPlanThreads / 32;
    const int grid = std::max(1, std::min((batch + warps - 1) / warps, kvc_host::sm_count()));
    if (kvc_host::launch_chained(page_release_kernel, dim3(grid), kPlanThreads, smem, static_cast<cudaStream_t>(stream_), a) !=
        cudaSuccess)
        return kvc_host::cuda_failed();
    return kvc_host::launch_status();
}

KVC_API kvc_status kvc_ragged_plan(const int32_t *cached, const int32_t *new_tokens, int32_t *block_table,
                                   int max_pages, int page_size, const int32_t *free_pages, int64_t n_pool_pages,
                                   const int32_t *free_count, int32_t *free_left, int batch, int tokens,
                                   int32_t *offsets, kvc_lengths len, int32_t *positions, int32_t *slots,
                                   int32_t *dev_status, void *stream_)
{
    const kvc_status st = check_pages(batch, max_pages, page_size, n_pool_pages);
    if (st != KVC_OK)
        return st;
    if (tokens < 0)
        return KVC_ERR_SHAPE;
    if (tokens > kMaxTokens)
        return KVC_ERR_CAPACITY;
    if (!free_pages || !free_count || !free_left || !offsets || (tokens > 0 && (!positions || !slots)) ||
        (batch > 0 && (!cached || !new_tokens || !block_table || !kvc_host::lengths_ok(len))))
        return KVC_ERR_NULL;
    if (!kvc_host::aligned16(positions) || !kvc_host::aligned16(slots))
        return KVC_ERR_ALIGN;
    // (every block reads what the requests hold and bring, block 0 writes: a step's `cached` may not be the lengths
    // that the step before wrote into the same plan)
    const size_t rows = (size_t)batch * sizeof(int32_t), one = sizeof(int32_t), places = tokens * one;
    const std::initializer_list<kvc_host::Span> read = {
        {cached, rows}, {new_tokens, rows}, {free_pages, n_pool_pages * one}, {free_count, one}};
    if (kvc_host::collide({{block_table, rows * max_pages}, {offsets, rows + one}, {positions, places}, {slots, places},
                           {free_left, one}}, read))
        return KVC_ERR_SHAPE;
    for (const void *p : {len.past_abs, len.cache_past, len.total_abs, len.cache_total, len.evict})
        if (kvc_host::collide({{p, rows}}, read) ||
            kvc_host::collide({{p, rows}}, {{block_table, rows * max_pages}, {offsets, rows + one}, {positions, places},
                                            {slots, places}, {free_left, one}}))
            return KVC_ERR_SHAPE;
    const PlanArgs a{cached, new_tokens, block_table, max_pages, page_size, free_pages, {free_count, n_pool_pages},
                     free_left, batch, tokens, offsets, len, positions, slots, dev_status};
    const size_t smem = words_of_plan(batch) * sizeof(int32_t);
    if (!allow_smem<words_of_plan(kMaxRequests) * (int)sizeof(int32_t)>(ragged_plan_kernel))
        return kvc_host::cuda_failed();
    const int grid = std::max(1, (int)(((int64_t)tokens + kPlanTokens - 1) / kPlanTokens));
    if (kvc_host::launch_chained(ragged_plan_kernel, dim3(grid), kPlanThreads, smem, static_cast<cudaStream_t>(stream_), a) !=
        cudaSuccess)
        return kvc_host::cuda_failed();
    return kvc_host::launch_status();
}

KVC_API kvc_status kvc_rope_tables(float *cos_table, float *sin_table, int64_t first, int64_t positions,
                                   int rotary_dim, double base, int scaling, double factor, int64_t trained, double low,
                                   double high, double magnitude, void *stream_)
{
    if (positions < 0 || positions > INT32_MAX || first < 0 || first > kMaxPositions - positions || rotary_dim < 2 || rotary_dim % 2)
        return KVC_ERR_SHAPE;
    if (rotary_dim > 2 * kMaxPairs || scaling < KVC_ROPE_PLAIN || scaling > KVC_ROPE_PARTS)
        return KVC_ERR_UNSUPPORTED;
    if (!(base > 0.0) || !std::isfinite(base) || !std::isfinite((float)magnitude))
        return KVC_ERR_SHAPE;
    if (scaling != KVC_ROPE_PLAIN && (!(factor > 0.0) || !std::isfinite(factor)))
        return KVC_ERR_SHAPE;
    if (scaling == KVC_ROPE_BASE && rotary_dim == 2)
        return KVC_ERR_SHAPE;
    if (scaling == KVC_ROPE_PARTS && (trained < 1 || !(low < high) || !std::isfinite(low) || !std::isfinite(high)))
        return KVC_ERR_SHAPE;
    if (positions == 0)
        return KVC_OK;
    if (!cos_table || !sin_table)
        return KVC_ERR_NULL;
    if ((reinterpret_cast<uintptr_t>(cos_table) | reinterpret_cast<uintptr_t>(sin_table)) & 3u)
        return KVC_ERR_ALIGN;
    const int half = rotary_dim / 2;
    const size_t bytes = (size_t)positions * half * sizeof(float);
    if (kvc_host::overlaps(cos_table, bytes, sin_table, bytes))
        return KVC_ERR_SHAPE;
    constexpr double kTurn = 6.283185307179586476925286766559;
    if (scaling == KVC_ROPE_BASE)
        base *= std::pow(factor, (double)rotary_dim / (rotary_dim - 2));
    TurnRates rates{};
    for (int i = 0; i < half; ++i) {
        double speed = std::pow(base, -2.0 * i / rotary_dim);
        if (scaling == KVC_ROPE_LINEAR) {
            speed /= factor;
        } else if (scaling == KVC_ROPE_PARTS) {
            const double keep = std::min(1.0, std::max(0.0, (trained * (speed / kTurn) - low) / (high - low)));
            speed = speed * keep + speed / factor * (1.0 - keep);
        }
        if (!std::isfinite(speed))
            return KVC_ERR_SHAPE;
        rates.per[i] = turns_of(speed);
    }
    const int vec = half % 4 == 0 && kvc_host::aligned16(cos_table) && kvc_host::aligned16(sin_table) ? 4 : 1;
    // as many blocks as run at once, and four positions a thread before that (8192 x 64: one 4.0, two 3.1, four 3.0,
    // eight 3.8 us; a thread's rates are as much work as a position)
    const int64_t blocks = std::min<int64_t>((positions * (half / vec) + kTableBlock - 1) / kTableBlock, 6 * kvc_host::sm_count());
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    if (vec == 4)
        rope_tables_kernel<4><<<(unsigned)blocks, 256, 0, stream>>>(cos_table, sin_table, first, positions, half, rates,
                                                                    (float)magnitude);
    else
        rope_tables_kernel<1><<<(unsigned)blocks, 256, 0, stream>>>(cos_table, sin_table, first, positions, half, rates,
                                                                    (float)magnitude);
    return kvc_host::launch_status();
}

KVC_API kvc_status kvc_ragged_append(void *q_out, void *k_pool, void *v_pool, const void *q, const void *k,
                                     const void *v, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                                     const void *q_weight, const void *k_weight, float eps, const int32_t *positions,
                                     const int32_t *slots, int tokens, int q_heads, int kv_heads, int64_t n_pool_pages,
                                     int page_size, int head_dim, int dtype, int rotary_dim, int interleaved,
                                     const float *rope_cos, const float *rope_sin, int64_t rope_max_pos,
                                     int32_t *dev_status, void *stream_)
{
    if (kvc_host::elem_bytes_of(dtype) == 0)
        return KVC_ERR_DTYPE;
    if (dtype == KVC_F32)
        return KVC_ERR_UNSUPPORTED;
    if (tokens < 0 || q_heads < 1 || kv_heads < 1 || n_pool_pages < 1 || page_size < 1 || head_dim < 1)
        return KVC_ERR_SHAPE;
    if (head_dim % 16 || head_dim > 256 || q_heads > 32767 || kv_heads > 32767)
        return KVC_ERR_UNSUPPORTED;
    if (n_pool_pages > INT32_MAX || n_pool_pages * page_size > INT32_MAX || tokens > kMaxTokens)
        return KVC_ERR_CAPACITY;
    if ((rope_cos == nullptr) != (rope_sin == nullptr))
        return KVC_ERR_NULL;
    if (rope_cos) {
        if (rope_max_pos < 1 || rotary_dim < 2 || rotary_dim > head_dim)
            return KVC_ERR_SHAPE;
        if (rotary_dim % 16)
            return KVC_ERR_UNSUPPORTED;
    }
    if ((q_weight || k_weight) && !(eps >= 0.f && std::isfinite(eps)))
        return KVC_ERR_SHAPE;
    const int64_t q_row = (int64_t)q_heads * head_dim, kv_row = (int64_t)kv_heads * head_dim;
    if (tokens > 1 && (q_stride < q_row || k_stride < kv_row || v_stride < kv_row))
        return KVC_ERR_SHAPE;
    if (tokens == 0)
        return KVC_OK;
    if (!q_out || !k_pool || !v_pool || !q || !k || !v || !positions || !slots)
        return KVC_ERR_NULL;
    for (const void *p : {(const void *)q_out, (const void *)k_pool, (const void *)v_pool, q, k, v, q_weight, k_weight,
                          (const void *)rope_cos, (const void *)rope_sin})
        if (p && !kvc_host::aligned16(p))
            return KVC_ERR_ALIGN;
    if (tokens > 1 && (q_stride % 8 || k_stride % 8 || v_stride % 8))
        return KVC_ERR_ALIGN;
    if (tokens == 1)
        q_stride = q_row, k_stride = v_stride = kv_row;
    if (q_stride > INT64_MAX / 4 / tokens || k_stride > INT64_MAX / 4 / tokens || v_stride > INT64_MAX / 4 / tokens)
        return KVC_ERR_SHAPE;
    // what is written shares no bytes with what is read (q_out == q, packed alike, is the one way in place)
    const size_t pool = (size_t)n_pool_pages * page_size * kv_row * 2, out = (size_t)tokens * q_row * 2;
    const size_t q_bytes = ((size_t)(tokens - 1) * q_stride + q_row) * 2,
                 k_bytes = ((size_t)(tokens - 1) * k_stride + kv_row) * 2,
                 v_bytes = ((size_t)(tokens - 1) * v_stride + kv_row) * 2;
    const bool in_place = q_out == q && q_stride == q_row;
    if (kvc_host::overlaps(k_pool, pool, v_pool, pool) || kvc_host::overlaps(q_out, out, k_pool, pool) ||
        kvc_host::overlaps(q_out, out, v_pool, pool) || (!in_place && kvc_host::overlaps(q_out, out, q, q_bytes)) ||
        kvc_host::overlaps(q_out, out, k, k_bytes) || kvc_host::overlaps(q_out, out, v, v_bytes))
        return KVC_ERR_SHAPE;
    for (const void *p : {(const void *)k_pool, (const void *)v_pool})
        if (kvc_host::overlaps(p, pool, q, q_bytes) || kvc_host::overlaps(p, pool, k, k_bytes) ||
            kvc_host::overlaps(p, pool, v, v_bytes))
            return KVC_ERR_SHAPE;
    // (positions are 32-bit: no row of the tables past 2^31 is read)
    const size_t list = tokens * sizeof(int32_t), weight = head_dim * 2,
                 table = rope_cos ? (size_t)std::min<int64_t>(rope_max_pos, (int64_t)1 << 31) * (rotary_dim / 2) * 4 : 0;
    for (const kvc_host::Span &w : {kvc_host::Span{q_out, out}, kvc_host::Span{k_pool, pool}, kvc_host::Span{v_pool, pool}})
        if (kvc_host::collide({w}, {{positions, list}, {slots, list}, {rope_cos, table}, {rope_sin, table},
                                    {q_weight, q_weight ? weight : 0}, {k_weight, k_weight ? weight : 0}}))
            return KVC_ERR_SHAPE;
    const AppendArgs a{q_out, k_pool, v_pool, q, k, v, q_stride, k_stride, v_stride, q_weight, k_weight, eps, positions,
                       slots, tokens, q_heads, kv_heads, head_dim, page_size, n_pool_pages * page_size,
                       rope_cos ? rotary_dim : 0, interleaved, rope_cos, rope_sin, rope_max_pos, 1, dev_status};
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    if ((dtype == KVC_BF16 ? launch_append<__nv_bfloat16>(a, stream) : launch_append<__half>(a, stream)) != cudaSuccess)
        return kvc_host::cuda_failed();
    return kvc_host::launch_status();
}
