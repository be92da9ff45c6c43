// kvc_tree.cu -- a tree of drafted tokens verified over a persistent cache
// ("Persistent KV Cache and Decode Performance Roadmap", "Phase 1" and
// "Phase 2": grouped-query attention over a contiguous or paged cache).
//
// N drafted tokens follow the P tokens of a cache as a tree: node i continues
// its parent's line, so it stands at position P + depth_i and sees the cache,
// its ancestors and itself, whatever the row its key lies in (P + i).  After
// the model has judged the drafts, one line of the tree is kept.
//
//   tree_mask_kernel     parents -> ancestor bits and depths
//   tree_append_kernel   the drafts' K/V rows at rows [P, P + N), K rotated at
//                        P + depth
//   tree_attn_kernel     the attention of the N drafts
//   tree_commit_kernel   the kept line's rows to [P, P + n), the next seqlens_k
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "kvc_common.cuh"
#include "kvc_flat.cuh"
#include "kvc_tc.cuh"

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxNodes = 256;
constexpr int kAbsent = -2;   // parent of a node that is not there

// where the rows of a cache lie: [B, kv_heads, rows, D], or pages of a pool
struct CacheRows {
    const int32_t *table;  // NULL: contiguous
    int max_pages, page_size;
    int64_t n_pool, rows;  // rows: capacity (contiguous) or max_pages * page_size
};

// element offset of row r of (batch row b, kv head h); the caller has checked
// that r < rows and (paged) that the page exists
__device__ __forceinline__ int64_t row_index(const CacheRows &c, int b, int h, int kv_heads, int64_t r)
{
    if (!c.table)
        return ((int64_t)b * kv_heads + h) * c.rows + r;
    const int64_t id = c.table[(int64_t)b * c.max_pages + r / c.page_size];
    return (id * kv_heads + h) * c.page_size + r % c.page_size;
}

// the pages of rows [r0, r1) all name pages of the pool
__device__ __forceinline__ bool pages_ok(const CacheRows &c, int b, int64_t r0, int64_t r1)
{
    if (!c.table || r1 <= r0)
        return true;
    for (int64_t p = r0 / c.page_size; p <= (r1 - 1) / c.page_size; ++p) {
        const int64_t id = c.table[(int64_t)b * c.max_pages + p];
        if (id < 0 || id >= c.n_pool)
            return false;
    }
    return true;
}

// --------------------------------------------------------------------------
// parents -> masks and depths
// --------------------------------------------------------------------------

// One block a batch row, one thread a node: a node's parent comes before it,
// so the walk to the root ends after at most i steps.
__global__ void __launch_bounds__(kMaxNodes)
tree_mask_kernel(const int32_t *__restrict__ parents, int nodes, uint32_t *__restrict__ mask,
                 int32_t *__restrict__ depth, int32_t *status)
{
    __shared__ int32_t up[kMaxNodes];
    __shared__ uint32_t bits[kMaxNodes][kMaxNodes / 32];
    const int b = blockIdx.x, i = threadIdx.x;
    const int words = (nodes + 31) / 32;
    if (i < nodes) {
        int p = parents[(int64_t)b * nodes + i];
        if (p < kAbsent || p >= i) {
            kvc::raise_status(status, KVC_DEV_INDEX_OOB);
            p = kAbsent;
        }
        up[i] = p;
        for (int w = 0; w < words; ++w)
            bits[i][w] = 0;
    }
    __syncthreads();
    if (i >= nodes)
        return;
    int d = -1, p = i;
    for (; p >= 0; p = up[p]) {
        bits[i][p >> 5] |= 1u << (p & 31);
        ++d;
    }
    // a line that ends at an absent node is absent
    const bool there = p == -1;
    depth[(int64_t)b * nodes + i] = there ? d : -1;
    for (int w = 0; w < words; ++w)
        mask[((int64_t)b * nodes + i) * words + w] = there ? bits[i][w] : 0;
}

// --------------------------------------------------------------------------
// append
// --------------------------------------------------------------------------

struct TreeRows {
    void *k, *v;
    const void *new_k, *new_v;
    const int32_t *depth;
    CacheRows at;
    kvc_lengths len;
    int batch, kv_heads, nodes, D;
    const float *cos_t, *sin_t;
    int64_t rope_max_pos;
    int32_t *status;
};

// eight columns of one row of K and of V a thread; the rotation's other half
// is read again by the thread that needs it
template <typename T>
__global__ void __launch_bounds__(128)
tree_append_kernel(const TreeRows a)
{
    const int h = blockIdx.y, b = blockIdx.z;
    const int P = a.len.past_abs[b];
    if (a.len.cache_total[b] < 0 || P < 0)
        return;
    const bool lead = threadIdx.x == 0 && blockIdx.x == 0 && h == 0;
    if (a.cos_t && (int64_t)P + a.nodes > a.rope_max_pos) {
        if (lead)
            kvc::raise_status(a.status, KVC_DEV_ROPE_RANGE);
        return;
    }
    if ((int64_t)P + a.nodes > a.at.rows) {
        if (lead)
            kvc::raise_status(a.status, KVC_DEV_CAPACITY);
        return;
    }
    if (!pages_ok(a.at, b, P, (int64_t)P + a.nodes)) {
        if (lead)
            kvc::raise_status(a.status, KVC_DEV_INDEX_OOB);
        return;
    }
    const int pieces = a.D / 8, half = a.D / 2;
    for (int w = blockIdx.x * blockDim.x + threadIdx.x; w < a.nodes * pieces; w += gridDim.x * blockDim.x) {
        const int i = w / pieces, c0 = (w % pieces) * 8;
        const int d = a.depth[(int64_t)b * a.nodes + i];
        if (d < 0 || d >= a.nodes) {
            if (d >= a.nodes)
                kvc::raise_status(a.status, KVC_DEV_INDEX_OOB);
            continue;
        }
        const int64_t src = (((int64_t)b * a.kv_heads + h) * a.nodes + i) * a.D;
        const int64_t dst = row_index(a.at, b, h, a.kv_heads, (int64_t)P + i) * a.D;
        const T *nk = static_cast<const T *>(a.new_k) + src;
        uint4 k = *reinterpret_cast<const uint4 *>(nk + c0);
        const uint4 v = *reinterpret_cast<const uint4 *>(static_cast<const T *>(a.new_v) + src + c0);
        if (a.cos_t) {
            const bool low = c0 < half;
            const int p0 = low ? c0 : c0 - half;
            const uint4 o = *reinterpret_cast<const uint4 *>(nk + (low ? c0 + half : c0 - half));
            T *x = reinterpret_cast<T *>(&k);
            const T *y = reinterpret_cast<const T *>(&o);
            const float *cs = a.cos_t + ((int64_t)P + d) * half + p0, *sn = a.sin_t + ((int64_t)P + d) * half + p0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float mine = kvc::Elem<T>::to_f32(x[e]), other = kvc::Elem<T>::to_f32(y[e]);
                float lo = low ? mine : other, hi = low ? other : mine;
                kvc::rope_pair(lo, hi, cs[e], sn[e]);
                x[e] = kvc::Elem<T>::from_f32(low ? lo : hi);
            }
        }
        *reinterpret_cast<uint4 *>(static_cast<T *>(a.k) + dst + c0) = k;
        *reinterpret_cast<uint4 *>(static_cast<T *>(a.v) + dst + c0) = v;
    }
}

// --------------------------------------------------------------------------
// commit
// --------------------------------------------------------------------------

struct CommitArgs {
    void *k, *v;
    const int32_t *path, *accepted;
    int path_len;
    CacheRows at;
    kvc_lengths len;
    int32_t *seqlens;
    int kv_heads, nodes, row_vecs;  // row_vecs: 16-byte pieces of a row
    int32_t *status;
};

// A thread owns one 16-byte column of a (batch row, head, K or V) and moves
// rows P + path[j] to P + j for j = 0, 1, ...: path[j] >= j and path ascends,
// so the row read at step j has not been written by an earlier step.  Rows
// are read kBatch ahead of their stores, which keeps that order.
__global__ void __launch_bounds__(64)
tree_commit_kernel(const CommitArgs a)
{
    constexpr int kBatch = 8;
    __shared__ int32_t path[kMaxNodes];
    const int h = blockIdx.x >> 1, b = blockIdx.y;
    const bool is_v = blockIdx.x & 1;
    const int P = a.len.past_abs[b];
    if (a.len.cache_total[b] < 0 || P < 0)
        return;
    const bool lead = threadIdx.x == 0 && blockIdx.x == 0;
    const int n = a.accepted[b];
    bool ok = n >= 0 && n <= a.path_len && n <= a.nodes;
    if (ok)
        for (int j = threadIdx.x; j < n; j += blockDim.x) {
            const int at = a.path[(int64_t)b * a.path_len + j];
            const int before = j ? a.path[(int64_t)b * a.path_len + j - 1] : -1;
            path[j] = at;
            ok = ok && at > before && at >= j && at < a.nodes;
        }
    ok = __syncthreads_and(ok);
    const bool fits = (int64_t)P + a.nodes <= a.at.rows;
    if (!ok || !fits || !pages_ok(a.at, b, P, (int64_t)P + a.nodes)) {
        if (lead)
            kvc::raise_status(a.status, fits ? KVC_DEV_INDEX_OOB : KVC_DEV_CAPACITY);
        return;
    }
    if (lead)
        a.seqlens[b] = P + n - 1;
    uint4 *rows = static_cast<uint4 *>(is_v ? a.v : a.k);
    for (int c = threadIdx.x; c < a.row_vecs; c += blockDim.x) {
        for (int j0 = 0; j0 < n; j0 += kBatch) {
            uint4 x[kBatch];
#pragma unroll
            for (int e = 0; e < kBatch; ++e)
                if (j0 + e < n && path[j0 + e] != j0 + e)
                    x[e] = rows[row_index(a.at, b, h, a.kv_heads, (int64_t)P + path[j0 + e]) * a.row_vecs + c];
#pragma unroll
            for (int e = 0; e < kBatch; ++e)
                if (j0 + e < n && path[j0 + e] != j0 + e)
                    rows[row_index(a.at, b, h, a.kv_heads, (int64_t)P + j0 + e) * a.row_vecs + c] = x[e];
        }
    }
}

// --------------------------------------------------------------------------
// attention
// --------------------------------------------------------------------------
//
// The group's G heads x N nodes are the rows of the query matrix of one (batch
// row, kv head), in tiles of 128: row m is head m / N, node m % N, as they lie
// in memory.  Each (batch row, kv head, row tile) streams its keys past the
// tensor cores in tiles of 128, and every CTA (one an SM) takes the same number
// of key tiles, whatever the lengths (kvc_flat.cuh), in segments of one row
// each; rows that several CTAs worked on are joined by tree_merge_kernel.
// (Keys read once for all rows of a group: 4 G N products for each byte of bf16 keys
// and values.)
//
//   tree_prep_kernel  the queries rotated at their positions, and for each node
//                     the drafts that it sees (mask, window and absences in one)
//   TMEM columns  O [0, D) fp32 | S / P double buffer [D, D + 256)
//   shared        Q (128 x D, 128-byte swizzled) | ring of slabs of 64 or 128 rows
//   warp 0        TMA of the queries and the score products S_0, S_1, ...: S_{j+2}
//                 once PV_j has read the weights in its place
//   warps 1-8     softmax and output: two threads a row (= TMEM lane), each half
//                 of the columns
//   warps 9, 10   TMA producers of K and of V into one ring in the order of use
//                 (K_0, K_1, V_0, K_2, ...), through the next segment's tiles
//                 without a stop
//   warp 11       the output products PV_0, PV_1, ... (one thread that issued all
//                 products in turn was behind the softmax at every tile)
// so that from one segment to the next the stream of keys does not stop: while
// the softmax warps write one segment's output, the next one's first scores are
// on their way.  (With the queries loaded and rotated by the softmax warps
// between segments, each segment cost 22,000 clocks, as much as ten tiles.)
//
// A slab is KR = 128 rows (a whole tile of K or of V) where that is 32 KB at most,
// else 64.  It is one TMA box, or, where a page may end inside a tile, two rows of
// boxes of 64 rows and 64 columns.  (Slabs of 64 rows there made each product one
// of 64 keys, which takes the tensor cores as long as one of 128.)
//
// Three roundings to 16 bits meet in an output: of the rotated query, of the
// weights and of the result, each about as large as the others.  One of the first
// two is taken out with a second product, whose time the tensor cores have to
// spare: with head_dim <= 128 the query is a sum of two 16-bit numbers (two query
// tiles fit beside the ring), with 256 the weights are (their second parts fit
// beside the first in the score columns; they are work for the softmax warps, which
// made head_dim 128 slower that way: 137 us instead of 123).
//
// Only key tiles that hold drafts, or that a window's edge may cut, are masked
// ("cut" tiles).  A NaN or an infinity in a column of V makes that column of the output
// NaN for the rows that see it, and for no other.  In the other tiles the products do
// that by themselves (every row sees every key, and what comes out infinite is made
// NaN).  In the cut tiles 0 x NaN would reach the rows that do not see it: there the
// softmax warps look through V in shared memory, write down for each row the columns
// of such values that it sees, and put zeros in their place.
//
// 32 nodes of 32 heads over 32 x 8 cache rows of up to 8160 keys (581 MB, bf16,
// head_dim 128): 97 us for this kernel, 6.0 TB/s, 115 us for the call.  Memory bounds
// it; a tile's softmax (2300 clocks, 1024 of them the exponentials' unit) is close
// behind the 2788 clocks of its bytes.  With head_dim 64 or few keys a row the softmax
// does: 61 nodes of 64 heads under a window of 1000 (19 MB) take 29 us.

constexpr int kBM = 128, kBN = 128;
constexpr int kSoftmaxWarps = 8;
constexpr int kAttnThreads = 32 * (1 + kSoftmaxWarps + 3);
constexpr float kRescale = 8.f;  // log2 units by which a score may exceed the reference maximum

struct TreeArgs {
    void *out;
    const void *q;
    const uint32_t *mask;
    const int32_t *depth;
    CacheRows at;
    kvc_lengths len;
    int batch, q_heads, kv_heads, group, nodes;
    int row_tiles;  // ceil(group * nodes / 128)
    int box_rows;   // rows of a TMA box of K or V
    int window;
    float scale_log2;
    const float *cos_t, *sin_t;
    int64_t rope_max_pos;
    int grid, row_cost;
    float *ws_o, *ws_m, *ws_l;  // [2 * grid][D / 4][128][4], [2 * grid][128]
    void *ws_q;                 // rotated queries, as q: rounded, then (q_split) what that left
    int q_split;
    uint32_t *see;              // drafts that each node sees, as mask
    int4 *split;                // [grid] the row of which a CTA has the first keys but not the last: batch row, row,
                                // parts (0: there is none), slot of its own part
    int32_t *status;
};

template <int D, int KR> struct TreeSmem {
    static constexpr bool SPLIT_Q = D <= 128;  // two query tiles; else two parts of the weights
    static constexpr int Q_TILE = kBM * D * 2, Q_BYTES = SPLIT_Q ? 2 * Q_TILE : Q_TILE;
    static constexpr int SLAB = KR * D * 2;
    static constexpr int SPT = kBN / KR;  // slabs of a tile of K (or V)
    static constexpr int BUDGET = 227 * 1024;
    static constexpr int NBAR = 10;       // beside the ring's
    static constexpr int MISC = (2 * 12 + NBAR) * 8 + 16 + 4 * kBM * 4 + 16;
    static constexpr int FIT = (BUDGET - Q_BYTES - MISC) / SLAB;
    static constexpr int NSLAB = FIT < 12 ? FIT : 12;
    static constexpr int RING_OFF = Q_BYTES;
    static constexpr int BAR_OFF = RING_OFF + NSLAB * SLAB;
    // full[NSLAB], empty[NSLAB], s_full[2], p_full[2], o_done[2], q_full, q_empty, drain[2]
    static constexpr int MISC_OFF = BAR_OFF + (2 * NSLAB + NBAR) * 8;
    static constexpr int RED_OFF = (MISC_OFF + 8 + 15) / 16 * 16;  // row maximum / sum exchange
    static constexpr int BAD_OFF = RED_OFF + 4 * kBM * 4;
    static constexpr int TOTAL = BAD_OFF + 16;
    static_assert(TOTAL <= BUDGET && NSLAB >= 2 * SPT, "a tile of K and one of V must fit");
    static constexpr uint32_t COL_O = 0, COL_S = D, TMEM_COLS = 512;
};

// batch row b: its past length, first key row of its tiles and their number (0:
// nothing to do)
__device__ __forceinline__ int tree_tiles(const TreeArgs &a, int b, int &P, int &lo, uint32_t &bad)
{
    P = a.len.past_abs[b];
    const int L = a.len.cache_total[b];
    bad = 0;
    lo = 0;
    if (L < 0 || P < 0)
        return 0;
    const int64_t T = (int64_t)P + a.nodes;
    if (a.cos_t && T > a.rope_max_pos)
        bad = KVC_DEV_ROPE_RANGE;
    else if (T > a.at.rows)
        bad = KVC_DEV_CAPACITY;
    if (bad)
        return 0;
    if (a.window > 0)
        lo = max(0, P - a.window + 1) & ~(a.box_rows - 1);  // what a node of depth 0 sees
    return (int)((T - lo + kBN - 1) / kBN);
}

// Tiles of a row on the line that the CTAs share: those of its keys, and kRowCost
// that hold none but stand for what a segment costs beside them (scores of the first
// tile, output).
constexpr int kRowCost = 4;
__device__ __forceinline__ int line_tiles(const TreeArgs &a, int n) { return n > 0 ? n + a.row_cost : 0; }

// The segments of a CTA's share, one at a time: tiles [t0, t1) of the n tiles of
// line row (b, head, row tile).
struct Segment {
    int b, row, P, lo, n, t0, t1, end;  // end: of the row on the line
};
struct Walk {
    int x, x_end, b, base, P, lo, n;
    __device__ __forceinline__ void load(const TreeArgs &a)
    {
        uint32_t bad;
        n = tree_tiles(a, b, P, lo, bad);
    }
    __device__ __forceinline__ bool next(const TreeArgs &a, Segment &s)
    {
        const int rows = a.kv_heads * a.row_tiles;
        while (x < x_end) {
            while (x >= base + line_tiles(a, n) * rows) {
                base += line_tiles(a, n) * rows;
                ++b;
                load(a);
            }
            const int line = line_tiles(a, n);
            s.b = b;
            s.P = P;
            s.lo = lo;
            s.n = n;
            s.row = (x - base) / line;
            s.end = base + (s.row + 1) * line;
            const int p0 = (x - base) - s.row * line, p1 = min(line, p0 + (x_end - x));
            x += p1 - p0;
            // the tiles that stand for the row's cost hold no keys
            s.t0 = max(0, p0 - a.row_cost);
            s.t1 = p1 - a.row_cost;
            if (s.t1 > s.t0)
                return true;
        }
        return false;
    }
};

// The ring holds, for a segment of n tiles, K_0, K_1, then V_j and K_{j+2} while
// there is one, then the last V's: the places of K_j and of V_j in that order.
__device__ __forceinline__ int k_group(int j, int) { return j < 2 ? j : 2 * j - 1; }
__device__ __forceinline__ int v_group(int j, int n)
{
    const int lead = n < 2 ? n : 2, paired = n - lead;
    return j < paired ? lead + 2 * j : lead + paired + j;
}

// the 16-bit halves of w that are NaN or infinite, as 0xffff each
template <typename T> __device__ __forceinline__ uint32_t not_finite(uint32_t w)
{
    constexpr uint32_t ex = std::is_same<T, __half>::value ? 0x7c007c00u : 0x7f807f80u;
    return __vcmpeq2(w & ex, ex);
}

// Blocks [0, q_blocks): eight rotation pairs of a query row a thread.  The others:
// a word of a node's drafts a thread.
template <typename T>
__global__ void __launch_bounds__(256)
tree_prep_kernel(const TreeArgs a, int D, unsigned q_blocks)
{
    kvc::grid_dep_launch();
    const int N = a.nodes;
    if (blockIdx.x < q_blocks) {
        const int pieces = D / 16;
        const int64_t w = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
        const int64_t row = w / pieces;
        const int c0 = (int)(w % pieces) * 8;
        if (row >= (int64_t)a.batch * a.q_heads * N)
            return;
        const int b = (int)(row / ((int64_t)a.q_heads * N));
        const int d = __ldg(a.depth + (int64_t)b * N + row % N);
        const T *q = static_cast<const T *>(a.q) + row * D + c0;
        uint4 lo = __ldg(reinterpret_cast<const uint4 *>(q)), hi = __ldg(reinterpret_cast<const uint4 *>(q + D / 2));
        int P, first;
        uint32_t bad;
        if (tree_tiles(a, b, P, first, bad) == 0 || d < 0 || d >= N)
            return;  // never looked at
        const int64_t at = ((int64_t)P + d) * (D / 2) + c0;
        float cs[8], sn[8];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float4 x = __ldg(reinterpret_cast<const float4 *>(a.cos_t + at) + e);
            const float4 y = __ldg(reinterpret_cast<const float4 *>(a.sin_t + at) + e);
            cs[4 * e] = x.x, cs[4 * e + 1] = x.y, cs[4 * e + 2] = x.z, cs[4 * e + 3] = x.w;
            sn[4 * e] = y.x, sn[4 * e + 1] = y.y, sn[4 * e + 2] = y.z, sn[4 * e + 3] = y.w;
        }
        T *x = reinterpret_cast<T *>(&lo), *y = reinterpret_cast<T *>(&hi);
        uint4 lo2, hi2;
        T *x2 = reinterpret_cast<T *>(&lo2), *y2 = reinterpret_cast<T *>(&hi2);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float u = kvc::Elem<T>::to_f32(x[e]), v = kvc::Elem<T>::to_f32(y[e]);
            kvc::rope_pair(u, v, cs[e], sn[e]);
            x[e] = kvc::Elem<T>::from_f32(u);
            y[e] = kvc::Elem<T>::from_f32(v);
            x2[e] = kvc::Elem<T>::from_f32(u - kvc::Elem<T>::to_f32(x[e]));
            y2[e] = kvc::Elem<T>::from_f32(v - kvc::Elem<T>::to_f32(y[e]));
        }
        T *to = static_cast<T *>(a.ws_q) + row * D + c0;
        *reinterpret_cast<uint4 *>(to) = lo;
        *reinterpret_cast<uint4 *>(to + D / 2) = hi;
        if (a.q_split) {
            to += (int64_t)a.batch * a.q_heads * N * D;
            *reinterpret_cast<uint4 *>(to) = lo2;
            *reinterpret_cast<uint4 *>(to + D / 2) = hi2;
        }
        return;
    }
    const int words = (N + 31) / 32;
    const int64_t w = (int64_t)(blockIdx.x - q_blocks) * blockDim.x + threadIdx.x;
    if (w >= (int64_t)a.batch * N * words)
        return;
    const int64_t row = w / words;
    const int b = (int)(row / N), j0 = (int)(w % words) * 32;
    const int32_t *depth = a.depth + (int64_t)b * N;
    const int d = __ldg(depth + row % N);
    uint32_t left = a.mask[w], bits = 0;
    if (d >= N && j0 == 0)
        kvc::raise_status(a.status, KVC_DEV_INDEX_OOB);
    if (d < 0 || d >= N)
        left = 0;
    while (left) {
        const int c = __ffs(left) - 1;
        left &= left - 1;
        const int dj = j0 + c < N ? __ldg(depth + j0 + c) : -1;
        if (dj >= 0 && dj < N && (a.window <= 0 || d - dj < a.window))
            bits |= 1u << c;
    }
    a.see[w] = bits;
}

template <typename T, int D, int KR>
__global__ void __launch_bounds__(kAttnThreads, 1)
tree_attn_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                 const __grid_constant__ CUtensorMap tmap_v, const TreeArgs a)
{
    using SM = TreeSmem<D, KR>;
    using kvc_tc::wait_or_abort;
    constexpr int NSLAB = SM::NSLAB, SPT = SM::SPT;
    constexpr uint32_t AB = std::is_same<T, __half>::value ? 0u : 1u;
    constexpr uint32_t IDESC_S = kvc_tc::f16_idesc(AB, 0, kBM, KR);
    constexpr uint32_t IDESC_O = kvc_tc::f16_idesc(AB, 1, kBM, D);

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    {
        // the swizzled tiles need a 1024-byte aligned base
        uint32_t dyn;
        asm("mov.u32 %0, %%dynamic_smem_size;" : "=r"(dyn));
        if ((uint32_t)(smem - smem_raw) + SM::TOTAL > dyn) {
            if (threadIdx.x == 0)
                kvc::raise_status(a.status, KVC_DEV_CAPACITY);
            return;
        }
    }
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + SM::BAR_OFF), *empty = full + NSLAB,
             *s_full = full + 2 * NSLAB, *p_full = s_full + 2, *o_done = s_full + 4, *q_full = s_full + 6,
             *q_empty = s_full + 7, *drain = s_full + 8;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + SM::MISC_OFF);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + SM::MISC_OFF + 4);

    kvc::grid_dep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < NSLAB; ++i) {
            kvc::mbar_init(&full[i], 1);
            kvc::mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            kvc::mbar_init(&s_full[i], 1);
            kvc::mbar_init(&p_full[i], kSoftmaxWarps);
            kvc::mbar_init(&o_done[i], 1);
        }
        kvc::mbar_init(q_full, 1);
        kvc::mbar_init(q_empty, 1);
        kvc::mbar_init(&drain[0], 1);
        kvc::mbar_init(&drain[1], 1);
        *abort_flag = 0;
        for (int i = 0; i < 4; ++i)
            reinterpret_cast<uint32_t *>(smem + SM::BAD_OFF)[i] = 0;
        kvc::fence_mbar_init();
    }
    if (warp == 0) {
        kvc_tc::tmem_alloc(tmem_slot, SM::TMEM_COLS);
        kvc_tc::fence_before();
    }
    const int N = a.nodes, rows = a.group * N, line_rows = a.kv_heads * a.row_tiles;
    Walk walk;
    kvc_flat::Shares shares(0, 1);
    {
        auto count = [&](int b) {
            int P, lo;
            uint32_t bad;
            const int n = tree_tiles(a, b, P, lo, bad);
            if (bad && blockIdx.x == 0 && warp == 0)
                kvc::raise_status(a.status, bad);
            return line_tiles(a, n);
        };
        // (a CTA without a share falls through its loops)
        shares = kvc_flat::share_of_cta(a.batch, line_rows, count, a.grid, blockIdx.x, walk.x, walk.x_end, walk.b,
                                        walk.base);
        if (walk.x < walk.x_end)
            walk.load(a);
    }
    __syncthreads();
    kvc_tc::fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t smem_base = kvc::smem_u32(smem);
    // each role looks one segment ahead, so that the lengths are there when it gets to it
    Segment cur, nxt;
    bool more = walk.next(a, cur);

    if (warp == 1 + kSoftmaxWarps || warp == 2 + kSoftmaxWarps) {
        // ======================= TMA producers of K and of V =======================
        // (the cache's rows are those of the kernels before tree_prep_kernel: no wait for it)
        // Each lane finds the place of one of the next 32 slabs: one thread alone spent 1500 clocks a slab
        // on a page's number, its division and the latency of the table.
        const bool mine_v = warp == 2 + kSoftmaxWarps;
        const CUtensorMap *tmap = mine_v ? &tmap_v : &tmap_k;
        if (lane == 0)
            kvc::tma_prefetch_desc(tmap);
        if (!mine_v && lane == 0)
            a.split[blockIdx.x] = make_int4(0, 0, 0, 0);
        int q0 = 0;  // slabs of the segments before
        bool ok = true, first_segment = true;
        const int boxes = KR / a.box_rows;  // of a slab's rows: 1 or 2
        uint32_t filled = 0, phase = 0;  // slots that this warp has filled, with the parity of the last time
        while (ok && more) {
            const int h = cur.row / a.row_tiles, nt = cur.t1 - cur.t0;
            const uint32_t end = (uint32_t)cur.P + N, first = (uint32_t)cur.lo + cur.t0 * kBN;
            const bool again = walk.next(a, nxt);
            if (!mine_v && lane == 0 && cur.t0 == 0 && nt != cur.n)
                a.split[blockIdx.x] =
                    make_int4(cur.b, cur.row, shares.of(cur.end - 1) - (int)blockIdx.x + 1, first_segment ? 0 : 1);
            first_segment = false;
            int32_t place = -1;
            for (int u = 0; u < SPT * nt; ++u) {
                if ((u * boxes & 31) == 0) {
                    const int w = u * boxes + lane;
                    const uint32_t r = first + (uint32_t)w * a.box_rows;
                    place = -1;
                    if (w < SPT * nt * boxes && r < end) {
                        if (a.at.table) {
                            const uint32_t page = r / (uint32_t)a.at.page_size;
                            const int32_t id = __ldg(a.at.table + (int64_t)cur.b * a.at.max_pages + page);
                            if (id >= 0 && id < a.at.n_pool)
                                place = (id * a.kv_heads + h) * a.at.page_size + (int32_t)(r - page * a.at.page_size);
                            else
                                kvc::raise_status(a.status, KVC_DEV_INDEX_OOB);
                        } else {
                            place = (int32_t)(((int64_t)cur.b * a.kv_heads + h) * a.at.rows + r);
                        }
                    }
                }
                const int32_t y0 = __shfl_sync(0xffffffffu, place, u * boxes & 31);
                const int32_t y1 = __shfl_sync(0xffffffffu, place, (u * boxes + 1) & 31);
                const int q = q0 + SPT * (mine_v ? v_group(u / SPT, nt) : k_group(u / SPT, nt)) + u % SPT;
                const int slot = q % NSLAB;
                if (q >= NSLAB)
                    ok = wait_or_abort(&empty[slot], ((q / NSLAB) - 1) & 1, abort_flag, a.status);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok)
                    break;
                if (lane == 0) {
                    uint8_t *to = smem + SM::RING_OFF + slot * SM::SLAB;
                    if (boxes == 1) {
                        if (y0 < 0) {
                            // nothing to read: the slot keeps what it holds, and its columns are masked
                            kvc::mbar_arrive(&full[slot]);
                        } else {
                            kvc::mbar_arrive_expect_tx(&full[slot], SM::SLAB);
                            kvc::tma_load_3d(to, tmap, 0, y0, 0, &full[slot]);
                        }
                    } else {
                        // half a slab's rows a box, of 64 columns
                        const int n = (y0 >= 0) + (y1 >= 0);
                        if (n == 0)
                            kvc::mbar_arrive(&full[slot]);
                        else
                            kvc::mbar_arrive_expect_tx(&full[slot], n * (SM::SLAB / 2));
                        for (int c = 0; c < D / 64; ++c) {
                            if (y0 >= 0)
                                kvc::tma_load_3d(to + c * (KR * 128), tmap, 0, y0, c, &full[slot]);
                            if (y1 >= 0)
                                kvc::tma_load_3d(to + c * (KR * 128) + KR / 2 * 128, tmap, 0, y1, c, &full[slot]);
                        }
                    }
                }
                __syncwarp();
                filled |= 1u << slot;
                phase = (phase & ~(1u << slot)) | ((uint32_t)((q / NSLAB) & 1) << slot);
            }
            q0 += 2 * SPT * nt;
            cur = nxt;
            more = again;
        }
        if (*abort_flag && lane == 0)
            // wind-down: let the loads in flight land before the CTA exits
            for (int i = 0; i < NSLAB; ++i)
                if (filled >> i & 1)
                    kvc::mbar_wait(&full[i], phase >> i & 1);
    } else if (warp == 3 + kSoftmaxWarps) {
        // ======================= output products =======================
        if (lane == 0) {
            const uint64_t v_ring = kvc_tc::sw128_desc(smem_base + SM::RING_OFF, KR * 128);
            int q0 = 0, J = 0;  // slabs of the segments before, tiles so far
            bool ok = true;
            while (ok && more) {
                const int nt = cur.t1 - cur.t0;
                more = walk.next(a, nxt);
                for (int j = 0; j < nt; ++j, ++J) {
                    const int s = J & 1;
                    if (!(ok = wait_or_abort(&p_full[s], (J >> 1) & 1, abort_flag, a.status)))
                        break;
                    kvc_tc::fence_after();
                    for (int hf = 0; hf < SPT; ++hf) {
                        const int q = q0 + SPT * v_group(j, nt) + hf, slot = q % NSLAB;
                        if (!(ok = wait_or_abort(&full[slot], (q / NSLAB) & 1, abort_flag, a.status)))
                            break;
                        kvc_tc::fence_after();
                        const uint64_t vd = v_ring + (uint64_t)(slot * (SM::SLAB / 16));
                        const uint32_t pa = tmem + SM::COL_S + s * kBN + hf * (KR / 2);
#pragma unroll
                        for (int part = 0; part < (SM::SPLIT_Q ? 1 : 2); ++part) {
#pragma unroll
                            for (int k2 = 0; k2 < KR / 16; ++k2)
                                kvc_tc::mma_ts(tmem + SM::COL_O, pa + part * 64 + k2 * 8,
                                               vd + (uint64_t)(k2 * (2048 / 16)), IDESC_O,
                                               j > 0 || hf > 0 || part > 0 || k2 > 0);
                        }
                        kvc_tc::commit(&empty[slot]);
                    }
                    if (!ok)
                        break;
                    kvc_tc::commit(&o_done[s]);
                }
                q0 += 2 * SPT * nt;
                cur = nxt;
            }
            // everything issued above has completed once this arrives
            kvc_tc::commit(&drain[1]);
            kvc::mbar_wait(&drain[1], 0);
        }
    } else if (warp == 0) {
        // ======================= queries, score products =======================
        if (lane == 0) {
            kvc::tma_prefetch_desc(&tmap_q);
            int q0 = 0, J = 0;  // slabs of the segments before, tiles so far
            bool ok = true;
            const int q_parts = SM::SPLIT_Q && a.q_split ? 2 : 1;
            const uint64_t q_desc = kvc_tc::sw128_desc(smem_base, 16);
            const uint64_t k_ring = kvc_tc::sw128_desc(smem_base + SM::RING_OFF, 16);
            kvc::grid_dep_wait();  // tree_prep_kernel's
            for (int s_no = 0; ok && more; ++s_no) {
                // the last segment's scores are done: the queries' place is free
                if (s_no > 0 && !wait_or_abort(q_empty, (s_no - 1) & 1, abort_flag, a.status))
                    break;
                const int nt = cur.t1 - cur.t0;
                {
                    const int h = cur.row / a.row_tiles, mt = cur.row % a.row_tiles;
                    const int y = (cur.b * a.kv_heads + h) * rows + mt * kBM;
                    kvc::mbar_arrive_expect_tx(q_full, q_parts * SM::Q_TILE);
                    kvc::tma_load_3d(smem, &tmap_q, 0, y, 0, q_full);
                    if (q_parts > 1)
                        kvc::tma_load_3d(smem + SM::Q_TILE, &tmap_q, 0, y + a.batch * a.q_heads * N, 0, q_full);
                }
                more = walk.next(a, nxt);
                if (!(ok = wait_or_abort(q_full, s_no & 1, abort_flag, a.status))) {
                    kvc::mbar_wait(q_full, s_no & 1);  // (let the loads land before the CTA exits)
                    break;
                }
                kvc_tc::fence_after();
                for (int j = 0; ok && j < nt; ++j, ++J) {
                    const int buf = J & 1;
                    // S_J is written where PV_{J-2} reads its weights.  Products follow one another in the order
                    // of their issue only when they share accumulator and shape, which these two do not: the
                    // wait for PV_{J-2} is what keeps its weights.  (With S_J issued right behind PV_{J-2} and no
                    // wait, head_dim 64 came out wrong in every second tile when the products of S were written
                    // out and so followed closely; with the wait both forms are right.)
                    if (J >= 2 && !(ok = wait_or_abort(&o_done[buf], ((J >> 1) - 1) & 1, abort_flag, a.status)))
                        break;
                    for (int hf = 0; hf < SPT; ++hf) {
                        const int q = q0 + SPT * k_group(j, nt) + hf, slot = q % NSLAB;
                        if (!(ok = wait_or_abort(&full[slot], (q / NSLAB) & 1, abort_flag, a.status)))
                            break;
                        kvc_tc::fence_after();
                        const uint64_t kd = k_ring + (uint64_t)(slot * (SM::SLAB / 16));
                        const uint32_t d_s = tmem + SM::COL_S + buf * kBN + hf * KR;
#pragma unroll
                        for (int part = 0; part < (SM::SPLIT_Q ? 2 : 1); ++part) {
                            if (part == q_parts)
                                break;
                            const uint64_t qd = q_desc + (uint64_t)(part * (SM::Q_TILE / 16));
#pragma unroll
                            for (int ks = 0; ks < D / 16; ++ks)
                                kvc_tc::mma_ss(d_s, qd + (uint64_t)(((ks >> 2) * (kBM * 128) + (ks & 3) * 32) / 16),
                                               kd + (uint64_t)(((ks >> 2) * (KR * 128) + (ks & 3) * 32) / 16), IDESC_S,
                                               part > 0 || ks > 0);
                        }
                        kvc_tc::commit(&empty[slot]);
                    }
                    if (!ok)
                        break;
                    kvc_tc::commit(&s_full[buf]);
                    if (j == nt - 1)
                        kvc_tc::commit(q_empty);
                }
                q0 += 2 * SPT * nt;
                cur = nxt;
            }
            // everything issued above has completed once this arrives
            kvc_tc::commit(&drain[0]);
            kvc::mbar_wait(&drain[0], 0);
        }
    } else {
        // ======================= softmax =======================
        const int sw = warp - 1, tid = threadIdx.x - 32;
        const int quad = warp & 3, half = sw >> 2;   // TMEM lane quadrant; columns [0, 64) or [64, 128)
        const int m = quad * 32 + lane;
        const uint32_t lane_addr = tmem + ((uint32_t)(quad * 32) << 16);
        float *red = reinterpret_cast<float *>(smem + SM::RED_OFF);
        uint32_t *bad_sh = reinterpret_cast<uint32_t *>(smem + SM::BAD_OFF);
        constexpr uint32_t all_bar = 1;
        const int words = (N + 31) / 32;
        const float c_log2 = fabsf(a.scale_log2);
        // this thread's row of a segment: its node's depth (-1: absent, or no row)
        auto row_depth = [&](const Segment &sg) {
            const int r = sg.row % a.row_tiles * kBM + m;
            return r < rows ? __ldg(a.depth + (int64_t)sg.b * N + r % N) : -1;
        };
        int d_next = more ? row_depth(cur) : -1;
        kvc::grid_dep_wait();  // tree_prep_kernel's
        int q0 = 0, J = 0;     // slabs before the segment, tiles so far
        // `ok` is the warp's own; the softmax warps leave their loops together, at a barrier
        bool ok = true, stop = false;
        for (int s_no = 0; more; ++s_no) {
            const int mt = cur.row % a.row_tiles, h = cur.row / a.row_tiles, nt = cur.t1 - cur.t0;
            const int P = cur.P;
            const int r = mt * kBM + m;
            const bool active = mt * kBM + quad * 32 < rows;  // of the warp: it has rows at all
            const int d = d_next >= 0 && d_next < N ? d_next : -1;
            // (ordinary loads: tree_prep_kernel still writes them when this kernel's life begins)
            const uint32_t *see_words = a.see + ((int64_t)cur.b * N + r % N) * words;
            // the words that hold the drafts of this thread's columns of tile j
            uint32_t w_next[3];
            auto load_words = [&](int j) {
                const int j0 = cur.lo + (cur.t0 + j) * kBN + 64 * half - P;  // draft of the first column
                w_next[0] = w_next[1] = w_next[2] = 0;
                if (j0 + 64 > 0 && r < rows) {
                    const int w0 = j0 >> 5;
#pragma unroll
                    for (int e = 0; e < 3; ++e)
                        w_next[e] = w0 + e >= 0 && w0 + e < words ? see_words[w0 + e] : 0u;
                }
            };
            load_words(0);
            more = walk.next(a, nxt);
            d_next = more ? row_depth(nxt) : -1;
            // cache rows from r_lo on are visible
            const int r_lo = a.window > 0 ? max(0, P + d - a.window + 1) : 0;
            // those among the keys [k0, k0 + 32), a bit each
            auto cache_keys = [&](int k0) {
                uint32_t bits = 0;
                if (d >= 0 && k0 < P && k0 + 32 > r_lo) {
                    bits = k0 < r_lo ? ~0u << (r_lo - k0) : ~0u;
                    if (k0 + 32 > P)
                        bits &= ~0u >> (k0 + 32 - P);
                }
                return bits;
            };
            // this half's output columns in which the row has seen a NaN or an infinity, in the cut tiles
            uint32_t nan_cols[D / 64] = {};
            float m_run = -INFINITY, l_run = 0.f;
            for (int j = 0; j < nt; ++j, ++J) {
                const int s = J & 1;
                const int t_lo = cur.lo + (cur.t0 + j) * kBN, c0 = t_lo + 64 * half;
                const bool cut = t_lo + kBN > P || (a.window > 0 && t_lo < P + N - a.window);
                // the keys that this row sees, a bit a column
                uint32_t see[2] = {~0u, ~0u};
                if (cut || d < 0) {
                    const int sh = (c0 - P) & 31;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        see[e] = cache_keys(c0 + 32 * e) | __funnelshift_r(w_next[e], w_next[e + 1], sh);
                    }
                }
                load_words(j + 1);
                ok = ok && wait_or_abort(&s_full[s], (J >> 1) & 1, abort_flag, a.status);
                kvc_tc::fence_after();
                if (cut) {
                    // V rows with a NaN or an infinity in them, a bit each in bad_sh (zero before)
                    bool found = false;
#pragma unroll
                    for (int hf = 0; hf < SPT; ++hf) {
                        const int qi = q0 + SPT * v_group(j, nt) + hf;
                        ok = ok && wait_or_abort(&full[qi % NSLAB], (qi / NSLAB) & 1, abort_flag, a.status);
                        if (!ok)
                            break;
                        const uint4 *v = reinterpret_cast<const uint4 *>(smem + SM::RING_OFF + (qi % NSLAB) * SM::SLAB);
#pragma unroll
                        for (int e = 0; e < SM::SLAB / 16 / 256; ++e) {
                            const uint4 x = v[tid + 256 * e];
                            if (not_finite<T>(x.x) | not_finite<T>(x.y) | not_finite<T>(x.z) | not_finite<T>(x.w)) {
                                const int vr = hf * KR + (((tid + 256 * e) >> 3) & (KR - 1));
                                atomicOr(&bad_sh[vr >> 5], 1u << (vr & 31));
                                found = true;
                            }
                        }
                    }
                    if (kvc_tc::named_bar_any(all_bar, 32 * kSoftmaxWarps, found)) {
                        // what this row sees of them is written down by column, then they are zeros for all
#pragma unroll 1
                        for (int e = 0; e < 4 && d >= 0; ++e) {
                            const int k0 = t_lo + 32 * e, w0 = (k0 - P) >> 5;
                            auto word = [&](int w) { return w >= 0 && w < words ? see_words[w] : 0u; };
                            uint32_t left = bad_sh[e] & (cache_keys(k0) | __funnelshift_r(word(w0), word(w0 + 1), (k0 - P) & 31));
                            while (left) {
                                const int vr = 32 * e + __ffs(left) - 1, in = vr & (KR - 1);
                                left &= left - 1;
                                const uint8_t *slab =
                                    smem + SM::RING_OFF + (q0 + SPT * v_group(j, nt) + vr / KR) % NSLAB * SM::SLAB;
#pragma unroll 1
                                for (int w = 0; w < D / 64; ++w) {
                                    uint32_t cols = 0;
#pragma unroll
                                    for (int c = 0; c < 4; ++c) {
                                        const int ch = half * (D / 16) + 4 * w + c;  // 16 bytes of the row
                                        const uint4 x = *reinterpret_cast<const uint4 *>(
                                            slab + (ch >> 3) * (KR * 128) + in * 128 + ((ch & 7) ^ (in & 7)) * 16);
                                        const uint32_t nf[4] = {not_finite<T>(x.x), not_finite<T>(x.y), not_finite<T>(x.z),
                                                                not_finite<T>(x.w)};
#pragma unroll
                                        for (int i = 0; i < 4; ++i)
                                            cols |= ((nf[i] & 1u) | (nf[i] >> 30 & 2u)) << (8 * c + 2 * i);
                                    }
                                    nan_cols[w] |= cols;
                                }
                            }
                        }
                        kvc_tc::named_bar_sync(all_bar, 32 * kSoftmaxWarps);
                        if (tid < 4)
                            bad_sh[tid] = 0;
#pragma unroll 1
                        for (int hf = 0; hf < SPT && ok; ++hf) {
                            uint4 *v = reinterpret_cast<uint4 *>(
                                smem + SM::RING_OFF + (q0 + SPT * v_group(j, nt) + hf) % NSLAB * SM::SLAB);
#pragma unroll 1
                            for (int at = tid; at < SM::SLAB / 16; at += 256) {
                                const uint4 x = v[at];
                                const uint4 nf = make_uint4(not_finite<T>(x.x), not_finite<T>(x.y), not_finite<T>(x.z),
                                                            not_finite<T>(x.w));
                                if (nf.x | nf.y | nf.z | nf.w)
                                    v[at] = make_uint4(x.x & ~nf.x, x.y & ~nf.y, x.z & ~nf.z, x.w & ~nf.w);
                            }
                        }
                        kvc::fence_proxy_async_smem();
                    }
                }
                float v[64];
                if (active) {
                    uint32_t *raw = reinterpret_cast<uint32_t *>(v);
                    kvc_tc::ld32(lane_addr + SM::COL_S + s * kBN + 64 * half, raw);
                    kvc_tc::ld32(lane_addr + SM::COL_S + s * kBN + 64 * half + 32, raw + 32);
                    kvc_tc::wait_ld();
                    if (a.scale_log2 < 0.f) {
#pragma unroll
                        for (int c = 0; c < 64; ++c)
                            v[c] = -v[c];
                    }
                    if (cut || d < 0) {
#pragma unroll
                        for (int c = 0; c < 64; ++c)
                            v[c] = see[c >> 5] >> (c & 31) & 1u ? v[c] : -INFINITY;
                    }
                    float mx0 = fmaxf(v[0], v[1]), mx1 = fmaxf(v[2], v[3]);
#pragma unroll
                    for (int c = 4; c < 64; c += 4) {
                        mx0 = fmaxf(mx0, fmaxf(v[c], v[c + 1]));
                        mx1 = fmaxf(mx1, fmaxf(v[c + 2], v[c + 3]));
                    }
                    red[(s * 2 + half) * kBM + m] = fmaxf(mx0, mx1);
                }
                // One barrier a tile of all softmax warps: the maxima are there, both halves' S has been
                // read before either writes P, and a warp whose wait gave up takes the others with it.
                if (kvc_tc::named_bar_any(all_bar, 32 * kSoftmaxWarps, !ok)) {
                    stop = true;
                    break;
                }
                if (active) {
                    const float top = fmaxf(red[(s * 2 + half) * kBM + m], red[(s * 2 + (half ^ 1)) * kBM + m]) * c_log2;
                    float alpha = 1.f;
                    bool rescale = false;
                    if (top > m_run + kRescale || (m_run == -INFINITY && top > -INFINITY)) {
                        if (j > 0 && m_run > -INFINITY) {
                            alpha = kvc_tc::fast_exp2(m_run - top);
                            rescale = true;
                        }
                        m_run = top;
                    }
                    const float neg_m = m_run == -INFINITY ? 0.f : -m_run;
                    float ps0 = 0.f, ps1 = 0.f;
                    uint32_t pk[32], pk2[SM::SPLIT_Q ? 1 : 32];
#pragma unroll
                    for (int c = 0; c < 64; c += 2) {
                        const float p0 = kvc_tc::fast_exp2(fmaf(v[c], c_log2, neg_m));
                        const float p1 = kvc_tc::fast_exp2(fmaf(v[c + 1], c_log2, neg_m));
                        ps0 += p0;
                        ps1 += p1;
                        pk[c / 2] = kvc_tc::pack2<T>(p0, p1);
                        if constexpr (!SM::SPLIT_Q) {
                            const T *w = reinterpret_cast<const T *>(&pk[c / 2]);
                            pk2[c / 2] =
                                kvc_tc::pack2<T>(p0 - kvc::Elem<T>::to_f32(w[0]), p1 - kvc::Elem<T>::to_f32(w[1]));
                        }
                    }
                    l_run = l_run * alpha + (ps0 + ps1);
                    kvc_tc::st32(lane_addr + SM::COL_S + s * kBN + 32 * half, pk);
                    if constexpr (!SM::SPLIT_Q)
                        kvc_tc::st32(lane_addr + SM::COL_S + s * kBN + 64 + 32 * half, pk2);
                    if (__any_sync(0xffffffffu, rescale)) {
                        // the reference moved: rescale this half of the O row (PV of the tile before is done;
                        // a wait that gives up is reported at the next barrier)
                        ok = wait_or_abort(&o_done[(J - 1) & 1], ((J - 1) >> 1) & 1, abort_flag, a.status);
                        kvc_tc::fence_after();
#pragma unroll 1
                        for (int cc = half * (D / 2); cc < (half + 1) * (D / 2); cc += 32) {
                            uint32_t o[32];
                            kvc_tc::ld32(lane_addr + SM::COL_O + cc, o);
                            kvc_tc::wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                            kvc_tc::st32(lane_addr + SM::COL_O + cc, o);
                        }
                    }
                    kvc_tc::wait_st();
                }
                kvc_tc::fence_before();
                __syncwarp();
                if (lane == 0)
                    kvc::mbar_arrive(&p_full[s]);
            }
            if (stop)
                break;
            q0 += 2 * SPT * nt;

            // ---- output rows ----
            // (the next segment's first PV waits for its p_full, which every warp gives after this)
            // The sums change hands where the last tile's maxima did: its PV is done, so every warp has read
            // those.  The next segment's first tile writes the other pair, and its barrier lies between these
            // reads and the next use of this one.
            const int sums = ((J - 1) & 1) * 2;
            ok = ok && wait_or_abort(&o_done[(J - 1) & 1], ((J - 1) >> 1) & 1, abort_flag, a.status);
            kvc_tc::fence_after();
            if (active)
                red[(sums + half) * kBM + m] = l_run;
            if (kvc_tc::named_bar_any(all_bar, 32 * kSoftmaxWarps, !ok))
                break;
            if (active) {
                const float l = l_run + red[(sums + (half ^ 1)) * kBM + m];
                const bool whole = nt == cur.n;
                const int64_t part = 2 * (int64_t)blockIdx.x + (s_no == 0 ? 0 : 1);
                // a row that saw nothing holds no sum: zeros, whatever O is
                const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
                for (int cc = half * (D / 2); cc < (half + 1) * (D / 2); cc += 32) {
                    uint32_t o[32];
                    kvc_tc::ld32(lane_addr + SM::COL_O + cc, o);
                    kvc_tc::wait_ld();
                    if (r >= rows)
                        continue;
                    if (const uint32_t bad = nan_cols[(cc - half * (D / 2)) / 32]) {
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            o[c] = bad >> c & 1u ? 0x7fc00000u : o[c];
                    }
                    if (whole) {
                        const int64_t row0 = ((int64_t)cur.b * a.kv_heads + h) * rows + (int64_t)mt * kBM;
                        T *to = static_cast<T *>(a.out) + (row0 + m) * D + cc;
#pragma unroll
                        for (int c = 0; c < 32; c += 8) {
                            uint4 x;
                            uint32_t *w = reinterpret_cast<uint32_t *>(&x);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float f0 = l == 0.f ? 0.f : __uint_as_float(o[c + 2 * e]) * inv;
                                const float f1 = l == 0.f ? 0.f : __uint_as_float(o[c + 2 * e + 1]) * inv;
                                w[e] = kvc_tc::pack2<T>(kvc_tc::finite_or_nan(f0), kvc_tc::finite_or_nan(f1));
                            }
                            *reinterpret_cast<uint4 *>(to + c) = x;
                        }
                    } else {
                        // four columns of all 128 rows side by side, so that a warp's store is one run
                        uint4 *to = reinterpret_cast<uint4 *>(a.ws_o) + (part * (D / 4) + cc / 4) * kBM + m;
#pragma unroll
                        for (int c = 0; c < 32; c += 4)
                            to[c / 4 * kBM] = make_uint4(o[c], o[c + 1], o[c + 2], o[c + 3]);
                    }
                }
                if (!whole && half == 0 && r < rows) {
                    a.ws_m[part * kBM + m] = m_run;
                    a.ws_l[part * kBM + m] = l;
                }
            }
            kvc_tc::fence_before();
            cur = nxt;
        }
    }

    kvc::grid_dep_wait();
    __syncthreads();
    if (warp == 0) {
        kvc_tc::fence_after();
        kvc_tc::tmem_dealloc(tmem, SM::TMEM_COLS);
    }
}

// Joins the partial results of 16 query rows that several CTAs worked on:
// out = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i.  A split row's first keys are in
// the share of exactly one CTA, which the block takes its number from and which has
// written down which row that is.  (With each of 2400 blocks finding that out from the
// lengths, the join of 32 x 8 rows took 4 us longer.  A join by the CTA that ends last
// cost the rows under way as much as the launch.)
constexpr int kMergeRows = 16;
template <typename T, int D>
__global__ void __launch_bounds__(256)
tree_merge_kernel(const TreeArgs a)
{
    kvc::grid_dep_wait();
    const int c0 = blockIdx.x, lane = threadIdx.x & 31, rows = a.group * a.nodes;
    const int4 split = a.split[c0];
    const int b = split.x, row = split.y, parts = split.z, slot0 = split.w;
    const int m0 = blockIdx.y * kMergeRows, r0 = row % a.row_tiles * kBM + m0;  // of the tile, of the head's rows
    if (parts == 0 || r0 >= rows)
        return;
    // the row's segment is the first of its CTA, but in the first CTA if that began before the row
    auto part = [&](int i) { return 2 * ((int64_t)c0 + i) + (i == 0 ? slot0 : 0); };
    // Weights: a warp two rows.  Columns: a row a thread's low bits, so that 16 threads read a run of
    // 256 bytes; those of the first parts are under way while the weights are found.
    constexpr int R = kMergeRows, W = R / 8;
    constexpr int COLS = D / 4, LANES = 256 / R, PER = COLS / LANES;  // float4 columns, of a thread
    __shared__ float w_sh[R][33], sum_sh[R];
    const int warp = threadIdx.x >> 5, mine = threadIdx.x % R, c4 = threadIdx.x / R;
    constexpr int AHEAD = PER <= 2 ? 4 : 2;  // parts under way
    float4 acc[PER], x[AHEAD][PER];
    auto load = [&](int i) {
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const float4 *o =
                reinterpret_cast<const float4 *>(a.ws_o) + (part(min(i + k, parts - 1)) * COLS + c4) * kBM + m0 + mine;
#pragma unroll
            for (int e = 0; e < PER; ++e)
                x[k][e] = o[e * LANES * kBM];
        }
    };
    load(0);
#pragma unroll
    for (int e = 0; e < PER; ++e)
        acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    float top[W], sum[W];
#pragma unroll
    for (int k = 0; k < W; ++k) {
        top[k] = -INFINITY;
        sum[k] = 0.f;
    }
    auto stat = [&](int i, int k) { return part(i) * kBM + m0 + W * warp + k; };
    for (int i = lane; i < parts; i += 32)
#pragma unroll
        for (int k = 0; k < W; ++k)
            top[k] = fmaxf(top[k], a.ws_l[stat(i, k)] == 0.f ? -INFINITY : a.ws_m[stat(i, k)]);
#pragma unroll
    for (int d = 16; d; d >>= 1)
#pragma unroll
        for (int k = 0; k < W; ++k)
            top[k] = fmaxf(top[k], __shfl_xor_sync(0xffffffffu, top[k], d));
    for (int i0 = 0; i0 < parts; i0 += 32) {
        __syncthreads();
#pragma unroll
        for (int k = 0; k < W; ++k) {
            // a part's weight a lane; a part that saw nothing (no sum) has none (-1), whatever its O holds; one
            // that is too small for a number still has its part's NaN
            float w = -1.f;
            if (i0 + lane < parts) {
                const float l = a.ws_l[stat(i0 + lane, k)], mc = a.ws_m[stat(i0 + lane, k)];
                if (l != 0.f) {
                    w = mc == top[k] || mc == -INFINITY ? 1.f : exp2f(mc - top[k]);
                    sum[k] += l * w;
                }
            }
            w_sh[W * warp + k][lane] = w;
        }
        __syncthreads();
        const int here = min(32, parts - i0);
        for (int i = 0; i < here; i += AHEAD) {
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                const float w = w_sh[mine][i + k];  // (-1 past the last part)
                if (w >= 0.f) {
#pragma unroll
                    for (int e = 0; e < PER; ++e) {
                        acc[e].x += x[k][e].x * w;
                        acc[e].y += x[k][e].y * w;
                        acc[e].z += x[k][e].z * w;
                        acc[e].w += x[k][e].w * w;
                    }
                }
            }
            if (i0 + i + AHEAD < parts)
                load(i0 + i + AHEAD);
        }
    }
#pragma unroll
    for (int k = 0; k < W; ++k) {
#pragma unroll
        for (int d = 16; d; d >>= 1)
            sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], d);
        if (lane == 0)
            sum_sh[W * warp + k] = sum[k];
    }
    __syncthreads();
    if (r0 + mine >= rows)
        return;
    const float total = sum_sh[mine], inv = total == 0.f ? 0.f : 1.f / total;
    T *to = static_cast<T *>(a.out) + (((int64_t)b * a.kv_heads + row / a.row_tiles) * rows + r0 + mine) * D;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
        uint2 y;
        y.x = total == 0.f ? 0u : kvc_tc::pack2<T>(kvc_tc::finite_or_nan(acc[e].x * inv), kvc_tc::finite_or_nan(acc[e].y * inv));
        y.y = total == 0.f ? 0u : kvc_tc::pack2<T>(kvc_tc::finite_or_nan(acc[e].z * inv), kvc_tc::finite_or_nan(acc[e].w * inv));
        *reinterpret_cast<uint2 *>(to + 4 * (c4 + LANES * e)) = y;
    }
}

template <typename... A>
cudaError_t launch_after(void (*kern)(A...), dim3 grid, int threads, size_t smem, cudaStream_t stream, A... args)
{
    // may start while the kernel before it runs, and waits for it where it needs it
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <typename T, int D, int KR>
kvc_status launch_attn_dim(TreeArgs &a, const void *k, const void *v, cudaStream_t stream)
{
    using SM = TreeSmem<D, KR>;
    const CUtensorMapDataType tt = std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                                  : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const uint64_t rows = (a.at.table ? (uint64_t)a.at.n_pool * a.at.page_size : (uint64_t)a.batch * a.at.rows) *
                          a.kv_heads;
    const int64_t q_rows = (int64_t)a.batch * a.q_heads * a.nodes;
    a.q_split = SM::SPLIT_Q && a.cos_t;  // (an unrotated query is 16-bit as it is)
    const int blocks = a.box_rows == KR ? D / 64 : 1;  // column blocks of a box of K or V
    CUtensorMap tq, tk, tv;
    if (!kvc_host::encode_3d_sw128(&tq, a.cos_t ? a.ws_q : a.q, (uint64_t)q_rows * (a.q_split ? 2 : 1), D, kBM, D / 64,
                                   tt) ||
        !kvc_host::encode_3d_sw128(&tk, k, rows, D, a.box_rows, blocks, tt) ||
        !kvc_host::encode_3d_sw128(&tv, v, rows, D, a.box_rows, blocks, tt))
        return kvc_host::cuda_failed();
    int dev = 0, optin = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess)
        return kvc_host::cuda_failed();
    const size_t smem = std::min<size_t>((size_t)SM::TOTAL + 1024, (size_t)optin);
    if (smem < (size_t)SM::TOTAL)
        return KVC_ERR_UNSUPPORTED;
    auto kern = tree_attn_kernel<T, D, KR>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return kvc_host::cuda_failed();
    const unsigned q_blocks = a.cos_t ? (unsigned)((q_rows * (D / 16) + 255) / 256) : 0u;
    const int64_t words = (int64_t)a.batch * a.nodes * ((a.nodes + 31) / 32);
    tree_prep_kernel<T><<<q_blocks + (unsigned)((words + 255) / 256), 256, 0, stream>>>(a, D, q_blocks);
    if (launch_after(kern, dim3(a.grid), kAttnThreads, smem, stream, tq, tk, tv, a) != cudaSuccess)
        return kvc_host::cuda_failed();
    if (a.grid > 1 && launch_after(tree_merge_kernel<T, D>,
                                   dim3(a.grid - 1, (std::min(kBM, a.group * a.nodes) + kMergeRows - 1) / kMergeRows), 256, 0,
                                   stream,
                                   a) != cudaSuccess)
        return kvc_host::cuda_failed();
    return kvc_host::launch_status();
}

template <typename T>
kvc_status launch_attn(TreeArgs &a, const void *k, const void *v, int D, cudaStream_t stream)
{
    a.box_rows = D <= 128 && (!a.at.table || a.at.page_size % kBN == 0) ? kBN : 64;
    switch (D) {
    case 64:
        return launch_attn_dim<T, 64, 128>(a, k, v, stream);
    case 128:
        return launch_attn_dim<T, 128, 128>(a, k, v, stream);
    default:
        return launch_attn_dim<T, 256, 64>(a, k, v, stream);
    }
}

// sizes that the calls on the cache's rows share; rows_out: rows a sequence may have
kvc_status check_rows(const int32_t *table, int max_pages, int64_t n_pool, int page_size, int batch, int kv_heads,
                      int nodes, int64_t capacity, int head_dim, int dtype, CacheRows &at)
{
    if (kvc_host::elem_bytes_of(dtype) == 0)
        return KVC_ERR_DTYPE;
    if (dtype == KVC_F32)
        return KVC_ERR_UNSUPPORTED;
    if (batch < 0 || batch > 65535 || kv_heads < 1 || kv_heads > 32767 || nodes < 1)
        return KVC_ERR_SHAPE;
    if (nodes > kMaxNodes || (head_dim != 64 && head_dim != 128 && head_dim != 256))
        return KVC_ERR_UNSUPPORTED;
    if (table) {
        if (page_size < 64 || page_size % 64 != 0 || max_pages < 1 || n_pool < 1)
            return KVC_ERR_SHAPE;
        capacity = (int64_t)max_pages * page_size;
        if (capacity > (int64_t)INT32_MAX || n_pool * kv_heads * (int64_t)page_size > (int64_t)INT32_MAX)
            return KVC_ERR_CAPACITY;
    } else if (capacity < 1 || capacity > (int64_t)INT32_MAX ||
               (int64_t)batch * kv_heads * capacity > (int64_t)INT32_MAX) {
        return KVC_ERR_CAPACITY;
    }
    at = CacheRows{table, max_pages, page_size, n_pool, capacity};
    return KVC_OK;
}

size_t cache_bytes(const CacheRows &at, int batch, int kv_heads, int D)
{
    const size_t rows = at.table ? (size_t)at.n_pool * at.page_size : (size_t)batch * at.rows;
    return rows * kv_heads * D * 2;
}

kvc_status check_rope(const float *cos_t, const float *sin_t, int64_t max_pos)
{
    if ((cos_t == nullptr) != (sin_t == nullptr))
        return KVC_ERR_NULL;
    if (cos_t && max_pos < 1)
        return KVC_ERR_SHAPE;
    return KVC_OK;
}

// the workspace: two partial results of a row tile for each CTA (one an SM), the
// rotated queries, the drafts that each node sees
struct TreeLayout {
    size_t split, q, see, total;
};
TreeLayout tree_layout(int batch, int q_heads, int nodes, int D)
{
    TreeLayout l;
    l.split = 2 * (size_t)kvc_host::sm_count() * kBM * (D + 2) * sizeof(float);
    l.q = l.split + (size_t)kvc_host::sm_count() * sizeof(int4);
    l.see = l.q + (size_t)batch * q_heads * nodes * D * 2 * 2;
    l.total = l.see + (size_t)batch * nodes * ((nodes + 31) / 32) * 4;
    return l;
}

bool all_aligned(std::initializer_list<const void *> ptrs)
{
    for (const void *p : ptrs)
        if (p && !kvc_host::aligned16(p))
            return false;
    return true;
}

} // namespace

KVC_API kvc_status kvc_tree_mask(const int32_t *parents, int batch, int nodes, uint32_t *mask, int32_t *depth,
                                 int32_t *dev_status, void *stream_)
{
    if (batch < 0 || nodes < 1)
        return KVC_ERR_SHAPE;
    if (nodes > kMaxNodes)
        return KVC_ERR_UNSUPPORTED;
    if (batch == 0)
        return KVC_OK;
    if (!parents || !mask || !depth)
        return KVC_ERR_NULL;
    tree_mask_kernel<<<batch, (nodes + 31) / 32 * 32, 0, static_cast<cudaStream_t>(stream_)>>>(parents, nodes, mask,
                                                                                              depth, dev_status);
    return kvc_host::launch_status();
}

KVC_API kvc_status kvc_tree_append(void *k_cache, void *v_cache, const void *new_k, const void *new_v,
                                   const int32_t *depth, const int32_t *block_table, int max_pages,
                                   int64_t n_pool_pages, int page_size, kvc_lengths len, int batch, int kv_heads,
                                   int nodes, int64_t capacity, int head_dim, int dtype, const float *rope_cos,
                                   const float *rope_sin, int64_t rope_max_pos, int32_t *dev_status, void *stream_)
{
    CacheRows at;
    kvc_status st = check_rows(block_table, max_pages, n_pool_pages, page_size, batch, kv_heads, nodes, capacity,
                               head_dim, dtype, at);
    if (st == KVC_OK)
        st = check_rope(rope_cos, rope_sin, rope_max_pos);
    if (st != KVC_OK)
        return st;
    if (batch == 0)
        return KVC_OK;
    if (!k_cache || !v_cache || !new_k || !new_v || !depth || !kvc_host::lengths_ok(len))
        return KVC_ERR_NULL;
    if (!all_aligned({k_cache, v_cache, new_k, new_v, rope_cos, rope_sin}))
        return KVC_ERR_ALIGN;
    const size_t bytes = cache_bytes(at, batch, kv_heads, head_dim);
    if (kvc_host::overlaps(k_cache, bytes, v_cache, bytes))
        return KVC_ERR_SHAPE;
    TreeRows a{k_cache, v_cache, new_k, new_v, depth, at, len, batch, kv_heads, nodes, head_dim, rope_cos, rope_sin,
               rope_max_pos, dev_status};
    const dim3 grid((nodes * head_dim / 8 + 127) / 128, kv_heads, batch);
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    if (dtype == KVC_BF16)
        tree_append_kernel<__nv_bfloat16><<<grid, 128, 0, stream>>>(a);
    else
        tree_append_kernel<__half><<<grid, 128, 0, stream>>>(a);
    return kvc_host::launch_status();
}

KVC_API size_t kvc_gqa_tree_workspace_size(int batch, int q_heads, int kv_heads, int nodes, int head_dim)
{
    if (batch < 1 || kv_heads < 1 || q_heads < 1 || q_heads % kv_heads != 0 || nodes < 1 || head_dim < 1)
        return 0;
    // (o, m, l), then the rotated queries and the words of the drafts seen
    return tree_layout(batch, q_heads, nodes, head_dim).total;
}

KVC_API kvc_status kvc_gqa_tree(void *out, const void *q, const void *k_cache, const void *v_cache,
                                const uint32_t *mask, const int32_t *depth, const int32_t *block_table, int max_pages,
                                int64_t n_pool_pages, int page_size, kvc_lengths len, int batch, int q_heads,
                                int kv_heads, int nodes, int64_t capacity, int head_dim, int dtype,
                                int local_window_size, float scale, const float *rope_cos, const float *rope_sin,
                                int64_t rope_max_pos, void *workspace, size_t workspace_bytes, int32_t *dev_status,
                                void *stream_)
{
    CacheRows at;
    kvc_status st = check_rows(block_table, max_pages, n_pool_pages, page_size, batch, kv_heads, nodes, capacity,
                               head_dim, dtype, at);
    if (st == KVC_OK)
        st = check_rope(rope_cos, rope_sin, rope_max_pos);
    if (st != KVC_OK)
        return st;
    if (q_heads < 1 || q_heads % kv_heads != 0)
        return KVC_ERR_SHAPE;
    if (q_heads / kv_heads > 16)
        return KVC_ERR_UNSUPPORTED;
    if (batch == 0)
        return KVC_OK;
    if (!out || !q || !k_cache || !v_cache || !mask || !depth || !kvc_host::lengths_ok(len))
        return KVC_ERR_NULL;
    if (!all_aligned({out, q, k_cache, v_cache, rope_cos, rope_sin}))
        return KVC_ERR_ALIGN;
    const size_t bytes = cache_bytes(at, batch, kv_heads, head_dim);
    if (kvc_host::overlaps(k_cache, bytes, v_cache, bytes))
        return KVC_ERR_SHAPE;
    const size_t need = kvc_gqa_tree_workspace_size(batch, q_heads, kv_heads, nodes, head_dim);
    if (!workspace || workspace_bytes < need)
        return KVC_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u)
        return KVC_ERR_ALIGN;
    TreeArgs a{};
    a.out = out;
    a.q = q;
    a.mask = mask;
    a.depth = depth;
    a.at = at;
    a.len = len;
    a.batch = batch;
    a.q_heads = q_heads;
    a.kv_heads = kv_heads;
    a.group = q_heads / kv_heads;
    a.nodes = nodes;
    a.window = local_window_size;
    a.scale_log2 = (scale == 0.f ? 1.0f / sqrtf((float)head_dim) : scale) * kLog2e;
    a.cos_t = rope_cos;
    a.sin_t = rope_sin;
    a.rope_max_pos = rope_max_pos;
    a.status = dev_status;
    a.row_tiles = (a.group * nodes + kBM - 1) / kBM;
    const int64_t units = (int64_t)batch * kv_heads * a.row_tiles * ((at.rows + kBN - 1) / kBN + kRowCost);
    if (units > (int64_t)INT32_MAX || (int64_t)batch * q_heads * nodes > (int64_t)INT32_MAX / 32)
        return KVC_ERR_SHAPE;
    // One CTA an SM over all rows, or, where the rows are so few that this leaves each too many parts: a
    // tile takes a CTA 1.4 us, and joining four parts 0.8, so that a row of t tiles is done soonest by about
    // sqrt(7 t) CTAs (one row of 126 tiles: 32 us with 126).  Rows then begin with a CTA each and cost nothing
    // beside their keys.
    const int64_t line_rows = (int64_t)batch * kv_heads * a.row_tiles, t = (at.rows + kBN - 1) / kBN;
    const int64_t few = std::min(t, (int64_t)std::ceil(std::sqrt(7.0 * (double)t)));
    const bool alone = line_rows * few <= kvc_host::sm_count();
    a.grid = (int)(alone ? line_rows * few : std::min<int64_t>(units, kvc_host::sm_count()));
    a.row_cost = alone ? 0 : kRowCost;
    const int64_t parts = 2 * (int64_t)kvc_host::sm_count() * kBM;
    a.ws_o = static_cast<float *>(workspace);
    a.ws_m = a.ws_o + parts * head_dim;
    a.ws_l = a.ws_m + parts;
    const TreeLayout layout = tree_layout(batch, q_heads, nodes, head_dim);
    a.ws_q = static_cast<uint8_t *>(workspace) + layout.q;
    a.see = reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(workspace) + layout.see);
    a.split = reinterpret_cast<int4 *>(static_cast<uint8_t *>(workspace) + layout.split);
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    return dtype == KVC_BF16 ? launch_attn<__nv_bfloat16>(a, k_cache, v_cache, head_dim, stream)
                             : launch_attn<__half>(a, k_cache, v_cache, head_dim, stream);
}

KVC_API kvc_status kvc_tree_commit(void *k_cache, void *v_cache, const int32_t *path, const int32_t *accepted,
                                   int path_len, const int32_t *block_table, int max_pages, int64_t n_pool_pages,
                                   int page_size, kvc_lengths len, int32_t *seqlens_k, int batch, int kv_heads,
                                   int nodes, int64_t capacity, int head_dim, int dtype, int32_t *dev_status,
                                   void *stream_)
{
    CacheRows at;
    const kvc_status st = check_rows(block_table, max_pages, n_pool_pages, page_size, batch, kv_heads, nodes, capacity,
                                     head_dim, dtype, at);
    if (st != KVC_OK)
        return st;
    if (path_len < 1)
        return KVC_ERR_SHAPE;
    if (batch == 0)
        return KVC_OK;
    if (!k_cache || !v_cache || !path || !accepted || !seqlens_k || !kvc_host::lengths_ok(len))
        return KVC_ERR_NULL;
    if (!all_aligned({k_cache, v_cache}))
        return KVC_ERR_ALIGN;
    const size_t bytes = cache_bytes(at, batch, kv_heads, head_dim);
    if (kvc_host::overlaps(k_cache, bytes, v_cache, bytes))
        return KVC_ERR_SHAPE;
    CommitArgs a{k_cache, v_cache, path, accepted, path_len, at, len, seqlens_k, kv_heads, nodes, head_dim * 2 / 16,
                 dev_status};
    tree_commit_kernel<<<dim3(2 * kv_heads, batch), 64, 0, static_cast<cudaStream_t>(stream_)>>>(a);
    return kvc_host::launch_status();
}
