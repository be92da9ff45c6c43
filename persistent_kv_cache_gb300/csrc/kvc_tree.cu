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
#include <type_traits>

#include "kvc_common.cuh"

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

struct TreeArgs {
    void *out;
    const void *q;
    const void *k, *v;
    const uint32_t *mask;
    const int32_t *depth;
    CacheRows at;
    kvc_lengths len;
    int batch, q_heads, kv_heads, group, nodes;
    int window;
    float scale_log2;
    const float *cos_t, *sin_t;
    int64_t rope_max_pos;
    int32_t *status;
};

// One block per (node, kv head, batch row), a warp per query head: 32 keys at
// a time, one a lane for the scores, then all lanes over the columns.
template <typename T, int D>
__global__ void __launch_bounds__(128)
tree_attn_kernel(const TreeArgs a)
{
    __shared__ float q_sh[4][D], p_sh[4][32];
    __shared__ int64_t row_sh[4][32];
    const int i = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int P = a.len.past_abs[b];
    if (a.len.cache_total[b] < 0 || P < 0)
        return;
    const bool lead = threadIdx.x == 0 && i == 0 && h == 0;
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
    const int d = a.depth[(int64_t)b * a.nodes + i];
    const bool there = d >= 0 && d < a.nodes;
    if (d >= a.nodes && threadIdx.x == 0 && h == 0)
        kvc::raise_status(a.status, KVC_DEV_INDEX_OOB);
    const int words = (a.nodes + 31) / 32;
    const uint32_t *mask = a.mask + ((int64_t)b * a.nodes + i) * words;
    const int64_t pos = (int64_t)P + d;
    for (int r = warp; r < a.group; r += 4) {
        const int64_t qrow = (((int64_t)b * a.q_heads + h * a.group + r) * a.nodes + i) * D;
        const T *q = static_cast<const T *>(a.q) + qrow;
        T *out = static_cast<T *>(a.out) + qrow;
        if (!there) {
            for (int c = lane; c < D; c += 32)
                out[c] = kvc::Elem<T>::from_f32(0.f);
            continue;
        }
        for (int c = lane; c < D / 2; c += 32) {
            float lo = kvc::Elem<T>::to_f32(q[c]), hi = kvc::Elem<T>::to_f32(q[c + D / 2]);
            if (a.cos_t)
                kvc::rope_pair(lo, hi, a.cos_t[pos * (D / 2) + c], a.sin_t[pos * (D / 2) + c]);
            q_sh[warp][c] = lo;
            q_sh[warp][c + D / 2] = hi;
        }
        __syncwarp();
        float acc[D / 32], m = -INFINITY, l = 0.f;
#pragma unroll
        for (int e = 0; e < D / 32; ++e)
            acc[e] = 0.f;
        const int64_t lo = a.window > 0 ? max((int64_t)0, pos - a.window + 1) : 0;
        for (int64_t r0 = min(lo, (int64_t)P); r0 < (int64_t)P + a.nodes; r0 += 32) {
            const int64_t row = r0 + lane;
            bool see = row < P;
            if (row >= P && row < (int64_t)P + a.nodes) {
                const int j = (int)(row - P);
                const int dj = a.depth[(int64_t)b * a.nodes + j];
                see = (mask[j >> 5] >> (j & 31) & 1u) && dj >= 0 && dj < a.nodes &&
                      (a.window <= 0 || d - dj < a.window);
            }
            int64_t at = -1;
            if (see) {
                if (a.at.table) {
                    const int64_t id = a.at.table[(int64_t)b * a.at.max_pages + row / a.at.page_size];
                    if (id < 0 || id >= a.at.n_pool) {
                        kvc::raise_status(a.status, KVC_DEV_INDEX_OOB);
                        see = false;
                    }
                }
                if (see)
                    at = row_index(a.at, b, h, a.kv_heads, row) * D;
            }
            float s = -INFINITY;
            if (see) {
                s = 0.f;
                const T *k = static_cast<const T *>(a.k) + at;
                for (int c = 0; c < D; c += 8) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(k + c);
                    const T *e = reinterpret_cast<const T *>(&x);
#pragma unroll
                    for (int u = 0; u < 8; ++u)
                        s += q_sh[warp][c + u] * kvc::Elem<T>::to_f32(e[u]);
                }
                s *= a.scale_log2;
            }
            float top = s;
#pragma unroll
            for (int x = 16; x; x >>= 1)
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
            const float m_new = fmaxf(m, top);
            const float f = m == m_new ? 1.f : exp2f(m - m_new);
            m = m_new;
            const float p = see ? exp2f(s - (m == -INFINITY ? 0.f : m)) : 0.f;
            l = l * f + p;
#pragma unroll
            for (int e = 0; e < D / 32; ++e)
                acc[e] *= f;
            p_sh[warp][lane] = p;
            row_sh[warp][lane] = at;
            __syncwarp();
            for (int j = 0; j < 32; ++j) {
                const int64_t vr = row_sh[warp][j];
                if (vr < 0)
                    continue;
                const float w = p_sh[warp][j];
#pragma unroll
                for (int e = 0; e < D / 32; ++e)
                    acc[e] += w * kvc::Elem<T>::to_f32(static_cast<const T *>(a.v)[vr + lane + 32 * e]);
            }
            __syncwarp();
        }
#pragma unroll
        for (int x = 16; x; x >>= 1)
            l += __shfl_xor_sync(0xffffffffu, l, x);
#pragma unroll
        for (int e = 0; e < D / 32; ++e)
            out[lane + 32 * e] = kvc::Elem<T>::from_f32(l == 0.f ? 0.f : acc[e] / l);
        __syncwarp();
    }
}

template <typename T> kvc_status launch_attn(const TreeArgs &a, int D, cudaStream_t stream)
{
    const dim3 grid(a.nodes, a.kv_heads, a.batch);
    if (D == 64)
        tree_attn_kernel<T, 64><<<grid, 128, 0, stream>>>(a);
    else if (D == 128)
        tree_attn_kernel<T, 128><<<grid, 128, 0, stream>>>(a);
    else
        tree_attn_kernel<T, 256><<<grid, 128, 0, stream>>>(a);
    return kvc_host::launch_status();
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
    return 256;
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
    a.k = k_cache;
    a.v = v_cache;
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
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    return dtype == KVC_BF16 ? launch_attn<__nv_bfloat16>(a, head_dim, stream) : launch_attn<__half>(a, head_dim, stream);
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
