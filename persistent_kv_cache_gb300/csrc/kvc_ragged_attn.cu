// kvc_ragged_attn.cu -- attention of a packed batch's new tokens over a paged
// cache ("Persistent KV Cache and Decode Performance Roadmap", "Phase 1" and
// "Phase 2": streaming online softmax, pages read through a page table).
#include <algorithm>
#include <cmath>

#include "kvc_common.cuh"

namespace {

struct RaggedArgs {
    void *out;
    const void *q, *k, *v;
    const int32_t *offsets, *table;
    int max_pages, page_size;
    int64_t n_pool;
    kvc_lengths len;
    int batch, tokens, q_heads, kv_heads, group;
    int window;
    float scale;
    int32_t *status;
};

// The new tokens of request b: how many, the first one's row and position.  0 for
// a request that was rejected; one whose lengths and offsets do not go together
// is too.
__device__ __forceinline__ int request(const RaggedArgs &a, int b, int &row0, int &P, uint32_t &bad)
{
    const int o0 = a.offsets[b], o1 = a.offsets[b + 1], T = a.len.total_abs[b];
    row0 = o0;
    P = a.len.past_abs[b];
    bad = 0;
    if (a.len.cache_total[b] < 0 || P < 0)
        return 0;
    if (T < P || o0 < 0 || o1 < o0 || o1 > a.tokens || T - P != o1 - o0)
        bad = KVC_DEV_SEQLEN_RANGE;
    else if (T > (int64_t)a.max_pages * a.page_size)
        bad = KVC_DEV_CAPACITY;
    return bad ? 0 : o1 - o0;
}

// A block a token and kv head, a warp a query head, the keys one by one.
template <typename T, int D>
__global__ void __launch_bounds__(512)
ragged_attn_kernel(const RaggedArgs a)
{
    constexpr int PER = D / 32;
    const int t = blockIdx.x, h = blockIdx.y, lane = threadIdx.x & 31, head = h * a.group + (threadIdx.x >> 5);
    int b = 0, n = 0, row0 = 0, P = 0;
    if (t == 0 && h == 0)
        for (int i = threadIdx.x; i < a.batch; i += blockDim.x) {
            uint32_t bad;
            request(a, i, row0, P, bad);
            if (bad)
                kvc::raise_status(a.status, bad);
        }
    for (; b < a.batch; ++b) {
        uint32_t bad;
        n = request(a, b, row0, P, bad);
        if (n && t >= row0 && t < row0 + n)
            break;
    }
    if (b == a.batch)
        return;
    const int pos = P + t - row0, first = a.window > 0 ? max(0, pos - a.window + 1) : 0;
    float q[PER], o[PER], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
        q[e] = kvc::Elem<T>::to_f32(static_cast<const T *>(a.q)[((int64_t)t * a.q_heads + head) * D + lane + 32 * e]);
        o[e] = 0.f;
    }
    for (int r = first; r <= pos; ++r) {
        const int64_t id = a.table[(int64_t)b * a.max_pages + r / a.page_size];
        if (id < 0 || id >= a.n_pool) {
            if (lane == 0)
                kvc::raise_status(a.status, KVC_DEV_INDEX_OOB);
            continue;
        }
        const int64_t at = ((id * a.kv_heads + h) * a.page_size + r % a.page_size) * D + lane;
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < PER; ++e)
            s = fmaf(q[e], kvc::Elem<T>::to_f32(static_cast<const T *>(a.k)[at + 32 * e]), s);
#pragma unroll
        for (int d = 16; d; d >>= 1)
            s += __shfl_xor_sync(0xffffffffu, s, d);
        s *= a.scale;
        const float top = fmaxf(m, s), old = m == -INFINITY ? 0.f : expf(m - top), p = expf(s - top);
        l = l * old + p;
        m = top;
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const float v = kvc::Elem<T>::to_f32(static_cast<const T *>(a.v)[at + 32 * e]);
            o[e] = o[e] * old + p * fmaf(v, 0.f, v);  // (an infinity counts as NaN)
        }
    }
#pragma unroll
    for (int e = 0; e < PER; ++e)
        static_cast<T *>(a.out)[((int64_t)t * a.q_heads + head) * D + lane + 32 * e] = kvc::Elem<T>::from_f32(o[e] / l);
}

template <typename T> void launch_attn(const RaggedArgs &a, int D, cudaStream_t stream)
{
    const dim3 grid(a.tokens, a.kv_heads);
    if (D == 64)
        ragged_attn_kernel<T, 64><<<grid, 32 * a.group, 0, stream>>>(a);
    else if (D == 128)
        ragged_attn_kernel<T, 128><<<grid, 32 * a.group, 0, stream>>>(a);
    else
        ragged_attn_kernel<T, 256><<<grid, 32 * a.group, 0, stream>>>(a);
}

} // namespace

KVC_API size_t kvc_gqa_ragged_workspace_size(int batch, int tokens, int q_heads, int kv_heads, int head_dim)
{
    if (batch < 1 || tokens < 1 || kv_heads < 1 || q_heads < 1 || q_heads % kv_heads != 0 || head_dim < 1)
        return 0;
    return 256;
}

KVC_API kvc_status kvc_gqa_ragged(void *out, const void *q, const void *k_pool, const void *v_pool,
                                  const int32_t *offsets, const int32_t *block_table, int max_pages,
                                  int64_t n_pool_pages, int page_size, kvc_lengths len, int batch, int tokens,
                                  int q_heads, int kv_heads, int head_dim, int dtype, int local_window_size,
                                  float scale, void *workspace, size_t workspace_bytes, int32_t *dev_status,
                                  void *stream_)
{
    if (kvc_host::elem_bytes_of(dtype) == 0)
        return KVC_ERR_DTYPE;
    if (dtype == KVC_F32)
        return KVC_ERR_UNSUPPORTED;
    if (batch < 0 || tokens < 0 || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads != 0 || max_pages < 1 ||
        n_pool_pages < 1 || page_size < 16 || page_size % 16 != 0)
        return KVC_ERR_SHAPE;
    if ((head_dim != 64 && head_dim != 128 && head_dim != 256) || q_heads / kv_heads > 16 || kv_heads > 32767 ||
        batch > 65535)
        return KVC_ERR_UNSUPPORTED;
    if ((int64_t)max_pages * page_size > INT32_MAX || n_pool_pages > INT32_MAX ||
        n_pool_pages * page_size > INT32_MAX / kv_heads || (int64_t)tokens * q_heads > INT32_MAX)
        return KVC_ERR_CAPACITY;
    if (batch == 0 || tokens == 0)
        return KVC_OK;
    if (!out || !q || !k_pool || !v_pool || !offsets || !block_table || !kvc_host::lengths_ok(len))
        return KVC_ERR_NULL;
    for (const void *p : {(const void *)out, q, k_pool, v_pool})
        if (!kvc_host::aligned16(p))
            return KVC_ERR_ALIGN;
    const size_t pool = (size_t)n_pool_pages * page_size * kv_heads * head_dim * 2,
                 rows = (size_t)tokens * q_heads * head_dim * 2;
    if (kvc_host::overlaps(out, rows, q, rows) || kvc_host::overlaps(out, rows, k_pool, pool) ||
        kvc_host::overlaps(out, rows, v_pool, pool))
        return KVC_ERR_SHAPE;
    if (!workspace || workspace_bytes < kvc_gqa_ragged_workspace_size(batch, tokens, q_heads, kv_heads, head_dim))
        return KVC_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u)
        return KVC_ERR_ALIGN;
    const RaggedArgs a{out, q, k_pool, v_pool, offsets, block_table, max_pages, page_size, n_pool_pages, len, batch,
                       tokens, q_heads, kv_heads, q_heads / kv_heads, local_window_size,
                       scale == 0.f ? 1.0f / sqrtf((float)head_dim) : scale, dev_status};
    if (dtype == KVC_BF16)
        launch_attn<__nv_bfloat16>(a, head_dim, static_cast<cudaStream_t>(stream_));
    else
        launch_attn<__half>(a, head_dim, static_cast<cudaStream_t>(stream_));
    return kvc_host::launch_status();
}
