// kvc_quant.cu -- a KV cache whose rows are quantised as they are written, and
// its readers ("Persistent KV Cache and Decode Performance Roadmap", "Phase 3:
// cache quantization and fusion"; the ring of "Stateful decode & KV cache",
// "Sliding-window ring buffer").
//
// A row x of head_dim values (K rotated at its absolute position, in float32)
// is held as 8-bit codes and one float32 scale:
//     s = max|x| / 127 (int8) or / 448 (e4m3),  code = nearest(x / s)
// so that code * s is the row read back.  A row of zeros has s = 0; a row with
// a NaN or an infinity has s = NaN and codes 0, so it reads back as NaN.
//
//   quant_append_kernel   new rows -> codes and scales
//   dequant_rows_kernel   rows [0, L) back to 16 or 32 bits
//   quant_decode_kernel   one-token GQA attention over the codes
//   quant_merge_kernel    joins the partial results of rows that several CTAs
//                         worked on
#include <algorithm>
#include <cmath>
#include <type_traits>

#include <cuda_fp8.h>

#include "kvc_common.cuh"
#include "kvc_flat.cuh"

namespace {

constexpr float kLog2e = 1.4426950408889634f;

template <int FMT> constexpr float kTop = FMT == KVC_INT8 ? 127.f : 448.f;

// --------------------------------------------------------------------------
// writing
// --------------------------------------------------------------------------

// eight values of a row, as they lie in memory
template <typename T> struct Raw8 { uint32_t w[sizeof(T) * 2]; };

template <typename T> __device__ __forceinline__ Raw8<T> load8(const T *p)
{
    Raw8<T> r;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
        const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p) + i);
        r.w[4 * i] = v.x, r.w[4 * i + 1] = v.y, r.w[4 * i + 2] = v.z, r.w[4 * i + 3] = v.w;
    }
    return r;
}
template <typename T> __device__ __forceinline__ void to_f32(const Raw8<T> &r, float (&x)[8])
{
    const T *e = reinterpret_cast<const T *>(r.w);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        x[i] = kvc::Elem<T>::to_f32(e[i]);
}

__device__ __forceinline__ float max_nan(float x, float y)
{
    float z;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
    return z;
}

// Eight values of a row, LPR lanes a row, to codes.  The maximum carries a NaN,
// so a row that is not finite shows in it.  x / s is needed to the last bit (a
// code hangs on it), and s is a row's: with r the correctly rounded 1 / s, and no
// overflow or underflow on the way, q = x r corrected by its remainder,
// q + (x - q s) r, is the correctly rounded quotient (Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990): three
// operations a value in the place of a division's ten or more; the scale itself is
// top / 127 in the same way.  Rows with a maximum outside [2^-100, 2^100] divide.
template <int FMT, int LPR>
__device__ __forceinline__ uint2 quantise8(const float (&x)[8], float &scale)
{
    float top = fabsf(x[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i)
        top = max_nan(top, fabsf(x[i]));
#pragma unroll
    for (int d = 1; d < LPR; d <<= 1)
        top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, d));
    uint2 out = make_uint2(0, 0);
    if (!(top < INFINITY)) {
        scale = __uint_as_float(0x7fc00000u);
        return out;
    }
    float y[8];
    const bool usual = top >= 7.8886091e-31f && top <= 1.2676506e30f;  // 2^-100, 2^100
    if (usual) {
        constexpr float rt = 1.f / kTop<FMT>;
        const float q0 = __fmul_rn(top, rt);
        scale = __fmaf_rn(__fmaf_rn(-q0, kTop<FMT>, top), rt, q0);
        const float r = __frcp_rn(scale);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float q = __fmul_rn(x[i], r);
            y[i] = __fmaf_rn(__fmaf_rn(-q, scale, x[i]), r, q);
        }
    } else {
        scale = __fdiv_rn(top, kTop<FMT>);
        if (scale == 0.f)
            return out;
        // (a subnormal scale may round the quotient past the largest code)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            y[i] = fminf(fmaxf(__fdiv_rn(x[i], scale), -kTop<FMT>), kTop<FMT>);
    }
    uint32_t w[2];
    if constexpr (FMT == KVC_INT8) {
        uint32_t n[8];
        // y + 1.5 2^23 rounds y to a whole number, ties to even, in the low bits
#pragma unroll
        for (int i = 0; i < 8; ++i)
            n[i] = __float_as_uint(y[i] + 12582912.f);
#pragma unroll
        for (int h = 0; h < 2; ++h)
            w[h] = __byte_perm(__byte_perm(n[4 * h], n[4 * h + 1], 0x0040), __byte_perm(n[4 * h + 2], n[4 * h + 3], 0x0040),
                               0x5410);
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            w[h] = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(y[4 * h], y[4 * h + 1]), __NV_SATFINITE, __NV_E4M3) |
                   (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(y[4 * h + 2], y[4 * h + 3]), __NV_SATFINITE, __NV_E4M3)
                       << 16;
    }
    return make_uint2(w[0], w[1]);
}

struct AppendArgs {
    uint8_t *kq, *vq;
    float *ks, *vs;
    const void *new_k, *new_v;
    kvc_lengths len;
    int batch, kv_heads, S, D;
    int64_t C;
    int ring;
    const float *cos_t, *sin_t;
    int64_t rope_max_pos;
    int32_t *status;
};

// LPR lanes write one row of K and the same row of V: eight columns a lane
// (lanes past head_dim idle along), the rotation's partner columns c +- D / 2
// fetched from the lane that holds them.  A block walks the rows of one (batch
// row, head) with the next rows under way while it works on these; the first
// are asked for before the lengths say where they go.
// 2 x 64 x 2048 rows of 128 (67 MB in, 34 out, bf16 to int8): 32 us, 3.1 TB/s.  The
// instructions bound it (69 % of the issue slots: maximum, scale, exact quotients,
// packing); with a row a block and nothing ahead it took 46 us.
constexpr int kAppendThreads = 256;
template <typename T, int FMT, int LPR>
__global__ void __launch_bounds__(kAppendThreads)
quant_append_kernel(const AppendArgs a)
{
    constexpr int RPB = kAppendThreads / LPR;
    const int sub = threadIdx.x % LPR, t = threadIdx.x / LPR;
    const int slice = blockIdx.y, b = slice / a.kv_heads;
    const int c0 = 8 * sub, half = a.D / 2;
    const bool low = c0 < half, col = c0 < a.D;
    const T *nk = static_cast<const T *>(a.new_k) + (int64_t)slice * a.S * a.D + c0;
    const T *nv = static_cast<const T *>(a.new_v) + (int64_t)slice * a.S * a.D + c0;
    Raw8<T> kn = {}, vn = {};
    int base = blockIdx.x * RPB;
    if (col && base + t < a.S) {
        kn = load8(nk + (int64_t)(base + t) * a.D);
        vn = load8(nv + (int64_t)(base + t) * a.D);
    }
    const int P = a.len.past_abs[b];
    bool write = a.len.cache_total[b] >= 0 && P >= 0;
    const bool lead = threadIdx.x == 0 && blockIdx.x == 0 && slice % a.kv_heads == 0;
    if (write && a.cos_t && (int64_t)P + a.S > a.rope_max_pos) {
        if (lead)
            kvc::raise_status(a.status, KVC_DEV_ROPE_RANGE);
        write = false;
    }
    if (write && !a.ring && (int64_t)P + a.S > a.C) {
        // lengths computed for another capacity: refuse rather than overrun
        if (lead)
            kvc::raise_status(a.status, KVC_DEV_CAPACITY);
        write = false;
    }
    if (!write)
        return;  // the whole block
    // D is a multiple of 16, so the partner columns are one lane's
    const int from = ((threadIdx.x & 31) - sub + (low ? sub + half / 8 : sub - half / 8)) & 31;
    const float sign = low ? -1.f : 1.f;
    const int step = gridDim.x * RPB;
    for (; base < a.S; base += step) {
        const int i = base + t;
        const bool in = col && i < a.S;
        const int pos = P + i;
        const Raw8<T> kr = kn, vr = vn;
        float cs[8] = {}, sn[8] = {};
        if (a.cos_t && in) {
            const int64_t at = (int64_t)pos * half + (low ? c0 : c0 - half);
            to_f32(load8(a.cos_t + at), cs);
            to_f32(load8(a.sin_t + at), sn);
        }
        if (col && i + step < a.S) {
            kn = load8(nk + (int64_t)(i + step) * a.D);
            vn = load8(nv + (int64_t)(i + step) * a.D);
        }
        float k[8], v[8], vs, ks;
        to_f32(vr, v);
        const uint2 vc = quantise8<FMT, LPR>(v, vs);
        to_f32(kr, k);
        if (a.cos_t) {
            Raw8<T> orow;
#pragma unroll
            for (int e = 0; e < (int)sizeof(T) * 2; ++e)
                orow.w[e] = __shfl_sync(0xffffffffu, kr.w[e], from);
            float other[8];
            to_f32(orow, other);
            // lo cos - hi sin for a column of the lower half, hi cos + lo sin for one of the upper
#pragma unroll
            for (int e = 0; e < 8; ++e)
                k[e] = __fadd_rn(__fmul_rn(k[e], cs[e]), __fmul_rn(other[e], __fmul_rn(sn[e], sign)));
            if (a.D != 8 * LPR && !col) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    k[e] = 0.f;  // (a lane past the columns has turned another row's)
            }
        }
        const uint2 kc = quantise8<FMT, LPR>(k, ks);
        // a ring keeps only the last C rows of the step
        if (in && !(a.ring && (int64_t)i < (int64_t)a.S - a.C)) {
            const int64_t r = (int64_t)slice * a.C + (a.ring ? (int)((uint32_t)pos % (uint32_t)a.C) : pos);
            *reinterpret_cast<uint2 *>(a.kq + r * a.D + c0) = kc;
            *reinterpret_cast<uint2 *>(a.vq + r * a.D + c0) = vc;
            if (sub == 0) {
                a.ks[r] = ks;
                a.vs[r] = vs;
            }
        }
    }
}

// --------------------------------------------------------------------------
// reading back
// --------------------------------------------------------------------------

// four codes of a word as floats
template <int FMT> __device__ __forceinline__ void codes4(uint32_t w, float (&f)[4])
{
    if constexpr (FMT == KVC_INT8) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f[i] = (float)(int)(signed char)(w >> (8 * i));
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (16 * i)), __NV_E4M3);
            const float2 v = __half22float2(__half2(h));
            f[2 * i] = v.x;
            f[2 * i + 1] = v.y;
        }
    }
}

struct DequantArgs {
    void *k_out, *v_out;
    const uint8_t *kq, *vq;
    const float *ks, *vs;
    kvc_lengths len;
    int batch, kv_heads, D;
    int64_t C, R;
    int ring;
    int32_t *status;
};

// Eight codes a thread (16 bytes out, side by side over a warp), D / 8 threads a
// row, kRowsAhead rows under way.
// 2 x 64 x 4096 rows of 128 (69 MB in, 134 out): 25 us, part of the writes still in
// L2 at the end; 31 us with 16 codes a thread.
constexpr int kRowsAhead = 4;
constexpr int kDequantCtas = 12;
template <typename T, int FMT>
__global__ void __launch_bounds__(256)
dequant_rows_kernel(const DequantArgs a)
{
    const int slice = blockIdx.y;
    const int b = slice / a.kv_heads;
    const int L = a.len.cache_total[b], total = a.len.total_abs[b];
    if (L < 0)
        return;
    if (L > a.R || L > a.C || total < L) {
        if (threadIdx.x == 0 && blockIdx.x == 0 && slice % a.kv_heads == 0)
            kvc::raise_status(a.status, KVC_DEV_CAPACITY);
        return;
    }
    const int pieces = a.D / 8, rpb = 256 / pieces;
    const int c0 = threadIdx.x % pieces * 8, sub = threadIdx.x / pieces;
    if (sub >= rpb)
        return;
    const uint32_t cap = (uint32_t)a.C, first = a.ring ? (uint32_t)(total - L) % cap : 0u;
    const uint8_t *src = (blockIdx.z == 0 ? a.kq : a.vq) + (int64_t)slice * a.C * a.D + c0;
    const float *scales = (blockIdx.z == 0 ? a.ks : a.vs) + (int64_t)slice * a.C;
    T *dst = static_cast<T *>(blockIdx.z == 0 ? a.k_out : a.v_out) + (int64_t)slice * a.R * a.D + c0;
    const int64_t step = (int64_t)gridDim.x * kRowsAhead * rpb;
    uint2 q[kRowsAhead];
    float s[kRowsAhead];
    auto fetch = [&](int64_t r0) {
#pragma unroll
        for (int u = 0; u < kRowsAhead; ++u) {
            // (a row past the last is the last again)
            const uint32_t r = (uint32_t)min(r0 + u * rpb, (int64_t)L - 1) + first;
            const uint32_t slot = min(r, r - cap);
            q[u] = __ldg(reinterpret_cast<const uint2 *>(src + (uint64_t)slot * a.D));
            s[u] = __ldg(scales + slot);
        }
    };
    int64_t r0 = (int64_t)blockIdx.x * kRowsAhead * rpb + sub;
    if (r0 < L)
        fetch(r0);
    for (; r0 < L; r0 += step) {
        Raw8<T> out[kRowsAhead];
#pragma unroll
        for (int u = 0; u < kRowsAhead; ++u) {
            float f[8];
            codes4<FMT>(q[u].x, *reinterpret_cast<float (*)[4]>(f));
            codes4<FMT>(q[u].y, *reinterpret_cast<float (*)[4]>(f + 4));
            T *e = reinterpret_cast<T *>(out[u].w);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                e[i] = kvc::Elem<T>::from_f32(f[i] * s[u]);
        }
        if (r0 + step < L)
            fetch(r0 + step);
#pragma unroll
        for (int u = 0; u < kRowsAhead; ++u) {
            const int64_t r = r0 + u * rpb;
            if (r < L) {
                uint4 *to = reinterpret_cast<uint4 *>(dst + r * a.D);
#pragma unroll
                for (int i = 0; i < (int)sizeof(T) / 2; ++i)
                    to[i] = make_uint4(out[u].w[4 * i], out[u].w[4 * i + 1], out[u].w[4 * i + 2], out[u].w[4 * i + 3]);
            }
        }
    }
}

// --------------------------------------------------------------------------
// one-token attention over the codes
// --------------------------------------------------------------------------

constexpr int kWarps = 4;
constexpr int kRowCost = 2;         // units (kvc_flat.cuh) that a row costs beside its keys
constexpr float kNone = -1e30f;     // a reference maximum before any score (finite: differences stay numbers)
constexpr float kSlack = 8.f;       // log2 units a score may exceed its reference by

struct QuantDecodeArgs {
    void *out;
    const void *q;
    const uint8_t *kq, *vq;
    const float *ks, *vs;
    kvc_lengths len;
    int batch, q_heads, kv_heads, group;
    int64_t C;
    int ring, window;
    float scale_log2;
    const float *cos_t, *sin_t;
    int64_t rope_max_pos;
    int unit;                        // keys of a unit of work
    int grid, row_cost;              // CTAs of the attention launch, units that a row costs beside its keys
    float *ws_o, *ws_m, *ws_l;       // [2 * grid][group] (x D)
    int32_t *status;
};

// the visible keys of batch row b, at absolute length T with L rows resident
__device__ __forceinline__ int visible(const QuantDecodeArgs &a, int b, int &T, int &L, uint32_t &bad)
{
    L = a.len.cache_total[b];
    T = a.len.total_abs[b];
    bad = L < 0 ? 0u
          : L > a.C || T < L ? (uint32_t)KVC_DEV_CAPACITY
          : a.cos_t && (int64_t)T > a.rope_max_pos ? (uint32_t)KVC_DEV_ROPE_RANGE : 0u;
    if (L < 0 || bad)
        return 0;
    return a.window > 0 ? min(L, a.window) : L;
}
// The slot of the first of them (they wrap at C).  Position p of a ring lies in slot
// p mod C; row r of a contiguous cache holds position T - L + r, and T may be more
// than L, or than C (a window or a compaction has moved the rows down), so the last
// n rows start at L - n, not at T - n.
__device__ __forceinline__ uint32_t first_slot(const QuantDecodeArgs &a, int n, int T, int L)
{
    return a.ring ? (uint32_t)(T - n) % (uint32_t)a.C : (uint32_t)(L - n);
}

// Units of a row on the line that the CTAs share: its keys', and kRowCost that hold
// none but stand for what a CTA spends on a row beside its keys.
__device__ __forceinline__ int row_units(const QuantDecodeArgs &a, int n, int unit)
{
    return n > 0 ? (n + unit - 1) / unit + a.row_cost : 0;
}

__device__ __forceinline__ float fast_exp2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float fast_log2(float x)
{
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t movm_trans(uint32_t x)
{
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Four codes as two pairs of halves: bytes 0 and 2 in `even`, 1 and 3 in `odd` for
// int8, bytes 0, 1 and 2, 3 for e4m3 (its conversion takes neighbours).  Every
// e4m3 value is a half.  An int8 code c with its sign bit flipped is the byte
// u = c + 128:
//   BIASED: u alone in a half is the subnormal u 2^-24, so one logic operation
//     masks and flips two codes at once, and the sum over d of q_d u_d is
//     corrected by 128 sum q_d, a constant of the head (both are sums of about the
//     same size, so no digits go);
//   else: under the high byte 0x64 it is the half 1024 + u; subtracting 1152
//     leaves c.  (A bias of 128 on the values would be far above what their
//     weighted mean leaves.)
// The shift of the odd bytes is a multiplication, for the pipe that has room: the
// logic pipe takes a warp's instruction in two clocks and bounds the kernel.
template <int FMT, bool BIASED> __device__ __forceinline__ void codes_to_halves(uint32_t w, uint32_t &even, uint32_t &odd)
{
    if constexpr (FMT == KVC_INT8) {
        constexpr uint32_t flip = BIASED ? 0x00800080u : 0x64806480u;
        even = (w & 0x00ff00ffu) ^ flip;
        odd = (__umulhi(w, 1u << 24) & 0x00ff00ffu) ^ flip;
        if constexpr (!BIASED) {
            asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(even) : "r"(0x64806480u));
            asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(odd) : "r"(0x64806480u));
        }
    } else {
        asm("{\n\t.reg .b16 l, h;\n\t"
            "mov.b32 {l, h}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
            "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=r"(even), "=r"(odd)
            : "r"(w));
    }
}
// the codes of columns 2 e and 2 e + 1 of two keys' words x, y as the pairs
// (x_2e, y_2e), (x_2e+1, y_2e+1)
template <int FMT>
__device__ __forceinline__ void pairs_of(uint32_t x, uint32_t y, int e, uint32_t &first, uint32_t &second)
{
    constexpr uint32_t sel[2] = {FMT == KVC_INT8 ? 0x5410u : 0x5140u, FMT == KVC_INT8 ? 0x7632u : 0x7362u};
    codes_to_halves<FMT, false>(__byte_perm(x, y, sel[e]), first, second);
}

// asynchronous copies to shared memory: 16 bytes of codes past L1, 4 of a scale
__device__ __forceinline__ void copy16(uint32_t to, const uint8_t *from)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t to, const float *from)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ uint4 lds16(uint32_t p)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t p)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(p) : "memory");
    return v;
}
// Tiles of 16 keys that a warp takes in one step: two where registers and shared
// memory allow, whose chains of products, exponentials and conversions fill each
// other's waits.  A unit of work is a step of the four warps.
__host__ __device__ constexpr int tiles_of(int D, int HB) { return D * HB <= 128 ? 2 : 1; }
__host__ __device__ constexpr int unit_of(int D, int HB) { return 16 * tiles_of(D, HB) * kWarps; }
// resident CTAs an SM, by the registers that O and the query fragments take
__host__ __device__ constexpr int ctas_per_sm(int D, int HB) { return D * HB <= 256 ? 3 : 2; }

template <int D, int HB, bool F16> struct QuantSmem {
    static constexpr int HEADS = 8 * HB;
    static constexpr int Q_ROWS = F16 ? 2 * HEADS : HEADS;  // fp16: what a row's rounding left, in a second one
    static constexpr int Q_PITCH = D * 2 + 8;     // bytes: a fragment's 16 half-warp reads hit 16 distinct 8-byte banks
    static constexpr int Q_BYTES = Q_ROWS * Q_PITCH;
    // A stage of a warp's ring, a tile of 16 keys: K piece by piece, each lane's own 16 bytes; V row by
    // row, its 16-byte chunks swizzled (v_chunk); a scale a lane
    static constexpr int K_PIECES = 2 * (D / 64), V_OFF = K_PIECES * 512, S_OFF = V_OFF + 16 * D;
    static constexpr int TILE = S_OFF + 128;                // and a scale
    static constexpr int TILES = tiles_of(D, HB), STAGE = TILES * TILE;
    static constexpr int RING_OFF = (Q_BYTES + 15) / 16 * 16;
    // each query row's factor and bias, then m and l of each warp
    static constexpr int ML_BYTES = (2 * Q_ROWS + 2 * kWarps * HEADS) * 4;
    static constexpr int FIXED = RING_OFF + ML_BYTES;
    static constexpr int FIT = ((228 * 1024 / ctas_per_sm(D, HB) - 1024) - FIXED) / (kWarps * STAGE);
    static constexpr int STAGES = FIT < 4 ? FIT : 4;
    static constexpr int WARP_RING = STAGES * STAGE;
    static constexpr int ML_OFF = RING_OFF + kWarps * WARP_RING;
    static constexpr int TOTAL = ML_OFF + ML_BYTES;
    // at a segment's end a warp's O takes the place of its ring
    static constexpr int O_PITCH = D + 4;                   // floats
    static_assert(STAGES >= 2 && HEADS * O_PITCH * 4 <= WARP_RING, "two stages, and O in their place");
};

// byte offset of the 16-byte chunk c of row r of a tile of V: such that the eight
// lanes of a phase, which read two neighbouring chunks (or, for D = 64, four
// halves of two) of rows 2 t, hit distinct banks
template <int D> __device__ __forceinline__ uint32_t v_chunk(int r, int c)
{
    if constexpr (D == 64)
        return (r >> 1) * 128 + ((((r & 1) << 2) | c) ^ ((r >> 1 & 3) << 1)) * 16;
    else
        return r * D + (c ^ (r & 7)) * 16;
}

// Attention of one query over the codes of a flat share of the batch
// (kvc_flat.cuh), a warp taking 16 keys at a time into the operands of mma.sync
// m16n8k16:
//   scores  S^T[key][head] = K[key][:] . Q[head][:]    A = K codes as halves
//   output  O^T[d][head] += V^T[d][key] w[key][head]   A = V codes as halves
// The sum over d does not care for the order of d, so lane (g, t) takes 16
// consecutive codes of key g (and g + 8) as its share of four k-steps, and the
// query's fragments are laid out to match: one 16-byte load feeds four MMAs.
// Likewise the rows d of O^T are taken in the order in which lane (g, .) holds
// the 16 (or 8) consecutive codes of its keys' V rows; the bytes of two keys
// are interleaved with one permute for each two codes.  So a lane needs only
// 16-byte pieces.  A warp copies them asynchronously into a ring of its own in
// shared memory, a few tiles ahead, and reads them back without conflicts.
// The keys' scales stay out of the products: s = (q . code) * ks in float32,
// and a value's weight is 2^(s + log2(vs) - mo), with a reference maximum mo
// of its own beside the m of the sum l = sum 2^(s - m).  So the weights are
// rounded to halves near 1 however the rows' scales differ (a value row of
// tiny scale may carry all of the probability).
// The query is scaled by a power of two to [2^14, 2^15) at its largest and
// rounded to halves: 11 bits, three more than a bf16 query has, whose result's
// own rounding hides it.  For fp16 what the roundings of the query and of the
// weights leave is taken along as halves too (the error falls from 5e-4 to the 2e-4
// of the result's own rounding).  With groups of four heads or fewer half of the
// eight columns are free, and column r + 4 takes what column r leaves: the two
// columns' scores are added before the softmax and their outputs at the end, at the
// price of four shuffles a tile (3 % of the time).  With more heads it is a second
// product into the same sums.
// 32 x 8 rows of 512 to 8192 keys, head_dim 128, int8 (295 MB): 61 us, 4.8 TB/s; a
// ring of 8 x 8 x 4096 keys of 256, e4m3: 29 us.  HBM bounds it while every CTA runs,
// 5.2 TB/s, but the SMs do not get equal parts of it and the last ends 15 % late; the
// logic pipe, which the codes' conversion takes, is half full.
template <typename T, int FMT, int D, int HB>
__global__ void __launch_bounds__(32 * kWarps, ctas_per_sm(D, HB))
quant_decode_kernel(const QuantDecodeArgs a)
{
    constexpr bool F16 = std::is_same<T, __half>::value;
    using SM = QuantSmem<D, HB, F16>;
    constexpr int HEADS = SM::HEADS;
    constexpr int KV4 = D / 64;               // 16-byte pieces of K a lane takes of one key
    constexpr int VW = D / 32;                // 32-bit words of V a lane takes of one key
    constexpr bool QREG = HB == 1;            // query fragments in registers
    const bool split = F16 && HB == 1 && a.group <= 4;  // columns r + 4
    const bool twice = F16 && !split;                  // second products
    constexpr int TILES = SM::TILES, kUnit = unit_of(D, HB);
    extern __shared__ __align__(16) uint8_t smem[];
    float *q_factor = reinterpret_cast<float *>(smem + SM::ML_OFF);
    float *q_bias = q_factor + SM::Q_ROWS;
    float *m_sh = q_bias + SM::Q_ROWS, *l_sh = m_sh + kWarps * HEADS;

    kvc::grid_dep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int c = blockIdx.x;
    auto units = [&](int b) {
        int T, L;
        uint32_t bad;
        const int n = visible(a, b, T, L, bad);
        if (bad && c == 0 && warp == 0)
            kvc::raise_status(a.status, bad);
        return row_units(a, n, kUnit);
    };
    int x, x_end, b, base;
    kvc_flat::share_of_cta(a.batch, a.kv_heads, units, a.grid, c, x, x_end, b, base);

    for (int seg = 0; x < x_end; ++seg) {
        int T_abs, L;
        uint32_t bad;
        const int n = visible(a, b, T_abs, L, bad);
        const int line = row_units(a, n, kUnit), nu = line - a.row_cost;
        const int h = (x - base) / line;
        const int p0 = (x - base) - h * line, p1 = min(line, p0 + (x_end - x));
        // the units that stand for the row's cost hold no keys
        const int u0 = max(0, p0 - a.row_cost), u1 = p1 - a.row_cost;
        if (u1 <= u0)
            break;  // (the share ends in them)
        const int64_t slice = (int64_t)b * a.kv_heads + h;

        const uint8_t *kb = a.kq + slice * a.C * D + 16 * t, *vb = a.vq + slice * a.C * D + 16 * (lane % (D / 16));
        const float *ksb = a.ks + slice * a.C, *vsb = a.vs + slice * a.C;
        const uint32_t cap = (uint32_t)a.C, start = first_slot(a, n, T_abs, L);
        // 16 keys whose rows follow one another: one address each for the keys, the values and the
        // scales, and constant steps.  Else (the last keys, or a ring's end among them) each row has its
        // own, a key past the last being the last again: its score is masked, and what is loaded is
        // finite or seen.  start + j wraps at C at most once.
        auto in_line = [&](int j0) {
            const uint32_t r = start + (uint32_t)j0;
            return j0 + 16 <= n && (r >= cap || r + 16 <= cap);
        };
        auto slot = [&](int j) {
            const uint32_t r = start + (uint32_t)min(j, n - 1);
            return min(r, r - cap);  // (r - cap is huge below cap)
        };
        const uint32_t ring = kvc::smem_u32(smem) + SM::RING_OFF + warp * SM::WARP_RING;
        const uint32_t my16 = ring + lane * 16, my_s = ring + SM::S_OFF + lane * 4;
        // V comes in whole rows, D / 16 lanes a row: with each lane fetching what it needs itself (32
        // bytes of four rows for eight lanes) the memory system moved twice the bytes of V to the SM
        constexpr int V_LANES = D / 16, V_ROWS = 32 / V_LANES;  // rows a load covers
        const int v_row = lane / V_LANES, v_col = lane % V_LANES;
        uint32_t v_to[16 / V_ROWS];
#pragma unroll
        for (int i = 0; i < 16 / V_ROWS; ++i)
            v_to[i] = ring + SM::V_OFF + v_chunk<D>(i * V_ROWS + v_row, v_col);
        // lane (g, t) fetches the scale of key g (t even) or g + 8, K's (t < 2) or V's: four side by side
        const float *scales = t < 2 ? ksb : vsb;
        auto fetch = [&](int j0, uint32_t at) {
            if (in_line(j0)) {
                const uint32_t rk = slot(j0 + g);
                const uint8_t *k = kb + (uint64_t)rk * D, *v = vb + (uint64_t)slot(j0 + v_row) * D;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int i = 0; i < KV4; ++i)
                        copy16(my16 + at + (e * KV4 + i) * 512, k + 8 * e * D + 64 * i);
                }
                copy4(my_s + at, scales + rk + 8 * (t & 1));
#pragma unroll
                for (int i = 0; i < 16 / V_ROWS; ++i)
                    copy16(v_to[i] + at, v + i * V_ROWS * D);
            } else {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t r = slot(j0 + g + 8 * e);
#pragma unroll
                    for (int i = 0; i < KV4; ++i)
                        copy16(my16 + at + (e * KV4 + i) * 512, kb + (uint64_t)r * D + 64 * i);
                }
                copy4(my_s + at, scales + slot(j0 + g + 8 * (t & 1)));
#pragma unroll
                for (int i = 0; i < 16 / V_ROWS; ++i)
                    copy16(v_to[i] + at, vb + (uint64_t)slot(j0 + i * V_ROWS + v_row) * D);
            }
        };
        // the first keys are under way while the queries are made ready
        const int j_end = min(n, u1 * kUnit);
        int j0 = u0 * kUnit + 16 * TILES * warp;
        auto fetch_step = [&](int j0, uint32_t at) {
#pragma unroll
            for (int u = 0; u < TILES; ++u)
                if (u == 0 || j0 + 16 * u < j_end)
                    fetch(j0 + 16 * u, at + u * SM::TILE);
        };
        __syncthreads();  // the last segment's reads of shared memory are done
#pragma unroll
        for (int st = 0; st < SM::STAGES; ++st) {
            if (j0 + st * kUnit < j_end)
                fetch_step(j0 + st * kUnit, st * SM::STAGE);
            copy_commit();
        }

        // ---- the group's queries: rotated, scaled by a power of two, halves ----
        {
            const int64_t pos = (int64_t)T_abs - 1;
            const T *q = static_cast<const T *>(a.q) + slice * a.group * D;
            for (int r = warp; r < (twice ? SM::Q_ROWS : HEADS); r += kWarps) {
                constexpr int PPL = D / 64;  // rotation pairs a lane
                const int first_rest = split ? 4 : HEADS;
                const bool rest = F16 && r >= first_rest;
                const int qr = rest ? r - first_rest : r;
                float lo[PPL], hi[PPL], top = 0.f;
#pragma unroll
                for (int e = 0; e < PPL; ++e) {
                    const int p = lane + 32 * e;
                    lo[e] = hi[e] = 0.f;
                    if (qr < a.group) {
                        lo[e] = kvc::Elem<T>::to_f32(q[qr * D + p]);
                        hi[e] = kvc::Elem<T>::to_f32(q[qr * D + D / 2 + p]);
                        if (a.cos_t)
                            kvc::rope_pair(lo[e], hi[e], a.cos_t[pos * (D / 2) + p], a.sin_t[pos * (D / 2) + p]);
                    }
                    top = fmaxf(top, fmaxf(fabsf(lo[e]), fabsf(hi[e])));
                }
#pragma unroll
                for (int d = 16; d; d >>= 1)
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                // top in [2^(ex - 127), 2^(ex - 126)); both powers of two stay normal
                // (column d of the row goes where codes_to_halves() leaves the code of column d)
                auto place = [](int d) { return FMT == KVC_INT8 ? (d & ~3) | ((d & 1) << 1) | ((d >> 1) & 1) : d; };
                const int ex = min(max((int)(__float_as_uint(top) >> 23), 40), 250);
                const float up = __uint_as_float((uint32_t)(127 + 14 + 127 - ex) << 23);
                const float down = __uint_as_float((uint32_t)(ex - 14) << 23);
                float sum = 0.f;
#pragma unroll
                for (int e = 0; e < PPL; ++e) {
                    __half *row = reinterpret_cast<__half *>(smem + r * SM::Q_PITCH);
                    __half x = __float2half_rn(lo[e] * up), y = __float2half_rn(hi[e] * up);
                    if (rest) {
                        x = __float2half_rn(lo[e] * up - __half2float(x));
                        y = __float2half_rn(hi[e] * up - __half2float(y));
                    }
                    row[place(lane + 32 * e)] = x;
                    row[place(D / 2 + lane + 32 * e)] = y;
                    sum += __half2float(x) + __half2float(y);
                }
                if constexpr (FMT == KVC_INT8) {
#pragma unroll
                    for (int d = 16; d; d >>= 1)
                        sum += __shfl_xor_sync(0xffffffffu, sum, d);
                }
                if (lane == 0) {
                    // score / scale of the key = factor * (products) - bias
                    q_factor[r] = down * a.scale_log2 * (FMT == KVC_INT8 ? 16777216.f : 1.f);
                    q_bias[r] = FMT == KVC_INT8 ? down * a.scale_log2 * 128.f * sum : 0.f;
                }
            }
        }
        __syncthreads();
        auto q_frag = [&](int hb, int step, int rest = 0) {
            // k-step `step` = (span of 64 columns, word of the 16-byte piece)
            return *reinterpret_cast<const uint2 *>(smem + (rest + hb * 8 + g) * SM::Q_PITCH +
                                                    2 * (64 * (step >> 2) + 16 * t + 4 * (step & 3)));
        };
        uint2 qf[QREG ? HB : 1][QREG ? D / 16 : 1];
        if constexpr (QREG) {
#pragma unroll
            for (int hb = 0; hb < HB; ++hb)
#pragma unroll
                for (int st = 0; st < D / 16; ++st)
                    qf[hb][st] = q_frag(hb, st);
        }
        float qs[HB][2], qb[HB][2];
#pragma unroll
        for (int hb = 0; hb < HB; ++hb)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                qs[hb][e] = q_factor[hb * 8 + 2 * t + e];
                qb[hb][e] = q_bias[hb * 8 + 2 * t + e] + (twice ? q_bias[HEADS + hb * 8 + 2 * t + e] : 0.f);
            }

        float o[HB][D / 16][4], m[HB][2], mo[HB][2], l[HB][2];
#pragma unroll
        for (int hb = 0; hb < HB; ++hb) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
                o[hb][i][0] = o[hb][i][1] = o[hb][i][2] = o[hb][i][3] = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m[hb][e] = mo[hb][e] = kNone;
                l[hb][e] = 0.f;
            }
        }

        uint32_t at = 0;  // the stage
        for (; j0 < j_end; j0 += kUnit) {
            copy_wait<SM::STAGES - 1>();
            __syncwarp();  // the values and scales are fetched by all for all
            // ---- scores: two chains of products a head block and tile ----
            float s[TILES][HB][4], s2[TILES][HB][4];
#pragma unroll
            for (int u = 0; u < TILES; ++u)
#pragma unroll
                for (int hb = 0; hb < HB; ++hb)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        s[u][hb][e] = s2[u][hb][e] = 0.f;
#pragma unroll
            for (int i = 0; i < KV4; ++i) {
                uint32_t wa[TILES][4], wb[TILES][4];
#pragma unroll
                for (int u = 0; u < TILES; ++u) {
                    const uint4 ka = lds16(my16 + at + u * SM::TILE + i * 512);
                    const uint4 kc = lds16(my16 + at + u * SM::TILE + (KV4 + i) * 512);
                    wa[u][0] = ka.x, wa[u][1] = ka.y, wa[u][2] = ka.z, wa[u][3] = ka.w;
                    wb[u][0] = kc.x, wb[u][1] = kc.y, wb[u][2] = kc.z, wb[u][3] = kc.w;
                }
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    uint2 f[HB];
#pragma unroll
                    for (int hb = 0; hb < HB; ++hb) {
                        if constexpr (QREG)
                            f[hb] = qf[hb][4 * i + w];
                        else
                            f[hb] = q_frag(hb, 4 * i + w);
                    }
#pragma unroll
                    for (int u = 0; u < TILES; ++u) {
                        uint32_t a0, a1, a2, a3;
                        codes_to_halves<FMT, true>(wa[u][w], a0, a2);
                        codes_to_halves<FMT, true>(wb[u][w], a1, a3);
#pragma unroll
                        for (int hb = 0; hb < HB; ++hb)
                            mma_f16(w & 1 ? s2[u][hb] : s[u][hb], a0, a1, a2, a3, f[hb].x, f[hb].y);
                        if (twice) {
#pragma unroll
                            for (int hb = 0; hb < HB; ++hb) {
                                const uint2 r = q_frag(hb, 4 * i + w, HEADS);
                                mma_f16(w & 1 ? s2[u][hb] : s[u][hb], a0, a1, a2, a3, r.x, r.y);
                            }
                        }
                    }
                }
            }
            const bool tail = j0 + 16 * TILES > n;
            float lv[TILES][2];

            // ---- softmax: x = s - m, y = s + log2(vs) - mo ----
            float x[TILES][HB][4], y[TILES][HB][4], top = kNone;
#pragma unroll
            for (int u = 0; u < TILES; ++u) {
                const uint4 sc = lds16(ring + SM::S_OFF + g * 16 + at + u * SM::TILE);
                const float kk[2] = {__uint_as_float(sc.x), __uint_as_float(sc.y)};
                lv[u][0] = fast_log2(__uint_as_float(sc.z));
                lv[u][1] = fast_log2(__uint_as_float(sc.w));
#pragma unroll
                for (int hb = 0; hb < HB; ++hb) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float sum = s[u][hb][e] + s2[u][hb][e];
                        float z = FMT == KVC_INT8 ? fmaf(sum, qs[hb][e & 1], -qb[hb][e & 1]) : sum * qs[hb][e & 1];
                        if (split)
                            z += __shfl_xor_sync(0xffffffffu, z, 2);
                        z *= kk[e >> 1];
                        float lz = lv[u][e >> 1];
                        if (tail && j0 + 16 * u + g + 8 * (e >> 1) >= n) {
                            z = -INFINITY;
                            lz = 0.f;  // (what a tile past the last holds is not looked at)
                        }
                        s[u][hb][e] = z;
                        x[u][hb][e] = z - m[hb][e & 1];
                        y[u][hb][e] = z + lz - mo[hb][e & 1];
                        top = fmaxf(top, fmaxf(x[u][hb][e], y[u][hb][e]));
                    }
                }
            }
            if (__any_sync(0xffffffffu, top > kSlack)) {
                // a reference is left behind: raise both to the step's maxima
#pragma unroll
                for (int hb = 0; hb < HB; ++hb) {
                    float shrink[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float mx = kNone, my = kNone;
#pragma unroll
                        for (int u = 0; u < TILES; ++u) {
                            mx = fmaxf(mx, fmaxf(s[u][hb][e], s[u][hb][2 + e]));
                            my = fmaxf(my, fmaxf(s[u][hb][e] + lv[u][0], s[u][hb][2 + e] + lv[u][1]));
                        }
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) {
                            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                            my = fmaxf(my, __shfl_xor_sync(0xffffffffu, my, d));
                        }
                        // (fmaxf drops a NaN: the references stay numbers)
                        mx = fmaxf(mx, m[hb][e]);
                        my = fmaxf(my, mo[hb][e]);
                        l[hb][e] *= fast_exp2(m[hb][e] - mx);
                        shrink[e] = fast_exp2(mo[hb][e] - my);
#pragma unroll
                        for (int u = 0; u < TILES; ++u)
#pragma unroll
                            for (int i = e; i < 4; i += 2) {
                                // (a masked key stays at -infinity)
                                x[u][hb][i] += m[hb][e] - mx;
                                y[u][hb][i] += mo[hb][e] - my;
                                if (m[hb][e] == kNone)
                                    x[u][hb][i] = s[u][hb][i] - mx;
                                if (mo[hb][e] == kNone)
                                    y[u][hb][i] = s[u][hb][i] == -INFINITY ? -INFINITY : s[u][hb][i] + lv[u][i >> 1] - my;
                            }
                        m[hb][e] = mx;
                        mo[hb][e] = my;
                    }
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        o[hb][i][0] *= shrink[0];
                        o[hb][i][1] *= shrink[1];
                        o[hb][i][2] *= shrink[0];
                        o[hb][i][3] *= shrink[1];
                    }
                }
            }
            uint32_t b0[TILES][HB], b1[TILES][HB];
            uint32_t r0[F16 ? TILES : 1][F16 ? HB : 1], r1[F16 ? TILES : 1][F16 ? HB : 1];  // (twice) what b0, b1 leave
#pragma unroll
            for (int u = 0; u < TILES; ++u)
#pragma unroll
                for (int hb = 0; hb < HB; ++hb) {
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        l[hb][e] += fast_exp2(x[u][hb][e]) + fast_exp2(x[u][hb][2 + e]);
                    float w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        w[e] = fast_exp2(y[u][hb][e]);
                    __half2 h0 = __floats2half2_rn(w[0], w[1]), h1 = __floats2half2_rn(w[2], w[3]);
                    if constexpr (F16) {
                        const float2 f0 = __half22float2(h0), f1 = __half22float2(h1);
                        const __half2 g0 = __floats2half2_rn(w[0] - f0.x, w[1] - f0.y);
                        const __half2 g1 = __floats2half2_rn(w[2] - f1.x, w[3] - f1.y);
                        if (twice) {
                            r0[u][hb] = movm_trans(*reinterpret_cast<const uint32_t *>(&g0));
                            r1[u][hb] = movm_trans(*reinterpret_cast<const uint32_t *>(&g1));
                        } else if (t >= 2) {
                            h0 = g0;
                            h1 = g1;
                        }
                    }
                    b0[u][hb] = movm_trans(*reinterpret_cast<const uint32_t *>(&h0));
                    b1[u][hb] = movm_trans(*reinterpret_cast<const uint32_t *>(&h1));
                }

            // ---- output ----
            constexpr int VP = D == 64 ? 2 : 4;  // words of a piece
#pragma unroll
            for (int u = 0; u < TILES; ++u) {
                // (a whole tile past the last: its values may be anything, and its weights are zeros)
                if (u > 0 && j0 + 16 * u >= n)
                    break;
#pragma unroll
                for (int p = 0; p < VW / VP; ++p) {
                    uint32_t vr[4][VP];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        // columns of lane (g, .): the 16 (D = 64: 8) from 16 g (8 g) of each 128 on
                        const int row = 2 * t + (e & 1) + 8 * (e >> 1);
                        const uint32_t from = ring + SM::V_OFF + u * SM::TILE + at;
                        if constexpr (D == 64) {
                            const uint2 v = lds8(from + v_chunk<D>(row, g >> 1) + (g & 1) * 8);
                            vr[e][0] = v.x;
                            vr[e][1] = v.y;
                        } else {
                            const uint4 v = lds16(from + v_chunk<D>(row, 8 * p + g));
                            vr[e][0] = v.x;
                            vr[e][1] = v.y;
                            vr[e][2] = v.z;
                            vr[e][3] = v.w;
                        }
                    }
#pragma unroll
                    for (int w = 0; w < VP; ++w) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            // columns 4 w + 2 e and + 1 of keys 2 t, 2 t + 1 and of 2 t + 8, 2 t + 9
                            uint32_t a0, a1, a2, a3;
                            pairs_of<FMT>(vr[0][w], vr[1][w], e, a0, a1);
                            pairs_of<FMT>(vr[2][w], vr[3][w], e, a2, a3);
#pragma unroll
                            for (int hb = 0; hb < HB; ++hb)
                                mma_f16(o[hb][2 * (p * VP + w) + e], a0, a1, a2, a3, b0[u][hb], b1[u][hb]);
                            if constexpr (F16) {
                                if (twice) {
#pragma unroll
                                    for (int hb = 0; hb < HB; ++hb)
                                        mma_f16(o[hb][2 * (p * VP + w) + e], a0, a1, a2, a3, r0[u][hb], r1[u][hb]);
                                }
                            }
                        }
                    }
                }
            }
            __syncwarp();  // every byte of the stage has been read
            if (j0 + SM::STAGES * kUnit < j_end)
                fetch_step(j0 + SM::STAGES * kUnit, at);
            copy_commit();
            at = at + SM::STAGE == SM::WARP_RING ? 0 : at + SM::STAGE;
        }
        copy_wait<0>();

        // ---- join the warps: m, l, then O relative to the common m ----
#pragma unroll
        for (int hb = 0; hb < HB; ++hb) {
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
        }
        __syncthreads();
        float f[HB][2];
#pragma unroll
        for (int hb = 0; hb < HB; ++hb)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float top = -INFINITY;
#pragma unroll
                for (int w = 0; w < kWarps; ++w)
                    top = fmaxf(top, m_sh[w * HEADS + hb * 8 + 2 * t + e]);
                f[hb][e] = exp2f(mo[hb][e] - top);  // O is relative to mo
            }
        auto o_of = [&](int w) { return reinterpret_cast<float *>(smem + SM::RING_OFF + w * SM::WARP_RING); };
        {
            // tile i holds columns 2 i and 2 i + 1 of the lane's run of consecutive columns
            constexpr int RUN = D == 64 ? 8 : 16;
#pragma unroll
            for (int hb = 0; hb < HB; ++hb)
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int i = 0; i < D / 16; i += 2) {
                        const int col = (2 * i / RUN) * 128 + RUN * g + 2 * i % RUN;
                        const float x = f[hb][e];
                        *reinterpret_cast<float4 *>(o_of(warp) + (hb * 8 + 2 * t + e) * SM::O_PITCH + col) =
                            make_float4(o[hb][i][e] * x, o[hb][i][2 + e] * x, o[hb][i + 1][e] * x, o[hb][i + 1][2 + e] * x);
                    }
        }
        __syncthreads();
        const bool whole = u0 == 0 && u1 == nu;
        const int64_t part = 2 * (int64_t)c + (seg == 0 ? 0 : 1);
        for (int idx = threadIdx.x; idx < a.group * D; idx += 32 * kWarps) {
            const int r = idx / D, d = idx % D;
            float top = -INFINITY, sum = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                top = fmaxf(top, m_sh[w * HEADS + r]);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                sum += l_sh[w * HEADS + r] * exp2f(m_sh[w * HEADS + r] - top);
            }
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                v += o_of(w)[r * SM::O_PITCH + d] + (split ? o_of(w)[(r + 4) * SM::O_PITCH + d] : 0.f);
            if (whole) {
                static_cast<T *>(a.out)[slice * a.group * D + idx] = kvc::Elem<T>::from_f32(v / sum);
            } else {
                a.ws_o[(part * a.group + r) * D + d] = v;
                if (d == 0) {
                    a.ws_m[part * a.group + r] = top;
                    a.ws_l[part * a.group + r] = sum;
                }
            }
        }
        x += p1 - p0;
        if (x == base + line * a.kv_heads && x < x_end) {
            base = x;
            do {
                ++b;
            } while (visible(a, b, T_abs, L, bad) == 0);
        }
    }
}

// Joins the partial results of one query head: out = sum_i 2^(m_i - m) o_i /
// sum_i 2^(m_i - m) l_i over the CTAs whose shares cover its row.  The parts'
// m and l are read at once, a part a thread; then D / 4 threads take the
// columns of a part and the block's groups of them the parts in turn.
constexpr int kMergeThreads = 128;
constexpr int kMaxParts = 4096;  // at least the CTAs of the attention launch

template <typename T, int D>
__global__ void __launch_bounds__(kMergeThreads)
quant_merge_kernel(const QuantDecodeArgs a)
{
    constexpr int CT = D / 4, GROUPS = kMergeThreads / CT;
    __shared__ float w_sh[kMaxParts];
    __shared__ float red[2][kMergeThreads / 32];
    __shared__ float4 o_sh[GROUPS][CT];
    const int slice = blockIdx.x, r = blockIdx.y;
    const int b = slice / a.kv_heads, h = slice % a.kv_heads;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto units = [&](int bb) {
        int T, L;
        uint32_t bad;
        return row_units(a, visible(a, bb, T, L, bad), a.unit);
    };
    int b_out, base;
    const int U = kvc_flat::locate(a.batch, a.kv_heads, units, b, b_out, base);
    const int line = units(b);
    const kvc_flat::Shares shares(U, a.grid);
    const int x0 = base + h * line;
    kvc::grid_dep_wait();
    if (line == 0)
        return;
    const int c0 = shares.of(x0 + a.row_cost), n = shares.of(x0 + line - 1) - c0 + 1;
    if (n == 1)
        return;  // written by that CTA
    // the row's segment is the first of its CTA, but in CTA c0 if that began before the row
    const int slot0 = shares.begin(c0) < x0 ? 1 : 0;
    auto part = [&](int i) { return ((int64_t)2 * (c0 + i) + (i == 0 ? slot0 : 0)) * a.group + r; };
    float top = -INFINITY;
    for (int i = threadIdx.x; i < n; i += kMergeThreads) {
        w_sh[i] = a.ws_m[part(i)];
        top = fmaxf(top, w_sh[i]);
    }
#pragma unroll
    for (int d = 16; d; d >>= 1)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    if (lane == 0)
        red[0][warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kMergeThreads / 32; ++w)
        top = fmaxf(top, red[0][w]);
    float sum = 0.f;
    for (int i = threadIdx.x; i < n; i += kMergeThreads) {
        const float w = exp2f(w_sh[i] - top);
        w_sh[i] = w;
        sum += w * a.ws_l[part(i)];
    }
#pragma unroll
    for (int d = 16; d; d >>= 1)
        sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (lane == 0)
        red[1][warp] = sum;
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < kMergeThreads / 32; ++w)
        sum += red[1][w];
    const int col = threadIdx.x % CT, grp = threadIdx.x / CT;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = grp; i < n; i += GROUPS) {
        const float4 o = *(reinterpret_cast<const float4 *>(a.ws_o + part(i) * D) + col);
        const float w = w_sh[i];
        acc.x += w * o.x;
        acc.y += w * o.y;
        acc.z += w * o.z;
        acc.w += w * o.w;
    }
    o_sh[grp][col] = acc;
    __syncthreads();
    if (grp == 0) {
#pragma unroll
        for (int e = 1; e < GROUPS; ++e) {
            const float4 o = o_sh[e][col];
            acc.x += o.x;
            acc.y += o.y;
            acc.z += o.z;
            acc.w += o.w;
        }
        T *to = static_cast<T *>(a.out) + ((int64_t)slice * a.group + r) * D + 4 * col;
        to[0] = kvc::Elem<T>::from_f32(acc.x / sum);
        to[1] = kvc::Elem<T>::from_f32(acc.y / sum);
        to[2] = kvc::Elem<T>::from_f32(acc.z / sum);
        to[3] = kvc::Elem<T>::from_f32(acc.w / sum);
    }
}

// One wave of resident CTAs over all rows, or, where the rows are so few that this
// leaves each too many parts: a unit takes a CTA 0.5 us, and joining 16 parts 0.4 to
// 0.8, so that a row of t units is done soonest by about sqrt(20 t) CTAs (one row of
// 16000 keys of 256: 23 us with 250).  Rows then begin with a CTA each and cost
// nothing beside their keys.
struct Grid {
    int ctas, row_cost;
};
Grid decode_grid(int batch, int kv_heads, int group, int64_t C, int D)
{
    const int hb = group > 8 ? 2 : 1, unit = unit_of(D, hb);
    const int64_t rows = (int64_t)batch * kv_heads, t = (C + unit - 1) / unit;
    const int64_t wave = std::min((int64_t)kvc_host::sm_count() * ctas_per_sm(D, hb), (int64_t)kMaxParts);
    const int64_t few = std::min(t, (int64_t)std::ceil(std::sqrt(20.0 * (double)t)));
    if (rows * few <= wave)
        return {(int)std::max<int64_t>(1, rows * few), 0};
    return {(int)std::min(rows * (t + kRowCost), wave), kRowCost};
}

template <typename T, int FMT, int D, int HB> kvc_status launch_decode(const QuantDecodeArgs &a, cudaStream_t stream)
{
    constexpr int smem = QuantSmem<D, HB, std::is_same<T, __half>::value>::TOTAL;
    auto kern = quant_decode_kernel<T, FMT, D, HB>;
    if (smem > 32 * 1024 &&
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return KVC_ERR_CUDA;
    kern<<<a.grid, 32 * kWarps, smem, stream>>>(a);
    // a row of one unit is never split
    if (a.C > a.unit) {
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(a.batch * a.kv_heads, a.group);
        cfg.blockDim = dim3(kMergeThreads);
        cfg.stream = stream;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        if (cudaLaunchKernelEx(&cfg, quant_merge_kernel<T, D>, a) != cudaSuccess)
            return KVC_ERR_CUDA;
    }
    return kvc_host::launch_status();
}

template <typename T, int FMT> kvc_status launch_decode_dim(const QuantDecodeArgs &a, int D, cudaStream_t stream)
{
    const bool two = a.group > 8;
    switch (D) {
    case 64:
        return two ? launch_decode<T, FMT, 64, 2>(a, stream) : launch_decode<T, FMT, 64, 1>(a, stream);
    case 128:
        return two ? launch_decode<T, FMT, 128, 2>(a, stream) : launch_decode<T, FMT, 128, 1>(a, stream);
    default:
        return two ? launch_decode<T, FMT, 256, 2>(a, stream) : launch_decode<T, FMT, 256, 1>(a, stream);
    }
}

bool format_ok(int format) { return format == KVC_INT8 || format == KVC_E4M3; }

template <typename T> kvc_status launch_append(const AppendArgs &a, int format, cudaStream_t stream)
{
    const int lpr = a.D <= 64 ? 8 : a.D <= 128 ? 16 : 32;
    // 12 blocks an SM over all slices, or a block for every row tile: 31 us for 100 MB with 8, 35 with 6
    const int slices = a.batch * a.kv_heads;
    const int64_t tiles = ((int64_t)a.S * lpr + kAppendThreads - 1) / kAppendThreads;
    const dim3 n((unsigned)std::min<int64_t>(tiles, (int64_t)kvc_host::sm_count() * 12 / slices + 1), slices);
    if (format == KVC_INT8) {
        if (lpr == 8)
            quant_append_kernel<T, KVC_INT8, 8><<<n, kAppendThreads, 0, stream>>>(a);
        else if (lpr == 16)
            quant_append_kernel<T, KVC_INT8, 16><<<n, kAppendThreads, 0, stream>>>(a);
        else
            quant_append_kernel<T, KVC_INT8, 32><<<n, kAppendThreads, 0, stream>>>(a);
    } else {
        if (lpr == 8)
            quant_append_kernel<T, KVC_E4M3, 8><<<n, kAppendThreads, 0, stream>>>(a);
        else if (lpr == 16)
            quant_append_kernel<T, KVC_E4M3, 16><<<n, kAppendThreads, 0, stream>>>(a);
        else
            quant_append_kernel<T, KVC_E4M3, 32><<<n, kAppendThreads, 0, stream>>>(a);
    }
    return kvc_host::launch_status();
}

template <typename T> kvc_status launch_dequant(const DequantArgs &a, int format, cudaStream_t stream)
{
    // a block for every kRowsAhead * rpb rows, or one wave of resident blocks over all slices of K and V
    const int slices = a.batch * a.kv_heads, rpb = 256 / (a.D / 8);
    int64_t nx = (std::min(a.C, a.R) + kRowsAhead * rpb - 1) / (kRowsAhead * rpb);
    nx = std::min<int64_t>(nx, (int64_t)kvc_host::sm_count() * kDequantCtas / (2 * slices) + 1);
    const dim3 grid((unsigned)nx, slices, 2);
    if (format == KVC_INT8)
        dequant_rows_kernel<T, KVC_INT8><<<grid, 256, 0, stream>>>(a);
    else
        dequant_rows_kernel<T, KVC_E4M3><<<grid, 256, 0, stream>>>(a);
    return kvc_host::launch_status();
}

// what the three calls ask of the quantised cache's buffers
kvc_status check_cache(const void *kq, const void *vq, const void *ks, const void *vs, int batch, int kv_heads,
                       int64_t C, int D)
{
    if (!kq || !vq || !ks || !vs)
        return KVC_ERR_NULL;
    for (const void *p : {kq, vq, ks, vs})
        if (!kvc_host::aligned16(p))
            return KVC_ERR_ALIGN;
    const size_t rows = (size_t)batch * kv_heads * C;
    const void *at[4] = {kq, vq, ks, vs};
    const size_t bytes[4] = {rows * D, rows * D, rows * 4, rows * 4};
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < i; ++j)
            if (kvc_host::overlaps(at[i], bytes[i], at[j], bytes[j]))
                return KVC_ERR_SHAPE;
    return KVC_OK;
}

} // namespace

KVC_API kvc_status kvc_quant_append(void *kq_cache, void *vq_cache, float *k_scale, float *v_scale,
                                    const void *new_k, const void *new_v, kvc_lengths len, int batch,
                                    int kv_heads, int new_tokens, int64_t capacity, int head_dim, int dtype,
                                    int format, int windowed, const float *rope_cos, const float *rope_sin,
                                    int64_t rope_max_pos, int32_t *dev_status, void *stream_)
{
    if (kvc_host::elem_bytes_of(dtype) == 0 || !format_ok(format))
        return KVC_ERR_DTYPE;
    if (batch < 0 || kv_heads < 1 || new_tokens < 1 || head_dim < 1 || (int64_t)batch * kv_heads > 65535)
        return KVC_ERR_SHAPE;
    if (windowed != KVC_CONTIGUOUS && windowed != KVC_RING)
        return KVC_ERR_UNSUPPORTED;
    if (head_dim > 256 || head_dim % 16 != 0)
        return KVC_ERR_UNSUPPORTED;
    if (capacity < 1 || capacity > (int64_t)INT32_MAX)
        return KVC_ERR_CAPACITY;
    if ((rope_cos == nullptr) != (rope_sin == nullptr))
        return KVC_ERR_NULL;
    if (rope_cos && rope_max_pos < 1)
        return KVC_ERR_SHAPE;
    if (batch == 0)
        return KVC_OK;
    if (!new_k || !new_v || !kvc_host::lengths_ok(len))
        return KVC_ERR_NULL;
    const kvc_status st = check_cache(kq_cache, vq_cache, k_scale, v_scale, batch, kv_heads, capacity, head_dim);
    if (st != KVC_OK)
        return st;
    for (const void *p : {new_k, new_v, (const void *)rope_cos, (const void *)rope_sin})
        if (p && !kvc_host::aligned16(p))
            return KVC_ERR_ALIGN;
    AppendArgs a{static_cast<uint8_t *>(kq_cache), static_cast<uint8_t *>(vq_cache), k_scale, v_scale, new_k, new_v,
                 len, batch, kv_heads, new_tokens, head_dim, capacity, windowed == KVC_RING, rope_cos, rope_sin,
                 rope_max_pos, dev_status};
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    switch (dtype) {
    case KVC_F32:
        return launch_append<float>(a, format, stream);
    case KVC_BF16:
        return launch_append<__nv_bfloat16>(a, format, stream);
    default:
        return launch_append<__half>(a, format, stream);
    }
}

KVC_API kvc_status kvc_dequant_rows(void *k_out, void *v_out, const void *kq_cache, const void *vq_cache,
                                    const float *k_scale, const float *v_scale, kvc_lengths len, int batch,
                                    int kv_heads, int64_t capacity, int64_t rows_out, int head_dim, int dtype,
                                    int format, int windowed, int32_t *dev_status, void *stream_)
{
    const int eb = kvc_host::elem_bytes_of(dtype);
    if (eb == 0 || !format_ok(format))
        return KVC_ERR_DTYPE;
    if (batch < 0 || kv_heads < 1 || head_dim < 1 || (int64_t)batch * kv_heads > 65535)
        return KVC_ERR_SHAPE;
    if (windowed != KVC_CONTIGUOUS && windowed != KVC_RING)
        return KVC_ERR_UNSUPPORTED;
    if (head_dim > 256 || head_dim % 16 != 0)
        return KVC_ERR_UNSUPPORTED;
    if (capacity < 1 || capacity > (int64_t)INT32_MAX || rows_out < 1 || rows_out > (int64_t)INT32_MAX)
        return KVC_ERR_CAPACITY;
    if (batch == 0)
        return KVC_OK;
    if (!k_out || !v_out || !kvc_host::lengths_ok(len))
        return KVC_ERR_NULL;
    const kvc_status st = check_cache(kq_cache, vq_cache, k_scale, v_scale, batch, kv_heads, capacity, head_dim);
    if (st != KVC_OK)
        return st;
    for (const void *p : {(const void *)k_out, (const void *)v_out})
        if (!kvc_host::aligned16(p))
            return KVC_ERR_ALIGN;
    const size_t in_rows = (size_t)batch * kv_heads * capacity;
    const size_t out_bytes = (size_t)batch * kv_heads * rows_out * head_dim * eb;
    if (kvc_host::overlaps(k_out, out_bytes, v_out, out_bytes))
        return KVC_ERR_SHAPE;
    for (const void *o : {(const void *)k_out, (const void *)v_out}) {
        for (const void *p : {kq_cache, vq_cache})
            if (kvc_host::overlaps(o, out_bytes, p, in_rows * head_dim))
                return KVC_ERR_SHAPE;
        for (const void *p : {(const void *)k_scale, (const void *)v_scale})
            if (kvc_host::overlaps(o, out_bytes, p, in_rows * 4))
                return KVC_ERR_SHAPE;
    }
    DequantArgs a{k_out, v_out, static_cast<const uint8_t *>(kq_cache), static_cast<const uint8_t *>(vq_cache),
                  k_scale, v_scale, len, batch, kv_heads, head_dim, capacity, rows_out, windowed == KVC_RING,
                  dev_status};
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    switch (dtype) {
    case KVC_F32:
        return launch_dequant<float>(a, format, stream);
    case KVC_BF16:
        return launch_dequant<__nv_bfloat16>(a, format, stream);
    default:
        return launch_dequant<__half>(a, format, stream);
    }
}

KVC_API size_t kvc_gqa_decode_quant_workspace_size(int batch, int q_heads, int kv_heads, int64_t capacity,
                                                   int head_dim)
{
    if (batch < 1 || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads != 0 || capacity < 1 || head_dim < 1)
        return 0;
    if (capacity <= unit_of(head_dim, q_heads / kv_heads > 8 ? 2 : 1))
        return 0;
    const size_t parts = 2 * (size_t)decode_grid(batch, kv_heads, q_heads / kv_heads, capacity, head_dim).ctas *
                         (q_heads / kv_heads);
    return parts * (head_dim + 2) * sizeof(float);
}

KVC_API kvc_status kvc_gqa_decode_quant(void *out, const void *q, const void *kq_cache, const void *vq_cache,
                                        const float *k_scale, const float *v_scale, kvc_lengths len, int batch,
                                        int q_heads, int kv_heads, int64_t capacity, int head_dim, int dtype,
                                        int format, int windowed, int local_window_size, float scale,
                                        const float *rope_cos, const float *rope_sin, int64_t rope_max_pos,
                                        void *workspace, size_t workspace_bytes, int32_t *dev_status, void *stream_)
{
    if (kvc_host::elem_bytes_of(dtype) == 0 || !format_ok(format))
        return KVC_ERR_DTYPE;
    if (dtype == KVC_F32)
        return KVC_ERR_UNSUPPORTED;
    if (batch < 0 || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads != 0)
        return KVC_ERR_SHAPE;
    if (windowed != KVC_CONTIGUOUS && windowed != KVC_RING)
        return KVC_ERR_UNSUPPORTED;
    if ((head_dim != 64 && head_dim != 128 && head_dim != 256) || q_heads / kv_heads > 16)
        return KVC_ERR_UNSUPPORTED;
    if (capacity < 1 || capacity > (int64_t)INT32_MAX)
        return KVC_ERR_CAPACITY;
    if ((int64_t)batch * kv_heads * ((capacity + 63) / 64 + kRowCost) > (int64_t)INT32_MAX)
        return KVC_ERR_SHAPE;
    if ((rope_cos == nullptr) != (rope_sin == nullptr))
        return KVC_ERR_NULL;
    if (rope_cos && rope_max_pos < 1)
        return KVC_ERR_SHAPE;
    if (batch == 0)
        return KVC_OK;
    if (!out || !q || !kvc_host::lengths_ok(len))
        return KVC_ERR_NULL;
    const kvc_status st = check_cache(kq_cache, vq_cache, k_scale, v_scale, batch, kv_heads, capacity, head_dim);
    if (st != KVC_OK)
        return st;
    for (const void *p : {(const void *)out, q})
        if (!kvc_host::aligned16(p))
            return KVC_ERR_ALIGN;
    const size_t need = kvc_gqa_decode_quant_workspace_size(batch, q_heads, kv_heads, capacity, head_dim);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return KVC_ERR_WORKSPACE;
    if (need > 0 && (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return KVC_ERR_ALIGN;
    QuantDecodeArgs a{};
    a.out = out;
    a.q = q;
    a.kq = static_cast<const uint8_t *>(kq_cache);
    a.vq = static_cast<const uint8_t *>(vq_cache);
    a.ks = k_scale;
    a.vs = v_scale;
    a.len = len;
    a.batch = batch;
    a.q_heads = q_heads;
    a.kv_heads = kv_heads;
    a.group = q_heads / kv_heads;
    a.C = capacity;
    a.ring = windowed == KVC_RING;
    a.window = local_window_size;
    a.scale_log2 = (scale == 0.f ? 1.0f / sqrtf((float)head_dim) : scale) * kLog2e;
    a.cos_t = rope_cos;
    a.sin_t = rope_sin;
    a.rope_max_pos = rope_max_pos;
    a.unit = unit_of(head_dim, a.group > 8 ? 2 : 1);
    const Grid grid = decode_grid(batch, kv_heads, a.group, capacity, head_dim);
    a.grid = grid.ctas;
    a.row_cost = grid.row_cost;
    const int64_t parts = 2 * (int64_t)a.grid * a.group;
    a.ws_o = static_cast<float *>(workspace);
    a.ws_m = a.ws_o ? a.ws_o + parts * head_dim : nullptr;
    a.ws_l = a.ws_m ? a.ws_m + parts : nullptr;
    a.status = dev_status;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    if (dtype == KVC_BF16)
        return format == KVC_INT8 ? launch_decode_dim<__nv_bfloat16, KVC_INT8>(a, head_dim, stream)
                                  : launch_decode_dim<__nv_bfloat16, KVC_E4M3>(a, head_dim, stream);
    return format == KVC_INT8 ? launch_decode_dim<__half, KVC_INT8>(a, head_dim, stream)
                              : launch_decode_dim<__half, KVC_E4M3>(a, head_dim, stream);
}
