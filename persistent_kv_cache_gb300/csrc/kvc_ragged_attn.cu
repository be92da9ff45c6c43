// kvc_ragged_attn.cu -- attention of a packed batch's new tokens over a paged
// cache ("Persistent KV Cache and Decode Performance Roadmap", "Phase 1" and
// "Phase 2": streaming online softmax, a KV block read once per query-head
// group, pages read through a page table).
//
// The queries of one kv head's G heads at `toks` = 128 / G consecutive tokens
// are the 128 rows of a query tile (row m: token m / G, head m % G, as they lie in
// memory).  An item is one or, with head_dim <= 128, two such tiles of one
// (request, kv head), and streams the keys that its last token sees past the
// tensor cores in tiles of 128.
//
//   ragged_attn_kernel   the attention; every CTA (one an SM) takes the same share
//                        of the keys of all items, in segments of one item each
//   ragged_merge_kernel  joins the items that several CTAs worked on
#include <algorithm>
#include <climits>
#include <cmath>
#include <type_traits>

#include "kvc_common.cuh"
#include "kvc_tc.cuh"

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kBM = 128, kBN = 128;
constexpr float kRescale = 8.f;  // log2 units by which a score may exceed the reference maximum
// Keys that stand for what an item costs beside its keys (256, 512, 768, 1024, 1536: chunks of 8 prompts 718, 673, 656,
// 659, 676 us, windowed 614, 602, 601, 601, 609, decoding and prompts 111, 105, 105, 106, 106).
constexpr int kItemCost = 768;
constexpr int kMaxRequests = 65535;
constexpr int kMaxKeys = INT_MAX - 511;  // of a request: rows are rounded up to tiles and items in 32 bits

struct RaggedArgs {
    void *out;
    const int32_t *offsets, *table;
    int max_pages, page_size;
    int64_t n_pool;
    kvc_lengths len;
    int batch, tokens, q_heads, kv_heads, group;
    int toks, item;  // tokens of a query tile, of an item
    int one, two;    // what a key of an item of one, of two query tiles counts
    int rounds;      // at most so many
    int key_bytes;   // of a key and its value, all kv heads
    int streams;     // of softmax and products in a CTA
    int box_rows;    // rows of a TMA box of K (of V: up to a slab's)
    int window;
    float scale_log2;
    float *ws_o, *ws_m, *ws_l;  // partial results: [2 * pieces * tiles][D / 4][128][4], [..][128]
    int4 *split;  // [pieces] the item of which a piece has the first keys but not the last: its first row, its tokens, kv
                  // head, 2 * parts + slot of its own part (parts 0: there is none)
    int32_t *status;
};

// --------------------------------------------------------------------------
// the items and their shares
// --------------------------------------------------------------------------

// The new tokens of request b.  n = 0 for a request that was rejected; one whose
// lengths and offsets do not go together is too.
struct Request {
    int row0, P, n, items;
};
__device__ __forceinline__ Request request(const RaggedArgs &a, int b, uint32_t &bad)
{
    const int o0 = a.offsets[b], o1 = a.offsets[b + 1], T = a.len.total_abs[b], L = a.len.cache_total[b];
    Request r;
    r.row0 = o0;
    r.P = a.len.past_abs[b];
    r.n = 0;
    bad = 0;
    if (L >= 0 && r.P >= 0) {
        if (T < r.P || o0 < 0 || o1 < o0 || o1 > a.tokens || T - r.P != o1 - o0)
            bad = KVC_DEV_SEQLEN_RANGE;
        else if (T > min((int64_t)a.max_pages * a.page_size, (int64_t)kMaxKeys))
            bad = KVC_DEV_CAPACITY;
        else
            r.n = o1 - o0;
    }
    r.items = (int)((uint32_t)(r.n + a.item - 1) / (uint32_t)a.item);
    return r;
}

// first key row that item i's tokens see, and one past the last
__device__ __forceinline__ void key_range(const RaggedArgs &a, const Request &r, int i, int &lo, int &hi)
{
    lo = a.window > 0 ? max(0, r.P + i * a.item - a.window + 1) : 0;
    hi = r.P + min(r.n, (i + 1) * a.item);
}

// keys of the items before j: the sum over i < j of hi - lo, in closed form
__device__ __forceinline__ int64_t keys_before(const RaggedArgs &a, const Request &r, int j)
{
    // items of item tokens among them (all but perhaps the last)
    const int K = a.item, full = j == r.items && j * K != r.n ? j - 1 : j;
    int64_t sum = (int64_t)j * r.P + (int64_t)K * ((int64_t)full * (full + 1) / 2) + (j > full ? r.n : 0);
    if (a.window > 0) {
        const int i0 = r.P >= a.window ? 0 : (int)(((uint32_t)(a.window - r.P) + (uint32_t)(K - 1)) / (uint32_t)K);  // first with lo > 0
        if (j > i0) {
            const int64_t count = j - i0;
            sum -= count * ((int64_t)r.P - a.window + 1) + K * ((i0 + (int64_t)j - 1) * count / 2);
        }
    }
    return sum;
}

// what a key of item i counts
__device__ __forceinline__ int weight_of(const RaggedArgs &a, const Request &r, int i)
{
    return r.n - i * a.item <= a.toks ? a.one : a.two;
}

// the same of the items before j, with what each key counts (all items but the last
// have two query tiles) and with every item's cost
__device__ __forceinline__ int64_t units_before(const RaggedArgs &a, const Request &r, int j, int cost)
{
    int64_t sum = keys_before(a, r, j) * a.two + (int64_t)j * cost;
    if (j > 0 && j == r.items) {
        int lo, hi;
        key_range(a, r, j - 1, lo, hi);
        sum -= (int64_t)(hi - lo) * (a.two - weight_of(a, r, j - 1));
    }
    return sum;
}

// x / y for x >= 0, y > 0 (in 32 bits where they fit: the other takes a thousand clocks of a CTA's start)
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t y)
{
    if (((x | y) >> 32) == 0)
        return (uint32_t)x / (uint32_t)y;
    return x / y;
}

// All items laid end to end (request, then kv head, then item; each as long as its
// keys count and `cost`) are one line, cut into equal shares: every CTA gets the
// same work whatever the lengths, and the split is the same on every run.
// A CTA's share is in one piece, or in up to `rounds` of them, a grid's pieces apart:
// then the CTAs are at work in a part of the line at a time, whose keys and values L2
// can hold.  (head_dim 256, where a key tile is read for 128 query rows only: windowed
// chunks of 8 prompts read each key from memory seven times.  A round costs each CTA two
// partial results, and its pieces are long enough for that to be little.)
constexpr int kRounds = 4;
constexpr int64_t kRoundBytes = 64 << 20, kRoundUnits = 64 * kBN;
struct Line {
    int grid, cost, rounds;  // grid: pieces of the line
    int64_t each, longer;  // shares [0, longer) are one longer than `each`
    __device__ __forceinline__ int64_t begin(int64_t c) const { return c * each + min(c, longer); }
    __device__ __forceinline__ int of(int64_t x) const
    {
        const int64_t head = longer * (each + 1);
        return (int)(x < head ? quotient(x, each + 1) : longer + quotient(x - head, each));
    }
};

// What `streams` key tiles of a row take a CTA, the join of two parts takes for each: a
// row of t such is done soonest by about sqrt(7 t) CTAs.  With so few rows that this
// leaves CTAs over, an item costs nothing beside its keys, and a row of a few tiles has its
// CTAs to itself.  Rows of less than a share's least (a tile's keys, two with two streams) then
// stand behind one another in a CTA, each with its start and end: 6 requests of 8 kv heads with
// 17 keys have 3 CTAs and take 75 us, where 7, whose items' cost counts, take 12.
__device__ __forceinline__ Line make_line(const RaggedArgs &a, int64_t units, int64_t rows, int64_t keys, int grid)
{
    Line l;
    l.rounds = 1;
    l.cost = kItemCost * a.one;
    const float t = fmaxf(1.f, (float)units / (128.f * a.one * a.streams * (float)max(rows, (int64_t)1)));
    const int64_t few = rows * (int64_t)ceilf(sqrtf(7.f * t));
    l.grid = grid;
    if (few <= grid) {
        l.grid = (int)max(few, (int64_t)1);
        l.cost = 0;
    }
    int64_t total = units + rows * l.cost;
    // no share shorter than a tile (no segment of a row between two others is empty), nor than one for each stream
    l.grid = (int)max((int64_t)1, min((int64_t)l.grid, quotient(total, kBN * max(a.two, a.streams * a.one))));
    if (a.rounds > 1 && l.grid == grid) {
        const int64_t fit = quotient(keys * a.key_bytes + kRoundBytes - 1, kRoundBytes), longest = quotient(total, grid * kRoundUnits);
        l.rounds = (int)max((int64_t)1, min((int64_t)a.rounds, min(fit, longest)));
        l.grid *= l.rounds;
    }
    l.each = quotient(total, l.grid);
    l.longer = total - l.each * l.grid;
    return l;
}

struct Segment {
    int b, h, i;
    int row0, P, n;    // of the request
    int lo, t0, t1, tiles;  // key tiles [t0, t1) of `tiles` from key row lo on
    int slot;               // of its partial result: two a piece of the line, the first for the piece's first segment
    int64_t end;            // of the item on the line
};

// x / weight, for the weights that there are: 1, 2, 3
__device__ __forceinline__ int over_weight(uint32_t x, int weight)
{
    return (int)(weight == 3 ? x / 3u : x >> (weight - 1));
}

// The segments of a CTA's share, one at a time.
struct Walk {
    int64_t x, x_end, base;  // base: of the item at (b, h, i)
    int b, h, i;
    int round, slot;         // which of the CTA's pieces; of the piece's next segment
    Request r;
    // `pieces`: the CTA's later ones, as they begin
    __device__ __forceinline__ bool next(const RaggedArgs &a, int cost, int rounds, const Walk *pieces, Segment &s)
    {
        for (;;) {
            if (x >= x_end) {
                if (round + 1 >= rounds)
                    return false;
                *this = pieces[round];
                continue;
            }
            while (i >= r.items) {
                i = 0;
                if (r.items == 0 || ++h == a.kv_heads) {
                    h = 0;
                    ++b;
                    uint32_t bad;
                    r = request(a, b, bad);
                }
            }
            int lo, hi;
            key_range(a, r, i, lo, hi);
            const int weight = weight_of(a, r, i);
            const int64_t end = base + (int64_t)(hi - lo) * weight + cost;
            s.b = b;
            s.h = h;
            s.i = i;
            s.row0 = r.row0;
            s.P = r.P;
            s.n = r.n;
            s.lo = lo & ~(a.box_rows - 1);
            s.tiles = (hi - s.lo + kBN - 1) / kBN;
            s.end = end;
            // (what stands for the item's cost comes first and holds no keys; positions over 128 fit 32 bits)
            const int64_t p0 = x - base - cost, p1 = x_end - base - cost;
            s.t0 = p0 <= 0 ? 0 : over_weight((uint32_t)(p0 / kBN), weight);
            s.t1 = x_end >= end ? s.tiles : p1 <= 0 ? 0 : over_weight((uint32_t)(p1 / kBN), weight);
            if (x_end >= end) {
                x = base = end;
                ++i;
            } else {
                x = x_end;
            }
            if (s.t1 > s.t0) {
                s.slot = 2 * (int)(blockIdx.x + round * gridDim.x) + slot;
                slot = 1;
                return true;
            }
        }
    }
};

// sum over a warp of x (0 <= x < 2^54, which no tokens and keys that fit a GPU's memory reach)
__device__ __forceinline__ int64_t warp_sum(int64_t x)
{
    const uint32_t low = __reduce_add_sync(0xffffffffu, (uint32_t)x & 0x7ffffffu);
    return (int64_t)low + ((int64_t)__reduce_add_sync(0xffffffffu, (uint32_t)(x >> 27)) << 27);
}

// inclusive prefix sum over a warp
template <typename U> __device__ __forceinline__ U warp_scan(U x)
{
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const U y = __shfl_up_sync(0xffffffffu, x, d);
        x += (int)(threadIdx.x & 31) >= d ? y : 0;
    }
    return x;
}

// Where unit x of the line is: the group of 32 requests (whose sums are in units and
// rows), the request, the kv head and the item.  `mine`: of a single group, this lane's
// request.
__device__ __forceinline__ void locate(const RaggedArgs &a, const int64_t *units, const int *rows, int groups, int cost,
                                       const Request &mine, Walk &w)
{
    const int lane = threadIdx.x & 31;
    int64_t before = 0;
    int at = 0;
    for (int g0 = 0; groups > 1 && g0 < groups; g0 += 32) {
        const int g = g0 + lane;
        const int64_t len = g < groups ? (units[g] + (int64_t)rows[g] * cost) * a.kv_heads : 0;
        const int64_t inc = warp_scan(len);
        const uint32_t past = __ballot_sync(0xffffffffu, before + inc > w.x);
        if (past) {
            const int first = __ffs(past) - 1;
            at = g0 + first;
            before += __shfl_sync(0xffffffffu, inc - len, first);
            break;
        }
        before += __shfl_sync(0xffffffffu, inc, 31);
    }
    {
        const int b = 32 * at + lane;
        uint32_t bad;
        Request r = mine;
        if (groups > 1 && b < a.batch)
            r = request(a, b, bad);
        const int64_t len = units_before(a, r, r.items, cost) * a.kv_heads;
        // (the group's units, in 32 bits where they fit)
        const int64_t group = warp_sum(len);
        const int64_t inc = group >> 31 ? warp_scan(len) : (int64_t)warp_scan((int)len);
        const int first = __ffs(__ballot_sync(0xffffffffu, before + inc > w.x)) - 1;
        w.b = 32 * at + first;
        before += __shfl_sync(0xffffffffu, inc - len, first);
        w.r.row0 = __shfl_sync(0xffffffffu, r.row0, first);
        w.r.P = __shfl_sync(0xffffffffu, r.P, first);
        w.r.n = __shfl_sync(0xffffffffu, r.n, first);
        w.r.items = __shfl_sync(0xffffffffu, r.items, first);
    }
    const int64_t head = units_before(a, w.r, w.r.items, cost);
    w.h = (int)quotient(w.x - before, head);
    before += w.h * head;
    int low = 0, count = w.r.items;  // the last item that begins at x or before it, among [low, low + count)
    while (count > 1) {
        const int step = (count + 31) / 32, j = low + lane * step;
        const bool begun = lane * step < count && before + units_before(a, w.r, j, cost) <= w.x;
        const int last = 31 - __clz(__ballot_sync(0xffffffffu, begun));
        low += last * step;
        count = min(step, count - last * step);
    }
    w.i = low;
    w.base = before + units_before(a, w.r, low, cost);
}

// The CTA's share: the requests' units, items and keys summed by groups of 32 (a warp a
// group), the sums in shared memory, and where the share's pieces begin.  `scratch` holds
// 20 bytes a group.
template <int THREADS>
__device__ __forceinline__ Line find_share(const RaggedArgs &a, uint8_t *scratch, Walk &w, Walk *pieces)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, groups = (a.batch + 31) / 32;
    int64_t *units = reinterpret_cast<int64_t *>(scratch), *seen = units + groups;
    int *rows = reinterpret_cast<int *>(seen + groups);
    // (a single group: every warp has it in registers)
    Request mine{0, 0, 0, 0};
    int64_t k = 0, n = 0, keys = 0;
    auto count = [&](int b, Request &r, int64_t &k, int64_t &keys) {
        uint32_t bad;
        r = request(a, b, bad);
        if (bad && blockIdx.x == 0)
            kvc::raise_status(a.status, bad);
        k = units_before(a, r, r.items, 0);
        keys = r.n == 0 ? 0 : a.window > 0 ? r.n + min(r.P, a.window - 1) : r.n + r.P;
    };
    if (groups == 1 && lane < a.batch) {
        count(lane, mine, k, keys);
        n = mine.items;
    }
    for (int g = groups == 1 ? groups : warp; g < groups; g += THREADS / 32) {
        const int b = 32 * g + lane;
        Request r{0, 0, 0, 0};
        int64_t mine_k = 0, mine_keys = 0;
        if (b < a.batch)
            count(b, r, mine_k, mine_keys);
        mine_k = warp_sum(mine_k);
        mine_keys = warp_sum(mine_keys);
        const int items = __reduce_add_sync(0xffffffffu, r.items);
        if (lane == 0) {
            units[g] = mine_k;
            seen[g] = mine_keys;
            rows[g] = items;
        }
    }
    if (groups > 1) {
        __syncthreads();
        for (int g = lane; g < groups; g += 32) {
            k += units[g];
            keys += seen[g];
            n += rows[g];
        }
    }
    k = warp_sum(k);
    n = warp_sum(n);
    if (a.rounds > 1)
        keys = warp_sum(keys);
    const Line line = make_line(a, k * a.kv_heads, n * a.kv_heads, keys, gridDim.x);
    w.x = w.x_end = 0;
    w.round = w.slot = 0;
    if (n > 0) {
#pragma unroll 1
        for (int round = line.rounds - 1; round >= 0; --round) {
            const int piece = blockIdx.x + round * gridDim.x;
            if (piece >= line.grid)
                break;
            w.round = round;
            w.x = line.begin(piece);
            w.x_end = line.begin(piece + 1);
            locate(a, units, rows, groups, line.cost, mine, w);
            if (round > 0 && threadIdx.x == 0)
                pieces[round - 1] = w;
        }
    }
    __syncthreads();
    return line;
}

// --------------------------------------------------------------------------
// the attention
// --------------------------------------------------------------------------
//
//   TMEM columns  an output O of D columns and a score buffer S of 128 for each of two
//                 streams, the weights over the scores (64: in 64 columns of their
//                 own; 256: one O, two buffers S)
//   shared        queries (two tiles; 256: one) | ring of slabs of K and V
//   warp 0        TMA of the queries, the score products
//   warps 1, 2    TMA of K and of V into one ring in the order of use
//   warp 3        the output products
//   other warps   softmax and output: eight a stream, two threads a row (= TMEM
//                 lane), each half of the columns
//
// head_dim <= 128: the warps 4-11 and 12-19 are two streams, each with a score buffer
// and an output of its own, so that one's softmax runs while the other's products
// do.  An item of two query tiles gives each stream one of them, over the same keys
// (read once for both); an item of one tile (a decoding request, the end of a prompt)
// gives each stream every second key tile, and the two results are joined
// from tensor memory at the end.
// head_dim 256: no room for two outputs; one stream, the two score buffers in turn.
//
// What bounds it (one GB300, bf16; times of the whole call, with the join; means of 16
// drawn batches and the products of the pairs that are seen; times of steps, here and below,
// are of three such batches):
//   chunks of 8 prompts, head_dim 128, group 4, 737 GFLOP: 643 us, 60 % of the measured
//   bf16 peak (58 to 63).  A pair of tiles takes 3800 clocks where its products need 2048: a
//   stream's chain (scores 512, their maximum 370, weights 1150, output products 512, the
//   barriers between them) is longer than two streams hide.  Three streams, or scores a
//   tile ahead, want more than the 512 columns of tensor memory; the maximum and the weights
//   each read the scores, of which a thread's 64 do not fit the 96 registers that all
//   threads are compiled for (another split of the registers between the warps has not been
//   tried in this form).  Steps on the way: one
//   thread a row, unrolled, with its scores in registers 869 us (the code missed the
//   instruction cache; a spilled register in the loop costs the release of every
//   arrival behind it hundreds of clocks); two threads a row and rolled loops 650.
//   windowed chunks, head_dim 256, 718 GFLOP: 597 us, 63 %.  128 KB of K and V a tile for
//   16.8 MFLOP: L2 delivers about 11 TB/s.
//   decoding batch, 544 MB: 97 us, 83 % of the measured copy rate.
//   decoding and prompts, head_dim 64, window 1000, pages of 16 (116 MB): 102 us; nine
//   tiles an item, three of them cut, and the exponentials of 128 rows for a decoding
//   request's eight.
//   17 tokens of one user over 700: 18.4 us (20 with a cold L2), a chain of loads (lengths, table, rows, join).
//
// Only key tiles that hold the last tokens' own rows, or that a window's edge cuts,
// are masked ("cut" tiles).  A NaN or an infinity in a column of V makes that column of
// the output NaN for the rows that see it, and for no other.  In whole tiles the
// products do that by themselves.  In cut tiles 0 x NaN would reach the rows that
// do not see it, and rows that no token of the item sees (behind the last one, before a
// window) may hold anything: there the softmax warps look through V in shared memory,
// write down for each row the columns of such values that it sees, and put zeros in
// their place.  (Zeros for the rows that none sees, without looking, took longer: by the
// warp of the output products, or by the stream's warps before they give the weights,
// 672 and 665 us for 645 in chunks of 8 prompts.)

// The segments of a stream's softmax warps: one warp looks one ahead for all.
struct Kept {
    Walk walk;
    Segment seg[2];
    int more[2];
};

template <int D> struct Smem {
    static constexpr int TILES = D <= 128 ? 2 : 1;  // query tiles, streams
    static constexpr int SOFTMAX = TILES * 256;     // threads of the softmax warps: two a row
    static constexpr int THREADS = 128 + SOFTMAX;
    static constexpr int KR = D <= 128 ? 128 : 64;  // rows of a slab of V
    static constexpr int SPT = kBN / KR;            // slabs of a tile of K (or V)
    static constexpr int Q_TILE = kBM * D * 2, Q_BYTES = TILES * Q_TILE;
    static constexpr int SLAB = KR * D * 2;
    static constexpr int BUDGET = 227 * 1024;
    static constexpr int NBAR = 12;  // beside the ring's
    // beside the queries and n slabs: barriers, tensor memory's address and a flag, maxima and sums, rows, `Kept`, pieces
    static constexpr int misc(int n)
    {
        return (2 * n + NBAR) * 8 + 16 + 4 * kBM * 4 + 16 + 2 * (int)sizeof(Kept) + (kRounds - 1) * (int)sizeof(Walk);
    }
    static constexpr int fit()
    {
        int n = 12;
        while (Q_BYTES + n * SLAB + misc(n) > BUDGET)
            --n;
        return n;
    }
    static constexpr int NSLAB = fit();
    static constexpr int RING_OFF = Q_BYTES;
    static constexpr int BAR_OFF = RING_OFF + NSLAB * SLAB;
    // full[NSLAB], empty[NSLAB], s_full[2], p_full[2], o_done[2], q_full, q_empty, drain[2], h_full[2]
    static constexpr int HALF_OFF = BAR_OFF + (2 * NSLAB + 10) * 8;  // h_full
    static constexpr int MISC_OFF = BAR_OFF + (2 * NSLAB + NBAR) * 8;
    static constexpr int RED_OFF = (MISC_OFF + 8 + 15) / 16 * 16;  // 4 x 128 floats: maxima and sums that change hands
    static constexpr int BAD_OFF = RED_OFF + 4 * kBM * 4;
    static constexpr int WALK_OFF = BAD_OFF + 16;  // of each stream
    static constexpr int PIECES_OFF = WALK_OFF + 2 * (int)sizeof(Kept);
    static constexpr int TOTAL = PIECES_OFF + (kRounds - 1) * (int)sizeof(Walk);
    static_assert(TOTAL <= BUDGET && NSLAB >= 2 * SPT + 1, "a tile of K, one of V and the next slab must fit");
    static_assert(NSLAB * SLAB >= 20 * ((kMaxRequests + 31) / 32), "the groups' sums lie where the ring will");
    // the weights have columns of their own where there are some left: the next scores need not wait for them to be read
    static constexpr bool OWN_P = D == 64;
    // head_dim 128: the output products of half of a tile's keys start while the other half's weights are made (632 ->
    // 614 us, chunks of 8 prompts; at 64, whose products are short, 106 -> 113, decoding and prompts in one call)
    static constexpr bool EARLY = D == 128;
    static constexpr uint32_t COL_S = TILES * D, COL_P = OWN_P ? COL_S + 2 * kBN : COL_S, TMEM_COLS = 512;
    static_assert(COL_S + 2 * kBN + (OWN_P ? 2 * 64 : 0) <= TMEM_COLS, "tensor memory");
};

// The ring holds, for a segment of n tiles, K_0, K_1, then V_j and K_{j+2} while
// there is one, then the last V's: the places of K_j and of V_j in that order.
__device__ __forceinline__ int k_group(int j) { return j < 2 ? j : 2 * j - 1; }
__device__ __forceinline__ int v_group(int j, int n)
{
    const int lead = n < 2 ? n : 2, paired = n - lead;
    return j < paired ? lead + 2 * j : lead + paired + j;
}

// The 16-bit halves of w that are NaN or infinite: bit 15 of each (the other bits are
// anything), which an exponent of ones carries into; then 0xffff for each.  (Comparing
// halves took several instructions more a word: chunks 617 -> 608, windowed 620 -> 604 us.)
template <typename T> __device__ __forceinline__ uint32_t odd_bits(uint32_t w)
{
    constexpr bool H = std::is_same<T, __half>::value;
    return (w & (H ? 0x7c007c00u : 0x7f807f80u)) + (H ? 0x04000400u : 0x00800080u);
}
template <typename T> __device__ __forceinline__ uint32_t not_finite(uint32_t w)
{
    return (odd_bits<T>(w) >> 15 & 0x10001u) * 0xffffu;
}

// Scores of up to 32 columns: those outside [lo, hi] become -infinity, and a negative
// scale turns the others' sign (the maximum is of scale * score / |scale|).
template <int N> __device__ __forceinline__ void seen_only(uint32_t (&x)[N], int lo, int hi, uint32_t flip)
{
    uint32_t bits = lo > 0 ? lo < 32 ? ~0u << lo : 0u : ~0u;
    bits &= hi < 0 ? 0u : hi < 31 ? (2u << hi) - 1u : ~0u;
#pragma unroll
    for (int c = 0; c < N; ++c)
        x[c] = bits >> c & 1u ? x[c] ^ flip : 0xff800000u;
}

template <int N> __device__ __forceinline__ float top_of(const uint32_t (&x)[N])
{
    float m[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        m[e] = fmaxf(__uint_as_float(x[e]), __uint_as_float(x[4 + e]));
#pragma unroll
    for (int c = 8; c < N; c += 8)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            m[e] = fmaxf(fmaxf(m[e], __uint_as_float(x[c + e])), __uint_as_float(x[c + 4 + e]));
    return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// scores -> weights 2^(x c - m), summed in float32 and packed to 16-bit pairs in the first half of x.
// (The output products take both operands in one 16-bit type, V's.  A weight is rounded once, by at most half a
// step of itself, which a result's own rounding exceeds a little: the relative error against 64 bits goes from 1.7e-3,
// a result that is only rounded, to 2.3e-3 with bf16, from 2.1e-4 to 2.9e-4 with fp16.  A second product with what
// the rounding left over would make the output products, half of all, twice as long.)
template <typename T, int N>
__device__ __forceinline__ void weights(uint32_t (&x)[N], float c_log2, float neg_m, float2 (&sum)[2])
{
    const float2 c2 = make_float2(c_log2, c_log2), m2 = make_float2(neg_m, neg_m);
#pragma unroll
    for (int e = 0; e < N; e += 2) {
        const float2 z = kvc_tc::fma2(make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), c2, m2);
        const float2 p = make_float2(kvc_tc::fast_exp2(z.x), kvc_tc::fast_exp2(z.y));
        sum[e / 2 % 2] = kvc_tc::add2(sum[e / 2 % 2], p);
        x[e / 2] = kvc_tc::pack2<T>(p.x, p.y);
    }
}

// The maximum of a row's CT scores in tensor memory, found as they are loaded; then of
// those of the columns [lo, hi].
template <int CT> __device__ __forceinline__ float row_top(uint32_t from)
{
    uint32_t x[32];
    float mx = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < CT; c += 32) {
        float top = kvc_tc::ld32_max(from + c, x);
        kvc_tc::wait_ld_max(top);
        mx = fmaxf(mx, top);
    }
    return mx;
}
template <int CT> __device__ __forceinline__ float row_top(uint32_t from, int lo, int hi, uint32_t flip)
{
    uint32_t x[32];
    float mx = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < CT; c += 32) {
        kvc_tc::ld32(from + c, x);
        kvc_tc::wait_ld32(x);
        seen_only(x, lo - c, hi - c, flip);
        mx = fmaxf(mx, top_of(x));
    }
    return mx;
}

// Scores -> weights in tensor memory, and their sum.  MASK: the scores of the columns
// [lo, hi] count.  Read 32 at a time in a rolled loop: with a row's scores in registers
// from the maximum to the exponential, and the code unrolled over them, a tile was
// longer than the instruction cache next to the tensor cores' issue loops.
template <typename T, int CT, bool MASK>
__device__ __forceinline__ float row_weights(uint32_t from, uint32_t to, int lo, int hi, uint32_t flip, float c_log2,
                                             float neg_m, uint32_t half_there)
{
    uint32_t x[32];
    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
    for (int c = 0; c < CT; c += 32) {
        kvc_tc::ld32(from + c, x);
        kvc_tc::wait_ld32(x);
        if (MASK)
            seen_only(x, lo - c, hi - c, flip);
        weights<T>(x, c_log2, neg_m, sum);
        kvc_tc::st16(to + c / 2, x);
        kvc_tc::wait_st();
        if (c == 0 && half_there) {
            kvc_tc::fence_before();
            __syncwarp();
            if ((threadIdx.x & 31) == 0)
                kvc_tc::arrive_at(half_there);
        }
    }
    return (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
}

// What the streams do in a segment: `two` query tiles over the same keys, the first
// of which needs the first n0 of the tiles only; or one, whose tiles alternate.
struct Streams {
    bool two;
    int n, n0;
    template <int TILES>
    static __device__ __forceinline__ Streams of(const RaggedArgs &a, const Segment &s)
    {
        Streams r;
        const int first = s.i * a.item;  // token
        r.n = s.t1 - s.t0;
        r.two = TILES == 2 && s.n - first > a.toks;
        // the last token of the first tile sees the rows up to its own
        r.n0 = r.two ? max(0, min(r.n, (s.P + first + a.toks - s.lo + kBN - 1) / kBN - s.t0)) : r.n;
        return r;
    }
    // does stream k work on tile j, and is it the tile's last one
    __device__ __forceinline__ bool has(int k, int j) const { return two ? k == 1 || j < n0 : (j & 1) == k; }
    __device__ __forceinline__ int tiles(int k) const { return two ? (k ? n : n0) : (n + 1 - k) >> 1; }
};

template <typename T, int D>
__global__ void __launch_bounds__(Smem<D>::THREADS, 1)
ragged_attn_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                   const __grid_constant__ CUtensorMap tmap_v, const RaggedArgs a)
{
    using SM = Smem<D>;
    using kvc_tc::wait_or_abort;
    using kvc_tc::warp_wait_or_abort;
    constexpr int NSLAB = SM::NSLAB, SPT = SM::SPT, KR = SM::KR, TILES = SM::TILES, kSoftmax = SM::SOFTMAX, THREADS = SM::THREADS;
    constexpr uint32_t AB = std::is_same<T, __half>::value ? 0u : 1u;
    constexpr uint32_t IDESC_S = kvc_tc::f16_idesc(AB, 0, kBM, kBN);
    constexpr uint32_t IDESC_O = kvc_tc::f16_idesc(AB, 1, kBM, D);

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    {
        // the swizzled tiles need a 1024-byte aligned base
        uint32_t dyn;
        asm("mov.u32 %0, %%dynamic_smem_size;" : "=r"(dyn));
        if ((uint32_t)(smem - smem_raw) + SM::TOTAL > dyn) {
            // (the call before may still join by what is written here, and what comes after counts on its end)
            kvc::grid_dep_wait();
            if (threadIdx.x == 0) {
                kvc::raise_status(a.status, KVC_DEV_CAPACITY);
                for (int p = 0; p < a.rounds; ++p)
                    a.split[blockIdx.x + p * gridDim.x] = make_int4(0, 0, 0, 0);
            }
            return;
        }
    }
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + SM::BAR_OFF), *empty = full + NSLAB,
             *s_full = full + 2 * NSLAB, *p_full = s_full + 2, *o_done = s_full + 4, *q_full = s_full + 6,
             *q_empty = s_full + 7, *drain = s_full + 8, *h_full = s_full + 10;
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
            kvc::mbar_init(&p_full[i], 8);
            kvc::mbar_init(&o_done[i], 1);
            kvc::mbar_init(&h_full[i], 8);
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
    kvc::grid_dep_wait();  // the kernels before: lengths, queries, cache, this workspace's last use
    Walk walk;
    Walk *later = reinterpret_cast<Walk *>(smem + SM::PIECES_OFF);
    const Line line = find_share<THREADS>(a, smem + SM::RING_OFF, walk, later);
    const int rounds = TILES == 1 ? line.rounds : 1;
    if (TILES == 2)
        walk.round = 0;  // (known to the compiler)
    // (the sums were read from where the ring's first slabs will be written)
    kvc::fence_proxy_async_smem();
    __syncthreads();
    kvc_tc::fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t smem_base = kvc::smem_u32(smem);
    // (products and softmax look one segment ahead, so that the lengths are there when they get to it)
    Segment cur, nxt;
    bool more = walk.next(a, line.cost, rounds, later, cur);

    if (warp < 4) {
        if (warp == 1 || warp == 2) {
            // ======================= TMA producers of K and of V =======================
            // A slab of K is all 128 rows and D / SPT columns of a tile, one of V KR rows and all columns (so that every
            // product has 128 keys or D columns to its name).  Each lane finds the place of one of the next 32
            // boxes' rows, and issues one of a slab's boxes.
            const bool mine_v = warp == 2;
            const CUtensorMap *tmap = mine_v ? &tmap_v : &tmap_k;
            if (lane == 0)
                kvc::tma_prefetch_desc(tmap);
            if (!mine_v && lane == 0)
                for (int p = 0; p < a.rounds; ++p)
                    a.split[blockIdx.x + p * gridDim.x] = make_int4(0, 0, 0, 0);
            int q0 = 0;  // slabs of the segments before
            bool ok = true;
            const int box = mine_v ? min(a.box_rows, KR) : a.box_rows, slab_rows = mine_v ? KR : kBN;
            const int per_tile = kBN / box, pieces = slab_rows / box;  // boxes of a tile's, of a slab's rows: powers of two up to 8
            const int blocks = mine_v ? D / 64 : D / 64 / SPT;         // column blocks of a slab
            const int piece = lane / blocks, block = lane % blocks;
            uint32_t filled = 0, phase = 0;  // slots that this warp has filled, with the parity of the last time
            while (ok && more) {
                const int nt = cur.t1 - cur.t0;
                const uint32_t end = (uint32_t)cur.P + min(cur.n, (cur.i + 1) * a.item), first = (uint32_t)cur.lo + cur.t0 * kBN;
                if (!mine_v && lane == 0 && cur.t0 == 0 && nt != cur.tiles)
                    a.split[cur.slot >> 1] = make_int4(cur.row0 + cur.i * a.item, min(cur.n - cur.i * a.item, a.item), cur.h,
                                                       2 * (line.of(cur.end - 1) - (cur.slot >> 1) + 1) + (cur.slot & 1));
                int32_t place = -1;
                for (int j = 0; ok && j < nt; ++j) {
                    if ((j * per_tile & 31) == 0) {
                        const int w = j * per_tile + lane;
                        const uint32_t r = first + (uint32_t)w * box;
                        place = -1;
                        if (w < nt * per_tile && r < end) {
                            const uint32_t page = r / (uint32_t)a.page_size;
                            // (an ordinary load: this kernel's life may begin while a plan still writes the table)
                            const int32_t id = a.table[(int64_t)cur.b * a.max_pages + page];
                            if (id >= 0 && id < a.n_pool)
                                place = (id * a.kv_heads + cur.h) * a.page_size + (int32_t)(r - page * a.page_size);
                            else
                                kvc::raise_status(a.status, KVC_DEV_INDEX_OOB);
                        }
                    }
                    for (int u = 0; u < SPT; ++u) {
                        const int q = q0 + SPT * (mine_v ? v_group(j, nt) : k_group(j)) + u, slot = q % NSLAB;
                        if (q >= NSLAB)
                            ok = warp_wait_or_abort(&empty[slot], ((q / NSLAB) - 1) & 1, abort_flag, a.status);
                        if (!ok)
                            break;
                        uint8_t *to = smem + SM::RING_OFF + slot * SM::SLAB;
                        const int at = j * per_tile + (mine_v ? u * pieces : 0), block0 = mine_v ? 0 : u * blocks;
                        const int32_t y = __shfl_sync(0xffffffffu, place, (at + (pieces == 1 ? 0 : piece)) & 31);
                        if (pieces == 1) {
                            if (lane == 0) {
                                if (y < 0) {
                                    // nothing to read: the slot keeps what it holds, and its columns are masked
                                    kvc::mbar_arrive(&full[slot]);
                                } else {
                                    kvc::mbar_arrive_expect_tx(&full[slot], SM::SLAB);
                                    kvc::tma_load_3d(to, tmap, 0, y, block0, &full[slot]);
                                }
                            }
                        } else {
                            // boxes of 64 columns, piece by piece
                            const bool load = piece < pieces && y >= 0;
                            const int n = __popc(__ballot_sync(0xffffffffu, load));
                            if (lane == 0) {
                                if (n == 0)
                                    kvc::mbar_arrive(&full[slot]);
                                else
                                    kvc::mbar_arrive_expect_tx(&full[slot], n * box * 128);
                            }
                            __syncwarp();
                            if (load)
                                kvc::tma_load_3d(to + block * (slab_rows * 128) + piece * box * 128, tmap, 0, y,
                                                 block0 + block, &full[slot]);
                        }
                        __syncwarp();
                        filled |= 1u << slot;
                        phase = (phase & ~(1u << slot)) | ((uint32_t)((q / NSLAB) & 1) << slot);
                    }
                }
                q0 += 2 * SPT * nt;
                more = walk.next(a, line.cost, rounds, later, cur);
            }
            if (*abort_flag && lane == 0)
                // wind-down: let the loads in flight land before the CTA exits
                for (int i = 0; i < NSLAB; ++i)
                    if (filled >> i & 1)
                        kvc::mbar_wait(&full[i], phase >> i & 1);
        } else if (warp == 3) {
            // ======================= output products =======================
            if (lane == 0) {
                const uint64_t v_ring = kvc_tc::sw128_desc(smem_base + SM::RING_OFF, KR * 128);
                int q0 = 0;                 // slabs of the segments before
                uint32_t used[2] = {0, 0};  // tiles that went through each score buffer
                bool ok = true;
                while (ok && more) {
                    const Streams st = Streams::of<TILES>(a, cur);
                    more = walk.next(a, line.cost, rounds, later, nxt);
                    for (int j = 0; ok && j < st.n; ++j) {
#pragma unroll
                        for (int k = 0; k < TILES; ++k) {
                            if (TILES == 2 && !st.has(k, j))
                                continue;
                            const int s = TILES == 2 ? k : (int)(used[0] & 1);
                            uint32_t &u = used[TILES == 2 ? k : 0];
                            const uint32_t parity = TILES == 2 ? u & 1 : (u >> 1) & 1;
                            const bool fresh = TILES == 2 && !st.two ? j < 2 : j == 0;  // first of the stream
                            const bool last = TILES == 1 || !st.two || k == 1;          // of the tile
                            // (EARLY: the products with each thread's first 32 weights, then the others)
                            constexpr int PARTS = SM::EARLY ? 2 : 1;
#pragma unroll
                            for (int part = 0; ok && part < PARTS; ++part) {
                                if (!(ok = wait_or_abort(SM::EARLY && part == 0 ? &h_full[s] : &p_full[s], parity, abort_flag, a.status)))
                                    break;
                                kvc_tc::fence_after();
                                for (int hf = 0; hf < SPT; ++hf) {
                                    const int q = q0 + SPT * v_group(j, st.n) + hf, slot = q % NSLAB;
                                    if (part == 0 && !(ok = wait_or_abort(&full[slot], (q / NSLAB) & 1, abort_flag, a.status)))
                                        break;
                                    kvc_tc::fence_after();
                                    const uint64_t vd = v_ring + (uint64_t)(slot * (SM::SLAB / 16));
                                    // (the weights of 64 keys are 32 columns; over the scores, the next ones' begin 64 further on)
                                    const uint32_t pa = tmem + SM::COL_P + s * (SM::OWN_P ? 64 : kBN) + hf * 64;
#pragma unroll
                                    for (int k2 = 0; k2 < KR / 16; ++k2) {
                                        if (SM::EARLY && (k2 >> 1 & 1) != part)
                                            continue;
                                        kvc_tc::mma_ts(tmem + (TILES == 2 ? k * D : 0),
                                                       pa + k2 / 4 * (SM::OWN_P ? 32 : 64) + k2 % 4 * 8,
                                                       vd + (uint64_t)(k2 * (2048 / 16)), IDESC_O,
                                                       !fresh || hf > 0 || k2 > 0);
                                    }
                                    if (last && part == PARTS - 1)
                                        kvc_tc::commit(&empty[slot]);
                                }
                            }
                            if (!ok)
                                break;
                            kvc_tc::commit(&o_done[s]);
                            ++u;
                        }
                    }
                    q0 += 2 * SPT * st.n;
                    cur = nxt;
                }
                // everything issued above has completed once this arrives
                kvc_tc::commit(&drain[1]);
                kvc::mbar_wait(&drain[1], 0);
            }
        } else {
            // ======================= queries, score products =======================
            if (lane == 0) {
                kvc::tma_prefetch_desc(&tmap_q);
                int q0 = 0;
                uint32_t used[2] = {0, 0};
                bool ok = true;
                const uint64_t q_desc = kvc_tc::sw128_desc(smem_base, 16);
                const uint64_t k_ring = kvc_tc::sw128_desc(smem_base + SM::RING_OFF, 16);
                const uint32_t q_box = (uint32_t)a.toks * a.group * 128;
                for (int s_no = 0; ok && more; ++s_no) {
                    // the last segment's scores are done: the queries' place is free
                    if (s_no > 0 && !wait_or_abort(q_empty, (s_no - 1) & 1, abort_flag, a.status))
                        break;
                    const Streams st = Streams::of<TILES>(a, cur);
                    const int tiles = st.two ? 2 : 1;
                    kvc::mbar_arrive_expect_tx(q_full, tiles * (D / 64) * q_box);
                    for (int k = 0; k < tiles; ++k)
                        for (int c = 0; c < D / 64; ++c)
                            kvc::tma_load_4d(smem + k * SM::Q_TILE + c * (kBM * 128), &tmap_q, 0, cur.h * a.group,
                                             cur.row0 + cur.i * a.item + k * a.toks, c, q_full);
                    more = walk.next(a, line.cost, rounds, later, nxt);
                    if (!(ok = wait_or_abort(q_full, s_no & 1, abort_flag, a.status))) {
                        kvc::mbar_wait(q_full, s_no & 1);  // (let the loads land before the CTA exits)
                        break;
                    }
                    kvc_tc::fence_after();
                    for (int j = 0; ok && j < st.n; ++j) {
#pragma unroll
                        for (int k = 0; k < TILES; ++k) {
                            if (TILES == 2 && !st.has(k, j))
                                continue;
                            const int s = TILES == 2 ? k : (int)(used[0] & 1);
                            uint32_t &u = used[TILES == 2 ? k : 0];
                            // Scores are written where the output products of the tile before (256: before last) read
                            // their weights.  Products of another accumulator or shape are not ordered by their
                            // issue: the wait for those is what keeps the weights.  (Weights in columns of their own:
                            // where the softmax warps read the scores before, until they gave the weights.)
                            const uint32_t before = TILES == 2 ? u : u >> 1;
                            if (before > 0 && !(ok = wait_or_abort(SM::OWN_P ? &p_full[s] : &o_done[s], (before - 1) & 1,
                                                                   abort_flag, a.status)))
                                break;
                            kvc_tc::fence_after();
                            const bool last = TILES == 1 || !st.two || k == 1;
                            for (int hf = 0; hf < SPT; ++hf) {
                                const int q = q0 + SPT * k_group(j) + hf, slot = q % NSLAB;
                                if (!(ok = wait_or_abort(&full[slot], (q / NSLAB) & 1, abort_flag, a.status)))
                                    break;
                                kvc_tc::fence_after();
                                const uint64_t qd = q_desc + (uint64_t)(((st.two ? k : 0) * SM::Q_TILE + hf * (D / 64 / SPT) * (kBM * 128)) / 16);
                                const uint64_t kd = k_ring + (uint64_t)(slot * (SM::SLAB / 16));
                                const uint32_t d_s = tmem + SM::COL_S + s * kBN;
#pragma unroll
                                for (int ks = 0; ks < D / 16 / SPT; ++ks)
                                    kvc_tc::mma_ss(d_s, qd + (uint64_t)(((ks >> 2) * (kBM * 128) + (ks & 3) * 32) / 16),
                                                   kd + (uint64_t)(((ks >> 2) * (kBN * 128) + (ks & 3) * 32) / 16), IDESC_S,
                                                   hf > 0 || ks > 0);
                                if (last)
                                    kvc_tc::commit(&empty[slot]);
                            }
                            if (!ok)
                                break;
                            kvc_tc::commit(&s_full[s]);
                            ++u;
                        }
                        if (ok && j == st.n - 1)
                            kvc_tc::commit(q_empty);
                    }
                    q0 += 2 * SPT * st.n;
                    cur = nxt;
                }
                // everything issued above has completed once this arrives
                kvc_tc::commit(&drain[0]);
                kvc::mbar_wait(&drain[0], 0);
            }
        }
        __syncwarp();
    } else {
        // ======================= softmax =======================
        // A wait that gives up has set the flag that ends all others, and the warps go on through the
        // tiles, whatever they find there, up to the stores, which ask for the flag: lanes give up one
        // by one, and the barriers below, which have no limit, want every warp and tensor memory whole
        // ones, so that nothing on the way may hang on a wait's answer.  (With a vote a tile, or each
        // lane's answer carried along, calls took 1 to 3 % longer.)
        constexpr int CT = kBN / 2, OT = D / 2;  // columns of S and of O of a thread
        const int tid = threadIdx.x - 128, quad = warp & 3, half = ((warp - 4) >> 2) & 1, stream = (warp - 4) >> 3;
        const int m = quad * 32 + lane;  // row of the tile
        const uint32_t lane_addr = tmem + ((uint32_t)(quad * 32) << 16);
        float *red = reinterpret_cast<float *>(smem + SM::RED_OFF);
        uint32_t *bad_sh = reinterpret_cast<uint32_t *>(smem + SM::BAD_OFF);
        constexpr uint32_t all_bar = 1;
        const uint32_t pair_bar = 2 + 4 * stream + quad;  // of a row's two threads
        const float c_log2 = fabsf(a.scale_log2);
        const uint32_t flip = a.scale_log2 < 0.f ? 0x80000000u : 0u;
        const uint32_t stream_bar = 10 + stream;
        // what a tile does not need, kept apart from the registers that its scores take
        Kept *kept = reinterpret_cast<Kept *>(smem + SM::WALK_OFF) + stream;
        // of a stream's warps, the one that looks ahead: one that a decoding request's few rows leave idle
        const bool scout = quad == 3 && half == 1;
        if (scout && lane == 0) {
            kept->walk = walk;
            kept->seg[0] = cur;
            kept->more[0] = more;
        }
        kvc_tc::named_bar_sync(stream_bar, 256);
        int q0 = 0;         // slabs before the segment
        uint32_t used = 0;  // tiles that this stream has had
        for (int s_no = 0; *(volatile int *)&kept->more[s_no & 1]; ++s_no) {
            Streams st;
            bool active;           // the warp has rows at all
            int head_cut, tail_cut;  // tiles [0, head_cut) and from tail_cut on are cut
            {
                const Segment seg = kept->seg[s_no & 1];
                st = Streams::of<TILES>(a, seg);
                active = seg.i * a.item + (st.two ? stream * a.toks : 0) + quad * 32 / a.group < seg.n;
                // what every row of the item sees: up to its first token, from the last one's window on
                const int lo0 = seg.lo + seg.t0 * kBN, hi = seg.P + seg.i * a.item;
                const int lo = a.window > 0 ? seg.P + min(seg.n, (seg.i + 1) * a.item) - a.window : 0;
                head_cut = lo > lo0 ? (lo - lo0 + kBN - 1) / kBN : 0;
                tail_cut = hi + 1 > lo0 ? (hi + 1 - lo0) / kBN : 0;
            }
            // This row sees the key rows [r_lo, r_hi], counted from tile j's first one; a row without a query
            // nothing in particular.  (Made again for each cut tile: kept, they cost registers in all others.)
            auto rows_seen = [&](int j, int &r_lo, int &r_hi) {
                const Segment &seg = kept->seg[s_no & 1];
                const int tok = m / a.group, i = seg.i * a.item + (st.two ? stream * a.toks : 0) + tok;
                const int pos = seg.P + i - (seg.lo + (seg.t0 + j) * kBN);
                const bool there = tok < a.toks && i < seg.n;
                r_hi = there ? pos : INT_MAX / 2;
                r_lo = there && a.window > 0 ? pos - a.window + 1 : INT_MIN / 2;
            };
            if (scout && lane == 0) {
                Walk next = kept->walk;
                kept->more[(s_no + 1) & 1] = next.next(a, line.cost, rounds, later, kept->seg[(s_no + 1) & 1]);
                kept->walk = next;
            }
            __syncwarp();
            // output columns in which the row has seen a NaN or an infinity, in cut tiles (written once there is one)
            volatile uint32_t nan_cols[OT / 32];
            bool nans = false;
            float m_run = -INFINITY, l_run = 0.f;
            for (int j = 0; j < st.n; ++j) {
                const bool cut = j < head_cut || j >= tail_cut;
                // Before the scores are waited for with two streams, so that both come to it at once and before the
                // first output products of EARLY; with one stream after the weights, by when V is there (608 -> 604 us).
                auto scan = [&]() {
                    // V rows with a NaN or an infinity in them, a bit each in bad_sh (zero before).
                    // Rows that all of the item's tokens see need none of that: looked at are groups of kRows rows with
                    // another among them (604 -> 589 us, windowed chunks at 256; at 64, whose groups are one load of a
                    // thread, finding out took longer: 107.7 -> 109.2, decoding and prompts).
                    constexpr int kRows = kSoftmax / 8, kGroups = KR / kRows;
                    int all_lo = 0, all_hi = -1;
                    if (D > 64) {
                        const Segment &seg = kept->seg[s_no & 1];
                        const int base = seg.lo + (seg.t0 + j) * kBN;
                        all_hi = seg.P + seg.i * a.item - base;
                        all_lo = a.window > 0 ? seg.P + min(seg.n, (seg.i + 1) * a.item) - a.window - base : INT_MIN / 2;
                    }
                    auto looked_at = [&](int row) { return row < all_lo || row + kRows - 1 > all_hi; };
                    bool found = false;
#pragma unroll
                    for (int hf = 0; hf < SPT; ++hf) {
                        const int qi = q0 + SPT * v_group(j, st.n) + hf;
                        wait_or_abort(&full[qi % NSLAB], (qi / NSLAB) & 1, abort_flag, a.status);
                        const uint4 *v = reinterpret_cast<const uint4 *>(smem + SM::RING_OFF + (qi % NSLAB) * SM::SLAB);
#pragma unroll
                        for (int g = 0; g < kGroups; ++g) {
                            if (!looked_at(hf * KR + g * kRows))
                                continue;
                            uint32_t odd = 0;
#pragma unroll
                            for (int c = 0; c < D / 64; ++c) {
                                const uint4 x = v[tid + kSoftmax * (g + c * kGroups)];
                                odd |= odd_bits<T>(x.x) | odd_bits<T>(x.y) | odd_bits<T>(x.z) | odd_bits<T>(x.w);
                            }
                            if (odd & 0x80008000u) {
                                const int vr = hf * KR + g * kRows + (tid >> 3);
                                atomicOr(&bad_sh[vr >> 5], 1u << (vr & 31));
                                found = true;
                            }
                        }
                    }
                    if (kvc_tc::named_bar_any(all_bar, kSoftmax, found)) {
                        // what this row sees of them is written down by column, then they are zeros for all
                        int r_lo, r_hi;
                        rows_seen(j, r_lo, r_hi);
#pragma unroll 1
                        for (int e = 0; e < 4; ++e) {
                            uint32_t left = r_hi < INT_MAX / 2 ? bad_sh[e] : 0u;
                            while (left) {
                                const int vr = 32 * e + __ffs(left) - 1, in = vr & (KR - 1);
                                left &= left - 1;
                                if (vr < r_lo || vr > r_hi)
                                    continue;
                                if (!nans)
                                    for (int w = 0; w < OT / 32; ++w)
                                        nan_cols[w] = 0;
                                nans = true;
                                const uint8_t *slab =
                                    smem + SM::RING_OFF + (q0 + SPT * v_group(j, st.n) + vr / KR) % NSLAB * SM::SLAB;
#pragma unroll 1
                                for (int w = 0; w < OT / 32; ++w) {
                                    uint32_t cols = 0;
#pragma unroll 1
                                    for (int c = 0; c < 4; ++c) {
                                        const int ch = half * (OT / 8) + 4 * w + c;  // 16 bytes of the row
                                        const uint4 x = *reinterpret_cast<const uint4 *>(
                                            slab + (ch >> 3) * (KR * 128) + in * 128 + ((ch & 7) ^ (in & 7)) * 16);
                                        const uint32_t nf[4] = {not_finite<T>(x.x), not_finite<T>(x.y), not_finite<T>(x.z),
                                                                not_finite<T>(x.w)};
#pragma unroll
                                        for (int i = 0; i < 4; ++i)
                                            cols |= ((nf[i] & 1u) | (nf[i] >> 30 & 2u)) << (8 * c + 2 * i);
                                    }
                                    nan_cols[w] = nan_cols[w] | cols;
                                }
                            }
                        }
                        kvc_tc::named_bar_sync(all_bar, kSoftmax);
                        if (tid < 4)
                            bad_sh[tid] = 0;
#pragma unroll 1
                        for (int hf = 0; hf < SPT; ++hf) {
                            uint4 *v = reinterpret_cast<uint4 *>(
                                smem + SM::RING_OFF + (q0 + SPT * v_group(j, st.n) + hf) % NSLAB * SM::SLAB);
#pragma unroll 1
                            for (int e = 0; e < SM::SLAB / 16 / kSoftmax; ++e) {
                                if (!looked_at(hf * KR + e % kGroups * kRows))
                                    continue;
                                const int at = tid + kSoftmax * e;
                                const uint4 x = v[at];
                                const uint4 nf = make_uint4(not_finite<T>(x.x), not_finite<T>(x.y), not_finite<T>(x.z),
                                                            not_finite<T>(x.w));
                                if (nf.x | nf.y | nf.z | nf.w)
                                    v[at] = make_uint4(x.x & ~nf.x, x.y & ~nf.y, x.z & ~nf.z, x.w & ~nf.w);
                            }
                        }
                        kvc::fence_proxy_async_smem();
                        // (either stream's products may come first)
                        kvc_tc::named_bar_sync(all_bar, kSoftmax);
                    }
                };
                if (TILES == 2 && cut)
                    scan();
                if (TILES == 2 && !st.has(stream, j))
                    continue;
                const int s = TILES == 2 ? stream : (int)(used & 1);
                const uint32_t parity = TILES == 2 ? used & 1 : (used >> 1) & 1;
                const uint32_t s_col = lane_addr + SM::COL_S + s * kBN;
                wait_or_abort(&s_full[s], parity, abort_flag, a.status);
                ++used;
                kvc_tc::fence_after();
                // the weights of either half go where its own scores were, so that neither waits for the other
                const uint32_t from = s_col + CT * half;
                const uint32_t to = SM::OWN_P ? lane_addr + SM::COL_P + s * 64 + 32 * half : from;
                float top = -INFINITY;
                const uint32_t half_there = SM::EARLY ? smem_base + (uint32_t)SM::HALF_OFF + 8u * stream : 0u;
                // (every row sees all of a whole tile)
                const bool plain = !cut && !flip;
                int lo = 0, hi = 0;
                if (!plain) {
                    rows_seen(j, lo, hi);
                    lo -= CT * half;
                    hi -= CT * half;
                }
                if (active)
                    top = plain ? row_top<CT>(from) : row_top<CT>(from, lo, hi, flip);
                red[(s * 2 + half) * kBM + m] = top;
                kvc_tc::named_bar_sync(pair_bar, 64);
                if (active) {
                    top = fmaxf(top, red[(s * 2 + (half ^ 1)) * kBM + m]) * c_log2;
                    float alpha = 1.f;
                    bool rescale = false;
                    if (top > m_run + kRescale || (m_run == -INFINITY && top > -INFINITY)) {
                        if (m_run > -INFINITY) {
                            alpha = kvc_tc::fast_exp2(m_run - top);
                            rescale = true;
                        }
                        m_run = top;
                    }
                    if (__any_sync(0xffffffffu, rescale)) {
                        // the reference moved: rescale this thread's part of the O row
                        // (the products of the tile before; with two streams they were done before S was written)
                        if (TILES == 2)
                            wait_or_abort(&o_done[s], (used - 2) & 1, abort_flag, a.status);
                        else
                            wait_or_abort(&o_done[s ^ 1], ((used - 2) >> 1) & 1, abort_flag, a.status);
                        kvc_tc::fence_after();
#pragma unroll 1
                        for (int cc = half * OT; cc < (half + 1) * OT; cc += 32) {
                            uint32_t o[32];
                            kvc_tc::ld32(lane_addr + stream * D + cc, o);
                            kvc_tc::wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                            kvc_tc::st32(lane_addr + stream * D + cc, o);
                        }
                        kvc_tc::wait_st();
                    }
                    const float neg_m = m_run == -INFINITY ? 0.f : -m_run;
                    if (SM::OWN_P && used > 1) {
                        // the products of the tile before have read its weights
                        wait_or_abort(&o_done[s], (used - 2) & 1, abort_flag, a.status);
                        kvc_tc::fence_after();
                    }
                    const float sum = plain ? row_weights<T, CT, false>(from, to, lo, hi, flip, c_log2, neg_m, half_there)
                                            : row_weights<T, CT, true>(from, to, lo, hi, flip, c_log2, neg_m, half_there);
                    l_run = l_run * alpha + sum;
                } else if (half_there) {
                    kvc_tc::fence_before();
                    __syncwarp();
                    if (lane == 0)
                        kvc_tc::arrive_at(half_there);
                }
                if (TILES == 1 && cut)
                    scan();
                kvc_tc::fence_before();
                __syncwarp();
                if (lane == 0)
                    kvc::mbar_arrive(&p_full[s]);
            }
            q0 += 2 * SPT * st.n;

            // ---- output rows ----
            // (the next segment's first output products wait for its p_full, which every warp gives after this)
            if (st.tiles(stream) > 0) {
                const uint32_t last = used - 1;
                if (TILES == 2)
                    wait_or_abort(&o_done[stream], last & 1, abort_flag, a.status);
                else
                    wait_or_abort(&o_done[last & 1], (last >> 1) & 1, abort_flag, a.status);
            }
            kvc_tc::fence_after();
            const Segment seg = kept->seg[s_no & 1];
            const int first = seg.i * a.item + (st.two ? stream * a.toks : 0), tok = m / a.group;
            const bool there = tok < a.toks && first + tok < seg.n && !*abort_flag, whole = seg.t1 - seg.t0 == seg.tiles;
            const int64_t out_row = (int64_t)(seg.row0 + first + tok) * a.q_heads + seg.h * a.group + (m - tok * a.group);
            const int64_t part = (int64_t)seg.slot * TILES + (st.two ? stream : 0);
            float l = l_run, ref = m_run;
            float w0 = 1.f, w1 = 0.f;  // what the two streams' outputs of a row count
            int col0 = half * OT, cols = OT;  // output columns of this thread
            // The halves' sums change hands where the maxima did (of the last tile: read, or its products would
            // not be done; two buffers in turn: in the other one).
            const uint32_t at = TILES == 2 ? stream : (used & 1);
            red[(at * 2 + half) * kBM + m] = l_run;
            kvc_tc::named_bar_sync(pair_bar, 64);
            l += red[(at * 2 + (half ^ 1)) * kBM + m];
            const bool share = TILES == 2 && !st.two;
            if (share) {
                // one query tile, two streams of keys: four threads have the row, each joins a quarter of the columns
                kvc_tc::fence_before();
                kvc_tc::named_bar_sync(all_bar, kSoftmax);
                kvc_tc::fence_after();
                red[(stream * 2 + half) * kBM + m] = half ? l : m_run;
                kvc_tc::named_bar_sync(all_bar, kSoftmax);
                const float m0 = red[m], l0 = red[kBM + m], m1 = red[2 * kBM + m], l1 = red[3 * kBM + m];
                // (a stream without a visible key has no sum, and its output may hold anything)
                ref = fmaxf(l0 == 0.f ? -INFINITY : m0, l1 == 0.f ? -INFINITY : m1);
                w0 = l0 == 0.f ? -1.f : m0 == ref || ref == -INFINITY ? 1.f : kvc_tc::fast_exp2(m0 - ref);
                w1 = l1 == 0.f ? -1.f : m1 == ref || ref == -INFINITY ? 1.f : kvc_tc::fast_exp2(m1 - ref);
                l = (l0 == 0.f ? 0.f : l0 * w0) + (l1 == 0.f ? 0.f : l1 * w1);
                cols = OT / 2;
                col0 += stream * cols;
            }
            if (active) {
                const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
                for (int cc = col0; cc < col0 + cols; cc += 16) {
                    uint32_t o[16];
                    if (!share) {
                        kvc_tc::ld16(lane_addr + stream * D + cc, o);
                        kvc_tc::wait_ld();
                    } else {
                        uint32_t o1[16];
                        kvc_tc::ld16(lane_addr + cc, o);
                        kvc_tc::ld16(lane_addr + D + cc, o1);
                        kvc_tc::wait_ld();
#pragma unroll
                        for (int c = 0; c < 16; ++c) {
                            const float x = w0 >= 0.f ? __uint_as_float(o[c]) * w0 : 0.f;
                            o[c] = __float_as_uint(w1 >= 0.f ? fmaf(__uint_as_float(o1[c]), w1, x) : x);
                        }
                    }
                    if (!there)
                        continue;
                    const uint32_t bad = nans ? nan_cols[(cc - half * OT) / 32] >> (cc & 16) : 0u;
                    if (bad) {
#pragma unroll
                        for (int c = 0; c < 16; ++c)
                            o[c] = bad >> c & 1u ? 0x7fc00000u : o[c];
                    }
                    if (whole) {
                        T *to = static_cast<T *>(a.out) + out_row * D + cc;
#pragma unroll
                        for (int c = 0; c < 16; c += 8) {
                            uint4 x;
                            uint32_t *w = reinterpret_cast<uint32_t *>(&x);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                w[e] = kvc_tc::pack2<T>(kvc_tc::finite_or_nan(__uint_as_float(o[c + 2 * e]) * inv),
                                                        kvc_tc::finite_or_nan(__uint_as_float(o[c + 2 * e + 1]) * inv));
                            *reinterpret_cast<uint4 *>(to + c) = x;
                        }
                    } else {
                        // four columns of all 128 rows side by side, so that a warp's store is one run
                        uint4 *to = reinterpret_cast<uint4 *>(a.ws_o) + (part * (D / 4) + cc / 4) * kBM + m;
#pragma unroll
                        for (int c = 0; c < 16; c += 4)
                            to[c / 4 * kBM] = make_uint4(o[c], o[c + 1], o[c + 2], o[c + 3]);
                    }
                }
                if (!whole && there && col0 == 0) {
                    a.ws_m[part * kBM + m] = ref;
                    a.ws_l[part * kBM + m] = l;
                }
            }
            kvc_tc::fence_before();
            if (share)
                // both streams' outputs have been read, and the sums: the next segment may write them
                kvc_tc::named_bar_sync(all_bar, kSoftmax);
            // the next segment is there, and this one's rows and sums have been read
            kvc_tc::named_bar_sync(stream_bar, 256);
        }
    }

    __syncthreads();
    if (warp == 0) {
        kvc_tc::fence_after();
        kvc_tc::tmem_dealloc(tmem, SM::TMEM_COLS);
    }
}

// Joins the partial results of an item's rows that several CTAs worked on:
// out = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i.  The item's first keys are in the
// piece of exactly one CTA, which the block takes its number from and which has
// written down which item that is.  A block takes 16 rows at a time: a row a
// thread's low bits, so that 16 threads read a run of 256 bytes.
constexpr int kMergeRows = 16;
template <typename T, int D>
__global__ void __launch_bounds__(256)
ragged_merge_kernel(const RaggedArgs a)
{
    constexpr int TILES = Smem<D>::TILES;
    kvc::grid_dep_wait();
    const int c0 = blockIdx.x, lane = threadIdx.x & 31;
    const int4 split = a.split[c0];
    const int parts = split.w >> 1, slot0 = split.w & 1;
    if (parts == 0)
        return;
    const int row0 = split.x, left = split.y, h = split.z;
    // the item's segment is the first of its CTA, but in the first CTA if that began before it
    auto part = [&](int p, int tile) { return (2 * ((int64_t)c0 + p) + (p == 0 ? slot0 : 0)) * TILES + tile; };
    constexpr int R = kMergeRows, W = R / 8;
    constexpr int COLS = D / 4, LANES = 256 / R, PER = COLS / LANES;  // float4 columns, of a thread
    __shared__ float w_sh[R][33], sum_sh[R];
    const int warp = threadIdx.x >> 5, mine = threadIdx.x % R, c4 = threadIdx.x / R;
    constexpr int AHEAD = PER <= 2 ? 4 : 2;  // parts under way
    for (int g = blockIdx.y; g < TILES * kBM / R; g += gridDim.y) {
        const int tile = g / (kBM / R), m0 = g % (kBM / R) * R;
        // rows of the tile that hold queries
        const int rows = min(left - tile * a.toks, a.toks) * a.group;
        if (m0 >= rows)
            continue;
        float4 acc[PER], x[AHEAD][PER];
        auto load = [&](int p) {
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                const float4 *o = reinterpret_cast<const float4 *>(a.ws_o) +
                                  (part(min(p + k, parts - 1), tile) * COLS + c4) * kBM + m0 + mine;
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
        auto stat = [&](int p, int k) { return part(p, tile) * kBM + m0 + W * warp + k; };
        auto row_there = [&](int k) { return m0 + W * warp + k < rows; };
        for (int p = lane; p < parts; p += 32)
#pragma unroll
            for (int k = 0; k < W; ++k)
                if (row_there(k))
                    top[k] = fmaxf(top[k], a.ws_l[stat(p, k)] == 0.f ? -INFINITY : a.ws_m[stat(p, k)]);
#pragma unroll
        for (int d = 16; d; d >>= 1)
#pragma unroll
            for (int k = 0; k < W; ++k)
                top[k] = fmaxf(top[k], __shfl_xor_sync(0xffffffffu, top[k], d));
        for (int p0 = 0; p0 < parts; p0 += 32) {
            __syncthreads();
#pragma unroll
            for (int k = 0; k < W; ++k) {
                // a part's weight a lane; a part that saw nothing (no sum) has none (-1), whatever its O holds; one
                // that is too small for a number still has its part's NaN
                float w = -1.f;
                if (p0 + lane < parts && row_there(k)) {
                    const float l = a.ws_l[stat(p0 + lane, k)], mc = a.ws_m[stat(p0 + lane, k)];
                    if (l != 0.f) {
                        w = mc == top[k] || mc == -INFINITY ? 1.f : exp2f(mc - top[k]);
                        sum[k] += l * w;
                    }
                }
                w_sh[W * warp + k][lane] = w;
            }
            __syncthreads();
            const int here = min(32, parts - p0);
            for (int p = 0; p < here; p += AHEAD) {
#pragma unroll
                for (int k = 0; k < AHEAD; ++k) {
                    const float w = w_sh[mine][p + k];  // (-1 past the last part)
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
                if (p0 + p + AHEAD < parts)
                    load(p0 + p + AHEAD);
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
        const int m = m0 + mine;
        if (m < rows) {
            const float total = sum_sh[mine], inv = total == 0.f ? 0.f : 1.f / total;
            const int tok = m / a.group;
            const int64_t row = (int64_t)(row0 + tile * a.toks + tok) * a.q_heads + h * a.group +
                                (m - tok * a.group);
            T *to = static_cast<T *>(a.out) + row * D;
#pragma unroll
            for (int e = 0; e < PER; ++e) {
                uint2 y;
                y.x = kvc_tc::pack2<T>(kvc_tc::finite_or_nan(acc[e].x * inv), kvc_tc::finite_or_nan(acc[e].y * inv));
                y.y = kvc_tc::pack2<T>(kvc_tc::finite_or_nan(acc[e].z * inv), kvc_tc::finite_or_nan(acc[e].w * inv));
                *reinterpret_cast<uint2 *>(to + 4 * (c4 + LANES * e)) = y;
            }
        }
        __syncthreads();
    }
}

// The packed queries [tokens, q_heads, D] as (64 columns, heads, tokens, D / 64 column
// blocks): a box of (64, group, toks, 1) is a column block of a query tile.
bool encode_queries(CUtensorMap *map, const void *q, const RaggedArgs &a, int D, CUtensorMapDataType type)
{
    const PFN_cuTensorMapEncodeTiled_v12000 encode = kvc_host::tensor_map_encoder();
    if (!encode)
        return false;
    const cuuint64_t dims[4] = {64, (cuuint64_t)a.q_heads, (cuuint64_t)a.tokens, (cuuint64_t)D / 64};
    const cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)a.q_heads * D * 2, 128};
    const cuuint32_t box[4] = {64, (cuuint32_t)a.group, (cuuint32_t)a.toks, 1}, step[4] = {1, 1, 1, 1};
    return encode(map, type, 4, const_cast<void *>(q), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

template <typename T, int D>
kvc_status launch_attn(RaggedArgs &a, const void *q, const void *k, const void *v, int grid, cudaStream_t stream)
{
    using SM = Smem<D>;
    const CUtensorMapDataType tt = std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                                  : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const uint64_t rows = (uint64_t)a.n_pool * a.page_size * a.kv_heads;
    // column blocks of a box: a slab's, where the box has all its rows
    const int k_blocks = a.box_rows == kBN ? D / 64 / SM::SPT : 1, v_rows = std::min(a.box_rows, SM::KR),
              v_blocks = v_rows == SM::KR ? D / 64 : 1;
    CUtensorMap tq, tk, tv;
    if (!encode_queries(&tq, q, a, D, tt) ||
        !kvc_host::encode_3d_sw128(&tk, k, rows, D, a.box_rows, k_blocks, tt) ||
        !kvc_host::encode_3d_sw128(&tv, v, rows, D, v_rows, v_blocks, tt))
        return kvc_host::cuda_failed();
    auto kern = ragged_attn_kernel<T, D>;
    int dev = 0, optin = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess)
        return kvc_host::cuda_failed();
    const size_t smem = std::min<size_t>((size_t)SM::TOTAL + 1024, (size_t)optin);
    if (smem < (size_t)SM::TOTAL)
        return KVC_ERR_UNSUPPORTED;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return kvc_host::cuda_failed();
    if (kvc_host::launch_chained(kern, dim3(grid), SM::THREADS, smem, stream, tq, tk, tv, a) != cudaSuccess)
        return kvc_host::cuda_failed();
    if (grid * a.rounds > 1) {
        // blocks for the rows that an item has if requests are alike (they go round for more)
        const int64_t rows_each = (int64_t)((a.tokens + a.batch - 1) / a.batch) * a.group;
        const int64_t blocks = std::min<int64_t>((rows_each + kMergeRows - 1) / kMergeRows, SM::TILES * kBM / kMergeRows);
        if (kvc_host::launch_chained(ragged_merge_kernel<T, D>, dim3(grid * a.rounds - 1, (unsigned)blocks), 256, 0, stream, a) != cudaSuccess)
            return kvc_host::cuda_failed();
    }
    return kvc_host::launch_status();
}

template <typename T>
kvc_status dispatch(RaggedArgs &a, const void *q, const void *k, const void *v, int D, int grid, cudaStream_t stream)
{
    switch (D) {
    case 64:
        return launch_attn<T, 64>(a, q, k, v, grid, stream);
    case 128:
        return launch_attn<T, 128>(a, q, k, v, grid, stream);
    default:
        return launch_attn<T, 256>(a, q, k, v, grid, stream);
    }
}

// the workspace: two partial results of an item for each piece of each CTA (one an SM)
struct Layout {
    int grid, rounds;
    int64_t parts;  // of a query tile
    size_t m, l, split, total;
};
Layout layout_of(int head_dim)
{
    Layout w;
    w.grid = kvc_host::sm_count();
    w.rounds = head_dim <= 128 ? 1 : kRounds;
    w.parts = 2 * (int64_t)w.grid * w.rounds * (head_dim <= 128 ? 2 : 1);
    w.m = (size_t)w.parts * kBM * head_dim * sizeof(float);
    w.l = w.m + (size_t)w.parts * kBM * sizeof(float);
    w.split = w.l + (size_t)w.parts * kBM * sizeof(float);
    w.total = w.split + (size_t)w.grid * w.rounds * sizeof(int4);
    return w;
}

} // namespace

KVC_API size_t kvc_gqa_ragged_workspace_size(int batch, int tokens, int q_heads, int kv_heads, int head_dim)
{
    if (batch < 1 || tokens < 1 || kv_heads < 1 || q_heads < 1 || q_heads % kv_heads != 0 || head_dim < 1)
        return 0;
    return layout_of(head_dim).total;
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
    const size_t each = (size_t)batch * sizeof(int32_t);
    const kvc_host::Span offs{offsets, each + sizeof(int32_t)}, table{block_table, each * max_pages}, past{len.past_abs, each},
        total{len.total_abs, each}, resident{len.cache_total, each};
    if (kvc_host::collide({{out, rows}}, {offs, table, past, total, resident}) ||
        kvc_host::collide({{workspace, workspace_bytes}}, {{out, rows}, {q, rows}, {k_pool, pool}, {v_pool, pool}, offs, table, past,
                                                           total, resident}))
        return KVC_ERR_SHAPE;
    RaggedArgs a{};
    a.out = out;
    a.offsets = offsets;
    a.table = block_table;
    a.max_pages = max_pages;
    a.page_size = page_size;
    a.n_pool = n_pool_pages;
    a.len = len;
    a.batch = batch;
    a.tokens = tokens;
    a.q_heads = q_heads;
    a.kv_heads = kv_heads;
    a.group = q_heads / kv_heads;
    a.toks = kBM / a.group;
    a.item = a.toks * (head_dim <= 128 ? 2 : 1);
    // (an item of one query tile has both streams for its keys: half the time for each, but with head_dim 128 its
    // bytes take more than that)
    a.one = head_dim == 128 ? 2 : 1;
    a.two = head_dim == 128 ? 3 : head_dim == 64 ? 2 : 1;
    a.streams = head_dim <= 128 ? 2 : 1;
    // rows of a box: as many of a tile's that no page's end cuts
    a.box_rows = kBN;
    while (page_size % a.box_rows)
        a.box_rows /= 2;
    a.window = local_window_size;
    a.scale_log2 = (scale == 0.f ? 1.0f / sqrtf((float)head_dim) : scale) * kLog2e;
    a.status = dev_status;
    const Layout w = layout_of(head_dim);
    a.rounds = w.rounds;
    a.key_bytes = kv_heads * head_dim * 4;
    uint8_t *base = static_cast<uint8_t *>(workspace);
    a.ws_o = reinterpret_cast<float *>(base);
    a.ws_m = reinterpret_cast<float *>(base + w.m);
    a.ws_l = reinterpret_cast<float *>(base + w.l);
    a.split = reinterpret_cast<int4 *>(base + w.split);
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    return dtype == KVC_BF16 ? dispatch<__nv_bfloat16>(a, q, k_pool, v_pool, head_dim, w.grid, stream)
                             : dispatch<__half>(a, q, k_pool, v_pool, head_dim, w.grid, stream);
}
