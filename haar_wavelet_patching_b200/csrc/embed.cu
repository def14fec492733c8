// Embedding of codes and its gradient.
//
// Forward: y[n] = scale table[c_n], one row in and one out, bound by HBM.  A thread holds 16 bytes of a
// row (fewer where rows are not so aligned), up to kPer of them.
//
// Gradient: grad_table[v] = scale sum over the tokens n of code v of g[n].  Every row of the table is written and
// every row of g read once, so it is bound by HBM as well, if no row is added to twice: the tokens are sorted by
// code, stable, so the order of a sum is that of the tokens and no atomics are needed.
//
//   sort_kernel: one cluster sorts (code, token) pairs by digits of 8 or 10 bits, a slice of the pairs to a CTA and a
//   contiguous part of it to a warp.  Each pass counts digits per warp, adds the counts up over warps, CTAs and
//   digits, and moves each pair to its place.  (2 passes up to 2^20 codes.)
//
//   sum_kernel: the table's row ends and the tokens, merged in the order of codes, are one sequence of V + N
//   elements of equal cost (a row written, a row read); a group of threads takes kLen of them in turn, whatever the
//   codes' frequencies.  Where a border cuts a row with fewer than kAbsorb tokens behind it, the
//   group before takes these too; else both store partial sums (fp32), and join_kernel adds them up.
//
// Measured, 56,320 tokens, a table of 64,000 x 2048 bf16: forward 60 us (461 MB of rows in and out), gradient 113 us:
// sorting 20, sums 77 (493 MB, 6.4 TB/s), joining and the launches' gaps 16.  10,395 tokens, 64,000 x 1004 fp32,
// both: 83 us, of which the sort's chain of barriers counts for more.  80 tokens, forward: 1.7 us, the launch.
#include <algorithm>
#include <utility>

#include "tma.cuh"
#include "tok_common.cuh"
#include "tok_internal.h"
#include "umma.cuh"

namespace tok {
namespace {

constexpr int64_t kMaxV = 1 << 18;

// ---------------------------------------------------------------------------
// Forward.
// ---------------------------------------------------------------------------
constexpr int kThreads = 128;
constexpr int kPer = 4; // vectors of a row per thread

struct EmbedArgs {
    const int32_t *codes;
    const void *table;
    void *y;
    int32_t *bad_count;
    int64_t table_row, y_row;
    int V, units, lanes; // vectors per row, threads per row
    FastDiv lanes_div;
    uint32_t n0, items;
    float scale;
};

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) embed_kernel(const EmbedArgs g)
{
    const uint32_t item = blockIdx.x * kThreads + threadIdx.x;
    if (item >= g.items)
        return;
    const uint32_t ln = g.lanes_div.div(item);
    const int lane = (int)(item - ln * g.lanes_div.d);
    const int64_t n = (int64_t)g.n0 + ln;
    const int c = g.codes[n];
    const bool ok = (uint32_t)c < (uint32_t)g.V;
    if (!ok && lane == 0 && g.bad_count)
        atomicAdd(g.bad_count, 1);
    const T *src = static_cast<const T *>(g.table) + (ok ? c : 0) * g.table_row;
    T *dst = static_cast<T *>(g.y) + n * g.y_row;
    float v[kPer][V];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int u = lane + k * g.lanes;
        if (ok && u < g.units)
            Row<T, V, (V > 1)>::load(src + (int64_t)u * V, v[k]);
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int u = lane + k * g.lanes;
        if (u < g.units) {
#pragma unroll
            for (int e = 0; e < V; ++e)
                v[k][e] = ok ? v[k][e] * g.scale : __int_as_float(0x7FC00000);
            Row<T, V, (V > 1)>::store(dst + (int64_t)u * V, v[k]);
        }
    }
}

// Elements per vector: the most, of at most 16 bytes each, that the row length, strides and addresses allow.
int vector_of(int most, int64_t D, std::initializer_list<std::pair<const void *, int64_t>> rows, int64_t size)
{
    int v = most;
    for (; v > 1; v /= 2) {
        const int64_t vb = std::min<int64_t>(16, v * size);
        bool fits = D % v == 0;
        for (const auto &r : rows)
            fits = fits && aligned(r.first, vb) && r.second * size % vb == 0;
        if (fits)
            break;
    }
    return v;
}

template <typename T> void launch_embed(int v, const EmbedArgs &g, cudaStream_t stream)
{
    const unsigned blocks = (g.items + kThreads - 1) / kThreads;
    if constexpr (sizeof(T) == 2)
        if (v == 8) {
            embed_kernel<T, 8><<<blocks, kThreads, 0, stream>>>(g);
            return;
        }
    if (v == 4)
        embed_kernel<T, 4><<<blocks, kThreads, 0, stream>>>(g);
    else if (v == 2)
        embed_kernel<T, 2><<<blocks, kThreads, 0, stream>>>(g);
    else
        embed_kernel<T, 1><<<blocks, kThreads, 0, stream>>>(g);
}

// ---------------------------------------------------------------------------
// Gradient: sorting.
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kMaxSortCtas = 16; // (beyond 8 a cluster is not portable, but this GPU holds it)
constexpr int kAbsorb = 8;

struct SortArgs {
    const int32_t *codes;
    uint64_t *pairs[2]; // (code, token)
    uint2 *bounds;      // [chunks + 1]: first token (in sorted order) and row of each chunk
    uint32_t *joins;    // number of rows to join (cleared here)
    uint32_t N, V;
    int passes;
    uint32_t chunks, len;
};

// Exclusive scan of one value per thread over the block; all threads.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t *warp_sums)
{
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    uint32_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(~0u, x, o);
        if (lane >= o)
            x += y;
    }
    if (lane == 31)
        warp_sums[w] = x;
    __syncthreads();
    uint32_t s = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(~0u, s, o);
        if (lane >= o)
            s += y;
    }
    const uint32_t before = __shfl_sync(~0u, s, (w + 31) & 31);
    __syncthreads();
    return x - v + (w ? before : 0);
}

__device__ __forceinline__ uint32_t load_cluster(const uint32_t *p, uint32_t rank)
{
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(smem_addr(p), rank)) : "memory");
    return v;
}

template <int kBits> // of a digit
__global__ void __launch_bounds__(kSortThreads, 1) sort_kernel(const SortArgs g, int C)
{
    constexpr int digits = 1 << kBits;
    extern __shared__ uint32_t hist[]; // [warps][digits]
    __shared__ uint32_t totals[digits], base[digits], sums[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = C > 1 ? cluster_rank() : 0;
    // This warp's pairs: contiguous parts of contiguous slices, whole 32s.
    const uint32_t per = (((g.N + C * kSortWarps - 1) / (C * kSortWarps)) + 31) & ~31u;
    const uint64_t first = (uint64_t)(rank * kSortWarps + warp) * per;
    const uint32_t i0 = (uint32_t)min((uint64_t)g.N, first), i1 = (uint32_t)min((uint64_t)g.N, first + per);
    uint32_t *mine = hist + warp * digits;
    if (rank == 0 && tid == 0)
        *g.joins = 0;
    asm volatile("griddepcontrol.launch_dependents;");
    for (int pass = 0; pass < g.passes; ++pass) {
        const uint64_t *src = g.pairs[(pass + 1) & 1];
        uint64_t *dst = g.pairs[pass & 1];
        const int shift = pass * kBits;
        auto pair = [&](uint32_t i) -> uint64_t {
            if (pass > 0)
                return src[i];
            const uint32_t c = (uint32_t)g.codes[i];
            return (uint64_t)(c < g.V ? c : g.V) << 32 | i; // (codes outside the table behind all others)
        };
        // f(pair, whether there is one) for this warp's pairs, 32 at a time in order, kAtOnce x 32 loads on their way;
        // what fits into one batch is loaded once per pass.
        constexpr int kAtOnce = 8;
        uint64_t held[kAtOnce];
        auto batches = [&](bool load, auto &&f) {
            for (uint32_t i = i0; i < i1; i += 32 * kAtOnce) {
                if (load || i1 - i0 > 32 * kAtOnce) {
#pragma unroll
                    for (int e = 0; e < kAtOnce; ++e)
                        held[e] = i + 32 * e + lane < i1 ? pair(i + 32 * e + lane) : 0;
                }
#pragma unroll
                for (int e = 0; e < kAtOnce; ++e)
                    if (i + 32 * e < i1)
                        f(held[e], i + 32 * e + lane < i1);
            }
        };
        // The lanes with the same digit, by a vote per bit (the instruction that matches whole values takes 10 times as
        // long with 32 warps at it).
        auto alike = [&](uint32_t d, bool on) {
            uint32_t same = __ballot_sync(~0u, on);
#pragma unroll
            for (int b = 0; b < kBits; ++b) {
                const bool bit = d >> b & 1;
                const uint32_t set = __ballot_sync(~0u, bit);
                same &= bit ? set : ~set;
            }
            return same;
        };
        for (int d = lane; d < digits; d += 32)
            mine[d] = 0;
        __syncwarp();
        batches(true, [&](uint64_t p, bool on) {
            if (on)
                atomicAdd(&mine[(uint32_t)(p >> 32) >> shift & (digits - 1)], 1u);
        });
        __syncthreads();
        for (int d = tid; d < digits; d += kSortThreads) { // counts of the warps before
            uint32_t run = 0;
#pragma unroll 8
            for (int w = 0; w < kSortWarps; ++w) {
                const uint32_t x = hist[w * digits + d];
                hist[w * digits + d] = run;
                run += x;
            }
            totals[d] = run;
        }
        if (C > 1)
            cluster_sync();
        else
            __syncthreads();
        uint32_t before = 0, all = 0;
        if (tid < digits) {
            uint32_t x[kMaxSortCtas];
#pragma unroll
            for (int c = 0; c < kMaxSortCtas; ++c)
                x[c] = c >= C ? 0 : C > 1 ? load_cluster(&totals[tid], c) : totals[tid];
#pragma unroll
            for (int c = 0; c < kMaxSortCtas; ++c) {
                before += c < (int)rank ? x[c] : 0;
                all += x[c];
            }
        }
        const uint32_t at = block_scan(all, sums);
        if (tid < digits)
            base[tid] = at + before;
        __syncthreads();
        batches(false, [&](uint64_t p, bool on) {
            const uint32_t d = (uint32_t)(p >> 32) >> shift & (digits - 1), same = alike(d, on);
            const uint32_t below = __popc(same & ((1u << lane) - 1));
            if (on)
                dst[base[d] + mine[d] + below] = p;
            __syncwarp();
            if (on && below == 0)
                mine[d] += __popc(same);
            __syncwarp();
        });
        if (C > 1)
            cluster_sync(); // (also: nobody reads totals any more)
        else
            __syncthreads();
    }
    // The chunks' borders.  Token i of code k is element i + k of the merged sequence (k row ends lie before it);
    // thread i finds the borders between its element and that of the token before.
    const uint64_t *sorted = g.pairs[(g.passes - 1) & 1];
    auto key = [&](uint32_t i) -> uint32_t { return i < g.N ? (uint32_t)(sorted[i] >> 32) : g.V; };
    const uint32_t step = C * kSortThreads;
    constexpr int kAtOnce = 4, kAlone = 96; // (borders that a lane writes by itself)
    for (uint64_t j0 = rank * kSortThreads + warp * 32; j0 <= g.N; j0 += (uint64_t)step * kAtOnce) {
        const uint64_t j = j0 + lane;
        uint32_t ks[kAtOnce], kps[kAtOnce];
#pragma unroll
        for (int e = 0; e < kAtOnce; ++e) {
            const uint32_t i = (uint32_t)min(j + (uint64_t)step * e, (uint64_t)g.N);
            ks[e] = key(i);
            kps[e] = i ? key(i - 1) : 0;
        }
#pragma unroll
        for (int e = 0; e < kAtOnce; ++e) {
            const uint64_t at = j + (uint64_t)step * e;
            const uint32_t i = (uint32_t)at, k = ks[e], kp = kps[e];
            const bool is = at <= g.N && !(i && kp == g.V); // (no elements behind a code outside the table)
            uint32_t lo = is && i ? (i - 1 + kp) / g.len + 1 : 0, end = 0; // its borders: [lo, end)
            if (is)
                end = (k == g.V ? g.chunks : (i + k) / g.len) + 1;
            uint32_t rem = 0; // tokens of the code before from here on (up to kAbsorb)
            if (lo < end && i && k == kp) {
                uint32_t more = 0;
#pragma unroll
                for (int r = 0; r < kAbsorb; ++r)
                    more |= (uint32_t)(key(i + r) == kp) << r;
                rem = __ffs(~more) - 1; // (bit kAbsorb is not set)
            }
            auto border = [&](uint32_t c, uint32_t i, uint32_t kp, uint32_t rem) {
                uint2 b = make_uint2(i, min(c * g.len - i, g.V)); // the row of element c * len
                if (i && b.y == kp && rem < kAbsorb) // the border cuts a row: its rest goes to the chunk before
                    b = make_uint2(i + rem, kp + 1);
                g.bounds[c] = b;
            };
            for (int n = 0; n < kAlone && lo < end; ++n)
                border(lo++, i, kp, rem);
            __syncwarp();
            // More between two tokens (of few ones in a large table): all lanes (1 token, 64,000 x 512: 37 -> 22 us;
            // with 4 borders to a lane 110 tokens took 34 us for 33).
            for (uint32_t many = __ballot_sync(~0u, lo < end); many; many &= many - 1) {
                const int from = __ffs(many) - 1;
                const uint32_t c0 = __shfl_sync(~0u, lo, from), c1 = __shfl_sync(~0u, end, from);
                const uint32_t fi = __shfl_sync(~0u, i, from), fk = __shfl_sync(~0u, kp, from);
                const uint32_t fr = __shfl_sync(~0u, rem, from);
                for (uint32_t c = c0 + lane; c < c1; c += 32)
                    border(c, fi, fk, fr);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Gradient: sums.
// ---------------------------------------------------------------------------
constexpr int kSumThreads = 256;
constexpr int kBatch = 4; // rows of g on their way

struct SumArgs {
    const uint64_t *sorted;
    const uint2 *bounds;
    const void *grad;
    void *table;
    uint32_t *joins; // their number, then the chunks that a row ends in which was begun before
    float *part; // [chunks][2][D]: sums of a chunk's first row (begun before it), of its last one (going on behind)
    int64_t grad_row, table_row;
    uint32_t N, V, chunks;
    int D, units, slab; // vectors of a row, of a row's part
    int tg;             // threads to a group
    float scale;
};

// V elements as they lie in memory.
template <int kBytes> struct RawOf;
template <> struct RawOf<16> {
    using type = uint4;
};
template <> struct RawOf<8> {
    using type = uint2;
};
template <> struct RawOf<4> {
    using type = uint32_t;
};
template <> struct RawOf<2> {
    using type = unsigned short;
};
template <typename T, int V> struct Raw {
    using type = typename RawOf<V * (int)sizeof(T)>::type;
    static __device__ __forceinline__ void add(const type &x, float *acc)
    {
        const T *v = reinterpret_cast<const T *>(&x);
#pragma unroll
        for (int e = 0; e < V; ++e)
            acc[e] += (float)v[e];
    }
};

template <typename TG, typename TT, int V>
__global__ void __launch_bounds__(kSumThreads, 3) sum_kernel(const SumArgs g)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int group = threadIdx.x / g.tg, u = (int)blockIdx.y * g.slab + threadIdx.x % g.tg;
    const uint32_t c = blockIdx.x * (kSumThreads / g.tg) + group;
    if (c >= g.chunks || u >= min(g.units, ((int)blockIdx.y + 1) * g.slab))
        return;
    const uint2 b0 = g.bounds[c], b1 = g.bounds[c + 1];
    const int64_t d = (int64_t)u * V;
    const TG *src = static_cast<const TG *>(g.grad) + d;
    TT *dst = static_cast<TT *>(g.table) + d;
    uint32_t v = b0.y;
    bool begun = b0.x > 0 && (uint32_t)(g.sorted[b0.x - 1] >> 32) == v; // the first row's tokens begin before
    if (begun && v < b1.y && u == 0)
        g.joins[1 + atomicAdd(g.joins, 1u)] = c; // (their order does not matter)
    float acc[V];
#pragma unroll
    for (int e = 0; e < V; ++e)
        acc[e] = 0.0f;
    auto emit = [&]() {
        if (begun) {
            Row<float, V, (V > 1)>::store(g.part + (int64_t)c * 2 * g.D + d, acc);
            begun = false;
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e)
                acc[e] *= g.scale;
            Row<TT, V, (V > 1)>::store(dst + (int64_t)v * g.table_row, acc);
        }
#pragma unroll
        for (int e = 0; e < V; ++e)
            acc[e] = 0.0f;
        ++v;
    };
    // Tokens' rows one batch ahead of the sums, the tokens two.
    using R = Raw<TG, V>;
    uint64_t p[kBatch], q[kBatch];
    typename R::type x[kBatch], y[kBatch];
    auto tokens = [&](uint32_t t, uint64_t (&to)[kBatch]) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            to[k] = t + k < b1.x ? g.sorted[t + k] : 0;
    };
    auto rows = [&](uint32_t t, const uint64_t (&of)[kBatch], typename R::type (&to)[kBatch]) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (t + k < b1.x)
                to[k] = *reinterpret_cast<const typename R::type *>(src + (int64_t)(uint32_t)of[k] * g.grad_row);
    };
    tokens(b0.x, p);
    rows(b0.x, p, x);
    tokens(b0.x + kBatch, q);
    for (uint32_t t = b0.x; t < b1.x; t += kBatch) {
        rows(t + kBatch, q, y);
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (t + k < b1.x) {
                while (v < (uint32_t)(p[k] >> 32))
                    emit();
                R::add(x[k], acc);
            }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            x[k] = y[k];
            p[k] = q[k];
        }
        tokens(t + 2 * kBatch, q);
    }
    while (v < b1.y)
        emit();
    if (b1.x > b0.x && (uint32_t)(g.sorted[b1.x - 1] >> 32) == v) // tokens of a row that goes on
        Row<float, V, (V > 1)>::store(g.part + ((int64_t)c * 2 + 1) * g.D + d, acc);
}

// Rows that were begun in an earlier chunk: the partial sums, in order within each of kJoinParts interleaved
// parts, then of the parts.  A CTA takes 32 channels of a row at a time.
constexpr int kJoinParts = 8;

template <typename TT>
__global__ void __launch_bounds__(32 * kJoinParts) join_kernel(const SumArgs g)
{
    __shared__ float sums[kJoinParts][32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, part = tid >> 5;
    const uint32_t slabs = (uint32_t)(g.D + 31) / 32, items = g.joins[0] * slabs;
    for (uint32_t item = blockIdx.x; item < items; item += gridDim.x) {
        const uint32_t c = g.joins[1 + item / slabs], row = g.bounds[c].y;
        auto inside = [&](uint32_t x) { // chunk x starts inside the row
            const uint2 b = g.bounds[x];
            return b.x > 0 && b.y == row && (uint32_t)(g.sorted[b.x - 1] >> 32) == row;
        };
        uint32_t first = c; // the chunk that the row begins in
        for (;;) {
            const bool in = first > (uint32_t)tid && inside(first - tid);
            const int n = __syncthreads_count(in); // (the chunks first - t, t < n, start inside)
            first -= n;
            if (n < 32 * kJoinParts)
                break;
        }
        const int d = (int)(item % slabs) * 32 + lane;
        float acc = 0.0f;
        if (d < g.D)
#pragma unroll 8
            for (uint32_t x = first + part; x < c; x += kJoinParts)
                acc += g.part[((int64_t)x * 2 + 1) * g.D + d];
        sums[part][lane] = acc;
        __syncthreads();
        if (part == 0 && d < g.D) {
            for (int j = 1; j < kJoinParts; ++j)
                acc += sums[j][lane];
            acc = (acc + g.part[(int64_t)c * 2 * g.D + d]) * g.scale;
            Row<TT, 1, false>::store(static_cast<TT *>(g.table) + (int64_t)row * g.table_row + d, &acc);
        }
    }
}

// How the gradient is shared out.
struct Plan {
    int64_t len, chunks; // elements of a chunk of the merged sequence
    int C, passes, bits;
    int64_t at_order, at_bounds, at_joins, at_part, bytes;
    Plan(int64_t N, int64_t V, int64_t D)
    {
        // Chunks of a group of 256 threads that hold up to 2048 channels: four rounds of 3 CTAs per SM.
        const int64_t groups = 148 * 12 * std::max<int64_t>(1, 2048 / std::max<int64_t>(D, 64));
        len = std::max<int64_t>(4 * kAbsorb, (N + V + groups - 1) / groups);
        chunks = (N + V + len - 1) / len;
        int width = 1; // bits of the largest key, V
        while (V >> width)
            ++width;
        passes = width <= 8 ? 1 : 2;
        bits = width <= 16 ? 8 : 10;
        C = 1;
        while (C < kMaxSortCtas && N > (int64_t)C * kSortThreads)
            C *= 2;
        auto up = [](int64_t x) { return (x + 15) / 16 * 16; };
        at_order = up(N * 8);
        at_bounds = at_order + up(N * 8);
        at_joins = at_bounds + up((chunks + 1) * 8);
        at_part = at_joins + up((chunks + 1) * 4);
        bytes = at_part + chunks * 2 * D * 4;
    }
};

bool embed_dims_ok(int64_t N, int64_t V, int64_t D)
{
    return N >= 0 && N < ((int64_t)1 << 30) && V >= 1 && V <= kMaxV && D >= 1 && D <= 65536;
}

// Bytes from the first to the last element of [n, D] with rows `row` apart; false where the stride does not fit.
bool rows_ok(int64_t n, int64_t row, int64_t D, int64_t size, int64_t *bytes)
{
    if (n <= 1) {
        *bytes = n * D * size;
        return true;
    }
    if (row < D || row >= ((int64_t)1 << 38) / n)
        return false;
    *bytes = ((n - 1) * row + D) * size;
    return true;
}

template <typename TG, typename TT> tok_status launch_sums(int v, const SumArgs &g, dim3 grid, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.stream = stream;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kSumThreads);
    void (*sums)(SumArgs) = v == 4   ? sum_kernel<TG, TT, 4>
                            : v == 2 ? sum_kernel<TG, TT, 2>
                                     : sum_kernel<TG, TT, 1>;
    if constexpr (sizeof(TG) == 2)
        if (v == 8)
            sums = sum_kernel<TG, TT, 8>;
    cudaError_t e = cudaLaunchKernelEx(&cfg, sums, g);
    if (e == cudaSuccess) {
        cfg.gridDim = dim3((unsigned)std::min<int64_t>(148 * 4, (int64_t)g.chunks * ((g.D + 31) / 32)));
        cfg.blockDim = dim3(32 * kJoinParts);
        e = cudaLaunchKernelEx(&cfg, join_kernel<TT>, g);
    }
    if (e != cudaSuccess) {
        record_cuda_error(e);
        cudaGetLastError();
        return TOK_ERR_CUDA;
    }
    return launch_status();
}

} // namespace
} // namespace tok

extern "C" tok_status tok_embed_codes(const int32_t *codes, const void *table, void *y, int32_t *bad_count,
                                      tok_dtype dtype, int64_t N, int64_t V, int64_t D, int64_t table_row,
                                      int64_t y_row, float scale, cudaStream_t stream)
{
    using namespace tok;
    if (dtype != TOK_F32 && dtype != TOK_BF16)
        return TOK_ERR_DTYPE;
    const int64_t size = dtype == TOK_F32 ? 4 : 2;
    int64_t tb, yb;
    if (!embed_dims_ok(N, V, D))
        return TOK_ERR_SHAPE;
    if (N == 0)
        return TOK_OK;
    if (!rows_ok(V, table_row, D, size, &tb) || !rows_ok(N, y_row, D, size, &yb))
        return TOK_ERR_SHAPE;
    if (!codes || !table || !y)
        return TOK_ERR_NULL;
    if (!aligned(codes, 4) || !aligned(table, size) || !aligned(y, size) || !aligned(bad_count, 4))
        return TOK_ERR_ALIGN;
    if (overlaps(y, yb, table, tb) || overlaps(y, yb, codes, 4 * N) ||
        (bad_count && (overlaps(bad_count, 4, y, yb) || overlaps(bad_count, 4, table, tb) ||
                       overlaps(bad_count, 4, codes, 4 * N))))
        return TOK_ERR_ALIAS;
    const int v = vector_of(size == 4 ? 4 : 8, D, {{table, V > 1 ? table_row : 0}, {y, N > 1 ? y_row : 0}}, size);
    EmbedArgs g{};
    g.codes = codes;
    g.table = table;
    g.y = y;
    g.bad_count = bad_count;
    g.table_row = table_row;
    g.y_row = y_row;
    g.V = (int)V;
    g.units = (int)(D / v);
    g.lanes = (g.units + kPer - 1) / kPer;
    g.lanes_div = FastDiv((uint32_t)g.lanes);
    g.scale = scale;
    const int64_t most = (((int64_t)1 << 31) - 1) / g.lanes; // tokens of a launch (items are 32-bit)
    tok_status st = TOK_OK;
    for (int64_t n0 = 0; n0 < N && st == TOK_OK; n0 += most) {
        g.n0 = (uint32_t)n0;
        g.items = (uint32_t)(std::min(most, N - n0) * g.lanes);
        dtype == TOK_F32 ? launch_embed<float>(v, g, stream) : launch_embed<__nv_bfloat16>(v, g, stream);
        st = launch_status();
    }
    return st;
}

extern "C" int64_t tok_embed_codes_backward_workspace_size(int64_t N, int64_t V, int64_t D)
{
    return tok::embed_dims_ok(N, V, D) ? tok::Plan(N, V, D).bytes : -1;
}

extern "C" tok_status tok_embed_codes_backward(const int32_t *codes, const void *grad_y, void *grad_table,
                                               tok_dtype grad_dtype, tok_dtype table_dtype, int64_t N, int64_t V,
                                               int64_t D, int64_t grad_row, int64_t table_row, float scale,
                                               void *workspace, int64_t workspace_bytes, cudaStream_t stream)
{
    using namespace tok;
    for (tok_dtype t : {grad_dtype, table_dtype})
        if (t != TOK_F32 && t != TOK_BF16)
            return TOK_ERR_DTYPE;
    const int64_t gs = grad_dtype == TOK_F32 ? 4 : 2, ts = table_dtype == TOK_F32 ? 4 : 2;
    int64_t gb, tb;
    if (!embed_dims_ok(N, V, D) || !rows_ok(N, grad_row, D, gs, &gb) || !rows_ok(V, table_row, D, ts, &tb))
        return TOK_ERR_SHAPE;
    const Plan plan(N, V, D);
    if (workspace_bytes < plan.bytes)
        return TOK_ERR_SHAPE;
    if (!grad_table || !workspace || (N > 0 && (!codes || !grad_y)))
        return TOK_ERR_NULL;
    if (!aligned(codes, 4) || !aligned(grad_y, gs) || !aligned(grad_table, ts) || !aligned(workspace, 16))
        return TOK_ERR_ALIGN;
    if (overlaps(grad_table, tb, workspace, plan.bytes) ||
        (N > 0 && (overlaps(grad_table, tb, grad_y, gb) || overlaps(grad_table, tb, codes, 4 * N) ||
                   overlaps(workspace, plan.bytes, grad_y, gb) || overlaps(workspace, plan.bytes, codes, 4 * N))))
        return TOK_ERR_ALIAS;

    char *ws = static_cast<char *>(workspace);
    SortArgs s{};
    s.codes = codes;
    s.pairs[0] = reinterpret_cast<uint64_t *>(ws);
    s.pairs[1] = reinterpret_cast<uint64_t *>(ws + plan.at_order);
    s.bounds = reinterpret_cast<uint2 *>(ws + plan.at_bounds);
    s.joins = reinterpret_cast<uint32_t *>(ws + plan.at_joins);
    s.N = (uint32_t)N;
    s.V = (uint32_t)V;
    s.passes = plan.passes;
    s.chunks = (uint32_t)plan.chunks;
    s.len = (uint32_t)plan.len;
    const int smem = (kSortWarps << plan.bits) * 4;
    void (*sort)(SortArgs, int) = plan.bits == 8 ? sort_kernel<8> : sort_kernel<10>;
    cudaError_t e = cudaFuncSetAttribute(sort, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(sort, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) {
        record_cuda_error(e);
        return TOK_ERR_CUDA;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)plan.C);
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)plan.C;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, sort, s, plan.C);
    if (e != cudaSuccess) {
        record_cuda_error(e);
        cudaGetLastError();
        return TOK_ERR_CUDA;
    }

    const int v = std::min(vector_of(gs == 4 ? 4 : 8, D, {{grad_y, N > 1 ? grad_row : 0}}, gs),
                           vector_of(8, D, {{grad_table, V > 1 ? table_row : 0}}, ts));
    SumArgs g{};
    g.sorted = s.pairs[(plan.passes - 1) & 1];
    g.bounds = s.bounds;
    g.joins = s.joins;
    g.grad = grad_y;
    g.table = grad_table;
    g.part = reinterpret_cast<float *>(ws + plan.at_part);
    g.grad_row = grad_row;
    g.table_row = table_row;
    g.N = (uint32_t)N;
    g.V = (uint32_t)V;
    g.chunks = (uint32_t)plan.chunks;
    g.D = (int)D;
    g.units = (int)(D / v);
    const int slabs = (g.units + kSumThreads - 1) / kSumThreads;
    g.slab = (g.units + slabs - 1) / slabs;
    g.tg = 1;
    while (g.tg < g.slab)
        g.tg *= 2;
    g.scale = scale;
    const int groups = kSumThreads / g.tg;
    const dim3 grid((unsigned)((plan.chunks + groups - 1) / groups), (unsigned)slabs);
    if (grad_dtype == TOK_F32)
        return table_dtype == TOK_F32 ? launch_sums<float, float>(v, g, grid, stream)
                                      : launch_sums<float, __nv_bfloat16>(v, g, grid, stream);
    return table_dtype == TOK_F32 ? launch_sums<__nv_bfloat16, float>(v, g, grid, stream)
                                  : launch_sums<__nv_bfloat16, __nv_bfloat16>(v, g, grid, stream);
}
