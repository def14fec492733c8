// Pages of a cache of keys and values: the streams' page tables and the new tokens' slots, pages given back,
// and keys and values written into the pages.
//
// tables_kernel is one cluster: each CTA adds up what all streams need (one pass of scans over B numbers, so no CTA
// waits for another), then the CTAs share the tokens' slots and the new pages.  Counts are written behind a cluster
// barrier, as they may replace the ones that were read.  It is bound by latency: the launch, the loads of the counts,
// a scan, the loads of table entries, the stores.  Measured: 16 streams of 5 tokens 4.8 us, 256 of 880 15.4 (eight
// slots of a thread at a time, their loads together: 16.8).
// write_kernel moves up to four pieces of 16 bytes per thread, bound by HBM: 28,160 tokens of 8 heads x 128, a quarter
// of them with slots of -1, 28.7 us (173 MB, 6.0 TB/s); 16 streams of 5 tokens 2.2 us, the launch.
#include <algorithm>

#include "pages.cuh"

namespace tok {
namespace {

// ---------------------------------------------------------------------------
// Tables.
// ---------------------------------------------------------------------------
constexpr int kThreads = 1024;
constexpr int kMaxCluster = 8;

struct TablesArgs {
    const int32_t *lens, *fresh, *held, *free_count;
    const int32_t *pages;
    int32_t *pages_out;
    int32_t *table, *slots, *held_out, *free_out, *bad_count;
    int B, N, M, F;
    int64_t table_row;
    FastDiv page, n_div;
};

// Inclusive scan of one value per thread over the block, *total the sum; all threads.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t *sums, int64_t *total)
{
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(~0u, v, o);
        if (lane >= o)
            v += y;
    }
    __syncthreads(); // `sums` may still be read from an earlier use
    if (lane == 31)
        sums[w] = v;
    __syncthreads();
    int64_t s = sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(~0u, s, o);
        if (lane >= o)
            s += y;
    }
    *total = __shfl_sync(~0u, s, 31);
    const int64_t before = __shfl_sync(~0u, s, (w + 31) & 31);
    return v + (w ? before : 0);
}

__device__ __forceinline__ int pages_of(const TablesArgs &g, int64_t tokens) // for up to M pages' tokens and one more
{
    return (int)g.page.div((uint32_t)(tokens + g.page.d - 1));
}

struct Stream {
    int len, fresh, held, need; // new tokens, 0 where the stream is not served; pages held; pages taken
    bool bad;
};

// What stream b asks for.
__device__ __forceinline__ Stream ask(const TablesArgs &g, int b)
{
    Stream s;
    s.len = g.lens[b];
    s.fresh = min(max(g.fresh ? g.fresh[b] : g.N, 0), g.N);
    s.held = min(max(g.held[b], 0), g.M);
    const int64_t tokens = (int64_t)s.len + s.fresh;
    s.bad = s.len < 0 || tokens > (int64_t)g.M * g.page.d;
    s.need = s.bad ? 0 : max(0, pages_of(g, tokens) - s.held);
    return s;
}

__global__ void __launch_bounds__(kThreads) tables_kernel(const TablesArgs g, int C)
{
    __shared__ int64_t sums[32];
    __shared__ int s_len[kThreads], s_fresh[kThreads], s_held[kThreads], s_need[kThreads];
    __shared__ int64_t s_top[kThreads]; // place of the stream's first new page in the list
    const int tid = threadIdx.x, rank = C > 1 ? (int)cluster_rank() : 0;
    const int free0 = min(max(*g.free_count, 0), g.F);
    int64_t run = 0, taken = 0;
    for (int b0 = 0; b0 < g.B; b0 += kThreads) {
        const int b = b0 + tid, nb = min(kThreads, g.B - b0);
        Stream s{};
        if (b < g.B)
            s = ask(g, b);
        int64_t total;
        const int64_t upto = run + block_scan(s.need, sums, &total);
        run += total;
        if (s.need > 0 && upto > free0) {
            s.bad = true;
            s.need = 0;
        }
        block_scan(s.need, sums, &total);
        taken += total;
        s_len[tid] = s.len;
        s_fresh[tid] = s.bad ? 0 : s.fresh;
        s_held[tid] = s.held;
        s_need[tid] = s.need;
        s_top[tid] = free0 - 1 - (upto - s.need);
        if (rank == 0 && b < g.B && s.bad && g.bad_count)
            atomicAdd(g.bad_count, 1);
        __syncthreads();
        // New pages: a warp per stream.
        for (int i = rank * 32 + (tid >> 5); i < nb; i += C * 32)
            for (int j = tid & 31; j < s_need[i]; j += 32)
                g.table[(b0 + i) * g.table_row + s_held[i] + j] = g.pages[s_top[i] - j];
        // Slots.
        const uint32_t items = (uint32_t)nb * (uint32_t)g.N;
        for (uint32_t e = rank * kThreads + tid; e < items; e += C * kThreads) {
            const int i = (int)g.n_div.div(e), n = (int)(e - i * g.n_div.d);
            int64_t slot = -1;
            if (n < s_fresh[i]) {
                const uint32_t at = (uint32_t)(s_len[i] + n), p = g.page.div(at);
                const int j = (int)p - s_held[i];
                const int64_t page = j < 0 ? g.table[(b0 + i) * g.table_row + p] : g.pages[s_top[i] - j];
                slot = page * g.page.d + (at - p * g.page.d);
                slot = page < 0 || slot > 0x7FFFFFFF ? -1 : slot;
            }
            g.slots[(int64_t)b0 * g.N + e] = (int)slot;
        }
        if (g.B > kThreads)
            __syncthreads(); // (the streams' numbers are overwritten)
    }
    if (C > 1)
        cluster_sync(); // every CTA has read the counts
    else
        __syncthreads();
    if (rank != 0)
        return;
    run = 0;
    for (int b0 = 0; b0 < g.B; b0 += kThreads) {
        const int b = b0 + tid;
        Stream s{};
        if (b < g.B)
            s = ask(g, b);
        int64_t total;
        const int64_t upto = run + block_scan(s.need, sums, &total);
        run += total;
        if (b < g.B)
            g.held_out[b] = s.held + (upto > free0 ? 0 : s.need);
    }
    if (tid == 0)
        *g.free_out = (int)(free0 - taken);
}

// One CTA.
__global__ void __launch_bounds__(kThreads) release_kernel(const TablesArgs g)
{
    __shared__ int64_t sums[32];
    __shared__ int s_keep[kThreads], s_back[kThreads];
    __shared__ int64_t s_top[kThreads];
    const int tid = threadIdx.x;
    const int free0 = min(max(*g.free_count, 0), g.F);
    auto back_of = [&](int b, int &held) { // pages of stream b that go back
        held = min(max(g.held[b], 0), g.M);
        const int64_t len = min((int64_t)max(g.lens[b], 0), (int64_t)g.M * g.page.d);
        return max(0, held - pages_of(g, len));
    };
    int64_t all = 0;
    for (int b0 = 0; b0 < g.B; b0 += kThreads) {
        int held;
        int64_t total;
        block_scan(b0 + tid < g.B ? back_of(b0 + tid, held) : 0, sums, &total);
        all += total;
    }
    const bool fits = all <= g.F - free0;
    int64_t run = 0;
    for (int b0 = 0; b0 < g.B; b0 += kThreads) {
        const int b = b0 + tid, nb = min(kThreads, g.B - b0);
        int held = 0;
        const int back = b < g.B && fits ? back_of(b, held) : 0;
        int64_t total;
        const int64_t upto = run + block_scan(back, sums, &total);
        run += total;
        s_keep[tid] = held - back;
        s_back[tid] = back;
        s_top[tid] = free0 + all - 1 - (upto - back);
        if (b < g.B)
            g.held_out[b] = fits ? held - back : min(max(g.held[b], 0), g.M);
        __syncthreads();
        for (int i = tid >> 5; i < nb; i += 32)
            for (int j = tid & 31; j < s_back[i]; j += 32) {
                int32_t *entry = g.table + (b0 + i) * g.table_row + s_keep[i] + j;
                g.pages_out[s_top[i] - j] = *entry;
                *entry = -1;
            }
        __syncthreads();
    }
    if (tid == 0) {
        *g.free_out = (int)(free0 + run);
        if (!fits && g.bad_count)
            atomicAdd(g.bad_count, 1);
    }
}

// ---------------------------------------------------------------------------
// Writing.
// ---------------------------------------------------------------------------
constexpr int kWriteThreads = 256;
constexpr int kWritePer = 4; // 16-byte pieces of a token per thread

struct WriteArgs {
    HeadsView k, v;
    PagesView kp, vp;
    const int32_t *slots;
    int32_t *bad_count;
    int64_t slots_all;
    int units, lanes; // pieces of a token's keys or values; threads for them
    uint32_t items;   // of the launch
    uint32_t n0;
    FastDiv lanes_div, n_div, chunks, page;
};

__global__ void __launch_bounds__(kWriteThreads) write_kernel(const WriteArgs g)
{
    const uint32_t item = blockIdx.x * kWriteThreads + threadIdx.x;
    if (item >= g.items)
        return;
    const uint32_t row = g.lanes_div.div(item), lane = item - row * g.lanes_div.d, token = g.n0 + (row >> 1);
    const bool is_v = row & 1;
    const int64_t slot = g.slots[token];
    if (slot < 0 || slot >= g.slots_all) {
        if (slot >= 0 && !is_v && lane == 0 && g.bad_count)
            atomicAdd(g.bad_count, 1);
        return;
    }
    const uint32_t b = g.n_div.div(token), n = token - b * g.n_div.d, p = g.page.div((uint32_t)slot);
    const HeadsView &src = is_v ? g.v : g.k;
    const PagesView &dst = is_v ? g.vp : g.kp;
    const __nv_bfloat16 *from = src.row(b, n, 0);
    __nv_bfloat16 *to = dst.row(p, (int64_t)slot - (int64_t)p * g.page.d, 0);
    uint4 x[kWritePer];
    int64_t at[kWritePer];
#pragma unroll
    for (int i = 0; i < kWritePer; ++i) {
        const uint32_t u = lane + i * g.lanes;
        if (u < (uint32_t)g.units) {
            const uint32_t h = g.chunks.div(u), d = 8 * (u - h * g.chunks.d);
            x[i] = *reinterpret_cast<const uint4 *>(from + h * src.h + d);
            at[i] = h * dst.h + d;
        }
    }
#pragma unroll
    for (int i = 0; i < kWritePer; ++i)
        if (lane + i * g.lanes < (uint32_t)g.units)
            *reinterpret_cast<uint4 *>(to + at[i]) = x[i];
}

constexpr int64_t kIntMax = ((int64_t)1 << 31) - 1;

bool tables_ok(int64_t B, int64_t N, int64_t M, int64_t F, int64_t page_size, int64_t table_row)
{
    int64_t p;
    return B >= 0 && B <= 65535 && N >= 0 && M >= 0 && F >= 0 && F <= kIntMax && page_size >= 1 &&
           page_size <= kIntMax && N <= kIntMax && M <= kIntMax && prod_ok({M, page_size}, &p) && p <= kIntMax &&
           prod_ok({B, N}, &p) && p <= kIntMax && prod_ok({B, M}, &p) && p <= kIntMax &&
           (B <= 1 || (table_row >= M && table_row < ((int64_t)1 << 38) / B));
}

int64_t table_bytes(int64_t B, int64_t M, int64_t table_row) { return B > 0 ? 4 * ((B - 1) * table_row + M) : 0; }

// Whether any of the arrays that are written meets another one (an in-place pair is passed once).
struct Range {
    const void *p;
    int64_t bytes;
    bool written;
};
bool any_meet(std::initializer_list<Range> ranges)
{
    for (const Range &a : ranges)
        for (const Range &b : ranges)
            if (&a != &b && a.written && a.p && b.p && a.bytes > 0 && b.bytes > 0 && overlaps(a.p, a.bytes, b.p, b.bytes))
                return true;
    return false;
}

} // namespace
} // namespace tok

extern "C" tok_status tok_page_tables(const int32_t *lens, const int32_t *fresh, const int32_t *held,
                                      const int32_t *free_count, const int32_t *pages, int32_t *table,
                                      int32_t *slots, int32_t *held_out, int32_t *free_out, int32_t *bad_count,
                                      int64_t B, int64_t N, int64_t M, int64_t F, int64_t page_size,
                                      int64_t table_row, cudaStream_t stream)
{
    using namespace tok;
    if (!tables_ok(B, N, M, F, page_size, table_row))
        return TOK_ERR_SHAPE;
    if (B == 0 && (!free_count || !free_out))
        return TOK_OK;
    if (!free_count || !free_out ||
        (B > 0 && (!lens || !held || !held_out || (F > 0 && !pages) || (M > 0 && !table) || (N > 0 && !slots))))
        return TOK_ERR_NULL;
    for (const void *p : {(const void *)lens, (const void *)fresh, (const void *)held, (const void *)free_count,
                          (const void *)pages, (const void *)table, (const void *)slots, (const void *)held_out,
                          (const void *)free_out, (const void *)bad_count})
        if (!aligned(p, 4))
            return TOK_ERR_ALIGN;
    if (any_meet({{lens, 4 * B, false}, {fresh, 4 * B, false}, {held == held_out ? nullptr : held, 4 * B, false},
                  {free_count == free_out ? nullptr : free_count, 4, false}, {pages, 4 * F, false},
                  {table, table_bytes(B, M, table_row), true}, {slots, 4 * B * N, true}, {held_out, 4 * B, true},
                  {free_out, 4, true}, {bad_count, 4, true}}))
        return TOK_ERR_ALIAS;
    TablesArgs g{};
    g.lens = lens;
    g.fresh = fresh;
    g.held = held;
    g.free_count = free_count;
    g.pages = pages;
    g.table = table;
    g.slots = slots;
    g.held_out = held_out;
    g.free_out = free_out;
    g.bad_count = bad_count;
    g.B = (int)B;
    g.N = (int)N;
    g.M = (int)M;
    g.F = (int)F;
    g.table_row = table_row;
    g.page = FastDiv((uint32_t)page_size);
    g.n_div = FastDiv((uint32_t)std::max<int64_t>(N, 1));
    int C = 1;
    while (C < kMaxCluster && B * N > (int64_t)C * kThreads)
        C *= 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)C);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)C;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, tables_kernel, g, C);
    if (e != cudaSuccess) {
        record_cuda_error(e);
        cudaGetLastError();
        return TOK_ERR_CUDA;
    }
    return launch_status();
}

extern "C" tok_status tok_page_release(const int32_t *lens, const int32_t *held, const int32_t *free_count,
                                       int32_t *pages, int32_t *table, int32_t *held_out, int32_t *free_out,
                                       int32_t *bad_count, int64_t B, int64_t M, int64_t F, int64_t page_size,
                                       int64_t table_row, cudaStream_t stream)
{
    using namespace tok;
    if (!tables_ok(B, 0, M, F, page_size, table_row))
        return TOK_ERR_SHAPE;
    if (B == 0 && (!free_count || !free_out))
        return TOK_OK;
    if (!free_count || !free_out ||
        (B > 0 && (!lens || !held || !held_out || (F > 0 && !pages) || (M > 0 && !table))))
        return TOK_ERR_NULL;
    for (const void *p : {(const void *)lens, (const void *)held, (const void *)free_count, (const void *)pages,
                          (const void *)table, (const void *)held_out, (const void *)free_out,
                          (const void *)bad_count})
        if (!aligned(p, 4))
            return TOK_ERR_ALIGN;
    if (any_meet({{lens, 4 * B, false}, {held == held_out ? nullptr : held, 4 * B, false},
                  {free_count == free_out ? nullptr : free_count, 4, false}, {pages, 4 * F, true},
                  {table, table_bytes(B, M, table_row), true}, {held_out, 4 * B, true}, {free_out, 4, true},
                  {bad_count, 4, true}}))
        return TOK_ERR_ALIAS;
    TablesArgs g{};
    g.lens = lens;
    g.held = held;
    g.free_count = free_count;
    g.pages_out = pages;
    g.table = table;
    g.held_out = held_out;
    g.free_out = free_out;
    g.bad_count = bad_count;
    g.B = (int)B;
    g.M = (int)M;
    g.F = (int)F;
    g.table_row = table_row;
    g.page = FastDiv((uint32_t)page_size);
    release_kernel<<<1, kThreads, 0, stream>>>(g);
    return launch_status();
}

extern "C" tok_status tok_paged_write(const tok_heads *k, const tok_heads *v, const int32_t *slots,
                                      const tok_pages *k_pages, const tok_pages *v_pages, int32_t *bad_count,
                                      int64_t B, int64_t N, int64_t H, int64_t D, int64_t P, int64_t page_size,
                                      cudaStream_t stream)
{
    using namespace tok;
    int64_t tokens, all;
    if (B < 0 || B > 65535 || N < 0 || H < 1 || H > 65535 || D < 8 || D > 128 || D % 8 || P < 0 || page_size < 1 ||
        !prod_ok({B, N}, &tokens) || tokens > kIntMax || !prod_ok({P, page_size}, &all) || all > kIntMax ||
        page_size > kIntMax)
        return TOK_ERR_SHAPE;
    if (tokens == 0)
        return TOK_OK;
    if (!k || !v || !k_pages || !v_pages || !k->ptr || !v->ptr || !slots || (P > 0 && (!k_pages->ptr || !v_pages->ptr)))
        return TOK_ERR_NULL;
    const View vk{k, B, N, H, D, true}, vv{v, B, N, H, D, true};
    const PoolView pk{k_pages, P, page_size, H, D}, pv{v_pages, P, page_size, H, D};
    for (const View &x : {vk, vv})
        if (!x.strides_ok())
            return TOK_ERR_SHAPE;
    for (const PoolView &x : {pk, pv})
        if (!x.strides_ok() || (P > 0 && !x.distinct()))
            return TOK_ERR_SHAPE;
    for (const View &x : {vk, vv})
        if (!x.aligned16())
            return TOK_ERR_ALIGN;
    for (const PoolView &x : {pk, pv})
        if (P > 0 && !x.aligned16())
            return TOK_ERR_ALIGN;
    if (!aligned(slots, 4) || !aligned(bad_count, 4))
        return TOK_ERR_ALIGN;
    if (P > 0) {
        if (pools_meet(pk, pv))
            return TOK_ERR_ALIAS;
        for (const PoolView &x : {pk, pv})
            if (x.meets(k->ptr, vk.span() * 2) || x.meets(v->ptr, vv.span() * 2) || x.meets(slots, 4 * tokens) ||
                x.meets(bad_count, 4))
                return TOK_ERR_ALIAS;
    }
    if (bad_count && (overlaps(bad_count, 4, k->ptr, vk.span() * 2) || overlaps(bad_count, 4, v->ptr, vv.span() * 2) ||
                      overlaps(bad_count, 4, slots, 4 * tokens)))
        return TOK_ERR_ALIAS;
    WriteArgs g{};
    g.k = view(k);
    g.v = view(v);
    g.kp = view(k_pages);
    g.vp = view(v_pages);
    g.slots = slots;
    g.bad_count = bad_count;
    g.slots_all = all;
    g.units = (int)(H * (D / 8));
    g.lanes = (g.units + kWritePer - 1) / kWritePer;
    g.lanes_div = FastDiv((uint32_t)g.lanes);
    g.n_div = FastDiv((uint32_t)N);
    g.chunks = FastDiv((uint32_t)(D / 8));
    g.page = FastDiv((uint32_t)page_size);
    const int64_t most = kIntMax / (2 * (int64_t)g.lanes); // tokens of a launch (items are 32-bit)
    tok_status st = TOK_OK;
    for (int64_t n0 = 0; n0 < tokens && st == TOK_OK; n0 += most) {
        g.n0 = (uint32_t)n0;
        g.items = (uint32_t)(std::min(most, tokens - n0) * 2 * g.lanes);
        write_kernel<<<(g.items + kWriteThreads - 1) / kWriteThreads, kWriteThreads, 0, stream>>>(g);
        st = launch_status();
    }
    return st;
}
