// Drawing codes from a model's logits: temperature, top-k, top-p and min-p filters, then
// one draw per row by a given number in [0, 1).
//
// With x the row, m its largest value and T the temperature, token i has the weight
// e_i = exp((x_i - m) / T).  The filters keep, in this order: the top_k largest tokens;
// of those, by falling weight, each one before which less than top_p of their weight lies
// (the largest always); of those, the ones with e_i >= min_p.  Equal logits rank by index.
// The drawn code is the first, in index order, at which the running sum of the kept weights
// exceeds u times their total.
//
// 64,000 borders lie in [0, 1), so sums in 32 bits would put draws on the wrong side of
// one: exponentials are taken in 64 bits and held as integers of 2^-44 (a weight below
// 2^-45 of the largest is zero; 2^18 weights sum to at most 2^62).  Integer sums do not
// depend on their order, so neither the split over threads and CTAs nor the order of
// the histogram's atomics shows in the result.
//
// The kernel is bound by latency: the chain of short steps of a row between barriers, at 40% of an SM's
// warps (1.6 to 2.1 instructions a cycle of 4; HBM and the issue slots are half idle or more).  So
// rows are streamed (re-reads come from L2), several to an SM, in few and short passes:
//   top_k up to kSmall: a histogram of a sample gives a value that a little more than top_k
//     tokens should reach; one pass picks these out (their count says whether they hold the top_k),
//     and the rest is done on the picked tokens by one CTA, which sorts up to kCap outright.
//   top_p without top_k: a histogram of weights relative to their bin's own (32-bit integers)
//     says in which bin the limit lies; one pass then sums the exact weights above that bin
//     and in all, and picks out the bin's tokens; sorted, they give the limit's token.  The
//     exact sums say whether the bin was the right one.
//   everything else, and what these two do not settle: a histogram of counts and exact weights
//     over 1024 bins of x, then the tokens of the limit's bin, sorted; a bin with more than
//     kCap tokens is narrowed on the bits of x, to a single value if need be, whose ties
//     are counted in index order.
// With few rows a cluster of up to 8 CTAs shares one, a contiguous slice each.
// Measured, rows of 64,000: 4 with all filters 17 us; 255 in fp32 under top_p 0.9 76 us (65 MB: 10 us
// of HBM); 880 in bf16 under top_k 500 63 us (17 us of HBM).  Sorting every picked token outright
// instead of the limit's bin only: 19 and 86 us for the first and the last.
#include <algorithm>

#include "tma.cuh"
#include "tok_common.cuh"
#include "tok_internal.h"
#include "umma.cuh"

namespace tok {
namespace {

// (a lambda that is not inlined keeps everything it captures in local memory)
#define TOK_INLINE __attribute__((always_inline))

constexpr int kMaxWarps = 16;
constexpr int kBins = 1024;
constexpr int kCap = 512;                            // tokens sorted outright
constexpr int kList = 2048;                          // picked tokens
constexpr int kSmall = 1024;                         // largest top_k that picks
constexpr int kMaxCluster = 8;
constexpr int64_t kMaxV = 1 << 18;
constexpr double kOne = 17592186044416.0; // 2^44
constexpr uint64_t kBias = 0x4330000000000000ull; // the bits of 2^52
constexpr float kReach = 31.25f;          // exp(-31.25) 2^44 < 1/2: no weight beyond
constexpr float kLowest = -3.402823466e+38f; // tokens that are not at least this (-inf, NaN) do not count

struct SampleArgs {
    const void *logits;
    const float *u;
    const float *temperature, *top_p, *min_p; // per row, or null: the values below
    const int32_t *top_k;
    float temperature_all, top_p_all, min_p_all;
    int32_t top_k_all;
    int32_t *idx;
    float *logprob; // or null
    int64_t row_stride;
    int V, slice;  // tokens per CTA
    int bucket;    // log2 of the tokens per index bucket: at most 1024 buckets
};

// Order-preserving bits of a float (no NaN); -0 counts as 0.
__device__ __forceinline__ uint32_t order_key(float x)
{
    const uint32_t b = __float_as_uint(x + 0.0f);
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// Loads from another CTA's shared memory.
__device__ __forceinline__ uint32_t ld_cluster(uint32_t addr, uint32_t rank)
{
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(addr, rank)) : "memory");
    return v;
}
__device__ __forceinline__ uint64_t ld_cluster64(uint32_t addr, uint32_t rank)
{
    uint64_t v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(mapa_shared(addr, rank)) : "memory");
    return v;
}

struct Shared {
    double table[64]; // 2^44 2^(j / 64)
    uint64_t warp64[kMaxWarps], range[kMaxWarps], cap[kCap], sorted[kCap], cap_w[kCap];
    uint64_t pub64[2]; // this CTA's weight sums, or best token
    uint64_t found_before, found_mass, mass;
    uint32_t cnt[kBins], lo[kBins], hi[kBins]; // histogram: tokens, weight in two words
    float list_x[kList];
    int list_idx[kList];
    uint32_t rank[kCap];
    int owner[kCap];
    uint32_t warp32[2][kMaxWarps];
    uint32_t pub[4]; // this CTA's: largest and smallest key, tokens picked, ties
    uint32_t found_bin, found_cnt, res_idx;
};

// 16 bytes are N tokens.
template <typename T> struct Vec;
template <> struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ float one(const float *p) { return __ldg(p); }
    static __device__ __forceinline__ float largest(const uint4 &v) // NaN gives way to numbers
    {
        return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
    }
    static __device__ __forceinline__ void split(const uint4 &v, float (&f)[4])
    {
        f[0] = __uint_as_float(v.x);
        f[1] = __uint_as_float(v.y);
        f[2] = __uint_as_float(v.z);
        f[3] = __uint_as_float(v.w);
    }
    static __device__ __forceinline__ float threshold(float least) { return least; }
    static __device__ __forceinline__ uint32_t at_least(const uint4 &v, float t) // bit k: token k >= t
    {
        return (uint32_t)(__uint_as_float(v.x) >= t) | (uint32_t)(__uint_as_float(v.y) >= t) << 1 |
               (uint32_t)(__uint_as_float(v.z) >= t) << 2 | (uint32_t)(__uint_as_float(v.w) >= t) << 3;
    }
};
template <> struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ float one(const __nv_bfloat16 *p)
    {
        return bf16_lo(__ldg(reinterpret_cast<const unsigned short *>(p)));
    }
    static __device__ __forceinline__ float largest(const uint4 &v)
    {
        const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&v);
        const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
        return fmaxf(__low2float(m), __high2float(m));
    }
    static __device__ __forceinline__ void split(const uint4 &v, float (&f)[8])
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            f[2 * k] = bf16_lo(w[k]);
            f[2 * k + 1] = bf16_hi(w[k]);
        }
    }
    static __device__ __forceinline__ __nv_bfloat162 threshold(float least) // the bf16 numbers >= least are those >= it
    {
        return __bfloat162bfloat162(__float2bfloat16_ru(least));
    }
    static __device__ __forceinline__ uint32_t at_least(const uint4 &v, __nv_bfloat162 t)
    {
        const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&v);
        const uint32_t m = (__hge2_mask(h[0], t) & 0x00010001u) | (__hge2_mask(h[1], t) & 0x00040004u) |
                           (__hge2_mask(h[2], t) & 0x00100010u) | (__hge2_mask(h[3], t) & 0x00400040u);
        return (m | m >> 15) & 0xFFu;
    }
};

// Inclusive scan over the block's threads; *total gets the sum.  All threads.
template <int kWarps>
__device__ __forceinline__ uint64_t warps_scan(uint64_t v, uint64_t *warp, uint64_t *total)
{
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    __syncthreads(); // `warp` may still be read from an earlier use
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t x = __shfl_up_sync(~0u, v, o);
        if (lane >= o)
            v += x;
    }
    if (lane == 31)
        warp[w] = v;
    __syncthreads();
    uint64_t before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        const uint64_t x = warp[i];
        before += i < w ? x : 0;
        all += x;
    }
    *total = all;
    return v + before;
}

template <typename T, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) sample_kernel(const SampleArgs g, int C)
{
    constexpr int N = Vec<T>::N, kWarps = kThreads / 32, kPer = kBins / kThreads; // bins per thread
    __shared__ Shared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = C > 1 ? cluster_rank() : 0;
    const int64_t row = blockIdx.x / C;
    // This CTA's tokens [begin, begin + n): `head` of them up to a 16-byte boundary, nv vectors, the
    // rest.  Each warp has a contiguous range of the vectors; the first one the head, the last the rest.
    const int begin = min(g.V, (int)rank * g.slice), n = min(g.slice, g.V - begin);
    const T *src = static_cast<const T *>(g.logits) + row * g.row_stride + begin;
    const int head = min(n, (int)((16 - ((uintptr_t)src & 15)) & 15) / (int)sizeof(T)), nv = (n - head) / N;
    const uint4 *vec = reinterpret_cast<const uint4 *>(src + head);
    const int per_warp = (nv + kWarps - 1) / kWarps, v0 = min(nv, warp * per_warp), v1 = min(nv, v0 + per_warp);
    const int odd0 = warp == 0 ? 0 : warp == kWarps - 1 ? head + nv * N : n; // of the head or the rest
    const int odd1 = warp == 0 ? head : n;

    float T1 = g.temperature ? g.temperature[row] : g.temperature_all;
    const float top_p = g.top_p ? g.top_p[row] : g.top_p_all;
    float min_p = g.min_p ? g.min_p[row] : g.min_p_all;
    min_p = min_p > 0.0f ? fminf(min_p, 1.0f) : 0.0f;
    int top_k = g.top_k ? g.top_k[row] : g.top_k_all;
    if (!(T1 > 0.0f) || top_p <= 0.0f) { // greedy; or the nucleus is the largest token alone
        top_k = 1;
        T1 = T1 > 0.0f ? T1 : 1.0f;
    }
    T1 = fminf(T1, 3.4e38f); // (an infinite one would turn infinite differences into NaN)
    const bool by_p = top_p < 1.0f && top_k != 1;
    bool by_k = top_k > 1 && top_k < g.V;

    // The set that ranks are taken in: the row over C CTAs, or the picked tokens in the first.
    int members = C, listed = -1; // listed >= 0: number of picked tokens
    float floor_x = kLowest;      // tokens that are not at least this do not count
    auto barrier = [&]() TOK_INLINE {
        if (members > 1)
            cluster_sync();
        else
            __syncthreads();
    };
    auto remote = [&](const void *p, int c) TOK_INLINE -> uint32_t {
        return members > 1 ? ld_cluster(smem_addr(p), c) : *static_cast<const uint32_t *>(p);
    };
    auto remote64 = [&](const void *p, int c) TOK_INLINE -> uint64_t {
        return members > 1 ? ld_cluster64(smem_addr(p), c) : *static_cast<const uint64_t *>(p);
    };
    auto leave = [&]() TOK_INLINE { // no CTA leaves while another reads its shared memory
        if (members > 1)
            cluster_sync();
    };
    auto value = [](uint32_t key) TOK_INLINE { return __uint_as_float((key & 0x80000000u) ? key & 0x7FFFFFFFu : ~key); };
    // A token's place in the order of ranks: falling value, then rising index.
    auto place_of = [](uint32_t key, int idx) TOK_INLINE -> uint64_t { return ((uint64_t)key << 32) | (uint32_t)~idx; };
    auto nothing = [&]() TOK_INLINE { // no token to draw from
        if (rank == 0 && tid == 0) {
            g.idx[row] = -1;
            if (g.logprob)
                g.logprob[row] = -INFINITY;
        }
    };
    // f(vectors, first indices, how many of them this lane has) for batches of 4 x 32 vectors, every
    // step-th 32 of each warp's, all loads of a batch in flight at once, all lanes of the warp together;
    // f1(value, index) for the odd tokens.
    constexpr int kBatch = 4;
    auto batches = [&](int step, auto &&f, auto &&f1) TOK_INLINE {
        for (int c0 = v0; c0 < v1; c0 += 32 * step * kBatch) {
            uint4 v[kBatch];
            int idx[kBatch], has = 0;
#pragma unroll
            for (int e = 0; e < kBatch; ++e) {
                const int c = c0 + lane + 32 * step * e;
                idx[e] = begin + head + c * N;
                if (c < v1) {
                    v[e] = __ldg(vec + c);
                    has = e + 1;
                }
            }
            f(v, idx, has);
        }
        for (int i = odd0 + lane; i < odd1; i += 32)
            f1(Vec<T>::one(src + i), begin + i);
    };
    auto vectors = [&](int step, auto &&f, auto &&f1) TOK_INLINE { // f(vector, first index)
        batches(
            step,
            [&](const uint4 (&v)[kBatch], const int (&idx)[kBatch], int has) {
#pragma unroll
                for (int e = 0; e < kBatch; ++e)
                    if (e < has)
                        f(v[e], idx[e]);
            },
            f1);
    };
    auto tokens = [&](auto &&f) TOK_INLINE { // f(value, index) for the tokens of this CTA's set that count
        if (listed >= 0) {
            for (int i = tid; i < listed; i += kThreads)
                if (sh.list_x[i] >= floor_x)
                    f(sh.list_x[i], sh.list_idx[i]);
        } else
            vectors(
                1,
                [&](const uint4 &v, int idx) {
                    float x[N];
                    Vec<T>::split(v, x);
#pragma unroll
                    for (int k = 0; k < N; ++k)
                        if (x[k] >= floor_x)
                            f(x[k], idx + k);
                },
                [&](float x, int idx) {
                    if (x >= floor_x)
                        f(x, idx);
                });
    };

    // ---- One token: the first of the largest. ----
    if (top_k == 1) {
        float best = -INFINITY;
        int at = 0x7FFFFFFF;
        auto take = [&](float x, int idx) TOK_INLINE { // indices rise within a thread but for the head, which is warp 0's last
            if (x > best || (x == best && idx < at)) {
                best = x;
                at = idx;
            }
        };
        vectors(
            1,
            [&](const uint4 &v, int idx) {
                if (Vec<T>::largest(v) >= best) {
                    float x[N];
                    Vec<T>::split(v, x);
#pragma unroll
                    for (int k = 0; k < N; ++k)
                        take(x[k], idx + k);
                }
            },
            take);
        uint64_t top = best > -INFINITY ? place_of(order_key(best), at) : 0ull;
#pragma unroll
        for (int o = 16; o; o >>= 1)
            top = max(top, __shfl_xor_sync(~0u, top, o));
        if (lane == 0)
            sh.warp64[warp] = top;
        __syncthreads();
        if (tid == 0) {
            for (int w = 0; w < kWarps; ++w)
                top = max(top, sh.warp64[w]);
            sh.pub64[0] = top;
        }
        barrier();
        if (rank == 0 && tid == 0) {
            for (int c = 0; c < C; ++c)
                top = max(top, remote64(&sh.pub64[0], c));
            if (top) {
                g.idx[row] = (int)~(uint32_t)top;
                if (g.logprob)
                    g.logprob[row] = 0.0f;
            } else
                nothing();
        }
        leave();
        return;
    }

    // Largest and lowest of all threads' (and, over the cluster, all members') values.
    auto extremes = [&](float &hi, float &lo) TOK_INLINE {
        uint32_t kmax = __reduce_max_sync(~0u, order_key(hi)), kmin = __reduce_min_sync(~0u, order_key(lo));
        __syncthreads();
        if (lane == 0) {
            sh.warp32[0][warp] = kmax;
            sh.warp32[1][warp] = kmin;
        }
        __syncthreads();
        kmax = __reduce_max_sync(~0u, sh.warp32[0][lane % kWarps]);
        kmin = __reduce_min_sync(~0u, sh.warp32[1][lane % kWarps]);
        if (members > 1) {
            if (tid == 0) {
                sh.pub[0] = kmax;
                sh.pub[1] = kmin;
            }
            cluster_sync();
            for (int c = 0; c < C; ++c) {
                kmax = max(kmax, ld_cluster(smem_addr(&sh.pub[0]), c));
                kmin = min(kmin, ld_cluster(smem_addr(&sh.pub[1]), c));
            }
        }
        hi = value(kmax);
        lo = value(kmin);
    };
    // Bins of equal width downwards from `top`, the highest in bin 0.  Rounding to nearest: any
    // monotone rule serves, and this one needs no conversion.
    float bin_top = 0.0f, per_bin = 0.0f;
    const float reach = kReach * T1;
    auto set_bins = [&](float top, float low) TOK_INLINE { // no further than weights reach
        const float span = fminf(reach, top - low);
        bin_top = top;
        per_bin = span > 0.0f ? fminf((float)(kBins - 1) / span, 3.4e38f) : 0.0f;
    };
    auto bin_of = [&](float x) TOK_INLINE -> int {
        const float d = fminf((bin_top - x) * per_bin, (float)(kBins - 1));
        return (int)(__float_as_uint(d + 8388608.0f) & 0x7FFFFFu);
    };
    auto clear_bins = [&]() TOK_INLINE {
        for (int i = tid; i < kBins; i += kThreads)
            sh.cnt[i] = sh.lo[i] = sh.hi[i] = 0;
        __syncthreads();
    };
    // All members' counts of bins kPer tid + e.
    auto merged_counts = [&](const uint32_t *bins, uint64_t (&out)[kPer]) TOK_INLINE {
#pragma unroll
        for (int e = 0; e < kPer; ++e)
            out[e] = 0;
#pragma unroll 4
        for (int c = 0; c < members; ++c)
#pragma unroll
            for (int e = 0; e < kPer; e += 2) {
                const uint64_t x = remote64(&bins[kPer * tid + e], c);
                out[e] += (uint32_t)x;
                out[e + 1] += x >> 32;
            }
    };
    // The bin of this thread's (c_at, w_at lie before them) in which the limit lies publishes itself: the
    // `want`-th token, or the last before which less than `limit` lies.
    auto publish = [&](bool count, uint64_t want, double limit, uint64_t c_at, uint64_t w_at,
                       const uint64_t (&c)[kPer], const uint64_t (&w)[kPer]) TOK_INLINE {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            if (count ? c_at < want && c_at + c[e] >= want : (double)w_at < limit && (double)(w_at + w[e]) >= limit) {
                sh.found_bin = (uint32_t)(kPer * tid + e);
                sh.found_cnt = (uint32_t)c[e];
                sh.found_before = c_at;
                sh.found_mass = w_at;
            }
            c_at += c[e];
            w_at += w[e];
        }
        __syncthreads();
    };
    auto sum_of = [](const uint64_t (&x)[kPer]) TOK_INLINE {
        uint64_t s = 0;
#pragma unroll
        for (int e = 0; e < kPer; ++e)
            s += x[e];
        return s;
    };
    const uint64_t none[kPer] = {};

    // ---- Pick the tokens among which the top_k largest are. ----
    float xmax = -INFINITY, xlow = INFINITY;
    if (by_k && top_k <= kSmall) {
        const int step = g.slice / N >= 32 * 16 * kWarps ? 8 : 1; // (the same in all CTAs)
        vectors(
            step,
            [&](const uint4 &v, int) {
                float x[N];
                Vec<T>::split(v, x);
                xmax = fmaxf(xmax, Vec<T>::largest(v));
                xlow = fminf(xlow, x[0] >= kLowest ? x[0] : INFINITY);
            },
            [&](float x, int) { xmax = fmaxf(xmax, x); });
        extremes(xmax, xlow);
        xlow = fminf(xlow, xmax);
        if (xmax > -INFINITY && xmax < INFINITY) {
            set_bins(xmax, xlow);
            clear_bins();
            auto add = [&](float x, int) TOK_INLINE {
                if (x >= kLowest)
                    atomicAdd(&sh.cnt[bin_of(x)], 1u);
            };
            vectors(
                step,
                [&](const uint4 &v, int) {
                    float x[N];
                    Vec<T>::split(v, x);
#pragma unroll
                    for (int k = 0; k < N; ++k)
                        add(x[k], 0);
                },
                add);
            if (tid == 0) {
                sh.found_bin = kBins; // fewer tokens than that
                sh.pub[2] = 0;
            }
            barrier();
            uint64_t c[kPer], total;
            merged_counts(sh.cnt, c);
            const uint64_t at = warps_scan<kWarps>(sum_of(c), sh.warp64, &total) - sum_of(c);
            // Of a sample: 1.5 top_k + 128 tokens, four standard deviations from too few.
            publish(true, step > 1 ? (uint64_t)((3 * top_k / 2 + 128) / step) : (uint64_t)top_k, 0.0, at, 0, c, none);
            const int bin = (int)sh.found_bin;
            // The bin's lower edge (or a little below it: what counts is the count).
            const float least =
                bin >= kBins - 1 || per_bin == 0.0f ? kLowest : fmaxf(xmax - ((float)bin + 0.51f) / per_bin, kLowest);
            const auto threshold = Vec<T>::threshold(least);
            batches( // indices only: the values are read again
                1,
                [&](const uint4 (&v)[kBatch], const int (&idx)[kBatch], int has) {
                    uint32_t m = 0;
#pragma unroll
                    for (int e = 0; e < kBatch; ++e)
                        m |= e < has ? Vec<T>::at_least(v[e], threshold) << (N * e) : 0u;
                    const uint32_t own = __popc(m);
                    if (!__any_sync(~0u, own))
                        return;
                    uint32_t to = own;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const uint32_t x = __shfl_up_sync(~0u, to, o);
                        if (lane >= o)
                            to += x;
                    }
                    uint32_t base = 0;
                    if (lane == 31)
                        base = atomicAdd(&sh.pub[2], to);
                    to += __shfl_sync(~0u, base, 31) - own;
                    for (; m; m &= m - 1, ++to) {
                        const int b = __ffs(m) - 1;
                        if (to < (uint32_t)kList)
                            sh.list_idx[to] = idx[0] + b / N * (32 * N) + b % N;
                    }
                },
                [&](float x, int idx) {
                    if (x >= least) {
                        const uint32_t to = atomicAdd(&sh.pub[2], 1u);
                        if (to < (uint32_t)kList)
                            sh.list_idx[to] = idx;
                    }
                });
            barrier();
            int upto[kMaxCluster], all = 0; // tokens of the members, added up
#pragma unroll
            for (int m = 0; m < kMaxCluster; ++m) {
                all += m < C ? (int)remote(&sh.pub[2], m) : 0;
                upto[m] = all;
            }
            if (all <= kList && (all >= top_k || least == kLowest)) {
                if (rank == 0) { // the first CTA has them all
                    const T *whole = src - begin;
                    for (int i = tid; i < all; i += kThreads) {
                        int m = 0, at = i;
#pragma unroll
                        for (int c2 = 0; c2 < kMaxCluster - 1; ++c2)
                            if (i >= upto[c2]) {
                                m = c2 + 1;
                                at = i - upto[c2];
                            }
                        const int idx = (int)remote(&sh.list_idx[at], m);
                        if (m)
                            sh.list_idx[i] = idx;
                        sh.list_x[i] = Vec<T>::one(whole + idx);
                    }
                }
                leave();
                if (rank != 0)
                    return;
                __syncthreads();
                listed = all;
                members = 1;
                by_k = listed > top_k;
            } else
                barrier(); // pub is read by others until here
        } else
            barrier(); // (likewise: the extremes are published anew below)
    }

    // ---- The largest token; what weights are relative to. ----
    xmax = -INFINITY, xlow = INFINITY;
    if (listed >= 0)
        tokens([&](float x, int) {
            xmax = fmaxf(xmax, x);
            xlow = fminf(xlow, x);
        });
    else
        vectors(
            1,
            [&](const uint4 &v, int) {
                xmax = fmaxf(xmax, Vec<T>::largest(v));
                float x[N];
                Vec<T>::split(v, x);
                xlow = fminf(xlow, x[0] >= kLowest ? x[0] : INFINITY); // (one of a vector is sample enough)
            },
            [&](float x, int) { xmax = fmaxf(xmax, x); });
    extremes(xmax, xlow);
    xlow = fminf(xlow, xmax);
    if (xmax == -INFINITY) {
        nothing();
        leave();
        return;
    }
    const bool infinite = xmax == INFINITY; // only infinite logits count, with equal weights
    floor_x = infinite ? INFINITY : kLowest;
    if (tid < kWarps)
        sh.range[tid] = 0;
    if (tid < 64)
        sh.table[tid] = kOne * exp2((double)tid / 64.0);
    // 2^44 exp((x - xmax) / T1) in 64 bits: with y = 64 log2(e) (x - xmax) / T1 = k + f,
    // 2^(k / 64) from a table and the exponent, 2^(f / 64) by its Taylor polynomial of
    // degree 4 (|f ln 2 / 64| <= 0.0055: what is left out is below 2^-44.5 relative, beside the
    // half unit, 2^-45, of rounding to an integer).
    const double per_t = 64.0 / 0.6931471805599453 / (double)T1, xmax_d = infinite ? 0.0 : (double)xmax;
    const float xcut = infinite ? INFINITY : fmaxf(xmax - reach, kLowest); // no weight below
    auto weight_at = [&](double d) TOK_INLINE -> double { // of d = x - xmax
        constexpr double kMagic = 6755399441055744.0; // 1.5 2^52: a sum's low bits are its integer part
        constexpr double c1 = 0.6931471805599453 / 64, c2 = c1 * c1 / 2, c3 = c2 * c1 / 3, c4 = c3 * c1 / 4;
        const double kd = fma(d, per_t, kMagic), f = fma(d, per_t, kMagic - kd);
        const int k = __double2loint(kd);
        const double q = fma(fma(fma(c4, f, c3), f, c2), f, c1) * f, t = sh.table[k & 63];
        const double w = fma(t, q, t);
        return __hiloint2double(__double2hiint(w) + ((k >> 6) << 20), __double2loint(w));
    };
    auto weight_d = [&](float x) TOK_INLINE { return weight_at(infinite ? 0.0 : (double)x - xmax_d); }; // x >= xcut
    auto to_fixed = [](double w) TOK_INLINE -> uint64_t { // nearest integer of 0 <= w < 2^51
        return (uint64_t)__double_as_longlong(w + 4503599627370496.0) & 0xFFFFFFFFFFFFFull;
    };
    auto weight = [&](float x) TOK_INLINE -> uint64_t { return x >= xcut ? to_fixed(weight_d(x)) : 0ull; };
    const double floor_w = (double)min_p * kOne;
    set_bins(xmax, infinite ? xmax : xlow); // (infinite logits: all in one bin, whichever it is)
    clear_bins();

    // The `total` (at most kCap) tokens of sh.cap by falling place into sh.sorted, cap_w of the key beside
    // them if `w`.
    auto sort_cap = [&](int total, bool w) TOK_INLINE {
        for (int i = tid; i < total; i += kThreads)
            sh.rank[i] = 0;
        __syncthreads();
        const int groups = (total + 31) / 32, parts = groups ? max(1, kWarps / groups) : 0;
        for (int job = warp; job < groups * parts; job += kWarps) {
            const int i = job % groups * 32 + lane, part = job / groups, per = (total + parts - 1) / parts;
            const uint64_t me = i < total ? sh.cap[i] : 0;
            uint32_t r = 0;
            const int j1 = min(total, (part + 1) * per);
#pragma unroll 4
            for (int j = part * per; j < j1; ++j)
                r += sh.cap[j] > me;
            if (i < total)
                atomicAdd(&sh.rank[i], r);
        }
        __syncthreads();
        for (int i = tid; i < total; i += kThreads) {
            const uint64_t me = sh.cap[i];
            sh.sorted[sh.rank[i]] = me;
            if (w)
                sh.cap_w[sh.rank[i]] = weight(value((uint32_t)(me >> 32)));
        }
        __syncthreads();
    };
    // All members' sh.cap into each one's, in turn; returns their number (more than kCap: none moved).
    auto share_cap = [&]() TOK_INLINE -> int {
        barrier();
        if (members == 1) {
            const int m = (int)sh.pub[2];
            __syncthreads();
            return m;
        }
        constexpr int kEach = kCap / kThreads;
        uint64_t me[kEach] = {};
        int total = 0;
        for (int c = 0; c < members; ++c) {
            const int m = (int)remote(&sh.pub[2], c);
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                const int i = tid + e * kThreads;
                if (m <= kCap && i >= total && i < total + m)
                    me[e] = remote64(&sh.cap[i - total], c);
            }
            total += m;
        }
        barrier();
#pragma unroll
        for (int e = 0; e < kEach; ++e)
            if (total <= kCap && tid + e * kThreads < total)
                sh.cap[tid + e * kThreads] = me[e];
        __syncthreads();
        return total;
    };
    // Of the sorted tokens, the prefix that `keep(position, weight before it)` holds for: its length; the
    // weight through it goes to sh.mass, that of all to *all.
    auto prefix = [&](int total, bool w, auto &&keep, uint64_t *all) TOK_INLINE -> int {
        constexpr int kEach = kCap / kThreads;
        uint64_t x[kEach], s = 0;
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            x[e] = w && kEach * tid + e < total ? sh.cap_w[kEach * tid + e] : 0;
            s += x[e];
        }
        uint64_t at = w ? warps_scan<kWarps>(s, sh.warp64, all) - s : 0;
        const uint64_t start = at;
        int mine = 0;
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            mine += kEach * tid + e < total && keep(kEach * tid + e, at);
            at += x[e];
        }
        uint64_t kept;
        warps_scan<kWarps>((uint64_t)mine, sh.warp64, &kept);
        at = start;
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            at += x[e];
            if (kEach * tid + e + 1 == (int)kept)
                sh.mass = at;
        }
        __syncthreads();
        return (int)kept;
    };

    uint64_t cut = 0;  // the place of the last token kept
    uint64_t mine = 0; // kept weight of this thread's tokens
    bool have_mine = false, settled = !by_k && !by_p;

    // ---- top_p alone: the bin of the limit from relative weights, then one exact pass. ----
    if (!settled && !by_k && listed < 0 && !infinite && per_bin > 0.0f && xmax - reach >= kLowest) {
        const float h = 1.0f / (per_bin * T1); // a bin's width over T1: at most 0.031
        auto add = [&](float x, int) TOK_INLINE {
            const float d = fminf((bin_top - x) * per_bin, (float)(kBins - 1)), m = d + 8388608.0f;
            const float e = ((m - 8388608.0f) - d) * h; // weight relative to the bin's middle, in 2^-14
            const float r = fmaf(e, fmaf(e, 8192.0f, 16384.0f), 16384.0f);
            if (x >= xcut)
                atomicAdd(&sh.lo[__float_as_uint(m) & 0x7FFFFFu], __float_as_uint(r + 8388608.0f) & 0x7FFFFFu);
        };
        vectors(
            1,
            [&](const uint4 &v, int) {
                float x[N];
                Vec<T>::split(v, x);
#pragma unroll
                for (int k = 0; k < N; ++k)
                    add(x[k], 0);
            },
            add);
        barrier();
        uint64_t w[kPer], total;
        merged_counts(sh.lo, w);
#pragma unroll
        for (int e = 0; e < kPer; ++e) // 2^16 more for the small ones
            w[e] = (uint64_t)((double)w[e] * (65536.0 * exp(-(double)(kPer * tid + e) * (double)h)));
        const uint64_t at = warps_scan<kWarps>(sum_of(w), sh.warp64, &total) - sum_of(w);
        publish(false, 0, fmin((double)top_p * (double)total, (double)total), 0, at, none, w);
        const int bin = (int)sh.found_bin;
        const float above = bin == 0 ? INFINITY : xmax - ((float)bin - 0.52f) / per_bin;
        const float least = fmaxf(bin == kBins - 1 ? kLowest : xmax - ((float)bin + 0.52f) / per_bin, xcut);
        if (tid == 0)
            sh.pub[2] = 0;
        __syncthreads();
        // Sums of the bits of 2^52 + w: the number of terms times the bits of 2^52 is taken off at the end.
        // A token without a weight (-inf, NaN or below xcut, which is rounded and may be xmax) counts as 2^52 + 0.
        uint64_t sum_all = 0, sum_above = 0;
        uint32_t n_all = 0, n_above = 0, n_mine = 0;
        auto pick = [&](float x, int idx) TOK_INLINE {
            const uint32_t to = atomicAdd(&sh.pub[2], 1u);
            if (to < (uint32_t)kCap) {
                sh.cap[to] = place_of(order_key(x), idx);
                sh.owner[to] = warp;
            }
        };
        auto weigh = [&](float x0) TOK_INLINE -> bool { // whether the token is one of the bin's
            const float x = fmaxf(x0, xcut);
            const double wd = weight_at((double)x - xmax_d);
            const uint64_t bits = x0 >= xcut ? (uint64_t)__double_as_longlong(wd + 4503599627370496.0) : kBias;
            sum_all += bits;
            const bool in = x >= above;
            if (in) {
                sum_above += bits;
                ++n_above;
            }
            if (floor_w > 0.0) {
                mine += in && wd >= floor_w ? bits : 0ull;
                n_mine += in && wd >= floor_w;
            }
            return !in && x0 >= least;
        };
        vectors(
            1,
            [&](const uint4 &v, int idx) {
                float x[N];
                Vec<T>::split(v, x);
                uint32_t m = 0;
                n_all += N;
#pragma unroll
                for (int k = 0; k < N; ++k)
                    m |= (uint32_t)weigh(x[k]) << k;
                for (; m; m &= m - 1) {
                    const int k = __ffs(m) - 1;
                    pick(Vec<T>::one(src + (idx + k - begin)), idx + k);
                }
            },
            [&](float x, int idx) {
                ++n_all;
                if (weigh(x))
                    pick(x, idx);
            });
        sum_all -= n_all * kBias;
        sum_above -= n_above * kBias;
        mine = floor_w > 0.0 ? mine - n_mine * kBias : sum_above;
        uint64_t cta_all, cta_above, z = 0, before = 0;
        warps_scan<kWarps>(sum_all, sh.warp64, &cta_all);
        warps_scan<kWarps>(sum_above, sh.warp64, &cta_above);
        if (tid == 0) {
            sh.pub64[0] = cta_all;
            sh.pub64[1] = cta_above;
        }
        const int own = (int)sh.pub[2]; // (final since the scans' barriers)
        constexpr int kEach = kCap / kThreads;
        uint64_t own_place[kEach];
#pragma unroll
        for (int e = 0; e < kEach; ++e)
            own_place[e] = tid + e * kThreads < min(own, kCap) ? sh.cap[tid + e * kThreads] : 0;
        const int picked = share_cap();
        for (int c = 0; c < C; ++c) {
            z += remote64(&sh.pub64[0], c);
            before += remote64(&sh.pub64[1], c);
        }
        const double limit = (double)top_p * (double)z;
        if (!(limit < (double)z)) // every token
            settled = true;
        else if (picked <= kCap && picked > 0) {
            sort_cap(picked, true);
            uint64_t all;
            const int kept = prefix(
                picked, true, [&](int, uint64_t at2) { return (double)(before + at2) < limit; }, &all);
            if ((double)before < limit && (double)(before + all) >= limit) {
                cut = sh.sorted[kept - 1];
                // The picked tokens' kept weights, to the ranges of the warps that hold them.
#pragma unroll
                for (int e = 0; e < kEach; ++e)
                    if (own_place[e] && own_place[e] >= cut) {
                        const double wd = weight_d(value((uint32_t)(own_place[e] >> 32)));
                        if (wd >= floor_w)
                            atomicAdd(reinterpret_cast<unsigned long long *>(&sh.range[sh.owner[tid + e * kThreads]]),
                                      (unsigned long long)to_fixed(wd));
                    }
                settled = have_mine = true;
            }
        }
        barrier();
    }
    // ---- Few picked tokens: all of them sorted. ----
    if (!settled && listed >= 0 && listed <= kCap) {
        __syncthreads();
        for (int i = tid; i < listed; i += kThreads)
            sh.cap[i] = place_of(order_key(sh.list_x[i]), sh.list_idx[i]);
        __syncthreads();
        sort_cap(listed, by_p);
        int kept = min(listed, top_k);
        if (by_p) { // the weight of the top_k, then the tokens before which less than its share lies
            uint64_t all;
            prefix(
                listed, true, [&](int i, uint64_t) { return i < kept; }, &all);
            const uint64_t z = sh.mass;
            const double limit = (double)top_p * (double)z;
            __syncthreads();
            if (limit < (double)z)
                kept = min(kept, prefix(
                                     listed, true, [&](int, uint64_t at) { return (double)at < limit; }, &all));
        }
        cut = sh.sorted[kept - 1];
        settled = true;
    }
    if (!settled) {
        // Histogram of the tokens with klo <= key <= khi: by bin_of (shift < 0) or the key's bits.
        // Every CTA adds up all members' bins.
        auto histogram = [&](uint32_t klo, uint32_t khi, int shift, uint64_t (&c_out)[kPer], uint64_t (&w_out)[kPer]) TOK_INLINE {
            clear_bins();
            tokens([&](float x, int) {
                const uint32_t k = order_key(x);
                if (k < klo || k > khi)
                    return;
                const int b = shift < 0 ? bin_of(x) : (int)((khi - k) >> shift);
                atomicAdd(&sh.cnt[b], 1u);
                const uint64_t w = by_p ? weight(x) : 0ull;
                if (w) {
                    const uint32_t wl = (uint32_t)w, old = atomicAdd(&sh.lo[b], wl);
                    const uint32_t wh = (uint32_t)(w >> 32) + (old + wl < old ? 1u : 0u);
                    if (wh)
                        atomicAdd(&sh.hi[b], wh);
                }
            });
            barrier();
            merged_counts(sh.cnt, c_out);
#pragma unroll
            for (int e = 0; e < kPer; ++e)
                w_out[e] = 0;
            if (by_p) {
                uint64_t h[kPer];
                merged_counts(sh.lo, w_out);
                merged_counts(sh.hi, h);
#pragma unroll
                for (int e = 0; e < kPer; ++e)
                    w_out[e] += h[e] << 32;
            }
            barrier(); // the bins may be cleared again
        };
        uint64_t cnt0[kPer], mass0[kPer], total_cnt, total_mass = 0;
        histogram(0u, ~0u, -1, cnt0, mass0);
        const uint64_t cnt_at = warps_scan<kWarps>(sum_of(cnt0), sh.warp64, &total_cnt) - sum_of(cnt0);
        const uint64_t mass_at = by_p ? warps_scan<kWarps>(sum_of(mass0), sh.warp64, &total_mass) - sum_of(mass0) : 0;

        // Index of the m-th (from 1) token with this very key, in index order: the tokens of equal
        // value are counted by index bucket, then picked out of the m-th one's bucket.
        auto nth_tie = [&](uint32_t key, uint64_t m) TOK_INLINE -> int {
            clear_bins();
            tokens([&](float x, int idx) {
                if (order_key(x) == key)
                    atomicAdd(&sh.cnt[idx >> g.bucket], 1u);
            });
            if (tid == 0)
                sh.pub[2] = 0;
            barrier();
            uint64_t c[kPer], total;
            merged_counts(sh.cnt, c);
            publish(true, m, 0.0, warps_scan<kWarps>(sum_of(c), sh.warp64, &total) - sum_of(c), 0, c, none);
            const int b = (int)sh.found_bin;
            const uint64_t before = sh.found_before;
            tokens([&](float x, int idx) {
                if (order_key(x) == key && idx >> g.bucket == b)
                    sh.cap[atomicAdd(&sh.pub[2], 1u)] = (uint32_t)~idx; // (a bucket has at most 256)
            });
            sort_cap(share_cap(), false);
            const int idx = (int)~(uint32_t)sh.sorted[m - before - 1];
            barrier();
            return idx;
        };

        // One limit: by count or by weight.  Tokens past `cut` do not count.  Returns the weight up to it.
        auto find = [&](bool count, uint64_t want, double limit) TOK_INLINE -> uint64_t {
            publish(count, want, limit, cnt_at, mass_at, cnt0, mass0);
            uint64_t before_c = sh.found_before, before_w = sh.found_mass;
            uint32_t m = sh.found_cnt, klo = 0, khi = 0;
            const int bin = (int)sh.found_bin;
            const bool narrow = m > (uint32_t)kCap;
            if (narrow) { // the bin's range of keys, then narrower ones
                float a = -INFINITY, z = INFINITY;
                tokens([&](float x, int) {
                    if (bin_of(x) == bin) {
                        a = fmaxf(a, x);
                        z = fminf(z, x);
                    }
                });
                extremes(a, z);
                khi = order_key(a);
                klo = order_key(z);
                barrier();
                while (m > (uint32_t)kCap && klo < khi) {
                    int shift = 0;
                    while (((khi - klo) >> shift) >= (uint32_t)kBins)
                        ++shift;
                    uint64_t c[kPer], w[kPer], tc, tw = 0;
                    histogram(klo, khi, shift, c, w);
                    const uint64_t ca = before_c + warps_scan<kWarps>(sum_of(c), sh.warp64, &tc) - sum_of(c);
                    const uint64_t wa = before_w + (by_p ? warps_scan<kWarps>(sum_of(w), sh.warp64, &tw) - sum_of(w) : 0);
                    publish(count, want, limit, ca, wa, c, w);
                    before_c = sh.found_before;
                    before_w = sh.found_mass;
                    m = sh.found_cnt;
                    khi -= sh.found_bin << shift;
                    klo = max(klo, khi - ((1u << shift) - 1));
                    __syncthreads(); // (found_* may be written again)
                }
            }
            if (m > (uint32_t)kCap) { // one value, more than kCap times: its first ties in index order
                const uint64_t w = by_p ? weight(value(klo)) : 0ull;
                uint64_t take = m;
                if (count)
                    take = want - before_c;
                else if (w) { // the most ties j with before + (j - 1) w < limit
                    const double room = ceil((limit - (double)before_w) / (double)w);
                    take = room < 1.0 ? 1 : room < (double)m ? (uint64_t)room : m;
                }
                cut = max(cut, place_of(klo, nth_tie(klo, take)));
                return before_w + take * w;
            }
            if (tid == 0)
                sh.pub[2] = 0;
            __syncthreads();
            tokens([&](float x, int idx) {
                const uint32_t k = order_key(x);
                if (narrow ? k >= klo && k <= khi : bin_of(x) == bin)
                    sh.cap[atomicAdd(&sh.pub[2], 1u)] = place_of(k, idx); // m <= kCap of them in all
            });
            const int total = share_cap();
            sort_cap(total, by_p);
            uint64_t all;
            const int kept = prefix(
                total, by_p,
                [&](int i, uint64_t at) {
                    return sh.sorted[i] >= cut && (count ? before_c + i < want : (double)(before_w + at) < limit);
                },
                &all);
            uint64_t mass = 0;
            if (kept > 0) {
                cut = sh.sorted[kept - 1];
                mass = before_w + sh.mass;
            }
            __syncthreads();
            return mass;
        };

        uint64_t z_mass = total_mass;
        if (by_k && total_cnt > (uint64_t)top_k)
            z_mass = find(true, (uint64_t)top_k, 0.0);
        if (by_p) {
            const double limit = (double)top_p * (double)z_mass;
            if (limit < (double)z_mass)
                find(false, 0, limit);
        }
    }

    // ---- The draw: the first token, in index order, at which the running sum of the kept weights
    // exceeds u * total.  An integer sum exceeds that exactly when it exceeds its floor. ----
    auto kept_weight = [&](float x, int idx) TOK_INLINE -> uint64_t {
        if (!(x >= xcut) || place_of(order_key(x), idx) < cut)
            return 0;
        const double w = weight_d(x);
        return w >= floor_w ? to_fixed(w) : 0ull;
    };
    const double u = fmin(fmax((double)g.u[row], 0.0), 1.0);
    auto target_of = [&](uint64_t total) TOK_INLINE { return min((uint64_t)(u * (double)total), total - 1); };
    auto emit = [&](float x, int idx, uint64_t total) TOK_INLINE {
        g.idx[row] = idx;
        if (g.logprob)
            g.logprob[row] = (float)((infinite ? 0.0 : ((double)x - xmax_d) / (double)T1) - log((double)total / kOne));
    };
    if (listed >= 0) { // sums by index bucket, then the tokens of the target's bucket in order
        __syncthreads();
        clear_bins();
        tokens([&](float x, int idx) {
            const uint64_t w = kept_weight(x, idx);
            if (w) {
                const uint32_t b = idx >> g.bucket, wl = (uint32_t)w, old = atomicAdd(&sh.lo[b], wl);
                const uint32_t wh = (uint32_t)(w >> 32) + (old + wl < old ? 1u : 0u);
                if (wh)
                    atomicAdd(&sh.hi[b], wh);
            }
        });
        if (tid == 0)
            sh.pub[2] = 0;
        __syncthreads();
        uint64_t w[kPer], total;
#pragma unroll
        for (int e = 0; e < kPer; ++e)
            w[e] = (uint64_t)sh.lo[kPer * tid + e] + ((uint64_t)sh.hi[kPer * tid + e] << 32);
        uint64_t run = warps_scan<kWarps>(sum_of(w), sh.warp64, &total) - sum_of(w);
        const uint64_t target = target_of(total);
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            if (run <= target && run + w[e] > target) {
                sh.found_bin = (uint32_t)(kPer * tid + e);
                sh.found_mass = run;
            }
            run += w[e];
        }
        __syncthreads();
        const int b = (int)sh.found_bin;
        tokens([&](float x, int idx) {
            if (idx >> g.bucket == b && kept_weight(x, idx))
                sh.cap[atomicAdd(&sh.pub[2], 1u)] = ((uint64_t)(uint32_t)~idx << 32) | order_key(x); // at most 256
        });
        __syncthreads();
        const int m = (int)sh.pub[2];
        sort_cap(m, false);
        uint64_t x = tid < m ? kept_weight(value((uint32_t)sh.sorted[tid]), (int)~(uint32_t)(sh.sorted[tid] >> 32)) : 0;
        uint64_t all;
        const uint64_t upto = sh.found_mass + warps_scan<kWarps>(x, sh.warp64, &all);
        if (upto > target && upto - x <= target)
            emit(value((uint32_t)sh.sorted[tid]), (int)~(uint32_t)(sh.sorted[tid] >> 32), total);
        return;
    }
    if (!have_mine && cut == 0 && !infinite && xmax - reach >= kLowest) {
        // No rank limit: as in the exact pass above, without a branch per token.
        uint32_t count = 0;
        auto sum = [&](float x0) TOK_INLINE {
            const double w = weight_at((double)fmaxf(x0, xcut) - xmax_d);
            // (xcut is rounded and may be xmax itself: what lies below it has no weight, whatever w is there)
            const bool in = x0 >= xcut && w >= floor_w;
            mine += in ? (uint64_t)__double_as_longlong(w + 4503599627370496.0) : 0ull;
            count += in;
        };
        mine = 0;
        vectors(
            1,
            [&](const uint4 &v, int) {
                float x[N];
                Vec<T>::split(v, x);
#pragma unroll
                for (int k = 0; k < N; ++k)
                    sum(x[k]);
            },
            [&](float x, int) { sum(x); });
        mine -= count * kBias;
    } else if (!have_mine) {
        mine = 0;
        tokens([&](float x, int idx) { mine += kept_weight(x, idx); });
    }
#pragma unroll
    for (int o = 16; o; o >>= 1)
        mine += __shfl_xor_sync(~0u, mine, o);
    if (lane == 0)
        sh.range[warp] += mine;
    __syncthreads();
    uint64_t own = 0, before = 0, total = 0;
    for (int w = 0; w < kWarps; ++w)
        own += sh.range[w];
    if (C > 1) {
        if (tid == 0)
            sh.pub64[0] = own;
        cluster_sync();
        for (int c = 0; c < C; ++c) {
            const uint64_t t = ld_cluster64(smem_addr(&sh.pub64[0]), c);
            before += c < (int)rank ? t : 0;
            total += t;
        }
    } else
        total = own;
    const uint64_t target = target_of(total);
    if (target >= before && target < before + own) { // this CTA: the warp's range, a thread's share, the token
        uint64_t run = before;
        int w = 0;
        for (; w < kWarps - 1 && run + sh.range[w] <= target; ++w)
            run += sh.range[w];
        const int lo = w == 0 ? 0 : head + min(nv, w * per_warp) * N;
        const int hi = w == kWarps - 1 ? n : head + min(nv, (w + 1) * per_warp) * N;
        const int per = (hi - lo + kThreads - 1) / kThreads;
        uint64_t s = 0, all;
        for (int i = lo + tid * per; i < min(hi, lo + (tid + 1) * per); ++i)
            s += kept_weight(Vec<T>::one(src + i), begin + i);
        run += warps_scan<kWarps>(s, sh.warp64, &all) - s;
        const uint32_t holds = __ballot_sync(~0u, run <= target && run + s > target);
        if (holds) { // one warp: the share that holds the target, 32 tokens at a time
            const int l = __ffs(holds) - 1, i0 = lo + (warp * 32 + l) * per, i1 = min(hi, i0 + per);
            run = __shfl_sync(~0u, run, l);
            for (int i = i0 + lane; i - lane < i1; i += 32) {
                const float x = i < i1 ? Vec<T>::one(src + i) : -INFINITY;
                const uint64_t wx = kept_weight(x, begin + i);
                uint64_t v = wx;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint64_t y = __shfl_up_sync(~0u, v, o);
                    if (lane >= o)
                        v += y;
                }
                if (run + v - wx <= target && run + v > target)
                    emit(x, begin + i, total);
                run += __shfl_sync(~0u, v, 31);
                if (run > target)
                    break;
            }
        }
    }
    leave();
}

template <typename T, int kThreads> tok_status launch(SampleArgs g, int64_t R, cudaStream_t stream)
{
    constexpr int N = Vec<T>::N;
    // CTAs per row: several while there are SMs without a row.
    auto slice_of = [&](int c) { return ((g.V + c - 1) / c + N - 1) / N * N; };
    int C = 1;
    while (C < kMaxCluster && R * C * 2 <= 148 && slice_of(C) > 4 * kThreads)
        C *= 2;
    g.slice = slice_of(C);
    g.bucket = 0;
    while (((g.V - 1) >> g.bucket) >= kBins)
        ++g.bucket;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(R * C));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)C;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, sample_kernel<T, kThreads>, g, C);
    if (e != cudaSuccess) {
        record_cuda_error(e);
        cudaGetLastError();
        return TOK_ERR_CUDA;
    }
    return launch_status();
}

} // namespace
} // namespace tok

extern "C" tok_status tok_sample_codes(const void *logits, tok_dtype dtype, int64_t R, int64_t V, int64_t row_stride,
                                       const float *u, const float *temperature, float temperature_all,
                                       const int32_t *top_k, int32_t top_k_all, const float *top_p, float top_p_all,
                                       const float *min_p, float min_p_all, int32_t *idx, float *logprob,
                                       cudaStream_t stream)
{
    using namespace tok;
    if (dtype != TOK_F32 && dtype != TOK_BF16)
        return TOK_ERR_DTYPE;
    const int64_t size = dtype == TOK_F32 ? 4 : 2;
    if (R < 0 || V < 1 || V > kMaxV || R > ((int64_t)1 << 27) || row_stride < 0)
        return TOK_ERR_SHAPE;
    if (R == 0)
        return TOK_OK;
    int64_t span;
    if (!mul_ok(R - 1, row_stride, &span) || span > ((int64_t)1 << 60))
        return TOK_ERR_SHAPE;
    if (!logits || !u || !idx)
        return TOK_ERR_NULL;
    if (!aligned(logits, size) || !aligned(u, 4) || !aligned(temperature, 4) || !aligned(top_k, 4) ||
        !aligned(top_p, 4) || !aligned(min_p, 4) || !aligned(idx, 4) || !aligned(logprob, 4))
        return TOK_ERR_ALIGN;
    const int64_t in_bytes = (span + V) * size, rb = 4 * R;
    const void *ins[] = {u, temperature, top_k, top_p, min_p};
    const void *outs[] = {idx, logprob};
    for (const void *o : outs) {
        if (!o)
            continue;
        if (overlaps(logits, in_bytes, o, rb))
            return TOK_ERR_ALIAS;
        for (const void *i : ins)
            if (i && overlaps(i, rb, o, rb))
                return TOK_ERR_ALIAS;
    }
    if (logprob && overlaps(idx, rb, logprob, rb))
        return TOK_ERR_ALIAS;

    SampleArgs g{};
    g.logits = logits;
    g.u = u;
    g.temperature = temperature;
    g.top_p = top_p;
    g.min_p = min_p;
    g.top_k = top_k;
    g.temperature_all = temperature_all;
    g.top_p_all = top_p_all;
    g.min_p_all = min_p_all;
    g.top_k_all = top_k_all;
    g.idx = idx;
    g.logprob = logprob;
    g.row_stride = row_stride;
    g.V = (int)V;
    // Rows in flight per SM: two of 512 threads where that holds all rows (255 rows of 64,000 under top_p:
    // 74 us against 88 with 256 threads), else four of 256 (880 rows under top_k: 62 us against 125 with 512).
    if (R <= 2 * 148)
        return dtype == TOK_F32 ? launch<float, 512>(g, R, stream) : launch<__nv_bfloat16, 512>(g, R, stream);
    return dtype == TOK_F32 ? launch<float, 256>(g, R, stream) : launch<__nv_bfloat16, 256>(g, R, stream);
}
