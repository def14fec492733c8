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
// A cluster of C CTAs holds one row in shared memory, a contiguous slice in each, and each
// thread a contiguous run of the slice: the row is read from HBM once.  The kernel is bound
// by instructions per token, so the passes over the row are few and short:
//   top_k up to kSmall: a histogram of a sample gives a value that a little more than top_k
//     tokens should reach; these are gathered in index order (the count says whether they hold the
//     top_k) and one CTA goes on with them alone.
//   top_p without top_k: a histogram of weights relative to their bin's own (32-bit integers)
//     says in which bin the limit lies; one pass then sums the exact weights above that bin
//     and in all, and picks out the bin's tokens; sorted, they give the limit's token.  The
//     exact sums say whether the bin was the right one.
//   everything else, and what these two do not settle: a histogram of counts and exact weights
//     over 1024 bins of x, then the tokens of the limit's bin, sorted; a bin with more than
//     kCap tokens is narrowed on the bits of x, to a single value if need be, whose ties
//     are counted in index order.
#include <algorithm>

#include "tma.cuh"
#include "tok_common.cuh"
#include "tok_internal.h"
#include "umma.cuh"

namespace tok {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 1024;   // two per thread
constexpr int kCap = 512;     // tokens sorted outright: one per thread
constexpr int kList = 2048;   // gathered tokens: four per thread
constexpr int kSmall = 1024;  // largest top_k that gathers
constexpr int kMaxCluster = 8;
constexpr int64_t kMaxV = 1 << 18;
constexpr double kOne = 17592186044416.0; // 2^44
constexpr float kReach = 31.25f;          // exp(-31.25) 2^44 < 1/2: no weight beyond

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
    int V, slice; // tokens per CTA
    int run;      // 16-byte vectors of a thread's run (odd: no bank conflicts between the runs)
    int vec;            // rows may be read 16 bytes at a time
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

__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t rank, uint32_t v)
{
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa_shared(addr, rank)), "r"(v) : "memory");
}

struct Shared {
    double table[64]; // 2^44 2^(j / 64)
    uint64_t warp64[kWarps], cap[kCap], sorted[kCap], cap_w[kCap];
    uint64_t pub64[2]; // this CTA's weight sums
    uint64_t found_before, found_mass;
    uint32_t cnt[kBins], lo[kBins], hi[kBins]; // histogram: tokens, weight in two words
    float list_x[kList];
    int list_idx[kList];
    uint32_t place[kCap];
    int owner[kCap];
    uint32_t warp32[2][kWarps];
    uint32_t pub[4]; // this CTA's: largest and smallest key, tokens picked, ties
    uint32_t found_bin, found_cnt;
    uint32_t res_idx;
};

// Tokens in shared memory: 16 bytes are N of them.
template <typename T> struct Vec;
template <> struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ float one(const float *p) { return *p; }
    static __device__ __forceinline__ void put(float *p, float x) { *p = x; }
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
};
template <> struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ float one(const __nv_bfloat16 *p)
    {
        return bf16_lo(*reinterpret_cast<const unsigned short *>(p));
    }
    static __device__ __forceinline__ void put(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }
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
};

// Inclusive scan over the block's threads; *total gets the sum.  All threads.
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t *warp, uint64_t *total)
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

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleArgs g, int C)
{
    constexpr int N = Vec<T>::N;
    constexpr float kLowest = -3.402823466e+38f; // tokens below it (-inf) and NaN do not count
    extern __shared__ __align__(16) unsigned char smem[];
    Shared &sh = *reinterpret_cast<Shared *>(smem);
    T *vals = reinterpret_cast<T *>(smem + (sizeof(Shared) + 15) / 16 * 16);
    const uint4 *vec = reinterpret_cast<const uint4 *>(vals);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = C > 1 ? cluster_rank() : 0;
    const int64_t row = blockIdx.x / C;
    const int begin = min(g.V, (int)rank * g.slice), n = min(g.slice, g.V - begin);
    const int vecs = (n + N - 1) / N; // vectors of the slice, the last one filled up with -inf
    const int v0 = min(vecs, tid * g.run), v1 = min(vecs, v0 + g.run); // this thread's run

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

    // The set that ranks are taken in: the row over C CTAs, or the gathered list in the first.
    int members = C, listed = -1; // listed >= 0: tokens of the list
    auto barrier = [&] {
        if (members > 1)
            cluster_sync();
        else
            __syncthreads();
    };
    auto remote = [&](const void *p, int c) -> uint32_t {
        return members > 1 ? ld_cluster(smem_addr(p), c) : *static_cast<const uint32_t *>(p);
    };
    auto remote64 = [&](const void *p, int c) -> uint64_t {
        return members > 1 ? ld_cluster64(smem_addr(p), c) : *static_cast<const uint64_t *>(p);
    };
    auto leave = [&] { // no CTA leaves while another reads its shared memory
        if (C > 1)
            cluster_sync();
    };

    // ---- The slice into shared memory; its largest value, and a low one of a sample. ----
    if (tid < 64)
        sh.table[tid] = kOne * exp2((double)tid / 64.0);
    float xmax = -INFINITY, xlow = INFINITY;
    {
        const T *src = static_cast<const T *>(g.logits) + row * g.row_stride + begin;
        if (g.vec) {
            const int whole = n / N;
#pragma unroll 4
            for (int c = tid; c < whole; c += kThreads) {
                const uint4 v = reinterpret_cast<const uint4 *>(src)[c];
                xmax = fmaxf(xmax, Vec<T>::largest(v));
                if (c < 4 * kThreads) {
                    float f[N];
                    Vec<T>::split(v, f);
                    xlow = fminf(xlow, f[0] >= kLowest ? f[0] : INFINITY);
                }
                reinterpret_cast<uint4 *>(vals)[c] = v;
            }
        }
        for (int i = (g.vec ? n / N * N : 0) + tid; i < vecs * N; i += kThreads) {
            const float x = i < n ? Vec<T>::one(src + i) : -INFINITY;
            xmax = fmaxf(xmax, x);
            xlow = fminf(xlow, x >= kLowest ? x : INFINITY);
            Vec<T>::put(vals + i, x);
        }
    }
    auto value = [](uint32_t key) { return __uint_as_float((key & 0x80000000u) ? key & 0x7FFFFFFFu : ~key); };
    {
        uint32_t kmax = __reduce_max_sync(~0u, order_key(xmax)), kmin = __reduce_min_sync(~0u, order_key(xlow));
        if (lane == 0) {
            sh.warp32[0][warp] = kmax;
            sh.warp32[1][warp] = kmin;
        }
        __syncthreads();
        kmax = __reduce_max_sync(~0u, sh.warp32[0][lane % kWarps]);
        kmin = __reduce_min_sync(~0u, sh.warp32[1][lane % kWarps]);
        if (C > 1) {
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
        xmax = value(kmax);
        xlow = fminf(value(kmin), xmax);
    }
    if (xmax == -INFINITY) { // nothing to draw from
        if (rank == 0 && tid == 0) {
            g.idx[row] = -1;
            if (g.logprob)
                g.logprob[row] = -INFINITY;
        }
        leave();
        return;
    }
    if (xmax == INFINITY) { // infinite logits: equal weights among them
        __syncthreads();
        for (int i = tid; i < vecs * N; i += kThreads)
            Vec<T>::put(vals + i, Vec<T>::one(vals + i) == INFINITY ? 0.0f : -INFINITY);
        xmax = xlow = 0.0f;
        __syncthreads();
    }

    // 2^44 exp((x - xmax) / T1) in 64 bits: with y = 64 log2(e) (x - xmax) / T1 = k + f,
    // 2^(k / 64) from a table and the exponent, 2^(f / 64) by its Taylor polynomial of
    // degree 4 (|f ln 2 / 64| <= 0.0055: what is left out is below 2^-44 relative).
    const double per_t = 64.0 / 0.6931471805599453 / (double)T1, xmax_d = (double)xmax;
    const float reach = kReach * T1, xcut = fmaxf(xmax - reach, kLowest); // no weight below
    auto weight_d = [&](float x) -> double {
        constexpr double kMagic = 6755399441055744.0; // 1.5 2^52: a sum's low bits are its integer part
        constexpr double c1 = 0.6931471805599453 / 64, c2 = c1 * c1 / 2, c3 = c2 * c1 / 3, c4 = c3 * c1 / 4;
        const double d = (double)x - xmax_d, kd = fma(d, per_t, kMagic), f = fma(d, per_t, kMagic - kd);
        const int k = __double2loint(kd);
        const double q = fma(fma(fma(c4, f, c3), f, c2), f, c1) * f, t = sh.table[k & 63];
        const double w = fma(t, q, t);
        return __hiloint2double(__double2hiint(w) + ((k >> 6) << 20), __double2loint(w));
    };
    auto to_fixed = [](double w) -> uint64_t { // nearest integer of 0 <= w < 2^51
        return (uint64_t)__double_as_longlong(w + 4503599627370496.0) & 0xFFFFFFFFFFFFFull;
    };
    auto weight = [&](float x) -> uint64_t { return x >= xcut ? to_fixed(weight_d(x)) : 0ull; };
    const double floor_w = (double)min_p * kOne;

    // Bins of equal width, the highest in bin 0, over the values that can have a weight and
    // no further than the sample's lowest.  Rounding to nearest: any monotone rule serves,
    // and this one needs no conversion.
    const float span = fminf(reach, xmax - xlow);
    const float per_bin = span > 0.0f ? fminf((float)(kBins - 1) / span, 3.4e38f) : 0.0f;
    auto bin_of = [&](float x) -> int {
        const float d = fminf((xmax - x) * per_bin, (float)(kBins - 1));
        return (int)(__float_as_uint(d + 8388608.0f) & 0x7FFFFFu);
    };
    // A token's place in the order of ranks: falling value, then rising index.
    auto place_of = [](uint32_t key, int idx) -> uint64_t { return ((uint64_t)key << 32) | (uint32_t)~idx; };
    uint64_t cut = 0; // the place of the last token kept
    const bool by_p = top_p < 1.0f && top_k != 1;
    bool by_k = top_k > 1 && top_k < g.V;

    auto each = [&](auto &&f) { // f(value, index) for the tokens of this CTA
        if (listed >= 0) {
            for (int i = tid; i < listed; i += kThreads)
                f(sh.list_x[i], sh.list_idx[i]);
        } else
            for (int c = v0; c < v1; ++c) {
                float x[N];
                Vec<T>::split(vec[c], x);
#pragma unroll
                for (int k = 0; k < N; ++k)
                    if (x[k] >= kLowest)
                        f(x[k], begin + c * N + k);
            }
    };
    auto clear_bins = [&] {
        for (int i = tid; i < kBins; i += kThreads)
            sh.cnt[i] = sh.lo[i] = sh.hi[i] = 0;
        __syncthreads();
    };

    // ---- One token: the first of the largest. ----
    if (top_k == 1) {
        if (tid == 0)
            sh.pub[2] = 0x7FFFFFFFu;
        __syncthreads();
        int first = 0x7FFFFFFF;
        for (int c = v1 - 1; c >= v0; --c) // falling, so the last hit is the first
            if (Vec<T>::largest(vec[c]) == xmax) {
                float x[N];
                Vec<T>::split(vec[c], x);
#pragma unroll
                for (int k = N - 1; k >= 0; --k)
                    first = x[k] == xmax ? begin + c * N + k : first;
            }
        first = __reduce_min_sync(~0u, first);
        if (lane == 0)
            atomicMin(&sh.pub[2], (uint32_t)first);
        barrier();
        if (rank == 0 && tid == 0) {
            uint32_t best = sh.pub[2];
            for (int c = 1; c < C; ++c)
                best = min(best, remote(&sh.pub[2], c));
            g.idx[row] = (int)best;
            if (g.logprob)
                g.logprob[row] = 0.0f;
        }
        leave();
        return;
    }

    // The bin of this thread's two (2 tid and the next; c_at, w_at lie before them) in which the limit
    // lies publishes itself: the `want`-th token, or the last before which less than `limit` lies.
    auto publish = [&](bool count, uint64_t want, double limit, uint64_t c_at, uint64_t w_at, const uint32_t (&c)[2],
                       const uint64_t (&w)[2]) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (count ? c_at < want && c_at + c[e] >= want : (double)w_at < limit && (double)(w_at + w[e]) >= limit) {
                sh.found_bin = (uint32_t)(2 * tid + e);
                sh.found_cnt = c[e];
                sh.found_before = c_at;
                sh.found_mass = w_at;
            }
            c_at += c[e];
            w_at += w[e];
        }
        __syncthreads();
    };

    // ---- Gather the tokens among which the top_k largest are. ----
    if (by_k && top_k <= kSmall) {
        // First by the runs' first vectors (where runs are long enough that this saves work), for 1.5
        // top_k + 128 tokens: four standard deviations from too few.  Then by all tokens, for top_k.
        for (int sampled = g.run >= 5 ? 1 : 0; sampled >= 0; --sampled) {
            clear_bins();
            for (int c = v0; c < (sampled ? min(v1, v0 + 1) : v1); ++c) {
                float x[N];
                Vec<T>::split(vec[c], x);
#pragma unroll
                for (int k = 0; k < N; ++k)
                    if (x[k] >= kLowest)
                        atomicAdd(&sh.cnt[bin_of(x[k])], 1u);
            }
            barrier();
            uint32_t c2[2] = {0, 0};
            for (int c = 0; c < C; ++c) {
                const uint64_t x = remote64(&sh.cnt[2 * tid], c);
                c2[0] += (uint32_t)x;
                c2[1] += (uint32_t)(x >> 32);
            }
            const uint64_t w2[2] = {0, 0};
            uint64_t total;
            const uint64_t at = block_scan((uint64_t)c2[0] + c2[1], sh.warp64, &total) - c2[0] - c2[1];
            const int want = sampled ? max(1, (3 * top_k / 2 + 128) / g.run) : top_k;
            if (tid == 0)
                sh.found_bin = kBins; // fewer tokens than that
            publish(true, (uint64_t)want, 0.0, at, 0, c2, w2);
            const int bin = (int)sh.found_bin;
            // The bin's lower edge (a little below it: what counts is the count).
            const float least = bin >= kBins - 1 || per_bin == 0.0f ? kLowest
                                                                     : fmaxf(xmax - ((float)bin + 0.51f) / per_bin, kLowest);
            uint32_t count = 0;
            for (int c = v0; c < v1; ++c)
                if (Vec<T>::largest(vec[c]) >= least) {
                    float x[N];
                    Vec<T>::split(vec[c], x);
#pragma unroll
                    for (int k = 0; k < N; ++k)
                        count += x[k] >= least;
                }
            uint64_t mine, before = 0, all = 0;
            const uint64_t upto = block_scan(count, sh.warp64, &mine);
            if (tid == 0)
                sh.pub[2] = (uint32_t)mine;
            barrier();
            for (int c = 0; c < C; ++c) {
                const uint32_t m = remote(&sh.pub[2], c);
                before += c < (int)rank ? m : 0;
                all += m;
            }
            if (all <= (uint64_t)kList && (all >= (uint64_t)top_k || least == kLowest)) {
                if (count) {
                    uint32_t to = (uint32_t)(before + upto) - count;
                    for (int c = v0; c < v1; ++c)
                        if (Vec<T>::largest(vec[c]) >= least) {
                            float x[N];
                            Vec<T>::split(vec[c], x);
#pragma unroll
                            for (int k = 0; k < N; ++k)
                                if (x[k] >= least) {
                                    const int idx = begin + c * N + k;
                                    if (C > 1) { // the first CTA has the list
                                        st_cluster(smem_addr(&sh.list_x[to]), 0, __float_as_uint(x[k]));
                                        st_cluster(smem_addr(&sh.list_idx[to]), 0, (uint32_t)idx);
                                    } else {
                                        sh.list_x[to] = x[k];
                                        sh.list_idx[to] = idx;
                                    }
                                    ++to;
                                }
                        }
                }
                listed = (int)all;
            }
            barrier();
            if (listed >= 0)
                break;
        }
        if (listed >= 0) {
            members = 1;
            by_k = listed > top_k;
            if (rank != 0) {
                leave();
                return;
            }
        }
    }

    // The `total` (at most kCap) tokens of sh.cap, sorted by place into sh.sorted, weights beside them.
    auto sort_cap = [&](int total) {
        if (tid < total)
            sh.place[tid] = 0;
        __syncthreads();
        const int groups = (total + 31) / 32, parts = groups ? kWarps / groups : 0;
        if (warp < groups * parts) {
            const int i = warp % groups * 32 + lane, part = warp / groups, per = (total + parts - 1) / parts;
            const uint64_t me = i < total ? sh.cap[i] : 0;
            uint32_t r = 0;
            const int j1 = min(total, (part + 1) * per);
#pragma unroll 4
            for (int j = part * per; j < j1; ++j)
                r += sh.cap[j] > me;
            if (i < total)
                atomicAdd(&sh.place[i], r);
        }
        __syncthreads();
        if (tid < total) {
            const uint64_t me = sh.cap[tid];
            sh.sorted[sh.place[tid]] = me;
            sh.cap_w[sh.place[tid]] = by_p ? weight(value((uint32_t)(me >> 32))) : 0ull;
        }
        __syncthreads();
    };
    // All members' sh.cap into each one's, in turn; returns their number (more than kCap: none moved).
    auto share_cap = [&]() -> int {
        barrier();
        int total = 0;
        uint64_t me = 0;
        for (int c = 0; c < members; ++c) {
            const int m = (int)remote(&sh.pub[2], c);
            if (m <= kCap && tid >= total && tid < total + m)
                me = remote64(&sh.cap[tid - total], c);
            total += m;
        }
        if (members > 1)
            barrier();
        if (total <= kCap && tid < total)
            sh.cap[tid] = me;
        return total;
    };

    // ---- Ranks. ----
    uint64_t mine = 0; // kept weight of this thread's run
    bool have_mine = false, settled = !by_k && !by_p;
    if (!settled && !by_k && listed < 0) {
        // top_p alone: the bin of the limit from relative weights, then one exact pass.
        clear_bins();
        const float h = per_bin > 0.0f ? 1.0f / (per_bin * T1) : 0.0f; // a bin's width over T1: at most 0.031
        each([&](float x, int) {
            const float d = fminf((xmax - x) * per_bin, (float)(kBins - 1)), b = (d + 8388608.0f) - 8388608.0f;
            const float e = (b - d) * h; // weight relative to the bin's middle, in 2^-14
            const float r = fmaf(e, fmaf(e, 8192.0f, 16384.0f), 16384.0f);
            if (x >= xcut)
                atomicAdd(&sh.lo[(int)(__float_as_uint(d + 8388608.0f) & 0x7FFFFFu)],
                          __float_as_uint(r + 8388608.0f) & 0x7FFFFFu);
        });
        barrier();
        uint64_t w2[2] = {0, 0};
        for (int c = 0; c < C; ++c) {
            const uint64_t x = remote64(&sh.lo[2 * tid], c);
            w2[0] += (uint32_t)x;
            w2[1] += x >> 32;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) // 2^16 more for the small ones
            w2[e] = (uint64_t)((double)w2[e] * (65536.0 * exp(-(double)(2 * tid + e) * h)));
        uint64_t total;
        const uint64_t at = block_scan(w2[0] + w2[1], sh.warp64, &total) - w2[0] - w2[1];
        const uint32_t c2[2] = {0, 0};
        publish(false, 0, fmin((double)top_p * (double)total, (double)total), 0, at, c2, w2);
        const int bin = (int)sh.found_bin;
        const float above = bin == 0 || per_bin == 0.0f ? INFINITY : xmax - ((float)bin - 0.52f) / per_bin;
        const float least = bin == kBins - 1 || per_bin == 0.0f ? kLowest : xmax - ((float)bin + 0.52f) / per_bin;
        if (tid == 0)
            sh.pub[2] = 0;
        __syncthreads();
        uint64_t sum_all = 0, sum_above = 0;
        each([&](float x, int idx) {
            if (x < xcut)
                return;
            const double wd = weight_d(x);
            const uint64_t w = to_fixed(wd);
            sum_all += w;
            if (x >= above) {
                sum_above += w;
                mine += wd >= floor_w ? w : 0ull;
            } else if (x >= least) {
                const uint32_t to = atomicAdd(&sh.pub[2], 1u);
                if (to < (uint32_t)kCap) {
                    sh.cap[to] = place_of(order_key(x), idx);
                    sh.owner[to] = tid;
                }
            }
        });
        uint64_t cta_all, cta_above, z = 0, before = 0;
        block_scan(sum_all, sh.warp64, &cta_all);
        block_scan(sum_above, sh.warp64, &cta_above);
        if (tid == 0) {
            sh.pub64[0] = cta_all;
            sh.pub64[1] = cta_above;
        }
        const int own = (int)sh.pub[2]; // (written before the scans' barriers)
        const uint64_t own_place = tid < own && own <= kCap ? sh.cap[tid] : 0;
        const int picked = share_cap();
        for (int c = 0; c < C; ++c) {
            z += remote64(&sh.pub64[0], c);
            before += remote64(&sh.pub64[1], c);
        }
        const double limit = (double)top_p * (double)z;
        if (!(limit < (double)z)) { // every token
            mine = 0;
            settled = true;
        } else if (picked <= kCap && picked > 0) {
            __syncthreads();
            sort_cap(picked);
            uint64_t tw;
            const uint64_t w = tid < picked ? sh.cap_w[tid] : 0, wi = block_scan(w, sh.warp64, &tw);
            if ((double)before < limit && (double)(before + tw) >= limit) {
                const bool keep = tid < picked && (double)(before + wi - w) < limit;
                const int kept = __syncthreads_count(keep); // a prefix
                cut = sh.sorted[kept - 1];
                // The picked tokens' kept weights to the threads whose runs hold them.
                uint64_t *extra = reinterpret_cast<uint64_t *>(sh.cnt);
                extra[tid] = 0;
                __syncthreads();
                if (own_place && own_place >= cut) {
                    const double wd = weight_d(value((uint32_t)(own_place >> 32)));
                    if (wd >= floor_w)
                        atomicAdd(reinterpret_cast<unsigned long long *>(&extra[sh.owner[tid]]),
                                  (unsigned long long)to_fixed(wd));
                }
                __syncthreads();
                mine += extra[tid];
                settled = have_mine = true;
            }
        }
        if (!have_mine)
            mine = 0;
        barrier();
    }
    if (!settled) {
        // Histogram of the tokens with klo <= key <= khi: by bin_of (shift < 0) or the key's bits.
        // Every CTA adds up all members' bins; thread j returns with bins 2j, 2j + 1.
        auto histogram = [&](uint32_t klo, uint32_t khi, int shift, uint32_t (&c_out)[2], uint64_t (&w_out)[2]) {
            clear_bins();
            each([&](float x, int) {
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
            c_out[0] = c_out[1] = 0;
            w_out[0] = w_out[1] = 0;
            for (int c = 0; c < members; ++c) {
                const uint64_t x = remote64(&sh.cnt[2 * tid], c);
                c_out[0] += (uint32_t)x;
                c_out[1] += (uint32_t)(x >> 32);
                if (by_p) {
                    const uint64_t l = remote64(&sh.lo[2 * tid], c), u = remote64(&sh.hi[2 * tid], c);
                    w_out[0] += (l & 0xFFFFFFFFull) + (u << 32);
                    w_out[1] += (l >> 32) + (u & 0xFFFFFFFF00000000ull);
                }
            }
            barrier(); // the bins may be cleared again
        };
        uint32_t cnt0[2];
        uint64_t mass0[2], total_cnt, total_mass = 0;
        histogram(0u, ~0u, -1, cnt0, mass0);
        const uint64_t cnt_at = block_scan((uint64_t)cnt0[0] + cnt0[1], sh.warp64, &total_cnt) - cnt0[0] - cnt0[1];
        const uint64_t mass_at = by_p ? block_scan(mass0[0] + mass0[1], sh.warp64, &total_mass) - mass0[0] - mass0[1] : 0;

        // Index of the m-th (from 1) token with this very key, in index order.
        auto nth_tie = [&](uint32_t key, uint32_t m) -> int {
            const int size = listed >= 0 ? listed : n, per = listed >= 0 ? kList / kThreads : g.run * N;
            const int i0 = min(size, tid * per), i1 = min(size, i0 + per);
            auto at = [&](int i) { return listed >= 0 ? sh.list_x[i] : Vec<T>::one(vals + i); };
            auto same = [&](int i) { return at(i) >= kLowest && order_key(at(i)) == key; };
            uint64_t c = 0, total;
            for (int i = i0; i < i1; ++i)
                c += same(i);
            uint64_t incl = block_scan(c, sh.warp64, &total);
            if (tid == 0) {
                sh.pub[3] = (uint32_t)total;
                sh.res_idx = 0;
            }
            barrier();
            if (members > 1)
                for (uint32_t r = 0; r < rank; ++r)
                    incl += remote(&sh.pub[3], r);
            if (c && incl >= m && incl - c < m) {
                uint64_t seen = incl - c;
                for (int i = i0; i < i1; ++i)
                    if (same(i) && ++seen == m)
                        sh.res_idx = (uint32_t)(listed >= 0 ? sh.list_idx[i] : begin + i) + 1;
            }
            barrier();
            uint32_t idx = 0; // the one member that has it wrote index + 1
            for (int c2 = 0; c2 < members; ++c2)
                idx = max(idx, remote(&sh.res_idx, c2));
            barrier();
            return (int)idx - 1;
        };

        // One limit: by count or by weight.  Tokens past `cut` do not count.  Returns the weight up to it.
        auto find = [&](bool count, uint64_t want, double limit) -> uint64_t {
            publish(count, want, limit, cnt_at, mass_at, cnt0, mass0);
            uint64_t before_c = sh.found_before, before_w = sh.found_mass;
            uint32_t m = sh.found_cnt, klo = 0, khi = 0;
            const int bin = (int)sh.found_bin;
            const bool narrow = m > (uint32_t)kCap;
            if (narrow) { // the bin's range of keys, then narrower ones
                uint32_t a = 0, z = ~0u;
                each([&](float x, int) {
                    if (bin_of(x) == bin) {
                        a = max(a, order_key(x));
                        z = min(z, order_key(x));
                    }
                });
                a = __reduce_max_sync(~0u, a);
                z = __reduce_min_sync(~0u, z);
                if (tid == 0) {
                    sh.pub[0] = 0;
                    sh.pub[1] = ~0u;
                }
                __syncthreads();
                if (lane == 0) {
                    atomicMax(&sh.pub[0], a);
                    atomicMin(&sh.pub[1], z);
                }
                barrier();
                klo = ~0u;
                for (int c = 0; c < members; ++c) {
                    khi = max(khi, remote(&sh.pub[0], c));
                    klo = min(klo, remote(&sh.pub[1], c));
                }
                barrier();
                while (m > (uint32_t)kCap && klo < khi) {
                    int shift = 0;
                    while (((khi - klo) >> shift) >= (uint32_t)kBins)
                        ++shift;
                    uint32_t c[2];
                    uint64_t w[2], tc, tw = 0;
                    histogram(klo, khi, shift, c, w);
                    const uint64_t ca = before_c + block_scan((uint64_t)c[0] + c[1], sh.warp64, &tc) - c[0] - c[1];
                    const uint64_t wa = before_w + (by_p ? block_scan(w[0] + w[1], sh.warp64, &tw) - w[0] - w[1] : 0);
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
                cut = max(cut, place_of(klo, nth_tie(klo, (uint32_t)take)));
                return before_w + take * w;
            }
            if (tid == 0)
                sh.pub[2] = 0;
            __syncthreads();
            each([&](float x, int idx) {
                const uint32_t k = order_key(x);
                if (narrow ? k >= klo && k <= khi : bin_of(x) == bin)
                    sh.cap[atomicAdd(&sh.pub[2], 1u)] = place_of(k, idx); // m <= kCap of them in all
            });
            const int total = share_cap();
            __syncthreads();
            sort_cap(total);
            uint64_t tw;
            const uint64_t w = tid < total ? sh.cap_w[tid] : 0, wi = by_p ? block_scan(w, sh.warp64, &tw) : 0;
            const bool keep = tid < total && sh.sorted[tid] >= cut &&
                              (count ? before_c + tid < want : (double)(before_w + wi - w) < limit);
            const int kept = __syncthreads_count(keep); // a prefix of the list
            if (kept > 0 && tid == kept - 1)
                sh.found_mass = before_w + wi;
            __syncthreads();
            uint64_t mass = 0;
            if (kept > 0) {
                cut = sh.sorted[kept - 1];
                mass = sh.found_mass;
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
    auto kept_weight = [&](float x, int idx) -> uint64_t {
        if (!(x >= xcut) || place_of(order_key(x), idx) < cut)
            return 0;
        const double w = weight_d(x);
        return w >= floor_w ? to_fixed(w) : 0ull;
    };
    const double u = fmin(fmax((double)g.u[row], 0.0), 1.0);
    auto target_of = [&](uint64_t total) { return min((uint64_t)(u * (double)total), total - 1); };
    auto emit = [&](float x, int idx, uint64_t total) {
        g.idx[row] = idx;
        if (g.logprob)
            g.logprob[row] = (float)(((double)x - xmax_d) / (double)T1 - log((double)total / kOne));
    };
    if (listed >= 0) {
        constexpr int kPer = kList / kThreads;
        uint64_t w[kPer], sum = 0, total;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const int i = kPer * tid + e;
            w[e] = i < listed ? kept_weight(sh.list_x[i], sh.list_idx[i]) : 0;
            sum += w[e];
        }
        uint64_t run = block_scan(sum, sh.warp64, &total) - sum;
        const uint64_t target = target_of(total);
        if (run <= target && run + sum > target) {
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
                if (run <= target && run + w[e] > target)
                    emit(sh.list_x[kPer * tid + e], sh.list_idx[kPer * tid + e], total);
                run += w[e];
            }
        }
        leave();
        return;
    }
    if (!have_mine)
        each([&](float x, int idx) { mine += kept_weight(x, idx); });
    uint64_t own, before = 0, total = 0;
    uint64_t run = block_scan(mine, sh.warp64, &own) - mine;
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
    run += before;
    const uint64_t target = target_of(total);
    const uint32_t holds = __ballot_sync(~0u, run <= target && run + mine > target);
    if (holds) { // one warp: the run that holds the target, 32 tokens at a time
        const int l = __ffs(holds) - 1, i0 = (warp * 32 + l) * g.run * N, i1 = min(n, i0 + g.run * N);
        run = __shfl_sync(~0u, run, l);
        for (int i = i0 + lane; i - lane < i1; i += 32) {
            const float x = i < i1 ? Vec<T>::one(vals + i) : -INFINITY;
            const uint64_t w = kept_weight(x, begin + i);
            uint64_t v = w;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint64_t y = __shfl_up_sync(~0u, v, o);
                if (lane >= o)
                    v += y;
            }
            if (run + v - w <= target && run + v > target)
                emit(x, begin + i, total);
            run += __shfl_sync(~0u, v, 31);
            if (run > target)
                break;
        }
    }
    leave();
}

template <typename T> tok_status launch(SampleArgs g, int64_t R, cudaStream_t stream)
{
    constexpr int N = Vec<T>::N;
    // CTAs per row: as few as let two CTAs share an SM (one loads while the other computes), more
    // (up to 8) while the GPU has room.
    auto slice_of = [&](int c) { return ((g.V + c - 1) / c + N - 1) / N * N; };
    auto bytes_of = [&](int c) { return (sizeof(Shared) + 15) / 16 * 16 + sizeof(T) * (size_t)slice_of(c); };
    int C = 1;
    while (C < kMaxCluster && (bytes_of(C) > 113 * 1024 || (R * C * 2 <= 148 && slice_of(C) > 2 * kThreads)))
        C *= 2;
    g.slice = slice_of(C);
    g.run = ((g.slice / N + kThreads - 1) / kThreads) | 1;
    const size_t smem = bytes_of(C);
    cudaError_t e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess) {
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3((unsigned)(R * C));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = stream;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)C;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, sample_kernel<T>, g, C);
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
    g.vec = aligned(logits, 16) && (R == 1 || row_stride * size % 16 == 0);
    return dtype == TOK_F32 ? launch<float>(g, R, stream) : launch<__nv_bfloat16>(g, R, stream);
}
